// mra_bias_tc.cu - the biased block-sparse attention on the 5th-generation
// tensor cores (tcgen05 MMA, tensor-memory accumulators, TMA tiles), bf16,
// head size 64: forward, and the three passes of the backward.
//
// One kernel body, four modes.  A block holds 128 rows (four adjacent block
// rows of a head: queries; in mode kCols four block columns: keys), row i of
// the tile on tensor-memory lane i, and walks the union of their lists kStack
// blocks at a time.  With rows A1 (Q or K), A2 (dO or V) and columns B1 (K or
// Q), B2 (V or dO):
//   X = A1 B1^T -> P,  dP = A2 B2^T,  dS = P (dP - delta)
//   kForward  acc1 += P B2           kDelta  delta = sum P dP
//   kRows     acc1 += dS B1, bias    kCols   acc1 += dS B1, acc2 += P B2
// X and dP are products of shared-memory tiles into tensor memory, two blocks
// (64 columns) a step.  Two softmax warps share a quarter of its lanes, a block
// row: one takes a step's first, the other its second block.  A thread reads
// its row's 32 scores and writes the weights back over them in bf16, the A
// operand of the second product.  A pair of row and block outside the lists
// costs no exponential, and the products leave out its 32 rows (by the lanes
// that they may write): with weights of 0 in their place, a NaN or an infinity
// in V, K, Q or dO would reach rows whose lists do not hold it.  So the
// accumulators are zeros at an item's start, which its last reader sees to.
// The two warps of a row share nothing in the loop: forward, each has a
// reference, a sum and an output accumulator of its own, joined at the end.
//
// Forward and delta have two buffers of scores in tensor memory: the next
// step's products run during this step's softmax.  With its accumulators kRows
// has room for two of X and one of dP (two blocks per SM, 256 columns each),
// kCols for one of each, whose weights both go over dP.  Their softmax waits
// for X and dP one by one: it starts on the next X while the products of the
// last weights and then dP run (train BigBird at 4096, B = 2, H = 12: 374 to 365
// us).  Products run in the order of their issue, so scores may be issued
// behind the products that read older weights from their columns.
//
// Blocks are persistent and take their items as they come (against items by
// block number: dense 4096 225 to 211 us, 16384 tokens 124 to 116 us).  The TMA
// warp fetches the next item's list, masks, biases and row statistics (four
// dependent loads, about 2 us) and its first tiles while this item is computed.
// The MMA warp runs its role converged and an elected lane issues (lane 0
// instead: 100 to 130 cycles to issue a product, train BigBird 370 us, not 343).
//
// What bounds it (clock stamps per role, all blocks, two blocks per SM): the
// chains of the softmax warps, four a scheduler.  A step of 64 columns takes them
// 1,500 cycles forward (N = 4096), 2,740 in kRows and 2,870 in kCols (N = 2048).
// Meanwhile the SM computes a step of each of its two blocks: 1,024 cycles of
// exponentials and 900 (forward) to 1,800 (kCols) in the tensor pipe, where a
// product with N = 64 is bound by reading its operands (50 cycles from shared
// memory, 65 with the weights in tensor memory, 32 of arithmetic).  Issue slots
// are 34 to 44 % used while blocks run; between two items the roles leave about
// 4,000 cycles (a split group's partial result: 7,000), which the SM's other
// block fills.
//
// Warps 0-7: softmax and epilogue; warp 8: items and TMA; warp 9: MMA issue.
// Every wait is bounded: on expiry MRA_DEV_TIMEOUT is raised, every role stops,
// copies and products in flight are waited for (bounded) and tensor memory is
// freed.
#include <algorithm>

#include "mra_bias_direct.cuh"
#include "mra_bias_warp.cuh"

namespace mra {
namespace bias {
namespace {

using tc::mma_commit;
using tc::mma_f16;
using tc::mma_f16_ts_rows;
using tc::sdesc;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_ld32;
using tc::tmem_st16;
using tc::tmem_st32;
using tc::tmem_wait_ld_regs;
using tc::tmem_wait_st;

enum Mode { kForward, kDelta, kRows, kCols };
constexpr int kTcRows = 4;                    // block rows per item
constexpr int kTileRows = kTcRows * kTokens;  // 128
constexpr int kSoftWarps = 8, kTmaWarp = 8, kMmaWarp = 9;
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kTcThreads = 32 * (kSoftWarps + 2);
constexpr int kD = 64;
constexpr int kTileBytes = kTokens * kD * 2;  // one block, 4 KB
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColAcc = 128;             // two accumulators of 64 columns
constexpr float kMove = 5.5f;                 // e^5.5 < 2^8

template <int kMode>
struct Shape {
    static constexpr bool two = kMode != kForward;           // A2 and dP
    static constexpr int stack = 2;                          // blocks per step
    static constexpr bool split = kMode == kRows || kMode == kCols;   // X and dP awaited one by one
    static constexpr int buffers = kMode == kCols ? 1 : 2;   // of X, and where not split of dP
    static constexpr int stages = kMode == kForward ? 4 : kMode == kRows ? 2 : 3;
    static constexpr uint32_t col_buffer = kMode == kDelta ? 128 : 64;
    // dP: kDelta in a buffer behind X, the others' only one
    static constexpr uint32_t col_dp = kMode == kRows ? 192 : 64;
};

// A work item as its roles see it; bh < 0: no more.
template <int kMode>
struct ItemInfo {
    Item it;
    BlockInfo info;
    int bucket[kMode == kRows ? kTcRows : 1][kMaxChunk];
    float stat[kMode == kRows ? 2 : 1][kMode == kDelta || kMode == kRows ? kTileRows : 1];   // minus lse, minus delta
    uint32_t rows_off[kTcRows];   // kRows, kCols: the item's rows without a gradient (padded)
};

template <int kMode>
struct TcSmem {
    using S = Shape<kMode>;
    __nv_bfloat16 a[S::two ? 2 : 1][kTileRows * kD];
    __nv_bfloat16 b[S::stages][2][S::stack * kTokens * kD];
    float stat[kMode == kCols ? S::stages : 1][S::stack][2][kTokens];   // minus lse, minus delta
    float diag[kMode == kRows ? kSoftWarps : 1][kTokens * kTokens];
    float half[2][2][2][kTileRows];   // by item parity: (max, sum) of each half of a row's blocks
    ItemInfo<kMode> item[2];
    unsigned long long item_full[2], item_empty[2], a_full, a_empty, full[S::stages], empty[S::stages],
        scores[S::buffers], scores_dp, weights[S::buffers], acc_empty, fin;
    uint32_t tmem;
    int abort, count, last, issued, issued_a;
};

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;\n" ::: "memory"); }
// barrier of the softmax threads that also ANDs a predicate
__device__ __forceinline__ bool soft_all(bool v) {
    uint32_t out;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.red.and.pred q, 1, 256, p;\n"
        " selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(out)
        : "r"((uint32_t)v)
        : "memory");
    return out != 0;
}
// true in one lane of a converged warp, the same one each time
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void store_32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// instruction descriptors (kind::f16): D fp32, A and B bf16, M = 128
__device__ __forceinline__ uint32_t idesc_scores(int blocks) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(32 * blocks) >> 3 << 17) | ((128u >> 4) << 24);
}
// acc += W tile: the tile read with its rows as K, N = 64
constexpr uint32_t kIdescAcc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((64u >> 3) << 17) | ((128u >> 4) << 24);

struct TcPtrs {
    const float *lse;           // kDelta
    __nv_bfloat16 *out, *out2;  // O; dQ; dK, dV
    float *lse_out;
};

// x (scores of this thread's row) with scale, bias and masks:
// several biases in the block (u = +inf), or tokens that take no part.
template <bool kTransposed, int kCount>
__device__ __forceinline__ void general_row(float (&x)[kCount], float scale, float u, const float *vec, int d0, bool masked,
                                            bool row_on, uint32_t cols) {
    // relative position of column j: d0 + j, or d0 - j with keys as rows
    if (u == INFINITY) {
#pragma unroll
        for (int j = 0; j < kCount; ++j) x[j] = fmaf(x[j], scale, vec[kTransposed ? d0 - j : d0 + j]);
    } else {
#pragma unroll
        for (int j = 0; j < kCount; ++j) x[j] = fmaf(x[j], scale, u);
    }
    if (masked) {
#pragma unroll
        for (int j = 0; j < kCount; ++j)
            if (!row_on || !((cols >> j) & 1u)) x[j] = -INFINITY;
    }
}

__device__ __forceinline__ void load_row(float (&x)[32], uint32_t addr) {
    uint32_t r[32];
    tmem_ld32(addr, r);
    tmem_wait_ld_regs(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void load_half(float (&x)[16], uint32_t addr) {
    uint32_t r[16];
    tmem_ld16(addr, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Bins of a block with several buckets, from a warp's 32 x 32 dS in shared
// memory: column j, row i at 32 j + 31 - i.  Diagonals run down the addresses
// 31 j + k: position k - 31 for j <= k, and position k from there on (the step
// past the end of a column lands in the diagonal 32 further up).  Constant
// offsets, and neither the writes nor the reads have bank conflicts.
__device__ __forceinline__ void bin_rows(const float *tile, float *bins, const int32_t *bucket, int buckets, int N,
                                         int d_row0, bool distinct, int lane) {
    __syncwarp();
    const int b0 = bucket_at(bucket, buckets, N, d_row0 + lane - 31, true);
    const int b1 = bucket_at(bucket, buckets, N, d_row0 + lane, lane > 0);
    float all[2] = {0.0f, 0.0f}, low[2] = {0.0f, 0.0f};
    const float *p = tile + lane;
#pragma unroll
    for (int j = 0; j < 33; ++j) {
        const float v = p[31 * j];
        if (j <= lane) low[j & 1] += v;
        else all[j & 1] += v;
    }
    bin_runs(low[0] + low[1], b0, bins, distinct, lane);
    bin_runs(all[0] + all[1], b1, bins, distinct, lane);
}

template <int kMode, bool kDirect>
__global__ void __launch_bounds__(kTcThreads, 2)
tc_kernel(const __grid_constant__ CUtensorMap ta1, const __grid_constant__ CUtensorMap ta2,
          const __grid_constant__ CUtensorMap tb1, const __grid_constant__ CUtensorMap tb2, const Call c, const TcPtrs g) {
    using S = Shape<kMode>;
    constexpr bool cols = kMode == kCols;
    constexpr int kStages = S::stages, kBuffers = S::buffers;
    extern __shared__ unsigned char raw[];
    TcSmem<kMode> &s = *reinterpret_cast<TcSmem<kMode> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Window &win = *reinterpret_cast<Window *>(&s + 1);                   // kDirect
    float *const bins = reinterpret_cast<float *>(&s + 1);               // kRows: [8][buckets]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(saddr(&s.item_full[i]), 1);
            mbar_init(saddr(&s.item_empty[i]), kSoftWarps + 1);
        }
        mbar_init(saddr(&s.a_full), 1);
        mbar_init(saddr(&s.a_empty), 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(saddr(&s.full[i]), 1);
            mbar_init(saddr(&s.empty[i]), 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(saddr(&s.scores[i]), 1);
            mbar_init(saddr(&s.weights[i]), kSoftWarps);
        }
        mbar_init(saddr(&s.scores_dp), 1);
        mbar_init(saddr(&s.acc_empty), kSoftWarps);
        mbar_init(saddr(&s.fin), 1);
        s.abort = s.issued = s.issued_a = 0;
        mbar_init_fence();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(saddr(&s.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    if (cols) columns_begin();
    else rows_begin(kMode == kRows);
    if (kDirect) {
        const int bh = (int)blockIdx.x / c.groups, group = (int)blockIdx.x % c.groups;
        make_list<kTcRows>(c, win, s.item[0].info, &s.count, bh / c.H, bh % c.H, group * kTcRows);
        if (tid == 0) s.item[0].it = Item{bh, group, 0, s.count, 1 << 16, 0};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *abort = &s.abort;
    auto wait = [&](unsigned long long *bar, uint32_t parity) { return guarded_wait(bar, parity, abort, c.status); };
    // the same answer for the whole warp, whose collective instructions follow
    auto wait_warp = [&](unsigned long long *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
    auto steps_of = [](int count) { return (count + S::stack - 1) / S::stack; };

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ items and tiles
        const Item *const items = cols ? c.col_item : c.row_item;
        int *const counters = c.counters + (cols ? kColItems : kRowItems);
        const int capacity = cols ? c.col_items : c.row_items;
        int split = 0, total = 1, t = 0, na = 0;
        bool started = false;
        if (!kDirect) {
            split = counters[1];
            total = split + counters[0];
        }
        for (int n = 0;; ++n) {
            ItemInfo<kMode> &x = s.item[n & 1];
            if (n >= 2 && !wait_warp(&s.item_empty[n & 1], ((n >> 1) - 1) & 1)) break;
            // heads with a refused list have no output
            Item it{-1, 0, 0, 0, 0, 0};
            if (kDirect) {
                if (n == 0) it = x.it;
            } else {
                // the first by the block's number, the others as they come: which
                // block has an item changes nothing in its result
                for (;; started = true) {
                    int idx = blockIdx.x;
                    if (started && lane == 0) idx = (int)gridDim.x + atomicAdd(c.counters + kTaken + kMode, 1);
                    if (started) idx = __shfl_sync(0xffffffffu, idx, 0);
                    if (idx >= total) break;
                    const Item next = items[idx < split ? idx : capacity - 1 - (idx - split)];
                    if (next.bh >= 0 && (!c.lists || !c.bad[next.bh])) {
                        it = next;
                        started = true;
                        break;
                    }
                }
            }
            if (it.bh >= 0 && !kDirect) {
                const int b = it.bh / c.H, h = it.bh - b * c.H, row0 = it.group * kTcRows;
                const int *list = (cols ? c.col_list : c.row_list) + it.start;
                for (int i = lane; i < it.count; i += 32) {
                    const int e = list[i], other = e & 0xffff;
                    x.info.entry[i] = e;
                    x.info.valid[i] = c.valid[b * c.nbr + other];
#pragma unroll
                    for (int r = 0; r < kTcRows; ++r) {
                        const bool on = row0 + r < c.nbr;
                        x.info.tile[r][i] = !on ? 0.0f : cols ? tile_bias(c, h, other, row0 + r) : tile_bias(c, h, row0 + r, other);
                        if (kMode == kRows) x.bucket[r][i] = on ? c.tile_bucket[other - row0 - r + c.nbr - 1] : -1;
                    }
                }
            }
            if ((kMode == kDelta || kMode == kRows) && it.bh >= 0) {
#pragma unroll
                for (int r = 0; r < kTcRows; ++r) {
                    const int row = it.group * kTcRows + r, pos = row * kTokens + lane, i = r * kTokens + lane;
                    if (kMode == kDelta) {
                        const float l = pos < c.N ? g.lse[(size_t)it.bh * c.N + pos] : -INFINITY;
                        x.stat[0][i] = l == -INFINITY ? -INFINITY : -l;
                    } else {
                        const float *p = c.rowstat + ((size_t)it.bh * c.nbr + row) * 2 * kTokens + lane;
                        x.stat[0][i] = row < c.nbr ? p[0] : -INFINITY;
                        x.stat[kMode == kRows ? 1 : 0][i] = row < c.nbr ? p[kTokens] : 0.0f;
                    }
                }
            }
            if ((kMode == kRows || cols) && it.bh >= 0 && lane < kTcRows) {
                const int row = it.group * kTcRows + lane;
                x.rows_off[lane] = row < c.nbr ? ~c.valid[it.bh / c.H * c.nbr + row] : 0xffffffffu;
            }
            if (lane == 0) x.it = it;
            __syncwarp();
            if (lane == 0) mbar_arrive(saddr(&s.item_full[n & 1]));
            if (it.bh < 0) break;
            const int steps = steps_of(it.count);
            if (steps == 0) continue;
            bool ok = na == 0 || wait_warp(&s.a_empty, (na - 1) & 1);
            if (ok && lane == 0) {
                const uint32_t bar = saddr(&s.a_full);
                mbar_expect_tx(bar, (S::two ? 2 : 1) * kTileRows * kD * 2);
                tma_load_3d(saddr(s.a[0]), &ta1, 0, it.group * kTileRows, it.bh, bar);
                if (S::two) tma_load_3d(saddr(s.a[S::two ? 1 : 0]), &ta2, 0, it.group * kTileRows, it.bh, bar);
                s.issued_a = na + 1;
            }
            ++na;
            for (int st = 0; ok && st < steps; ++st, ++t) {
                const int sg = t % kStages, k = min(S::stack, it.count - st * S::stack);
                if (t >= kStages && !(ok = wait_warp(&s.empty[sg], (t / kStages - 1) & 1))) break;
                if (lane == 0) {
                    const uint32_t bar = saddr(&s.full[sg]);
                    mbar_expect_tx(bar, k * (2 * kTileBytes + (cols ? 2 * kTokens * 4 : 0)));
                    for (int j = 0; j < k; ++j) {
                        const int o = x.info.entry[st * S::stack + j] & 0xffff;
                        tma_load_3d(saddr(s.b[sg][0] + j * kTokens * kD), &tb1, 0, o * kTokens, it.bh, bar);
                        tma_load_3d(saddr(s.b[sg][1] + j * kTokens * kD), &tb2, 0, o * kTokens, it.bh, bar);
                        if (cols)
                            bulk_load(saddr(s.stat[cols ? sg : 0][j]), c.rowstat + ((size_t)it.bh * c.nbr + o) * 2 * kTokens,
                                      2 * kTokens * 4, bar);
                    }
                    s.issued = t + 1;
                }
            }
            if (!ok) break;
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ products
        // The whole warp runs this role and one lane issues: descriptors and
        // counters then live in uniform registers.  (Issued from a branch of
        // one lane, a product took 90 to 180 cycles to issue, more than it
        // takes to run.)
        const uint64_t a1 = sdesc(saddr(s.a[0]), 16, 1024), a2 = sdesc(saddr(s.a[S::two ? 1 : 0]), 16, 1024);
        const uint64_t b1 = sdesc(saddr(s.b[0][0]), 16, 1024), b2 = sdesc(saddr(s.b[0][1]), 16, 1024);
        constexpr uint64_t kStage = (uint64_t)(2 * S::stack * kTileBytes) >> 4;
        // the rows that do not list each of a step's k blocks (found before the
        // step's weights are awaited)
        uint32_t off_rows[S::stack][kTcRows];
        auto rows_of = [&](const ItemInfo<kMode> &x, int st, int k) {
#pragma unroll
            for (int j = 0; j < S::stack; ++j) {
                const int e = j < k ? x.info.entry[st * S::stack + j] : 0;
#pragma unroll
                for (int r = 0; r < kTcRows; ++r)
                    off_rows[j][r] = (kMode == kForward ? 0u : x.rows_off[r]) | (((e >> (kMemberShift + r)) & 1) ? 0u : 0xffffffffu);
            }
        };
        // products of step t's weights; first: the item's first step (its
        // accumulators are zeros)
        auto accumulate = [&](int t, int k, bool first, int item) -> bool {
            const int sg = t % kStages, buf = t % kBuffers;
            if (!wait_warp(&s.weights[buf], (t / kBuffers) & 1)) return false;
            if (kMode == kDelta) {
                if (elect_one()) mbar_arrive(saddr(&s.empty[sg]));
                return true;
            }
            // the last item's accumulators have been read
            if (first && item > 0 && !wait_warp(&s.acc_empty, (item - 1) & 1)) return false;
            tc_fence_after();
            const uint64_t src1 = (kMode == kForward ? b2 : b1) + kStage * sg, src2 = b2 + kStage * sg;
            const uint32_t w = cols ? tmem + S::col_dp : tmem + buf * S::col_buffer;
            if (elect_one()) {
                // products into one accumulator wait for one another (about 100
                // cycles at these sizes): the two accumulators take turns
#pragma unroll
                for (int i = 0; i < 2 * S::stack; ++i) {
                    const int j = kMode == kForward ? i & 1 : i >> 1, kk = kMode == kForward ? i >> 1 : i & 1;
                    if (j >= k) continue;
                    const uint64_t off = (uint64_t)(j * kTileBytes + kk * 2048) >> 4;
                    // forward: each half of a row's blocks has its own accumulator
                    const uint32_t acc = kColAcc + (kMode == kForward ? 64 * j : 0);
                    const uint32_t from = w + 32 * j + (cols ? 16 : 8) * kk;     // kCols: P, then dS, 16 columns each
                    mma_f16_ts_rows(tmem + acc, from + (cols ? 8 : 0), src1 + off, kIdescAcc, off_rows[j]);
                    if (cols) mma_f16_ts_rows(tmem + kColAcc + 64, from, src2 + off, kIdescAcc, off_rows[j]);
                }
                mma_commit(saddr(&s.empty[sg]));
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        int t = 0, na = 0;
        for (int n = 0; ok; ++n) {
            if (!(ok = wait_warp(&s.item_full[n & 1], (n >> 1) & 1))) break;
            // (a reduction's result is known to be the same in every lane)
            const int count = __reduce_max_sync(0xffffffffu, s.item[n & 1].it.bh < 0 ? -1 : s.item[n & 1].it.count);
            const int steps = steps_of(max(count, 0));
            const ItemInfo<kMode> &x_item = s.item[n & 1];
            auto item_done = [&]() {
                __syncwarp();
                if (elect_one()) mbar_arrive(saddr(&s.item_empty[n & 1]));
            };
            if (count < 0) break;
            if (steps == 0) {
                item_done();
                continue;
            }
            if (!(ok = wait_warp(&s.a_full, na & 1))) break;
            // A1 (or A2) times a step's B1 (B2): 32 columns for each of its blocks
            auto product = [&](int st, int tt, uint32_t to, uint64_t a, uint64_t b) {
                const uint32_t id = idesc_scores(min(S::stack, count - st * S::stack));
                const uint64_t from = b + kStage * (tt % kStages);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_f16(to, a + 2 * ks, from + 2 * ks, id, ks > 0 ? 1u : 0u);
            };
            auto scores_x = [&](int st, int tt) {
                if (elect_one()) {
                    product(st, tt, tmem + (tt % kBuffers) * S::col_buffer, a1, b1);
                    mma_commit(saddr(&s.scores[tt % kBuffers]));
                }
                __syncwarp();
            };
            auto scores_dp = [&](int st, int tt) {
                if (elect_one()) {
                    product(st, tt, tmem + S::col_dp, a2, b2);
                    mma_commit(saddr(&s.scores_dp));
                    if (st == steps - 1) mma_commit(saddr(&s.a_empty));
                }
                __syncwarp();
            };
            if (S::split) {
                // Behind the weights of step st: kRows the next dP (its X is
                // there already), kCols, whose weights lie where dP was, the
                // next X.  The softmax starts with X, the products of st's
                // weights run meanwhile.
                if (!(ok = wait_warp(&s.full[t % kStages], (t / kStages) & 1))) break;
                tc_fence_after();
                scores_x(0, t);
                scores_dp(0, t);
                for (int st = 0; st + 1 < steps; ++st, ++t) {
                    if (!(ok = wait_warp(&s.full[(t + 1) % kStages], ((t + 1) / kStages) & 1))) break;
                    if (kMode == kRows) scores_x(st + 1, t + 1);
                    rows_of(x_item, st, S::stack);
                    if (!(ok = wait_warp(&s.weights[t % kBuffers], (t / kBuffers) & 1))) break;
                    tc_fence_after();
                    if (kMode == kRows) scores_dp(st + 1, t + 1);
                    else scores_x(st + 1, t + 1);
                    if (!(ok = accumulate(t, S::stack, st == 0, na))) break;
                    if (kMode == kCols) scores_dp(st + 1, t + 1);
                }
                ++t;
            } else {
                for (int st = 0; st < steps; ++st, ++t) {
                    const int sg = t % kStages, buf = t % kBuffers;
                    if (!(ok = wait_warp(&s.full[sg], (t / kStages) & 1))) break;
                    tc_fence_after();
                    const uint32_t x = tmem + buf * S::col_buffer;
                    if (elect_one()) {
                        const uint32_t id = idesc_scores(min(S::stack, count - st * S::stack));
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            mma_f16(x, a1 + 2 * ks, b1 + kStage * sg + 2 * ks, id, ks > 0 ? 1u : 0u);
                            if (S::two) mma_f16(x + S::col_dp, a2 + 2 * ks, b2 + kStage * sg + 2 * ks, id, ks > 0 ? 1u : 0u);
                        }
                        mma_commit(saddr(&s.scores[buf]));
                        if (st == steps - 1) mma_commit(saddr(&s.a_empty));
                    }
                    __syncwarp();
                    if (st > 0) {
                        if (kMode != kDelta) rows_of(x_item, st - 1, S::stack);
                        if (!(ok = accumulate(t - 1, S::stack, st == 1, na))) break;
                    }
                }
            }
            if (!ok) break;
            // the last step's at once: the item's end waits for it, and the
            // next item's first scores for its tiles
            const int last = count - (steps - 1) * S::stack;
            if (kMode != kDelta) rows_of(x_item, steps - 1, last);
            ok = accumulate(t - 1, last, steps == 1, na);
            item_done();
            ++na;
        }
        // every product issued here completes before tensor memory is freed
        if (elect_one()) {
            mma_commit(saddr(&s.fin));
            mbar_wait(saddr(&s.fin), 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax threads: one row each
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const int row = quarter * 32 + lane, nb = c.buckets;
        float *const my_bins = bins + (kMode == kRows ? warp * nb : 0);
        float *const my_diag = s.diag[kMode == kRows ? warp : 0];
        // this warp's part of the accumulators, zeros at every item's start
        auto clear = [&]() {
            const uint32_t zero[8] = {};
            const uint32_t own = lanes + kColAcc + (cols ? 64 : 32) * half;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                tmem_st8(own + 8 * k, zero);
                if (kMode == kForward) tmem_st8(own + 64 + 8 * k, zero);
                if (cols) tmem_st8(own + 32 + 8 * k, zero);
            }
            tmem_wait_st();
        };
        if (kMode != kDelta) clear();
        int t = 0;
        for (int n = 0;; ++n) {
            const ItemInfo<kMode> &x_item = s.item[n & 1];
            const bool got = wait(&s.item_full[n & 1], (n >> 1) & 1) && x_item.it.bh >= 0;
            if (!soft_all(got)) break;
            const Item it = x_item.it;
            const int b = it.bh / c.H, h = it.bh - b * c.H, row0 = it.group * kTcRows, steps = steps_of(it.count);
            const int r = row0 + quarter, pos = r * kTokens + lane;
            const uint32_t rows_on = r >= c.nbr ? 0u : kDirect ? win.valid[r] : c.valid[b * c.nbr + r];
            const bool row_on = (rows_on >> lane) & 1u, rows_all = rows_on == 0xffffffffu;
            const float *vec = kDirect ? win.vec + ((row0 + kTcRows) * kTokens - 1)
                                       : c.vec + ((size_t)h * 2 + 1) * c.nbr * kTokens;
            float *const stat = kMode == kDelta && r < c.nbr
                                    ? c.rowstat + ((size_t)it.bh * c.nbr + r) * 2 * kTokens + lane : nullptr;
            float m = -INFINITY, nlse = 0.0f, ndelta = 0.0f;
            float2 sum[2] = {both(0.0f), both(0.0f)};          // kForward: weights; kDelta: P dP
            float2 bin[2] = {both(0.0f), both(0.0f)};
            int bin_cur = -1;
            auto flush = [&]() {
                if (bin_cur < 0) return;
                float v = (bin[0].x + bin[0].y) + (bin[1].x + bin[1].y);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
                if (lane == 0) my_bins[bin_cur] += v;
                bin[0] = bin[1] = both(0.0f);
                __syncwarp();
            };
            if (kMode == kRows) {
                for (int i = lane; i < nb; i += 32) my_bins[i] = 0.0f;
                __syncwarp();
            }
            if (kMode == kDelta || kMode == kRows) nlse = x_item.stat[0][row];
            if (kMode == kRows) ndelta = x_item.stat[kMode == kRows ? 1 : 0][row];
            bool ok = true;
            for (int st = 0; ok && st < steps; ++st, ++t) {
                const int sg = t % kStages, buf = t % kBuffers, i = st * S::stack + half;
                if (c.expire && t == 0) {
                    *abort = 1;
                    atomicOr(c.status, kDevTimeout);
                }
                ok = !(c.expire && t == 0) && wait_warp(&s.scores[buf], (t / kBuffers) & 1);
                if (!ok) break;
                tc_fence_after();
                const int entry = i < it.count ? x_item.info.entry[i] : 0;
                const uint32_t at = lanes + buf * S::col_buffer + 32 * half,
                               at_dp = kMode == kDelta ? at + S::col_dp : lanes + S::col_dp + 32 * half;
                const uint32_t kv = i < it.count ? x_item.info.valid[i] : 0xffffffffu;
                if (!((entry >> (kMemberShift + quarter)) & 1)) {
                    if (S::split && !(ok = wait_warp(&s.scores_dp, t & 1))) break;
                    tc_fence_after();
                } else {
                    const int other = (entry & 0xffff) * kTokens;
                    const float u = x_item.info.tile[quarter][i];
                    const bool masked = kv != 0xffffffffu || (kMode != kForward && !rows_all);
                    const bool general = u == INFINITY || masked || (kMode == kForward && !(c.scale >= 0.0f));
                    const float sc = general ? 1.0f : c.scale, add = general ? 0.0f : u;
                    if (kMode == kForward) {
                        float x[32];
                        load_row(x, at);
                        if (general) general_row<false>(x, c.scale, u, vec, other - pos, masked, true, kv);
                        float y[4] = {max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[8]),
                                      max3(x[9], x[10], x[11])};
#pragma unroll
                        for (int e = 12; e < 32; e += 2) y[(e >> 1) & 3] = max3(y[(e >> 1) & 3], x[e], x[e + 1]);
                        const float top = fmaxf(max3(y[0], y[1], y[2]), y[3]), mx = fmaf(top, sc, add);
                        const bool move = mx > m + kMove || (m == -INFINITY && mx > m);
                        if (__any_sync(0xffffffffu, move)) {
                            const float f = move ? fast_exp2((m - mx) * kLog2e) : 1.0f;
                            if (move) m = mx;
                            sum[0] = mul2(sum[0], both(f));
                            sum[1] = mul2(sum[1], both(f));
                            if (move) sum[0].x += reference_rest(top, sc, add, mx);
                            if (st > 0) {
                                // the output so far, once the last step's products are in
                                wait_warp(&s.empty[(t - 1) % kStages], ((t - 1) / kStages) & 1);
                                tc_fence_after();
#pragma unroll 1
                                for (int k = 0; k < 4; ++k) {
                                    uint32_t o[16];
                                    tmem_ld16(lanes + kColAcc + 64 * half + 16 * k, o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st16(lanes + kColAcc + 64 * half + 16 * k, o);
                                }
                            }
                        }
                        const float2 ref = both((add - (m == -INFINITY ? 0.0f : m)) * kLog2e), k2 = both(sc * kLog2e);
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 p = fma2(make_float2(x[2 * e], x[2 * e + 1]), k2, ref);
                            p.x = fast_exp2(p.x);
                            p.y = fast_exp2(p.y);
                            sum[e & 1] = add2(sum[e & 1], p);
                            w[e] = pack_bf16(p.x, p.y);
                        }
                        tmem_st16(at, w);
                    } else {
                        const int tb = kMode == kRows ? x_item.bucket[kMode == kRows ? quarter : 0][i] : 0;
                        if (kMode == kRows && tb >= 0 && tb != bin_cur) {
                            flush();
                            bin_cur = tb;
                        }
                        if (kMode == kRows && tb < 0) __syncwarp();      // the tile of dS is free
                        // 16 columns at a time: the registers of two blocks per SM
                        float2 p[16];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float x[16];
                            load_half(x, at + 16 * k);
                            if (general)
                                general_row<cols>(x, c.scale, u, vec, cols ? pos - other - 16 * k : other - pos + 16 * k, masked,
                                                  row_on, kv >> (16 * k));
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float2 nl = both(nlse);
                                if (cols) nl = *reinterpret_cast<const float2 *>(&s.stat[cols ? sg : 0][half][0][16 * k + 2 * e]);
                                p[8 * k + e] = weight2(make_float2(x[2 * e], x[2 * e + 1]), sc, add, nl);
                            }
                        }
                        if (S::split && !(ok = wait_warp(&s.scores_dp, t & 1))) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float dp[16];
                            load_half(dp, at_dp + 16 * k);
                            // V or dO of a pair that does not count may hold anything
                            if (masked) {
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (!row_on || !((kv >> (16 * k + e)) & 1u)) dp[e] = 0.0f;
                            }
                            uint32_t w[8], w2[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 d = make_float2(dp[2 * e], dp[2 * e + 1]), q = p[8 * k + e];
                                if (kMode == kDelta) {
                                    sum[e & 1] = fma2(q, d, sum[e & 1]);
                                    continue;
                                }
                                float2 nd = both(ndelta);
                                if (cols) nd = *reinterpret_cast<const float2 *>(&s.stat[cols ? sg : 0][half][1][16 * k + 2 * e]);
                                const float2 ds = mul2(q, add2(d, nd));
                                if (cols) w[e] = pack_bf16(q.x, q.y);
                                w2[e] = pack_bf16(ds.x, ds.y);
                                if (kMode == kRows) {
                                    if (tb >= 0) {
                                        bin[e & 1] = add2(bin[e & 1], ds);
                                    } else {
                                        my_diag[32 * (16 * k + 2 * e) + 31 - lane] = ds.x;
                                        my_diag[32 * (16 * k + 2 * e + 1) + 31 - lane] = ds.y;
                                    }
                                }
                            }
                            // weights over scores already read: kRows over X,
                            // kCols both over dP, which leaves X free
                            if (kMode == kRows) tmem_st8(at + 8 * k, w2);
                            if (cols) {
                                tmem_st8(at_dp + 16 * k, w);
                                tmem_st8(at_dp + 16 * k + 8, w2);
                            }
                        }
                        if (kMode == kRows && tb < 0)
                            bin_rows(my_diag, my_bins, c.bucket, nb, c.N, other - r * kTokens, tb == -2, lane);
                    }
                }
                if (kMode != kDelta && kv != 0xffffffffu && quarter == 0 && !((kv >> lane) & 1u)) {
                    // a token that takes no part has weight 0; its row may hold
                    // anything, and 0 times a NaN must not be formed
                    uint4 *z1 = reinterpret_cast<uint4 *>(s.b[sg][0] + (half * kTokens + lane) * kD);
                    uint4 *z2 = reinterpret_cast<uint4 *>(s.b[sg][1] + (half * kTokens + lane) * kD);
#pragma unroll
                    for (int e = 0; e < kD / 8; ++e) {
                        if (kMode != kForward) z1[e] = make_uint4(0, 0, 0, 0);
                        if (kMode != kRows) z2[e] = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                if (kMode != kDelta) tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(saddr(&s.weights[buf]));
            }
            // ------------------------------------------------------------ epilogue: half of a row's columns each
            // (kCols: half 0 has dK, half 1 dV)
            if (ok && steps > 0 && kMode != kDelta) ok = wait_warp(&s.empty[(t - 1) % kStages], ((t - 1) / kStages) & 1);
            tc_fence_after();
            constexpr int kVals = kMode == kDelta ? 1 : cols ? 64 : 32;
            float o[kVals], total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
#pragma unroll
            for (int e = 0; e < kVals; ++e) o[e] = 0.0f;
            if (kMode == kForward || kMode == kDelta) {
                s.half[n & 1][half][0][row] = m;
                s.half[n & 1][half][1][row] = total;
                soft_sync();
            }
            if (kMode == kForward) {
                const float m0 = s.half[n & 1][0][0][row], m1 = s.half[n & 1][1][0][row];
                m = fmaxf(m0, m1);
                const float f0 = m0 == -INFINITY ? 0.0f : fast_exp2((m0 - m) * kLog2e);
                const float f1 = m1 == -INFINITY ? 0.0f : fast_exp2((m1 - m) * kLog2e);
                total = fmaf(s.half[n & 1][0][1][row], f0, s.half[n & 1][1][1][row] * f1);
                float x[32];
                if (it.count > 0) {
                    load_row(x, lanes + kColAcc + 32 * half);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e % kVals] = f0 == 0.0f ? 0.0f : x[e] * f0;
                }
                if (it.count > 1) {
                    load_row(x, lanes + kColAcc + 64 + 32 * half);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e % kVals] = f1 == 0.0f ? o[e % kVals] : fmaf(x[e], f1, o[e % kVals]);
                }
            } else if (kMode == kDelta) {
                total = s.half[n & 1][0][1][row] + s.half[n & 1][1][1][row];
            } else if (steps > 0) {
#pragma unroll
                for (int k = 0; k < kVals / 32; ++k) {
                    float x[32];
                    load_row(x, lanes + kColAcc + (cols ? 64 : 32) * half + 32 * k);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[(32 * k + e) % kVals] = x[e];
                }
            }
            if (kMode != kDelta && steps > 0) {
                // the accumulators are free for the next item
                clear();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(saddr(&s.acc_empty));
            }
            const int chunks = kDirect ? 1 : item_chunks(it);
            float *const group_bins = kMode == kRows ? c.bins + ((size_t)it.bh * c.groups + it.group) * nb : nullptr;
            auto warps_bin = [&](int i) {       // the eight warps' bins in warp order
                float v = bins[i];
#pragma unroll
                for (int w = 1; w < kSoftWarps; ++w) v += bins[w * nb + i];
                return v;
            };
            if (kMode == kRows) {
                flush();
                soft_sync();
                if (chunks == 1)
                    for (int i = tid; i < nb; i += kSoftThreads) group_bins[i] = warps_bin(i);
            }
            bool write = true;
            if (chunks > 1) {
                constexpr int kPart = kVals * kSoftThreads;      // then (max, sum) of each row
                const size_t per = kMode == kDelta ? kTileRows : kPart + (kMode == kForward ? 2 * kTileRows : kMode == kRows ? nb : 0);
                float *const base = (cols ? c.col_part : c.row_part) + (size_t)it.slot * per;
                float *const p = base + item_chunk(it) * per;
                if (kMode == kDelta) {
                    if (half == 0) p[row] = total;
                } else {
#pragma unroll
                    for (int e = 0; e < kVals; ++e) p[e * kSoftThreads + tid] = o[e];
                    if (kMode == kForward && half == 0) {
                        p[kPart + row] = m;
                        p[kPart + kTileRows + row] = total;
                    }
                    if (kMode == kRows)
                        for (int i = tid; i < nb; i += kSoftThreads) p[kPart + i] = warps_bin(i);
                }
                int *const counter = c.arrive + (size_t)((cols ? c.BH : 0) + it.bh) * c.groups + it.group;
                __threadfence();
                soft_sync();
                if (tid == 0) s.last = atomicAdd(counter, 1) == chunks - 1;
                soft_sync();
                __threadfence();
                write = s.last != 0;
                if (write) {
                    if (kMode == kDelta) {
                        total = 0.0f;
                        for (int k = 0; k < chunks; ++k) total += __ldcg(base + k * per + row);
                        if (tid == 0) *counter = 0;      // the next kernel's arrivals count from zero
                    } else {
                        float top = -INFINITY;
                        if (kMode == kForward)
                            for (int k = 0; k < chunks; ++k) top = fmaxf(top, __ldcg(base + k * per + kPart + row));
                        m = top;
                        total = 0.0f;
#pragma unroll
                        for (int e = 0; e < kVals; ++e) o[e] = 0.0f;
                        for (int k = 0; k < chunks; ++k) {
                            const float *pk = base + k * per;
                            float f = 1.0f;
                            if (kMode == kForward) {
                                const float mk = __ldcg(pk + kPart + row);
                                f = mk == -INFINITY ? 0.0f : fast_exp2((mk - top) * kLog2e);
                                total = fmaf(__ldcg(pk + kPart + kTileRows + row), f, total);
                            }
#pragma unroll
                            for (int e = 0; e < kVals; ++e) o[e] = fmaf(__ldcg(pk + e * kSoftThreads + tid), f, o[e]);
                        }
                        if (kMode == kRows)
                            for (int i = tid; i < nb; i += kSoftThreads) {
                                float v = 0.0f;
                                for (int k = 0; k < chunks; ++k) v += __ldcg(base + k * per + kPart + i);
                                group_bins[i] = v;
                            }
                    }
                }
            }
            if (ok && write && r < c.nbr) {
                if (kMode == kDelta) {
                    if (half == 0) {
                        stat[0] = nlse;
                        stat[kTokens] = -total;
                    }
                } else if (pos < c.N) {
                    float f = cols && half == 1 ? 1.0f : c.scale;
                    if (kMode == kForward) {
                        const bool live = row_on && total != 0.0f;      // (NaN: live)
                        f = 1.0f / total;
                        if (!live) {
                            f = 0.0f;
#pragma unroll
                            for (int e = 0; e < kVals; ++e) o[e] = 0.0f;
                        }
                        if (g.lse_out && half == 0)
                            g.lse_out[(size_t)it.bh * c.N + pos] = live ? m + logf(total) : -INFINITY;
                    }
                    const bool wide = ((uintptr_t)(cols && half == 1 ? g.out2 : g.out) & 31) == 0;
                    __nv_bfloat16 *dst = (cols && half == 1 ? g.out2 : g.out) + ((size_t)it.bh * c.N + pos) * kD +
                                         (cols ? 0 : 32 * half);
                    // 32 bytes a store: a row is a line of its own, and what a
                    // store costs is its 32 lines
#pragma unroll
                    for (int e = 0; e < kVals / 16; ++e) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = pack_bf16(o[16 * e + 2 * k] * f, o[16 * e + 2 * k + 1] * f);
                        if (wide) {
                            store_32(dst + 16 * e, w);
                        } else {
                            *reinterpret_cast<uint4 *>(dst + 16 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                            *reinterpret_cast<uint4 *>(dst + 16 * e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
            // the item's list and, with the barrier at the next item's start, the
            // bins are free
            __syncwarp();
            if (lane == 0) mbar_arrive(saddr(&s.item_empty[n & 1]));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort && tid == 0) {
        // copies in flight land before the shared memory is given up
        if (s.issued_a > 0) mbar_wait(saddr(&s.a_full), (s.issued_a - 1) & 1);
        for (int t = max(0, s.issued - kStages); t < s.issued; ++t)
            mbar_wait(saddr(&s.full[t % kStages]), (t / kStages) & 1);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols) : "memory");
    if (cols) table_gradient(c, kTcThreads / 32);
}

// The maps of an item's own rows and of the blocks that it walks.
struct Maps {
    CUtensorMap a1, a2, b1, b2;
};

template <int kMode, bool kDirect>
cudaError_t launch(const Call &c, const Maps &m, const TcPtrs &g, cudaStream_t s) {
    const size_t bin = kMode == kRows ? kSoftWarps * sizeof(float) : 0;
    const size_t fixed = sizeof(TcSmem<kMode>) + 1024 + (kDirect ? sizeof(Window) : 0), smem = fixed + bin * c.buckets;
    auto *kern = tc_kernel<kMode, kDirect>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_shared(kern, fixed + bin * kMaxBuckets, done);
    if (e != cudaSuccess) return e;
    const int grid = kDirect ? c.BH * c.groups : std::min(kMode == kCols ? c.col_items : c.row_items, 2 * device_sm_count());
    return launch_dependent(kern, dim3(grid), dim3(kTcThreads), smem, s, m.a1, m.a2, m.b1, m.b2, c, g);
}

}  // namespace

cudaError_t launch_forward_tc(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                              cudaStream_t s) {
    const TcPtrs g{nullptr, static_cast<__nv_bfloat16 *>(out), nullptr, lse};
    Maps m;
    if (!make_head_map(&m.a1, q, c.BH, c.N, kD, kTileRows) || !make_head_map(&m.b1, k, c.BH, c.N, kD, kTokens) ||
        !make_head_map(&m.b2, v, c.BH, c.N, kD, kTokens))
        return cudaErrorInvalidValue;
    m.a2 = m.a1;
    return c.direct ? launch<kForward, true>(c, m, g, s) : launch<kForward, false>(c, m, g, s);
}

cudaError_t launch_backward_tc(const Call &c, const void *q, const void *k, const void *v, const float *lse,
                               const void *dout, void *dq, void *dk, void *dv, cudaStream_t s, int *launches) {
    __nv_bfloat16 *oq = static_cast<__nv_bfloat16 *>(dq), *ok = static_cast<__nv_bfloat16 *>(dk),
                  *ov = static_cast<__nv_bfloat16 *>(dv);
    Maps rows, cols;
    const void *const by_rows[] = {q, dout, k, v};
    CUtensorMap *const tile[] = {&rows.a1, &rows.a2, &cols.a1, &cols.a2}, *const block[] = {&cols.b1, &cols.b2, &rows.b1, &rows.b2};
    for (int i = 0; i < 4; ++i)
        if (!make_head_map(tile[i], by_rows[i], c.BH, c.N, kD, kTileRows) ||
            !make_head_map(block[i], by_rows[i], c.BH, c.N, kD, kTokens))
            return cudaErrorInvalidValue;
    *launches += 3;
    cudaError_t e = launch<kDelta, false>(c, rows, TcPtrs{lse, nullptr, nullptr, nullptr}, s);
    if (e == cudaSuccess) e = launch<kRows, false>(c, rows, TcPtrs{nullptr, oq, nullptr, nullptr}, s);
    if (e == cudaSuccess) e = launch<kCols, false>(c, cols, TcPtrs{nullptr, ok, ov, nullptr}, s);
    return e;
}

}  // namespace bias
}  // namespace mra
