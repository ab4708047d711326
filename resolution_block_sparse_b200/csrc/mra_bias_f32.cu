// mra_bias_f32.cu - the biased block-sparse attention in fp32, forward and
// backward, on the FMA pipes (no TF32: fp32 products and sums throughout).
//
// One kernel body, four modes.  A block of 128 threads holds 64 rows (two
// block rows: queries; in mode kCols two block columns: keys) and walks the
// item's list 32 columns at a time; a thread owns rows ty, ty + 16, ty + 32,
// ty + 48 and every eighth column.  With rows A1 (Q or K), A2 (dO or V) and
// columns B1 (K or Q), B2 (V or dO):
//   x = A1 B1^T -> P,  dp = A2 B2^T,  dS = P (dp - delta)
//   kFwd    acc += P B2            kDelta  delta = sum P dp
//   kRows   acc += dS B1, bias     kCols   acc += dS B1, acc2 += P B2
// A row's 8 threads are in one warp, so its weights pass through shared memory
// with warp barriers only.  Columns come by asynchronous copies, one block ahead.
// Bound by the FMA pipes: 4 x 4 products from eight 16-byte shared loads.
#include "mra_bias.cuh"
#include "mra_f32x2.cuh"
#include "mra_internal.cuh"
#include "mra_mma.cuh"

namespace mra {
namespace bias {
namespace {

using mma::fast_exp2;

constexpr int kThreads = 128;
constexpr int kRowsTile = kGroup * kTokens;
constexpr int kPitchS = 36;
constexpr float kMove = 5.5f;
enum Mode { kFwd, kDelta, kRows, kCols };

template <int D, int kMode>
struct Smem {
    static constexpr int kPitch = D + 4;
    float a1[kRowsTile * kPitch];
    float a2[kMode == kFwd ? 4 : kRowsTile * kPitch];
    float b1[2][kTokens * kPitch], b2[2][kTokens * kPitch];
    float x[kRowsTile * kPitchS];
    float stat[2][2][kTokens];
    int last;
};

// rows of a [.][D] tensor into shared memory; rows that take no part are zeros
template <int D>
__device__ __forceinline__ void load_rows(float *dst, const float *src, int rows, const uint32_t *on, int tid) {
    constexpr int kPitch = D + 4, kPer = D / 4;
    for (int i = tid; i < rows * kPer; i += kThreads) {
        const int r = i / kPer, j = i % kPer;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if ((on[r >> 5] >> (r & 31)) & 1u) v = *reinterpret_cast<const float4 *>(src + (size_t)r * D + j * 4);
        *reinterpret_cast<float4 *>(dst + r * kPitch + j * 4) = v;
    }
}

// The same asynchronously, 16 bytes at a time (a size of 0 writes zeros).
template <int D>
__device__ __forceinline__ void load_rows_async(float *dst, const float *src, uint32_t on, int tid) {
    constexpr int kPitch = D + 4, kPer = D / 4;
    for (int i = tid; i < kTokens * kPer; i += kThreads) {
        const int r = i / kPer, j = i % kPer;
        const bool live = (on >> r) & 1u;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(mma::smem_u32(dst + r * kPitch + j * 4)),
                     "l"(src + (live ? (size_t)r * D + j * 4 : 0)), "r"(live ? 16 : 0)
                     : "memory");
    }
}

// x[i][j] = row ty + 16 i of a . row tx + 8 j of b, even and odd d apart (one
// instruction for two products)
template <int D>
__device__ __forceinline__ void mul_abt(float (&x)[4][4], const float *a, const float *b, int ty, int tx) {
    constexpr int kPitch = D + 4;
    float2 y[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i][j] = both(0.0f);
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 u[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = *reinterpret_cast<const float4 *>(a + (ty + 16 * i) * kPitch + d);
            v[i] = *reinterpret_cast<const float4 *>(b + (tx + 8 * i) * kPitch + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[i][j] = fma2(make_float2(u[i].x, u[i].y), make_float2(v[j].x, v[j].y), y[i][j]);
                y[i][j] = fma2(make_float2(u[i].z, u[i].w), make_float2(v[j].z, v[j].w), y[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = y[i][j].x + y[i][j].y;
}

// acc[i][.] += weights of row ty + 16 i (shared, 32 of them) times the rows of
// b, for kRows rows i from kFirst on; a thread's columns are 4 tx + 32 k .. + 3
template <int D, int kFirst, int kRows>
__device__ __forceinline__ void mul_ab_of(float (&acc)[4][D / 8], const float *w, const float *b, int ty, int tx) {
    constexpr int kPitch = D + 4;
#pragma unroll 2
    for (int n = 0; n < kTokens; n += 4) {
        float4 p[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) p[i] = *reinterpret_cast<const float4 *>(w + (ty + 16 * (kFirst + i)) * kPitchS + n);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const float4 v = *reinterpret_cast<const float4 *>(b + (n + m) * kPitch + 32 * k + 4 * tx);
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    float *const a = acc[kFirst + i] + 4 * k;
                    const float f = m == 0 ? p[i].x : m == 1 ? p[i].y : m == 2 ? p[i].z : p[i].w;
                    const float2 lo = fma2(both(f), make_float2(v.x, v.y), make_float2(a[0], a[1]));
                    const float2 hi = fma2(both(f), make_float2(v.z, v.w), make_float2(a[2], a[3]));
                    a[0] = lo.x;
                    a[1] = lo.y;
                    a[2] = hi.x;
                    a[3] = hi.y;
                }
            }
        }
    }
}

// The same for the block rows (members) that list the block, rows i = 0, 1 and
// 2, 3: another row's weights are 0, and 0 times a NaN of a block that it does
// not list must not be formed.
template <int D>
__device__ __forceinline__ void mul_ab(float (&acc)[4][D / 8], const float *w, const float *b, int ty, int tx, int members) {
    if (members == 3) mul_ab_of<D, 0, 4>(acc, w, b, ty, tx);
    else if (members == 1) mul_ab_of<D, 0, 2>(acc, w, b, ty, tx);
    else mul_ab_of<D, 2, 2>(acc, w, b, ty, tx);
}

__device__ __forceinline__ void put_weights(float *w, const float (&x)[4][4], int ty, int tx) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[(ty + 16 * i) * kPitchS + tx + 8 * j] = x[i][j];
    __syncwarp();
}

__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

template <int D>
__device__ __forceinline__ void write_rows(float *dst, const float (&acc)[4][D / 8], const float (&f)[4], int rows,
                                           int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ty + 16 * i >= rows) continue;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            *reinterpret_cast<float4 *>(dst + (size_t)(ty + 16 * i) * D + 32 * k + 4 * tx) =
                make_float4(acc[i][4 * k] * f[i], acc[i][4 * k + 1] * f[i], acc[i][4 * k + 2] * f[i],
                            acc[i][4 * k + 3] * f[i]);
    }
}

__device__ __forceinline__ bool last_to_arrive(int *counter, int chunks, int *s_last) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) *s_last = atomicAdd(counter, 1) == chunks - 1;
    __syncthreads();
    __threadfence();
    return *s_last != 0;
}

struct Ptrs {
    const float *a1, *a2, *b1, *b2;
    const float *lse;      // kDelta, kRows
    float *out, *out2;     // O; dQ; dK, dV
    float *lse_out;
};

template <int D, int kMode>
__device__ __forceinline__ void f32_item(const Call &c, const Ptrs &g, unsigned char *raw) {
    Smem<D, kMode> &s = *reinterpret_cast<Smem<D, kMode> *>(raw);
    float *const bins = reinterpret_cast<float *>(&s + 1);        // kRows: [4][buckets]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ty = tid >> 3, tx = tid & 7;
    constexpr bool cols = kMode == kCols;
    Item it;
    if (!take_item(cols ? c.col_item : c.row_item, c.counters + (cols ? kColItems : kRowItems),
                   cols ? c.col_items : c.row_items, &it))
        return;
    if (c.lists && c.bad[it.bh]) return;
    const int *list = cols ? c.col_list : c.row_list;
    const int b = it.bh / c.H, h = it.bh - b * c.H, row0 = it.group * kGroup, pos = row0 * kTokens;
    const size_t head = (size_t)it.bh * c.N * D;
    const float *vec = c.vec + (size_t)h * 2 * c.nbr * kTokens + c.nbr * kTokens;
    uint32_t on[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) on[k] = row0 + k < c.nbr ? c.valid[b * c.nbr + row0 + k] : 0u;
    load_rows<D>(s.a1, g.a1 + head + (size_t)pos * D, kRowsTile, on, tid);
    if (kMode != kFwd) load_rows<D>(s.a2, g.a2 + head + (size_t)pos * D, kRowsTile, on, tid);
    if (kMode == kRows)
        for (int i = tid; i < 4 * c.buckets; i += kThreads) bins[i] = 0.0f;

    float acc[4][D / 8], acc2[kMode == kCols ? 4 : 1][D / 8];
    float m[4], l[4], nlse[4], ndelta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < D / 8; ++k) acc[i][k] = acc2[kMode == kCols ? i : 0][k] = 0.0f;
        m[i] = -INFINITY;
        l[i] = 0.0f;
        const int r = ty + 16 * i, n = pos + r;
        if (kMode == kDelta || kMode == kRows) {
            const float x = n < c.N ? g.lse[(size_t)it.bh * c.N + n] : -INFINITY;
            nlse[i] = x == -INFINITY ? -INFINITY : -x;
            ndelta[i] = kMode == kRows && row0 + (r >> 5) < c.nbr
                           ? c.rowstat[(((size_t)it.bh * c.nbr + row0 + (r >> 5)) * 2 + 1) * kTokens + (r & 31)]
                           : 0.0f;
        }
    }

    // the next block is on its way while this one is computed
    int entry = 0, next_entry = it.count > 0 ? list[it.start] : 0;
    uint32_t cv = 0u, next_cv = 0u;
    // one bias (+inf: several) and bucket (negative: several) for each of the
    // group's blocks against the column block
    float u[kGroup], next_u[kGroup];
    int tb[kGroup], next_tb[kGroup];
    const float *tile = c.tile + (size_t)h * 2 * c.nbr + c.nbr - 1;
    auto fetch = [&](int buf) {
        const int col = next_entry & 0xffff;
        next_cv = c.valid[b * c.nbr + col];
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            const bool row = row0 + k < c.nbr;
            const int o = col - row0 - k;
            next_u[k] = row ? tile[cols ? -o : o] : 0.0f;
            next_tb[k] = kMode == kRows && row ? c.tile_bucket[o + c.nbr - 1] : -1;
        }
        load_rows_async<D>(s.b1[buf], g.b1 + head + (size_t)col * kTokens * D, next_cv, tid);
        load_rows_async<D>(s.b2[buf], g.b2 + head + (size_t)col * kTokens * D, next_cv, tid);
        if (cols && tid < 2 * kTokens / 4)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(mma::smem_u32(&s.stat[buf][0][0] + 4 * tid)),
                         "l"(c.rowstat + ((size_t)it.bh * c.nbr + col) * 2 * kTokens + 4 * tid)
                         : "memory");
        mma::cp_async_commit();
    };
    // bias gradient of blocks with one bucket: this thread's sum for each row of
    // blocks, added to the warp's bins when the bucket changes
    float bin[kGroup] = {0.0f, 0.0f};
    int bin_cur[kGroup] = {-1, -1};
    auto flush = [&](int k) {
        if (bin_cur[k] < 0) return;
        float v = bin[k];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) bins[warp * c.buckets + bin_cur[k]] += v;
        bin[k] = 0.0f;
        __syncwarp();
    };
    if (it.count > 0) fetch(0);
    for (int n = 0; n < it.count; ++n) {
        const int buf = n & 1;
        entry = next_entry;
        cv = next_cv;
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            u[k] = next_u[k];
            tb[k] = next_tb[k];
        }
        const int cpos = (entry & 0xffff) * kTokens, members = entry >> kMemberShift;
        bool row_on[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) row_on[i] = ((members >> (i >> 1)) & 1) && ((on[i >> 1] >> ((ty + 16 * i) & 31)) & 1u);
        if (n + 1 < it.count) {
            next_entry = list[it.start + n + 1];
            fetch(buf ^ 1);
            mma::cp_async_wait<1>();
        } else {
            mma::cp_async_wait<0>();
        }
        __syncthreads();
        float x[4][4];
        mul_abt<D>(x, s.a1, s.b1[buf], ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = cpos + tx + 8 * j - pos - r;
                const bool ok = row_on[i] && ((cv >> (tx + 8 * j)) & 1u);
                const float bias = u[i >> 1] == INFINITY ? __ldg(vec + (cols ? -d : d)) : u[i >> 1];
                x[i][j] = ok ? fmaf(x[i][j], c.scale, bias) : -INFINITY;
            }
        }
        if (kMode == kFwd) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mx = row_max(fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])));
                if (mx > m[i] + kMove || (m[i] == -INFINITY && mx > m[i])) {
                    const float f = fast_exp2((m[i] - mx) * kLog2e);
                    m[i] = mx;
                    l[i] *= f;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k) acc[i][k] *= f;
                }
                const float ref = m[i] == -INFINITY ? 0.0f : m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = fast_exp2((x[i][j] - ref) * kLog2e);
                    l[i] += x[i][j];
                }
            }
            put_weights(s.x, x, ty, tx);
            mul_ab<D>(acc, s.x, s.b2[buf], ty, tx, members);
            __syncthreads();
            continue;
        }
        float dp[4][4];
        mul_abt<D>(dp, s.a2, s.b2[buf], ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (a row that takes no part has weight 0, and its dP may be a NaN)
                const float p = row_on[i] ? fast_exp2((x[i][j] + (cols ? s.stat[buf][0][tx + 8 * j] : nlse[i])) * kLog2e) : 0.0f;
                if (kMode == kDelta && row_on[i]) l[i] = fmaf(p, dp[i][j], l[i]);
                x[i][j] = p;
                dp[i][j] = row_on[i] ? p * (dp[i][j] + (cols ? s.stat[buf][1][tx + 8 * j] : ndelta[i])) : 0.0f;
            }
        if (kMode == kDelta) {
            __syncthreads();
            continue;
        }
        if constexpr (kMode == kCols) {
            put_weights(s.x, x, ty, tx);
            mul_ab<D>(acc2, s.x, s.b2[buf], ty, tx, members);
        }
        put_weights(s.x, dp, ty, tx);
        mul_ab<D>(acc, s.x, s.b1[buf], ty, tx, members);
        if (kMode == kRows) {
            bool several = false;
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                if (!((entry >> (kMemberShift + k)) & 1)) continue;
                if (tb[k] < 0) {
                    several = true;
                    continue;
                }
                if (tb[k] != bin_cur[k]) {
                    flush(k);
                    bin_cur[k] = tb[k];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) bin[k] += dp[2 * k][j] + dp[2 * k + 1][j];
            }
            if (several) {
                // thread 64 * member + k: diagonal k - 31 of that block row's tile
                __syncthreads();
                const int member = tid >> 6, k = tid & 63;
                const bool live = k < 63 && ((entry >> (kMemberShift + member)) & 1) && (member ? tb[1] : tb[0]) < 0;
                float sum = 0.0f;
                if (live) {
#pragma unroll 8
                    for (int r = 0; r < kTokens; ++r) {      // neighbouring threads read neighbouring words
                        const int at = r + k - 31;
                        if (at >= 0 && at < kTokens) sum += s.x[(32 * member + r) * kPitchS + at];
                    }
                }
                bin_runs(sum, bucket_at(c.bucket, c.buckets, c.N, cpos - pos - 32 * member + k - 31, live),
                         bins + warp * c.buckets, false, lane);
            }
        }
        __syncthreads();      // this buffer is free for the block after the next
    }

    if (kMode == kRows) {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) flush(k);
        __syncthreads();
    }
    const int chunks = item_chunks(it);
    int *const counter = c.arrive + (size_t)((cols ? c.BH : 0) + it.bh) * c.groups + it.group;
    if (kMode == kFwd || kMode == kDelta) {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] = row_sum(l[i]);
    }
    if (kMode == kDelta) {
        if (chunks > 1) {
            float *p = c.row_part + (size_t)(it.slot + item_chunk(it)) * kRowsTile;
            if (tx == 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) p[ty + 16 * i] = l[i];
            if (!last_to_arrive(counter, chunks, &s.last)) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                l[i] = 0.0f;
                for (int k = 0; k < chunks; ++k) l[i] += __ldcg(c.row_part + (size_t)(it.slot + k) * kRowsTile + ty + 16 * i);
            }
            if (tid == 0) *counter = 0;      // the next kernel's arrivals count from zero
        }
        if (tx == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty + 16 * i;
                if (row0 + (r >> 5) >= c.nbr) continue;
                float *st = c.rowstat + ((size_t)it.bh * c.nbr + row0 + (r >> 5)) * 2 * kTokens + (r & 31);
                st[0] = nlse[i];
                st[kTokens] = -l[i];
            }
        return;
    }
    const int nb = c.buckets;
    float *const group_bins = kMode == kRows ? c.bins + ((size_t)it.bh * c.groups + it.group) * nb : nullptr;
    if (kMode == kRows) __syncthreads();
    if (chunks > 1) {
        constexpr int kAcc = D / 2;
        const size_t per = kMode == kFwd    ? (size_t)kThreads * (kAcc + 8)
                           : kMode == kRows ? (size_t)kThreads * kAcc + nb
                                            : (size_t)kThreads * 2 * kAcc;
        float *const base = (cols ? c.col_part : c.row_part) + (size_t)it.slot * per;
        float *const p = base + item_chunk(it) * per;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                p[(i * (D / 8) + k) * kThreads + tid] = acc[i][k];
                if (kMode == kCols) p[(kAcc + i * (D / 8) + k) * kThreads + tid] = acc2[kMode == kCols ? i : 0][k];
            }
            if (kMode == kFwd) {
                p[(kAcc + i) * kThreads + tid] = m[i];
                p[(kAcc + 4 + i) * kThreads + tid] = l[i];
            }
        }
        if (kMode == kRows)
            for (int i = tid; i < nb; i += kThreads)
                p[kThreads * kAcc + i] = ((bins[i] + bins[nb + i]) + bins[2 * nb + i]) + bins[3 * nb + i];
        if (!last_to_arrive(counter, chunks, &s.last)) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
            if (kMode == kFwd)
                for (int k = 0; k < chunks; ++k) top = fmaxf(top, __ldcg(base + k * per + (kAcc + i) * kThreads + tid));
            m[i] = top;
            l[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < D / 8; ++e) acc[i][e] = acc2[kMode == kCols ? i : 0][e] = 0.0f;
            for (int k = 0; k < chunks; ++k) {
                const float *pk = base + k * per + tid;
                float f = 1.0f;
                if (kMode == kFwd) {
                    const float mk = __ldcg(pk + (kAcc + i) * kThreads);
                    f = mk == -INFINITY ? 0.0f : fast_exp2((mk - top) * kLog2e);
                    l[i] = fmaf(__ldcg(pk + (kAcc + 4 + i) * kThreads), f, l[i]);
                }
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    acc[i][e] = fmaf(__ldcg(pk + (i * (D / 8) + e) * kThreads), f, acc[i][e]);
                    if (kMode == kCols)
                        acc2[kMode == kCols ? i : 0][e] += __ldcg(pk + (kAcc + i * (D / 8) + e) * kThreads);
                }
            }
        }
        if (kMode == kRows)
            for (int i = tid; i < nb; i += kThreads) {
                float v = 0.0f;
                for (int k = 0; k < chunks; ++k) v += __ldcg(base + k * per + kThreads * kAcc + i);
                group_bins[i] = v;
            }
    } else if (kMode == kRows) {
        for (int i = tid; i < nb; i += kThreads)
            group_bins[i] = ((bins[i] + bins[nb + i]) + bins[2 * nb + i]) + bins[3 * nb + i];
    }
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = c.scale;
        const int r = ty + 16 * i, n = pos + r;
        if (kMode != kFwd && !((on[i >> 1] >> (r & 31)) & 1u)) {
            // a padded row has no gradient, whatever its blocks hold
#pragma unroll
            for (int k = 0; k < D / 8; ++k) acc[i][k] = acc2[kMode == kCols ? i : 0][k] = 0.0f;
        }
        if (kMode == kFwd) {
            const bool live = ((on[i >> 1] >> (r & 31)) & 1u) && l[i] != 0.0f;      // (NaN: live)
            f[i] = live ? 1.0f / l[i] : 0.0f;
            if (!live)
#pragma unroll
                for (int k = 0; k < D / 8; ++k) acc[i][k] = 0.0f;
            if (g.lse_out && tx == 0 && n < c.N)
                g.lse_out[(size_t)it.bh * c.N + n] = live ? m[i] + logf(l[i]) : -INFINITY;
        }
    }
    write_rows<D>(g.out + head + (size_t)pos * D, acc, f, c.N - pos, ty, tx);
    if constexpr (kMode == kCols) {
        const float one[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        write_rows<D>(g.out2 + head + (size_t)pos * D, acc2, one, c.N - pos, ty, tx);
    }
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, D == 32 ? 4 : 2) f32_kernel(const Call c, const Ptrs g) {
    extern __shared__ __align__(16) unsigned char raw[];
    if (kMode == kCols) columns_begin();
    else rows_begin(kMode == kRows);
    f32_item<D, kMode>(c, g, raw);
    if (kMode == kCols) table_gradient(c, kThreads / 32);
}

template <int D, int kMode>
cudaError_t launch(const Call &c, const Ptrs &g, cudaStream_t s) {
    const size_t bin = kMode == kRows ? 4 * sizeof(float) : 0, smem = sizeof(Smem<D, kMode>) + bin * c.buckets;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_shared(f32_kernel<D, kMode>, sizeof(Smem<D, kMode>) + bin * kMaxBuckets, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(f32_kernel<D, kMode>, dim3(kMode == kCols ? c.col_items : c.row_items), dim3(kThreads), smem,
                            s, c, g);
}

template <int D>
cudaError_t backward(const Call &c, const float *q, const float *k, const float *v, const float *lse, const float *dout,
                     float *dq, float *dk, float *dv, cudaStream_t s) {
    cudaError_t e = launch<D, kDelta>(c, Ptrs{q, dout, k, v, lse, nullptr, nullptr, nullptr}, s);
    if (e == cudaSuccess) e = launch<D, kRows>(c, Ptrs{q, dout, k, v, lse, dq, nullptr, nullptr}, s);
    if (e == cudaSuccess) e = launch<D, kCols>(c, Ptrs{k, v, q, dout, nullptr, dk, dv, nullptr}, s);
    return e;
}

}  // namespace

cudaError_t launch_forward_f32(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                               cudaStream_t s) {
    const Ptrs g{static_cast<const float *>(q), nullptr, static_cast<const float *>(k), static_cast<const float *>(v),
                 nullptr, static_cast<float *>(out), nullptr, lse};
    return c.D == 64 ? launch<64, kFwd>(c, g, s) : launch<32, kFwd>(c, g, s);
}

cudaError_t launch_backward_f32(const Call &c, const void *q, const void *k, const void *v, const float *lse,
                                const void *dout, void *dq, void *dk, void *dv, cudaStream_t s, int *launches) {
    *launches += 3;
    const float *fq = static_cast<const float *>(q), *fk = static_cast<const float *>(k),
                *fv = static_cast<const float *>(v), *fg = static_cast<const float *>(dout);
    float *oq = static_cast<float *>(dq), *ok = static_cast<float *>(dk), *ov = static_cast<float *>(dv);
    return c.D == 64 ? backward<64>(c, fq, fk, fv, lse, fg, oq, ok, ov, s)
                     : backward<32>(c, fq, fk, fv, lse, fg, oq, ok, ov, s);
}

}  // namespace bias
}  // namespace mra
