// mra_bias_warp.cuh - pieces of the biased attention kernels in bf16 on
// warp-level tensor-core products: tile rings filled by TMA, the score
// fragments of one 16 x 32 tile with scale, bias and masks, and the products
// from registers.
//
// Fragment layout of a 16 x 32 tile x[4][4] in lane (g = lane / 4, c = lane %
// 4): x[t][e] is row g + 8 * (e / 2), column 8 t + 2 c + (e & 1).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "mra_async.cuh"
#include "mra_bias.cuh"
#include "mra_f32x2.cuh"
#include "mra_internal.cuh"
#include "mra_mma.cuh"
#include "mra_tcgen05.cuh"

namespace mra {
namespace bias {

using namespace async;
using mma::fast_exp2;
using mma::mma16816;
using mma::pack_bf16;
using mma::swz;

constexpr int kWarpThreads = 128;       // four warps, 16 rows each: 64 rows

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// [BH][N][D] bf16, boxes of box_rows x D, rows past N read as zeros; the
// swizzle is the one of mma::swz.
inline bool make_head_map(CUtensorMap *m, const void *base, int BH, int N, int D, unsigned box_rows) {
    tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * (cuuint64_t)N};
    cuuint32_t box[3] = {(cuuint32_t)D, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What an item's blocks need besides their tiles, gathered once per item.
struct BlockInfo {
    int entry[kMaxChunk];         // block | members << 16
    uint32_t valid[kMaxChunk];    // valid tokens of the block
    float tile[kMaxGroup][kMaxChunk];// bias of the block at each of the group's rows (columns)
};

__device__ __forceinline__ float tile_bias(const Call &c, int h, int row_block, int col_block) {
    return c.tile[(size_t)h * 2 * c.nbr + (col_block - row_block + c.nbr - 1)];
}

// Pipeline of K/V (or Q/dO) tiles: full[s] completes by TMA, empty[s] by one
// arrival of each warp.  The warps refill in turn; every wait is bounded and a wait
// that gives up raises the status word and stops the whole block.
template <int kStages>
struct Ring {
    unsigned long long full[kStages], empty[kStages], first;   // first: the item's own tiles
    int abort;
    int issued;
};

template <int kStages>
__device__ __forceinline__ void ring_init(Ring<kStages> &r, int warps = kWarpThreads / 32) {
    for (int i = 0; i < kStages; ++i) {
        mbar_init(saddr(&r.full[i]), 1);
        mbar_init(saddr(&r.empty[i]), warps);
    }
    mbar_init(saddr(&r.first), 1);
    r.abort = 0;
    r.issued = 0;
    mbar_init_fence();
}

__device__ __forceinline__ bool guarded_wait(unsigned long long *bar, uint32_t parity, volatile int *abort,
                                             unsigned int *status) {
    const uint32_t b = saddr(bar);
    if (mbar_try_wait(b, parity)) return true;
    if (*abort) return false;
    if (mbar_wait(b, parity)) return true;
    *abort = 1;
    atomicOr(status, kDevTimeout);
    return false;
}

// The same answer for the whole warp, whose collective instructions follow.
__device__ __forceinline__ bool warp_wait(unsigned long long *bar, uint32_t parity, volatile int *abort, unsigned int *status) {
    return __all_sync(0xffffffffu, guarded_wait(bar, parity, abort, status));
}

// A block's first wait; with the test hook it gives up at once.
__device__ __forceinline__ bool first_wait(unsigned long long *bar, volatile int *abort, const Call &c) {
    if (c.expire) {
        *abort = 1;
        atomicOr(c.status, kDevTimeout);
        return false;
    }
    return warp_wait(bar, 0, abort, c.status);
}

// The block's end, for all of its threads.  After a stop no copy of the block
// may land after its shared memory is given up: one thread waits (bounded) for
// every stage filled.
template <int kStages>
__device__ __forceinline__ void ring_end(Ring<kStages> &r) {
    if (!__syncthreads_or(*(volatile int *)&r.abort) || threadIdx.x != 0) return;
    mbar_wait(saddr(&r.first), 0);
    for (int t = max(0, r.issued - kStages); t < r.issued; ++t)
        mbar_wait(saddr(&r.full[t % kStages]), (t / kStages) & 1);
}

// ldmatrix at a register address plus a constant.  The 16-byte pieces of a
// tile's row lie at piece ^ f(row) (mma::swz) and f is the same for rows 8
// apart, so one address per lane and tile reaches every fragment: the piece by
// an exclusive or, the rows by the constant.
template <int kOffset>
__device__ __forceinline__ void ldsm(unsigned (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4 + %5];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(kOffset));
}
template <int kOffset>
__device__ __forceinline__ void ldsm_t(unsigned (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4 + %5];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(kOffset));
}
// Byte offsets of a lane in a tile: as the B operand of A . tile^T (row pairs
// 0..15, two pieces), and as the A operand or the B operand of W . tile.
template <int D>
struct Lane {
    uint32_t wide, tall;
    __device__ __forceinline__ explicit Lane(int lane) {
        const int r = (lane >> 4) * 8 + (lane & 7), q = lane & 15;
        wide = 2 * swz<D>(r, (lane >> 3) & 1);
        tall = 2 * swz<D>(q, lane >> 4);
    }
};

// A fragments (16 rows x D) of a swizzled tile [rows][D] from row row0 on.
template <int D>
__device__ __forceinline__ void load_a(unsigned (&a)[D / 16][4], const __nv_bfloat16 *tile, int row0, const Lane<D> &at) {
    const uint32_t base = mma::smem_u32(tile) + row0 * D * 2 + at.tall;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) ldsm<0>(a[ks], base ^ (ks << 5));
}

// x[i] (16 x 32) = A[i] (16 x D) . tile^T, tile [32][D], for kM fragments A.
// Every fragment of the tile is read once, one step ahead of its products: the
// latency of ldmatrix, not its rate, is what these loops would wait for.
template <int D, int kM>
__device__ __forceinline__ void mul_abt(float (&x)[kM][4][4], const unsigned (&a)[kM][D / 16][4],
                                        const __nv_bfloat16 *tile, const Lane<D> &at) {
    const uint32_t base = mma::smem_u32(tile) + at.wide;
    unsigned r[2][2][4];
    ldsm<0>(r[0][0], base);
    ldsm<16 * D * 2>(r[0][1], base);
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][t][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const int s = ks & 1;
        if (ks + 1 < D / 16) {
            ldsm<0>(r[s ^ 1][0], base ^ ((ks + 1) << 5));
            ldsm<16 * D * 2>(r[s ^ 1][1], base ^ ((ks + 1) << 5));
        }
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) mma16816(x[i][t], a[i][ks], r[s][t >> 1][2 * (t & 1)], r[s][t >> 1][2 * (t & 1) + 1]);
    }
}

// Two such products, x1 = A1 . tile1^T and x2 = A2 . tile2^T, in step.
template <int D>
__device__ __forceinline__ void mul_abt_two(float (&x1)[4][4], float (&x2)[4][4], const unsigned (&a1)[D / 16][4],
                                            const unsigned (&a2)[D / 16][4], const __nv_bfloat16 *tile1,
                                            const __nv_bfloat16 *tile2, const Lane<D> &at) {
    const uint32_t b1 = mma::smem_u32(tile1) + at.wide, b2 = mma::smem_u32(tile2) + at.wide;
    unsigned r[2][4][4];
    ldsm<0>(r[0][0], b1);
    ldsm<16 * D * 2>(r[0][1], b1);
    ldsm<0>(r[0][2], b2);
    ldsm<16 * D * 2>(r[0][3], b2);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x1[t][e] = x2[t][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const int s = ks & 1;
        if (ks + 1 < D / 16) {
            ldsm<0>(r[s ^ 1][0], b1 ^ ((ks + 1) << 5));
            ldsm<16 * D * 2>(r[s ^ 1][1], b1 ^ ((ks + 1) << 5));
            ldsm<0>(r[s ^ 1][2], b2 ^ ((ks + 1) << 5));
            ldsm<16 * D * 2>(r[s ^ 1][3], b2 ^ ((ks + 1) << 5));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) mma16816(x1[t], a1[ks], r[s][t >> 1][2 * (t & 1)], r[s][t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            mma16816(x2[t], a2[ks], r[s][2 + (t >> 1)][2 * (t & 1)], r[s][2 + (t >> 1)][2 * (t & 1) + 1]);
    }
}

// Registers of a B fragment whose tile rows do not take part, as zeros: such
// rows may hold anything, and 0 times a NaN must not be formed.
struct Keep {
    unsigned m[2][2];
    __device__ __forceinline__ Keep(uint32_t rows, int lane) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const uint32_t k = rows >> (kk * 16 + 2 * (lane & 3));
            m[kk][0] = ((k & 1u) ? 0xffffu : 0u) | ((k & 2u) ? 0xffff0000u : 0u);
            m[kk][1] = ((k & 256u) ? 0xffffu : 0u) | ((k & 512u) ? 0xffff0000u : 0u);
        }
    }
    __device__ __forceinline__ void apply(unsigned (&r)[4], int kk) const {
        r[0] &= m[kk][0];
        r[1] &= m[kk][1];
        r[2] &= m[kk][0];
        r[3] &= m[kk][1];
    }
};

// acc[i] (16 x D) += W[i] (16 x 32, bf16 fragments of a score tile) . tile;
// keep: the tile's rows that take part.  Fragments one step ahead, as above.
template <int D, int kM>
__device__ __forceinline__ void mul_ab(float (&acc)[kM][D / 8][4], const unsigned (&w)[kM][2][4],
                                       const __nv_bfloat16 *tile, const Lane<D> &at, int lane, uint32_t keep) {
    const uint32_t base = mma::smem_u32(tile) + at.tall;
    const Keep rows(keep, lane);
    const bool masked = keep != 0xffffffffu;
    constexpr int kSteps = D / 8;            // (kk, pair of column tiles)
    unsigned r[2][4];
    ldsm_t<0>(r[0], base);
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
        const int s = n & 1, kk = n / (kSteps / 2), t = n % (kSteps / 2) * 2;
        if (n + 1 < kSteps) {
            const int k1 = (n + 1) / (kSteps / 2), t1 = (n + 1) % (kSteps / 2) * 2;
            if (k1 == 0) ldsm_t<0>(r[s ^ 1], base ^ (t1 << 4));
            else ldsm_t<16 * D * 2>(r[s ^ 1], base ^ (t1 << 4));
        }
        if (masked) rows.apply(r[s], kk);
#pragma unroll
        for (int i = 0; i < kM; ++i) {
            mma16816(acc[i][t], w[i][kk], r[s][0], r[s][1]);
            mma16816(acc[i][t + 1], w[i][kk], r[s][2], r[s][3]);
        }
    }
}

// acc += (high + low) . tile: weights in two bf16 pieces.
template <int D>
__device__ __forceinline__ void mul_ab_pieces(float (&acc)[D / 8][4], const unsigned (&high)[2][4], const unsigned (&low)[2][4],
                                              const __nv_bfloat16 *tile, const Lane<D> &at, int lane, uint32_t keep) {
    const uint32_t base = mma::smem_u32(tile) + at.tall;
    const Keep rows(keep, lane);
    const bool masked = keep != 0xffffffffu;
    constexpr int kSteps = D / 8;
    unsigned r[2][4];
    ldsm_t<0>(r[0], base);
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
        const int s = n & 1, kk = n / (kSteps / 2), t = n % (kSteps / 2) * 2;
        if (n + 1 < kSteps) {
            const int k1 = (n + 1) / (kSteps / 2), t1 = (n + 1) % (kSteps / 2) * 2;
            if (k1 == 0) ldsm_t<0>(r[s ^ 1], base ^ (t1 << 4));
            else ldsm_t<16 * D * 2>(r[s ^ 1], base ^ (t1 << 4));
        }
        if (masked) rows.apply(r[s], kk);
        mma16816(acc[t], high[kk], r[s][0], r[s][1]);
        mma16816(acc[t + 1], high[kk], r[s][2], r[s][3]);
        mma16816(acc[t], low[kk], r[s][0], r[s][1]);
        mma16816(acc[t + 1], low[kk], r[s][2], r[s][3]);
    }
}

// Two neighbouring elements of a score tile, and their place in the A operand
// of mul_ab.  The weights enter the tensor cores as bf16: rounded once forward,
// a half step of the operand type, as large as that of the result's own type;
// in two pieces backward (mra_bias_bwd.cu).
__device__ __forceinline__ float2 pair_of(const float (&x)[4][4], int n, int k) {
    return make_float2(x[n][2 * k], x[n][2 * k + 1]);
}
__device__ __forceinline__ void put_operand(unsigned (&w)[2][4], int n, int k, float2 p) {
    w[n >> 1][(n & 1) * 2 + k] = pack_bf16(p.x, p.y);
}

// x = x * scale + bias of a 16 x 32 tile whose first row is position
// row0 and first column col0 (rows are queries, or keys with kTransposed).
// u: the block's one bias value, or +inf: read the vector (vec[j - i], 10 values a lane:
// a tile's bias depends on 8 t + 2 c + e - g - 8 * (row half) alone).
template <bool kTransposed>
__device__ __forceinline__ void add_bias(float (&x)[4][4], float scale, float u, const float *vec, int row0,
                                         int col0, int lane) {
    if (u != INFINITY) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = fmaf(x[t][e], scale, u);
        return;
    }
    const int d0 = col0 + 2 * (lane & 3) - row0 - (lane >> 2);
    float b[5][2];
#pragma unroll
    for (int t = 0; t < 5; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int d = d0 + 8 * (t - 1) + e;
            b[t][e] = vec[kTransposed ? -d : d];
        }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][e] = fmaf(x[t][e], scale, b[t + 1 - (e >> 1)][e & 1]);
}

// Whether element [t][e] of a tile takes part: row bits of this lane's two
// rows, column bits of the tile.
__device__ __forceinline__ bool pair_on(uint32_t rows, uint32_t cols, int t, int e, int lane) {
    return ((rows >> ((lane >> 2) + 8 * (e >> 1))) & 1u) && ((cols >> (8 * t + 2 * (lane & 3) + (e & 1))) & 1u);
}

// Scores of a block with several biases, or with rows or columns that take no
// part: with their bias, -inf where the pair does not count.
template <bool kTransposed>
__device__ __forceinline__ void general_scores(float (&x)[4][4], float scale, float u, const float *vec, int row0,
                                               int col0, bool masked, uint32_t rows, uint32_t cols, int lane) {
    add_bias<kTransposed>(x, scale, u, vec, row0, col0, lane);
    if (masked) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!pair_on(rows, cols, n, e, lane)) x[n][e] = -INFINITY;
    }
}

// exp(x * sc + add - lse) of two scores (nl: minus lse)
__device__ __forceinline__ float2 weight2(float2 x, float sc, float add, float2 nl) {
    const float2 z = mul2(add2(fma2(x, both(sc), both(add)), nl), both(kLog2e));
    return make_float2(fast_exp2(z.x), fast_exp2(z.y));
}

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// Writes a warp's 16 x D result as bf16 rows through its own 16 rows of a
// shared tile (16-byte stores, whole rows); rows at or past `rows` are left.
template <int D>
__device__ __forceinline__ void store_rows(__nv_bfloat16 *tile, int row0, const float (&acc)[D / 8][4], float f0,
                                           float f1, __nv_bfloat16 *dst, int rows, int lane) {
    const int g = lane >> 2, c2 = 2 * (lane & 3);
    __syncwarp();
#pragma unroll
    for (int t = 0; t < D / 8; ++t) {
        *reinterpret_cast<unsigned *>(tile + swz<D>(row0 + g, t) + c2) = pack_bf16(acc[t][0] * f0, acc[t][1] * f0);
        *reinterpret_cast<unsigned *>(tile + swz<D>(row0 + g + 8, t) + c2) = pack_bf16(acc[t][2] * f1, acc[t][3] * f1);
    }
    __syncwarp();
    constexpr int kPer = D / 8;
#pragma unroll
    for (int i = 0; i < 16 * kPer / 32; ++i) {
        const int e = i * 32 + lane, r = e / kPer, j = e % kPer;
        if (r < rows)
            *reinterpret_cast<uint4 *>(dst + (size_t)r * D + j * 8) =
                *reinterpret_cast<const uint4 *>(tile + swz<D>(row0 + r, j));
    }
    __syncwarp();
}

// Split group: true in every thread of the block that arrives last (the
// partial results of the other chunks are visible to it).
__device__ __forceinline__ bool last_to_arrive(int *counter, int chunks, int *s_last) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) *s_last = atomicAdd(counter, 1) == chunks - 1;
    __syncthreads();
    __threadfence();
    return *s_last != 0;
}

}  // namespace bias
}  // namespace mra
