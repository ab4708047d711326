// mra_bias_bwd.cu - backward pass of the biased block-sparse attention in
// bf16 on warp-level tensor-core products, without atomics on results: every
// gradient is summed in registers by the block that owns it, so two calls
// give the same bits.
//
//   row_kernel    (kDelta) delta_i = sum_j P_ij dP_ij, from the same fp32 P and dP that
//                 the gradients use.  (Taking it from the rounded output,
//                 dout . out, leaves the rounding of `out` in every dS_ij, as
//                 large as dS itself where one key holds most of a row's
//                 weight.)  Rows again, because all three need it.
//   row_kernel    by block rows: dQ += dS K, and the bias gradient: a block in
//                 one bucket adds its dS in registers; another one is summed
//                 along its diagonals through shared memory.
//   col_kernel    by block columns, on transposed tiles (keys are the rows of
//                 the fragments): dV += P^T dO, dK += dS^T Q, both weights
//                 straight from registers.
//
// Work items, rings and fragments as in the forward pass.
#include "mra_bias_warp.cuh"

namespace mra {
namespace bias {
namespace {

constexpr int kStages = 4;     // one streamed block each
// A 16 x 32 tile of dS in shared memory between zero margins, so that its
// diagonals are read without bounds; the pitch keeps fragment stores and
// diagonal reads free of bank conflicts.
constexpr int kDiag = 72, kMargin = 16;

// ---------------------------------------------------------------- rows: delta, dQ, bias gradient
template <int D>
struct RowSmem {
    __nv_bfloat16 kv[kStages][2][kTokens * D];
    __nv_bfloat16 q[2][kGroup * kTokens * D];          // Q, dO
    BlockInfo info;
    int bucket[kGroup][kMaxChunk];      // of each block at each row (Call::tile_bucket)
    Ring<kStages> ring;
    int last;
};

// Sums of dS by bucket over a warp's 16 rows.
struct BinSum {
    float *bins;        // [buckets], this warp's own
    float2 acc;         // this lane's sum over blocks of bucket `cur`
    int cur;
    __device__ __forceinline__ void flush(int lane) {
        if (cur < 0) return;
        float v = acc.x + acc.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) bins[cur] += v;
        acc = both(0.0f);
        __syncwarp();
    }
};

// Bins of a block with several buckets: the 47 diagonals of the 16 x 32 tile,
// lane l summing diagonals l and l + 32 through a skewed read.
__device__ __forceinline__ void bin_diagonals(const float (&ds)[4][4], float *tile, float *bins, const int32_t *bucket,
                                              int buckets, int N, int d_first, bool distinct, int lane) {
    float *const mine = tile + (lane >> 2) * kDiag + kMargin + 2 * (lane & 3);
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        *reinterpret_cast<float2 *>(mine + 8 * t) = make_float2(ds[t][0], ds[t][1]);
        *reinterpret_cast<float2 *>(mine + 8 * kDiag + 8 * t) = make_float2(ds[t][2], ds[t][3]);
    }
    __syncwarp();
    // diagonal k: column - row = k - 15, relative position d_first + k
    const int b0 = bucket_at(bucket, buckets, N, d_first + lane, true);
    const int b1 = bucket_at(bucket, buckets, N, d_first + 32 + lane, lane < 15);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const float *p = tile + r * (kDiag + 1) + kMargin - 15 + lane;
        s0 += p[0];
        if (lane < 16) s1 += p[32];
    }
    bin_runs(s0, b0, bins, distinct, lane);
    bin_runs(s1, b1, bins, distinct, lane);
}

// What the rounding of an operand to bf16 leaves.  P and dS enter their products
// in two bf16 pieces.  A weight's rounding and its result's are independent and of
// one size, so that weights rounded once give dq, dk and dv sqrt(2) times the
// error of the rounded exact result; with the rest in a second product it is that
// of the rounding alone, and costs 0 to 9 % (forward and backward, rounded once / in
// two pieces: 1 x 4 heads of 256 of 64 42.8 / 42.8 us, 1 x 2 of 2048 97.7 / 104; heads
// of 32: 8 x 12 of 512 120 / 127, 2 x 12 of 4096 1697 / 1850, BigBird 334 / 357).
__device__ __forceinline__ float2 residual(float2 v) {
    const unsigned h = mma::pack_bf16(v.x, v.y);
    return make_float2(v.x - __uint_as_float(h << 16), v.y - __uint_as_float(h & 0xffff0000u));
}

// Zeros the fragment rows of a warp's 16 x D result that are padded: they have no
// gradient, whatever the blocks that they meet hold (0 times a NaN among it).
template <int D>
__device__ __forceinline__ void clear_padded(float (&acc)[D / 8][4], uint32_t rows_on, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if ((rows_on >> ((lane >> 2) + 8 * i)) & 1u) continue;
#pragma unroll
        for (int t = 0; t < D / 8; ++t) acc[t][2 * i] = acc[t][2 * i + 1] = 0.0f;
    }
}

template <int D, bool kDelta>
__global__ void __launch_bounds__(kWarpThreads, 3)
row_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
           const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Call c,
           const float *lse, __nv_bfloat16 *dq) {
    extern __shared__ unsigned char raw[];
    RowSmem<D> &s = *reinterpret_cast<RowSmem<D> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    float *const diag = reinterpret_cast<float *>(&s + 1);          // dQ: [4][16][kDiag], then [4][buckets]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) ring_init(s.ring);
    rows_begin(!kDelta);
    Item it;
    if (!take_item(c.row_item, c.counters + kRowItems, c.row_items, &it)) return;
    if (c.lists && c.bad[it.bh]) return;
    const int b = it.bh / c.H, h = it.bh - b * c.H;
    const int row0 = it.group * kGroup;
    for (int i = tid; i < it.count; i += kWarpThreads) {
        const int e = c.row_list[it.start + i], col = e & 0xffff;
        s.info.entry[i] = e;
        s.info.valid[i] = c.valid[b * c.nbr + col];
#pragma unroll
        for (int r = 0; r < kGroup; ++r) {
            const bool on = row0 + r < c.nbr;
            s.info.tile[r][i] = on ? tile_bias(c, h, row0 + r, col) : 0.0f;
            if (!kDelta) s.bucket[r][i] = on ? c.tile_bucket[col - row0 - r + c.nbr - 1] : -1;
        }
    }
    float *const bins = diag + 4 * 16 * kDiag;
    if (!kDelta)
        for (int i = tid; i < 4 * 16 * kDiag + 4 * c.buckets; i += kWarpThreads) diag[i] = 0.0f;
    __syncthreads();

    auto fill = [&](int t) {
        const int sg = t % kStages, y = (s.info.entry[t] & 0xffff) * kTokens;
        const uint32_t bar = saddr(&s.ring.full[sg]);
        mbar_expect_tx(bar, 2 * kTokens * D * 2);
        tma_load_3d(saddr(s.kv[sg][0]), &tk, 0, y, it.bh, bar);
        tma_load_3d(saddr(s.kv[sg][1]), &tv, 0, y, it.bh, bar);
        s.ring.issued = t + 1;
    };
    if (tid == 0) {
        mbar_expect_tx(saddr(&s.ring.first), 2 * kGroup * kTokens * D * 2);
        tma_load_3d(saddr(s.q[0]), &tq, 0, row0 * kTokens, it.bh, saddr(&s.ring.first));
        tma_load_3d(saddr(s.q[1]), &tdo, 0, row0 * kTokens, it.bh, saddr(&s.ring.first));
        for (int t = 0; t < min(kStages, it.count); ++t) fill(t);
    }
    const int member = warp >> 1, r = row0 + member, wrow = warp * 16;
    const int qpos = row0 * kTokens + wrow, g = lane >> 2;
    const uint32_t rows_on = r < c.nbr ? c.valid[b * c.nbr + r] >> (wrow & 31) : 0u;
    const bool rows_all = (rows_on & 0xffffu) == 0xffffu;
    const float *vec = c.vec + ((size_t)h * 2 + 1) * c.nbr * kTokens;
    volatile int *abort = &s.ring.abort;
    float *const stat = r < c.nbr ? c.rowstat + ((size_t)it.bh * c.nbr + r) * 2 * kTokens + (wrow & 31) : nullptr;
    // minus lse (-inf: a row without a pair, whose weights are all 0) and minus
    // delta
    float nlse[2], ndelta[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = qpos + g + 8 * i;
        const float x = n < c.N ? lse[(size_t)it.bh * c.N + n] : -INFINITY;
        nlse[i] = x == -INFINITY ? -INFINITY : -x;
        if (!kDelta && stat) ndelta[i] = stat[kTokens + g + 8 * i];
    }

    bool ok = first_wait(&s.ring.first, abort, c);
    const Lane<D> at(lane);
    unsigned qa[1][D / 16][4], ga[1][D / 16][4];
    load_a<D>(qa[0], s.q[0], wrow, at);
    load_a<D>(ga[0], s.q[1], wrow, at);
    float acc[1][D / 8][4];
#pragma unroll
    for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][t][e] = 0.0f;
    BinSum bin{bins + warp * c.buckets, both(0.0f), -1};
    float2 sum[2] = {both(0.0f), both(0.0f)};

    for (int t = 0; ok && t < it.count; ++t) {
        const int sg = t % kStages;
        if (t >= 1 && t - 1 + kStages < it.count && warp == (t & 3) && lane == 0) {
            const int u = t - 1;
            if (guarded_wait(&s.ring.empty[u % kStages], (u / kStages) & 1, abort, c.status)) fill(u + kStages);
        }
        __syncwarp();
        ok = warp_wait(&s.ring.full[sg], (t / kStages) & 1, abort, c.status);
        if (!ok) break;
        const int entry = s.info.entry[t];
        if ((entry >> (kMemberShift + member)) & 1) {
            const int col = entry & 0xffff;
            const uint32_t kv = s.info.valid[t];
            const bool masked = kv != 0xffffffffu || !rows_all;
            const float u = s.info.tile[member][t];
            float x[1][4][4], dp[1][4][4];
            mul_abt_two<D>(x[0], dp[0], qa[0], ga[0], s.kv[sg][0], s.kv[sg][1], at);
            float sc = c.scale, add = u;
            if (u == INFINITY || masked) {
                general_scores<false>(x[0], sc, u, vec, qpos, col * kTokens, masked, rows_on, kv, lane);
                sc = 1.0f;
                add = 0.0f;
                if (masked) {
                    // V or dO of a pair that does not count may hold anything
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!pair_on(rows_on, kv, n, e, lane)) dp[0][n][e] = 0.0f;
                }
            }
            unsigned w[1][2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 nl = both(nlse[k]), nd = both(ndelta[k]);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    float2 p = weight2(pair_of(x[0], n, k), sc, add, nl);
                    const float2 d = pair_of(dp[0], n, k);
                    if (kDelta) {
                        sum[k] = fma2(p, d, sum[k]);
                    } else {
                        p = mul2(p, add2(d, nd));
                        put_operand(w[0], n, k, p);
                        x[0][n][2 * k] = p.x;
                        x[0][n][2 * k + 1] = p.y;
                    }
                }
            }
            if (!kDelta) {
                unsigned low[2][4];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) put_operand(low, n, k, residual(pair_of(x[0], n, k)));
                mul_ab_pieces<D>(acc[0], w[0], low, s.kv[sg][0], at, lane, kv);
                const int tb = s.bucket[member][t];
                if (tb >= 0) {
                    if (tb != bin.cur) {
                        bin.flush(lane);
                        bin.cur = tb;
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        bin.acc = add2(bin.acc, add2(pair_of(x[0], n, 0), pair_of(x[0], n, 1)));
                } else {
                    bin_diagonals(x[0], diag + warp * 16 * kDiag, bin.bins, c.bucket, c.buckets, c.N,
                                  col * kTokens - qpos - 15, tb == -2, lane);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(saddr(&s.ring.empty[sg]));
    }

    const int chunks = item_chunks(it);
    if (kDelta) {
        float total[2] = {quad_sum(sum[0].x + sum[0].y), quad_sum(sum[1].x + sum[1].y)};
        bool write = true;
        if (chunks > 1) {
            float *p = c.row_part + (size_t)(it.slot + item_chunk(it)) * 64 + wrow + g;
            if ((lane & 3) == 0) {
                p[0] = total[0];
                p[8] = total[1];
            }
            write = last_to_arrive(c.arrive + (size_t)it.bh * c.groups + it.group, chunks, &s.last);
            if (write) {
                total[0] = total[1] = 0.0f;
                for (int k = 0; k < chunks; ++k) {
                    const float *pk = c.row_part + (size_t)(it.slot + k) * 64 + wrow + g;
                    total[0] += __ldcg(pk);
                    total[1] += __ldcg(pk + 8);
                }
                // the next kernel's arrivals on this group count from zero
                if (tid == 0) c.arrive[(size_t)it.bh * c.groups + it.group] = 0;
            }
        }
        if (write && stat && (lane & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                stat[g + 8 * i] = nlse[i];
                stat[kTokens + g + 8 * i] = -total[i];
            }
        }
    } else {
        bin.flush(lane);
        __syncthreads();
        // the four warps' bins in warp order
        const int nb = c.buckets;
        float *const group_bins = c.bins + ((size_t)it.bh * c.groups + it.group) * nb;
        const int per = kWarpThreads * (D / 2);
        float *const part = c.row_part + (size_t)(it.slot + item_chunk(it)) * (per + nb);
        for (int i = tid; i < nb; i += kWarpThreads) {
            const float v = ((bins[i] + bins[nb + i]) + bins[2 * nb + i]) + bins[3 * nb + i];
            if (chunks > 1) part[per + i] = v;
            else group_bins[i] = v;
        }
        bool write = true;
        if (chunks > 1) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[(n * 4 + e) * kWarpThreads + tid] = acc[0][n][e];
            write = last_to_arrive(c.arrive + (size_t)it.bh * c.groups + it.group, chunks, &s.last);
            if (write) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[0][n][e] = 0.0f;
                const float *p0 = c.row_part + (size_t)it.slot * (per + nb);
                for (int k = 0; k < chunks; ++k) {
                    const float *pk = p0 + (size_t)k * (per + nb) + tid;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[0][n][e] += __ldcg(pk + (n * 4 + e) * kWarpThreads);
                }
                for (int i = tid; i < nb; i += kWarpThreads) {
                    float v = 0.0f;
                    for (int k = 0; k < chunks; ++k) v += __ldcg(p0 + (size_t)k * (per + nb) + per + i);
                    group_bins[i] = v;
                }
            }
        }
        clear_padded<D>(acc[0], rows_on, lane);
        if (ok && write)
            store_rows<D>(s.q[0], wrow, acc[0], c.scale, c.scale, dq + ((size_t)it.bh * c.N + qpos) * D, c.N - qpos, lane);
    }
    ring_end(s.ring);
}

// ---------------------------------------------------------------- columns: dK, dV
template <int D>
struct ColSmem {
    __nv_bfloat16 qg[kStages][2][kTokens * D];     // Q, dO
    __nv_bfloat16 kv[2][kGroup * kTokens * D];     // K, V of the item
    float stat[kStages][2][kTokens];               // minus lse, minus delta
    BlockInfo info;
    Ring<kStages> ring;
    int last;
};

template <int D>
__device__ __forceinline__ void col_item(const CUtensorMap &tq, const CUtensorMap &tdo, const CUtensorMap &tk,
                                         const CUtensorMap &tv, const Call &c, __nv_bfloat16 *dk, __nv_bfloat16 *dv,
                                         unsigned char *raw) {
    ColSmem<D> &s = *reinterpret_cast<ColSmem<D> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) ring_init(s.ring);
    Item it;
    if (!take_item(c.col_item, c.counters + kColItems, c.col_items, &it)) return;
    if (c.lists && c.bad[it.bh]) return;
    const int b = it.bh / c.H, h = it.bh - b * c.H;
    const int col0 = it.group * kGroup;
    for (int i = tid; i < it.count; i += kWarpThreads) {
        const int e = c.col_list[it.start + i], row = e & 0xffff;
        s.info.entry[i] = e;
        s.info.valid[i] = c.valid[b * c.nbr + row];
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
            s.info.tile[k][i] = col0 + k < c.nbr ? tile_bias(c, h, row, col0 + k) : 0.0f;
    }
    __syncthreads();

    auto fill = [&](int t) {
        const int sg = t % kStages, row = s.info.entry[t] & 0xffff;
        const uint32_t bar = saddr(&s.ring.full[sg]);
        mbar_expect_tx(bar, 2 * kTokens * D * 2 + 2 * kTokens * 4);
        tma_load_3d(saddr(s.qg[sg][0]), &tq, 0, row * kTokens, it.bh, bar);
        tma_load_3d(saddr(s.qg[sg][1]), &tdo, 0, row * kTokens, it.bh, bar);
        bulk_load(saddr(s.stat[sg]), c.rowstat + ((size_t)it.bh * c.nbr + row) * 2 * kTokens, 2 * kTokens * 4, bar);
        s.ring.issued = t + 1;
    };
    if (tid == 0) {
        mbar_expect_tx(saddr(&s.ring.first), 2 * kGroup * kTokens * D * 2);
        tma_load_3d(saddr(s.kv[0]), &tk, 0, col0 * kTokens, it.bh, saddr(&s.ring.first));
        tma_load_3d(saddr(s.kv[1]), &tv, 0, col0 * kTokens, it.bh, saddr(&s.ring.first));
        for (int t = 0; t < min(kStages, it.count); ++t) fill(t);
    }
    const int member = warp >> 1, col = col0 + member, wrow = warp * 16;
    const int kpos = col0 * kTokens + wrow;
    const uint32_t keys_on = col < c.nbr ? c.valid[b * c.nbr + col] >> (wrow & 31) : 0u;
    const bool keys_all = (keys_on & 0xffffu) == 0xffffu;
    const float *vec = c.vec + ((size_t)h * 2 + 1) * c.nbr * kTokens;
    volatile int *abort = &s.ring.abort;

    bool ok = first_wait(&s.ring.first, abort, c);
    const Lane<D> at(lane);
    unsigned ka[1][D / 16][4], va[1][D / 16][4];
    load_a<D>(ka[0], s.kv[0], wrow, at);
    load_a<D>(va[0], s.kv[1], wrow, at);
    float ak[1][D / 8][4], av[1][D / 8][4];
#pragma unroll
    for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) ak[0][t][e] = av[0][t][e] = 0.0f;

    for (int t = 0; ok && t < it.count; ++t) {
        const int sg = t % kStages;
        if (t >= 1 && t - 1 + kStages < it.count && warp == (t & 3) && lane == 0) {
            const int u = t - 1;
            if (guarded_wait(&s.ring.empty[u % kStages], (u / kStages) & 1, abort, c.status)) fill(u + kStages);
        }
        __syncwarp();
        ok = warp_wait(&s.ring.full[sg], (t / kStages) & 1, abort, c.status);
        if (!ok) break;
        const int entry = s.info.entry[t];
        if ((entry >> (kMemberShift + member)) & 1) {
            const uint32_t qv = s.info.valid[t];
            const bool part = qv != 0xffffffffu, masked = part || !keys_all;
            const float u = s.info.tile[member][t];
            float x[1][4][4], dp[1][4][4];
            mul_abt_two<D>(x[0], dp[0], ka[0], va[0], s.qg[sg][0], s.qg[sg][1], at);
            float sc = c.scale, add = u;
            if (u == INFINITY || masked) {
                general_scores<true>(x[0], sc, u, vec, kpos, (entry & 0xffff) * kTokens, masked, keys_on, qv, lane);
                sc = 1.0f;
                add = 0.0f;
                if (masked) {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!pair_on(keys_on, qv, n, e, lane)) dp[0][n][e] = 0.0f;
                }
            }
            // P in two pieces, then dS over them
            unsigned high[2][4], low[2][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 nl = *reinterpret_cast<const float2 *>(&s.stat[sg][0][8 * n + 2 * (lane & 3)]);
                const float2 nd = *reinterpret_cast<const float2 *>(&s.stat[sg][1][8 * n + 2 * (lane & 3)]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 p = weight2(pair_of(x[0], n, k), sc, add, nl);
                    const float2 ds = mul2(p, add2(pair_of(dp[0], n, k), nd));
                    put_operand(high, n, k, p);
                    put_operand(low, n, k, residual(p));
                    x[0][n][2 * k] = ds.x;
                    x[0][n][2 * k + 1] = ds.y;
                }
            }
            mul_ab_pieces<D>(av[0], high, low, s.qg[sg][1], at, lane, qv);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 ds = pair_of(x[0], n, k);
                    put_operand(high, n, k, ds);
                    put_operand(low, n, k, residual(ds));
                }
            mul_ab_pieces<D>(ak[0], high, low, s.qg[sg][0], at, lane, qv);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(saddr(&s.ring.empty[sg]));
    }

    const int chunks = item_chunks(it);
    if (chunks > 1) {
        const size_t per = (size_t)kWarpThreads * D;
        float *p = c.col_part + (size_t)(it.slot + item_chunk(it)) * per + tid;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[(n * 4 + e) * kWarpThreads] = ak[0][n][e];
                p[(D / 2 + n * 4 + e) * kWarpThreads] = av[0][n][e];
            }
        if (last_to_arrive(c.arrive + (size_t)(c.BH + it.bh) * c.groups + it.group, chunks, &s.last)) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) ak[0][n][e] = av[0][n][e] = 0.0f;
            for (int k = 0; k < chunks; ++k) {
                const float *pk = c.col_part + (size_t)(it.slot + k) * per + tid;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ak[0][n][e] += __ldcg(pk + (n * 4 + e) * kWarpThreads);
                        av[0][n][e] += __ldcg(pk + (D / 2 + n * 4 + e) * kWarpThreads);
                    }
            }
        } else {
            ok = false;
        }
    }
    if (ok) {
        const size_t at = ((size_t)it.bh * c.N + kpos) * D;
        clear_padded<D>(ak[0], keys_on, lane);
        clear_padded<D>(av[0], keys_on, lane);
        store_rows<D>(s.kv[0], wrow, ak[0], c.scale, c.scale, dk + at, c.N - kpos, lane);
        store_rows<D>(s.kv[1], wrow, av[0], 1.0f, 1.0f, dv + at, c.N - kpos, lane);
    }
    ring_end(s.ring);
}

template <int D>
__global__ void __launch_bounds__(kWarpThreads, 3)
col_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
           const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Call c,
           __nv_bfloat16 *dk, __nv_bfloat16 *dv) {
    extern __shared__ unsigned char raw[];
    columns_begin();
    col_item<D>(tq, tdo, tk, tv, c, dk, dv, raw);
    table_gradient(c, kWarpThreads / 32);
}

template <int D>
cudaError_t launch(const Call &c, const void *q, const void *k, const void *v, const float *lse, const void *dout,
                   void *dq, void *dk, void *dv, cudaStream_t s, int *launches) {
    CUtensorMap q64, g64, k32, v32, q32, g32, k64, v64;
    const unsigned two = kGroup * kTokens;
    if (!make_head_map(&q64, q, c.BH, c.N, D, two) || !make_head_map(&g64, dout, c.BH, c.N, D, two) ||
        !make_head_map(&k32, k, c.BH, c.N, D, kTokens) || !make_head_map(&v32, v, c.BH, c.N, D, kTokens) ||
        !make_head_map(&q32, q, c.BH, c.N, D, kTokens) || !make_head_map(&g32, dout, c.BH, c.N, D, kTokens) ||
        !make_head_map(&k64, k, c.BH, c.N, D, two) || !make_head_map(&v64, v, c.BH, c.N, D, two))
        return cudaErrorInvalidValue;
    const size_t row = sizeof(RowSmem<D>) + 1024;
    const size_t row_bins = row + (4 * 16 * kDiag + 4 * (size_t)c.buckets) * sizeof(float);
    const size_t col = sizeof(ColSmem<D>) + 1024;
    static std::atomic<unsigned long long> done[3] = {};
    const size_t most = row_bins + 4 * (size_t)(kMaxBuckets - c.buckets) * sizeof(float);
    cudaError_t e = allow_shared(row_kernel<D, true>, row, done[0]);
    if (e == cudaSuccess) e = allow_shared(row_kernel<D, false>, most, done[1]);
    if (e == cudaSuccess) e = allow_shared(col_kernel<D>, col, done[2]);
    if (e != cudaSuccess) return e;
    e = launch_dependent(row_kernel<D, true>, dim3(c.row_items), dim3(kWarpThreads), row, s, q64, g64, k32, v32, c, lse,
                         (__nv_bfloat16 *)nullptr);
    if (e != cudaSuccess) return e;
    e = launch_dependent(row_kernel<D, false>, dim3(c.row_items), dim3(kWarpThreads), row_bins, s, q64, g64, k32, v32, c,
                         lse, static_cast<__nv_bfloat16 *>(dq));
    if (e != cudaSuccess) return e;
    *launches += 3;
    return launch_dependent(col_kernel<D>, dim3(c.col_items), dim3(kWarpThreads), col, s, q32, g32, k64, v64, c,
                            static_cast<__nv_bfloat16 *>(dk), static_cast<__nv_bfloat16 *>(dv));
}

}  // namespace

cudaError_t launch_backward_bf16(const Call &c, const void *q, const void *k, const void *v, const float *lse,
                                 const void *dout, void *dq, void *dk, void *dv, cudaStream_t s, int *launches) {
    return c.D == 64 ? launch<64>(c, q, k, v, lse, dout, dq, dk, dv, s, launches)
                     : launch<32>(c, q, k, v, lse, dout, dq, dk, dv, s, launches);
}

}  // namespace bias
}  // namespace mra
