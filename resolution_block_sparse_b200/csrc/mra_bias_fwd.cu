// mra_bias_fwd.cu - forward pass of the biased block-sparse attention in bf16
// on warp-level tensor-core products, for heads of 32 (heads of 64 run on
// tcgen05, mra_bias_tc.cu).
//
// One block takes one work item: kRows block rows of one head, a warp for each
// (32 queries, two fragments, so that every fragment of K and V is read from
// shared memory once for two products), against a run of key blocks that come
// by TMA, one per pipeline stage.  A warp whose row does not list a block
// releases its stage at once.
//
// Softmax in one pass over the keys.  A row's reference moves only
// when some score exceeds it by 2^8, which a vote of the warp finds without
// exchanging maxima; weights then stay below 2^8, sums and outputs in fp32.
// Scale, bias and reference are one fused multiply-add per score where the
// block has one bias value.
//
// Over all blocks of a short sequence (kDirect) the block makes its bias
// window, masks and list itself: one launch and no workspace.
#include "mra_bias_direct.cuh"
#include "mra_bias_warp.cuh"

namespace mra {
namespace bias {
namespace {

constexpr float kMove = 5.5f;     // growth of a row's maximum that moves its reference: e^5.5 < 2^8

// stages that leave room for the blocks that the registers allow
constexpr int stages(int rows) { return rows == 4 ? 5 : 3; }

template <int D, int kRows>
struct Smem {
    __nv_bfloat16 kv[stages(kRows)][2][kTokens * D];
    __nv_bfloat16 q[kRows * kTokens * D];
    BlockInfo info;
    Ring<stages(kRows)> ring;
    int count, last;
};
template <int D, int kRows, bool kDirect>
__global__ void __launch_bounds__(32 * kRows, 12 / kRows)
forward_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, const Call c, __nv_bfloat16 *out, float *lse) {
    constexpr int kThreads = 32 * kRows, kStages = stages(kRows);
    extern __shared__ unsigned char raw[];
    Smem<D, kRows> &s = *reinterpret_cast<Smem<D, kRows> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Window &win = *reinterpret_cast<Window *>(&s + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) ring_init(s.ring, kRows);
    pdl_wait();
    Item it;
    if (kDirect) {
        it = Item{(int)blockIdx.x / c.groups, (int)blockIdx.x % c.groups, 0, 0, 1 << 16, 0};
    } else {
        if (!take_item(c.row_item, c.counters + kRowItems, c.row_items, &it)) return;
        if (c.lists && c.bad[it.bh]) return;
    }
    const int b = it.bh / c.H, h = it.bh - b * c.H;
    const int row0 = it.group * kRows;                       // first block row
    if (tid == 0) {
        mbar_expect_tx(saddr(&s.ring.first), kRows * kTokens * D * 2);
        tma_load_3d(saddr(s.q), &tq, 0, row0 * kTokens, it.bh, saddr(&s.ring.first));
    }
    if (kDirect) {
        make_list<kRows>(c, win, s.info, &s.count, b, h, row0);
        it.count = s.count;
    } else {
        for (int i = tid; i < it.count; i += kThreads) {
            const int e = c.row_list[it.start + i], col = e & 0xffff;
            s.info.entry[i] = e;
            s.info.valid[i] = c.valid[b * c.nbr + col];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                s.info.tile[r][i] = row0 + r < c.nbr ? tile_bias(c, h, row0 + r, col) : 0.0f;
        }
        __syncthreads();
    }

    auto fill = [&](int t) {
        const int sg = t % kStages, y = (s.info.entry[t] & 0xffff) * kTokens;
        const uint32_t bar = saddr(&s.ring.full[sg]);
        mbar_expect_tx(bar, 2 * kTokens * D * 2);
        tma_load_3d(saddr(s.kv[sg][0]), &tk, 0, y, it.bh, bar);
        tma_load_3d(saddr(s.kv[sg][1]), &tv, 0, y, it.bh, bar);
        s.ring.issued = t + 1;
    };
    if (tid == 0)
        for (int t = 0; t < min(kStages, it.count); ++t) fill(t);
    const int r = row0 + warp, qpos = r * kTokens;           // this warp's block row
    const uint32_t rows_on = r >= c.nbr ? 0u : kDirect ? win.valid[r] : c.valid[b * c.nbr + r];
    const float *vec = kDirect ? win.vec + ((row0 + kRows) * kTokens - 1)
                               : c.vec + ((size_t)h * 2 + 1) * c.nbr * kTokens;
    volatile int *abort = &s.ring.abort;

    bool ok = first_wait(&s.ring.first, abort, c);
    unsigned qa[2][D / 16][4];
    const Lane<D> at(lane);
    load_a<D>(qa[0], s.q, warp * 32, at);
    load_a<D>(qa[1], s.q, warp * 32 + 16, at);
    float o[2][D / 8][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][t][e] = 0.0f;
    float m[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
    float2 l[2][2] = {{both(0.0f), both(0.0f)}, {both(0.0f), both(0.0f)}};

    for (int t = 0; ok && t < it.count; ++t) {
        const int sg = t % kStages;
        // the stage of the block before is free once every warp has read it;
        // the warps refill in turn
        if (t >= 1 && t - 1 + kStages < it.count && warp == t % kRows && lane == 0) {
            const int u = t - 1;
            if (guarded_wait(&s.ring.empty[u % kStages], (u / kStages) & 1, abort, c.status)) fill(u + kStages);
        }
        __syncwarp();
        // every warp waits for every block, so that none releases a stage twice
        // before the others have released it once
        ok = warp_wait(&s.ring.full[sg], (t / kStages) & 1, abort, c.status);
        if (!ok) break;
        const int entry = s.info.entry[t];
        if ((entry >> (kMemberShift + warp)) & 1) {
            const float u = s.info.tile[warp][t];
            const uint32_t kv = s.info.valid[t];
            float x[2][4][4];
            mul_abt<D, 2>(x, qa, s.kv[sg][0], at);
            float sc = c.scale, add = u;
            if (u == INFINITY || kv != 0xffffffffu || !(sc >= 0.0f)) {
                // several biases, or padded keys: the finished scores first
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    general_scores<false>(x[i], sc, u, vec, qpos + 16 * i, (entry & 0xffff) * kTokens,
                                          kv != 0xffffffffu, 0xffffffffu, kv, lane);
                sc = 1.0f;
                add = 0.0f;
            }
            float top[2][2];      // before scale and bias
            bool move = false;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y = fmaxf(x[i][0][2 * k], x[i][0][2 * k + 1]);
#pragma unroll
                    for (int n = 1; n < 4; ++n) y = fmaxf(fmaxf(y, x[i][n][2 * k]), x[i][n][2 * k + 1]);
                    const float mx = fmaf(y, sc, add);
                    top[i][k] = y;
                    move = move || mx > m[i][k] + kMove || (m[i][k] == -INFINITY && mx > m[i][k]);
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float x_top = quad_max(top[i][k]), y = fmaf(x_top, sc, add);
                        if (y > m[i][k]) {
                            const float f = fast_exp2((m[i][k] - y) * kLog2e);
                            m[i][k] = y;
                            l[i][k] = mul2(l[i][k], both(f));
                            if ((lane & 3) == 0) l[i][k].x += reference_rest(x_top, sc, add, y);
#pragma unroll
                            for (int n = 0; n < D / 8; ++n) {
                                o[i][n][2 * k] *= f;
                                o[i][n][2 * k + 1] *= f;
                            }
                        }
                    }
            }
            unsigned w[2][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 ref = both((add - (m[i][k] == -INFINITY ? 0.0f : m[i][k])) * kLog2e);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        float2 p = fma2(pair_of(x[i], n, k), both(sc * kLog2e), ref);
                        p.x = fast_exp2(p.x);
                        p.y = fast_exp2(p.y);
                        l[i][k] = add2(l[i][k], p);
                        put_operand(w[i], n, k, p);
                    }
                }
            }
            mul_ab<D, 2>(o, w, s.kv[sg][1], at, lane, kv);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(saddr(&s.ring.empty[sg]));
    }
    float sum[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) sum[i][k] = quad_sum(l[i][k].x + l[i][k].y);

    const int chunks = item_chunks(it);
    if (!kDirect && chunks > 1) {
        // partial results in the registers' own layout
        constexpr int kPer = D + 16;
        float *p = c.row_part + ((size_t)(it.slot + item_chunk(it)) * kPer) * kThreads + tid;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) p[((i * (D / 8) + n) * 4 + e) * kThreads] = o[i][n][e];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                p[(D + 2 * i + k) * kThreads] = m[i][k];
                p[(D + 4 + 2 * i + k) * kThreads] = sum[i][k];
            }
        }
        if (last_to_arrive(c.arrive + (size_t)it.bh * c.groups + it.group, chunks, &s.last)) {
            const float *q0 = c.row_part + ((size_t)it.slot * kPer) * kThreads + tid;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    m[i][k] = -INFINITY;
                    sum[i][k] = 0.0f;
                    for (int n = 0; n < chunks; ++n)
                        m[i][k] = fmaxf(m[i][k], __ldcg(q0 + ((size_t)n * kPer + D + 2 * i + k) * kThreads));
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;
                for (int j = 0; j < chunks; ++j) {
                    const float *pk = q0 + (size_t)j * kPer * kThreads;
                    float f[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float mk = __ldcg(pk + (D + 2 * i + k) * kThreads);
                        f[k] = mk == -INFINITY ? 0.0f : fast_exp2((mk - m[i][k]) * kLog2e);
                        sum[i][k] = fmaf(__ldcg(pk + (D + 4 + 2 * i + k) * kThreads), f[k], sum[i][k]);
                    }
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i][n][e] = fmaf(__ldcg(pk + ((i * (D / 8) + n) * 4 + e) * kThreads), f[e >> 1], o[i][n][e]);
                }
            }
        } else {
            ok = false;      // another block of the group writes
        }
    }
    if (ok && r < c.nbr) {
        const int g = lane >> 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int n = 16 * i + 8 * k + g;
                const bool live = ((rows_on >> n) & 1u) && sum[i][k] != 0.0f;      // (NaN: live)
                f[k] = live ? 1.0f / sum[i][k] : 0.0f;
                if (!live) {
#pragma unroll
                    for (int t = 0; t < D / 8; ++t) o[i][t][2 * k] = o[i][t][2 * k + 1] = 0.0f;
                }
                if (lse && (lane & 3) == 0 && qpos + n < c.N)
                    lse[(size_t)it.bh * c.N + qpos + n] = live ? m[i][k] + logf(sum[i][k]) : -INFINITY;
            }
            store_rows<D>(s.q, warp * 32 + 16 * i, o[i], f[0], f[1], out + ((size_t)it.bh * c.N + qpos + 16 * i) * D,
                          c.N - qpos - 16 * i, lane);
        }
    }
    ring_end(s.ring);
}

template <int D, int kRows, bool kDirect>
cudaError_t launch(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse, cudaStream_t s) {
    CUtensorMap tq, tk, tv;
    if (!make_head_map(&tq, q, c.BH, c.N, D, kRows * kTokens) || !make_head_map(&tk, k, c.BH, c.N, D, kTokens) ||
        !make_head_map(&tv, v, c.BH, c.N, D, kTokens))
        return cudaErrorInvalidValue;
    const size_t smem = sizeof(Smem<D, kRows>) + (kDirect ? sizeof(Window) : 0) + 1024;
    auto *kern = forward_kernel<D, kRows, kDirect>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_shared(kern, smem, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(kDirect ? c.BH * c.groups : c.row_items), dim3(32 * kRows), smem, s, tq, tk, tv, c,
                            static_cast<__nv_bfloat16 *>(out), lse);
}

}  // namespace

cudaError_t launch_forward_direct(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                                  cudaStream_t s) {
    return launch<32, 4, true>(c, q, k, v, out, lse, s);
}

cudaError_t launch_forward_bf16(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                                cudaStream_t s) {
    return c.group == 4 ? launch<32, 4, false>(c, q, k, v, out, lse, s) : launch<32, 2, false>(c, q, k, v, out, lse, s);
}

}  // namespace bias
}  // namespace mra
