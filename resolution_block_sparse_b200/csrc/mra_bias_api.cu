// mra_bias_api.cu - C entry points of the block-sparse attention with a
// learned relative position bias: argument checks, the carving of the
// caller's workspace, the launch sequence, and the host generator of bucket
// maps.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "mra.h"
#include "mra_bias.cuh"
#include "mra_internal.cuh"

using namespace mra;

namespace {

using bias::Call;
using bias::Item;

long long div_up(long long a, long long b) { return (a + b - 1) / b; }

// Sizes that every entry point refuses, and the work-item plan.
int plan(int B, int H, int N, int D, int cap, bool lists, int buckets, int dtype, bool backward, Call *c) {
    if (B < 1 || H < 1 || N < 1 || buckets < 1) return MRA_ERR_INVALID_ARG;
    if (dtype != MRA_DTYPE_BF16 && dtype != MRA_DTYPE_F32) return MRA_ERR_INVALID_ARG;
    if ((D != 32 && D != 64) || N > kMaxN || buckets > bias::kMaxBuckets) return MRA_ERR_UNSUPPORTED;
    *c = Call{};
    c->B = B;
    c->H = H;
    c->N = N;
    c->D = D;
    c->nbr = (N + bias::kTokens - 1) / bias::kTokens;
    c->words = (c->nbr + 31) / 32;
    // tcgen05 kernels (bf16, heads of 64) or warp-level ones.  The first take four
    // block rows an item, pay for the union of their lists and need more work to
    // fill the GPU; listed: the blocks of all heads' lists.  Measured (us, warp-level
    // against tcgen05; B x H, N, blocks a row; in brackets listed blocks per SM):
    //  backward (with the forward), all blocks: 4x12, 512 [83]: 115 / 87; 1x3, 2048
    //   [83]: 130 / 119; 1x8, 1024 [55]: 101 / 95; 1x2, 2048 [55]: 104 / 110; 2x12,
    //   512 [42]: 80 / 78; 1x12, 512 [21]: 58 / 67
    //  backward, lists: 2x12, 4096, 8 [166]: 293 / 262, 4 [83]: 192 / 190; 1x4, 4096,
    //   28 [97]: 185 / 162; 1x2, 4096, 28 [48]: 124 / 123; 2x12, 1024, 8 [42]: 111 / 102
    //  forward (heads of 64 have the tcgen05 kernel alone), when both were there:
    //   2x12, 4096, all blocks: 453 / 236, BigBird 91 / 77, random lists of 3 to
    //   12 % within 10 % of each other
    const long long all = (long long)c->nbr * c->nbr, listed = (long long)B * H * (lists ? cap : all);
    const int sms = device_sm_count();
    c->tc = dtype == MRA_DTYPE_BF16 && D == 64 && (!backward || listed >= 68LL * sms);
    // The warp-level forward kernel (heads of 32) takes four rows an item where
    // every second block or more is listed (their union is then little longer
    // than one row, and the traffic from L2 halves again), else two.
    const bool dense = !lists || 2LL * cap >= all;
    c->group = c->tc || (dtype == MRA_DTYPE_BF16 && !backward && dense) ? 4 : bias::kGroup;
    c->groups = (c->nbr + c->group - 1) / c->group;
    c->buckets = buckets;
    const long long BH = (long long)B * H, pairs = (long long)c->groups * c->nbr;
    if (BH > 65535) return MRA_ERR_UNSUPPORTED;
    if (lists && (cap < 1 || (long long)cap > (long long)c->nbr * c->nbr)) return MRA_ERR_INVALID_ARG;
    // entries of the union lists are counted in 32 bits
    const long long total = BH * (lists ? std::min<long long>(cap, pairs) : pairs);
    if (total > 0x3fffffffLL || BH * c->groups > 0x3fffffffLL || (lists && BH * cap > 0x3fffffffLL)) return MRA_ERR_UNSUPPORTED;
    c->BH = (int)BH;
    c->cap = lists ? cap : 0;
    // Blocks per item.  An item costs its blocks, its own tiles, descriptors and
    // result (3 to 5 blocks) and, where its group is split, the join (4 more).
    const long long resident = (c->tc ? 2LL : c->group == 4 ? 3LL : dtype == MRA_DTYPE_BF16 && !backward ? 6LL : 3LL) * device_sm_count();
    auto in = [](long long x, long long lo, long long hi) { return (int)std::max(lo, std::min(hi, x)); };
    if (dtype == MRA_DTYPE_F32) {
        // fp32 items are long in time and a causal half of their blocks is
        // skipped: two rounds of short items level that (8 heads of 1000 causal
        // tokens of 32, step: 154 us with 4 blocks, 166 with 5, 191 with 12; 1500
        // tokens of 64: 831 us with 16, 864 with 6, 915 with 4).
        c->chunk = in(div_up(total, 2 * (D == 32 ? 4 : 2) * device_sm_count()), 1, 32);
        c->chunk = (c->chunk + 3) / 4 * 4;
    } else if (lists && c->tc) {
        // Unions of four rows, taken as they come: a split pays for the longest
        // rows only (BigBird at 4096, B = 2, H = 12: 64.4 us with 64 blocks, 68.2
        // with 32; at 2048, B = 1, H = 4, step: 102 us with 22, 121 with 8).
        c->chunk = in(div_up(total, resident), 20, bias::kMaxChunk);
    } else if (lists) {
        // enough items for two rounds of the blocks that the GPU holds
        c->chunk = in(div_up(total, 2 * resident), 8, 32);
    } else {
        // All blocks: the rows are equally long.  The split with the earliest end:
        // by rounds of items; persistent blocks, which take their items as they
        // come, by the items' sum and half an item's tail (dense 4096: 199.6 us in
        // 2 chunks, 212.8 in 3, 219.8 in 4; one head pair: 43.9, 42.7, 38.5).
        long long best = -1;
        for (int n = 1; n <= c->nbr; ++n) {
            const long long each = (c->nbr + n - 1) / n;
            if (each > bias::kMaxChunk) continue;
            if (n > 1 && each < 8 && best >= 0) break;
            const long long items = BH * c->groups * n, item = each + (c->tc ? (n > 1 ? 9 : 5) : n > 1 ? 5 : 3);
            const long long cost = items <= resident ? 2 * item
                                   : c->tc ? 2 * items * item / resident + item : 2 * div_up(items, resident) * item;
            if (best < 0 || cost < best) {
                best = cost;
                c->chunk = (int)each;
            }
        }
    }
    c->direct = !backward && dtype == MRA_DTYPE_BF16 && !lists && c->nbr <= bias::kDirectBlocks;
    c->row_items = (int)(BH * c->groups + total / c->chunk);
    c->col_items = c->row_items;
    return MRA_OK;
}

// Offsets of the workspace's parts; writes them into c when base is given.
size_t carve(Call *c, char *base, bool backward) {
    if (c->direct) return 0;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at = (at + bytes + 255) & ~(size_t)255;
        return base ? base + p : nullptr;
    };
    const size_t BH = c->BH, L = (size_t)c->nbr * bias::kTokens, groups = BH * c->groups;
    const size_t total = BH * std::min<size_t>(c->cap ? c->cap : (size_t)-1, (size_t)c->groups * c->nbr);
    // a split group of t entries takes ceil(t / chunk) <= 2 t / chunk slots
    const size_t slots = std::min<size_t>(c->row_items, 2 * total / c->chunk);
    c->valid = (uint32_t *)take(4ull * c->B * c->nbr);
    c->vec = (float *)take(4ull * c->H * 2 * L);
    c->tile = (float *)take(4ull * c->H * 2 * c->nbr);
    c->tile_bucket = (int *)take(4ull * 2 * c->nbr);
    c->counters = (int *)take(4ull * (bias::kCounters + BH + 2 * groups));
    if (base) {
        c->bad = c->counters + bias::kCounters;
        c->arrive = c->bad + BH;
    }
    c->rows = (uint32_t *)take(4ull * BH * c->nbr * c->words);
    c->row_list = (int *)take(4ull * total);
    c->row_item = (Item *)take(sizeof(Item) * (size_t)c->row_items);
    const size_t part = backward ? std::max<size_t>(bias::row_part_floats(c->D, c->group, c->buckets), 128)
                                 : bias::forward_part_floats(c->D, c->group);
    c->row_part = (float *)take(4ull * slots * part);
    if (backward) {
        c->col_list = (int *)take(4ull * total);
        c->col_item = (Item *)take(sizeof(Item) * (size_t)c->col_items);
        c->col_part = (float *)take(4ull * slots * bias::col_part_floats(c->D, c->group));
        c->rowstat = (float *)take(4ull * BH * L * 2);
        c->bins = (float *)take(4ull * groups * c->buckets);
    }
    return at;
}

bool misaligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

int prepare_call(const void *const *tensors, int n, const float *key_mask, const void *bias_table, const int32_t *bucket,
                 int num_buckets, float scale, const float *lse, int B, int H, int N, int D, const int32_t *block_idx,
                 int cap_sel, int dtype, void *workspace, size_t workspace_bytes, bool backward, Call *c) {
    int rc = plan(B, H, N, D, cap_sel, block_idx != nullptr, num_buckets, dtype, backward, c);
    if (rc != MRA_OK) return rc;
    for (int i = 0; i < n; ++i)
        if (!tensors[i] || misaligned(tensors[i], 16)) return MRA_ERR_INVALID_ARG;
    if (!bias_table || misaligned(bias_table, dtype == MRA_DTYPE_BF16 ? 2 : 4)) return MRA_ERR_INVALID_ARG;
    if (!bucket || misaligned(bucket, 4) || misaligned(block_idx, 4)) return MRA_ERR_INVALID_ARG;
    if (misaligned(key_mask, 4) || misaligned(lse, 4)) return MRA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(scale * bias::kLog2e)) return MRA_ERR_INVALID_ARG;
    if ((!workspace && !c->direct) || misaligned(workspace, 256)) return MRA_ERR_INVALID_ARG;
    if (workspace_bytes < carve(c, nullptr, backward)) return MRA_ERR_TOO_LARGE;
    rc = current_status_word(&c->status);
    if (rc != MRA_OK) return rc;
    carve(c, static_cast<char *>(workspace), backward);
    c->scale = scale;
    c->mask = key_mask;
    c->table = bias_table;
    c->bucket = bucket;
    c->lists = block_idx;
    // MRA_TEST_EXPIRE_WAIT=1 (read at every call): the first wait of every block
    // of the kernels that wait reports expiry without waiting, to test the way out
    const char *expire = getenv("MRA_TEST_EXPIRE_WAIT");
    c->expire = expire && expire[0] == '1' ? 1 : 0;
    return MRA_OK;
}

// A whole number for n^K first^m >= max^m first^K, in 32-bit limbs: at most 512
// factors below 2^31 and 512 of at most 512 (kMaxBuckets / 2), 656 limbs.  No
// memory of its own: an exception must not leave a C entry.
struct Whole {
    int n = 1;
    uint32_t limb[(bias::kMaxBuckets / 2) * (31 + 10) / 32 + 1] = {1};
    void times(uint32_t f) {
        uint64_t carry = 0;
        for (int i = 0; i < n; ++i) {
            carry += (uint64_t)limb[i] * f;
            limb[i] = (uint32_t)carry;
            carry >>= 32;
        }
        if (carry) limb[n++] = (uint32_t)carry;
    }
    Whole(uint32_t a, int ea, uint32_t b, int eb) {
        for (int i = 0; i < ea; ++i) times(a);
        for (int i = 0; i < eb; ++i) times(b);
    }
};
bool at_least(const Whole &a, const Whole &b) {
    if (a.n != b.n) return a.n > b.n;
    for (int i = a.n; i-- > 0;)
        if (a.limb[i] != b.limb[i]) return a.limb[i] > b.limb[i];
    return true;
}

}  // namespace

extern "C" {

size_t mra_blocksparse_attention_bias_workspace(int B, int H, int N, int D, int cap_sel, int num_buckets, int dtype,
                                                int backward) {
    Call c;
    if (plan(B, H, N, D, cap_sel, cap_sel != 0, num_buckets, dtype, backward != 0, &c) != MRA_OK) return 0;
    return carve(&c, nullptr, backward != 0);
}

int mra_blocksparse_attention_bias_fwd(const void *q, const void *k, const void *v, const float *key_mask,
                                       const void *bias_table, const int32_t *bucket, int num_buckets, float scale,
                                       void *out, float *lse, int B, int H, int N, int D, const int32_t *block_idx,
                                       int cap_sel, int dtype, void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
    const void *tensors[] = {q, k, v, out};
    Call c;
    int rc = prepare_call(tensors, 4, key_mask, bias_table, bucket, num_buckets, scale, lse, B, H, N, D, block_idx,
                          cap_sel, dtype, workspace, workspace_bytes, false, &c);
    if (rc != MRA_OK) return rc;
    const bool bf16 = dtype == MRA_DTYPE_BF16;
    int launches = 1;
    cudaError_t e = c.direct ? cudaSuccess : bias::launch_prepare(c, bf16, false, stream, &launches);
    if (e == cudaSuccess)
        e = c.tc ? bias::launch_forward_tc(c, q, k, v, out, lse, stream)
            : c.direct ? bias::launch_forward_direct(c, q, k, v, out, lse, stream)
            : bf16 ? bias::launch_forward_bf16(c, q, k, v, out, lse, stream)
                 : bias::launch_forward_f32(c, q, k, v, out, lse, stream);
    if (e != cudaSuccess) return MRA_ERR_CUDA;
    set_last_launches(launches);
    return MRA_OK;
}

int mra_blocksparse_attention_bias_bwd(const void *q, const void *k, const void *v, const float *key_mask,
                                       const void *bias_table, const int32_t *bucket, int num_buckets, float scale,
                                       const float *lse, const void *dout, void *dq, void *dk, void *dv,
                                       void *dbias_table, int B, int H, int N, int D, const int32_t *block_idx,
                                       int cap_sel, int dtype, void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
    const void *tensors[] = {q, k, v, dout, dq, dk, dv};
    Call c;
    if (!lse) return MRA_ERR_INVALID_ARG;
    if (!dbias_table || misaligned(dbias_table, dtype == MRA_DTYPE_BF16 ? 2 : 4)) return MRA_ERR_INVALID_ARG;
    int rc = prepare_call(tensors, 7, key_mask, bias_table, bucket, num_buckets, scale, lse, B, H, N, D, block_idx,
                          cap_sel, dtype, workspace, workspace_bytes, true, &c);
    if (rc != MRA_OK) return rc;
    const bool bf16 = dtype == MRA_DTYPE_BF16;
    int launches = 0;
    c.dtable = dbias_table;
    c.table_bf16 = bf16 ? 1 : 0;
    cudaError_t e = bias::launch_prepare(c, bf16, true, stream, &launches);
    if (e == cudaSuccess)
        e = c.tc ? bias::launch_backward_tc(c, q, k, v, lse, dout, dq, dk, dv, stream, &launches)
            : bf16 ? bias::launch_backward_bf16(c, q, k, v, lse, dout, dq, dk, dv, stream, &launches)
                 : bias::launch_backward_f32(c, q, k, v, lse, dout, dq, dk, dv, stream, &launches);
    if (e != cudaSuccess) return MRA_ERR_CUDA;
    set_last_launches(launches);
    return MRA_OK;
}

int mra_relative_buckets(int N, int num_buckets, int max_distance, int bidirectional, int32_t *out) {
    if (N < 1 || !out || misaligned(out, 4)) return MRA_ERR_INVALID_ARG;
    if (N > kMaxN || num_buckets > bias::kMaxBuckets) return MRA_ERR_UNSUPPORTED;
    if (bidirectional && (num_buckets & 1)) return MRA_ERR_INVALID_ARG;
    const int per = bidirectional ? num_buckets / 2 : num_buckets, first = per / 2, far = per - first;
    if (per < 2 || max_distance <= first) return MRA_ERR_INVALID_ARG;
    const double ratio = far / std::log((double)max_distance / first);
    for (int n = 0; n < N; ++n) {
        int b = n;
        if (n >= max_distance) {
            b = per - 1;
        } else if (n >= first) {
            const double t = ratio * std::log((double)n / first);
            int m = (int)t;
            // next to a border the whole-number comparison decides
            const int near = (int)std::lround(t);
            if (std::fabs(t - near) < 1e-6)
                m = near == 0 || at_least(Whole(n, far, first, near), Whole(max_distance, near, first, far))
                        ? near
                        : near - 1;
            b = std::min(first + m, per - 1);
        }
        out[N - 1 - n] = b;
        if (n > 0) out[N - 1 + n] = bidirectional ? per + b : -1;
    }
    return MRA_OK;
}

}  // extern "C"
