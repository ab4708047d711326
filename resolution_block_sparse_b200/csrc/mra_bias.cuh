// mra_bias.cuh - block-sparse attention with a learned bias per bucket of the
// relative position (forward and backward): what its kernels share.
//
//   S_ij = scale q_i . k_j + T[bucket(j - i)][h]       (listed 32x32 blocks)
//   P = softmax_j(S), O = P V, lse_i = log sum_j exp S_ij
//   dP = dO V^T, delta_i = sum_j P dP, dS = P (dP - delta)
//   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO
// Scores and references are kept in natural units: in the backward pass P =
// exp(S - lse) takes S rounded exactly as the forward pass rounded it, and only
// then the factor of the base-2 exponential.
//   dT[b][h] = sum of dS over the pairs whose relative position is in bucket b
//
// The bias of a head depends on j - i alone, so a 32x32 block at block offset
// c - r sees 63 values of one vector, and where all 63 fall into one bucket
// (every far block of a logarithmic bucket map) a single number.  The prepare
// kernel writes that vector and the per-offset number once per call; the
// attention kernels never touch the table or the map per element.
//
// Work is cut into items: two or four adjacent block rows (for dK and dV: block
// columns) of one head against a run of at most `chunk` blocks of
// the union of their lists.  Sharing each loaded block between the rows
// divides the traffic from L2, which bounds a kernel that takes single rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mra {
namespace bias {

constexpr int kTokens = 32;             // tokens per block
constexpr int kGroup = 2;               // block rows (columns) per work item, backward and fp32
constexpr int kMaxGroup = 4;            // forward in bf16: two or four
constexpr float kExcluded = -1e30f;     // table values at or below exclude the pair
constexpr int kMaxBuckets = 1024;
constexpr int kMaxChunk = 64;           // union blocks per work item, at most
constexpr float kLog2e = 1.4426950408889634f;
// counters of a call, for rows and for columns: whole groups, items of split
// groups (and partial slots), union entries; then the items that each kernel of
// persistent blocks (forward, delta, rows, columns) has taken
enum { kRowItems = 0, kRowSlots, kRowUnion, kColItems, kColSlots, kColUnion, kTaken, kCounters = 12 };

struct Item {
    int bh, group;
    int start, count;   // its entries of the union list
    int chunk;          // chunk | chunks of the group << 16
    int slot;           // the group's first partial slot (more than one chunk)
};
// Entry of a union list: block index | rows (columns) of the group that hold
// it << 16.
constexpr int kMemberShift = 16;

// One call's problem and workspace, passed to every kernel by value.
struct Call {
    int B, H, N, D, nbr, words, BH;
    int group, groups;              // block rows per item, items' groups per head
    int buckets, cap, chunk;
    int row_items, col_items;       // upper bounds: the grids
    int direct;                     // the blocks make their own lists: no plan, no workspace
    int tc;                         // tcgen05 kernels (bf16, D = 64), group 4
    float scale;
    const float *mask;
    const void *table;              // [buckets][H], element type of q
    const int32_t *bucket;          // [2N-1]
    const int32_t *lists;           // [BH][cap] or null (every block)
    unsigned int *status;
    int expire;                     // test hook: each block's first wait gives up at once
    // workspace
    uint32_t *valid;                // [B][nbr] valid tokens of each block
    float *vec;                     // [H][2*nbr*32] bias; j - i at index j - i + nbr*32
    float *tile;                    // [H][2*nbr] one value for the block offset c - r + nbr - 1:
                                    // a number, -inf (excluded) or +inf (several buckets)
    int *tile_bucket;               // [2*nbr] the bucket, -1 (excluded), -2 (several, each
                                    // in one run), -3 (several)
    int *counters, *bad, *arrive;   // [kCounters], [BH], [2][BH*groups]: cleared by the prepare kernel
    uint32_t *rows;                 // [BH][nbr][words] blocks of each block row
    int *row_list, *col_list;       // union entries
    Item *row_item, *col_item;
    float *row_part, *col_part;     // partial results of split groups
    // backward
    float *rowstat;                 // [BH][nbr][2][32] minus lse, minus delta
    float *bins;                    // [BH*groups][buckets] bias gradient of each group
    void *dtable;                   // [buckets][H], element type of q
    int table_bf16;
};

// The backward's two large kernels, dQ by rows and dK, dV by columns, depend on
// the same earlier ones and not on each other.  The row kernel lets the column
// kernel's blocks start as soon as its own all run, so that they fill the SMs
// that its tail leaves idle (measured with the figures of each column kernel).
//  - The row kernel triggers after its own wait: what the kernels before it
//    wrote is complete when the first column block starts.  The column kernel
//    does not wait there; its fence drops older lines of the SM's L1.
//  - Its last blocks wait for the row kernel at their end and turn its bins into
//    the table's gradient.  So the column kernel ends after the row kernel, and
//    what follows in the stream after both.
__device__ __forceinline__ void rows_begin(bool last_row_kernel) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (last_row_kernel) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
__device__ __forceinline__ void columns_begin() { __threadfence(); }

__device__ __forceinline__ float table_value(const void *table, int bf16, int buckets, int H, int bucket, int h) {
    if (bucket < 0 || bucket >= buckets) return -INFINITY;
    const size_t i = (size_t)bucket * H + h;
    const float x = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(table)[i])
                         : static_cast<const float *>(table)[i];
    return x <= kExcluded ? -INFINITY : x;
}

// The block's work item: split groups' first, then whole groups'; false past
// the last.
__device__ __forceinline__ bool take_item(const Item *items, const int *counters, int capacity, Item *it) {
    const int split = counters[1], i = blockIdx.x;
    if (i >= split + counters[0]) return false;
    *it = items[i < split ? i : capacity - 1 - (i - split)];
    return it->bh >= 0;
}
// The weight that exp2(x * (sc log2 e) + (add - m) log2 e) gives the score m = x *
// sc + add itself: 1 but for the exponent's rounding.  Where a row's reference
// moves to m, its sum is given 1 minus that: the reference then counts exactly 1,
// so that a row of one key has lse m and the backward pass finds its weight to be
// exactly 1 and its dS exactly 0, and no other key's weight is lost.
__device__ __forceinline__ float reference_rest(float x, float sc, float add, float m) {
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(w) : "f"(fmaf(x, sc * kLog2e, (add - m) * kLog2e)));
    return 1.0f - w;
}

__device__ __forceinline__ int item_chunk(const Item &it) { return it.chunk & 0xffff; }
__device__ __forceinline__ int item_chunks(const Item &it) { return it.chunk >> 16; }

// The bucket of relative position d; -1 where there is none.
__device__ __forceinline__ int bucket_at(const int32_t *bucket, int buckets, int N, int d, bool on) {
    if (!on || d <= -N || d >= N) return -1;
    const int b = __ldg(bucket + d + N - 1);
    return b < buckets ? b : -1;
}

// Adds the 32 lanes' sums to bins[]: neighbouring lanes of one bucket b (-1:
// none) are joined by a segmented scan and the end of each run adds.  Runs
// that share a bucket (not where they are known to be distinct) take turns,
// lowest lane first: one order, no atomics.
__device__ __forceinline__ void bin_runs(float sum, int b, float *bins, bool distinct, int lane) {
    const int before = __shfl_up_sync(0xffffffffu, b, 1);
    const unsigned heads = __ballot_sync(0xffffffffu, lane == 0 || b != before);
    const int head = 31 - __clz(heads & (0xffffffffu >> (31 - lane)));
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, sum, s);
        if (lane - s >= head) sum += v;
    }
    const bool add = b >= 0 && (lane == 31 || ((heads >> (lane + 1)) & 1u));
    if (distinct) {
        if (add) bins[b] += sum;
        __syncwarp();
        return;
    }
    const unsigned same = __match_any_sync(0xffffffffu, add ? b : -1 - lane);
    const int turn = add ? __popc(same & ((1u << lane) - 1u)) : 0;
    const int turns = __reduce_max_sync(0xffffffffu, turn);
    for (int i = 0; i <= turns; ++i) {
        if (add && turn == i) bins[b] += sum;
        __syncwarp();
    }
}

// End of a column kernel's block of `warps` warps: dT[b][h] = the groups' bins, a
// warp per value, added in a fixed order (the items' order does not matter).
// Values go to the grid's last blocks, which have the shortest items or none.
__device__ __forceinline__ void table_gradient(const Call &c, int warps) {
    const int lane = threadIdx.x & 31, n = c.B * c.groups;
    const long long values = (long long)c.buckets * c.H;
    long long i = (long long)(gridDim.x - 1 - blockIdx.x) * warps + (threadIdx.x >> 5);
    if (i >= values) return;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    for (; i < values; i += (long long)gridDim.x * warps) {
        const int bucket = (int)(i / c.H), h = (int)(i - (long long)bucket * c.H);
        float sum = 0.0f;
#pragma unroll 4
        for (int k = lane; k < n; k += 32) {
            const int b = k / c.groups, bh = b * c.H + h;
            if (!c.lists || !c.bad[bh]) sum += __ldcg(c.bins + ((size_t)bh * c.groups + (k - b * c.groups)) * c.buckets + bucket);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) {
            if (c.table_bf16) static_cast<__nv_bfloat16 *>(c.dtable)[i] = __float2bfloat16_rn(sum);
            else static_cast<float *>(c.dtable)[i] = sum;
        }
    }
}

// Floats of one work item's partial result, in the accumulators' own layout
// [value][128 threads]: (max, sum, O) forward; dQ and the bins, and dK with
// dV, backward.
inline size_t forward_part_floats(int D, int group) { return 32 * (size_t)group * (D + 16); }
inline size_t row_part_floats(int D, int group, int buckets) { return 32 * (size_t)group * D + (size_t)buckets; }
inline size_t col_part_floats(int D, int group) { return 64 * (size_t)group * D; }

cudaError_t launch_prepare(const Call &c, bool bf16, bool columns, cudaStream_t s, int *launches);
// bf16 over every block of at most kDirectBlocks blocks: one launch that makes
// its own bias window and block list (heads of 32; launch_forward_tc does the
// same for heads of 64).
constexpr int kDirectBlocks = 32;
cudaError_t launch_forward_direct(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                                  cudaStream_t s);
cudaError_t launch_forward_bf16(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                                cudaStream_t s);
cudaError_t launch_forward_f32(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                               cudaStream_t s);
cudaError_t launch_backward_bf16(const Call &c, const void *q, const void *k, const void *v, const float *lse,
                                 const void *dout, void *dq, void *dk, void *dv, cudaStream_t s, int *launches);
cudaError_t launch_backward_f32(const Call &c, const void *q, const void *k, const void *v, const float *lse,
                                const void *dout, void *dq, void *dk, void *dv, cudaStream_t s, int *launches);
cudaError_t launch_forward_tc(const Call &c, const void *q, const void *k, const void *v, void *out, float *lse,
                              cudaStream_t s);
cudaError_t launch_backward_tc(const Call &c, const void *q, const void *k, const void *v, const float *lse,
                               const void *dout, void *dq, void *dk, void *dv, cudaStream_t s, int *launches);

}  // namespace bias

}  // namespace mra
