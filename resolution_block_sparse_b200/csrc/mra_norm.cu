// mra_norm.cu - the norms after and before a block, fused with the block's
// gate and the scaled residual, forward and backward.
//
// Row by row (C columns), with x the residual stream and h the block's output:
//   n = post-norm(h) = (h - m1) r1 * post_w + post_b      (or n = h)
//   x' = a x + g * n                                       (gate row g, or 1)
//   y = pre-norm(x') = (x' - m2) r2 * pre_w + pre_b
// layer norm: m = mean, r = 1 / sqrt(var + eps); RMS norm: m = 0.
//
// Backward, for the gradients dx' and dy; x' and the normalised rows u = (h -
// m1) r1, v = (x' - m2) r2 are formed again from x, h and the statistics,
// which costs no more traffic than reading x' would:
//   t = dx' + r2 (dv - mean(dv) - v mean(dv v)),  dv = dy pre_w
//   dx = a t,  dg = sum over the gate's rows of t n,  dn = t g
//   dh = r1 (du - mean(du) - u mean(du u)),       du = dn post_w
//   dpre_w = sum dy v, dpre_b = sum dy, dpost_w = sum dn u, dpost_b = sum dn
// (RMS norm: without the mean(d) terms).
//
// All arithmetic in fp32.  Bound by HBM: each element is read and written
// once, and what decides is how many bytes are on their way while a row's
// reductions run.  So every row group is persistent and loads its next row
// (16 bytes a lane and load) before it computes the one it has.
// Forward: a row per warp (up to 1024 columns of bf16, 512 of fp32) or per
// block, held in registers, so that mean and variance are two passes over
// registers; the weights wait in shared memory.
// Backward: a block walks a run of rows and a thread owns eight columns (four in
// single elements: 20000 x 333 bf16, step: 103 to 86 us), whose five column sums and weights stay in its registers (the sums in shared
// memory above 4096 columns); each block writes its sums once and a second
// kernel adds them in block order, so equal calls give equal bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "mra.h"
#include "mra_f32x2.cuh"
#include "mra_internal.cuh"

using namespace mra;

namespace {

constexpr int kMaxHidden = 8192;
constexpr int kMaxRows = 0x3fffffff;
// Columns per thread, backward: eight, or four where single elements are loaded
// (rows that do not start on 16 bytes) and the block has room for the threads.
constexpr __host__ __device__ int own_columns(int hidden, int V) { return V == 1 && hidden <= 2048 ? 4 : 8; }
constexpr int kSums = 4;                   // dpost_w, dpost_b, dpre_w, dpre_b
constexpr int kSmemStep = 4096, kSmemSteps = 33;
constexpr int kBackwardThreads = 512;
// Threads of the backward kernel that one SM holds, by the registers they need:
// eight columns in 16-byte pieces of bf16 and four single ones fit 128, and two
// blocks of 320 with less beat one of 512 at every width that 320 threads have
// (1025 to 1280 single columns; 16000 rows, step, one / two: fp32 of 1025 239 / 201
// us, 1153 247 / 210, 1275 251 / 215, bf16 of 1025 224 / 207, 1275 235 / 219; 300
// rows: no difference).  More blocks of 256 with less do not (8000 x 1001 bf16:
// 81 to 88 us).
constexpr __host__ __device__ int resident_threads(int V, int threads) {
    return V == 1 && threads > 256 && threads <= 320 ? 640 : V != 4 ? kBackwardThreads : kBackwardThreads / 2;
}

struct Args {
    const void *x, *h, *gate, *post_w, *post_b, *pre_w, *pre_b;
    void *x_out, *y;
    float *stats;
    int rows, rows_per_gate;
    int hidden;
    int layer, post, pre;
    float a, eps;
    // backward
    const void *dx_out, *dy;
    void *dx, *dh, *dgate;
    float *part;       // [blocks][kSums][hidden], then [blocks][2][hidden] for split gates
    int blocks;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float *p) { *p = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 *p) { *p = __float2bfloat16_rn(v); }

// V elements as they lie in memory (16-byte aligned when V fills 16 bytes)
template <typename T, int V>
struct Raw {
    T e[V];
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 u;
};
template <>
struct Raw<float, 4> {
    uint4 u;
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> fetch(const T *p) {
    return *reinterpret_cast<const Raw<T, V> *>(p);
}

// a row of ones, for a weight or a gate that is not there
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> ones() {
    Raw<T, V> r;
    if constexpr (V == 1) from_f(1.0f, &r.e[0]);
    else r.u = sizeof(T) == 2 ? make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u)
                              : make_uint4(0x3f800000u, 0x3f800000u, 0x3f800000u, 0x3f800000u);
    return r;
}

// Arithmetic on pairs of fp32 (one instruction for two columns: the issue
// rate, not the FMA pipe, is what a row costs beside its bytes).  With V = 1
// only .x counts.
constexpr __host__ __device__ int pairs(int V) { return V > 1 ? V / 2 : 1; }
template <int V>
struct Vec {
    float2 p[pairs(V)];
};
template <int V>
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    if constexpr (V == 1) return make_float2(fmaf(a.x, b.x, c.x), 0.0f);
    else return mra::fma2(a, b, c);
}
template <int V>
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    if constexpr (V == 1) return make_float2(a.x * b.x, 0.0f);
    else return mra::mul2(a, b);
}
template <int V>
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    if constexpr (V == 1) return make_float2(a.x + b.x, 0.0f);
    else return mra::add2(a, b);
}
template <int V>
__device__ __forceinline__ float across(float2 v) {
    return V == 1 ? v.x : v.x + v.y;
}
template <typename T, int V>
__device__ __forceinline__ Vec<V> unpack(const Raw<T, V> &r) {
    Vec<V> v;
    if constexpr (V == 1) {
        v.p[0] = make_float2(to_f(r.e[0]), 0.0f);
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v.p[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
        v.p[0] = make_float2(__uint_as_float(r.u.x), __uint_as_float(r.u.y));
        v.p[1] = make_float2(__uint_as_float(r.u.z), __uint_as_float(r.u.w));
    }
    return v;
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const Vec<V> &v) {
    if constexpr (V == 1) {
        from_f(v.p[0].x, p);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v.p[i].x, v.p[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
    }
}
template <typename T>
__device__ __forceinline__ const T *at(const void *p, long long i) {
    return static_cast<const T *>(p) + i;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
// Sum over the kTpr threads of a row (a warp, or the whole block); `turn`
// alternates the scratch so that one barrier per sum is enough.
template <int kTpr>
__device__ __forceinline__ float row_sum(float v, float (*s)[32], int &turn) {
    v = warp_sum(v);
    if constexpr (kTpr == 32) return v;
    float *t = s[turn];
    turn ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) t[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < kTpr / 32 ? t[lane] : 0.0f);
}

// ---------------------------------------------------------------- forward
constexpr __host__ __device__ int weight_stride(int hidden, int V, bool wide) {
    return V == 8 && wide ? (hidden + 255) / 256 * 256 : hidden;
}
template <typename T, bool kWide>
struct Weight {
    using type = T;
};
template <typename T>
struct Weight<T, true> {
    using type = float;
};

template <typename T, int V, int kPer, int kTpr, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const Args a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ float s_sum[2][32];
    constexpr int P = pairs(V);
    int turn = 0;
    const int C = a.hidden, t = threadIdx.x % kTpr;
    const int stride = gridDim.x * (kThreads / kTpr);
    int row = blockIdx.x * (kThreads / kTpr) + threadIdx.x / kTpr;
    const float inv = 1.0f / (float)C;
    Raw<T, V> rx[kPer] = {}, rh[kPer] = {};
    auto fetch_row = [&](int r) {
        const long long base = (long long)r * C + t * V;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if ((t + kTpr * i) * V < C) {
                rx[i] = fetch<T, V>(at<T>(a.x, base + kTpr * i * V));
                if (a.h) rh[i] = fetch<T, V>(at<T>(a.h, base + kTpr * i * V));
            }
        }
    };
    pdl_wait();
    if (row < a.rows) fetch_row(row);
    // post_w, post_b, pre_w, pre_b, [hidden] each (1 and 0 where absent): as
    // fp32 where a warp holds a row, which saves it the conversions
    using W = typename Weight<T, kTpr == 32>::type;
    constexpr int U = V > 1 && kTpr == 32 ? 4 : V;
    // with V = 8 the two halves of a warp's 256 columns lie apart, so that its
    // lanes read neighbouring 16 bytes
    const int S = weight_stride(C, V, kTpr == 32);
    auto spot = [](int c, int e) {
        return V == 8 ? (c & ~255) + (e >> 2) * 128 + ((c >> 3) & 31) * 4 + (e & 3) : c + e;
    };
    W *const s_w = reinterpret_cast<W *>(s_raw);
    const void *const weight[4] = {a.post_w, a.post_b, a.pre_w, a.pre_b};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k < 2 ? !a.post : !a.pre) continue;
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            Raw<T, V> r = {};
            if (weight[k]) r = fetch<T, V>(at<T>(weight[k], c));
            else if (k % 2 == 0) r = ones<T, V>();
            if constexpr (kTpr == 32) {
                const Vec<V> v = unpack<T, V>(r);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    s_w[k * S + spot(c, 2 * j)] = v.p[j].x;
                    if (V > 1) s_w[k * S + spot(c, 2 * j + 1)] = v.p[j].y;
                }
            } else {
                *reinterpret_cast<Raw<T, V> *>(s_w + k * S + c) = r;
            }
        }
    }
    __syncthreads();
    auto held = [&](int k, int c) -> Vec<V> {
        if constexpr (kTpr == 32) {
            Vec<V> v;
#pragma unroll
            for (int j = 0; j < V / U; ++j) {
                const Vec<U> w = unpack<float, U>(*reinterpret_cast<const Raw<float, U> *>(s_w + k * S + spot(c, U * j)));
#pragma unroll
                for (int e = 0; e < pairs(U); ++e) v.p[pairs(U) * j + e] = w.p[e];
            }
            return v;
        } else {
            return unpack<T, V>(*reinterpret_cast<const Raw<T, V> *>(s_w + k * S + c));
        }
    };
    for (; row < a.rows; row += stride) {
        Vec<V> x[kPer], h[kPer];
        Raw<T, V> rg[kPer];
        const long long gate = a.gate ? (long long)((unsigned)row / (unsigned)a.rows_per_gate) * C : 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = (t + kTpr * i) * V;
            x[i] = unpack<T, V>(rx[i]);
            h[i] = unpack<T, V>(rh[i]);
            rg[i] = ones<T, V>();
            if (a.gate && c < C) rg[i] = fetch<T, V>(at<T>(a.gate, gate + c));
        }
        if (row + stride < a.rows) fetch_row(row + stride);
        const long long base = (long long)row * C;
        // mean and 1 / sqrt(variance + eps) of the row held in v
        auto moments = [&](const Vec<V> (&v)[kPer], float &mean, float &rstd) {
            mean = 0.0f;
            if (a.layer) {
                float2 s = both(0.0f);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
#pragma unroll
                    for (int j = 0; j < P; ++j) s = add2<V>(s, v[i].p[j]);
                mean = row_sum<kTpr>(across<V>(s), s_sum, turn) * inv;
            }
            float2 q = both(0.0f);
            const float2 m = both(-mean);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if ((t + kTpr * i) * V < C) {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const float2 d = add2<V>(v[i].p[j], m);
                        q = fma2<V>(d, d, q);
                    }
                }
            rstd = rsqrtf(row_sum<kTpr>(across<V>(q), s_sum, turn) * inv + a.eps);
        };
        // v = (v - mean) rstd * weight k + weight k + 1
        auto normalise = [&](Vec<V> &v, float mean, float rstd, int k, int c) {
            const float2 m = both(-mean), r = both(rstd);
            const Vec<V> w = held(k, c), o = held(k + 1, c);
#pragma unroll
            for (int j = 0; j < P; ++j)
                v.p[j] = fma2<V>(mul2<V>(add2<V>(v.p[j], m), r), w.p[j], o.p[j]);
        };
        float m1 = 0.0f, r1 = 0.0f, m2 = 0.0f, r2 = 0.0f;
        if (a.post) moments(h, m1, r1);
        const float2 scale = both(a.a);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = (t + kTpr * i) * V;
            if (c >= C) continue;
            if (a.post) normalise(h[i], m1, r1, 0, c);
            const Vec<V> w = unpack<T, V>(rg[i]);
#pragma unroll
            for (int j = 0; j < P; ++j) x[i].p[j] = fma2<V>(h[i].p[j], w.p[j], mul2<V>(scale, x[i].p[j]));
            if (a.x_out) store<T, V>(static_cast<T *>(a.x_out) + base + c, x[i]);
        }
        if (a.pre) {
            moments(x, m2, r2);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = (t + kTpr * i) * V;
                if (c >= C) continue;
                normalise(x[i], m2, r2, 2, c);
                store<T, V>(static_cast<T *>(a.y) + base + c, x[i]);
            }
        }
        if (a.stats && t == 0) {
            const size_t R = a.rows;
            a.stats[row] = m1;
            a.stats[R + row] = r1;
            a.stats[2 * R + row] = m2;
            a.stats[3 * R + row] = r2;
        }
    }
}

template <typename T, int V, int kPer, int kTpr>
cudaError_t forward(const Args &a, cudaStream_t s) {
    constexpr int kThreads = kTpr == 32 ? 128 : kTpr;
    auto *kern = norm_forward_kernel<T, V, kPer, kTpr, kThreads>;
    const int smem = 4 * weight_stride(a.hidden, V, kTpr == 32) * (int)sizeof(typename Weight<T, kTpr == 32>::type);
    // the limit of the longest row that this instance takes, not of this call's:
    // another thread may launch it between the two
    constexpr int kMost = 4 * weight_stride(std::min(kMaxHidden, kPer * kTpr * V), V, kTpr == 32) * (int)sizeof(typename Weight<T, kTpr == 32>::type);
    if (kMost > 40 * 1024) {
        static std::atomic<unsigned long long> done{0};
        const cudaError_t e = allow_shared(kern, kMost, done);
        if (e != cudaSuccess) return e;
    }
    // as many blocks as are resident at once, so that each walks its rows;
    // with fewer rows, no more than there are
    static std::atomic<int> resident[kSmemSteps];
    std::atomic<int> &cached = resident[std::min(smem / kSmemStep, kSmemSteps - 1)];
    int per_sm = cached.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem) != cudaSuccess || per_sm < 1)
            per_sm = 1;
        cached.store(per_sm, std::memory_order_relaxed);
    }
    const int per = kThreads / kTpr, want = (a.rows + per - 1) / per;
    return launch_dependent(kern, dim3(std::min(want, device_sm_count() * per_sm)), dim3(kThreads), smem, s, a);
}
// A warp holds a row of up to 512 (32 lanes x 16) or, in 16-byte loads of
// bf16, 1024 columns; longer rows take a block.  Registers decide how many
// rows are on their way, so there is a variant for each quarter, and one of
// five columns a thread for single columns up to 1280 (16000 rows, eight / five:
// fp32 of 1025 117 / 79 us, 1275 119 / 84; bf16 of 1025 96 / 79, 1275 99 / 84).
template <typename T>
cudaError_t launch_forward(const Args &a, bool vec, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int C = a.hidden;
    if (vec) {
        if (C <= 32 * V) return forward<T, V, 1, 32>(a, s);
        if (C <= 64 * V) return forward<T, V, 2, 32>(a, s);
        if (C <= 96 * V) return forward<T, V, 3, 32>(a, s);
        if (C <= 128 * V) return forward<T, V, 4, 32>(a, s);
        if (C <= 256 * V) return forward<T, V, 2, 128>(a, s);
        if (C <= 512 * V) return forward<T, V, 2, 256>(a, s);
        return forward<T, V, 2, 4096 / V>(a, s);
    }
    if (C <= 128) return forward<T, 1, 4, 32>(a, s);
    if (C <= 512) return forward<T, 1, 16, 32>(a, s);
    if (C <= 1024) return forward<T, 1, 8, 128>(a, s);
    if (C <= 1280) return forward<T, 1, 5, 256>(a, s);
    if (C <= 2048) return forward<T, 1, 8, 256>(a, s);
    return forward<T, 1, 8, 1024>(a, s);
}

// ---------------------------------------------------------------- backward
// Sums of two values over the block in one round: the halves of a warp take
// one value each after the first exchange.
__device__ __forceinline__ float2 block_sum2(float u, float v, float2 (*s)[32], int &turn) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool low = lane < 16;
    float w = (low ? u : v) + __shfl_xor_sync(0xffffffffu, low ? v : u, 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
    if (warps == 1) return make_float2(__shfl_sync(0xffffffffu, w, 0), __shfl_sync(0xffffffffu, w, 16));
    float2 *t = s[turn];
    turn ^= 1;
    if ((lane & 15) == 0) (low ? t[threadIdx.x >> 5].x : t[threadIdx.x >> 5].y) = w;
    __syncthreads();
    u = v = 0.0f;
#pragma unroll 4
    for (int i = 0; i < warps; ++i) {
        u += t[i].x;
        v += t[i].y;
    }
    return make_float2(u, v);
}

// Rows of the backward kernel's blocks: a run of r rows or r + 1.
struct Runs {
    int rows, blocks;
    __host__ __device__ int first(int block) const {
        const int each = rows / blocks, more = rows - each * blocks;
        return each * block + (block < more ? block : more);
    }
    __host__ __device__ int of(int row) const {      // the block that has this row
        const int each = rows / blocks, more = rows - each * blocks;
        return row < more * (each + 1) ? row / (each + 1) : more + (row - more * (each + 1)) / each;
    }
};

__device__ __forceinline__ void copy_16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
// Which kernels stage rows in shared memory.
template <typename T, int V>
constexpr __host__ __device__ bool staged(bool ahead, bool shared) {
    return !ahead && !shared && V * sizeof(T) == 16;
}

// kShared (above 4096 columns, 64 registers a thread): the column sums live in
// shared memory ([5][hidden]) and the weights are read again for every row.
// Up to 4096 columns in 16-byte pieces the next row waits in shared memory (4096
// x 4096 bf16, step: 131.5 to 117 us; above, where the sums are, it gained nothing).
// kAhead (up to 2048 columns): the next row is loaded before this one is
// computed; larger blocks have no registers for it.
template <typename T, int V, int kOwn, int kThreads, bool kShared, bool kAhead, bool kPost, bool kPre>
__global__ void __launch_bounds__(kThreads, std::max(1, resident_threads(V, kThreads) / kThreads))
norm_backward_kernel(const Args a) {
    extern __shared__ float s_acc[];
    __shared__ float2 s_sum[2][32];
    pdl_wait();
    constexpr int kPer = kOwn / V, P = pairs(V);
    int turn = 0;
    const int C = a.hidden, t = threadIdx.x, T0 = blockDim.x;
    const float inv = 1.0f / (float)C;
    const Runs runs{a.rows, a.blocks};
    const int r0 = runs.first(blockIdx.x), r1 = runs.first(blockIdx.x + 1);
    const size_t R = a.rows;
    // sums: 0 dpost_w, 1 dpost_b, 2 dpre_w, 3 dpre_b, 4 dgate
    Vec<V> acc[kShared ? 1 : 5][kPer] = {};
    auto shared_at = [&](int k, int i, int j, int e) -> float & {
        return s_acc[(size_t)k * C + (t + T0 * i) * V + 2 * j + e];
    };
    // columns past the row's end hold zeros throughout: no branch over them
    auto in = [&](int i) { return (t + T0 * i) * V < C; };
    auto add = [&](int k, int i, int j, float2 u, float2 v) {      // += u v
        if constexpr (kShared) {
            if (in(i)) {
                shared_at(k, i, j, 0) += u.x * v.x;
                if (V > 1) shared_at(k, i, j, 1) += u.y * v.y;
            }
        } else {
            acc[k][i].p[j] = fma2<V>(u, v, acc[k][i].p[j]);
        }
    };
    auto get = [&](int k, int i, int j, int e) -> float {
        if constexpr (kShared) return shared_at(k, i, j, e);
        else return e ? acc[k][i].p[j].y : acc[k][i].p[j].x;
    };
    auto clear = [&](int k) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if constexpr (kShared) {
                    if ((t + T0 * i) * V < C) {
                        shared_at(k, i, j, 0) = 0.0f;
                        if (V > 1) shared_at(k, i, j, 1) = 0.0f;
                    }
                } else {
                    acc[k][i].p[j] = both(0.0f);
                }
            }
    };
#pragma unroll
    for (int k = 0; k < 5; ++k) clear(k);

    // this thread's weights and gate row (1 and 0 where absent), and the next
    // row of each tensor (0 where absent)
    Raw<T, V> w_post[kPer], b_post[kPer] = {}, w_pre[kPer], rg[kPer], rx[kPer] = {}, rh[kPer] = {}, ry[kPer] = {},
        ro[kPer] = {};
    float st[4] = {};
    auto fetch_row = [&](int row) {
        const long long base = (long long)row * C + t * V;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (!in(i)) continue;
            const long long e = base + T0 * i * V;
            if (kPre) rx[i] = fetch<T, V>(at<T>(a.x, e));
            if (a.h) rh[i] = fetch<T, V>(at<T>(a.h, e));
            if (kPre) ry[i] = fetch<T, V>(at<T>(a.dy, e));
            if (a.dx_out) ro[i] = fetch<T, V>(at<T>(a.dx_out, e));
        }
        if (kPost) {
            st[0] = a.stats[row];
            st[1] = a.stats[R + row];
        }
        if (kPre) {
            st[2] = a.stats[2 * R + row];
            st[3] = a.stats[3 * R + row];
        }
    };
    // kStaged: the next row waits in one of two buffers in shared memory, each
    // thread's own pieces
    constexpr bool kStaged = staged<T, V>(kAhead, kShared);
    uint4 *const s_row = reinterpret_cast<uint4 *>(s_acc);
    float next_st[4] = {};
    auto piece = [&](int buf, int k, int i) -> uint4 * { return s_row + ((buf * 4 + k) * kPer + i) * T0 + t; };
    auto stage = [&](int row, int buf) {
        if constexpr (kStaged) {
            const long long base = (long long)row * C + t * V;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (!in(i)) continue;
                const long long e = base + T0 * i * V;
                if (kPre) copy_16(piece(buf, 0, i), at<T>(a.x, e));
                if (a.h) copy_16(piece(buf, 1, i), at<T>(a.h, e));
                if (kPre) copy_16(piece(buf, 2, i), at<T>(a.dy, e));
                if (a.dx_out) copy_16(piece(buf, 3, i), at<T>(a.dx_out, e));
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < 2 ? kPost : kPre) next_st[k] = a.stats[k * R + row];
        }
    };
    auto unstage = [&](int buf) {
        if constexpr (kStaged) {
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (!in(i)) continue;
                if (kPre) rx[i].u = *piece(buf, 0, i);
                if (a.h) rh[i].u = *piece(buf, 1, i);
                if (kPre) ry[i].u = *piece(buf, 2, i);
                if (a.dx_out) ro[i].u = *piece(buf, 3, i);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) st[k] = next_st[k];
        }
    };
    // gate row in rg, and the first row that needs the next one
    int gate_row = -1, gate_end = a.gate ? 0 : 0x7fffffff;
    auto fetch_gate = [&](int row) {
        if (row < gate_end) return;
        gate_row = row / a.rows_per_gate;
        gate_end = min((long long)a.rows, (gate_row + 1LL) * a.rows_per_gate);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (in(i)) rg[i] = fetch<T, V>(at<T>(a.gate, (long long)gate_row * C + (t + T0 * i) * V));
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = (t + T0 * i) * V;
        w_post[i] = w_pre[i] = rg[i] = ones<T, V>();
        if (!in(i) || kShared) continue;
        if (a.post_w) w_post[i] = fetch<T, V>(at<T>(a.post_w, c));
        if (a.post_b) b_post[i] = fetch<T, V>(at<T>(a.post_b, c));
        if (a.pre_w) w_pre[i] = fetch<T, V>(at<T>(a.pre_w, c));
    }
    auto weight = [&](const Raw<T, V> &held, const void *p, int i) -> Vec<V> {
        Raw<T, V> r = held;
        if (kShared && p && in(i)) r = fetch<T, V>(at<T>(p, (t + T0 * i) * V));
        return unpack<T, V>(r);
    };
    // the block's output after its norm, from the normalised row
    auto output = [&](Vec<V> f, int i) -> Vec<V> {
        if (kPost) {
            const Vec<V> w = weight(w_post[i], a.post_w, i), o = weight(b_post[i], a.post_b, i);
#pragma unroll
            for (int j = 0; j < P; ++j) f.p[j] = fma2<V>(f.p[j], w.p[j], o.p[j]);
        }
        return f;
    };
    if (kAhead) {
        fetch_row(r0);
        fetch_gate(r0);
    }
    if (kStaged && r0 < r1) stage(r0, 0);
    const float2 scale = both(a.a), one = both(1.0f);
    for (int row = r0; row < r1; ++row) {
        const int buf = (row - r0) & 1;
        if (!kAhead) {
            if (kStaged) {
                unstage(buf);
                if (row + 1 < r1) stage(row + 1, buf ^ 1);
            } else {
                fetch_row(row);
            }
            fetch_gate(row);
        }
        const long long base = (long long)row * C;
        const float q1 = st[1], q2 = st[3];
        Vec<V> u[kPer], n[kPer], v[kPer], d[kPer];   // u, gate (then dn), v, dv (then t)
        Raw<T, V> go[kPer];
        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            go[i] = ro[i];
            u[i] = unpack<T, V>(rh[i]);
            n[i] = unpack<T, V>(rg[i]);
            if (kPost) {
                const float2 r = both(q1), m = both(-st[0]);
#pragma unroll
                for (int j = 0; j < P; ++j) u[i].p[j] = mul2<V>(add2<V>(u[i].p[j], m), r);
            }
            if (kPre) {
                // v from n, then dv
                const Vec<V> x = unpack<T, V>(rx[i]), f = output(u[i], i), w = weight(w_pre[i], a.pre_w, i);
                d[i] = unpack<T, V>(ry[i]);
                const float2 r = both(q2), m = both(-st[2]);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 z = fma2<V>(f.p[j], n[i].p[j], mul2<V>(scale, x.p[j]));
                    v[i].p[j] = mul2<V>(add2<V>(z, m), r);
                    add(2, i, j, d[i].p[j], v[i].p[j]);
                    add(3, i, j, d[i].p[j], one);
                    d[i].p[j] = mul2<V>(d[i].p[j], w.p[j]);
                    s1 = add2<V>(s1, d[i].p[j]);
                    s2 = fma2<V>(d[i].p[j], v[i].p[j], s2);
                }
            }
        }
        const int this_gate = gate_row, this_end = gate_end;
        if (kAhead && row + 1 < r1) {
            fetch_row(row + 1);
            fetch_gate(row + 1);
        }
        if (kPre) {
            const float2 s = block_sum2(across<V>(s1), across<V>(s2), s_sum, turn);
            s1 = both(a.layer ? -s.x * inv : 0.0f);
            s2 = both(-s.y * inv);
        }
        float2 t1 = both(0.0f), t2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            Vec<V> w = unpack<T, V>(go[i]);
            if (kPre) {
                // r2 (dv - mean(dv) - v mean(dv v)), and dx'
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 z = fma2<V>(fma2<V>(v[i].p[j], s2, add2<V>(d[i].p[j], s1)), both(q2), w.p[j]);
                    d[i].p[j] = in(i) ? z : both(0.0f);
                }
            } else {
                d[i] = w;
            }
#pragma unroll
            for (int j = 0; j < P; ++j) w.p[j] = mul2<V>(scale, d[i].p[j]);
            if (in(i)) store<T, V>(static_cast<T *>(a.dx) + base + (t + T0 * i) * V, w);
            if (a.dgate) {
                w = output(u[i], i);
#pragma unroll
                for (int j = 0; j < P; ++j) add(4, i, j, d[i].p[j], w.p[j]);
            }
            if (kPost) w = weight(w_post[i], a.post_w, i);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                n[i].p[j] = mul2<V>(n[i].p[j], d[i].p[j]);      // dn
                if (kPost) {
                    add(0, i, j, n[i].p[j], u[i].p[j]);
                    add(1, i, j, n[i].p[j], one);
                    n[i].p[j] = mul2<V>(n[i].p[j], w.p[j]);     // du
                    t1 = add2<V>(t1, n[i].p[j]);
                    t2 = fma2<V>(n[i].p[j], u[i].p[j], t2);
                }
            }
        }
        if (kPost) {
            const float2 s = block_sum2(across<V>(t1), across<V>(t2), s_sum, turn);
            t1 = both(a.layer ? -s.x * inv : 0.0f);
            t2 = both(-s.y * inv);
        }
        if (a.h) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (kPost) {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        n[i].p[j] = mul2<V>(fma2<V>(u[i].p[j], t2, add2<V>(n[i].p[j], t1)), both(q1));
                }
                if (in(i)) store<T, V>(static_cast<T *>(a.dh) + base + (t + T0 * i) * V, n[i]);
            }
        }
        // the gate row ends here: written if all its rows are this block's,
        // left to the second kernel otherwise (slot 0: it began before this
        // block, slot 1: it goes on after it)
        if (a.dgate && (row + 1 == r1 || row + 1 == this_end)) {
            const bool before = (long long)this_gate * a.rows_per_gate < r0;
            const bool whole = !before && this_end <= r1;
            float *slot = a.part + ((size_t)a.blocks * kSums + (size_t)blockIdx.x * 2 + (before ? 0 : 1)) * C;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = (t + T0 * i) * V;
                if (c >= C) continue;
                Vec<V> w;
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    w.p[j] = make_float2(get(4, i, j, 0), V > 1 ? get(4, i, j, 1) : 0.0f);
                    if (!whole) {
                        slot[c + 2 * j] = w.p[j].x;
                        if (V > 1) slot[c + 2 * j + 1] = w.p[j].y;
                    }
                }
                if (whole) store<T, V>(static_cast<T *>(a.dgate) + (long long)this_gate * C + c, w);
            }
            clear(4);
        }
    }
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        if (k < 2 ? !kPost : !kPre) continue;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = (t + T0 * i) * V;
            if (c >= C) continue;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                float *p = a.part + ((size_t)blockIdx.x * kSums + k) * C + c + 2 * j;
                p[0] = get(k, i, j, 0);
                if (V > 1) p[1] = get(k, i, j, 1);
            }
        }
    }
}

constexpr int kRuns = 32;
struct Targets {
    void *d[kSums];
};

// Column sums of the blocks' partial results, 32 columns a block, in block
// order (32 interleaved runs, then run by run).  y < 4: the weights'
// gradients.  Above: the gate rows that several blocks share, by gate row
// (by_gate: there are fewer of those than blocks) or by the block whose first
// row splits one (the first such block of a gate row does it).
template <typename T>
__global__ void __launch_bounds__(32 * kRuns) norm_reduce_kernel(const Args a, const Targets w, const int by_gate) {
    __shared__ float s_run[kRuns][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, C = a.hidden;
    const Runs runs{a.rows, a.blocks};
    int from = 0, to = a.blocks;
    const float *base = a.part;
    size_t stride = (size_t)kSums * C;
    T *dst;
    if (blockIdx.y < kSums) {
        if (!w.d[blockIdx.y]) return;
        base += (size_t)blockIdx.y * C;
        dst = static_cast<T *>(w.d[blockIdx.y]);
    } else {
        const int k = blockIdx.y - kSums;
        const int g = by_gate ? k : runs.first(k + 1) / a.rows_per_gate;
        const long long g0 = (long long)g * a.rows_per_gate, g1 = min((long long)a.rows, g0 + a.rows_per_gate);
        from = runs.of((int)g0);
        to = runs.of((int)g1 - 1) + 1;
        if (to - from < 2 || (!by_gate && k != from)) return;      // one block's, or another's turn
        base += (size_t)a.blocks * kSums * C;
        stride = 2 * (size_t)C;
        dst = static_cast<T *>(a.dgate) + (long long)g * C;
    }
    float sum = 0.0f;
    if (c < C) {
        // six loads on their way at a time (100000 x 64 bf16, step: 118 to 111 us)
        constexpr int kAtOnce = 6;
        const float *p = base + c;
        for (int k = from + run; k < to; k += kRuns * kAtOnce) {
            float v[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int at = k + j * kRuns;
                v[j] = at < to ? __ldcg(p + at * stride + (blockIdx.y >= kSums && at == from ? C : 0)) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) sum += v[j];
        }
    }
    s_run[run][lane] = sum;
    __syncthreads();
    if (run == 0 && c < C) {
        for (int k = 1; k < kRuns; ++k) sum += s_run[k][lane];
        from_f(sum, dst + c);
    }
}

int backward_threads(int hidden, int V) {
    const int own = own_columns(hidden, V);
    return ((hidden + own - 1) / own + 31) / 32 * 32;
}
// Blocks of the backward kernel: a run of at least 8 rows each (more blocks cost
// the second kernel more than they save: 2000 x 256 bf16, step: 16 us, with 2 rows
// each 21) or 2 until every SM has one (600 x 8192: 146 to 114 us, 100 x 768: 17 to
// 11), at most what the GPU holds at once.
int backward_blocks(long long rows, int hidden, int V) {
    const int resident = std::max(1, resident_threads(V, backward_threads(hidden, V)) / backward_threads(hidden, V));
    const long long sms = device_sm_count(), want = std::max((rows + 7) / 8, std::min((rows + 1) / 2, sms));
    return (int)std::max(1LL, std::min(want, sms * resident));
}

template <typename T, int V, int kOwn, int kThreads, bool kShared, bool kAhead, bool kPost, bool kPre>
cudaError_t backward(const Args &a, cudaStream_t s) {
    auto *kernel = norm_backward_kernel<T, V, kOwn, kThreads, kShared, kAhead, kPost, kPre>;
    const size_t smem = kShared ? 5 * sizeof(float) * (size_t)a.hidden
                        : staged<T, V>(kAhead, kShared) ? (size_t)2 * 4 * (kOwn / V) * 16 * backward_threads(a.hidden, V) : 0;
    constexpr size_t kMost = kShared ? 5 * sizeof(float) * (size_t)kMaxHidden
                             : staged<T, V>(kAhead, kShared) ? (size_t)2 * 4 * (kOwn / V) * 16 * kThreads : 0;
    if (kMost > 40 * 1024) {
        static std::atomic<unsigned long long> done{0};
        const cudaError_t e = allow_shared(kernel, kMost, done);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kernel, dim3(a.blocks), dim3(backward_threads(a.hidden, V)), smem, s, a);
}
template <typename T, int V, bool kPost, bool kPre>
cudaError_t backward_by_size(const Args &a, cudaStream_t s) {
    constexpr int kOwn = own_columns(2048, V);
    if (V == 1 && a.hidden <= 1024) return backward<T, V, kOwn, 256, false, true, kPost, kPre>(a, s);
    if (V == 1 && a.hidden <= 1280) return backward<T, V, kOwn, 320, false, true, kPost, kPre>(a, s);
    if (a.hidden <= 2048) return backward<T, V, kOwn, 2048 / kOwn, false, true, kPost, kPre>(a, s);
    if (a.hidden <= 4096) return backward<T, V, 8, 512, false, false, kPost, kPre>(a, s);
    return backward<T, V, 8, 1024, true, false, kPost, kPre>(a, s);
}
template <typename T, int V>
cudaError_t backward_by_norms(const Args &a, cudaStream_t s) {
    if (a.post && a.pre) return backward_by_size<T, V, true, true>(a, s);
    if (a.post) return backward_by_size<T, V, true, false>(a, s);
    if (a.pre) return backward_by_size<T, V, false, true>(a, s);
    return backward_by_size<T, V, false, false>(a, s);
}
template <typename T>
cudaError_t launch_backward(const Args &a, const Targets &w, bool vec, cudaStream_t s) {
    cudaError_t e = vec ? backward_by_norms<T, 16 / sizeof(T)>(a, s) : backward_by_norms<T, 1>(a, s);
    if (e != cudaSuccess) return e;
    const bool split = a.dgate && a.rows_per_gate > 1;
    if (!split && !w.d[0] && !w.d[1] && !w.d[2] && !w.d[3]) return cudaSuccess;
    const int gates = split ? (a.rows + a.rows_per_gate - 1) / a.rows_per_gate : 0;
    const int by_gate = gates < a.blocks ? 1 : 0;
    const dim3 grid((a.hidden + 31) / 32, kSums + (by_gate ? gates : split ? a.blocks - 1 : 0));
    return launch_dependent(norm_reduce_kernel<T>, grid, dim3(32 * kRuns), 0, s, a, w, by_gate);
}

bool off(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

// Checks shared by both directions; vec: every row and weight starts on 16
// bytes, so that the kernels move 16 bytes at a time.
int check(const Args &a, int norm, int norms, int dtype, const void *const *row_tensors, int n_rows,
          const void *const *weights, int n_weights, bool *vec) {
    if (a.rows < 0 || a.hidden < 1 || a.rows_per_gate < (a.gate ? 1 : 0)) return MRA_ERR_INVALID_ARG;
    if (norm != MRA_LAYER_NORM && norm != MRA_RMS_NORM) return MRA_ERR_INVALID_ARG;
    if (norms & ~(MRA_NORM_POST | MRA_NORM_PRE)) return MRA_ERR_INVALID_ARG;
    if (dtype != MRA_DTYPE_BF16 && dtype != MRA_DTYPE_F32) return MRA_ERR_INVALID_ARG;
    if (a.hidden > kMaxHidden || a.rows > kMaxRows) return MRA_ERR_UNSUPPORTED;
    if (!std::isfinite(a.a) || !(a.eps >= 0.0f) || !std::isfinite(a.eps)) return MRA_ERR_INVALID_ARG;
    // a part that is not there has no weights
    if (!(norms & MRA_NORM_POST) && (a.post_w || a.post_b)) return MRA_ERR_INVALID_ARG;
    if (!(norms & MRA_NORM_PRE) && (a.pre_w || a.pre_b)) return MRA_ERR_INVALID_ARG;
    const uintptr_t e = dtype == MRA_DTYPE_BF16 ? 2 : 4;
    bool v = (size_t)a.hidden * e % 16 == 0;
    for (int i = 0; i < n_rows; ++i) {
        if (off(row_tensors[i], e)) return MRA_ERR_INVALID_ARG;
        v = v && !off(row_tensors[i], 16);
    }
    for (int i = 0; i < n_weights; ++i) {
        if (off(weights[i], e)) return MRA_ERR_INVALID_ARG;
        v = v && !off(weights[i], 16);
    }
    *vec = v;
    return MRA_OK;
}

size_t part_floats(int blocks, int hidden) { return (size_t)blocks * (kSums + 2) * hidden; }

}  // namespace

extern "C" {

size_t mra_residual_norm_workspace(long long rows, int hidden) {
    if (rows < 0 || rows > kMaxRows || hidden < 1 || hidden > kMaxHidden) return 0;
    // the form of the type and alignment with the most blocks
    return 4 * part_floats(std::max(backward_blocks(rows, hidden, 8), backward_blocks(rows, hidden, 1)), hidden);
}

int mra_residual_norm_fwd(const void *x, const void *h, const void *gate, long long rows_per_gate, const void *post_w,
                          const void *post_b, const void *pre_w, const void *pre_b, void *x_out, void *y, float *stats,
                          long long rows, int hidden, int norm, int norms, float residual_scale, float eps, int dtype,
                          cudaStream_t stream) {
    Args a{};
    a.x = x;
    a.h = h;
    a.gate = gate;
    a.rows_per_gate = gate ? (int)std::max<long long>(-1, std::min<long long>(rows_per_gate, kMaxRows)) : 1;
    a.post_w = post_w;
    a.post_b = post_b;
    a.pre_w = pre_w;
    a.pre_b = pre_b;
    a.x_out = x_out;
    a.y = y;
    a.stats = stats;
    a.rows = (int)std::max<long long>(-1, std::min<long long>(rows, kMaxRows + 1LL));
    a.hidden = hidden;
    a.layer = norm == MRA_LAYER_NORM;
    a.post = (norms & MRA_NORM_POST) != 0;
    a.pre = (norms & MRA_NORM_PRE) != 0;
    a.a = residual_scale;
    a.eps = eps;
    const void *row_tensors[] = {x, h, x_out, y}, *weights[] = {gate, post_w, post_b, pre_w, pre_b};
    bool vec;
    const int rc = check(a, norm, norms, dtype, row_tensors, 4, weights, 5, &vec);
    if (rc != MRA_OK) return rc;
    if (off(stats, 4)) return MRA_ERR_INVALID_ARG;
    if (rows == 0) return MRA_OK;
    if (!h && (a.post || gate)) return MRA_ERR_INVALID_ARG;
    if (!x || (a.pre ? !y : y != nullptr) || (!x_out && !y)) return MRA_ERR_INVALID_ARG;
    const cudaError_t e = dtype == MRA_DTYPE_BF16 ? launch_forward<__nv_bfloat16>(a, vec, stream)
                                                  : launch_forward<float>(a, vec, stream);
    if (e != cudaSuccess) return MRA_ERR_CUDA;
    set_last_launches(1);
    return MRA_OK;
}

int mra_residual_norm_bwd(const void *x, const void *h, const void *gate, long long rows_per_gate, const void *post_w,
                          const void *post_b, const void *pre_w, const void *pre_b, const float *stats,
                          const void *dx_out, const void *dy, void *dx, void *dh, void *dgate, void *dpost_w,
                          void *dpost_b, void *dpre_w, void *dpre_b, long long rows, int hidden, int norm, int norms,
                          float residual_scale, float eps, int dtype, void *workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
    Args a{};
    a.x = x;
    a.h = h;
    a.gate = gate;
    a.rows_per_gate = gate ? (int)std::max<long long>(-1, std::min<long long>(rows_per_gate, kMaxRows)) : 1;
    a.post_w = post_w;
    a.post_b = post_b;
    a.pre_w = pre_w;
    a.pre_b = pre_b;
    a.stats = const_cast<float *>(stats);
    a.rows = (int)std::max<long long>(-1, std::min<long long>(rows, kMaxRows + 1LL));
    a.hidden = hidden;
    a.layer = norm == MRA_LAYER_NORM;
    a.post = (norms & MRA_NORM_POST) != 0;
    a.pre = (norms & MRA_NORM_PRE) != 0;
    a.a = residual_scale;
    a.eps = eps;
    a.dx_out = dx_out;
    a.dy = dy;
    a.dx = dx;
    a.dh = dh;
    a.dgate = dgate;
    a.part = static_cast<float *>(workspace);
    const Targets w{{dpost_w, dpost_b, dpre_w, dpre_b}};
    const void *row_tensors[] = {x, h, dx_out, dy, dx, dh},
               *weights[] = {gate, post_w, post_b, pre_w, pre_b, dgate, dpost_w, dpost_b, dpre_w, dpre_b};
    bool vec;
    const int rc = check(a, norm, norms, dtype, row_tensors, 6, weights, 10, &vec);
    if (rc != MRA_OK) return rc;
    if (off(stats, 4) || off(workspace, 16) || (dgate && !gate)) return MRA_ERR_INVALID_ARG;
    if ((!a.post && (dpost_w || dpost_b)) || (!a.pre && (dpre_w || dpre_b))) return MRA_ERR_INVALID_ARG;
    if (rows == 0) {
        // no row: the weights' gradients are empty sums
        const size_t bytes = (size_t)hidden * (dtype == MRA_DTYPE_BF16 ? 2 : 4);
        for (void *d : w.d)
            if (d && cudaMemsetAsync(d, 0, bytes, stream) != cudaSuccess) return MRA_ERR_CUDA;
        return MRA_OK;
    }
    if (!h && (a.post || gate)) return MRA_ERR_INVALID_ARG;
    if (!x || !dx || (h ? !dh : dh != nullptr) || (a.pre ? !dy : dy != nullptr)) return MRA_ERR_INVALID_ARG;
    if ((!dx_out && !dy) || ((a.post || a.pre) && !stats) || !workspace) return MRA_ERR_INVALID_ARG;
    if (workspace_bytes < mra_residual_norm_workspace(rows, hidden)) return MRA_ERR_TOO_LARGE;
    a.blocks = backward_blocks(rows, hidden, vec ? (dtype == MRA_DTYPE_BF16 ? 8 : 4) : 1);
    const cudaError_t e = dtype == MRA_DTYPE_BF16 ? launch_backward<__nv_bfloat16>(a, w, vec, stream)
                                                  : launch_backward<float>(a, w, vec, stream);
    if (e != cudaSuccess) return MRA_ERR_CUDA;
    set_last_launches(2);
    return MRA_OK;
}

}  // extern "C"
