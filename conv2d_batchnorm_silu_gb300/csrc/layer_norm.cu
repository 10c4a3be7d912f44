// layer_norm.cu -- layer norm over the channels of each row, its gradient, and
// the quantisation of rows to 8-bit integers.
//
//   mean = sum_c x / C,  var = sum_c (x - mean)^2 / C,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) * rstd * gamma + beta
//
// and for the gradient, with h = (x - mean) * rstd and g = dy * gamma,
//
//   dx = rstd * (g - mean_c(g) - h * mean_c(g * h)),
//   dgamma = sum_rows dy * h,  dbeta = sum_rows dy.
//
// Statistics, sums and parameters are fp32 whatever the activations' type; the
// variance is summed around the mean (a second pass over the row), so rows far
// from zero lose nothing to cancellation.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cbs_internal.h"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

// A row whose largest magnitude is below this is quantised as if it were this: 127 / most
// stays finite, and a row of zeros needs no case of its own.
constexpr float kTiniest = 7.8886090522101181e-31f;  // 2^-100

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_float(float v, float *out) { *out = v; }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16 *out) { *out = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_float(float v, __half *out) { *out = __float2half_rn(v); }

template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float *scratch)
{
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < THREADS / 32; ++i) s += scratch[i];
    __syncthreads();
    return s;
}

template <int THREADS>
__device__ __forceinline__ unsigned block_max(unsigned v, unsigned *scratch)
{
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    unsigned s = 0;
    for (int i = 0; i < THREADS / 32; ++i) s = max(s, scratch[i]);
    __syncthreads();
    return s;
}

// The bits of |v|: ordered like the magnitudes, with NaN above infinity, so that a NaN
// anywhere in a row becomes the row's scale.
__device__ __forceinline__ unsigned magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Most magnitude of a row -> its scale, and the factor that takes values to [-127, 127].
// The values of a row that holds a NaN or an infinity all become 0 (conversion of NaN gives
// 0), with a scale that is not finite: what is computed from such a row is NaN.
__device__ __forceinline__ float row_scale_of(unsigned most_bits, float *inv)
{
    float most = __uint_as_float(most_bits);
    if (most < kTiniest) most = kTiniest;
    *inv = 127.0f / most;
    return most / 127.0f;
}

constexpr int kWideThreads = 256;

struct NormArgs {
    const void *x;
    void *y;
    int8_t *q;
    float *row_scale;
    float *stats;
    const float *gamma;
    const float *beta;
    long long x_stride, y_stride, q_stride;
    long long rows;
    int c;
    float eps;
    int normalise;
};

// One row per block at a time, read once for each sum it needs: any width, alignment and stride.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const NormArgs a)
{
    __shared__ float scratch[kWideThreads / 32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
        float mean = 0.0f, rstd = 1.0f;
        if (a.normalise) {
            float s = 0.0f;
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) s += to_float(x[i]);
            mean = block_sum<kWideThreads>(s, scratch) / (float)a.c;
            s = 0.0f;
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) {
                const float d = to_float(x[i]) - mean;
                s = fmaf(d, d, s);
            }
            rstd = 1.0f / sqrtf(block_sum<kWideThreads>(s, scratch) / (float)a.c + a.eps);
            if (a.stats && threadIdx.x == 0) {
                a.stats[r] = mean;
                a.stats[a.rows + r] = rstd;
            }
        }
        auto value = [&](int i) {
            const float v = to_float(x[i]);
            if (!a.normalise) return v;
            const float h = (v - mean) * rstd;
            return fmaf(h, a.gamma ? a.gamma[i] : 1.0f, a.beta ? a.beta[i] : 0.0f);
        };
        if (a.q) {
            unsigned most = 0;
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) most = max(most, magnitude_bits(value(i)));
            float inv;
            const float scale = row_scale_of(block_max<kWideThreads>(most, reinterpret_cast<unsigned *>(scratch)), &inv);
            if (threadIdx.x == 0) a.row_scale[r] = scale;
            int8_t *q = a.q + r * a.q_stride;
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) q[i] = (int8_t)__float2int_rn(value(i) * inv);
        } else {
            T *y = static_cast<T *>(a.y) + r * a.y_stride;
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) from_float(value(i), y + i);
        }
    }
}

struct GradArgs {
    const void *dy, *x;
    void *dx;
    const float *gamma;
    const float *stats;
    float *dgamma, *dbeta;
    float *partial;
    long long dy_stride, x_stride, dx_stride;
    long long rows;
    int c;
    int partial_rows;
};

// dx, one row per block at a time.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const GradArgs a)
{
    __shared__ float scratch[kWideThreads / 32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
        T *dx = static_cast<T *>(a.dx) + r * a.dx_stride;
        const float mean = a.stats[r], rstd = a.stats[a.rows + r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int i = threadIdx.x; i < a.c; i += kWideThreads) {
            const float g = to_float(dy[i]) * (a.gamma ? a.gamma[i] : 1.0f);
            s1 += g;
            s2 = fmaf(g, (to_float(x[i]) - mean) * rstd, s2);
        }
        s1 = block_sum<kWideThreads>(s1, scratch) / (float)a.c;
        s2 = block_sum<kWideThreads>(s2, scratch) / (float)a.c;
        for (int i = threadIdx.x; i < a.c; i += kWideThreads) {
            const float g = to_float(dy[i]) * (a.gamma ? a.gamma[i] : 1.0f);
            const float h = (to_float(x[i]) - mean) * rstd;
            from_float(rstd * (g - s1 - h * s2), dx + i);
        }
    }
}

// Partial sums of dy * h and dy over every partial_rows-th row, one column per thread.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_grad_columns_kernel(const GradArgs a)
{
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int i = blockIdx.x * kWideThreads + threadIdx.x;
    if (i >= a.c) return;
    float sg = 0.0f, sb = 0.0f;
    for (long long r = blockIdx.y; r < a.rows; r += a.partial_rows) {
        const float d = to_float(static_cast<const T *>(a.dy)[r * a.dy_stride + i]);
        const float h = (to_float(static_cast<const T *>(a.x)[r * a.x_stride + i]) - a.stats[r]) * a.stats[a.rows + r];
        sg = fmaf(d, h, sg);
        sb += d;
    }
    a.partial[(long long)blockIdx.y * 2 * a.c + i] = sg;
    a.partial[(long long)blockIdx.y * 2 * a.c + a.c + i] = sb;
}

// Column sums of partial[partial_rows][2c] in a fixed order: 32 columns per block, eight
// runs of rows summed side by side and joined in shared memory.
constexpr int kJoinRuns = 8;
__global__ void __launch_bounds__(32 * kJoinRuns) norm_grad_join_kernel(const GradArgs a)
{
    __shared__ float part[kJoinRuns][32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int i = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (i < 2 * a.c)
        for (int r = threadIdx.y; r < a.partial_rows; r += kJoinRuns) s += a.partial[(long long)r * 2 * a.c + i];
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && i < 2 * a.c) {
        for (int t = 1; t < kJoinRuns; ++t) s += part[t][threadIdx.x];
        if (i < a.c)
            a.dgamma[i] = s;
        else
            a.dbeta[i - a.c] = s;
    }
}

// ------------------------------------------------------------------ rows held in registers
// A row stays in the registers of TPR threads, NI vectors of V elements each, from its one
// load to its one store; sums go through warp shuffles and, above a warp, shared memory.
// V = 16 bytes' worth where every pointer, row distance and the width allow it, else 1.
template <typename T, int V>
struct Vec;
template <int V>
struct ParamOf { using type = __half; };  // any type whose vector has V elements
template <>
struct ParamOf<4> { using type = float; };
template <typename T>
struct Vec<T, 1> {
    T raw;
    __device__ __forceinline__ void load(const T *p) { raw = __ldcs(p); }
    __device__ __forceinline__ void get(float *v) const { v[0] = to_float(raw); }
    static __device__ __forceinline__ void store(T *p, const float *v) { from_float(v[0], p); }
    static __device__ __forceinline__ void store_q(int8_t *p, const int *q) { *p = (int8_t)q[0]; }
    static __device__ __forceinline__ void load_param(const float *p, float *v) { v[0] = __ldg(p); }
};
template <>
struct Vec<float, 4> {
    float4 raw;
    __device__ __forceinline__ void load(const float *p) { raw = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void from(const uint4 &w)
    {
        raw = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
    }
    __device__ __forceinline__ void get(float *v) const
    {
        v[0] = raw.x;
        v[1] = raw.y;
        v[2] = raw.z;
        v[3] = raw.w;
    }
    static __device__ __forceinline__ void store(float *p, const float *v)
    {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
    static __device__ __forceinline__ void store_q(int8_t *p, const int *q)
    {
        const uint32_t lo = __byte_perm(q[0], q[1], 0x0040), hi = __byte_perm(q[2], q[3], 0x0040);
        *reinterpret_cast<uint32_t *>(p) = __byte_perm(lo, hi, 0x5410);
    }
    static __device__ __forceinline__ void load_param(const float *p, float *v)
    {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    }
};
__device__ __forceinline__ float2 unpack(uint32_t w, __nv_bfloat16)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack(uint32_t w, __half)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __half)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T>
struct Vec<T, 8> {
    uint4 raw;
    __device__ __forceinline__ void load(const T *p) { raw = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void from(const uint4 &w) { raw = w; }
    __device__ __forceinline__ void get(float *v) const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack(w[i], T());
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(T *p, const float *v)
    {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack(v[0], v[1], T()), pack(v[2], v[3], T()),
                                                   pack(v[4], v[5], T()), pack(v[6], v[7], T()));
    }
    static __device__ __forceinline__ void store_q(int8_t *p, const int *q)
    {
        auto four = [&](int i) {
            const uint32_t lo = __byte_perm(q[i], q[i + 1], 0x0040), hi = __byte_perm(q[i + 2], q[i + 3], 0x0040);
            return __byte_perm(lo, hi, 0x5410);
        };
        *reinterpret_cast<uint2 *>(p) = make_uint2(four(0), four(4));
    }
    static __device__ __forceinline__ void load_param(const float *p, float *v)
    {
        Vec<float, 4>::load_param(p, v);
        Vec<float, 4>::load_param(p + 4, v + 4);
    }
};

// Two fp32 operations per instruction; each rounds like the scalar one.
__device__ __forceinline__ float2 pair(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// max(|a|, |b|, |c|); a NaN among them is the result.
__device__ __forceinline__ float most_of(float a, float b, float c)
{
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// Sum over the TPR threads of a row; `scratch` is this sum's own TPR / 32 floats, so that one
// barrier does.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *scratch)
{
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
        for (int i = 0; i < TPR / 32; ++i) v += scratch[i];
    }
    return v;
}

// Largest of non-negative values over the TPR threads, as bits: ordered like the values, NaN on top.
template <int TPR>
__device__ __forceinline__ float row_most(float v, float *scratch)
{
    unsigned m = __float_as_uint(v);
    if (TPR < 32)
        for (int o = TPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    else
        m = __reduce_max_sync(0xffffffffu, m);
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = __uint_as_float(m);
        __syncthreads();
        m = 0;
        for (int i = 0; i < TPR / 32; ++i) m = max(m, __float_as_uint(scratch[i]));
    }
    return __uint_as_float(m);
}

// Threads of a block in which TPR threads hold a row: one row, or as many as 128 threads hold
// while a row stays within a warp.
constexpr int norm_block(int tpr) { return tpr <= 32 ? 128 : tpr; }

// What becomes of row r once thread `lane` of its TPR threads has its part in v (zeros beyond the
// row): NI runs of V elements, run i at column (i * TPR + lane) * V.  params(i, g, b) gives run i's
// gamma and beta.  All threads of a block call this together; rows past the end store nothing.
template <typename T, int V, int NI, int TPR, bool QUANT, typename Params>
__device__ __forceinline__ void finish_row(const NormArgs &a, long long r, int lane, float (&v)[NI * V],
                                           float (*scratch)[TPR > 32 ? TPR / 32 : 1], const Params &params)
{
    static_assert(NI * V % 2 == 0, "elements are handled in pairs");
    const bool live = r < a.rows;
    auto inside = [&](int i) { return (i * TPR + lane) * V < a.c; };
    if (!QUANT || a.normalise) {
        float2 s = both(0.0f);
        for (int e = 0; e < NI * V; e += 2) s = __fadd2_rn(s, pair(v[e], v[e + 1]));
        const float mean = row_sum<TPR>(s.x + s.y, scratch[0]) / (float)a.c;
        s = both(0.0f);
        if (V == 1) {
            for (int i = 0; i < NI; ++i)
                if (inside(i)) {
                    v[i] -= mean;
                    s.x = fmaf(v[i], v[i], s.x);
                }
        } else {
            for (int i = 0; i < NI; ++i)
                if (inside(i))
                    for (int e = i * V; e < (i + 1) * V; e += 2) {
                        const float2 d = __fadd2_rn(pair(v[e], v[e + 1]), both(-mean));
                        s = __ffma2_rn(d, d, s);
                        v[e] = d.x;
                        v[e + 1] = d.y;
                    }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(s.x + s.y, scratch[1]) / (float)a.c + a.eps);
        if (a.stats && lane == 0 && live) {
            a.stats[r] = mean;
            a.stats[a.rows + r] = rstd;
        }
        for (int i = 0; i < NI; ++i)
            if (inside(i)) {
                float g[V], b[V];
                params(i, g, b);
                if (V == 1) {
                    v[i] = fmaf(v[i] * rstd, g[0], b[0]);
                } else {
                    for (int j = 0; j < V; j += 2) {
                        const int e = i * V + j;
                        const float2 h = __fmul2_rn(pair(v[e], v[e + 1]), both(rstd));
                        const float2 y = __ffma2_rn(h, pair(g[j], g[j + 1]), pair(b[j], b[j + 1]));
                        v[e] = y.x;
                        v[e + 1] = y.y;
                    }
                }
            }
    }
    if (QUANT) {
        float most = 0.0f;
        for (int e = 0; e < NI * V; e += 2) most = most_of(most, v[e], v[e + 1]);
        most = row_most<TPR>(most, scratch[2]);
        float inv;
        const float scale = row_scale_of(__float_as_uint(most), &inv);
        if (lane == 0 && live) a.row_scale[r] = scale;
        // Adding 1.5 * 2^23 leaves a whole number, rounded to nearest even, in the low bits.  The products
        // are scalar: a packed one is joined with the addition into one that rounds once, which tips values
        // next to a half to the other side (seen against the definition's own arithmetic).
        if (scale < __int_as_float(0x7f800000)) {
            for (int e = 0; e < NI * V; e += 2) {
                const float2 q = __fadd2_rn(pair(__fmul_rn(v[e], inv), __fmul_rn(v[e + 1], inv)), both(12582912.0f));
                v[e] = q.x;
                v[e + 1] = q.y;
            }
        } else {
            for (int e = 0; e < NI * V; ++e) v[e] = 0.0f;
        }
        for (int i = 0; i < NI; ++i)
            if (live && inside(i)) {
                int q[V];
                for (int j = 0; j < V; ++j) q[j] = __float_as_int(v[i * V + j]);
                Vec<T, V>::store_q(a.q + r * a.q_stride + (i * TPR + lane) * V, q);
            }
    } else {
        for (int i = 0; i < NI; ++i)
            if (live && inside(i))
                Vec<T, V>::store(static_cast<T *>(a.y) + r * a.y_stride + (i * TPR + lane) * V, v + i * V);
    }
}

template <int V>
__device__ __forceinline__ void load_params(const NormArgs &a, int c, float *g, float *b)
{
    using P = Vec<typename ParamOf<V>::type, V>;
    for (int j = 0; j < V; ++j) g[j] = 1.0f, b[j] = 0.0f;
    if (a.gamma) P::load_param(a.gamma + c, g);
    if (a.beta) P::load_param(a.beta + c, b);
}

// One row for each TPR threads.
template <typename T, int V, int NI, int TPR, bool QUANT>
__global__ void __launch_bounds__(norm_block(TPR)) norm_rows_kernel(const NormArgs a)
{
    __shared__ float scratch[3][TPR > 32 ? TPR / 32 : 1];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const long long r = (long long)blockIdx.x * (norm_block(TPR) / TPR) + threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
    Vec<T, V> raw[NI];
    float v[NI * V];
    for (int i = 0; i < NI; ++i) {
        const int c = (i * TPR + lane) * V;
        if (r < a.rows && c < a.c) raw[i].load(x + c);
    }
    for (int i = 0; i < NI; ++i) {
        if (r < a.rows && (i * TPR + lane) * V < a.c)
            raw[i].get(v + i * V);
        else
            for (int j = 0; j < V; ++j) v[i * V + j] = 0.0f;
    }
    finish_row<T, V, NI, TPR, QUANT>(a, r, lane, v, scratch, [&](int i, float *g, float *b) {
        load_params<V>(a, (i * TPR + lane) * V, g, b);
    });
}

// ------------------------------------------------------------------ many rows: parameters held, rows streamed
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Blocks that stay for many rows: each thread keeps the gamma and beta of its columns in registers and
// copies its own part of the coming STAGES - 1 rows to shared memory with cp.async (no barrier: nobody
// else reads it), so that memory stays busy while a row is summed.
constexpr int kNormVecs = 4;  // vectors of a row per thread
constexpr int kNormStages = 3;
constexpr int norm_stream_blocks(int tpr) { return 512 / norm_block(tpr); }  // per SM: 128 registers a thread
template <typename T, int TPR, bool QUANT>
__global__ void __launch_bounds__(norm_block(TPR), norm_stream_blocks(TPR)) norm_stream_kernel(const NormArgs a)
{
    constexpr int V = 16 / sizeof(T), NI = kNormVecs;
    constexpr int kBlock = norm_block(TPR), kGroups = kBlock / TPR;
    __shared__ uint4 ring[kNormStages][NI][kBlock];
    // Two sets: a row's first sum may be written while a slow warp still reads the last row's.
    __shared__ float scratch[2][3][TPR > 32 ? TPR / 32 : 1];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * kGroups;
    auto fetch = [&](long long r, int stage) {
        if (r < a.rows) {
            const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
            for (int i = 0; i < NI; ++i) {
                const int c = (i * TPR + lane) * V;
                if (c < a.c) copy_async(dev::smem_u32(&ring[stage][i][threadIdx.x]), x + c);
            }
        }
        copy_commit();
    };
    long long r = (long long)blockIdx.x * kGroups + threadIdx.x / TPR;
    for (int s = 0; s < kNormStages - 1; ++s) fetch(r + s * step, s);
    float g[NI][V], b[NI][V];
    for (int i = 0; i < NI; ++i)
        if ((i * TPR + lane) * V < a.c) load_params<V>(a, (i * TPR + lane) * V, g[i], b[i]);
    int stage = 0, parity = 0;
    for (long long base = (long long)blockIdx.x * kGroups; base < a.rows; base += step, r += step) {
        fetch(r + (kNormStages - 1) * step, stage == 0 ? kNormStages - 1 : stage - 1);
        copy_wait<kNormStages - 1>();
        float v[NI * V];
        for (int i = 0; i < NI; ++i) {
            if (r < a.rows && (i * TPR + lane) * V < a.c) {
                Vec<T, V> raw;
                raw.from(ring[stage][i][threadIdx.x]);
                raw.get(v + i * V);
            } else {
                for (int j = 0; j < V; ++j) v[i * V + j] = 0.0f;
            }
        }
        finish_row<T, V, NI, TPR, QUANT>(a, r, lane, v, scratch[parity], [&](int i, float *pg, float *pb) {
            for (int j = 0; j < V; ++j) pg[j] = g[i][j], pb[j] = b[i][j];
        });
        stage = stage + 1 == kNormStages ? 0 : stage + 1;
        parity ^= 1;
    }
    copy_wait<0>();
}

unsigned blocks_for_rows(long long rows) { return (unsigned)(rows < (1LL << 20) ? rows : (1LL << 20)); }

template <typename T, int V, int NI, int TPR>
cudaError_t norm_rows_launch(const NormArgs &a, cudaStream_t stream)
{
    constexpr int kRows = norm_block(TPR) / TPR;
    const dim3 grid((unsigned)((a.rows + kRows - 1) / kRows)), block(norm_block(TPR));
    return a.q ? launch_overlapped(norm_rows_kernel<T, V, NI, TPR, true>, grid, block, 0, stream, 1, a)
               : launch_overlapped(norm_rows_kernel<T, V, NI, TPR, false>, grid, block, 0, stream, 1, a);
}

template <typename T, int TPR>
cudaError_t norm_stream_launch(const NormArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int kRows = norm_block(TPR) / TPR;
    const long long need = (a.rows + kRows - 1) / kRows, room = (long long)sm_count * norm_stream_blocks(TPR);
    const dim3 grid((unsigned)(need < room ? need : room)), block(norm_block(TPR));
    return a.q ? launch_overlapped(norm_stream_kernel<T, TPR, true>, grid, block, 0, stream, 1, a)
               : launch_overlapped(norm_stream_kernel<T, TPR, false>, grid, block, 0, stream, 1, a);
}

bool aligned_for(const void *p, long long stride, int element, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * element % bytes == 0;
}

template <typename T>
cudaError_t norm_launch_t(const NormArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    if (a.rows < (1LL << 31)) {
        const bool wide_loads = a.c % V == 0 && aligned_for(a.x, a.x_stride, sizeof(T), 16) &&
                                (a.q ? aligned_for(a.q, a.q_stride, 1, V) : aligned_for(a.y, a.y_stride, sizeof(T), 16)) &&
                                aligned_for(a.gamma, 0, 4, 16) && aligned_for(a.beta, 0, 4, 16);
        const int nv = a.c / V;
        // Held parameters and streamed rows are the faster from few rows on: bf16, us with one row for
        // each TPR threads against this, 8x4096 3.2 / 2.5, 600x1024 2.9 / 2.8, 2048x2048 7.1 / 6.5,
        // 32768x4096 110 / 84 (6.4 TB/s), 32768x256 10.0 / 9.2.  TPR is the fewest threads that hold the
        // row in four vectors each: more threads sum over more lanes (8192x4096 on 256: 37 us).
        if (wide_loads) {
            if (nv <= 4) return norm_rows_launch<T, V, 1, 4>(a, stream);
            if (nv <= 16) return norm_stream_launch<T, 4>(a, sm_count, stream);
            if (nv <= 32) return norm_stream_launch<T, 8>(a, sm_count, stream);
            if (nv <= 64) return norm_stream_launch<T, 16>(a, sm_count, stream);
            if (nv <= 128) return norm_stream_launch<T, 32>(a, sm_count, stream);
            if (nv <= 256) return norm_stream_launch<T, 64>(a, sm_count, stream);
            if (nv <= 512) return norm_stream_launch<T, 128>(a, sm_count, stream);
            if (nv <= 1024) return norm_stream_launch<T, 256>(a, sm_count, stream);
            if (nv <= 2048) return norm_rows_launch<T, V, 4, 512>(a, stream);
        } else {
            if (a.c <= 32) return norm_rows_launch<T, 1, 4, 8>(a, stream);
            if (a.c <= 128) return norm_rows_launch<T, 1, 4, 32>(a, stream);
            if (a.c <= 512) return norm_rows_launch<T, 1, 16, 32>(a, stream);
            if (a.c <= 1024) return norm_rows_launch<T, 1, 8, 128>(a, stream);
            if (a.c <= 2048) return norm_rows_launch<T, 1, 16, 128>(a, stream);
            if (a.c <= 8192) return norm_rows_launch<T, 1, 32, 256>(a, stream);
        }
    }
    return launch_overlapped(norm_wide_kernel<T>, dim3(blocks_for_rows(a.rows)), dim3(kWideThreads), 0, stream, 1, a);
}

// ------------------------------------------------------------------ gradient, rows in registers
// As norm_stream_kernel: blocks stay for many rows, TPR threads hold a row of x and dy (NI runs of V
// elements each), and each thread keeps gamma and the running sums of dy * h and dy for its own columns
// in registers, so that x and dy are read once for all three gradients.  The two sums over a row share
// one barrier.  At the end the rows of a block are joined in shared memory, and each block writes one
// row of partial sums, which norm_grad_join_kernel adds up in order.
constexpr int kGradElements = 16;  // of a row per thread: sums, gamma, h and g of more would not fit 128 registers
constexpr int kGradStages = 3;
constexpr int grad_block(int tpr) { return tpr < 256 ? 256 : tpr; }
constexpr int grad_blocks_per_sm(int tpr) { return 512 / grad_block(tpr); }

// Sums of two values over the TPR threads of a row; scratch: 2 * TPR / 32 floats for each row of the block.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 *scratch)
{
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) scratch[warp] = v;
        __syncthreads();
        v = both(0.0f);
        for (int i = 0; i < TPR / 32; ++i) v = __fadd2_rn(v, scratch[warp / (TPR / 32) * (TPR / 32) + i]);
    }
    return v;
}

template <typename T, int V, int TPR>
__global__ void __launch_bounds__(grad_block(TPR), grad_blocks_per_sm(TPR)) norm_grad_stream_kernel(const GradArgs a)
{
    constexpr int E = kGradElements, NI = E / V, kBlock = grad_block(TPR), kGroups = kBlock / TPR;
    constexpr bool kRing = V > 1;  // single elements are loaded without one
    extern __shared__ uint4 grad_ring[];  // [stage][x, dy][NI][kBlock]; afterwards the join of the block's rows
    __shared__ float2 scratch[2][kBlock / 32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * kGroups;
    auto column = [&](int i) { return (i * TPR + lane) * V; };
    auto slot = [&](int stage, int which, int i) {
        return grad_ring + ((stage * 2 + which) * NI + i) * kBlock + threadIdx.x;
    };
    auto fetch = [&](long long r, int stage) {
        if constexpr (kRing) {
            if (r < a.rows) {
                const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
                const T *dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
                for (int i = 0; i < NI; ++i)
                    if (column(i) < a.c) {
                        copy_async(dev::smem_u32(slot(stage, 0, i)), x + column(i));
                        copy_async(dev::smem_u32(slot(stage, 1, i)), dy + column(i));
                    }
            }
            copy_commit();
        }
    };
    auto moments = [&](long long r) {
        return r < a.rows ? make_float2(__ldg(a.stats + r), __ldg(a.stats + a.rows + r)) : both(0.0f);
    };
    long long r = (long long)blockIdx.x * kGroups + threadIdx.x / TPR;
    for (int s = 0; s < kGradStages - 1; ++s) fetch(r + s * step, s);
    float2 next = moments(r);
    float gamma[E], dg[E], db[E];
    for (int i = 0; i < NI; ++i) {
        for (int j = 0; j < V; ++j) gamma[i * V + j] = 1.0f;
        if (a.gamma && column(i) < a.c) Vec<typename ParamOf<V>::type, V>::load_param(a.gamma + column(i), gamma + i * V);
    }
    for (int e = 0; e < E; ++e) dg[e] = db[e] = 0.0f;
    const float per_c = 1.0f / (float)a.c;
    int stage = 0, parity = 0;
    for (long long base = (long long)blockIdx.x * kGroups; base < a.rows; base += step, r += step) {
        fetch(r + (kGradStages - 1) * step, stage == 0 ? kGradStages - 1 : stage - 1);
        const float2 moment = next;
        next = moments(r + step);
        if (kRing) copy_wait<kGradStages - 1>();
        const float mean = moment.x, rstd = moment.y;
        float h[E], g[E];
        Vec<T, V> xs[NI], dys[NI];
        for (int i = 0; i < NI; ++i)
            if (r < a.rows && column(i) < a.c) {
                if constexpr (kRing) {
                    xs[i].from(*slot(stage, 0, i));
                    dys[i].from(*slot(stage, 1, i));
                } else {
                    xs[i].load(static_cast<const T *>(a.x) + r * a.x_stride + column(i));
                    dys[i].load(static_cast<const T *>(a.dy) + r * a.dy_stride + column(i));
                }
            }
        float2 s1 = both(0.0f), s2 = both(0.0f);
        for (int i = 0; i < NI; ++i) {
            if (r < a.rows && column(i) < a.c) {
                xs[i].get(h + i * V);
                dys[i].get(g + i * V);
            } else {  // adds nothing anywhere: h and dy are both 0
                for (int j = 0; j < V; ++j) h[i * V + j] = mean, g[i * V + j] = 0.0f;
            }
        }
        for (int e = 0; e < E; e += 2) {
            const float2 d = pair(g[e], g[e + 1]);
            const float2 hh = __fmul2_rn(__fadd2_rn(pair(h[e], h[e + 1]), both(-mean)), both(rstd));
            const float2 sum_g = __ffma2_rn(d, hh, pair(dg[e], dg[e + 1]));
            const float2 sum_b = __fadd2_rn(d, pair(db[e], db[e + 1]));
            const float2 gg = __fmul2_rn(d, pair(gamma[e], gamma[e + 1]));
            s1 = __fadd2_rn(s1, gg);
            s2 = __ffma2_rn(gg, hh, s2);
            dg[e] = sum_g.x, dg[e + 1] = sum_g.y;
            db[e] = sum_b.x, db[e + 1] = sum_b.y;
            h[e] = hh.x, h[e + 1] = hh.y;
            g[e] = gg.x, g[e + 1] = gg.y;
        }
        const float2 sums = row_sum2<TPR>(make_float2(s1.x + s1.y, s2.x + s2.y), scratch[parity]);
        const float m1 = sums.x * per_c, m2 = sums.y * per_c;
        for (int e = 0; e < E; e += 2) {
            const float2 t = __fadd2_rn(__ffma2_rn(pair(h[e], h[e + 1]), both(-m2), pair(g[e], g[e + 1])), both(-m1));
            const float2 d = __fmul2_rn(t, both(rstd));
            h[e] = d.x, h[e + 1] = d.y;
        }
        if (r < a.rows)
            for (int i = 0; i < NI; ++i)
                if (column(i) < a.c)
                    Vec<T, V>::store(static_cast<T *>(a.dx) + r * a.dx_stride + column(i), h + i * V);
        stage = stage + 1 == kGradStages ? 0 : stage + 1;
        parity ^= 1;
    }
    if (kRing) copy_wait<0>();
    float *out = a.partial + (long long)blockIdx.x * 2 * a.c;
    if constexpr (kGroups == 1) {
        for (int i = 0; i < NI; ++i)
            if (column(i) < a.c) {
                if constexpr (V == 1) {
                    out[column(i)] = dg[i];
                    out[a.c + column(i)] = db[i];
                } else {
                    for (int j = 0; j < V; j += 4) {
                        const int e = i * V + j;
                        *reinterpret_cast<float4 *>(out + column(i) + j) = make_float4(dg[e], dg[e + 1], dg[e + 2], dg[e + 3]);
                        *reinterpret_cast<float4 *>(out + a.c + column(i) + j) =
                            make_float4(db[e], db[e + 1], db[e + 2], db[e + 3]);
                    }
                }
            }
    } else {
        // The block's rows side by side in shared memory, [row][dgamma, dbeta][element][thread]; those of one
        // warp are joined by shuffles before.
        constexpr int kSide = TPR < 32 ? kBlock / 32 : kGroups;
        for (int o = TPR; o < 32; o <<= 1)
            for (int e = 0; e < E; ++e) {
                dg[e] += __shfl_xor_sync(0xffffffffu, dg[e], o);
                db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
            }
        float *join = reinterpret_cast<float *>(grad_ring);
        __syncthreads();  // the ring is no longer read
        if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
            float *mine = join + (TPR < 32 ? threadIdx.x / 32 : threadIdx.x / TPR) * (2 * E * TPR) + lane;
            for (int e = 0; e < E; ++e) {
                mine[e * TPR] = dg[e];
                mine[(E + e) * TPR] = db[e];
            }
        }
        __syncthreads();
        for (int col = threadIdx.x; col < 2 * a.c; col += kBlock) {
            const int c = col < a.c ? col : col - a.c;
            const int e = c / (TPR * V) * V + c % V + (col < a.c ? 0 : E);
            const float *at = join + e * TPR + c / V % TPR;
            float sum = at[0];
            for (int t = 1; t < kSide; ++t) sum += at[t * (2 * E * TPR)];
            out[col] = sum;
        }
    }
}

cudaError_t norm_grad_join(const GradArgs &a, cudaStream_t stream)
{
    return launch_overlapped(norm_grad_join_kernel, dim3((unsigned)((2LL * a.c + 31) / 32)), dim3(32, kJoinRuns), 0,
                             stream, 1, a);
}

template <typename T, int V, int TPR>
cudaError_t norm_grad_stream_launch(GradArgs a, int sm_count, cudaStream_t stream)
{
    constexpr int kRows = grad_block(TPR) / TPR;
    constexpr int kRing = V > 1 ? kGradStages * 2 * (kGradElements / V) * grad_block(TPR) * 16 : 0;
    constexpr int kJoin = kRows > 1 ? (TPR < 32 ? 8 : kRows) * 2 * kGradElements * TPR * 4 : 0;
    constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    static bool allowed[kMaxDevices] = {};
    if (kSmem > 46 * 1024) {  // the sums of a block take some of the first 48 KB
        cudaError_t e = allow_dynamic_smem(norm_grad_stream_kernel<T, V, TPR>, kSmem, allowed);
        if (e != cudaSuccess) return e;
    }
    const long long need = (a.rows + kRows - 1) / kRows, room = (long long)sm_count * grad_blocks_per_sm(TPR);
    a.partial_rows = (int)(need < room ? need : room);
    cudaError_t e = launch_overlapped(norm_grad_stream_kernel<T, V, TPR>, dim3((unsigned)a.partial_rows),
                                      dim3(grad_block(TPR)), kSmem, stream, 1, a);
    return e == cudaSuccess ? norm_grad_join(a, stream) : e;
}

template <typename T>
cudaError_t norm_grad_launch_t(const GradArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    const bool wide_loads = a.c % V == 0 && aligned_for(a.x, a.x_stride, sizeof(T), 16) &&
                            aligned_for(a.dy, a.dy_stride, sizeof(T), 16) &&
                            aligned_for(a.dx, a.dx_stride, sizeof(T), 16) && aligned_for(a.gamma, 0, 4, 16);
    if (wide_loads) {
        if (a.c <= 8 * kGradElements) return norm_grad_stream_launch<T, V, 8>(a, sm_count, stream);
        if (a.c <= 16 * kGradElements) return norm_grad_stream_launch<T, V, 16>(a, sm_count, stream);
        if (a.c <= 32 * kGradElements) return norm_grad_stream_launch<T, V, 32>(a, sm_count, stream);
        if (a.c <= 64 * kGradElements) return norm_grad_stream_launch<T, V, 64>(a, sm_count, stream);
        if (a.c <= 128 * kGradElements) return norm_grad_stream_launch<T, V, 128>(a, sm_count, stream);
        if (a.c <= 256 * kGradElements) return norm_grad_stream_launch<T, V, 256>(a, sm_count, stream);
        if (a.c <= 512 * kGradElements) return norm_grad_stream_launch<T, V, 512>(a, sm_count, stream);
    } else {
        if (a.c <= 8 * kGradElements) return norm_grad_stream_launch<T, 1, 8>(a, sm_count, stream);
        if (a.c <= 32 * kGradElements) return norm_grad_stream_launch<T, 1, 32>(a, sm_count, stream);
        if (a.c <= 128 * kGradElements) return norm_grad_stream_launch<T, 1, 128>(a, sm_count, stream);
        if (a.c <= 512 * kGradElements) return norm_grad_stream_launch<T, 1, 512>(a, sm_count, stream);
    }
    cudaError_t e = launch_overlapped(norm_grad_wide_kernel<T>, dim3(blocks_for_rows(a.rows)), dim3(kWideThreads), 0,
                                      stream, 1, a);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(norm_grad_columns_kernel<T>,
                          dim3((unsigned)((a.c + kWideThreads - 1) / kWideThreads), (unsigned)a.partial_rows),
                          dim3(kWideThreads), 0, stream, 1, a);
    return e == cudaSuccess ? norm_grad_join(a, stream) : e;
}

}  // namespace

cudaError_t norm_launch(const NormProblem &p, int sm_count, cudaStream_t stream)
{
    NormArgs a{};
    a.x = p.x.data;
    a.x_stride = p.x.stride;
    a.y = p.y.data;
    a.y_stride = p.y.stride;
    a.q = static_cast<int8_t *>(p.q.data);
    a.q_stride = p.q.stride;
    a.row_scale = p.row_scale;
    a.stats = p.stats;
    a.gamma = p.gamma;
    a.beta = p.beta;
    a.rows = p.rows;
    a.c = p.c;
    a.eps = p.eps;
    a.normalise = p.normalise;
    switch (p.dtype) {
    case kF32: return norm_launch_t<float>(a, sm_count, stream);
    case kBf16: return norm_launch_t<__nv_bfloat16>(a, sm_count, stream);
    default: return norm_launch_t<__half>(a, sm_count, stream);
    }
}

int norm_grad_partial_rows(long long rows, int c, int sm_count)
{
    (void)c;
    const long long most = 2LL * sm_count;  // norm_grad_stream_kernel's blocks at most
    return (int)(rows < most ? rows : most);
}

cudaError_t norm_grad_launch(const NormGradProblem &p, int sm_count, cudaStream_t stream)
{
    GradArgs a{};
    a.dy = p.dy.data;
    a.dy_stride = p.dy.stride;
    a.x = p.x.data;
    a.x_stride = p.x.stride;
    a.dx = p.dx.data;
    a.dx_stride = p.dx.stride;
    a.gamma = p.gamma;
    a.stats = p.stats;
    a.dgamma = p.dgamma;
    a.dbeta = p.dbeta;
    a.partial = p.partial;
    a.rows = p.rows;
    a.c = p.c;
    a.partial_rows = p.partial_rows;
    switch (p.dtype) {
    case kF32: return norm_grad_launch_t<float>(a, sm_count, stream);
    case kBf16: return norm_grad_launch_t<__nv_bfloat16>(a, sm_count, stream);
    default: return norm_grad_launch_t<__half>(a, sm_count, stream);
    }
}

}  // namespace cbs
