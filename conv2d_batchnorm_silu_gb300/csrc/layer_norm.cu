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
        *reinterpret_cast<char4 *>(p) = make_char4((char)q[0], (char)q[1], (char)q[2], (char)q[3]);
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
            return (uint32_t)(q[i] & 255) | (uint32_t)(q[i + 1] & 255) << 8 | (uint32_t)(q[i + 2] & 255) << 16 |
                   (uint32_t)q[i + 3] << 24;
        };
        *reinterpret_cast<uint2 *>(p) = make_uint2(four(0), four(4));
    }
    static __device__ __forceinline__ void load_param(const float *p, float *v)
    {
        Vec<float, 4>::load_param(p, v);
        Vec<float, 4>::load_param(p + 4, v + 4);
    }
};

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

template <int TPR>
__device__ __forceinline__ unsigned row_max(unsigned v, float *scratch)
{
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = __uint_as_float(v);
        __syncthreads();
        v = 0;
        for (int i = 0; i < TPR / 32; ++i) v = max(v, __float_as_uint(scratch[i]));
    }
    return v;
}

constexpr int norm_block(int tpr) { return tpr < 128 ? 128 : tpr; }

template <typename T, int V, int NI, int TPR, bool QUANT>
__global__ void __launch_bounds__(norm_block(TPR)) norm_rows_kernel(const NormArgs a)
{
    __shared__ float scratch[3][TPR > 32 ? TPR / 32 : 1];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const long long r = (long long)blockIdx.x * (norm_block(TPR) / TPR) + threadIdx.x / TPR;
    const bool live = r < a.rows;  // the same for all threads of a block of one row
    const T *x = static_cast<const T *>(a.x) + (live ? r * a.x_stride : 0);
    Vec<T, V> raw[NI];
    for (int i = 0; i < NI; ++i) {
        const int c = (i * TPR + lane) * V;
        if (live && c < a.c) raw[i].load(x + c);
    }
    float v[NI][V];
    for (int i = 0; i < NI; ++i) {
        if (live && (i * TPR + lane) * V < a.c)
            raw[i].get(v[i]);
        else
            for (int j = 0; j < V; ++j) v[i][j] = 0.0f;
    }
    if (!QUANT || a.normalise) {
        float s = 0.0f;
        for (int i = 0; i < NI; ++i)
            for (int j = 0; j < V; ++j) s += v[i][j];
        const float mean = row_sum<TPR>(s, scratch[0]) / (float)a.c;
        s = 0.0f;
        for (int i = 0; i < NI; ++i)
            if ((i * TPR + lane) * V < a.c)
                for (int j = 0; j < V; ++j) {
                    v[i][j] -= mean;
                    s = fmaf(v[i][j], v[i][j], s);
                }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, scratch[1]) / (float)a.c + a.eps);
        if (a.stats && live && lane == 0) {
            a.stats[r] = mean;
            a.stats[a.rows + r] = rstd;
        }
        for (int i = 0; i < NI; ++i) {
            const int c = (i * TPR + lane) * V;
            if (c < a.c) {
                float g[V], b[V];
                if (a.gamma)
                    Vec<T, V>::load_param(a.gamma + c, g);
                else
                    for (int j = 0; j < V; ++j) g[j] = 1.0f;
                if (a.beta)
                    Vec<T, V>::load_param(a.beta + c, b);
                else
                    for (int j = 0; j < V; ++j) b[j] = 0.0f;
                for (int j = 0; j < V; ++j) v[i][j] = fmaf(v[i][j] * rstd, g[j], b[j]);
            }
        }
    }
    if (QUANT) {
        unsigned most = 0;
        for (int i = 0; i < NI; ++i)
            for (int j = 0; j < V; ++j) most = max(most, magnitude_bits(v[i][j]));
        float inv;
        const float scale = row_scale_of(row_max<TPR>(most, scratch[2]), &inv);
        if (live && lane == 0) a.row_scale[r] = scale;
        for (int i = 0; i < NI; ++i) {
            const int c = (i * TPR + lane) * V;
            int q[V];
            for (int j = 0; j < V; ++j) q[j] = __float2int_rn(v[i][j] * inv);
            if (live && c < a.c) Vec<T, V>::store_q(a.q + r * a.q_stride + c, q);
        }
    } else {
        for (int i = 0; i < NI; ++i) {
            const int c = (i * TPR + lane) * V;
            if (live && c < a.c) Vec<T, V>::store(static_cast<T *>(a.y) + r * a.y_stride + c, v[i]);
        }
    }
}

unsigned blocks_for_rows(long long rows) { return (unsigned)(rows < (1LL << 20) ? rows : (1LL << 20)); }

template <typename T, int V, int NI, int TPR>
cudaError_t norm_rows_launch(const NormArgs &a, cudaStream_t stream)
{
    constexpr int kRows = norm_block(TPR) / TPR;
    const dim3 grid((unsigned)((a.rows + kRows - 1) / kRows));
    return a.q ? launch_overlapped(norm_rows_kernel<T, V, NI, TPR, true>, grid, dim3(norm_block(TPR)), 0, stream, 1, a)
               : launch_overlapped(norm_rows_kernel<T, V, NI, TPR, false>, grid, dim3(norm_block(TPR)), 0, stream, 1, a);
}

bool aligned_for(const void *p, long long stride, int element, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * element % bytes == 0;
}

template <typename T>
cudaError_t norm_launch_t(const NormArgs &a, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    if (a.rows < (1LL << 31)) {
        const bool wide_loads = a.c % V == 0 && aligned_for(a.x, a.x_stride, sizeof(T), 16) &&
                                (a.q ? aligned_for(a.q, a.q_stride, 1, V) : aligned_for(a.y, a.y_stride, sizeof(T), 16)) &&
                                aligned_for(a.gamma, 0, 4, 16) && aligned_for(a.beta, 0, 4, 16);
        // The fewest threads that hold the row, so that its sums cross as few lanes as possible, with at
        // most 32 elements each (registers), from four vectors a thread on more threads instead.
        if (wide_loads) {
            const int nv = a.c / V;
            if (nv <= 4) return norm_rows_launch<T, V, 1, 4>(a, stream);
            if (nv <= 16) return norm_rows_launch<T, V, 1, 16>(a, stream);
            if (nv <= 32) return norm_rows_launch<T, V, 1, 32>(a, stream);
            if (nv <= 64) return norm_rows_launch<T, V, 2, 32>(a, stream);
            if (nv <= 128) return norm_rows_launch<T, V, 4, 32>(a, stream);
            if (nv <= 256) return norm_rows_launch<T, V, 2, 128>(a, stream);
            if (nv <= 512) return norm_rows_launch<T, V, 4, 128>(a, stream);
            if (nv <= 1024) return norm_rows_launch<T, V, 4, 256>(a, stream);
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

template <typename T>
cudaError_t norm_grad_launch_t(const GradArgs &a, cudaStream_t stream)
{
    cudaError_t e = launch_overlapped(norm_grad_wide_kernel<T>, dim3(blocks_for_rows(a.rows)), dim3(kWideThreads), 0,
                                      stream, 1, a);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(norm_grad_columns_kernel<T>,
                          dim3((unsigned)((a.c + kWideThreads - 1) / kWideThreads), (unsigned)a.partial_rows),
                          dim3(kWideThreads), 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    return launch_overlapped(norm_grad_join_kernel, dim3((unsigned)((2LL * a.c + 31) / 32)), dim3(32, kJoinRuns), 0,
                             stream, 1, a);
}

}  // namespace

cudaError_t norm_launch(const NormProblem &p, cudaStream_t stream)
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
    case kF32: return norm_launch_t<float>(a, stream);
    case kBf16: return norm_launch_t<__nv_bfloat16>(a, stream);
    default: return norm_launch_t<__half>(a, stream);
    }
}

int norm_grad_partial_rows(long long rows, int c, int sm_count)
{
    (void)c;
    const long long most = 4LL * sm_count;
    return (int)(rows < most ? rows : most);
}

cudaError_t norm_grad_launch(const NormGradProblem &p, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
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
    case kF32: return norm_grad_launch_t<float>(a, stream);
    case kBf16: return norm_grad_launch_t<__nv_bfloat16>(a, stream);
    default: return norm_grad_launch_t<__half>(a, stream);
    }
}

}  // namespace cbs
