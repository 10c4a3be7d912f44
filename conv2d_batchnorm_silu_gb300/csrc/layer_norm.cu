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

unsigned blocks_for_rows(long long rows) { return (unsigned)(rows < (1LL << 20) ? rows : (1LL << 20)); }

template <typename T>
cudaError_t norm_launch_t(const NormArgs &a, cudaStream_t stream)
{
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
