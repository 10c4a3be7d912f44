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

// One row per block at a time, read once for each sum it needs: any width, alignment and stride.  What the
// kernels below do not hold comes here: rows of more than 16384 elements (f32 8192), and many rows of 8193 to 9500
// off 16-byte boundaries.  Bound by its element-wise loads: bf16, 14592x9001 214 us (2.5 TB/s).
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

// dx, one row per block at a time, for rows of more than 8192 elements.
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

// Column sums of partial[partial_rows][2c] in a fixed order: 32 columns per block, 32 runs of rows summed side by
// side and joined by shuffles.  A thread's loads are all in flight at once (two rows an SM are ten a thread): the
// kernel is one trip to L2 and its launch.
constexpr int kJoinRuns = 32, kJoinLoads = 10;
__global__ void __launch_bounds__(32 * kJoinRuns) norm_grad_join_kernel(const GradArgs a)
{
    __shared__ float part[kJoinRuns][33];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int i = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    for (int r0 = threadIdx.y; r0 < a.partial_rows; r0 += kJoinRuns * kJoinLoads) {
        float v[kJoinLoads];
#pragma unroll
        for (int j = 0; j < kJoinLoads; ++j) {
            const int r = r0 + j * kJoinRuns;
            v[j] = r < a.partial_rows && i < 2 * a.c ? a.partial[(long long)r * 2 * a.c + i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kJoinLoads; ++j) s += v[j];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = part[threadIdx.x][threadIdx.y];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int column = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && column < 2 * a.c) {
        if (column < a.c)
            a.dgamma[column] = s;
        else
            a.dbeta[column - a.c] = s;
    }
}

// ------------------------------------------------------------------ rows held in registers
// A row stays in the registers of TPR threads from its one load to its one store; sums go through warp
// shuffles and, above a warp, shared memory.  A thread holds NI runs of V elements, run i at column
// (i * TPR + lane) * V.  W is the bytes of a run: 16 where every pointer, row distance and the width allow
// it; else 4 for f32, one element, and 2 for the 16-bit types, one element of a row that its threads copied
// together (fetch_row).
__device__ __forceinline__ float2 unpack(uint32_t w, __nv_bfloat16)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack(uint32_t w, __half)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t pack(float2 v, __nv_bfloat16)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint32_t pack(float2 v, __half)
{
    const __half2 b = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Two fp32 operations per instruction; each rounds like the scalar one.
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Asynchronous copies to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One run of a row: copied to its thread's own SLOT bytes of shared memory, read from there as floats, stored.
// Only runs within the row are.
template <typename T, int W>
struct Run;

template <>
struct Run<float, 16> {
    static constexpr int V = 4, SLOT = 16;
    static __device__ __forceinline__ void copy(uint32_t dst, const float *p) { copy16(dst, p); }
    static __device__ __forceinline__ void get(const void *slot, float2 *v)
    {
        const float4 f = *static_cast<const float4 *>(slot);
        v[0] = make_float2(f.x, f.y);
        v[1] = make_float2(f.z, f.w);
    }
    static __device__ __forceinline__ void store(float *p, const float2 *v)
    {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
};
template <>
struct Run<float, 4> {
    static constexpr int V = 1, SLOT = 4;
    static __device__ __forceinline__ void copy(uint32_t dst, const float *p) { copy4(dst, p); }
    static __device__ __forceinline__ void get(const void *slot, float *v) { *v = *static_cast<const float *>(slot); }
    static __device__ __forceinline__ void store(float *p, const float *v) { *p = *v; }
};
template <typename T>
struct Run<T, 16> {
    static constexpr int V = 8, SLOT = 16;
    static __device__ __forceinline__ void copy(uint32_t dst, const T *p) { copy16(dst, p); }
    static __device__ __forceinline__ void get(const void *slot, float2 *v)
    {
        const uint4 w = *static_cast<const uint4 *>(slot);
        v[0] = unpack(w.x, T());
        v[1] = unpack(w.y, T());
        v[2] = unpack(w.z, T());
        v[3] = unpack(w.w, T());
    }
    static __device__ __forceinline__ void store(T *p, const float2 *v)
    {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack(v[0], T()), pack(v[1], T()), pack(v[2], T()), pack(v[3], T()));
    }
};
// Elements one by one, of a row that its threads copied together (fetch_row).
template <typename T>
struct Run<T, 2> {
    static constexpr int V = 1, SLOT = 2;
    static __device__ __forceinline__ void copy(uint32_t, const T *) {}
    static __device__ __forceinline__ void get(const void *slot, float *v) { *v = to_float(*static_cast<const T *>(slot)); }
    static __device__ __forceinline__ void store(T *p, const float *v) { from_float(*v, p); }
};

// A row at any alignment copied by its TPR threads in the aligned 16-byte pieces that hold it: row_bytes() of
// shared memory, in which the row starts where it does in its first piece.  (Every thread its own runs, as where
// rows are aligned, takes two 4-byte copies for a pair of elements: 3001x777 8.6 us against 5.9.)
constexpr int row_bytes(int elements) { return elements * 2 + 32; }
template <int TPR, typename T>
__device__ __forceinline__ void fetch_row(uint32_t dst, const T *row, int c, int lane)
{
    const uintptr_t from = reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15;
    const int pieces = (int)((reinterpret_cast<uintptr_t>(row + c) - from + 15) >> 4);
    for (int i = lane; i < pieces; i += TPR) copy16(dst + 16 * i, reinterpret_cast<const void *>(from + 16 * (uintptr_t)i));
}
template <typename T>
__device__ __forceinline__ int start_of(const T *row) { return (int)(reinterpret_cast<uintptr_t>(row) & 15); }

// V quantised values (in the low bytes of q) to memory.
template <int V>
__device__ __forceinline__ void store_q(int8_t *p, const int *q, int n)
{
    auto four = [&](int i) {
        const uint32_t lo = __byte_perm(q[i], q[i + 1], 0x0040), hi = __byte_perm(q[i + 2], q[i + 3], 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    };
    if constexpr (V == 8)
        *reinterpret_cast<uint2 *>(p) = make_uint2(four(0), four(4));
    else if constexpr (V == 4)
        *reinterpret_cast<uint32_t *>(p) = four(0);
    else
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = (int8_t)q[i];
}

// Parameters of n columns from column 0 of p, `otherwise` where there is no array and 0 where the row has
// no column.
template <int V>
__device__ __forceinline__ void load_params(const float *p, float otherwise, int n, float *v)
{
    for (int j = 0; j < V; ++j) v[j] = j < n ? otherwise : 0.0f;
    if (!p || n <= 0) return;
    if constexpr (V >= 4) {
        for (int j = 0; j < V; j += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p + j));
            v[j] = f.x;
            v[j + 1] = f.y;
            v[j + 2] = f.z;
            v[j + 3] = f.w;
        }
    } else {
        for (int j = 0; j < V; ++j)
            if (j < n) v[j] = __ldg(p + j);
    }
}

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
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
        for (int i = 0; i < TPR / 32; ++i) v += scratch[i];
    }
    return v;
}

// Largest of non-negative values over the TPR threads of a row, as bits: ordered like the values, NaN on top.
template <int TPR>
__device__ __forceinline__ float row_most(float v, float *scratch)
{
    unsigned m = __float_as_uint(v);
    if constexpr (TPR >= 32)
        m = __reduce_max_sync(0xffffffffu, m);
    else
        for (int o = TPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = __uint_as_float(m);
        __syncthreads();
        m = 0;
        for (int i = 0; i < TPR / 32; ++i) m = max(m, __float_as_uint(scratch[i]));
    }
    return __uint_as_float(m);
}

// Quotients by a row's width, which is known beforehand: products with its reciprocal in two parts, with one rounding
// at the end (Brisebarre, Muller and Raina, "Accelerating correctly rounded floating-point division when the divisor
// is known in advance", 2004).  A quotient that fp32 holds comes out exactly, so the mean of equal values is that
// value; by the rounded reciprocal alone a row of 1000 and 7 channels ended 0.02 off beta.  (f16, 3001x777 5.1 us; with
// ordinary divisions, which give the same, 6.4.)
struct Width {
    float hi, lo;
    __device__ __forceinline__ explicit Width(int c) : hi(1.0f / (float)c), lo(fmaf(-hi, (float)c, 1.0f) * hi) {}
    __device__ __forceinline__ float share(float sum) const
    {
        const float q = sum * hi;
        return fabsf(q) < __int_as_float(0x7f800000) ? fmaf(sum, hi, sum * lo) : q;  // infinities and NaN stay
    }
};

// Blocks stay for many rows.  Each thread keeps the gamma and beta of its columns in registers and copies
// its own part of the coming rows to shared memory with cp.async (no barrier: nobody else
// reads it), so that memory stays busy while a row is summed.  Short rows share a warp.
// Bound by memory: bf16, 16384x4096 45 us and 14592x8192 72 us (5.9 and 6.6 TB/s of 6.8 for a copy).  With
// quantisation 14592x4096 39 us, x8192 81 (4.6 and 4.4 TB/s), with neither memory nor any pipe full.
constexpr int norm_stages(int w) { return w == 2 ? 4 : 3; }
// Threads of a block: one row, or as many as 128 threads hold while a row stays within a warp.
constexpr int norm_block(int tpr) { return tpr <= 32 ? 128 : tpr; }
constexpr int kSmThreads = 512;  // on an SM: 128 registers a thread

template <typename T, int W, int NI, int TPR, bool QUANT>
__global__ void __launch_bounds__(norm_block(TPR), kSmThreads / norm_block(TPR)) norm_stream_kernel(const NormArgs a)
{
    using R = Run<T, W>;
    constexpr int V = R::V, E = NI * V, kBlock = norm_block(TPR), kGroups = kBlock / TPR;
    constexpr int kStages = norm_stages(W);
    constexpr bool kTogether = W == 2;  // a row's threads copy it together: what one reads, others have copied
    extern __shared__ __align__(16) unsigned char norm_ring[];  // [stage][run][thread] slots, or [stage][group] rows
    // Two sets: a row's first sum may be written while a slow warp still reads the last row's.
    __shared__ float scratch[2][3][TPR > 32 ? TPR / 32 : 1];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * kGroups;
    // Of what a thread may hold, nothing lies in the row from past(i)'s run or unused(e)'s pair on.  Looked at where
    // instructions set the pace: 14592x5120 quantised 82 -> 72 us, but 14592x16384 151 -> 162.
    constexpr bool kSkips = W == 4 || (W == 16 && QUANT);
    auto past = [&](int i) { return kSkips && i > 0 && i * V % (V < 4 ? 4 : V) == 0 && i * TPR * V >= a.c; };
    auto unused = [&](int e) { return kSkips && e > 0 && 2 * e % (V < 4 ? 4 : V) == 0 && 2 * e / V * TPR * V >= a.c; };
    auto column = [&](int i) { return (i * TPR + lane) * V; };
    auto row_at = [&](long long r) { return static_cast<const T *>(a.x) + r * a.x_stride; };
    auto row_ring = [&](int stage) { return norm_ring + (stage * kGroups + threadIdx.x / TPR) * row_bytes(E * TPR); };
    auto slot = [&](int stage, int i) { return norm_ring + ((stage * NI + i) * kBlock + threadIdx.x) * R::SLOT; };
    auto fetch = [&](long long r, int stage) {
        if (r < a.rows) {
            const T *x = row_at(r);
            if constexpr (kTogether) {
                fetch_row<TPR>(dev::smem_u32(row_ring(stage)), x, a.c, lane);
            } else {
                for (int i = 0; i < NI; ++i)
                    if (column(i) < a.c) R::copy(dev::smem_u32(slot(stage, i)), x + column(i));
            }
        }
        copy_commit();
    };
    long long r = (long long)blockIdx.x * kGroups + threadIdx.x / TPR;
    for (int s = 0; s < kStages - 1; ++s) fetch(r + s * step, s);
    float2 g[(E + 1) / 2], b[(E + 1) / 2];
    for (int i = 0; i < NI; ++i) {
        load_params<V>(a.gamma ? a.gamma + column(i) : nullptr, 1.0f, a.c - column(i), reinterpret_cast<float *>(g) + i * V);
        load_params<V>(a.beta ? a.beta + column(i) : nullptr, 0.0f, a.c - column(i), reinterpret_cast<float *>(b) + i * V);
    }
    if constexpr (kTogether) {
        copy_wait<kStages - 2>();
        __syncthreads();
    }
    const Width width(a.c);
    int stage = 0, parity = 0;
    // All groups of a block go round together; rows past the end are zeros and store nothing.
    for (long long base = (long long)blockIdx.x * kGroups; base < a.rows; base += step, r += step) {
        fetch(r + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        // Rows copied together are waited for one round ahead: the barrier of this row's sums is also theirs.
        copy_wait<kTogether ? kStages - 2 : kStages - 1>();
        const bool live = r < a.rows;
        const unsigned char *mine = row_ring(stage) + start_of(row_at(r));
        float2 v[E / 2];
        float *vs = reinterpret_cast<float *>(v);
#pragma unroll
        for (int i = 0; i < NI && !past(i); ++i) {
            if (live && column(i) < a.c) {
                if constexpr (kTogether)
                    R::get(mine + column(i) * sizeof(T), vs + i);
                else if constexpr (V == 1)
                    R::get(slot(stage, i), vs + i);
                else
                    R::get(slot(stage, i), v + i * (V / 2));
            } else {
                for (int j = 0; j < V; ++j) vs[i * V + j] = 0.0f;
            }
        }
        if (!QUANT || a.normalise) {
            float2 s = both(0.0f);
#pragma unroll
            for (int e = 0; e < E / 2 && !unused(e); ++e) s = __fadd2_rn(s, v[e]);
            const float mean = width.share(row_sum<TPR>(s.x + s.y, scratch[parity][0]));
            // Around the mean, and 0 again where the row has no element.
#pragma unroll
            for (int e = 0; e < E / 2 && !unused(e); ++e) v[e] = __fadd2_rn(v[e], both(-mean));
#pragma unroll
            for (int i = 0; i < NI && !past(i); ++i)
                if (column(i) + V > a.c)
                    for (int j = 0; j < V; ++j)
                        if (column(i) + j >= a.c) vs[i * V + j] = 0.0f;
            s = both(0.0f);
#pragma unroll
            for (int e = 0; e < E / 2 && !unused(e); ++e) s = __ffma2_rn(v[e], v[e], s);
            // One rounding of the variance more than a division, and 2 units in the last place of the root: a relative
            // error that the sum over the row has already.
            const float rstd = rsqrtf(row_sum<TPR>(s.x + s.y, scratch[parity][1]) * width.hi + a.eps);
            if (a.stats && lane == 0 && live) {
                a.stats[r] = mean;
                a.stats[a.rows + r] = rstd;
            }
#pragma unroll
            for (int e = 0; e < E / 2 && !unused(e); ++e) v[e] = __ffma2_rn(__fmul2_rn(v[e], both(rstd)), g[e], b[e]);
        }
        if (QUANT) {
            float most = 0.0f;
#pragma unroll
            for (int e = 0; e < E / 2 && !unused(e); ++e) most = most_of(most, v[e].x, v[e].y);
            most = row_most<TPR>(most, scratch[parity][2]);
            float inv;
            const float scale = row_scale_of(__float_as_uint(most), &inv);
            if (lane == 0 && live) a.row_scale[r] = scale;
            // Adding 1.5 * 2^23 leaves a whole number, rounded to nearest even, in the low bits.  The products
            // are scalar: a packed one is joined with the addition into one that rounds once, which tips values
            // next to a half to the other side (seen against the definition's own arithmetic).
            if (scale < __int_as_float(0x7f800000)) {
#pragma unroll
                for (int e = 0; e < E / 2 && !unused(e); ++e)
                    v[e] = __fadd2_rn(make_float2(__fmul_rn(v[e].x, inv), __fmul_rn(v[e].y, inv)), both(12582912.0f));
            } else {
#pragma unroll
                for (int e = 0; e < E / 2 && !unused(e); ++e) v[e] = both(0.0f);
            }
            if (live)
#pragma unroll
                for (int i = 0; i < NI && !past(i); ++i)
                    if (column(i) < a.c) {
                        int q[V];
                        for (int j = 0; j < V; ++j) q[j] = __float_as_int(vs[i * V + j]);
                        store_q<V>(a.q + r * a.q_stride + column(i), q, a.c - column(i));
                    }
        } else if (live) {
            T *y = static_cast<T *>(a.y) + r * a.y_stride;
#pragma unroll
            for (int i = 0; i < NI && !past(i); ++i)
                if (column(i) < a.c) {
                    if constexpr (V == 1)
                        R::store(y + column(i), vs + i);
                    else
                        R::store(y + column(i), v + i * (V / 2));
                }
        }
        if (kTogether && TPR <= 32) __syncwarp();
        stage = stage + 1 == kStages ? 0 : stage + 1;
        parity ^= 1;
    }
    copy_wait<0>();
}

unsigned blocks_for_rows(long long rows) { return (unsigned)(rows < (1LL << 20) ? rows : (1LL << 20)); }

template <typename T, int W, int NI, int TPR>
cudaError_t norm_stream_launch(const NormArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int kBlock = norm_block(TPR), kRows = kBlock / TPR;
    constexpr int kSmem = norm_stages(W) * (W == 2 ? kRows * row_bytes(NI * TPR)
                                                   : NI * kBlock * Run<T, W>::SLOT);
    const long long need = (a.rows + kRows - 1) / kRows, room = (long long)sm_count * (kSmThreads / kBlock);
    const dim3 grid((unsigned)(need < room ? need : room)), block(kBlock);
    static bool allowed[2][kMaxDevices] = {};
    if (kSmem > 46 * 1024) {  // the sums take some of the first 48 KB
        const cudaError_t e = a.q ? allow_dynamic_smem(norm_stream_kernel<T, W, NI, TPR, true>, kSmem, allowed[1])
                                  : allow_dynamic_smem(norm_stream_kernel<T, W, NI, TPR, false>, kSmem, allowed[0]);
        if (e != cudaSuccess) return e;
    }
    return a.q ? launch_overlapped(norm_stream_kernel<T, W, NI, TPR, true>, grid, block, kSmem, stream, 1, a)
               : launch_overlapped(norm_stream_kernel<T, W, NI, TPR, false>, grid, block, kSmem, stream, 1, a);
}

bool aligned_for(const void *p, long long stride, int element, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * element % bytes == 0;
}

// A row gets the fewest threads, a power of two of them, that hold it: more sum over more lanes (bf16,
// 8192x4096 on 256 threads of two vectors each 37 us, on 128 of four 25 us), and a number of warps that only
// the launch knows costs more than it saves (16384x4096 quantised 65 us against 47 us).
template <typename T, int W, int NI>
cudaError_t norm_stream_pick(const NormArgs &a, int sm_count, cudaStream_t stream, bool *done)
{
    constexpr int kHeld = NI * Run<T, W>::V;
    *done = true;
    if (a.c <= 4 * kHeld) return norm_stream_launch<T, W, NI, 4>(a, sm_count, stream);
    if (a.c <= 8 * kHeld) return norm_stream_launch<T, W, NI, 8>(a, sm_count, stream);
    if (a.c <= 16 * kHeld) return norm_stream_launch<T, W, NI, 16>(a, sm_count, stream);
    if (a.c <= 32 * kHeld) return norm_stream_launch<T, W, NI, 32>(a, sm_count, stream);
    if (a.c <= 64 * kHeld) return norm_stream_launch<T, W, NI, 64>(a, sm_count, stream);
    if (a.c <= 128 * kHeld) return norm_stream_launch<T, W, NI, 128>(a, sm_count, stream);
    if (a.c <= 256 * kHeld) return norm_stream_launch<T, W, NI, 256>(a, sm_count, stream);
    if (a.c <= 512 * kHeld) return norm_stream_launch<T, W, NI, 512>(a, sm_count, stream);
    *done = false;
    return cudaSuccess;
}

// 16-bit rows off 16-byte boundaries: 16 elements a thread, or 32 where 128 threads would not hold the row (the
// least that fits is the fastest: f16, 14592x1537 29 / 28, 3001x777 5.8 / 6.2 us with 16 / 32; x2051 58 / 49).
template <typename T>
cudaError_t norm_together_pick(const NormArgs &a, int sm_count, cudaStream_t stream, bool *done)
{
    *done = true;
    if (a.c <= 16 * 4) return norm_stream_launch<T, 2, 16, 4>(a, sm_count, stream);
    if (a.c <= 16 * 8) return norm_stream_launch<T, 2, 16, 8>(a, sm_count, stream);
    if (a.c <= 16 * 16) return norm_stream_launch<T, 2, 16, 16>(a, sm_count, stream);
    if (a.c <= 16 * 32) return norm_stream_launch<T, 2, 16, 32>(a, sm_count, stream);
    if (a.c <= 16 * 64) return norm_stream_launch<T, 2, 16, 64>(a, sm_count, stream);
    if (a.c <= 16 * 128) return norm_stream_launch<T, 2, 16, 128>(a, sm_count, stream);
    if (a.c <= 32 * 128) return norm_stream_launch<T, 2, 32, 128>(a, sm_count, stream);
    if (a.c <= 32 * 256) return norm_stream_launch<T, 2, 32, 256>(a, sm_count, stream);
    // Half of 512 threads have nothing of a row just beyond 8192, which only counts where there are many rows:
    // f16, this / norm_wide_kernel, 64x8193 5.5 / 9.6 us, 14592x8193 227 / 164, 14592x10001 235 / 244, x16001 272 / 362.
    if (a.c <= 32 * 512 && (a.c > 9500 || a.rows <= 1000)) return norm_stream_launch<T, 2, 32, 512>(a, sm_count, stream);
    *done = false;
    return cudaSuccess;
}

template <typename T>
cudaError_t norm_launch_t(const NormArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    const bool wide_loads = a.c % V == 0 && aligned_for(a.x, a.x_stride, sizeof(T), 16) &&
                            (a.q ? aligned_for(a.q, a.q_stride, 1, V) : aligned_for(a.y, a.y_stride, sizeof(T), 16)) &&
                            aligned_for(a.gamma, 0, 4, 16) && aligned_for(a.beta, 0, 4, 16);
    bool done = false;
    cudaError_t e;
    if (wide_loads)
        e = norm_stream_pick<T, 16, 4>(a, sm_count, stream, &done);
    else if constexpr (sizeof(T) == 4)
        e = norm_stream_pick<T, 4, 16>(a, sm_count, stream, &done);
    else
        e = norm_together_pick<T>(a, sm_count, stream, &done);
    if (done) return e;
    return launch_overlapped(norm_wide_kernel<T>, dim3(blocks_for_rows(a.rows)), dim3(kWideThreads), 0, stream, 1, a);
}

// ------------------------------------------------------------------ gradient, rows in registers
// As norm_stream_kernel, for x and dy: each thread keeps gamma and the running sums of dy * h and dy for its
// own columns in registers, so that x and dy are read once for all three gradients.  The two sums over a row
// share one barrier.  At the end the rows of a block are joined in shared memory, and each block writes one
// row of partial sums, which norm_grad_join_kernel adds up in order.  bf16 with the join: 14592x4096 64 us
// (5.6 TB/s), 14592x256 9 us, of which the join and the launches' ends are a third.  Rows off 16-byte
// boundaries: f32 in 4-byte runs, 14592x1536 56 us (4.8 TB/s); bf16 copied together, 14592x1537 41 us (3.2 TB/s),
// bound by its element-wise reads and stores (59 us in 4-byte runs, two of them to a pair).
constexpr int kGradElements = 16;  // of a row per thread: sums, gamma, h and g of more would not fit 128 registers
constexpr int grad_stages(int w) { return w == 2 ? 4 : 3; }
constexpr int grad_block(int tpr) { return tpr < 256 ? 256 : tpr; }

// Sums of two values over the TPR threads of a row; scratch: a float2 for each warp of the block.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 *scratch)
{
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TPR > 32) {
        constexpr int warps = TPR / 32;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) scratch[warp] = v;
        __syncthreads();
        v = both(0.0f);
        for (int i = 0; i < warps; ++i) v = __fadd2_rn(v, scratch[warp / warps * warps + i]);
    }
    return v;
}

template <typename T, int W, int TPR>
__global__ void __launch_bounds__(grad_block(TPR), kSmThreads / grad_block(TPR)) norm_grad_stream_kernel(const GradArgs a)
{
    using R = Run<T, W>;
    constexpr int V = R::V, E = kGradElements, NI = E / V, kBlock = grad_block(TPR), kGroups = kBlock / TPR;
    constexpr int kStages = grad_stages(W);
    constexpr bool kTogether = W == 2;  // as in norm_stream_kernel
    extern __shared__ __align__(16) unsigned char grad_ring[];  // [stage][x, dy][run][thread] slots or [group] rows; then the join
    __shared__ float2 scratch[2][kBlock / 32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * kGroups;
    // As in norm_stream_kernel: f32, 14592x5121 245 -> 210 us.
    constexpr bool kSkips = W != 2;
    auto past = [&](int i) { return kSkips && i > 0 && i * V % (V < 4 ? 4 : V) == 0 && i * TPR * V >= a.c; };
    auto unused = [&](int e) { return kSkips && e > 0 && 2 * e % (V < 4 ? 4 : V) == 0 && 2 * e / V * TPR * V >= a.c; };
    auto column = [&](int i) { return (i * TPR + lane) * V; };
    auto slot = [&](int stage, int which, int i) {
        return grad_ring + (((stage * 2 + which) * NI + i) * kBlock + threadIdx.x) * R::SLOT;
    };
    auto row_ring = [&](int stage, int which) {
        return grad_ring + ((stage * 2 + which) * kGroups + threadIdx.x / TPR) * row_bytes(E * TPR);
    };
    auto x_at = [&](long long r) { return static_cast<const T *>(a.x) + r * a.x_stride; };
    auto dy_at = [&](long long r) { return static_cast<const T *>(a.dy) + r * a.dy_stride; };
    auto fetch = [&](long long r, int stage) {
        if (r < a.rows) {
            const T *x = x_at(r), *dy = dy_at(r);
            if constexpr (kTogether) {
                fetch_row<TPR>(dev::smem_u32(row_ring(stage, 0)), x, a.c, lane);
                fetch_row<TPR>(dev::smem_u32(row_ring(stage, 1)), dy, a.c, lane);
            } else {
                for (int i = 0; i < NI; ++i)
                    if (column(i) < a.c) {
                        R::copy(dev::smem_u32(slot(stage, 0, i)), x + column(i));
                        R::copy(dev::smem_u32(slot(stage, 1, i)), dy + column(i));
                    }
            }
        }
        copy_commit();
    };
    auto moments = [&](long long r) {
        return r < a.rows ? make_float2(__ldg(a.stats + r), __ldg(a.stats + a.rows + r)) : both(0.0f);
    };
    long long r = (long long)blockIdx.x * kGroups + threadIdx.x / TPR;
    for (int s = 0; s < kStages - 1; ++s) fetch(r + s * step, s);
    float2 next = moments(r);
    float2 gamma[E / 2], dg[E / 2], db[E / 2];
    for (int i = 0; i < NI; ++i)
        load_params<V>(a.gamma ? a.gamma + column(i) : nullptr, 1.0f, a.c - column(i),
                       reinterpret_cast<float *>(gamma) + i * V);
    for (int e = 0; e < E / 2; ++e) dg[e] = db[e] = both(0.0f);
    if constexpr (kTogether) {
        copy_wait<kStages - 2>();
        __syncthreads();
    }
    const Width width(a.c);
    int stage = 0, parity = 0;
    for (long long base = (long long)blockIdx.x * kGroups; base < a.rows; base += step, r += step) {
        fetch(r + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        const float mean = next.x, rstd = next.y;
        next = moments(r + step);
        copy_wait<kTogether ? kStages - 2 : kStages - 1>();
        const bool live = r < a.rows;
        const unsigned char *my_x = row_ring(stage, 0) + start_of(x_at(r)), *my_dy = row_ring(stage, 1) + start_of(dy_at(r));
        float2 h[E / 2], g[E / 2];
        float *hs = reinterpret_cast<float *>(h), *gs = reinterpret_cast<float *>(g);
#pragma unroll
        for (int i = 0; i < NI && !past(i); ++i) {
            if (live && column(i) < a.c) {
                if constexpr (kTogether) {
                    R::get(my_x + column(i) * sizeof(T), hs + i);
                    R::get(my_dy + column(i) * sizeof(T), gs + i);
                } else if constexpr (V == 1) {
                    R::get(slot(stage, 0, i), hs + i);
                    R::get(slot(stage, 1, i), gs + i);
                } else {
                    R::get(slot(stage, 0, i), h + i * (V / 2));
                    R::get(slot(stage, 1, i), g + i * (V / 2));
                }
            } else {  // adds nothing anywhere: h and dy are both 0
                for (int j = 0; j < V; ++j) hs[i * V + j] = mean, gs[i * V + j] = 0.0f;
            }
        }
        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int e = 0; e < E / 2 && !unused(e); ++e) {
            const float2 d = g[e];
            h[e] = __fmul2_rn(__fadd2_rn(h[e], both(-mean)), both(rstd));
            dg[e] = __ffma2_rn(d, h[e], dg[e]);
            db[e] = __fadd2_rn(d, db[e]);
            g[e] = __fmul2_rn(d, gamma[e]);
            s1 = __fadd2_rn(s1, g[e]);
            s2 = __ffma2_rn(g[e], h[e], s2);
        }
        const float2 sums = row_sum2<TPR>(make_float2(s1.x + s1.y, s2.x + s2.y), scratch[parity]);
        const float m1 = width.share(sums.x), m2 = width.share(sums.y);
#pragma unroll
        for (int e = 0; e < E / 2 && !unused(e); ++e)
            h[e] = __fmul2_rn(__fadd2_rn(__ffma2_rn(h[e], both(-m2), g[e]), both(-m1)), both(rstd));
        if (live) {
            T *dx = static_cast<T *>(a.dx) + r * a.dx_stride;
#pragma unroll
            for (int i = 0; i < NI && !past(i); ++i)
                if (column(i) < a.c) {
                    if constexpr (V == 1)
                        R::store(dx + column(i), hs + i);
                    else
                        R::store(dx + column(i), h + i * (V / 2));
                }
        }
        if (kTogether && TPR <= 32) __syncwarp();
        stage = stage + 1 == kStages ? 0 : stage + 1;
        parity ^= 1;
    }
    copy_wait<0>();
    float *out = a.partial + (long long)blockIdx.x * 2 * a.c;
    float *dgs = reinterpret_cast<float *>(dg), *dbs = reinterpret_cast<float *>(db);
    if constexpr (kGroups == 1) {
        for (int i = 0; i < NI; ++i)
            for (int j = 0; j < V; ++j)
                if (column(i) + j < a.c) {
                    if constexpr (V >= 4) {
                        if (j % 4 == 0) {
                            const int e = i * V + j;
                            *reinterpret_cast<float4 *>(out + column(i) + j) =
                                make_float4(dgs[e], dgs[e + 1], dgs[e + 2], dgs[e + 3]);
                            *reinterpret_cast<float4 *>(out + a.c + column(i) + j) =
                                make_float4(dbs[e], dbs[e + 1], dbs[e + 2], dbs[e + 3]);
                        }
                    } else {
                        out[column(i) + j] = dgs[i * V + j];
                        out[a.c + column(i) + j] = dbs[i * V + j];
                    }
                }
    } else {
        // The block's rows side by side in shared memory, [row][dgamma, dbeta][element][thread]; those of one
        // warp are joined by shuffles before.
        constexpr int kSide = TPR < 32 ? kBlock / 32 : kGroups;
        for (int o = TPR; o < 32; o <<= 1)
            for (int e = 0; e < E; ++e) {
                dgs[e] += __shfl_xor_sync(0xffffffffu, dgs[e], o);
                dbs[e] += __shfl_xor_sync(0xffffffffu, dbs[e], o);
            }
        float *join = reinterpret_cast<float *>(grad_ring);
        __syncthreads();  // the ring is no longer read
        if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
            float *mine = join + (TPR < 32 ? threadIdx.x / 32 : threadIdx.x / TPR) * (2 * E * TPR) + lane;
            for (int e = 0; e < E; ++e) {
                mine[e * TPR] = dgs[e];
                mine[(E + e) * TPR] = dbs[e];
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

template <typename T, int W, int TPR>
cudaError_t norm_grad_stream_launch(GradArgs a, int sm_count, cudaStream_t stream)
{
    constexpr int kBlock = grad_block(TPR), kRows = kBlock / TPR;
    constexpr int kRing = grad_stages(W) * 2 * (W == 2 ? kRows * row_bytes(kGradElements * TPR)
                                                       : kGradElements / Run<T, W>::V * kBlock * Run<T, W>::SLOT);
    constexpr int kJoin = kRows > 1 ? (TPR < 32 ? kBlock / 32 : kRows) * 2 * kGradElements * TPR * 4 : 0;
    constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    static bool allowed[kMaxDevices] = {};
    if (kSmem > 46 * 1024) {  // the sums of a block take some of the first 48 KB
        cudaError_t e = allow_dynamic_smem(norm_grad_stream_kernel<T, W, TPR>, kSmem, allowed);
        if (e != cudaSuccess) return e;
    }
    const long long need = (a.rows + kRows - 1) / kRows, room = (long long)sm_count * (kSmThreads / kBlock);
    a.partial_rows = (int)(need < room ? need : room);
    cudaError_t e = launch_overlapped(norm_grad_stream_kernel<T, W, TPR>, dim3((unsigned)a.partial_rows), dim3(kBlock),
                                      kSmem, stream, 1, a);
    return e == cudaSuccess ? norm_grad_join(a, stream) : e;
}

template <typename T, int W>
cudaError_t norm_grad_stream_pick(const GradArgs &a, int sm_count, cudaStream_t stream)
{
    if (a.c <= 8 * kGradElements) return norm_grad_stream_launch<T, W, 8>(a, sm_count, stream);
    if (a.c <= 16 * kGradElements) return norm_grad_stream_launch<T, W, 16>(a, sm_count, stream);
    if (a.c <= 32 * kGradElements) return norm_grad_stream_launch<T, W, 32>(a, sm_count, stream);
    if (a.c <= 64 * kGradElements) return norm_grad_stream_launch<T, W, 64>(a, sm_count, stream);
    if (a.c <= 128 * kGradElements) return norm_grad_stream_launch<T, W, 128>(a, sm_count, stream);
    if (a.c <= 256 * kGradElements) return norm_grad_stream_launch<T, W, 256>(a, sm_count, stream);
    return norm_grad_stream_launch<T, W, 512>(a, sm_count, stream);
}

template <typename T>
cudaError_t norm_grad_launch_t(const GradArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    if (a.c <= 512 * kGradElements) {
        const bool wide_loads = a.c % V == 0 && aligned_for(a.x, a.x_stride, sizeof(T), 16) &&
                                aligned_for(a.dy, a.dy_stride, sizeof(T), 16) &&
                                aligned_for(a.dx, a.dx_stride, sizeof(T), 16) && aligned_for(a.gamma, 0, 4, 16);
        return wide_loads ? norm_grad_stream_pick<T, 16>(a, sm_count, stream)
                          : norm_grad_stream_pick<T, sizeof(T) == 4 ? 4 : 2>(a, sm_count, stream);
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

int norm_grad_partial_rows(long long rows, int sm_count)
{
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
