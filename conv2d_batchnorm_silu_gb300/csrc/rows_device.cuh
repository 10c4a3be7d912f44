// rows_device.cuh -- rows of activations held in registers: their copies through shared memory, sums
// over the threads of a row, and quantisation; shared by the norms (layer_norm.cu, rms_norm.cu).
#pragma once

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

// Threads of a block: one row, or as many as 128 threads hold while a row stays within a warp.
constexpr int norm_block(int tpr) { return tpr <= 32 ? 128 : tpr; }
constexpr int kSmThreads = 512;  // on an SM: 128 registers a thread

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

inline unsigned blocks_for_rows(long long rows) { return (unsigned)(rows < (1LL << 20) ? rows : (1LL << 20)); }

inline bool aligned_for(const void *p, long long stride, int element, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * element % bytes == 0;
}

}  // namespace
}  // namespace cbs
