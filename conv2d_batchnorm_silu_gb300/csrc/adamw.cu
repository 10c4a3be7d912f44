// adamw.cu -- the AdamW step of many tensors in one launch, with the moments in fp32 or in 8 bits.
//
//   g' = grad_scale * g,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
//   p = p - (lr decay p + lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps))
//
// in fp32, p rounded once to its own type.  In 8 bits m and sqrt(v) are e4m3 values with one scale for each 256 in a
// row (their largest magnitude / 448): sqrt(v), whose range is half of v's, and a float format, so that small values
// beside a large one keep their relative precision.  They are rounded to one of the two values around them with the
// odds that keep the value's mean: to nearest, a change of less than a sixteenth a step (beta2 = 0.999 changes v by a
// thousandth) would be lost each time.  The odds come from the place and the step alone.  sqrt(v) never becomes 0
// where it was not: m / (0 + eps) would be a step without bounds.  This step itself uses m and v before the rounding.
//
// What that costs: with d the distance of the values around a root r, a step of steady gradients changes the root by
// |c| = (1 - beta2) / 2 r |g^2 / v - 1|, 0.48 (1 - beta2) r on average over normal ones, and its rounding adds |c| d to the
// variance.  v, its square, grows by as much, until it lies above the gradients' own by 0.48 d / r, of which the root's
// variance is half: d / r is a sixteenth to an eighth, so roots spread by 12 to 17 % and v is 3 to 6 % too large, for any
// beta2 near 1 (a restatement over 8000 steps: 16.6 and 5.3).
//
// Measured: 66M fp32 elements with fp32 moments 263 us (7.1 TB/s, memory); 8.3M in 192 bf16 tensors with 8-bit moments
// 28.5 us (3.5 TB/s), bound by some 80 instructions an element, most of them the dither and the rounding to 8 bits, and by
// the host, whose part of such a call is 24 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cbs_internal.h"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = 256;  // elements that share a scale; a warp's work at a time
constexpr int kPerLane = kBlock / 32;
constexpr int kBlocksPerWarp = 1;
constexpr int kChunk = kBlock * kWarps * kBlocksPerWarp;  // elements of a CTA
constexpr float kTiniest = 7.8886090522101181e-31f;       // 2^-100: as for quantised rows
constexpr float kMost8 = 448.0f;                          // of e4m3; no rounding here reaches beyond it

// A tensor as the kernel sees it.
struct Entry {
    void *p;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    long long n;
    unsigned first;      // chunks of the tensors before it
    unsigned char p_type, g_type, wide, unused;
};

template <int N>
struct Table {
    unsigned end[N];  // chunks of a tensor and those before it; the last's in the place of those beyond
    Entry e[N];
};

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float get(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }

// A lane's eight neighbours at once: 32 bytes of fp32, 16 of the 16-bit types, 8 of the 8-bit one.
__device__ __forceinline__ void get8(const float *p, float *v)
{
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void put8(float *p, const float *v)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void get8(const T *p, float *v)
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const T *t = reinterpret_cast<const T *>(&w);
    for (int j = 0; j < 8; ++j) v[j] = get(t + j);
}
template <typename T>
__device__ __forceinline__ void put8(T *p, const float *v)
{
    uint4 w;
    T *t = reinterpret_cast<T *>(&w);
    for (int j = 0; j < 8; ++j) put(t + j, v[j]);
    *reinterpret_cast<uint4 *>(p) = w;
}

// Two 8-bit floats, in the low half of b, to fp32 and back (of values that they hold).
__device__ __forceinline__ float2 from_e4m3(uint32_t b)
{
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)b, __NV_E4M3)));
}
__device__ __forceinline__ uint32_t to_e4m3(float a, float b)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The mixed bits of a place and a step, two numbers of 16 bits: the 32-bit finaliser of Appleby's MurmurHash3.
__device__ __forceinline__ uint32_t dither(uint32_t z)
{
    z = (z ^ (z >> 16)) * 0x85EBCA6Bu;
    z = (z ^ (z >> 13)) * 0xC2B2AE35u;
    return z ^ (z >> 16);
}

// x in [0, 448] to the e4m3 value below it or the one above, by u / 65536 in [0, 1): the three highest bits of the mantissa
// stay, after u has been added to the twenty below.  Below 2^-6, where the format's values are 2^-9 apart, after adding
// 2^-6, which puts that distance there.
__device__ __forceinline__ float eighth(float x, uint32_t u)
{
    const float low = x < 0x1p-6f ? 0x1p-6f : 0.0f;
    return __uint_as_float((__float_as_uint(x + low) + u * 16u) & 0xfff00000u) - low;
}

// A root of 2^-23 and a quotient of 2 units in the last place, which the rounding of p hides or, for fp32, the update's
// smallness.  (IEEE's, with conversions and floors in place of what is above, made 192 tensors with 8-bit moments 43 us.)
__device__ __forceinline__ float root_of(float v)
{
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Largest of the warp's non-negative values, NaN on top.
__device__ __forceinline__ float warp_most(float v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))); }
__device__ __forceinline__ float either_most(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

struct Rates {
    float decay, step_size, inv_root_c2, grad_scale;  // decay: lr * decay
    uint32_t step;
};

// What a step multiplies with, from the host's numbers or the device's.
__device__ __forceinline__ Rates rates_of(const AdamWScalars &s)
{
    Rates r;
    const float lr = s.lr_at ? *s.lr_at : s.lr;
    r.grad_scale = s.grad_scale_at ? *s.grad_scale_at : s.grad_scale;
    float c1 = s.c1, root_c2 = s.root_c2;
    r.step = (uint32_t)s.step;
    if (s.step_at) {  // 1 - beta^t through the logarithm, which the host takes in 64 bits: no difference of near equals
        const long long t = *s.step_at;
        r.step = (uint32_t)t;
        c1 = -expm1f((float)t * s.ln_beta1);
        root_c2 = sqrtf(-expm1f((float)t * s.ln_beta2));
    }
    r.decay = lr * s.decay;
    r.step_size = lr / c1;
    r.inv_root_c2 = 1.0f / root_c2;
    return r;
}

// 256 elements from `at` on by one warp.  WIDE: all there, a lane's eight side by side; else a lane's are 32 apart.
template <typename P, typename G, bool EIGHT, bool WIDE>
__device__ __forceinline__ void step_block(const Entry &e, long long at, const AdamWScalars &s, const Rates &r)
{
    const int lane = threadIdx.x & 31;
    const int have = WIDE ? kBlock : (int)(e.n - at < kBlock ? e.n - at : kBlock);
    auto place = [&](int j) { return WIDE ? lane * kPerLane + j : j * 32 + lane; };
    P *p_at = static_cast<P *>(e.p) + at;
    const G *g_at = static_cast<const G *>(e.g) + at;
    float p[kPerLane], g[kPerLane], m[kPerLane], v[kPerLane];
    if constexpr (WIDE) {
        get8(p_at + place(0), p);
        get8(g_at + place(0), g);
    } else {
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            p[j] = place(j) < have ? get(p_at + place(j)) : 0.0f;
            g[j] = place(j) < have ? get(g_at + place(j)) : 0.0f;
        }
    }
    if constexpr (EIGHT) {
        const uint8_t *m_at = static_cast<const uint8_t *>(e.m) + at, *v_at = static_cast<const uint8_t *>(e.v) + at;
        const float ms = e.m_scale[at / kBlock], vs = e.v_scale[at / kBlock];
        uint32_t mb[kPerLane / 2], vb[kPerLane / 2];  // pairs
        if constexpr (WIDE) {
            const uint2 mw = *reinterpret_cast<const uint2 *>(m_at + place(0)), vw = *reinterpret_cast<const uint2 *>(v_at + place(0));
            mb[0] = mw.x, mb[1] = mw.x >> 16, mb[2] = mw.y, mb[3] = mw.y >> 16;
            vb[0] = vw.x, vb[1] = vw.x >> 16, vb[2] = vw.y, vb[3] = vw.y >> 16;
        } else {
            auto pair = [&](const uint8_t *b, int j) {
                return (place(j) < have ? b[place(j)] : 0u) | (place(j + 1) < have ? b[place(j + 1)] : 0u) << 8;
            };
#pragma unroll
            for (int j = 0; j < kPerLane / 2; ++j) {
                mb[j] = pair(m_at, 2 * j);
                vb[j] = pair(v_at, 2 * j);
            }
        }
#pragma unroll
        for (int j = 0; j < kPerLane / 2; ++j) {
            const float2 mm = __fmul2_rn(from_e4m3(mb[j] & 0xffffu), make_float2(ms, ms));
            const float2 vv = __fmul2_rn(from_e4m3(vb[j] & 0xffffu), make_float2(vs, vs)), square = __fmul2_rn(vv, vv);
            m[2 * j] = mm.x, m[2 * j + 1] = mm.y;
            v[2 * j] = square.x, v[2 * j + 1] = square.y;
        }
    } else {
        const float *m_at = static_cast<const float *>(e.m) + at, *v_at = static_cast<const float *>(e.v) + at;
        if constexpr (WIDE) {
            get8(m_at + place(0), m);
            get8(v_at + place(0), v);
        } else {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) {
                m[j] = place(j) < have ? m_at[place(j)] : 0.0f;
                v[j] = place(j) < have ? v_at[place(j)] : 0.0f;
            }
        }
    }
    float root[kPerLane];
    auto both = [](float v) { return make_float2(v, v); };
#pragma unroll
    for (int j = 0; j < kPerLane; j += 2) {  // two to an instruction
        const float2 gj = __fmul2_rn(make_float2(g[j], g[j + 1]), both(r.grad_scale));
        const float2 mj = __ffma2_rn(make_float2(m[j], m[j + 1]), both(s.beta1), __fmul2_rn(gj, both(s.rest1)));
        const float2 vj = __ffma2_rn(make_float2(v[j], v[j + 1]), both(s.beta2), __fmul2_rn(__fmul2_rn(gj, both(s.rest2)), gj));
        m[j] = mj.x, m[j + 1] = mj.y;
        v[j] = vj.x, v[j + 1] = vj.y;
        root[j] = root_of(vj.x), root[j + 1] = root_of(vj.y);
        const float2 under = __ffma2_rn(make_float2(root[j], root[j + 1]), both(r.inv_root_c2), both(s.eps));
        const float2 over = __fmul2_rn(mj, both(r.step_size));
        // What p loses, decay and update, before it is taken away: 1 - lr decay would round the decay itself to multiples of
        // 2^-24, for each element and step the same way (lr decay = 1e-7: by a fifth).
        const float2 loss = __ffma2_rn(make_float2(p[j], p[j + 1]), both(r.decay),
                                       make_float2(__fdividef(over.x, under.x), __fdividef(over.y, under.y)));
        p[j] -= loss.x, p[j + 1] -= loss.y;
    }
    if constexpr (WIDE) {
        put8(p_at + place(0), p);
    } else {
#pragma unroll
        for (int j = 0; j < kPerLane; ++j)
            if (place(j) < have) put(p_at + place(j), p[j]);
    }
    if constexpr (EIGHT) {
        float most_m = 0.0f, most_v = 0.0f;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            most_m = either_most(most_m, fabsf(m[j]));
            most_v = either_most(most_v, root[j]);
        }
        most_m = warp_most(most_m);
        most_v = warp_most(most_v);
        if (most_m < kTiniest) most_m = kTiniest;
        if (most_v < kTiniest) most_v = kTiniest;
        const float inv_m = kMost8 / most_m, inv_v = kMost8 / most_v;
        float mh[kPerLane], vh[kPerLane];
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            const uint32_t u = dither((uint32_t)(at + place(j)) + r.step * 0x9E3779B9u);
            mh[j] = copysignf(eighth(fabsf(m[j]) * inv_m, u >> 16), m[j]);
            // 2^-9 at least where the root is not 0: its least, 2^-75, times 2^100 is more.
            vh[j] = fmaxf(eighth(root[j] * inv_v, u & 0xffffu), fminf(root[j] * 0x1p100f, 0x1p-9f));
        }
        uint8_t *m_at = static_cast<uint8_t *>(e.m) + at, *v_at = static_cast<uint8_t *>(e.v) + at;
        uint32_t mb[kPerLane / 2], vb[kPerLane / 2];
#pragma unroll
        for (int j = 0; j < kPerLane / 2; ++j) {
            mb[j] = to_e4m3(mh[2 * j], mh[2 * j + 1]);
            vb[j] = to_e4m3(vh[2 * j], vh[2 * j + 1]);
        }
        if constexpr (WIDE) {
            *reinterpret_cast<uint2 *>(m_at + place(0)) = make_uint2(mb[0] | mb[1] << 16, mb[2] | mb[3] << 16);
            *reinterpret_cast<uint2 *>(v_at + place(0)) = make_uint2(vb[0] | vb[1] << 16, vb[2] | vb[3] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j)
                if (place(j) < have) {
                    m_at[place(j)] = (uint8_t)(mb[j / 2] >> j % 2 * 8);
                    v_at[place(j)] = (uint8_t)(vb[j / 2] >> j % 2 * 8);
                }
        }
        if (lane == 0) {  // after every lane's reading of the old ones: the reductions above
            e.m_scale[at / kBlock] = most_m / kMost8;
            e.v_scale[at / kBlock] = most_v / kMost8;
        }
    } else {
        float *m_at = static_cast<float *>(e.m) + at, *v_at = static_cast<float *>(e.v) + at;
        if constexpr (WIDE) {
            put8(m_at + place(0), m);
            put8(v_at + place(0), v);
        } else {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j)
                if (place(j) < have) {
                    m_at[place(j)] = m[j];
                    v_at[place(j)] = v[j];
                }
        }
    }
}

template <typename P, typename G, bool EIGHT>
__device__ __forceinline__ void step_chunk(const Entry &e, long long chunk, const AdamWScalars &s, const Rates &r)
{
    for (int b = 0; b < kBlocksPerWarp; ++b) {
        const long long at = chunk * kChunk + (b * kWarps + threadIdx.x / 32) * kBlock;
        if (at >= e.n) return;
        if (e.wide && at + kBlock <= e.n)
            step_block<P, G, EIGHT, true>(e, at, s, r);
        else
            step_block<P, G, EIGHT, false>(e, at, s, r);
    }
}

template <bool EIGHT, int N>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<N> table, const int count,
                                                         const __grid_constant__ AdamWScalars s)
{
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    // As many tensors end at or before this chunk as come before its own: all ends looked at at once, where a search by
    // halves waits for the parameters' memory each time.
    int mine = 0;
#pragma unroll
    for (int i = 0; i < N; i += kThreads)
        mine += __syncthreads_count(i + (int)threadIdx.x < count && table.end[i + threadIdx.x < N ? i + threadIdx.x : N - 1] <= blockIdx.x);
    const Entry &e = table.e[mine];
    const long long chunk = blockIdx.x - e.first;
    const Rates r = rates_of(s);
    switch (e.p_type * 3 + e.g_type) {
    case kF32 * 3 + kF32: return step_chunk<float, float, EIGHT>(e, chunk, s, r);
    case kF32 * 3 + kBf16: return step_chunk<float, __nv_bfloat16, EIGHT>(e, chunk, s, r);
    case kF32 * 3 + kF16: return step_chunk<float, __half, EIGHT>(e, chunk, s, r);
    case kBf16 * 3 + kF32: return step_chunk<__nv_bfloat16, float, EIGHT>(e, chunk, s, r);
    case kBf16 * 3 + kBf16: return step_chunk<__nv_bfloat16, __nv_bfloat16, EIGHT>(e, chunk, s, r);
    case kBf16 * 3 + kF16: return step_chunk<__nv_bfloat16, __half, EIGHT>(e, chunk, s, r);
    case kF16 * 3 + kF32: return step_chunk<__half, float, EIGHT>(e, chunk, s, r);
    case kF16 * 3 + kBf16: return step_chunk<__half, __nv_bfloat16, EIGHT>(e, chunk, s, r);
    default: return step_chunk<__half, __half, EIGHT>(e, chunk, s, r);
    }
}

template <int N>
cudaError_t launch_table(const Entry *entries, int count, const AdamWScalars &s, bool eight, cudaStream_t stream)
{
    Table<N> table;
    unsigned end = 0;
    for (int i = 0; i < N; ++i) {
        if (i < count) {
            table.e[i] = entries[i];
            end = entries[i].first + (unsigned)((entries[i].n + kChunk - 1) / kChunk);
        }
        table.end[i] = end;
    }
    const dim3 grid(end), block(kThreads);
    return eight ? launch_overlapped(adamw_kernel<true, N>, grid, block, 0, stream, 1, table, count, s)
                 : launch_overlapped(adamw_kernel<false, N>, grid, block, 0, stream, 1, table, count, s);
}

// As many tensors as a launch's parameters hold (32,764 bytes).  A launch carries its whole table, so that fewer tensors go
// in smaller ones, of half as many among them (192 tensors: 33.4 us of the host's time a call, in the whole one 35.3).
constexpr int kMostEntries = 440;

}  // namespace

cudaError_t adamw_launch(const AdamWTensor *tensors, int count, const AdamWScalars &s, bool eight, cudaStream_t stream)
{
    Entry entries[kMostEntries];
    int held = 0;
    long long chunks = 0;
    auto flush = [&]() {
        cudaError_t e = cudaSuccess;
        if (held) {
            e = held <= 8     ? launch_table<8>(entries, held, s, eight, stream)
                : held <= 64  ? launch_table<64>(entries, held, s, eight, stream)
                : held <= kMostEntries / 2 ? launch_table<kMostEntries / 2>(entries, held, s, eight, stream)
                              : launch_table<kMostEntries>(entries, held, s, eight, stream);
        }
        held = 0;
        chunks = 0;
        return e;
    };
    for (int i = 0; i < count; ++i) {
        const AdamWTensor &t = tensors[i];
        if (t.n == 0) continue;
        const long long need = (t.n + kChunk - 1) / kChunk;
        if (held == kMostEntries || chunks + need > 0x7fffffffLL) {
            const cudaError_t e = flush();
            if (e != cudaSuccess) return e;
        }
        auto aligned = [](const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
        Entry &e = entries[held++];
        e.p = t.p;
        e.g = t.g;
        e.m = t.m;
        e.v = t.v;
        e.m_scale = t.m_scale;
        e.v_scale = t.v_scale;
        e.n = t.n;
        e.first = (unsigned)chunks;
        chunks += need;
        e.p_type = (unsigned char)t.p_type;
        e.g_type = (unsigned char)t.g_type;
        e.wide = aligned(t.p, 8 * dtype_size(t.p_type)) && aligned(t.g, 8 * dtype_size(t.g_type)) &&
                 aligned(t.m, eight ? 8 : 32) && aligned(t.v, eight ? 8 : 32);
        e.unused = 0;
    }
    return flush();
}

}  // namespace cbs
