// adapters_device.cuh -- kernels of the low-rank adapters, for one element type (adapters.cu has the formulas).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "adapters.h"
#include "cbs_internal.h"
#include "ptx.cuh"

namespace cbs {
namespace {

// ------------------------------------------------------------------ matrix instructions
// A warp's m16n8 product.  Lane l has g = l / 4 and t = l % 4; of the first operand it holds rows g and g + 8, of the
// second column g, both at the K positions of t, and of the result rows g and g + 8 at columns 2t and 2t + 1.  Which
// elements stand at t's positions is free as long as both operands agree: here neighbours in memory, eight of a
// 32-element step (four of 16 for the second product), so that both operands come by wide loads from where they lie.
__device__ __forceinline__ void mma16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                      __nv_bfloat16)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                      __half)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma16_first(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                            __nv_bfloat16)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma16_first(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                            __half)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// fp32 as the sum of two of the instruction's 19-bit floats, to 2^-22 of it.
struct Parts {
    uint32_t hi, lo;
};
__device__ __forceinline__ Parts parts_of(float v)
{
    Parts p;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(p.hi) : "f"(v));
    // Of infinities and NaN the first part alone: their difference with themselves would be NaN.
    const float rest = fabsf(v) < __int_as_float(0x7f800000) ? v - __uint_as_float(p.hi) : 0.0f;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(p.lo) : "f"(rest));
    return p;
}
// The same with both operands in two parts: three products, without that of the small parts.
__device__ __forceinline__ void mma8_parts(float *c, Parts a0, Parts a1, Parts a2, Parts a3, Parts b0, Parts b1)
{
    mma8(c, a0.lo, a1.lo, a2.lo, a3.lo, b0.hi, b1.hi);
    mma8(c, a0.hi, a1.hi, a2.hi, a3.hi, b0.lo, b1.lo);
    mma8(c, a0.hi, a1.hi, a2.hi, a3.hi, b0.hi, b1.hi);
}

// ------------------------------------------------------------------ neighbours in memory
__device__ __forceinline__ float widened(float v) { return v; }
__device__ __forceinline__ float widened(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widened(__half v) { return __half2float(v); }
__device__ __forceinline__ void narrowed(float v, float *out) { *out = v; }
__device__ __forceinline__ void narrowed(float v, __nv_bfloat16 *out) { *out = __float2bfloat16_rn(v); }
__device__ __forceinline__ void narrowed(float v, __half *out) { *out = __float2half_rn(v); }

__device__ __forceinline__ uint32_t packed(float a, float b, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t packed(float a, float b, __half)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// N neighbours: words of two for the 16-bit types.
template <typename T, int N>
struct Near {
    uint32_t w[N / 2];
    __device__ __forceinline__ float at(int i) const { return widened(reinterpret_cast<const T *>(w)[i]); }
};
template <int N>
struct Near<float, N> {
    float w[N];
    __device__ __forceinline__ float at(int i) const { return w[i]; }
};

// A load of what nothing writes while the kernel runs, or of what the same thread writes afterwards.
template <bool KEPT, typename W>
__device__ __forceinline__ W load(const W *p)
{
    if constexpr (KEPT) return __ldg(p);
    else return *p;
}

// `have` of N neighbours from p on (none where it is 0 or less), zeros in the place of the others.  WIDE: N or none,
// on a boundary of their size (16 bytes at most).
template <bool WIDE, typename T, int N, bool KEPT = true>
__device__ __forceinline__ Near<T, N> near(const T *p, int have)
{
    Near<T, N> v;
    constexpr int kBytes = N * (int)sizeof(T);
    if constexpr (WIDE) {
        uint32_t *w = reinterpret_cast<uint32_t *>(v.w);
        if (have > 0) {
            if constexpr (kBytes >= 16) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i) {
                    const uint4 u = load<KEPT>(reinterpret_cast<const uint4 *>(p) + i);
                    w[4 * i] = u.x;
                    w[4 * i + 1] = u.y;
                    w[4 * i + 2] = u.z;
                    w[4 * i + 3] = u.w;
                }
            } else if constexpr (kBytes == 8) {
                const uint2 u = load<KEPT>(reinterpret_cast<const uint2 *>(p));
                w[0] = u.x;
                w[1] = u.y;
            } else {
                w[0] = load<KEPT>(reinterpret_cast<const uint32_t *>(p));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) w[i] = 0;
        }
    } else {
        T *out = reinterpret_cast<T *>(v.w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            T e;
            narrowed(0.0f, &e);
            if (i < have) e = p[i];
            out[i] = e;
        }
    }
    return v;
}

__device__ __forceinline__ void store_piece(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, bool there)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n @p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n}" ::"l"(p), "r"(a), "r"(b),
                 "r"(c), "r"(d), "r"((int)there)
                 : "memory");
}

template <bool WIDE, typename T>
__device__ __forceinline__ void store_near(T *p, const float *v, int have)
{
    if constexpr (WIDE) {
        if constexpr (sizeof(T) == 4) {
            store_piece(p, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]), have > 0);
            store_piece(p + 4, __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]), have > 0);
        } else {
            store_piece(p, packed(v[0], v[1], T()), packed(v[2], v[3], T()), packed(v[4], v[5], T()), packed(v[6], v[7], T()), have > 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < have) narrowed(v[i], p + i);
    }
}

// 32 elements of K: rows g (lo) and g + 8 (hi), column g, eight neighbours a lane.
template <typename T>
__device__ __forceinline__ void mma_eight(float *c, const Near<T, 8> &lo, const Near<T, 8> &hi, const Near<T, 8> &col)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            mma8_parts(c, parts_of(lo.w[2 * s]), parts_of(hi.w[2 * s]), parts_of(lo.w[2 * s + 1]), parts_of(hi.w[2 * s + 1]),
                       parts_of(col.w[2 * s]), parts_of(col.w[2 * s + 1]));
    } else {
        mma16(c, lo.w[0], hi.w[0], lo.w[1], hi.w[1], col.w[0], col.w[1], T());
        mma16(c, lo.w[2], hi.w[2], lo.w[3], hi.w[3], col.w[2], col.w[3], T());
    }
}
// 16 elements of K, four neighbours a lane.
template <typename T>
__device__ __forceinline__ void mma_four(float *c, const Near<T, 4> &lo, const Near<T, 4> &hi, const Near<T, 4> &col)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            mma8_parts(c, parts_of(lo.w[2 * s]), parts_of(hi.w[2 * s]), parts_of(lo.w[2 * s + 1]), parts_of(hi.w[2 * s + 1]),
                       parts_of(col.w[2 * s]), parts_of(col.w[2 * s + 1]));
    } else {
        mma16(c, lo.w[0], hi.w[0], lo.w[1], hi.w[1], col.w[0], col.w[1], T());
    }
}

// 16 elements of K, or 8 in fp32, by the operands' registers; `first`: instead of adding to c.
template <typename T, typename W>
__device__ __forceinline__ void mma_quad(float *c, uint4 a, W b0, W b1, bool first)
{
    if constexpr (sizeof(T) == 4) {
        if (first) c[0] = c[1] = c[2] = c[3] = 0.0f;
        mma8_parts(c, parts_of(__uint_as_float(a.x)), parts_of(__uint_as_float(a.y)), parts_of(__uint_as_float(a.z)),
                   parts_of(__uint_as_float(a.w)), parts_of(b0), parts_of(b1));
    } else if (first) {
        mma16_first(c, a.x, a.y, a.z, a.w, b0, b1, T());
    } else {
        mma16(c, a.x, a.y, a.z, a.w, b0, b1, T());
    }
}

// Neighbours from shared memory, on a boundary of their size (16 bytes at most).
template <typename T, int N>
__device__ __forceinline__ void from_shared(uint32_t p, Near<T, N> *v)
{
    constexpr int kBytes = N * (int)sizeof(T);
    uint32_t *w = reinterpret_cast<uint32_t *>(v->w);
    if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                         : "r"(p + 16 * i));
    } else if constexpr (kBytes == 8) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
    } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(p));
    }
}

// What a row's N values of this lane are multiplied with before they are rounded to f16, whose range the sums may
// leave: a power of two that takes the row's largest, over the four lanes that share it, to [1, 2).  *s takes its
// inverse.
template <typename T, int N>
__device__ __forceinline__ float narrow_factor(const float *v, float *s)
{
    if constexpr (!__is_same(T, __half)) return 1.0f;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) most = fmaxf(most, fabsf(v[i]));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    int e = (int)(__float_as_uint(most) >> 23);  // 127 + its exponent; 255 where it is infinite
    e = e < 2 ? 2 : e > 252 ? 252 : e;
    *s *= __uint_as_float((unsigned)e << 23);
    return __uint_as_float((unsigned)(254 - e) << 23);
}

// Parts of a hidden row in the second product: 16-bit activations' type holds it in two, to 2^-16 of bf16 and 2^-22 of
// f16 values.
template <typename T>
constexpr int hidden_parts() { return sizeof(T) == 4 ? 1 : 2; }

// N rows of N neighbours -> for each neighbour the N values of its rows, as the second operand wants them.
template <typename T, int K, int N>
__device__ __forceinline__ void turned(const Near<T, N> (&rows)[K], Near<T, K> (&out)[N])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < K; ++i) out[j].w[i] = rows[i].w[j];
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < K / 2; ++i)
                out[j].w[i] = __byte_perm(rows[2 * i].w[j / 2], rows[2 * i + 1].w[j / 2], j % 2 ? 0x7632 : 0x5410);
    }
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t v;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(v));
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float4 load_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// ------------------------------------------------------------------ y = base + s (x W1) W2
// A cluster takes a tile of 16 rows of one adapter.  Its CTAs share K for the first product and the output's columns
// for the second; in between the partial sums [rows][rank] are added up through the cluster's shared memory, in the
// same order by every CTA.  So x, base, y and, per tile, the weights go by once, and nothing goes through memory in
// between.  Operands are loaded from where they lie into the registers that the instruction wants, so a tile is a few
// loads, the exchange and a few stores: latency bounds it.  bf16, 4096x4096, rank 16: one row 4.5 us of GPU time, 128
// rows of 64 adapters 8.5 (17 MB), 256 rows of 4 adapters 9; rank 64, 128 rows of 64 adapters 19.7.
// (One CTA a tile: one row 14.4 us, 128 rows 17.8.  The second product's weights and base prefetched into L2 during the
// first: 9.4 -> 10.0.)
template <int RT>
constexpr int hidden_pitch() { return RT == 1 ? 16 : 16 * RT + 16; }  // floats; 16-byte reads without bank conflicts
template <int RT, int WM>
constexpr int adapter_smem()
{
    constexpr int kRows = 16 * WM, kK = kAdapterThreads / 32 / WM;
    return (kK + 1) * kRows * hidden_pitch<RT>() * 4;
}

template <typename T, int RT, int WM, bool TURNED, bool WIDE>
__global__ void __launch_bounds__(kAdapterThreads, RT <= 2 || (RT == 4 && sizeof(T) == 2) ? 2 : 1) adapter_products_kernel(const AdapterArgs a)
{
    constexpr int kRows = 16 * WM, kWarps = kAdapterThreads / 32, kSplit = kWarps / WM, kPitch = hidden_pitch<RT>();
    extern __shared__ __align__(16) float adapter_sums[];  // [kSplit][kRows][kPitch] partial sums, then [kRows][kPitch] whole ones
    __shared__ int rows[kRows];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int part = (int)dev::cluster_ctarank(), parts = (int)cluster_size();
    const int tile = (int)blockIdx.x / parts;
    int adapter, count;
    if (a.tiles) {
        if (tile >= *a.tile_count) return;
        const AdapterTile my = a.tiles[tile];
        adapter = my.adapter;
        count = my.count;
        if ((int)threadIdx.x < count) rows[threadIdx.x] = a.order[my.first + threadIdx.x];
    } else if (a.counted) {
        // Up to 1024 rows of few adapters: every CTA counts them all, for each adapter and 32 rows, and finds its tile.
        __shared__ int counts[32][kCountedBins];
        __shared__ int totals[kCountedBins];
        __shared__ int mine[3];  // adapter, first of its rows, rows
        const int bins = a.adapters + 1;
        int of[4], before[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = j * kAdapterThreads + (int)threadIdx.x;
            const int v = i < a.m ? a.index[i] : -1;
            of[j] = i >= a.m ? -1 : v < 0 || v >= a.adapters ? a.adapters : v;
        }
        for (int i = threadIdx.x; i < 32 * kCountedBins; i += kAdapterThreads) counts[i / kCountedBins][i % kCountedBins] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned same = __match_any_sync(0xffffffffu, of[j]);
            before[j] = __popc(same & ((1u << lane) - 1));
            if (of[j] >= 0 && before[j] == 0) counts[j * kWarps + warp][of[j]] = __popc(same);
        }
        __syncthreads();
        if ((int)threadIdx.x < bins) {
            int c[32], sum = 0;
#pragma unroll
            for (int w = 0; w < 32; ++w) c[w] = counts[w][threadIdx.x];
#pragma unroll
            for (int w = 0; w < 32; ++w) {
                counts[w][threadIdx.x] = sum;
                sum += c[w];
            }
            totals[threadIdx.x] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            int left = tile;  // tiles of the adapters from here on that come before this one
            for (int b0 = 0; b0 < bins; b0 += 32) {
                const int total = b0 + lane < bins ? totals[b0 + lane] : 0, tiles = (total + kRows - 1) / kRows;
                int upto = tiles;
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                if (left >= 0 && left >= upto - tiles && left < upto) {
                    mine[0] = b0 + lane;
                    mine[1] = (left - (upto - tiles)) * kRows;
                    mine[2] = total;
                }
                left -= __shfl_sync(0xffffffffu, upto, 31);
            }
            if (lane == 0 && left >= 0) mine[0] = -1;  // one more than there are
        }
        __syncthreads();
        adapter = mine[0];
        if (adapter < 0) return;
        const int first = mine[1];
        count = mine[2] - first < kRows ? mine[2] - first : kRows;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int rank = of[j] == adapter ? counts[j * kWarps + warp][adapter] + before[j] - first : -1;
            if (rank >= 0 && rank < kRows) rows[rank] = j * kAdapterThreads + (int)threadIdx.x;
        }
    } else {
        // Few rows: a cluster for each.  Those whose row is the first, or the 17th and so on, of its adapter take it and
        // the next ones of the adapter; the others have nothing to do.
        __shared__ int before_warp[kWarps];
        auto of = [&](int i) {
            const int v = a.index[i];
            return v < 0 || v >= a.adapters ? a.adapters : v;
        };
        adapter = of(tile);
        const int i = threadIdx.x;
        const bool same = i < a.m && of(i) == adapter;
        const int before = __syncthreads_count(same && i < tile);
        if (before % kRows != 0) return;
        const unsigned mine = __ballot_sync(0xffffffffu, same && i >= tile);
        if (lane == 0) before_warp[warp] = __popc(mine);
        __syncthreads();
        int rank = __popc(mine & ((1u << lane) - 1));
        count = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) rank += before_warp[w];
            count += before_warp[w];
        }
        if (same && i >= tile && rank < kRows) rows[rank] = i;
        count = count < kRows ? count : kRows;
    }
    __syncthreads();
    const bool live = adapter < a.adapters;
    const int wm = warp % WM, ws = warp / WM;
    const int row_lo = 16 * wm + g, row_hi = row_lo + 8;
    const bool has_lo = row_lo < count, has_hi = row_hi < count;
    const long long at_lo = has_lo ? rows[row_lo] : 0, at_hi = has_hi ? rows[row_hi] : 0;
    float *whole = adapter_sums + kSplit * kRows * kPitch;

    if (live) {
        const T *x_lo = static_cast<const T *>(a.x) + at_lo * a.x_stride, *x_hi = static_cast<const T *>(a.x) + at_hi * a.x_stride;
        const T *w1 = static_cast<const T *>(a.w1) + (long long)adapter * a.rank * a.k;
        float acc[2 * RT][4] = {};
        const int steps = (a.k + 31) / 32, from = (int)((long long)steps * part / parts), to = (int)((long long)steps * (part + 1) / parts);
        // This warp's rows may all be beyond the tile's.
        if (16 * wm < count) {
#pragma unroll(RT <= 2 ? 2 : 1)
            for (int s = from + ws; s < to; s += kSplit) {
                const int k0 = 32 * s + 8 * t, have = a.k - k0;
                const Near<T, 8> lo = near<WIDE, T, 8>(x_lo + k0, has_lo ? have : 0);
                const Near<T, 8> hi = near<WIDE, T, 8>(x_hi + k0, has_hi ? have : 0);
                if constexpr (!TURNED) {
                    // W1 is [rank][k]: column j's values are neighbours.
#pragma unroll
                    for (int j = 0; j < 2 * RT; ++j) {
                        const int r = 8 * j + g;
                        mma_eight<T>(acc[j], lo, hi, near<WIDE, T, 8>(w1 + (long long)r * a.k + k0, r < a.rank ? have : 0));
                    }
                } else {
                    // W1 is [k][rank]: a lane loads its columns' neighbours in its eight rows, and turns them.
                    constexpr int kC = 2 * RT < 8 ? 2 * RT : 8;  // columns at a time
#pragma unroll
                    for (int c = 0; c < 2 * RT; c += kC) {
                        const int r = 2 * RT * g + c;
                        Near<T, kC> in[8];
                        Near<T, 8> col[kC];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            in[i] = near<WIDE, T, kC>(w1 + (long long)(k0 + i) * a.rank + r, i < have ? a.rank - r : 0);
                        turned<T, 8, kC>(in, col);
#pragma unroll
                        for (int j = 0; j < kC; ++j) mma_eight<T>(acc[c + j], lo, hi, col[j]);
                    }
                }
            }
        }
        float *mine = adapter_sums + (ws * kRows + 16 * wm) * kPitch;
#pragma unroll
        for (int j = 0; j < 2 * RT; ++j) {
            const int r0 = TURNED ? 2 * RT * (2 * t) + j : 8 * j + 2 * t, r1 = TURNED ? 2 * RT * (2 * t + 1) + j : r0 + 1;
            mine[g * kPitch + r0] = acc[j][0];
            mine[g * kPitch + r1] = acc[j][1];
            mine[(g + 8) * kPitch + r0] = acc[j][2];
            mine[(g + 8) * kPitch + r1] = acc[j][3];
        }
        __syncthreads();
        constexpr int kQuads = 4 * RT;  // of a row
        if constexpr (kSplit > 1) {
            for (int i = threadIdx.x; i < kRows * kQuads; i += kAdapterThreads) {
                float4 *at = reinterpret_cast<float4 *>(adapter_sums + i / kQuads * kPitch) + i % kQuads;
                float4 v = *at;
                for (int s = 1; s < kSplit; ++s) {
                    const float4 u = at[s * kRows * kPitch / 4];
                    v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                }
                *at = v;
            }
        }
        cluster_arrive();
        cluster_wait();
        const uint32_t sums = dev::smem_u32(adapter_sums);
        for (int i = threadIdx.x; i < kRows * kQuads; i += kAdapterThreads) {
            const int offset = i / kQuads * kPitch + i % kQuads * 4;
            float4 v = load_cluster(dev::mapa_cluster(sums + 4 * offset, 0));
            for (int p = 1; p < parts; ++p) {
                const float4 u = load_cluster(dev::mapa_cluster(sums + 4 * offset, (uint32_t)p));
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            *reinterpret_cast<float4 *>(whole + offset) = v;
        }
        __syncthreads();
        cluster_arrive();  // nobody leaves before all have read its sums: waited for at the end
    }
    if (a.hidden) {
        for (int i = threadIdx.x; i < count * a.rank; i += kAdapterThreads) {
            const int row = i / a.rank;
            if (row % parts == part)
                a.hidden[(long long)rows[row] * a.rank + i % a.rank] = live ? whole[row * kPitch + i % a.rank] : 0.0f;
        }
    }
    if (16 * wm < count && (live || a.base != a.y)) {
        // Rows of the first operand.  16-bit: in two parts of the activations' type, f16, whose range the sums may leave,
        // after division by a power of two near the row's largest.
        constexpr int kParts = hidden_parts<T>();
        Near<T, 4> h_lo[kParts][RT], h_hi[kParts][RT];
        float s_lo = live ? (a.scale ? a.scale[adapter] : 1.0f) : 0.0f, s_hi = s_lo;
        if (live) {
            auto take = [&](int row, auto &h, float *s) {
                float v[RT][4];
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float4 u = *reinterpret_cast<const float4 *>(whole + row * kPitch + 16 * i + 4 * t);
                    v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
                }
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int i = 0; i < RT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) h[0][i].w[j] = v[i][j];
                } else {
                    const float factor = narrow_factor<T, 4 * RT>(&v[0][0], s);
#pragma unroll
                    for (int i = 0; i < RT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[i][j] *= factor;
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            h[part][i].w[0] = packed(v[i][0], v[i][1], T());
                            h[part][i].w[1] = packed(v[i][2], v[i][3], T());
                            // What is left; of infinities and NaN nothing, as their difference with themselves is NaN.
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                v[i][j] = fabsf(v[i][j]) < __int_as_float(0x7f800000) ? v[i][j] - h[part][i].at(j) : 0.0f;
                        }
                }
            };
            take(row_lo, h_lo, &s_lo);
            take(row_hi, h_hi, &s_hi);
        }
        const T *w2 = static_cast<const T *>(a.w2) + (live ? (long long)adapter * a.rank * a.n : 0);
        const T *b_lo = static_cast<const T *>(a.base) + at_lo * a.base_stride, *b_hi = static_cast<const T *>(a.base) + at_hi * a.base_stride;
        T *y_lo = static_cast<T *>(a.y) + at_lo * a.y_stride, *y_hi = static_cast<T *>(a.y) + at_hi * a.y_stride;
        const int steps = (a.n + 31) / 32, from = (int)((long long)steps * part / parts), to = (int)((long long)steps * (part + 1) / parts);
#pragma unroll(RT <= 2 ? 2 : 1)
        for (int s = from + ws; s < to; s += kSplit) {
            // Of 32 columns: as the second operand the lane's are 4g to 4g + 3, as the result 8t to 8t + 7.
            const int n0 = 32 * s + 8 * t, have = a.n - n0;
            Near<T, 8> old_lo, old_hi;
            if (a.base) {
                old_lo = near<WIDE, T, 8, false>(b_lo + n0, has_lo ? have : 0);
                old_hi = near<WIDE, T, 8, false>(b_hi + n0, has_hi ? have : 0);
            }
            float acc[4][4] = {};
            if (live) {
                const int c0 = 32 * s + 4 * g;
                if constexpr (!TURNED) {
                    // W2 is [n][rank].
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            const Near<T, 4> col = near<WIDE, T, 4>(w2 + (long long)(c0 + q) * a.rank + 16 * i + 4 * t,
                                                                    c0 + q < a.n ? a.rank - 16 * i - 4 * t : 0);
#pragma unroll
                            for (int part = kParts - 1; part >= 0; --part) mma_four<T>(acc[q], h_lo[part][i], h_hi[part][i], col);
                        }
                } else {
                    // W2 is [rank][n].
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        Near<T, 4> in[4], col[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 16 * i + 4 * t + j;
                            in[j] = near<WIDE, T, 4>(w2 + (long long)r * a.n + c0, r < a.rank ? a.n - c0 : 0);
                        }
                        turned<T, 4, 4>(in, col);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int part = kParts - 1; part >= 0; --part) mma_four<T>(acc[q], h_lo[part][i], h_hi[part][i], col[q]);
                    }
                }
            }
            float v_lo[8], v_hi[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v_lo[q] = acc[q][0] * s_lo;
                v_lo[4 + q] = acc[q][1] * s_lo;
                v_hi[q] = acc[q][2] * s_hi;
                v_hi[4 + q] = acc[q][3] * s_hi;
            }
            if (a.base) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v_lo[j] = live ? old_lo.at(j) + v_lo[j] : old_lo.at(j);
                    v_hi[j] = live ? old_hi.at(j) + v_hi[j] : old_hi.at(j);
                }
            }
            if (has_lo) store_near<WIDE, T>(y_lo + n0, v_lo, have);
            if (has_hi) store_near<WIDE, T>(y_hi + n0, v_hi, have);
        }
    }
    if (live) cluster_wait();
}

// ------------------------------------------------------------------ the same for many rows of an adapter
// Tiles of 128 rows.  The first product goes in steps of 64 of K through a ring in shared memory that asynchronous
// copies fill some steps ahead: the step's weights, which all warps read, and each thread's own eight elements of its
// four rows of x, which nobody else reads; a warp takes 32 rows and a half of each step.  For the second, the small
// rows wait in shared memory as the first operand's registers lie, and each warp goes through strips of 32 output
// columns: it holds the strip's weights in registers and takes 32 rows of base at a time, the coming ones on their way
// through its threads' own places in the ring, with no barrier.
// bf16, 8192x4096x16384, rank 64: 156 us with the order (4.0 TB/s; 394 with the kernel above and 64 rows a tile, whose
// weight loads each touched eight lines; rank 16: 114, rank 128 245).  Some 340 instructions for 32x32 outputs, of which 64
// are products, and 15 KB through shared memory, 8 of them the small rows' two parts again for each strip, on 16 warps an
// SM: the tensor pipe is busy for 51 % of the time and L1 for 72, in turns rather than together.  (One part, which left y
// off by up to 2^-8 of the terms s b h: 127.)
constexpr int kManyStep = 64;

// Own elements in the ring: eight on their boundary, or the aligned pieces that they lie in.
template <typename T, bool WIDE>
constexpr int own_pieces() { return sizeof(T) == 4 || !WIDE ? 2 : 1; }
// A step's weights are [rank][64] ("flat") or [64][rank]: bytes of a row, an odd number of 64 where they are read 64
// from two rows at a time, which keeps those off each other's banks.
template <typename T, int RT, bool FLAT>
constexpr int weight_pitch()
{
    constexpr int bytes = (FLAT ? kManyStep : 16 * RT) * (int)sizeof(T);
    return FLAT ? bytes + 16 : bytes % 128 == 0 ? bytes + 64 : bytes;
}
template <typename T, int RT, bool FLAT>
constexpr int weight_rows() { return FLAT ? 16 * RT : kManyStep; }
template <typename T, int RT>
constexpr int weight_bytes()
{
    constexpr int flat = weight_rows<T, RT, true>() * weight_pitch<T, RT, true>(), tall = weight_rows<T, RT, false>() * weight_pitch<T, RT, false>();
    return flat > tall ? flat : tall;
}
template <typename T, int RT, bool WIDE>
constexpr int many_stage() { return 4 * kAdapterThreads * 16 * own_pieces<T, WIDE>() + weight_bytes<T, RT>(); }
constexpr int kManyStages = 3, kManyAhead = 4;  // of the first and the second product
// Bytes of the second product's small rows, in the parts of the activations' type, then their places in memory, and what
// they are multiplied with.
template <typename T, int RT>
constexpr int small_parts() { return 16 * RT * (int)sizeof(T) * hidden_parts<T>(); }  // of a row
template <typename T, int RT>
constexpr int small_rows() { return kAdapterManyRows * (small_parts<T, RT>() + 8 + 8 + 4); }
// The whole sums, behind the partial ones, which other CTAs read, and behind where the small rows go from them.
template <typename T, int RT>
constexpr int whole_sums()
{
    constexpr int partial = kAdapterManyRows * hidden_pitch<RT>() * 4;
    return partial > small_rows<T, RT>() ? partial : small_rows<T, RT>();
}
template <typename T, int RT, bool WIDE>
constexpr int many_smem()
{
    constexpr int ring = kManyStages * many_stage<T, RT, WIDE>(), sums = whole_sums<T, RT>() + kAdapterManyRows * hidden_pitch<RT>() * 4;
    constexpr int second = small_rows<T, RT>() + kManyAhead * 4 * kAdapterThreads * 16 * own_pieces<T, WIDE>();
    return ring > sums ? (ring > second ? ring : second) : (sums > second ? sums : second);
}

// Ranks that a lane has side by side in the second product: 8 of 32 in 16 bits, as one load of 16 bytes, else 4 of 16.
template <typename T, int RT>
constexpr int many_near() { return sizeof(T) == 2 && RT % 2 == 0 ? 8 : 4; }

__device__ __forceinline__ void copy_piece(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_word(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// N elements from p, `have` of them there, to their thread's pieces of 16 bytes, kAdapterThreads pieces apart.
template <bool WIDE, typename T, int N = 8>
__device__ __forceinline__ void copy_own(uint32_t dst, const T *p, int have)
{
    constexpr int kApart = 16 * kAdapterThreads, kBytes = N * (int)sizeof(T);
    if constexpr (WIDE && kBytes == 8) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(p), "r"(have > 0 ? 8 : 0) : "memory");
    } else if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) copy_piece(dst + i * kApart, reinterpret_cast<const char *>(p) + 16 * i, have > 0);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) copy_word(dst + i / 4 * kApart + i % 4 * 4, p + (i < have ? i : 0), i < have);
    } else {
        // The aligned pieces that hold some of them.
        const uintptr_t at = reinterpret_cast<uintptr_t>(p), from = at & ~(uintptr_t)15;
        const int bytes = (int)(at - from) + 2 * (have < N ? have : N);
        copy_piece(dst, reinterpret_cast<const void *>(from), have > 0);
        copy_piece(dst + kApart, reinterpret_cast<const void *>(bytes > 16 ? from + 16 : from), have > 0 && bytes > 16);
    }
}
// They again, from the pieces at `src`, zeros beyond `have`.
template <bool WIDE, typename T, int N = 8>
__device__ __forceinline__ Near<T, N> own_of(uint32_t src, const T *p, int have)
{
    constexpr int kApart = 16 * kAdapterThreads, kWords = N * (int)sizeof(T) / 4;
    Near<T, N> v;
    uint32_t *w = reinterpret_cast<uint32_t *>(v.w);
    const uint4 u = dev::lds_v4(src);
    if constexpr (sizeof(T) == 4 || WIDE) {
        w[0] = u.x, w[1] = u.y;
        if constexpr (kWords >= 4) w[2] = u.z, w[3] = u.w;
        if constexpr (kWords == 8) {
            const uint4 o = dev::lds_v4(src + kApart);
            w[4] = o.x, w[5] = o.y, w[6] = o.z, w[7] = o.w;
        }
    } else {
        const uint4 o = dev::lds_v4(src + kApart);
        const unsigned off = (unsigned)reinterpret_cast<uintptr_t>(p) & 15u;
        uint32_t all[8] = {u.x, u.y, u.z, u.w, o.x, o.y, o.z, o.w};
        // Down by whole words, two and one at a time, then by half a word.
#pragma unroll
        for (int i = 0; i < 6; ++i) all[i] = off & 8 ? all[i + 2] : all[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) all[i] = off & 4 ? all[i + 1] : all[i];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            w[i] = __funnelshift_r(all[i], all[i + 1], (off & 2) * 8);
            const int left = have - 2 * i;
            if (left < 2) w[i] = left < 1 ? 0u : w[i] & 0xffffu;
        }
    }
    return v;
}

template <typename T, int RT, bool TURNED, bool WIDE>
__global__ void __launch_bounds__(kAdapterThreads, WIDE && RT <= 4 && sizeof(T) == 2 ? 2 : 1) adapter_many_kernel(const AdapterArgs a)
{
    constexpr int kRows = kAdapterManyRows, kPitch = hidden_pitch<RT>(), kNear = many_near<T, RT>(), kSteps = 16 * RT / (4 * kNear);
    constexpr int kQuads = RT * (int)sizeof(T) / 2;  // of the first operand's registers in the second product, of one part
    constexpr int kParts = hidden_parts<T>();
    constexpr int kStages = kManyStages, kStage = many_stage<T, RT, WIDE>();
    constexpr int kOwn = 16 * kAdapterThreads * own_pieces<T, WIDE>();  // bytes of all threads' elements of one row
    extern __shared__ __align__(16) float adapter_sums[];  // a ring; [2][kRows][kPitch] partial and whole sums; small rows and a ring
    __shared__ int rows[kRows];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int part = (int)dev::cluster_ctarank(), parts = (int)cluster_size();
    const int tile = (int)blockIdx.x / parts;
    if (tile >= *a.tile_count) return;
    const AdapterTile my = a.tiles[tile];
    const int adapter = my.adapter, count = my.count;
    if ((int)threadIdx.x < count) rows[threadIdx.x] = a.order[my.first + threadIdx.x];
    __syncthreads();
    const bool live = adapter < a.adapters;
    const int wm = warp % 4, ws = warp / 4;  // 32 rows of the tile; a half of each step
    const bool busy = 32 * wm < count;
    bool has[4];
    int row[4];  // g, g + 8, g + 16 and g + 24 of the warp's; the tile's last in the place of those beyond, which are loaded but not stored
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 32 * wm + 8 * i + g;
        has[i] = r < count;
        row[i] = rows[has[i] ? r : count - 1];
    }
    float *whole = adapter_sums + whole_sums<T, RT>() / 4;
    unsigned char *ring = reinterpret_cast<unsigned char *>(adapter_sums);

    // Steps of a product that this CTA takes.
    auto share = [&](int length, int *first, int *stop) {
        const long long steps = (length + kManyStep - 1) / kManyStep;
        *first = (int)(steps * part / parts);
        *stop = (int)(steps * (part + 1) / parts);
    };
    const int own_column = 32 * ws + 8 * t;  // of a step
    const uint32_t ring_at = dev::smem_u32(ring), my_slot = ring_at + threadIdx.x * 16;
    // Goes through a product's steps: copies the weights [64 of `length` a step] and this thread's elements of the rows
    // at `own` (from the first step's on), and calls step(step, stage) when a step's are there for all.
    auto stream = [&](auto flat, const T *weights, bool pieces, int length, const T *const *own, bool owns, int first, int stop,
                      auto &&step) {
        constexpr bool kFlat = decltype(flat)::value;
        constexpr int kWRows = weight_rows<T, RT, kFlat>(), kWPitch = weight_pitch<T, RT, kFlat>();
        constexpr int kLong = kFlat ? kManyStep : 16 * RT, kPiece = 16 / (int)sizeof(T), kPieces = kLong / kPiece;
        constexpr int kAtOnce = kAdapterThreads / kPieces;  // rows of the weights that the threads copy at once
        const int my_row = (int)threadIdx.x / kPieces, my_piece = (int)threadIdx.x % kPieces * kPiece;
        const long long row_pitch = kFlat ? length : a.rank;
        const T *my_weights = weights + my_row * row_pitch + my_piece;
        const int apart = kAtOnce * (int)row_pitch;
        const uint32_t my_weight_slot = ring_at + 4 * kOwn + my_row * kWPitch + my_piece * (int)sizeof(T);
        auto fetch = [&](int j, int stage) {
            if (j < stop) {
                if (owns) {
                    const int have = length - j * kManyStep - own_column;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        copy_own<WIDE, T>(my_slot + stage * kStage + i * kOwn, own[i] + (have > 0 ? (j - first) * kManyStep : 0), have);
                }
                if (pieces) {
                    const T *from = my_weights + (kFlat ? (long long)j * kManyStep : (long long)(j * kManyStep) * a.rank);
#pragma unroll
                    for (int q = 0; q < (kWRows + kAtOnce - 1) / kAtOnce; ++q) {
                        const int r = my_row + q * kAtOnce;
                        const bool there = (kFlat ? r : my_piece) < a.rank && j * kManyStep + (kFlat ? my_piece : r) < length;
                        if (kWRows % kAtOnce == 0 || r < kWRows)
                            copy_piece(my_weight_slot + stage * kStage + q * kAtOnce * kWPitch, there ? from + q * apart : weights, there);
                    }
                } else {
                    unsigned char *to = ring + stage * kStage + 4 * kOwn;
                    for (int i = threadIdx.x; i < kWRows * kLong; i += kAdapterThreads) {
                        const int r = i / kLong, c = i % kLong;
                        const int rank = kFlat ? r : c, at = j * kManyStep + (kFlat ? c : r);
                        T v;
                        narrowed(0.0f, &v);
                        if (rank < a.rank && at < length) v = weights[kFlat ? (long long)rank * length + at : (long long)at * a.rank + rank];
                        reinterpret_cast<T *>(to + r * kWPitch)[c] = v;
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int j = 0; j < kStages - 1; ++j) fetch(first + j, j);
        int stage = 0;
        for (int j = first; j < stop; ++j) {
            // The step's copies are there, for all, and the step before it is read by all.
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncthreads();
            fetch(j + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
            if (busy) step(j, stage * kStage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
    };

    if (live) {
        const std::integral_constant<bool, !TURNED> flat{};
        constexpr int kWPitch = weight_pitch<T, RT, !TURNED>();
        const T *w1 = static_cast<const T *>(a.w1) + (long long)adapter * a.rank * a.k;
        float acc[2][2 * RT][4] = {};
        int first, stop;
        share(a.k, &first, &stop);
        const T *own[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) own[i] = static_cast<const T *>(a.x) + row[i] * a.x_stride + (first * kManyStep + own_column < a.k ? first * kManyStep + own_column : 0);
        const uint32_t my_weights = ring_at + 4 * kOwn + (TURNED ? own_column * kWPitch + 2 * RT * g * (int)sizeof(T) : g * kWPitch + own_column * (int)sizeof(T));
        stream(flat, w1, a.w1_pieces, a.k, own, true, first, stop, [&](int step, uint32_t at) {
            Near<T, 8> v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = own_of<WIDE, T>(my_slot + at + i * kOwn, own[i] + (step - first) * kManyStep, a.k - step * kManyStep - own_column);
            const uint32_t w = my_weights + at;
            if constexpr (!TURNED) {
#pragma unroll
                for (int j = 0; j < 2 * RT; ++j) {
                    Near<T, 8> col;
                    from_shared(w + 8 * j * kWPitch, &col);
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma_eight<T>(acc[h][j], v[2 * h], v[2 * h + 1], col);
                }
            } else {
                constexpr int kC = 2 * RT < 8 ? 2 * RT : 8;
#pragma unroll
                for (int c = 0; c < 2 * RT; c += kC) {
                    Near<T, kC> in[8];
                    Near<T, 8> col[kC];
#pragma unroll
                    for (int i = 0; i < 8; ++i) from_shared(w + i * kWPitch + c * (int)sizeof(T), &in[i]);
                    turned<T, 8, kC>(in, col);
#pragma unroll
                    for (int j = 0; j < kC; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) mma_eight<T>(acc[h][c + j], v[2 * h], v[2 * h + 1], col[j]);
                }
            }
        });
        __syncthreads();  // the ring is read; what was copied ahead of it, nothing
        // The two halves of the steps: the second's sums beside, where the whole ones will be.
        float *mine = (ws ? whole : adapter_sums) + 32 * wm * kPitch;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2 * RT; ++j) {
                const int r0 = TURNED ? 2 * RT * (2 * t) + j : 8 * j + 2 * t, r1 = TURNED ? 2 * RT * (2 * t + 1) + j : r0 + 1;
                mine[(16 * h + g) * kPitch + r0] = acc[h][j][0];
                mine[(16 * h + g) * kPitch + r1] = acc[h][j][1];
                mine[(16 * h + g + 8) * kPitch + r0] = acc[h][j][2];
                mine[(16 * h + g + 8) * kPitch + r1] = acc[h][j][3];
            }
        __syncthreads();
        constexpr int kFours = 4 * RT;  // of a row
        for (int i = threadIdx.x; i < count * kFours; i += kAdapterThreads) {
            const int offset = i / kFours * kPitch + i % kFours * 4;
            float4 *at = reinterpret_cast<float4 *>(adapter_sums + offset);
            const float4 u = *reinterpret_cast<const float4 *>(whole + offset);
            *at = make_float4(at->x + u.x, at->y + u.y, at->z + u.z, at->w + u.w);
        }
        cluster_arrive();
        cluster_wait();
        const uint32_t sums = dev::smem_u32(adapter_sums);
        for (int i = threadIdx.x; i < kRows * kFours; i += kAdapterThreads) {
            const int offset = i / kFours * kPitch + i % kFours * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < count * kFours) {
                v = load_cluster(dev::mapa_cluster(sums + 4 * offset, 0));
                for (int p = 1; p < parts; ++p) {
                    const float4 u = load_cluster(dev::mapa_cluster(sums + 4 * offset, (uint32_t)p));
                    v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                }
            }
            *reinterpret_cast<float4 *>(whole + offset) = v;
        }
        __syncthreads();
        cluster_arrive();  // waited for before the ring takes the sums' place
    }
    if (a.hidden) {
        for (int i = threadIdx.x; i < count * a.rank; i += kAdapterThreads) {
            const int r = i / a.rank;
            if (r % parts == part) a.hidden[(long long)rows[r] * a.rank + i % a.rank] = live ? whole[r * kPitch + i % a.rank] : 0.0f;
        }
    }
    const int strips = (a.n + 31) / 32;
    const int first = (int)((long long)strips * part / parts), stop = (int)((long long)strips * (part + 1) / parts);
    if (live) {
        cluster_wait();
        // The small rows in the parts of the activations' type (f16 after division by a power of two near the row's
        // largest), as the first operand's registers lie in a lane: 16 rows by each warp.  One part alone would leave y off
        // by 2^-8 (f16 2^-11) of the terms s b h, many times its own rounding where they cancel each other or the base.
        unsigned char *const small = ring;
        const char **const base_row = reinterpret_cast<const char **>(small + kRows * small_parts<T, RT>());
        char **const y_row = reinterpret_cast<char **>(small + kRows * (small_parts<T, RT>() + 8));
        float *const factors = reinterpret_cast<float *>(y_row + kRows);
        constexpr bool kFactors = __is_same(T, __half);  // else the small rows take the scale before they are split
        {
            float v[2][kSteps][kNear];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * warp + 8 * i + g;
                float s = a.scale ? a.scale[adapter] : 1.0f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int q = 0; q < kNear; q += 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(whole + r * kPitch + 4 * kNear * k + kNear * t + q);
                        v[i][k][q] = u.x, v[i][k][q + 1] = u.y, v[i][k][q + 2] = u.z, v[i][k][q + 3] = u.w;
                    }
                const float factor = narrow_factor<T, kSteps * kNear>(&v[i][0][0], &s);
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int q = 0; q < kNear; ++q) v[i][k][q] *= kFactors ? factor : s;
                if (t == 0) {
                    const long long at = rows[r < count ? r : count - 1];
                    factors[r] = s;
                    base_row[r] = static_cast<const char *>(a.base) + at * a.base_stride * (int)sizeof(T);
                    y_row[r] = static_cast<char *>(a.y) + at * a.y_stride * (int)sizeof(T);
                }
            }
            uint4 *const to = reinterpret_cast<uint4 *>(small) + warp * kParts * kQuads * 32 + lane;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int q = 0; q < kNear; q += 8 / (int)sizeof(T))
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        uint4 u;
                        if constexpr (sizeof(T) == 4) {
                            u = make_uint4(__float_as_uint(v[0][k][q]), __float_as_uint(v[1][k][q]), __float_as_uint(v[0][k][q + 1]), __float_as_uint(v[1][k][q + 1]));
                        } else {
                            uint32_t w[2][2];
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float *const pair = &v[i][k][q + 2 * h];
                                    w[i][h] = packed(pair[0], pair[1], T());
                                    // What is left; of infinities and NaN nothing, as their difference with themselves is NaN.
#pragma unroll
                                    for (int j = 0; j < 2; ++j)
                                        pair[j] = fabsf(pair[j]) < __int_as_float(0x7f800000) ? pair[j] - widened(reinterpret_cast<const T *>(&w[i][h])[j]) : 0.0f;
                                }
                            u = make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]);
                        }
                        to[(p * kQuads + (k * kNear + q) / (8 / (int)sizeof(T))) * 32] = u;
                    }
        }
        __syncthreads();  // they are there, and the sums read
        const T *w2 = static_cast<const T *>(a.w2) + (long long)adapter * a.rank * a.n;
        const bool adds = a.base != nullptr;
        if (!adds) {  // what is added is then zeros
            uint4 *const zeros = reinterpret_cast<uint4 *>(ring + small_rows<T, RT>());
            for (int i = threadIdx.x; i < kManyAhead * 4 * kOwn / 16; i += kAdapterThreads) zeros[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        }
        const int groups = (count + 31) / 32;  // of rows
        const uint32_t slots = dev::smem_u32(ring + small_rows<T, RT>()) + threadIdx.x * 16;
        const uint32_t small_at = dev::smem_u32(small) + lane * 16;
        // As the second operand, the lane's columns of a strip are 8 (g / 2) + g % 2 and every second from there; as the
        // result, 8t to 8t + 7, two of each instruction's.
        const unsigned odd = g % 2 ? 0x7632 : 0x5410;
        constexpr int kRaw = TURNED ? kNear : 4, kRawNear = TURNED ? 8 : kNear;
        using Raw = Near<T, kRawNear>[kSteps][kRaw];
        auto weights_of = [&](int strip, Raw &raw) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int q = 0; q < kRaw; ++q) {
                    const int rank = 4 * kNear * k + kNear * t + (TURNED ? q : 0), column = 32 * strip + 8 * (g / 2) + (TURNED ? 0 : g % 2 + 2 * q);
                    const T *from = w2 + (TURNED ? (long long)rank * a.n + column : (long long)column * a.rank + rank);
                    const int have = strip >= stop ? 0 : TURNED ? (rank < a.rank ? a.n - column : 0) : (column < a.n ? a.rank - rank : 0);
                    raw[k][q] = a.w2_wide ? near<true, T, kRawNear>(from, have) : near<false, T, kRawNear>(from, have);
                }
        };
        int next_strip = first + warp, next_group = 0, next_stage = 0;
        auto fetch = [&]() {
            if (next_strip < stop && adds) {
                const int c = 32 * next_strip + 8 * t, have = a.n - c;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    copy_own<WIDE, T>(slots + (next_stage * 4 + i) * kOwn,
                                      reinterpret_cast<const T *>(base_row[32 * next_group + 8 * i + g] + (have > 0 ? c : 0) * (int)sizeof(T)), have);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            next_stage = next_stage + 1 == kManyAhead ? 0 : next_stage + 1;
            if (++next_group == groups) {
                next_group = 0;
                next_strip += kAdapterThreads / 32;
            }
        };
        for (int i = 0; i < kManyAhead - 1; ++i) fetch();
        constexpr bool kAhead = !TURNED || RT <= 2;  // the coming strip's weights too, where registers are left
        Raw raw;
        if (kAhead) weights_of(first + warp, raw);
        int stage = 0;
        for (int strip = first + warp; strip < stop; strip += kAdapterThreads / 32) {
            if (!kAhead) weights_of(strip, raw);
            Near<T, kNear> w[kSteps][4];
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (!TURNED) {
                        w[k][q] = raw[k][q];
                    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
                        for (int r = 0; r < kNear; ++r) w[k][q].w[r] = g % 2 ? raw[k][r].w[2 * q + 1] : raw[k][r].w[2 * q];
                    } else {
#pragma unroll
                        for (int r = 0; r < kNear / 2; ++r) w[k][q].w[r] = __byte_perm(raw[k][2 * r].w[q], raw[k][2 * r + 1].w[q], odd);
                    }
                }
            if (kAhead) weights_of(strip + kAdapterThreads / 32, raw);
            const int column = 32 * strip + 8 * t, have = a.n - column;
            for (int group = 0; group < groups; ++group) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kManyAhead - 2) : "memory");
                fetch();
                float acc[2][4][4];
#pragma unroll
                for (int p = kParts - 1; p >= 0; --p)  // the small parts' sums first
#pragma unroll
                    for (int j = 0; j < kQuads; ++j)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint4 h = dev::lds_v4(small_at + (((2 * group + m) * kParts + p) * kQuads + j) * 512);
                            constexpr int kPairs = kNear * (int)sizeof(T) / 8;  // of a lane's weights of a column
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mma_quad<T>(acc[m][q], h, w[j / kPairs][q].w[2 * (j % kPairs)], w[j / kPairs][q].w[2 * (j % kPairs) + 1],
                                            j == 0 && p == kParts - 1);
                        }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 32 * group + 8 * i + g;
                    float2 v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = make_float2(acc[i / 2][q][i % 2 * 2], acc[i / 2][q][i % 2 * 2 + 1]);
                    const Near<T, 8> old = own_of<WIDE, T>(slots + (stage * 4 + i) * kOwn,
                                                           WIDE ? nullptr : reinterpret_cast<const T *>(base_row[r]) + column, have);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 o = make_float2(old.at(2 * q), old.at(2 * q + 1));
                        if constexpr (kFactors)
                            v[q] = __ffma2_rn(v[q], make_float2(factors[r], factors[r]), o);
                        else
                            v[q] = __fadd2_rn(v[q], o);
                    }
                    store_near<WIDE, T>(reinterpret_cast<T *>(y_row[r] + column * (int)sizeof(T)), reinterpret_cast<const float *>(v), r < count ? have : 0);
                }
                stage = stage + 1 == kManyAhead ? 0 : stage + 1;
            }
        }
    } else if (a.base != a.y) {
        // Rows without an adapter: base, or zeros; eight loads of a lane in flight, two of each of four rows.
        const int from = 32 * first, to = 32 * stop < a.n ? 32 * stop : a.n;
        constexpr int kTogether = 4;
        for (int r0 = kTogether * warp; r0 < count; r0 += kTogether * kAdapterThreads / 32)
            for (int c0 = from + 8 * lane; c0 < to; c0 += 512) {
                Near<T, 8> old[kTogether][2];
#pragma unroll
                for (int i = 0; i < kTogether; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = c0 + 256 * j, have = a.base && r0 + i < count ? to - c : 0;
                        old[i][j] = near<WIDE, T, 8, false>(static_cast<const T *>(a.base) + rows[r0 + i < count ? r0 + i : 0] * a.base_stride + c, have);
                    }
#pragma unroll
                for (int i = 0; i < kTogether; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = c0 + 256 * j;
                        float v[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] = old[i][j].at(q);
                        store_near<WIDE, T>(static_cast<T *>(a.y) + rows[r0 + i < count ? r0 + i : 0] * a.y_stride + c, v, r0 + i < count ? to - c : 0);
                    }
            }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ gradients of the weights
// What adapter_tc_weights_kernel does not take: f16 and f32, rows off 16-byte boundaries, ranks above 64, adapters of few
// rows.  Sums over an adapter's rows of outer products, [columns][rank]: a CTA takes a strip of columns of x (for dA) or dy
// (for dB), 64 a warp (32 for large ranks), and a chunk of the rows in the order by adapter, 16 at a time.  A lane's
// eight (four) neighbouring columns of four rows come through its own places in a ring of asynchronous copies and are
// turned into the first operand.  The second, the small rows, is the same for all warps: they make it together for a
// batch of rows in shared memory, fp32 in three bf16 parts (f16 and f32 activations: two 19-bit ones), so that the sums
// keep fp32's bits.  An adapter within the chunk is written as it is, one that reaches beyond it into the chunk's two
// rows of partial sums, which adapter_join_kernel adds up in order.  bf16, 8192x4096x4096, rank 16: 69 us (2 TB/s), by
// its instructions for each element, where the tensor cores' own kernel takes 31.
template <typename T, int RT>
struct WeightSizes {
    static constexpr int kNear = RT <= 2 ? 8 : 4, kWarpColumns = 8 * kNear;
    static constexpr int kColumns = kWarpColumns * kAdapterThreads / 32;
    static constexpr int kBatch = RT <= 2 ? 64 : 32;                  // rows
    static constexpr int kItems = kBatch / 16 * 2 * RT * 32;          // lanes' parts of a batch's second operand
    static constexpr bool kThree = __is_same(T, __nv_bfloat16);
    static constexpr int kItemBytes = kThree ? 24 : 32;
    static constexpr int kBatchBytes = kItems * kItemBytes;
};
template <typename T, int RT, bool WIDE>
constexpr int weights_pieces()  // of a thread's columns of a row
{
    return !WIDE ? 2 : WeightSizes<T, RT>::kNear * (int)sizeof(T) > 16 ? 2 : 1;
}
template <typename T, int RT, bool WIDE>
constexpr int weights_stages() { return 3; }
// CTAs on an SM: what shared memory holds, where the registers do.
template <typename T, int RT, bool WIDE>
constexpr int weights_resident() { return sizeof(T) == 2 && WIDE ? (RT == 1 ? 3 : RT <= 4 ? 2 : 1) : 1; }
template <typename T, int RT, bool WIDE>
constexpr int weights_smem()
{
    return weights_stages<T, RT, WIDE>() * 4 * kAdapterThreads * 16 * weights_pieces<T, RT, WIDE>() + 2 * WeightSizes<T, RT>::kBatchBytes +
           kAdapterChunkRows * 12;
}

template <typename T, int RT, bool WIDE>
__global__ void __launch_bounds__(kAdapterThreads, weights_resident<T, RT, WIDE>()) adapter_weights_kernel(const AdapterGradArgs a)
{
    using S = WeightSizes<T, RT>;
    constexpr int kNear = S::kNear, kBatchSteps = S::kBatch / 16, kMine = S::kItems / kAdapterThreads;
    constexpr int kStages = weights_stages<T, RT, WIDE>(), kOwn = kAdapterThreads * 16 * weights_pieces<T, RT, WIDE>();
    extern __shared__ __align__(16) unsigned char weights_ring[];  // [kStages][4] rows' own pieces; [2] batches; the chunk's rows
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int x_strips = (a.k + S::kColumns - 1) / S::kColumns;
    const bool of_x = (int)blockIdx.x < x_strips;
    const int width = of_x ? a.k : a.n;
    const T *data = static_cast<const T *>(of_x ? a.x : a.dy);
    const long long stride = of_x ? a.x_stride : a.dy_stride;
    const float *small = of_x ? a.dhidden : a.hidden;
    const int chunk = blockIdx.y, valid = a.starts[a.adapters], chunk_from = chunk * a.chunk_rows;
    const int stop = chunk_from + a.chunk_rows < valid ? chunk_from + a.chunk_rows : valid;
    const int column = ((int)blockIdx.x - (of_x ? 0 : x_strips)) * S::kColumns + S::kWarpColumns * warp + kNear * g, have = width - column;
    unsigned char *const batches = weights_ring + kStages * 4 * kOwn;
    // The chunk's rows, as the numbers of their first elements.
    long long *const rows = reinterpret_cast<long long *>(batches + 2 * S::kBatchBytes);
    int *const row_numbers = reinterpret_cast<int *>(rows + kAdapterChunkRows);
    for (int i = threadIdx.x; i < stop - chunk_from; i += kAdapterThreads) {
        const int row = a.order[chunk_from + i];
        rows[i] = row * stride;
        row_numbers[i] = row;
    }
    __syncthreads();
    const uint32_t slots = dev::smem_u32(weights_ring) + threadIdx.x * 16;
    for (int at = chunk_from; at < stop;) {
        // The adapter of position `at`: as many as end at or before it come first.
        int adapter = 0;
        for (int i = 0; i < a.adapters; i += kAdapterThreads)
            adapter += __syncthreads_count(i + (int)threadIdx.x < a.adapters && a.starts[i + threadIdx.x + 1] <= at);
        const int first = a.starts[adapter], last = a.starts[adapter + 1], end = last < stop ? last : stop;
        const long long *const mine = rows + (at - chunk_from);
        const int *const numbers = row_numbers + (at - chunk_from);
        const int count = end - at, steps = (count + 15) / 16;
        // A batch's second operand: thread's items are lanes' of a step of 16 rows and 8 ranks, four rows each.
        float held[kMine][4];
        auto load = [&](int batch) {
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int item = q * kAdapterThreads + threadIdx.x, l = item % 32, rank = item / 32 % (2 * RT) * 8 + l / 4;
                const int from = batch * S::kBatch + item / (64 * RT) * 16 + l % 4 * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    held[q][i] = rank < a.rank && from + i < count ? __ldg(small + (long long)numbers[from + i] * a.rank + rank) : 0.0f;
            }
        };
        auto keep = [&](int batch) {
            unsigned char *const to = batches + batch % 2 * S::kBatchBytes;
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int item = q * kAdapterThreads + threadIdx.x;
                if constexpr (S::kThree) {
                    float v[4] = {held[q][0], held[q][1], held[q][2], held[q][3]};
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        uint32_t w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            w[i] = packed(v[2 * i], v[2 * i + 1], T());
                            // What is left; of infinities and NaN nothing, as their difference with themselves is NaN.
                            const float top = __int_as_float(0x7f800000);
                            v[2 * i] = fabsf(v[2 * i]) < top ? v[2 * i] - __uint_as_float(w[i] << 16) : 0.0f;
                            v[2 * i + 1] = fabsf(v[2 * i + 1]) < top ? v[2 * i + 1] - __uint_as_float(w[i] & 0xffff0000u) : 0.0f;
                        }
                        reinterpret_cast<uint2 *>(to)[part * S::kItems + item] = make_uint2(w[0], w[1]);
                    }
                } else {
                    // 8 rows an instruction.
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const Parts b0 = parts_of(held[q][2 * i]), b1 = parts_of(held[q][2 * i + 1]);
                        reinterpret_cast<uint4 *>(to)[i * S::kItems + item] = make_uint4(b0.hi, b1.hi, b0.lo, b1.lo);
                    }
                }
            }
        };
        const T *const my_data = data + (have > 0 ? column : 0);
        auto fetch = [&](int step, uint32_t to) {
            if (step < steps) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = 16 * step + 4 * t + i;
                    copy_own<WIDE, T, kNear>(to + i * kOwn, my_data + (p < count ? mine[p] : 0), p < count ? have : 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int i = 0; i < kStages - 1; ++i) fetch(i, slots + i * 4 * kOwn);
        int stage = 0;
        load(0);
        keep(0);
        __syncthreads();
        float acc[kNear / 2][2 * RT][4] = {};
        for (int batch = 0; batch * kBatchSteps < steps; ++batch) {
            const bool more = (batch + 1) * kBatchSteps < steps;
            if (more) load(batch + 1);
            const int to = (batch + 1) * kBatchSteps < steps ? (batch + 1) * kBatchSteps : steps;
            uint32_t operand = dev::smem_u32(batches + batch % 2 * S::kBatchBytes) + lane * (S::kThree ? 8 : 16);
            for (int step = batch * kBatchSteps; step < to; ++step, operand += 2 * RT * 32 * (S::kThree ? 8 : 16)) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                Near<T, kNear> in[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = 16 * step + 4 * t + i;
                    in[i] = own_of<WIDE, T, kNear>(slots + (stage * 4 + i) * kOwn, WIDE ? nullptr : my_data + (p < count ? mine[p] : 0),
                                                   p < count ? have : 0);
                }
                fetch(step + kStages - 1, slots + (stage == 0 ? kStages - 1 : stage - 1) * 4 * kOwn);
                stage = stage + 1 == kStages ? 0 : stage + 1;
                if constexpr (S::kThree) {
                    Near<T, 4> col[kNear];
                    turned<T, 4, kNear>(in, col);
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int j = 0; j < 2 * RT; ++j) {
                            Near<T, 4> b;
                            from_shared(operand + (part * S::kItems + j * 32) * 8, &b);
#pragma unroll
                            for (int c = 0; c < kNear / 2; ++c)
                                mma16(acc[c][j], col[2 * c].w[0], col[2 * c + 1].w[0], col[2 * c].w[1], col[2 * c + 1].w[1], b.w[0], b.w[1], T());
                        }
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int j = 0; j < 2 * RT; ++j) {
                            const uint4 b = dev::lds_v4(operand + (s * S::kItems + j * 32) * 16);
#pragma unroll
                            for (int c = 0; c < kNear / 2; ++c) {
                                const float v0 = in[2 * s].at(2 * c), v1 = in[2 * s].at(2 * c + 1), v2 = in[2 * s + 1].at(2 * c),
                                            v3 = in[2 * s + 1].at(2 * c + 1);
                                if constexpr (sizeof(T) == 4) {
                                    mma8_parts(acc[c][j], parts_of(v0), parts_of(v1), parts_of(v2), parts_of(v3), Parts{b.x, b.z}, Parts{b.y, b.w});
                                } else {  // exact
                                    const uint32_t a0 = __float_as_uint(v0), a1 = __float_as_uint(v1), a2 = __float_as_uint(v2),
                                                   a3 = __float_as_uint(v3);
                                    mma8(acc[c][j], a0, a1, a2, a3, b.z, b.w);
                                    mma8(acc[c][j], a0, a1, a2, a3, b.x, b.y);
                                }
                            }
                        }
                }
            }
            if (more) keep(batch + 1);
            __syncthreads();
        }
        const float s = a.scale ? a.scale[adapter] : 1.0f;
        float *out = of_x ? a.da + (long long)adapter * a.rank * a.k : a.db + (long long)adapter * a.rank * a.n;
        if (first < chunk_from || last > stop) {
            out = a.partial + (2LL * chunk + (first >= chunk_from)) * a.rank * ((long long)a.k + a.n);
            if (!of_x) out += (long long)a.rank * a.k;
        }
#pragma unroll
        for (int j = 0; j < 2 * RT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rank = 8 * j + 2 * t + e;
#pragma unroll
                for (int i = 0; i < kNear; ++i)
                    if (rank < a.rank && i < have)
                        out[of_x ? (long long)rank * a.k + column + i : (long long)(column + i) * a.rank + rank] = s * acc[i / 2][j][i % 2 * 2 + e];
            }
        at = end;
    }
}

// ------------------------------------------------------------------ launches
template <typename T, int RT, bool TURNED, bool WIDE>
cudaError_t many_launch(const AdapterArgs &a, int clusters, int cluster_size, cudaStream_t stream)
{
    constexpr int kSmem = many_smem<T, RT, WIDE>();
    static bool allowed[kMaxDevices] = {};
    const cudaError_t e = allow_dynamic_smem(adapter_many_kernel<T, RT, TURNED, WIDE>, kSmem, allowed);
    if (e != cudaSuccess) return e;
    return launch_overlapped(adapter_many_kernel<T, RT, TURNED, WIDE>, dim3((unsigned)clusters * (unsigned)cluster_size),
                             dim3(kAdapterThreads), kSmem, stream, cluster_size, a);
}

template <typename T, int RT, int WM, bool TURNED, bool WIDE>
cudaError_t products_launch(const AdapterArgs &a, int clusters, int cluster_size, cudaStream_t stream)
{
    constexpr int kSmem = adapter_smem<RT, WM>();
    static bool allowed[kMaxDevices] = {};
    if (kSmem > 32 * 1024) {  // the counts take some of the first 48 KB
        const cudaError_t e = allow_dynamic_smem(adapter_products_kernel<T, RT, WM, TURNED, WIDE>, kSmem, allowed);
        if (e != cudaSuccess) return e;
    }
    return launch_overlapped(adapter_products_kernel<T, RT, WM, TURNED, WIDE>, dim3((unsigned)clusters * (unsigned)cluster_size),
                             dim3(kAdapterThreads), kSmem, stream, cluster_size, a);
}

template <typename T, int RT>
cudaError_t products_pick(const AdapterArgs &a, bool turned, bool many, int clusters, int cluster_size, cudaStream_t stream)
{
    const bool wide = a.x_wide && a.y_wide && (many || (a.w1_wide && a.w2_wide));
    auto pick = [&](auto t, auto w) {
        constexpr bool kTurned = decltype(t)::value, kWide = decltype(w)::value;
        return many ? many_launch<T, RT, kTurned, kWide>(a, clusters, cluster_size, stream)
                    : products_launch<T, RT, 1, kTurned, kWide>(a, clusters, cluster_size, stream);
    };
    constexpr std::true_type yes;
    constexpr std::false_type no;
    return turned ? (wide ? pick(yes, yes) : pick(yes, no)) : (wide ? pick(no, yes) : pick(no, no));
}

template <typename T, int RT, bool WIDE>
cudaError_t weights_launch(const AdapterGradArgs &a, cudaStream_t stream)
{
    using S = WeightSizes<T, RT>;
    constexpr int kSmem = weights_smem<T, RT, WIDE>();
    static_assert(S::kColumns == (RT <= 2 ? kAdapterColumns : kAdapterColumns / 2), "as the workspace is laid out");
    static bool allowed[kMaxDevices] = {};
    const cudaError_t e = allow_dynamic_smem(adapter_weights_kernel<T, RT, WIDE>, kSmem, allowed);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.k + S::kColumns - 1) / S::kColumns + (a.n + S::kColumns - 1) / S::kColumns), (unsigned)a.chunks);
    return launch_overlapped(adapter_weights_kernel<T, RT, WIDE>, grid, dim3(kAdapterThreads), kSmem, stream, 1, a);
}
template <typename T, int RT>
cudaError_t weights_pick(const AdapterGradArgs &a, cudaStream_t stream)
{
    return a.x_wide && a.dy_wide ? weights_launch<T, RT, true>(a, stream) : weights_launch<T, RT, false>(a, stream);
}

}  // namespace

template <typename T>
cudaError_t adapter_products_launch(const AdapterArgs &a, bool transposed, bool many, int clusters, int cluster_size,
                                    cudaStream_t stream)
{
    switch (adapter_rank_tiles(a.rank)) {
    case 1: return products_pick<T, 1>(a, transposed, many, clusters, cluster_size, stream);
    case 2: return products_pick<T, 2>(a, transposed, many, clusters, cluster_size, stream);
    case 4: return products_pick<T, 4>(a, transposed, many, clusters, cluster_size, stream);
    default: return products_pick<T, 8>(a, transposed, many, clusters, cluster_size, stream);
    }
}

template <typename T>
cudaError_t adapter_weights_launch(const AdapterGradArgs &a, cudaStream_t stream)
{
    switch (adapter_rank_tiles(a.rank)) {
    case 1: return weights_pick<T, 1>(a, stream);
    case 2: return weights_pick<T, 2>(a, stream);
    case 4: return weights_pick<T, 4>(a, stream);
    default: return weights_pick<T, 8>(a, stream);
    }
}

}  // namespace cbs
