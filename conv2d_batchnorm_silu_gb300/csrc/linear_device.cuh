// linear_device.cuh -- shared by the int8 linear layer's kernels: loads of int8, their widening to
// f16, and what becomes of a sum:
//   y = act(sum * (a_scale[m] * w_scale[n]) + bias[n]) [+ residual[m][n]], rounded once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "conv_bn_silu.h"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {

struct LinearEpilogue {
    const float *a_scale, *w_scale, *bias;
    const void *residual;
    void *y;
    long long residual_stride, y_stride;
    long long m;
    int n;
    int activation;
    int vec_y;         // rows of y 16-byte aligned
    int vec_residual;  // rows of the residual 16-byte aligned
};

inline LinearEpilogue linear_epilogue_of(const LinearProblem &p)
{
    const int size = dtype_size(p.out_dtype);
    auto rows16 = [&](const Rows &r) {
        return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.stride * size % 16 == 0;
    };
    LinearEpilogue e{};
    e.a_scale = p.a_scale;
    e.w_scale = p.w_scale;
    e.bias = p.bias;
    e.residual = p.residual.data;
    e.residual_stride = p.residual.stride;
    e.y = p.y.data;
    e.y_stride = p.y.stride;
    e.m = p.m;
    e.n = p.n;
    e.activation = p.activation;
    e.vec_y = rows16(p.y);
    e.vec_residual = rows16(p.residual);
    return e;
}

#ifdef __CUDACC__
namespace {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_float(float v, float *out) { *out = v; }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16 *out) { *out = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_float(float v, __half *out) { *out = __float2half_rn(v); }

// Brings `bytes` bytes (a multiple of 16, from a 16-byte boundary) into L2.  Only a hint, so it may run
// before grid_dependency_wait(): weights are on their way while the kernel before still quantises the rows.
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// A predicated 16-byte load straight into its registers, zeros without it: behind a branch the value would
// be moved, and the warp wait for it, where the branches meet.
__device__ __forceinline__ uint4 load_or_zero(const void *p, bool exists)
{
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)exists));
    return v;
}

// 16 values of a row from k0 on, at any alignment: the two aligned 16-byte pieces of memory that hold them,
// shifted together.  A piece is read only if it holds a byte of the row, so it may reach up to 15 bytes past
// either end of it, within the 16-byte unit, and so the page and the allocation, of that byte.
struct RawPiece {
    uint4 lo, hi;
};
__device__ __forceinline__ RawPiece load_raw(const int8_t *row, int k0, int k)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(row) + k0, end = reinterpret_cast<uintptr_t>(row) + k;
    const uintptr_t base = p & ~static_cast<uintptr_t>(15);
    return RawPiece{load_or_zero(reinterpret_cast<const void *>(base), k0 < k && base < end),
                    load_or_zero(reinterpret_cast<const void *>(base + 16), base != p && base + 16 < end)};
}
// The values of a piece; what it holds past k is left as it is.
__device__ __forceinline__ uint4 shifted(const RawPiece &r, const int8_t *row, int k0)
{
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) + k0) & 15u;
    uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = off & 4u ? w[i + 1] : w[i];
    const uint32_t bits = 8 * (off & 3u);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
// Zeros for the values past k.
__device__ __forceinline__ uint4 within(uint4 v, int k0, int k)
{
    auto keep = [&](uint32_t w, int first) {
        const int n = k - k0 - first;  // bytes of the word that stay
        return n >= 4 ? w : (n <= 0 ? 0u : w & (0xffffffffu >> (8 * (4 - n))));
    };
    return make_uint4(keep(v.x, 0), keep(v.y, 4), keep(v.z, 8), keep(v.w, 12));
}

// Four int8 of a word -> two words of f16 pairs, bytes 0 and 2, then 1 and 3 (an order of K that both
// operands share).  The well-known conversion through a biased mantissa.  Biased to 0..255, a byte below 0x64 is the f16 1024 + byte, and subtracting 1152
// leaves the value; the masking, the bias and the 0x64 are one three-input operation.
__device__ __forceinline__ uint2 widen4(uint32_t w)
{
    const uint32_t lo = (w & 0x00ff00ffu) ^ 0x64806480u, hi = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&hi), bias);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Waits for a barrier's phase while the hardware holds the thread back, up to 20 us at a time, so that
// waiting warps leave the issue slots to the working ones.  False if the abort flag is raised or timeout_ns
// pass.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const volatile int *abort_flag,
                                             uint64_t timeout_ns)
{
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 7u) == 7) {
            if (abort_flag != nullptr && *abort_flag) return false;
            const uint64_t now = dev::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > timeout_ns) return false;
        }
    }
}

// Instruction descriptor of kind::f16 with f16 A and B (format 0), both K-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

constexpr float kLog2E = 1.44269504f;                                       // log2(e) rounded
constexpr float kLog2ERest = (float)(1.4426950408889634 - (double)kLog2E);  // and what that leaves

// The activation of a sum whose output is of type T.  SiLU to the type's accuracy: for fp32 the library's exponential
// and a quotient, each within 2 units in the last place, and -0 from -88.8 on, where e^-z leaves the range; for the
// 16-bit types the fast exponential, off by some 1.2 |z| units of fp32, and -0 from -87.4 on, where the fast quotient
// gives 0 and SiLU is above -1.1e-36.
template <typename T>
__device__ __forceinline__ float activated(float z, int activation)
{
    if (activation == CBS_ACT_SILU) {
        if constexpr (sizeof(T) == 4) {
            const float s = 1.0f + expf(-z), k = s > 8.0e37f ? 0.00390625f : 1.0f;
            return __fdividef(z, s * k) * k;
        }
        return __fdividef(z, 1.0f + __expf(-z));
    }
    if (activation == CBS_ACT_RELU) return z < 0.0f ? 0.0f : z;  // keeps NaN
    return z;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float2 lds_pair(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_pair(uint32_t addr, float2 v)
{
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

// One output: the general form.
template <typename T>
__device__ __forceinline__ void finish_one(const LinearEpilogue &e, float sum, long long m, int n)
{
    float z = sum * (__ldg(e.a_scale + m) * __ldg(e.w_scale + n));
    if (e.bias) z += __ldg(e.bias + n);
    z = activated<T>(z, e.activation);
    if (e.residual) z += to_float(static_cast<const T *>(e.residual)[m * e.residual_stride + n]);
    from_float(z, static_cast<T *>(e.y) + m * e.y_stride + n);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// min(a, b, c); a NaN among them is the result.
__device__ __forceinline__ float least_of(float a, float b, float c)
{
    float m;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// 1 + e^-z of two values, with e^-z = 2^-u, u = z log2(e), for z from -43 to 10^30.  For fp32 with what u loses in its
// rounding and in that of log2(e): 2^(-u + d) = 2^-u (1 + d ln 2) but for d^2, where d is below 2^-16 unless e^-z is 0.
template <typename T>
__device__ __forceinline__ float2 one_plus_exp_of_minus(float2 z)
{
    const float2 one = make_float2(1.0f, 1.0f), u = __fmul2_rn(z, make_float2(kLog2E, kLog2E));
    const float2 e = make_float2(exp2_approx(-u.x), exp2_approx(-u.y));
    if constexpr (sizeof(T) != 4) return __fadd2_rn(e, one);
    float2 d = __ffma2_rn(z, make_float2(-kLog2E, -kLog2E), u);
    d = __ffma2_rn(z, make_float2(-kLog2ERest, -kLog2ERest), d);
    return __ffma2_rn(e, __ffma2_rn(d, make_float2(0.693147181f, 0.693147181f), one), one);
}

// SiLU of 32 values, two at a time with one reciprocal between them, 1/a = b * (1 / (a b)): three
// special-function operations a pair instead of four, which set the pace.  Values of -43 and below, for
// which a b could leave the range, and NaN, which would spread to its neighbour, take the single form.  Accurate to
// the type T of the output, as in activated().  `stg` is the warp's own shared memory (finish_block): the single form
// in fp32, which is long, goes through it a value at a time, so that it stands in the code once.
template <typename T>
__device__ __forceinline__ void silu32(float *v, uint32_t stg, int lane)
{
    float least = v[0];
#pragma unroll
    for (int i = 1; i < 31; i += 2) least = least_of(least, v[i], v[i + 1]);
    least = least_of(least, v[31], v[31]);
    bool paired = least > -43.0f;
    if constexpr (sizeof(T) == 4) {
        float most = v[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) most = fmaxf(most, v[i]);
        paired = paired && most < 1e30f;
    }
    if (__all_sync(0xffffffffu, paired)) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 z = make_float2(v[i], v[i + 1]), s = one_plus_exp_of_minus<T>(z);
            const float r = __fdividef(1.0f, s.x * s.y);
            const float2 y = __fmul2_rn(z, __fmul2_rn(make_float2(s.y, s.x), make_float2(r, r)));
            v[i] = y.x;
            v[i + 1] = y.y;
        }
    } else if constexpr (sizeof(T) == 4) {
        __syncwarp();  // the block before has been read
        const uint32_t mine = stg + 4 * (uint32_t)lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) dev::sts_u32(mine + 128 * i, __float_as_uint(v[i]));
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            dev::sts_u32(mine + 128 * i,
                         __float_as_uint(activated<T>(__uint_as_float(dev::lds_u32(mine + 128 * i)), CBS_ACT_SILU)));
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(dev::lds_u32(mine + 128 * i));
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = activated<T>(v[i], CBS_ACT_SILU);
    }
}

// A warp's 32 rows x 32 columns of a TMEM accumulator from column `col` on, in the layout of a matrix
// instruction's result: with g = lane / 4 and t = lane % 4, v[16 h + 4 j + 2 i + e] is row 16 h + 8 i + g,
// column 8 j + 2 t + e.  A lane so holds 8 columns of 4 rows and needs the scales of those only.
__device__ __forceinline__ void load_block(uint32_t taddr, uint32_t col, uint32_t *v)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t *r = v + 16 * h;
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32"
            " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr + ((uint32_t)(16 * h) << 16) + col));
    }
}

// What becomes of such a block, from row row0 and column col0 of the output: sums in v, row_scale[i] the
// scale of row 8 i + g, the columns' 32 scales and 32 biases in shared memory at `params`.  Rows and
// columns past the end are computed and not stored.  `stg` is the warp's own 32 x 32 elements of shared
// memory, through which lanes exchange pairs for runs of a row, so that each store covers whole sectors; its
// 16-byte pieces are swizzled so that neither direction meets a bank twice.  (With a row to each lane
// instead, 64 of a block's 112 shared-memory cycles went to the columns' scales: 25600x1024x256 took 25.9 us
// with its widening, this layout 24.9.)
template <typename T>
__device__ __forceinline__ void finish_block(const LinearEpilogue &e, const uint32_t *sums, uint32_t params,
                                             const float *row_scale, long long row0, int col0, uint32_t stg, int lane)
{
    constexpr int kPieces = 32 * sizeof(T) / 16;  // 16-byte pieces of a row
    constexpr int kPer = 16 / sizeof(T);          // elements of a piece
    const int g = lane >> 2, t = lane & 3;
    const bool whole = col0 + 32 <= e.n;
    const int rows = e.m - row0 < 32 ? (int)(e.m - row0) : 32;
    // Where piece q of row r lies, and this lane's pair j of row r.
    auto piece_at = [&](int r, int q) {
        const int turn = kPieces == 8 ? 2 * (r & 3) : (r >> 1) & 3;
        return stg + (uint32_t)(r * (32 * (int)sizeof(T)) + ((q ^ turn) * 16));
    };
    auto pair_at = [&](int r, int j) {
        return sizeof(T) == 4 ? piece_at(r, 2 * j + (t >> 1)) + (uint32_t)(t & 1) * 8 : piece_at(r, j) + (uint32_t)t * 4;
    };
    auto row_of = [&](int i) { return 8 * i + g; };  // rows 0 to 3 of this lane
    const int q = lane % kPieces, r0 = lane / kPieces;  // this lane's piece on the way to or from memory
    constexpr int kRowsAtOnce = 32 / kPieces;
    float2 v[16];  // [row of this lane][j]
    {
        float2 scale[4], bias[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            scale[j] = lds_pair(params + 4 * (8 * j + 2 * t));
            bias[j] = lds_pair(params + 128 + 4 * (8 * j + 2 * t));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t *s = sums + 16 * (i >> 1) + 4 * j + 2 * (i & 1);
                v[4 * i + j] = __ffma2_rn(make_float2(__uint_as_float(s[0]), __uint_as_float(s[1])),
                                          __fmul2_rn(scale[j], make_float2(row_scale[i], row_scale[i])), bias[j]);
            }
    }
    if (e.activation == CBS_ACT_SILU) {
        silu32<T>(reinterpret_cast<float *>(v), stg, lane);
    } else if (e.activation == CBS_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = make_float2(activated<T>(v[i].x, CBS_ACT_RELU), activated<T>(v[i].y, CBS_ACT_RELU));
    }
    __syncwarp();  // the block before has been read
    if (e.residual) {
        const T *res = static_cast<const T *>(e.residual) + row0 * e.residual_stride + col0;
        if (whole && e.vec_residual) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int r = i * kRowsAtOnce + r0;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < rows) w = *reinterpret_cast<const uint4 *>(res + r * e.residual_stride + q * kPer);
                dev::sts_v4(piece_at(r, q), w.x, w.y, w.z, w.w);
            }
        } else if (col0 + lane < e.n) {
            // An element a lane, a row at a time (a lane loading its own pairs took eight rows' sectors an
            // instruction: 1872x10746x320 92 us, this 53).
#pragma unroll 8
            for (int r = 0; r < rows; ++r) {
                const uint32_t addr = piece_at(r, lane / kPer) + (uint32_t)(lane % kPer * (int)sizeof(T));
                if constexpr (sizeof(T) == 4)
                    dev::sts_u32(addr, reinterpret_cast<const uint32_t *>(res + r * e.residual_stride)[lane]);
                else
                    dev::sts_u16(addr, reinterpret_cast<const unsigned short *>(res + r * e.residual_stride)[lane]);
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4)
                    v[4 * i + j] = __fadd2_rn(v[4 * i + j], lds_pair(pair_at(row_of(i), j)));
                else
                    v[4 * i + j] = __fadd2_rn(v[4 * i + j], unpack2(dev::lds_u32(pair_at(row_of(i), j)), T()));
            }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4)
                sts_pair(pair_at(row_of(i), j), v[4 * i + j]);
            else
                dev::sts_u32(pair_at(row_of(i), j), pack2(v[4 * i + j].x, v[4 * i + j].y, T()));
        }
    __syncwarp();
    T *y = static_cast<T *>(e.y) + row0 * e.y_stride + col0;
    if (whole && e.vec_y) {
        uint4 w[kPieces];  // all loaded before the first is stored
#pragma unroll
        for (int i = 0; i < kPieces; ++i) w[i] = dev::lds_v4(piece_at(i * kRowsAtOnce + r0, q));
        T *to = y + r0 * e.y_stride + q * kPer;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (i * kRowsAtOnce + r0 < rows) *reinterpret_cast<uint4 *>(to + i * kRowsAtOnce * e.y_stride) = w[i];
    } else if (col0 + lane < e.n) {
        for (int r = 0; r < rows; ++r) {
            const uint32_t addr = piece_at(r, lane / kPer) + (uint32_t)(lane % kPer * (int)sizeof(T));
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(y + r * e.y_stride)[lane] = dev::lds_u32(addr);
            else
                reinterpret_cast<unsigned short *>(y + r * e.y_stride)[lane] = (unsigned short)dev::lds_u16(addr);
        }
    }
}

}  // namespace
#endif

}  // namespace cbs
