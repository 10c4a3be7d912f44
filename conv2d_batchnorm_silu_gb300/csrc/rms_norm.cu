// rms_norm.cu -- root-mean-square norm over the channels of each row, after the residual's addition
// where there is one, and its gradient.
//
//   total = x + residual, rounded to the activations' type (without a residual: x)
//   rstd = 1 / sqrt(sum_c total^2 / C + eps),  y = total * rstd * gamma
//
// and for the gradient, with h = total * rstd and g = dy * gamma,
//
//   dx = rstd * (g - h * mean_c(g * h)) [+ the gradient that arrives at total past the norm],
//   dgamma = sum_rows dy * h.
//
// The norm is of the rounded total: that is what the residual stream keeps, and what the gradient, which has
// nothing else, is the gradient of.  Sums, statistics and parameters are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cbs_internal.h"
#include "ptx.cuh"
#include "rows_device.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

struct RmsArgs {
    const void *x, *residual;
    void *total, *y;
    int8_t *q;
    float *row_scale;
    float *rstd;
    const float *gamma;
    long long x_stride, residual_stride, total_stride, y_stride, q_stride;
    long long rows;
    int c;
    float eps;
};

__device__ __forceinline__ float2 rounded(float2 v, float) { return v; }
template <typename T>
__device__ __forceinline__ float2 rounded(float2 v, T t) { return unpack(pack(v, t), t); }
__device__ __forceinline__ float rounded(float v, float) { return v; }
template <typename T>
__device__ __forceinline__ float rounded(float v, T)
{
    T t;
    from_float(v, &t);
    return to_float(t);
}

// One row per block at a time, read again for each sum and store: any width, alignment and stride.  Rows of more
// than 16384 elements (f32 8192) come here.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) rms_wide_kernel(const RmsArgs a)
{
    __shared__ float scratch[kWideThreads / 32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
        float s = 0.0f;
        if (a.residual) {
            // The total is written once and read back by the thread that wrote it: it may be the residual's own memory.
            const T *res = static_cast<const T *>(a.residual) + r * a.residual_stride;
            T *total = static_cast<T *>(a.total) + r * a.total_stride;
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) {
                const float v = rounded(to_float(x[i]) + to_float(res[i]), T());
                from_float(v, total + i);
                s = fmaf(v, v, s);
            }
            x = total;
        } else {
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) {
                const float v = to_float(x[i]);
                s = fmaf(v, v, s);
            }
        }
        const float rstd = 1.0f / sqrtf(block_sum<kWideThreads>(s, scratch) / (float)a.c + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
        auto value = [&](int i) { return to_float(x[i]) * rstd * (a.gamma ? a.gamma[i] : 1.0f); };
        unsigned most = 0;
        for (int i = threadIdx.x; i < a.c; i += kWideThreads) {
            const float v = value(i);
            if (a.y) from_float(v, static_cast<T *>(a.y) + r * a.y_stride + i);
            most = max(most, magnitude_bits(v));
        }
        if (a.q) {
            float inv;
            const float scale = row_scale_of(block_max<kWideThreads>(most, reinterpret_cast<unsigned *>(scratch)), &inv);
            if (threadIdx.x == 0) a.row_scale[r] = scale;
            int8_t *q = a.q + r * a.q_stride;
            for (int i = threadIdx.x; i < a.c; i += kWideThreads) q[i] = (int8_t)__float2int_rn(value(i) * inv);
        }
    }
}

// As norm_stream_kernel of the layer norm: blocks stay for many rows, a thread keeps gamma's columns in registers,
// and the coming rows of x and of the residual are copied to shared memory meanwhile, so that memory stays busy
// while a row is summed.  The residual's run is added as it is read, so a row takes no more registers than without.
// Bound by memory: bf16 with the residual, 16384x4096 89 us (6.0 TB/s).  Rows off 16-byte boundaries by their
// element-wise reads and stores: f16, 3001x777 8.3 us (2.2 TB/s).
constexpr int kRmsStages = 3;

template <typename T, int W, int NI, int TPR, bool QUANT>
__global__ void __launch_bounds__(norm_block(TPR), kSmThreads / norm_block(TPR)) rms_stream_kernel(const RmsArgs a)
{
    using R = Run<T, W>;
    constexpr int V = R::V, E = NI * V, kBlock = norm_block(TPR), kGroups = kBlock / TPR;
    constexpr bool kTogether = W == 2;  // a row's threads copy it together: what one reads, others have copied
    extern __shared__ __align__(16) unsigned char rms_ring[];  // [stage][x, residual][run][thread] slots, or [group] rows
    __shared__ float scratch[2][2][TPR > 32 ? TPR / 32 : 1];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const int inputs = a.residual ? 2 : 1;
    const long long step = (long long)gridDim.x * kGroups;
    // Of what a thread may hold, nothing lies in the row from past(i)'s run or unused(e)'s pair on.
    constexpr bool kSkips = W != 2;
    auto past = [&](int i) { return kSkips && i > 0 && i * V % (V < 4 ? 4 : V) == 0 && i * TPR * V >= a.c; };
    auto unused = [&](int e) { return kSkips && e > 0 && 2 * e % (V < 4 ? 4 : V) == 0 && 2 * e / V * TPR * V >= a.c; };
    auto column = [&](int i) { return (i * TPR + lane) * V; };
    auto x_at = [&](long long r) { return static_cast<const T *>(a.x) + r * a.x_stride; };
    auto residual_at = [&](long long r) { return static_cast<const T *>(a.residual) + r * a.residual_stride; };
    auto row_ring = [&](int stage, int which) {
        return rms_ring + ((stage * inputs + which) * kGroups + threadIdx.x / TPR) * row_bytes(E * TPR);
    };
    auto slot = [&](int stage, int which, int i) {
        return rms_ring + (((stage * inputs + which) * NI + i) * kBlock + threadIdx.x) * R::SLOT;
    };
    auto fetch = [&](long long r, int stage) {
        if (r < a.rows) {
            const T *x = x_at(r), *res = a.residual ? residual_at(r) : nullptr;
            if constexpr (kTogether) {
                fetch_row<TPR>(dev::smem_u32(row_ring(stage, 0)), x, a.c, lane);
                if (res) fetch_row<TPR>(dev::smem_u32(row_ring(stage, 1)), res, a.c, lane);
            } else {
                for (int i = 0; i < NI; ++i)
                    if (column(i) < a.c) {
                        R::copy(dev::smem_u32(slot(stage, 0, i)), x + column(i));
                        if (res) R::copy(dev::smem_u32(slot(stage, 1, i)), res + column(i));
                    }
            }
        }
        copy_commit();
    };
    long long r = (long long)blockIdx.x * kGroups + threadIdx.x / TPR;
    for (int s = 0; s < kRmsStages - 1; ++s) fetch(r + s * step, s);
    float2 g[(E + 1) / 2];
    for (int i = 0; i < NI; ++i)
        load_params<V>(a.gamma ? a.gamma + column(i) : nullptr, 1.0f, a.c - column(i), reinterpret_cast<float *>(g) + i * V);
    if constexpr (kTogether) {
        copy_wait<kRmsStages - 2>();
        __syncthreads();
    }
    const Width width(a.c);
    int stage = 0, parity = 0;
    // All groups of a block go round together; rows past the end are zeros and store nothing.
    for (long long base = (long long)blockIdx.x * kGroups; base < a.rows; base += step, r += step) {
        fetch(r + (kRmsStages - 1) * step, stage == 0 ? kRmsStages - 1 : stage - 1);
        // Rows copied together are waited for one round ahead: the barrier of this row's sums is also theirs.
        copy_wait<kTogether ? kRmsStages - 2 : kRmsStages - 1>();
        const bool live = r < a.rows;
        float2 v[E / 2];
        float *vs = reinterpret_cast<float *>(v);
#pragma unroll
        for (int i = 0; i < NI && !past(i); ++i) {
            if (live && column(i) < a.c) {
                if constexpr (kTogether)
                    R::get(row_ring(stage, 0) + start_of(x_at(r)) + column(i) * sizeof(T), vs + i);
                else if constexpr (V == 1)
                    R::get(slot(stage, 0, i), vs + i);
                else
                    R::get(slot(stage, 0, i), v + i * (V / 2));
                if (a.residual) {
                    T *total = static_cast<T *>(a.total) + r * a.total_stride + column(i);
                    if constexpr (V == 1) {
                        float t;
                        if constexpr (kTogether)
                            R::get(row_ring(stage, 1) + start_of(residual_at(r)) + column(i) * sizeof(T), &t);
                        else
                            R::get(slot(stage, 1, i), &t);
                        vs[i] = rounded(vs[i] + t, T());
                        R::store(total, vs + i);
                    } else {
                        float2 t[V / 2];
                        R::get(slot(stage, 1, i), t);
                        for (int j = 0; j < V / 2; ++j) v[i * (V / 2) + j] = rounded(__fadd2_rn(v[i * (V / 2) + j], t[j]), T());
                        R::store(total, v + i * (V / 2));
                    }
                }
            } else {
                for (int j = 0; j < V; ++j) vs[i * V + j] = 0.0f;
            }
        }
        float2 s = both(0.0f);
#pragma unroll
        for (int e = 0; e < E / 2 && !unused(e); ++e) s = __ffma2_rn(v[e], v[e], s);
        // One rounding of the mean square more than a division, and 2 units in the last place of the root.
        const float rstd = rsqrtf(row_sum<TPR>(s.x + s.y, scratch[parity][0]) * width.hi + a.eps);
        if (a.rstd && lane == 0 && live) a.rstd[r] = rstd;
#pragma unroll
        for (int e = 0; e < E / 2 && !unused(e); ++e) v[e] = __fmul2_rn(__fmul2_rn(v[e], both(rstd)), g[e]);
        if (live && (!QUANT || a.y)) {
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
        if (QUANT) {
            float most = 0.0f;
#pragma unroll
            for (int e = 0; e < E / 2 && !unused(e); ++e) most = most_of(most, v[e].x, v[e].y);
            most = row_most<TPR>(most, scratch[parity][1]);
            float inv;
            const float scale = row_scale_of(__float_as_uint(most), &inv);
            if (lane == 0 && live) a.row_scale[r] = scale;
            // Rounded to nearest even by adding 1.5 * 2^23; scalar products, as in norm_stream_kernel.
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
        }
        if (kTogether && TPR <= 32) __syncwarp();
        stage = stage + 1 == kRmsStages ? 0 : stage + 1;
        parity ^= 1;
    }
    copy_wait<0>();
}

template <typename T, int W, int NI, int TPR>
cudaError_t rms_stream_launch(const RmsArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int kBlock = norm_block(TPR), kRows = kBlock / TPR;
    constexpr int kInput = kRmsStages * (W == 2 ? kRows * row_bytes(NI * TPR) : NI * kBlock * Run<T, W>::SLOT);
    const int smem = kInput * (a.residual ? 2 : 1);
    const long long need = (a.rows + kRows - 1) / kRows, room = (long long)sm_count * (kSmThreads / kBlock);
    const dim3 grid((unsigned)(need < room ? need : room)), block(kBlock);
    static bool allowed[2][kMaxDevices] = {};
    if (2 * kInput > 46 * 1024) {  // the sums take some of the first 48 KB
        const cudaError_t e = a.q ? allow_dynamic_smem(rms_stream_kernel<T, W, NI, TPR, true>, 2 * kInput, allowed[1])
                                  : allow_dynamic_smem(rms_stream_kernel<T, W, NI, TPR, false>, 2 * kInput, allowed[0]);
        if (e != cudaSuccess) return e;
    }
    return a.q ? launch_overlapped(rms_stream_kernel<T, W, NI, TPR, true>, grid, block, smem, stream, 1, a)
               : launch_overlapped(rms_stream_kernel<T, W, NI, TPR, false>, grid, block, smem, stream, 1, a);
}

// The fewest threads, a power of two of them, that hold a row, as for the layer norm.
template <typename T, int W, int NI>
cudaError_t rms_stream_pick(const RmsArgs &a, int sm_count, cudaStream_t stream, bool *done)
{
    constexpr int kHeld = NI * Run<T, W>::V;
    *done = true;
    if (a.c <= 4 * kHeld) return rms_stream_launch<T, W, NI, 4>(a, sm_count, stream);
    if (a.c <= 8 * kHeld) return rms_stream_launch<T, W, NI, 8>(a, sm_count, stream);
    if (a.c <= 16 * kHeld) return rms_stream_launch<T, W, NI, 16>(a, sm_count, stream);
    if (a.c <= 32 * kHeld) return rms_stream_launch<T, W, NI, 32>(a, sm_count, stream);
    if (a.c <= 64 * kHeld) return rms_stream_launch<T, W, NI, 64>(a, sm_count, stream);
    if (a.c <= 128 * kHeld) return rms_stream_launch<T, W, NI, 128>(a, sm_count, stream);
    if (a.c <= 256 * kHeld) return rms_stream_launch<T, W, NI, 256>(a, sm_count, stream);
    if (a.c <= 512 * kHeld) return rms_stream_launch<T, W, NI, 512>(a, sm_count, stream);
    *done = false;
    return cudaSuccess;
}

// 16-bit rows off 16-byte boundaries: 16 elements a thread, or 32 where 128 threads would not hold the row.
template <typename T>
cudaError_t rms_together_pick(const RmsArgs &a, int sm_count, cudaStream_t stream, bool *done)
{
    *done = true;
    if (a.c <= 16 * 8) return rms_stream_launch<T, 2, 16, 8>(a, sm_count, stream);
    if (a.c <= 16 * 16) return rms_stream_launch<T, 2, 16, 16>(a, sm_count, stream);
    if (a.c <= 16 * 32) return rms_stream_launch<T, 2, 16, 32>(a, sm_count, stream);
    if (a.c <= 16 * 64) return rms_stream_launch<T, 2, 16, 64>(a, sm_count, stream);
    if (a.c <= 16 * 128) return rms_stream_launch<T, 2, 16, 128>(a, sm_count, stream);
    if (a.c <= 32 * 128) return rms_stream_launch<T, 2, 32, 128>(a, sm_count, stream);
    if (a.c <= 32 * 256) return rms_stream_launch<T, 2, 32, 256>(a, sm_count, stream);
    if (a.c <= 32 * 512) return rms_stream_launch<T, 2, 32, 512>(a, sm_count, stream);
    *done = false;
    return cudaSuccess;
}

template <typename T>
cudaError_t rms_launch_t(const RmsArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    const bool wide_loads = a.c % V == 0 && aligned_for(a.x, a.x_stride, sizeof(T), 16) &&
                            (!a.residual || (aligned_for(a.residual, a.residual_stride, sizeof(T), 16) &&
                                             aligned_for(a.total, a.total_stride, sizeof(T), 16))) &&
                            (!a.y || aligned_for(a.y, a.y_stride, sizeof(T), 16)) &&
                            (!a.q || aligned_for(a.q, a.q_stride, 1, V)) && aligned_for(a.gamma, 0, 4, 16);
    bool done = false;
    cudaError_t e;
    if (wide_loads)
        e = rms_stream_pick<T, 16, 4>(a, sm_count, stream, &done);
    else if constexpr (sizeof(T) == 4)
        e = rms_stream_pick<T, 4, 16>(a, sm_count, stream, &done);
    else
        e = rms_together_pick<T>(a, sm_count, stream, &done);
    if (done) return e;
    return launch_overlapped(rms_wide_kernel<T>, dim3(blocks_for_rows(a.rows)), dim3(kWideThreads), 0, stream, 1, a);
}

}  // namespace

cudaError_t rms_norm_launch(const RmsNormProblem &p, int sm_count, cudaStream_t stream)
{
    RmsArgs a{};
    a.x = p.x.data;
    a.x_stride = p.x.stride;
    a.residual = p.residual.data;
    a.residual_stride = p.residual.stride;
    a.total = p.total.data;
    a.total_stride = p.total.stride;
    a.y = p.y.data;
    a.y_stride = p.y.stride;
    a.q = static_cast<int8_t *>(p.q.data);
    a.q_stride = p.q.stride;
    a.row_scale = p.row_scale;
    a.rstd = p.rstd;
    a.gamma = p.gamma;
    a.rows = p.rows;
    a.c = p.c;
    a.eps = p.eps;
    switch (p.dtype) {
    case kF32: return rms_launch_t<float>(a, sm_count, stream);
    case kBf16: return rms_launch_t<__nv_bfloat16>(a, sm_count, stream);
    default: return rms_launch_t<__half>(a, sm_count, stream);
    }
}

}  // namespace cbs
