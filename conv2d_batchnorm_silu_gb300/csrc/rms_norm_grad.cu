// rms_norm_grad.cu -- the gradient of the root-mean-square norm (rms_norm.cu has the formulas).
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

struct RmsGradArgs {
    const void *dy, *x, *residual;
    void *dx;
    const float *gamma;
    const float *rstd;
    float *dgamma;
    float *partial;
    long long dy_stride, x_stride, residual_stride, dx_stride;
    long long rows;
    int c;
    int partial_rows;
};

// dx, one row per block at a time, for rows of more than 8192 elements.  The addition may be in dx's own memory.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) rms_grad_wide_kernel(const RmsGradArgs a)
{
    __shared__ float scratch[kWideThreads / 32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
        const T *res = a.residual ? static_cast<const T *>(a.residual) + r * a.residual_stride : nullptr;
        T *dx = static_cast<T *>(a.dx) + r * a.dx_stride;
        const float rstd = a.rstd[r];
        float s = 0.0f;
        for (int i = threadIdx.x; i < a.c; i += kWideThreads)
            s = fmaf(to_float(dy[i]) * (a.gamma ? a.gamma[i] : 1.0f), to_float(x[i]) * rstd, s);
        s = block_sum<kWideThreads>(s, scratch) / (float)a.c;
        for (int i = threadIdx.x; i < a.c; i += kWideThreads) {
            const float g = to_float(dy[i]) * (a.gamma ? a.gamma[i] : 1.0f);
            const float v = rstd * fmaf(-s, to_float(x[i]) * rstd, g);
            from_float(res ? v + to_float(res[i]) : v, dx + i);
        }
    }
}

// Partial sums of dy * h over every partial_rows-th row, one column per thread.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) rms_grad_columns_kernel(const RmsGradArgs a)
{
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int i = blockIdx.x * kWideThreads + threadIdx.x;
    if (i >= a.c) return;
    float s = 0.0f;
    for (long long r = blockIdx.y; r < a.rows; r += a.partial_rows)
        s = fmaf(to_float(static_cast<const T *>(a.dy)[r * a.dy_stride + i]),
                 to_float(static_cast<const T *>(a.x)[r * a.x_stride + i]) * a.rstd[r], s);
    a.partial[(long long)blockIdx.y * a.c + i] = s;
}

// Column sums of partial[partial_rows][c] in a fixed order, as the layer norm's join: 32 columns per block, 32 runs of
// rows summed side by side, all of a thread's loads in flight at once.
constexpr int kJoinRuns = 32, kJoinLoads = 10;
__global__ void __launch_bounds__(32 * kJoinRuns) rms_grad_join_kernel(const RmsGradArgs a)
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
            v[j] = r < a.partial_rows && i < a.c ? a.partial[(long long)r * a.c + i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kJoinLoads; ++j) s += v[j];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = part[threadIdx.x][threadIdx.y];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int column = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && column < a.c) a.dgamma[column] = s;
}

// As the layer norm's gradient: each thread keeps gamma and the running sums of dy * h for its own columns in
// registers while x, dy and the gradient past the norm stream by, so that each is read once.  At the end the rows of
// a block are joined in shared memory, and each block writes one row of partial sums, which rms_grad_join_kernel
// adds up in order.  bf16 with the join: 16384x4096 with the gradient past the norm 82 us (6.6 TB/s), 25600x256 without it
// 8.6, of which the join and the launches' ends are a third.
constexpr int kGradElements = 16;  // of a row per thread
constexpr int grad_block(int tpr) { return tpr < 256 ? 256 : tpr; }
// Rounds of the ring: as many as 512 threads' rings find room for in an SM's shared memory.
template <typename T, int W, bool ADDS>
constexpr int grad_stages() { return sizeof(T) == 4 ? (ADDS ? 2 : 3) : (W == 2 && !ADDS ? 4 : 3); }

// Sum over the TPR threads of a row; scratch: a float for each warp of the block.
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float *scratch)
{
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        constexpr int warps = TPR / 32;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) scratch[warp] = v;
        __syncthreads();
        v = 0.0f;
        for (int i = 0; i < warps; ++i) v += scratch[warp / warps * warps + i];
    }
    return v;
}

template <typename T, int W, int TPR, bool ADDS>
__global__ void __launch_bounds__(grad_block(TPR), kSmThreads / grad_block(TPR)) rms_grad_stream_kernel(const RmsGradArgs a)
{
    using R = Run<T, W>;
    constexpr int V = R::V, E = kGradElements, NI = E / V, kBlock = grad_block(TPR), kGroups = kBlock / TPR;
    constexpr int kStages = grad_stages<T, W, ADDS>(), kInputs = ADDS ? 3 : 2;
    constexpr bool kTogether = W == 2;  // a row's threads copy it together: what one reads, others have copied
    extern __shared__ __align__(16) unsigned char grad_ring[];  // [stage][x, dy, residual][run][thread] slots or [group] rows; then the join
    __shared__ float scratch[2][kBlock / 32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int lane = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * kGroups;
    constexpr bool kSkips = W != 2;
    auto past = [&](int i) { return kSkips && i > 0 && i * V % (V < 4 ? 4 : V) == 0 && i * TPR * V >= a.c; };
    auto unused = [&](int e) { return kSkips && e > 0 && 2 * e % (V < 4 ? 4 : V) == 0 && 2 * e / V * TPR * V >= a.c; };
    auto column = [&](int i) { return (i * TPR + lane) * V; };
    auto slot = [&](int stage, int which, int i) {
        return grad_ring + (((stage * kInputs + which) * NI + i) * kBlock + threadIdx.x) * R::SLOT;
    };
    auto row_ring = [&](int stage, int which) {
        return grad_ring + ((stage * kInputs + which) * kGroups + threadIdx.x / TPR) * row_bytes(E * TPR);
    };
    auto row_at = [&](int which, long long r) {
        const void *p = which == 0 ? a.x : which == 1 ? a.dy : a.residual;
        return static_cast<const T *>(p) + r * (which == 0 ? a.x_stride : which == 1 ? a.dy_stride : a.residual_stride);
    };
    auto fetch = [&](long long r, int stage) {
        if (r < a.rows) {
#pragma unroll
            for (int which = 0; which < kInputs; ++which) {
                const T *row = row_at(which, r);
                if constexpr (kTogether) {
                    fetch_row<TPR>(dev::smem_u32(row_ring(stage, which)), row, a.c, lane);
                } else {
                    for (int i = 0; i < NI; ++i)
                        if (column(i) < a.c) R::copy(dev::smem_u32(slot(stage, which, i)), row + column(i));
                }
            }
        }
        copy_commit();
    };
    auto moment = [&](long long r) { return r < a.rows ? __ldg(a.rstd + r) : 0.0f; };
    // Run i of an input's row r, as floats.
    auto get = [&](int stage, int which, long long r, int i, float2 *v) {
        if constexpr (kTogether)
            R::get(row_ring(stage, which) + start_of(row_at(which, r)) + column(i) * sizeof(T), reinterpret_cast<float *>(v) + i);
        else if constexpr (V == 1)
            R::get(slot(stage, which, i), reinterpret_cast<float *>(v) + i);
        else
            R::get(slot(stage, which, i), v + i * (V / 2));
    };
    long long r = (long long)blockIdx.x * kGroups + threadIdx.x / TPR;
    for (int s = 0; s < kStages - 1; ++s) fetch(r + s * step, s);
    float next = moment(r);
    float2 gamma[E / 2], dg[E / 2];
    for (int i = 0; i < NI; ++i)
        load_params<V>(a.gamma ? a.gamma + column(i) : nullptr, 1.0f, a.c - column(i),
                       reinterpret_cast<float *>(gamma) + i * V);
    for (int e = 0; e < E / 2; ++e) dg[e] = both(0.0f);
    if constexpr (kTogether) {
        copy_wait<kStages - 2>();
        __syncthreads();
    }
    const Width width(a.c);
    int stage = 0, parity = 0;
    for (long long base = (long long)blockIdx.x * kGroups; base < a.rows; base += step, r += step) {
        fetch(r + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        const float rstd = next;
        next = moment(r + step);
        copy_wait<kTogether ? kStages - 2 : kStages - 1>();
        const bool live = r < a.rows;
        // The added gradient: read along with the others where the ring is not a thread's own, as the barrier of the sum
        // lets other threads copy over it, and else just before it is added.
        float2 h[E / 2], g[E / 2], t[kTogether && ADDS ? E / 2 : 1];
        float *hs = reinterpret_cast<float *>(h), *gs = reinterpret_cast<float *>(g);
#pragma unroll
        for (int i = 0; i < NI && !past(i); ++i) {
            if (live && column(i) < a.c) {
                get(stage, 0, r, i, h);
                get(stage, 1, r, i, g);
                if constexpr (kTogether && ADDS) get(stage, 2, r, i, t);
            } else {
                for (int j = 0; j < V; ++j) hs[i * V + j] = gs[i * V + j] = 0.0f;
            }
        }
        float2 s = both(0.0f);
#pragma unroll
        for (int e = 0; e < E / 2 && !unused(e); ++e) {
            const float2 d = g[e];
            h[e] = __fmul2_rn(h[e], both(rstd));
            dg[e] = __ffma2_rn(d, h[e], dg[e]);
            g[e] = __fmul2_rn(d, gamma[e]);
            s = __ffma2_rn(g[e], h[e], s);
        }
        const float mean = width.share(group_sum<TPR>(s.x + s.y, scratch[parity]));
#pragma unroll
        for (int e = 0; e < E / 2 && !unused(e); ++e) h[e] = __fmul2_rn(__ffma2_rn(h[e], both(-mean), g[e]), both(rstd));
        if (live) {
            T *dx = static_cast<T *>(a.dx) + r * a.dx_stride;
#pragma unroll
            for (int i = 0; i < NI && !past(i); ++i)
                if (column(i) < a.c) {
                    if constexpr (ADDS) {
                        if constexpr (!kTogether) get(stage, 2, r, i, g);
                        if constexpr (kTogether)
                            hs[i] += reinterpret_cast<float *>(t)[i];
                        else if constexpr (V == 1)
                            hs[i] += gs[i];
                        else
                            for (int j = 0; j < V / 2; ++j) h[i * (V / 2) + j] = __fadd2_rn(h[i * (V / 2) + j], g[i * (V / 2) + j]);
                    }
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
    float *out = a.partial + (long long)blockIdx.x * a.c;
    float *dgs = reinterpret_cast<float *>(dg);
    if constexpr (kGroups == 1) {
        for (int i = 0; i < NI; ++i)
            for (int j = 0; j < V; ++j)
                if (column(i) + j < a.c) {
                    if constexpr (V >= 4) {
                        const int e = i * V + j;
                        if (j % 4 == 0)
                            *reinterpret_cast<float4 *>(out + column(i) + j) =
                                make_float4(dgs[e], dgs[e + 1], dgs[e + 2], dgs[e + 3]);
                    } else {
                        out[column(i) + j] = dgs[i * V + j];
                    }
                }
    } else {
        // The block's rows side by side in shared memory, [row][element][thread]; those of one warp are joined by
        // shuffles before.
        constexpr int kSide = TPR < 32 ? kBlock / 32 : kGroups;
        for (int o = TPR; o < 32; o <<= 1)
            for (int e = 0; e < E; ++e) dgs[e] += __shfl_xor_sync(0xffffffffu, dgs[e], o);
        float *join = reinterpret_cast<float *>(grad_ring);
        __syncthreads();  // the ring is no longer read
        if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
            float *mine = join + (TPR < 32 ? threadIdx.x / 32 : threadIdx.x / TPR) * (E * TPR) + lane;
            for (int e = 0; e < E; ++e) mine[e * TPR] = dgs[e];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.c; c += kBlock) {
            const int e = c / (TPR * V) * V + c % V;
            const float *at = join + e * TPR + c / V % TPR;
            float sum = at[0];
            for (int t = 1; t < kSide; ++t) sum += at[t * (E * TPR)];
            out[c] = sum;
        }
    }
}

cudaError_t rms_grad_join(const RmsGradArgs &a, cudaStream_t stream)
{
    return launch_overlapped(rms_grad_join_kernel, dim3((unsigned)((a.c + 31LL) / 32)), dim3(32, kJoinRuns), 0, stream, 1, a);
}

template <typename T, int W, int TPR, bool ADDS>
cudaError_t rms_grad_stream_launch(RmsGradArgs a, int sm_count, cudaStream_t stream)
{
    constexpr int kBlock = grad_block(TPR), kRows = kBlock / TPR;
    constexpr int kRing = grad_stages<T, W, ADDS>() * (ADDS ? 3 : 2) *
                          (W == 2 ? kRows * row_bytes(kGradElements * TPR)
                                  : kGradElements / Run<T, W>::V * kBlock * Run<T, W>::SLOT);
    constexpr int kJoin = kRows > 1 ? (TPR < 32 ? kBlock / 32 : kRows) * kGradElements * TPR * 4 : 0;
    constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    static bool allowed[kMaxDevices] = {};
    if (kSmem > 46 * 1024) {  // the sums of a block take some of the first 48 KB
        cudaError_t e = allow_dynamic_smem(rms_grad_stream_kernel<T, W, TPR, ADDS>, kSmem, allowed);
        if (e != cudaSuccess) return e;
    }
    const long long need = (a.rows + kRows - 1) / kRows, room = (long long)sm_count * (kSmThreads / kBlock);
    a.partial_rows = (int)(need < room ? need : room);
    cudaError_t e = launch_overlapped(rms_grad_stream_kernel<T, W, TPR, ADDS>, dim3((unsigned)a.partial_rows), dim3(kBlock),
                                      kSmem, stream, 1, a);
    return e == cudaSuccess ? rms_grad_join(a, stream) : e;
}

template <typename T, int W, bool ADDS>
cudaError_t rms_grad_stream_pick(const RmsGradArgs &a, int sm_count, cudaStream_t stream)
{
    if (a.c <= 8 * kGradElements) return rms_grad_stream_launch<T, W, 8, ADDS>(a, sm_count, stream);
    if (a.c <= 16 * kGradElements) return rms_grad_stream_launch<T, W, 16, ADDS>(a, sm_count, stream);
    if (a.c <= 32 * kGradElements) return rms_grad_stream_launch<T, W, 32, ADDS>(a, sm_count, stream);
    if (a.c <= 64 * kGradElements) return rms_grad_stream_launch<T, W, 64, ADDS>(a, sm_count, stream);
    if (a.c <= 128 * kGradElements) return rms_grad_stream_launch<T, W, 128, ADDS>(a, sm_count, stream);
    if (a.c <= 256 * kGradElements) return rms_grad_stream_launch<T, W, 256, ADDS>(a, sm_count, stream);
    return rms_grad_stream_launch<T, W, 512, ADDS>(a, sm_count, stream);
}

template <typename T>
cudaError_t rms_grad_launch_t(const RmsGradArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T), W = sizeof(T) == 4 ? 4 : 2;
    if (a.c <= 512 * kGradElements) {
        const bool wide_loads = a.c % V == 0 && aligned_for(a.x, a.x_stride, sizeof(T), 16) &&
                                aligned_for(a.dy, a.dy_stride, sizeof(T), 16) &&
                                aligned_for(a.residual, a.residual_stride, sizeof(T), 16) &&
                                aligned_for(a.dx, a.dx_stride, sizeof(T), 16) && aligned_for(a.gamma, 0, 4, 16);
        if (a.residual)
            return wide_loads ? rms_grad_stream_pick<T, 16, true>(a, sm_count, stream)
                              : rms_grad_stream_pick<T, W, true>(a, sm_count, stream);
        return wide_loads ? rms_grad_stream_pick<T, 16, false>(a, sm_count, stream)
                          : rms_grad_stream_pick<T, W, false>(a, sm_count, stream);
    }
    // dgamma's sums first: dx may be written over the gradient that is added, but over nothing else.
    cudaError_t e = launch_overlapped(rms_grad_columns_kernel<T>,
                                      dim3((unsigned)((a.c + kWideThreads - 1) / kWideThreads), (unsigned)a.partial_rows),
                                      dim3(kWideThreads), 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    e = rms_grad_join(a, stream);
    if (e != cudaSuccess) return e;
    return launch_overlapped(rms_grad_wide_kernel<T>, dim3(blocks_for_rows(a.rows)), dim3(kWideThreads), 0, stream, 1, a);
}

}  // namespace

int rms_grad_partial_rows(long long rows, int sm_count)
{
    const long long most = 2LL * sm_count;  // rms_grad_stream_kernel's blocks at most
    return (int)(rows < most ? rows : most);
}

cudaError_t rms_norm_grad_launch(const RmsNormGradProblem &p, int sm_count, cudaStream_t stream)
{
    RmsGradArgs a{};
    a.dy = p.dy.data;
    a.dy_stride = p.dy.stride;
    a.x = p.x.data;
    a.x_stride = p.x.stride;
    a.residual = p.residual.data;
    a.residual_stride = p.residual.stride;
    a.dx = p.dx.data;
    a.dx_stride = p.dx.stride;
    a.gamma = p.gamma;
    a.rstd = p.rstd;
    a.dgamma = p.dgamma;
    a.partial = p.partial;
    a.rows = p.rows;
    a.c = p.c;
    a.partial_rows = p.partial_rows;
    switch (p.dtype) {
    case kF32: return rms_grad_launch_t<float>(a, sm_count, stream);
    case kBf16: return rms_grad_launch_t<__nv_bfloat16>(a, sm_count, stream);
    default: return rms_grad_launch_t<__half>(a, sm_count, stream);
    }
}

}  // namespace cbs
