// linear_int8.cu -- the linear layer over 8-bit integers:
//
//   y[m][n] = act( (sum_k a[m][k] * w[n][k]) * (a_scale[m] * w_scale[n]) + bias[n] ) [+ residual[m][n]]
//
// a row's scale and a channel's scale multiply the whole sum, so the sum itself
// is of integers and the scales, bias, activation and residual are an epilogue
// on it, applied before the one rounding to the output's type.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cbs_internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

struct LinearArgs {
    LinearEpilogue e;
    const int8_t *a, *w;
    long long a_stride, w_stride;
    int k;
};

// 64 x 64 outputs per block of 256 threads (4 x 4 each), K in steps of 64 through shared
// memory, four products per __dp4a: any size, alignment and stride.
constexpr int kTile = 64;
constexpr int kStepK = 64;
template <typename T>
__global__ void __launch_bounds__(256) linear_tile_kernel(const LinearArgs a)
{
    __shared__ int sa[kTile][kStepK / 4 + 1], sw[kTile][kStepK / 4 + 1];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const long long m0 = (long long)blockIdx.x * kTile;
    const int n0 = blockIdx.y * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < a.k; k0 += kStepK) {
        for (int i = threadIdx.x; i < kTile * kStepK; i += 256) {
            const int r = i / kStepK, c = i % kStepK, k = k0 + c;
            int8_t va = 0, vw = 0;
            if (k < a.k && m0 + r < a.e.m) va = a.a[(m0 + r) * a.a_stride + k];
            if (k < a.k && n0 + r < a.e.n) vw = a.w[(long long)(n0 + r) * a.w_stride + k];
            reinterpret_cast<int8_t *>(sa[r])[c] = va;
            reinterpret_cast<int8_t *>(sw[r])[c] = vw;
        }
        __syncthreads();
        for (int c = 0; c < kStepK / 4; ++c)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(sa[ty + 16 * i][c], sw[tx + 16 * j][c], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long m = m0 + ty + 16 * i;
            const int n = n0 + tx + 16 * j;
            if (m < a.e.m && n < a.e.n) finish_one<T>(a.e, (float)acc[i][j], m, n);
        }
}

template <typename T>
cudaError_t linear_launch_t(const LinearArgs &a, cudaStream_t stream)
{
    const dim3 grid((unsigned)((a.e.m + kTile - 1) / kTile), (unsigned)((a.e.n + kTile - 1) / kTile));
    return launch_overlapped(linear_tile_kernel<T>, grid, dim3(256), 0, stream, 1, a);
}

}  // namespace

bool linear_on_tensor_cores(long long m, int n, int k) { return m > 16 && k > 0 && tc_linear_supported(m, n, k); }

long long linear_workspace_bytes(long long m, int n, int k, int sm_count)
{
    (void)sm_count;
    return m > 0 && n > 0 && linear_on_tensor_cores(m, n, k) ? tc_linear_workspace_bytes(m, n, k) : 0;
}

cudaError_t linear_launch(const LinearProblem &p, int sm_count, cudaStream_t stream)
{
    if (linear_on_tensor_cores(p.m, p.n, p.k)) return tc_linear_launch(p, sm_count, stream);
    LinearArgs a{};
    a.e = linear_epilogue_of(p);
    a.a = static_cast<const int8_t *>(p.a.data);
    a.a_stride = p.a.stride;
    a.w = static_cast<const int8_t *>(p.w.data);
    a.w_stride = p.w.stride;
    a.k = p.k;
    switch (p.out_dtype) {
    case kF32: return linear_launch_t<float>(a, stream);
    case kBf16: return linear_launch_t<__nv_bfloat16>(a, stream);
    default: return linear_launch_t<__half>(a, stream);
    }
}

}  // namespace cbs
