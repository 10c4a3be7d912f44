// linear_tile.cu -- the int8 linear layer for small products, in one launch at any alignment.
//
// Where a call is bound by its launches, one kernel that takes int8 as it lies is faster than two that
// widen it for the fast tensor cores first.  32 x 64 outputs per block of four warps; K in steps of 128
// through shared memory, the next step's bytes loading meanwhile; products by the 8-bit integer matrix
// instruction (150 TOP/s on this part, like __dp4a: the reason for the other kernels), exact in 32 bits.
// Bound by its launch and the latency of its steps: 64x256x256 5.5 us a call, 512x512x256 5.7 (the widened
// product 7.4, two launches).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cbs_internal.h"
#include "linear_device.cuh"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

constexpr int kRows = 32, kChannels = 64, kStep = 128;
constexpr int kPitch = kStep + 16;  // bytes of a row in shared memory: eight rows at one k meet 32 banks
constexpr int kThreads = 128;
constexpr int kPieces = (kRows + kChannels) * (kStep / 16) / kThreads;

struct TileArgs {
    LinearEpilogue e;
    const int8_t *a, *w;
    long long a_stride, w_stride;
    int k;
};

__device__ __forceinline__ void mma_s8(int (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// ALIGNED: rows of both on 16-byte boundaries.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) linear_tile_kernel(const TileArgs a)
{
    __shared__ __align__(16) uint8_t sm[kRows + kChannels][kPitch];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * kChannels, m0 = blockIdx.y * kRows;
    // This thread's pieces: 16 bytes at 16 * (tid % 8) of rows tid / 8 + 16 i, rows of a first.
    const int q = tid & 7, r0 = tid >> 3;
    const int8_t *src[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int r = r0 + 16 * i;
        src[i] = r < kRows ? a.a + (long long)min(m0 + r, (int)a.e.m - 1) * a.a_stride
                           : a.w + (long long)min(n0 + r - kRows, a.e.n - 1) * a.w_stride;
    }
    RawPiece next[kPieces];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (ALIGNED)
                next[i].lo = load_or_zero(src[i] + k0 + q * 16, k0 + q * 16 < a.k);
            else
                next[i] = load_raw(src[i], k0 + q * 16, a.k);
        }
    };
    // What was loaded for the step at k0.  Rows of a are zeros past k, which makes what the weights hold there
    // harmless.
    auto piece = [&](int i, int k0) {
        const uint4 v = ALIGNED ? next[i].lo : shifted(next[i], src[i], k0 + q * 16);
        return i < kRows / 16 ? within(v, k0 + q * 16, a.k) : v;
    };
    load(0);
    int acc[4][4] = {};
    const int wm = (warp & 1) * 16, wn = kRows + (warp >> 1) * 32;  // the warp's 16 rows, and 32 channels
    for (int k0 = 0; k0 < a.k; k0 += kStep) {
        __syncthreads();  // the step before has been read
#pragma unroll
        for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4 *>(&sm[r0 + 16 * i][q * 16]) = piece(i, k0);
        __syncthreads();
        if (k0 + kStep < a.k) load(k0 + kStep);
#pragma unroll
        for (int kk = 0; kk < kStep; kk += 32) {
            auto word = [&](int r, int b) { return *reinterpret_cast<const uint32_t *>(&sm[r][kk + b]); };
            const uint32_t fa[4] = {word(wm + g, 4 * t), word(wm + g + 8, 4 * t), word(wm + g, 4 * t + 16),
                                    word(wm + g + 8, 4 * t + 16)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t fb[2] = {word(wn + 8 * j + g, 4 * t), word(wn + 8 * j + g, 4 * t + 16)};
                mma_s8(acc[j], fa, fb);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long m = m0 + wm + g + (i >> 1) * 8;
            const int n = n0 + wn - kRows + 8 * j + 2 * t + (i & 1);
            if (m < a.e.m && n < a.e.n) finish_one<T>(a.e, (float)acc[j][i], m, n);
        }
}

}  // namespace

float linear_tile_time(long long m, int n, int k, int sm_count)
{
    // Its launch, a block's own steps or all products at what the instruction reaches here, and the blocks'
    // epilogues.
    const float step = (float)((k + kStep - 1) / kStep);
    const float blocks = (float)((m + kRows - 1) / kRows) * (float)((n + kChannels - 1) / kChannels);
    const float all = blocks * kRows * kChannels * 2.0f * (float)k / 0.9e8f;
    return 3.0f + (step > all ? step : all) + 0.9f * blocks / (float)sm_count;
}

void linear_tile_plan(long long m, int n, int k, LinearPlan *plan)
{
    plan->kernel = CBS_LINEAR_TILE;
    plan->tile_rows = kRows;
    plan->tile_channels = kChannels;
    plan->k_steps = (k + kStep - 1) / kStep;
    plan->tiles = plan->workers = (int)((m + kRows - 1) / kRows * ((n + kChannels - 1) / kChannels));
}

bool linear_tile_supported(long long m, int n) { return (m + kRows - 1) / kRows <= 65535 && n > 0; }

template <bool ALIGNED>
static cudaError_t tile_launch(const TileArgs &a, int out_dtype, cudaStream_t stream)
{
    const dim3 grid((unsigned)((a.e.n + kChannels - 1) / kChannels), (unsigned)((a.e.m + kRows - 1) / kRows));
    switch (out_dtype) {
    case kF32: return launch_overlapped(linear_tile_kernel<float, ALIGNED>, grid, dim3(kThreads), 0, stream, 1, a);
    case kBf16: return launch_overlapped(linear_tile_kernel<__nv_bfloat16, ALIGNED>, grid, dim3(kThreads), 0, stream, 1, a);
    default: return launch_overlapped(linear_tile_kernel<__half, ALIGNED>, grid, dim3(kThreads), 0, stream, 1, a);
    }
}

cudaError_t linear_tile_launch(const LinearProblem &p, cudaStream_t stream)
{
    auto rows16 = [](const Rows &r) { return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.stride % 16 == 0; };
    TileArgs a{};
    a.e = linear_epilogue_of(p);
    a.a = static_cast<const int8_t *>(p.a.data);
    a.a_stride = p.a.stride;
    a.w = static_cast<const int8_t *>(p.w.data);
    a.w_stride = p.w.stride;
    a.k = p.k;
    return rows16(p.a) && rows16(p.w) ? tile_launch<true>(a, p.out_dtype, stream) : tile_launch<false>(a, p.out_dtype, stream);
}

}  // namespace cbs
