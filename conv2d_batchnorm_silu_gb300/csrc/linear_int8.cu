// linear_int8.cu -- the linear layer over 8-bit integers:
//
//   y[m][n] = act( (sum_k a[m][k] * w[n][k]) * (a_scale[m] * w_scale[n]) + bias[n] ) [+ residual[m][n]]
//
// a row's scale and a channel's scale multiply the whole sum, so the sum itself
// is of integers and the scales, bias, activation and residual are an epilogue
// on it, applied before the one rounding to the output's type.
//
// Sizes in the linear layer's comments are rows x channels x K, times of one call without the host's part.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "cbs_internal.h"
#include "linear_device.cuh"
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

// ------------------------------------------------------------------ few rows
// Up to eight rows of a: the weights are read once, at memory speed, and four products at a time go
// into 32-bit integers with __dp4a.  A warp (or, where there are few channels, two to eight warps that
// split K) takes kFewChannels channels; a lane holds 16 bytes of each of their weights and goes through
// the rows of a with them, so a's bytes, which stay in L1, are read once for all the channels.  8192x8192
// weights, kernel alone: one row 12.1 us (5.5 TB/s of 6.8 for a copy; the start and the end of 2048 blocks are the
// rest), two 12.6, four 16.0, eight 20.1, where the products' rate counts (53 of 150 TOP/s, a's bytes from L1).
constexpr int kFewChannels = 4;
constexpr int kFewWarps = 8;

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int acc)
{
    acc = __dp4a((int)a.x, (int)b.x, acc);
    acc = __dp4a((int)a.y, (int)b.y, acc);
    acc = __dp4a((int)a.z, (int)b.z, acc);
    return __dp4a((int)a.w, (int)b.w, acc);
}

// 16 values from k0 < k.  ALIGNED: rows on 16-byte boundaries and k a multiple of 16.
template <bool ALIGNED>
struct Piece {
    uint4 v;
    __device__ __forceinline__ void load(const int8_t *row, int k0, int) { v = __ldg(reinterpret_cast<const uint4 *>(row + k0)); }
    __device__ __forceinline__ uint4 get(const int8_t *, int, int) const { return v; }
};
template <>
struct Piece<false> {
    RawPiece raw;
    __device__ __forceinline__ void load(const int8_t *row, int k0, int k) { raw = load_raw(row, k0, k); }
    __device__ __forceinline__ uint4 get(const int8_t *row, int k0, int) const { return shifted(raw, row, k0); }
};

template <typename T, int ROWS, bool ALIGNED>
__global__ void __launch_bounds__(32 * kFewWarps, ALIGNED && ROWS <= 2 ? 4 : (ROWS <= 2 || (ALIGNED && ROWS <= 4) ? 3 : 2)) linear_few_kernel(const LinearArgs a, int split_log2)
{
    constexpr int R = kFewChannels;
    __shared__ int part[kFewWarps][R * ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = 1 << split_log2, groups = kFewWarps >> split_log2;
    const int n0 = (blockIdx.x * groups + (warp >> split_log2)) * R;
    const int m = (int)a.e.m;
    if constexpr (ALIGNED) {
        const int n = blockIdx.x * groups * R + threadIdx.x;
        if (threadIdx.x < groups * R && n < a.e.n && a.k > 0) prefetch_l2(a.w + n * a.w_stride, (uint32_t)a.k);
    }
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    // This thread's output, whose scales load along with the weights.
    const int out_e = threadIdx.x % (R * ROWS), out_i = out_e / R;
    const int out_n = (blockIdx.x * groups + threadIdx.x / (R * ROWS)) * R + out_e % R;
    const bool has_out = threadIdx.x < groups * R * ROWS && out_i < m && out_n < a.e.n;
    float scale = 0.0f, bias = 0.0f, residual = 0.0f;
    if (has_out) {
        scale = __ldg(a.e.a_scale + out_i) * __ldg(a.e.w_scale + out_n);
        if (a.e.bias) bias = __ldg(a.e.bias + out_n);
        if (a.e.residual) residual = to_float(static_cast<const T *>(a.e.residual)[out_i * a.e.residual_stride + out_n]);
    }
    const int8_t *w[R], *x[ROWS];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = a.w + (long long)min(n0 + r, a.e.n - 1) * a.w_stride;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) x[i] = a.a + min(i, m - 1) * a.a_stride;
    int acc[R][ROWS] = {};
    const int step = split * 512;
    constexpr int kUnroll = ALIGNED && ROWS <= 4 ? 2 : 1;
#pragma unroll kUnroll
    for (int k0 = ((warp & (split - 1)) * 32 + lane) * 16; k0 < a.k; k0 += step) {
        Piece<ALIGNED> raw[R];
#pragma unroll
        for (int r = 0; r < R; ++r) raw[r].load(w[r], k0, a.k);
        uint4 wv[R];
#pragma unroll
        for (int r = 0; r < R; ++r) wv[r] = raw[r].get(w[r], k0, a.k);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            Piece<ALIGNED> rx;
            rx.load(x[i], k0, a.k);
            uint4 xv = rx.get(x[i], k0, a.k);
            if constexpr (!ALIGNED) xv = within(xv, k0, a.k);  // zeros here make what wv holds past k harmless
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r][i] = dot16(wv[r], xv, acc[r][i]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int s = __reduce_add_sync(0xffffffffu, acc[r][i]);
            if (lane == 0) part[warp][i * R + r] = s;
        }
    __syncthreads();
    static_assert(R * ROWS * kFewWarps <= 32 * kFewWarps, "one output a thread");
    if (has_out) {
        const int g = threadIdx.x / (R * ROWS);
        int s = 0;
        for (int t = 0; t < split; ++t) s += part[g * split + t][out_e];
        const float z = activated<T>(fmaf((float)s, scale, bias), a.e.activation) + residual;
        from_float(z, static_cast<T *>(a.e.y) + out_i * a.e.y_stride + out_n);
    }
}

// K is split among the warps of a block while each has two passes (1 KB) of it: many short blocks
// fill the SMs evenly.
int few_split_log2(int k)
{
    int split_log2 = 0;
    while (split_log2 < 3 && k >= 2048 << split_log2) ++split_log2;
    return split_log2;
}
int few_per_block(int split_log2) { return kFewChannels * (kFewWarps >> split_log2); }  // of a block

template <typename T, bool ALIGNED>
cudaError_t linear_few_launch(const LinearArgs &a, cudaStream_t stream)
{
    const int split_log2 = few_split_log2(a.k), per_block = few_per_block(split_log2);
    const dim3 grid((unsigned)((a.e.n + per_block - 1) / per_block)), block(32 * kFewWarps);
    if (a.e.m == 1) return launch_overlapped(linear_few_kernel<T, 1, ALIGNED>, grid, block, 0, stream, 1, a, split_log2);
    if (a.e.m == 2) return launch_overlapped(linear_few_kernel<T, 2, ALIGNED>, grid, block, 0, stream, 1, a, split_log2);
    if (a.e.m <= 4) return launch_overlapped(linear_few_kernel<T, 4, ALIGNED>, grid, block, 0, stream, 1, a, split_log2);
    return launch_overlapped(linear_few_kernel<T, 8, ALIGNED>, grid, block, 0, stream, 1, a, split_log2);
}

template <typename T>
cudaError_t linear_few_launch_t(const LinearArgs &a, cudaStream_t stream)
{
    auto rows16 = [](const int8_t *p, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 16 == 0;
    };
    return a.k % 16 == 0 && rows16(a.a, a.a_stride) && rows16(a.w, a.w_stride) ? linear_few_launch<T, true>(a, stream)
                                                                                  : linear_few_launch<T, false>(a, stream);
}

}  // namespace

// Rows up to which linear_few_kernel is the faster.
constexpr int kFewRows = 8;
// The kernels for more rows, chosen by what they are modelled to take: linear_tile.cu's one launch, weights
// widened on their way to the tensor cores (tc_linear_stream.cu), rows on theirs (the same kernel with the operands'
// sides changed), or both widened before (tc_linear.cu).
enum Path { kTile, kStreamed, kTurned, kWidened };

// Measured, us, tile / streamed / widened before: 24x614x243 5.2 / - / 6.0 (8.6 with the host's part), 64x1024x1024
// 11.2 / 5.3 / 8.9, 64 rows of 8192x8192 - / 21 / 74, 512 rows - / 81 / 87, 1024 rows - / 152 / 123.  Streamed with
// the sides changed / widened before: 25984x40x4800 37 / 132, 11609x128x4512 24 / 58, 100000x16x256 15 / 28,
// 25600x256x1024 39 / 31, 16384x512x512 36 / 17.
// A call takes the longer of its kernels and what its launches cost the host.
Path best_path(long long m, int n, int k, int sm_count, int align)
{
    const float tile = linear_tile_supported(m, n) ? linear_tile_time(m, n, k, sm_count) : 1e30f;
    const float before = tc_linear_time(m, n, k, sm_count);
    // Beyond 4096 rows sixteen row tiles would each widen the weights again.
    const float on_the_way = align > 0 && m <= 4096 ? tc_stream_time(m, n, k, align, false, sm_count) : 1e30f;
    const bool few_channels = n <= 1024 && m <= (1 << 30) && m * k < (1LL << 42);  // its steps fit an int
    const float turned = align > 0 && few_channels ? tc_stream_time(n, (int)m, k, align, true, sm_count) : 1e30f;
    const float times[4] = {fmaxf(tile, 4.6f), fmaxf(on_the_way, 7.4f), fmaxf(turned, 7.4f), fmaxf(before, 8.6f)};
    int best = kWidened;
    for (int i = 0; i < 3; ++i)
        if (times[i] < times[best]) best = i;
    return (Path)best;
}

long long path_workspace(Path path, long long m, int n, int k, int sm_count)
{
    switch (path) {
    case kTile: return 0;
    case kStreamed: return tc_stream_workspace_bytes(m, n, k, sm_count);
    case kTurned: return tc_stream_workspace_bytes(n, (int)m, k, sm_count);
    default: return tc_linear_workspace_bytes(m, n, k);
    }
}

long long linear_workspace_bytes(long long m, int n, int k, int sm_count)
{
    if (m <= kFewRows || n <= 0) return 0;
    // For any alignment that the call's matrices may have.
    long long most = 0;
    for (int align : {16, 4, 1, 0}) {
        const long long bytes = path_workspace(best_path(m, n, k, sm_count, align), m, n, k, sm_count);
        if (bytes > most) most = bytes;
    }
    return most;
}

LinearPlan linear_plan(long long m, int n, int k, int align, int sm_count)
{
    LinearPlan plan{};
    if (m == 0 || n == 0) return plan;
    plan.align = align == 16 ? 16 : 1;  // what the kernels but the streamed ones tell apart
    while (align > 1 && k % align != 0) align = align == 16 ? 4 : 1;
    if (m <= kFewRows) {
        plan.align = align == 16 ? 16 : 1;
        plan.kernel = CBS_LINEAR_FEW;
        plan.tile_rows = m <= 2 ? (int)m : (m <= 4 ? 4 : kFewRows);
        plan.tile_channels = few_per_block(few_split_log2(k));
        plan.k_steps = (k + (512 << few_split_log2(k)) - 1) / (512 << few_split_log2(k));
        plan.tiles = plan.workers = (n + plan.tile_channels - 1) / plan.tile_channels;
        return plan;
    }
    switch (best_path(m, n, k, sm_count, k > 0 ? align : 0)) {
    case kTile: linear_tile_plan(m, n, k, &plan); break;
    case kStreamed: tc_stream_plan(m, n, k, align, false, sm_count, &plan); break;
    case kTurned: tc_stream_plan(n, (int)m, k, align, true, sm_count, &plan); break;
    default: tc_linear_plan(m, n, k, sm_count, &plan);
    }
    return plan;
}

// Whether a kernel that may record an error was launched, or captured, since the library was loaded.
static std::atomic<bool> g_recorders_launched{false};

cudaError_t linear_launch(const LinearProblem &p, int sm_count, cudaStream_t stream)
{
    if (p.m > kFewRows) {
        const Path path = best_path(p.m, p.n, p.k, sm_count, tc_stream_align(p));
        if (path == kTile) return linear_tile_launch(p, stream);
        g_recorders_launched.store(true, std::memory_order_relaxed);
        switch (path) {
        case kStreamed: return tc_stream_launch(p, false, sm_count, stream);
        case kTurned: return tc_stream_launch(p, true, sm_count, stream);
        default: return tc_linear_launch(p, sm_count, stream);
        }
    }
    LinearArgs a{};
    a.e = linear_epilogue_of(p);
    a.a = static_cast<const int8_t *>(p.a.data);
    a.a_stride = p.a.stride;
    a.w = static_cast<const int8_t *>(p.w.data);
    a.w_stride = p.w.stride;
    a.k = p.k;
    switch (p.out_dtype) {
    case kF32: return linear_few_launch_t<float>(a, stream);
    case kBf16: return linear_few_launch_t<__nv_bfloat16>(a, stream);
    default: return linear_few_launch_t<__half>(a, stream);
    }
}

cudaError_t linear_read_and_clear_error(cudaStream_t stream, unsigned int *out)
{
    // Each word is a copy and a wait, 10 us of a check, which programs without these kernels need not pay.
    *out = 0;
    if (!g_recorders_launched.load(std::memory_order_relaxed)) return cudaSuccess;
    unsigned int a = 0, b = 0;
    cudaError_t e = tc_linear_read_and_clear_error(stream, &a);
    if (e == cudaSuccess) e = tc_stream_read_and_clear_error(stream, &b);
    *out = a | b;
    return e;
}

}  // namespace cbs
