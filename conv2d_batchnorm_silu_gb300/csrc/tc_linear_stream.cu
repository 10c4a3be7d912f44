// tc_linear_stream.cu -- the int8 linear layer for tens to hundreds of rows, where the weights' bytes
// count: they are read once as int8 and widened to f16 between global and shared memory.
//
// D[channel][row] = W * A^T with 128 channels on the tensor core's M side and NT rows on its N side.
// Eight warps hold the int8 of the coming steps in registers (kAhead steps of 128 K elements, 48 KB of
// weights per SM in flight, whole 128-byte lines of each row), widen a step of weights and rows at a time into swizzled f16 tiles, and hand them
// to the issuing warp.  Every CTA takes an equal run of the (channel tile, row tile, K step) sequence,
// so that all SMs read the same share of the weights; a tile whose K steps fall to several CTAs is
// left as fp32 partial sums in the workspace, which a second kernel adds in K order and finishes.
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

__device__ unsigned int g_stream_error = 0;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far beyond any legitimate wait

constexpr int kChannels = 128;  // of a tile
constexpr int kStep = 128;      // K elements per step: two swizzle spans of f16
constexpr int kWidenWarps = 8;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (kWidenWarps + kEpiWarps + 1);

template <int NT>
struct StreamCfg {
    static constexpr int A_BYTES = kChannels * kStep * 2;
    static constexpr int B_BYTES = NT * kStep * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = NT <= 64 ? 4 : (NT <= 128 ? 3 : 2);
    static constexpr int SMEM = 1024 + STAGES * STAGE + 256;
    static constexpr int ROW_LOADS = NT / 32;  // 16-byte pieces of rows per thread and step
    static constexpr int kAhead = NT <= 128 ? 3 : 2;  // steps held in registers
    static constexpr int TMEM_COLS = 2 * NT;
};

struct StreamArgs {
    LinearEpilogue e;
    const int8_t *a, *w;
    long long a_stride, w_stride;
    int k, k_steps;
    int row_tiles, tiles;      // tile = channel tile * row_tiles + row tile
    long long steps;           // tiles * k_steps
    int workers;               // CTAs that share them
    float *partial;            // [workers + tiles][NT][kChannels]
};

__device__ __forceinline__ void give_up(unsigned int bit, volatile int *abort_flag)
{
    atomicOr(&g_stream_error, bit);
    *abort_flag = 1;
}

// As mbar_wait_bounded; waits here are often a little early, and reading the clock at the first
// unsuccessful poll would cost more than most of them last.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const volatile int *abort_flag,
                                             uint64_t timeout_ns)
{
    for (int i = 0; i < 64; ++i)
        if (dev::mbar_try_wait(bar, parity)) return true;
    return dev::mbar_wait_bounded(bar, parity, abort_flag, timeout_ns);
}

// One predicated load straight into its registers: behind a branch the value would be moved, and the
// warp wait for it, where the branches meet.
__device__ __forceinline__ void load_or_zero(uint4 &v, const int8_t *p, bool exists)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)exists));
}

// First step of worker b's run, and the worker that has step g.
__device__ __forceinline__ long long run_start(const StreamArgs &a, int b) { return a.steps * b / a.workers; }
__device__ __forceinline__ int worker_of(const StreamArgs &a, long long g)
{
    return (int)(((g + 1) * a.workers - 1) / a.steps);
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_stream_kernel(const StreamArgs a)
{
    using C = StreamCfg<NT>;
    constexpr int STAGES = C::STAGES, AHEAD = C::kAhead, LOADS = 4 + C::ROW_LOADS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *sm_a = smem, *sm_b = smem + STAGES * C::A_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * C::STAGE);
    uint64_t *empty = full + STAGES, *tfull = empty + STAGES, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMmaWarp = kWidenWarps + kEpiWarps;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            dev::mbar_init(dev::smem_u32(&full[i]), kWidenWarps);
            dev::mbar_init(dev::smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            dev::mbar_init(dev::smem_u32(&tfull[i]), 1);
            dev::mbar_init(dev::smem_u32(&tempty[i]), kEpiWarps);
        }
        dev::mbar_init(dev::smem_u32(drain), 1);
        *abort_flag = 0;
        dev::fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
        dev::tmem_alloc<1>(dev::smem_u32(tmem_slot), C::TMEM_COLS);
        dev::tmem_relinquish_alloc_permit<1>();
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    dev::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const long long g0 = run_start(a, blockIdx.x), g1 = run_start(a, blockIdx.x + 1);
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();

    if (warp < kWidenWarps) {
        // ---------------------------------------------------------- loads and widening
        // Piece j of this thread: 16 bytes of K from 16 * (tid % 8) of weights rows tid / 8 + 32 j for
        // j < 4, then of rows of a.
        const int tid = threadIdx.x, q = tid & 7, r8 = tid >> 3;
        int tile = (int)(g0 / a.k_steps), ks = (int)(g0 - (long long)tile * a.k_steps);  // of the next load
        const int8_t *w0 = nullptr, *a0 = nullptr;  // of piece 0 of either
        int w_count = 0, a_count = 0;               // pieces whose row exists; the others read as zeros
        auto rows_of_tile = [&]() {
            const int ct = tile / a.row_tiles, rt = tile - ct * a.row_tiles;
            const int n = ct * kChannels + r8;
            const long long m = (long long)rt * NT + r8;
            w0 = a.w + n * a.w_stride;
            a0 = a.a + m * a.a_stride;
            w_count = n < a.e.n ? (a.e.n - n + 31) / 32 : 0;
            a_count = m < a.e.m ? (int)((a.e.m - m + 31) / 32) : 0;
        };
        rows_of_tile();
        uint4 held[AHEAD][LOADS];
        long long loaded = g0;
        auto load = [&](uint4 (&to)[LOADS]) {
            const int k0 = ks * kStep + q * 16;
            const bool any = loaded < g1 && k0 < a.k;  // k is a multiple of 16
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const bool exists = any && (j < 4 ? j < w_count : j - 4 < a_count);
                const int8_t *src = j < 4 ? w0 + j * 32 * a.w_stride : a0 + (j - 4) * 32 * a.a_stride;
                load_or_zero(to[j], src + k0, exists);
            }
            ++loaded;
            if (++ks == a.k_steps && loaded < g1) {
                ks = 0;
                ++tile;
                rows_of_tile();
            }
        };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) load(held[d]);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (long long g = g0; g < g1 && ok; g += AHEAD) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                if (g + d >= g1 || !ok) break;
                ok = __all_sync(0xffffffffu, wait_bounded(dev::smem_u32(&empty[stage]), phase ^ 1u,
                                                                    abort_flag, kWaitNs));
                if (!ok) {
                    if (lane == 0 && !*abort_flag) give_up(kErrTimeoutProducer, abort_flag);
                    break;
                }
                const uint32_t ta = dev::smem_u32(sm_a + stage * C::A_BYTES);
                const uint32_t tb = dev::smem_u32(sm_b + stage * C::B_BYTES);
                // Bytes 16 q .. 16 q + 15 become the f16 pieces 2 q and 2 q + 1 of the row's 256 bytes, in the
                // first span (q < 4) or the second; the two spans take them in the other order, so that eight
                // lanes of a row meet eight different banks.
                const uint32_t swap = (uint32_t)q >> 2, piece = ((uint32_t)q & 3u) * 2, turn = (uint32_t)r8 & 7u;
                const uint32_t o0 = ((piece + swap) ^ turn) << 4, o1 = ((piece + (swap ^ 1u)) ^ turn) << 4;
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const uint32_t row = (uint32_t)((j < 4 ? j : j - 4) * 32 + r8);
                    const uint4 v = held[d][j];
                    const uint2 p0 = widen4(v.x), p1 = widen4(v.y), p2 = widen4(v.z), p3 = widen4(v.w);
                    const uint4 lo = make_uint4(p0.x, p0.y, p1.x, p1.y), hi = make_uint4(p2.x, p2.y, p3.x, p3.y);
                    const uint4 first = swap ? hi : lo, second = swap ? lo : hi;
                    const uint32_t at = (j < 4 ? ta + swap * (C::A_BYTES / 2) : tb + swap * (C::B_BYTES / 2)) + row * 128;
                    dev::sts_v4(at + o0, first.x, first.y, first.z, first.w);
                    dev::sts_v4(at + o1, second.x, second.y, second.z, second.w);
                }
                dev::fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(dev::smem_u32(&full[stage]));
                load(held[d]);
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMAs
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16(kChannels, NT);
            const uint64_t desc_a = dev::smem_desc_kmajor(dev::smem_u32(sm_a), 128);
            const uint64_t desc_b = dev::smem_desc_kmajor(dev::smem_u32(sm_b), 128);
            int stage = 0, piece = 0;
            uint32_t phase = 0;
            bool ok = true;
            int ks = (int)(g0 % a.k_steps);
            bool start = true;
            for (long long g = g0; g < g1; ++g) {
                const int buf = piece & 1;
                if (start) {
                    if (!wait_bounded(dev::smem_u32(&tempty[buf]), ((uint32_t)(piece >> 1) & 1u) ^ 1u,
                                                abort_flag, kWaitNs)) {
                        if (!*abort_flag) give_up(kErrTimeoutMma, abort_flag);
                        break;
                    }
                }
                ok = wait_bounded(dev::smem_u32(&full[stage]), phase, abort_flag, kWaitNs);
                if (!ok) {
                    if (!*abort_flag) give_up(kErrTimeoutMma, abort_flag);
                    break;
                }
                dev::tc_fence_after_sync();
                const uint64_t da = desc_a + (uint64_t)(stage * (C::A_BYTES >> 4));
                const uint64_t db = desc_b + (uint64_t)(stage * (C::B_BYTES >> 4));
                const uint32_t d = tmem + (uint32_t)(buf * NT);
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk) {
                    const uint64_t span = (uint64_t)(kk / 4), in = (uint64_t)(2 * (kk % 4));
                    dev::tc_mma_bf16<1>(d, da + span * (C::A_BYTES / 2 >> 4) + in, db + span * (C::B_BYTES / 2 >> 4) + in,
                                        idesc, !start || kk > 0 ? 1u : 0u);
                }
                dev::tc_commit<1>(dev::smem_u32(&empty[stage]));
                if (++stage == STAGES) stage = 0, phase ^= 1u;
                start = false;
                if (++ks == a.k_steps || g + 1 == g1) {
                    dev::tc_commit<1>(dev::smem_u32(&tfull[buf]));
                    ks = 0;
                    ++piece;
                    start = true;
                }
            }
            // Every MMA must have finished before tensor memory is freed.
            dev::tc_commit<1>(dev::smem_u32(drain));
            if (!wait_bounded(dev::smem_u32(drain), 0, nullptr, kWaitNs)) give_up(kErrTimeoutDrain, abort_flag);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- epilogue: lane = channel, column = row of a
        const int quarter = warp & 3;
        int piece = 0;
        for (long long g = g0; g < g1; ++piece) {
            const int tile = (int)(g / a.k_steps), ks = (int)(g - (long long)tile * a.k_steps);
            const long long end = g + (a.k_steps - ks) < g1 ? g + (a.k_steps - ks) : g1;
            const bool whole = ks == 0 && end - g == a.k_steps;
            const int ct = tile / a.row_tiles, rt = tile - ct * a.row_tiles;
            const int buf = piece & 1;
            int ok = 1;
            if (lane == 0)
                ok = wait_bounded(dev::smem_u32(&tfull[buf]), (uint32_t)(piece >> 1) & 1u, abort_flag, kWaitNs);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                if (lane == 0 && !*abort_flag) give_up(kErrTimeoutEpilogue, abort_flag);
                break;
            }
            dev::tc_fence_after_sync();
            const uint32_t taddr = tmem + (uint32_t)(buf * NT) + ((uint32_t)(quarter * 32) << 16);
            const long long m0 = (long long)rt * NT;
            const int n = ct * kChannels + quarter * 32 + lane;
            float *out = a.partial + ((long long)(blockIdx.x + tile) * NT) * kChannels + quarter * 32 + lane;
            for (int c = 0; c < NT && m0 + c < a.e.m; c += 16) {
                uint32_t v[16];
                dev::tmem_ld_32x32b_x16(taddr + (uint32_t)c, v);
                dev::tmem_ld_wait();
                dev::reg_fence16(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (m0 + c + i >= a.e.m) continue;
                    if (!whole)
                        out[(c + i) * kChannels] = __uint_as_float(v[i]);
                    else if (n < a.e.n)
                        finish_one<T>(a.e, __uint_as_float(v[i]), m0 + c + i, n);
                }
            }
            dev::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(dev::smem_u32(&tempty[buf]));
            g = end;
        }
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        dev::tc_fence_after_sync();
        dev::tmem_dealloc<1>(tmem, C::TMEM_COLS);
    }
}

// Tiles whose K steps several workers share: their partial sums added in K order, and finished.  A
// thread takes four channels of a row; eight workers' sums load at a time.
constexpr int kJoinRows = 4;
template <typename T, int NT>
__global__ void __launch_bounds__(32 * kJoinRows) linear_join_kernel(const StreamArgs a)
{
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int tile = blockIdx.x;
    const long long g = (long long)tile * a.k_steps;
    const int b0 = worker_of(a, g), b1 = worker_of(a, g + a.k_steps - 1);
    if (b0 == b1) return;  // finished by the worker itself
    const int ct = tile / a.row_tiles, rt = tile - ct * a.row_tiles;
    const int i = blockIdx.y * kJoinRows + threadIdx.y, c = threadIdx.x * 4;
    const long long m = (long long)rt * NT + i;
    if (i >= NT || m >= a.e.m) return;
    const float *from = a.partial + ((long long)(b0 + tile) * NT + i) * kChannels + c;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b = b0; b <= b1; b += 8) {
        float4 v[8];
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (b + t <= b1) v[t] = *reinterpret_cast<const float4 *>(from + (long long)(b - b0 + t) * NT * kChannels);
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (b + t <= b1) s.x += v[t].x, s.y += v[t].y, s.z += v[t].z, s.w += v[t].w;
    }
    const float sum[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (ct * kChannels + c + j < a.e.n) finish_one<T>(a.e, sum[j], m, ct * kChannels + c + j);
}

// Row tile and CTAs for m rows: the smallest tile that holds them, all SMs, and no CTA with fewer than
// two steps or less than a sixteenth of a tile (a join of many short runs costs more than it saves).
int row_tile_of(long long m) { return m <= 32 ? 32 : (m <= 64 ? 64 : (m <= 128 ? 128 : 256)); }

struct StreamPlan {
    int nt, k_steps, row_tiles, tiles, workers;
    long long steps;
};

StreamPlan plan_of(long long m, int n, int k, int sm_count)
{
    StreamPlan p{};
    p.nt = row_tile_of(m);
    p.k_steps = k > 0 ? (k + kStep - 1) / kStep : 1;
    p.row_tiles = (int)((m + p.nt - 1) / p.nt);
    p.tiles = (n + kChannels - 1) / kChannels * p.row_tiles;
    p.steps = (long long)p.tiles * p.k_steps;
    const int fewest = p.k_steps > 32 ? (p.k_steps + 15) / 16 : 2;
    const long long most = p.steps / fewest > 0 ? p.steps / fewest : 1;
    p.workers = (int)(most < sm_count ? most : sm_count);
    return p;
}

template <typename T, int NT>
cudaError_t stream_launch(const StreamArgs &a, cudaStream_t stream)
{
    using C = StreamCfg<NT>;
    static bool allowed[kMaxDevices] = {};
    cudaError_t e = allow_dynamic_smem(linear_stream_kernel<T, NT>, C::SMEM, allowed);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(linear_stream_kernel<T, NT>, dim3((unsigned)a.workers), dim3(kThreads), (size_t)C::SMEM, stream,
                          1, a);
    // Equal runs that are whole tiles leave nothing to join.
    if (e != cudaSuccess || (a.steps % a.workers == 0 && a.steps / a.workers % a.k_steps == 0)) return e;
    const int rows = (int)(a.e.m < NT ? a.e.m : NT);
    return launch_overlapped(linear_join_kernel<T, NT>, dim3((unsigned)a.tiles, (unsigned)((rows + kJoinRows - 1) / kJoinRows)),
                             dim3(32, kJoinRows), 0, stream, 1, a);
}

template <typename T>
cudaError_t stream_launch_t(const StreamArgs &a, int nt, cudaStream_t stream)
{
    switch (nt) {
    case 32: return stream_launch<T, 32>(a, stream);
    case 64: return stream_launch<T, 64>(a, stream);
    case 128: return stream_launch<T, 128>(a, stream);
    default: return stream_launch<T, 256>(a, stream);
    }
}

}  // namespace

bool tc_stream_supported(const LinearProblem &p)
{
    auto rows16 = [](const Rows &r) { return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.stride % 16 == 0; };
    return p.k > 0 && p.k % 16 == 0 && rows16(p.a) && rows16(p.w);
}

long long tc_stream_workspace_bytes(long long m, int n, int k, int sm_count)
{
    const StreamPlan p = plan_of(m, n, k, sm_count);
    return ((long long)p.workers + p.tiles) * p.nt * kChannels * 4;
}

cudaError_t tc_stream_launch(const LinearProblem &p, int sm_count, cudaStream_t stream)
{
    const StreamPlan plan = plan_of(p.m, p.n, p.k, sm_count);
    StreamArgs a{};
    a.e = linear_epilogue_of(p);
    a.a = static_cast<const int8_t *>(p.a.data);
    a.a_stride = p.a.stride;
    a.w = static_cast<const int8_t *>(p.w.data);
    a.w_stride = p.w.stride;
    a.k = p.k;
    a.k_steps = plan.k_steps;
    a.row_tiles = plan.row_tiles;
    a.tiles = plan.tiles;
    a.steps = plan.steps;
    a.workers = plan.workers;
    a.partial = static_cast<float *>(p.workspace);
    switch (p.out_dtype) {
    case kF32: return stream_launch_t<float>(a, plan.nt, stream);
    case kBf16: return stream_launch_t<__nv_bfloat16>(a, plan.nt, stream);
    default: return stream_launch_t<__half>(a, plan.nt, stream);
    }
}

cudaError_t tc_stream_read_and_clear_error(cudaStream_t stream, unsigned int *out)
{
    return read_and_clear_word(g_stream_error, stream, out);
}

}  // namespace cbs
