// tc_adapters.cu -- the adapters' weight gradients on the fifth-generation tensor cores (adapters.cu has the formulas).
//
// For bf16 activations in 16-byte aligned rows and adapters of many rows: sums over rows of outer products, as products
// with K over the rows.  A CTA takes 128 columns of x (for dA) or dy (for dB) and a chunk of the rows in the order by
// adapter, 64 at a time.  The rows come by gathering TMA loads, four rows of 64 columns each, in the swizzled tiles
// that tcgen05.mma reads with its first operand's M along memory; so x and dy pass through no register.  Four warps make
// the second operand: the small fp32 rows in three bf16 parts, side by side along N, which keep fp32's bits; each part
// has its own sums in tensor memory, and the epilogue adds them up.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "adapters.h"
#include "cbs_internal.h"
#include "linear_device.cuh"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

__device__ unsigned int g_adapters_error = 0;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far beyond any legitimate wait
std::atomic<bool> g_launched{false};

constexpr int kTcThreads = 192;   // loads, MMAs, and four warps that finish
constexpr int kTileBytes = 128 * kTcStepRows * 2;  // two boxes of 64 columns

template <int RT>
struct TcSizes {
    static constexpr int kRanks = 16 * RT, kN = 3 * kRanks;
    static constexpr int kOperand = kN * 128;  // bytes a step: 64 rows of K for each rank and part
    static constexpr int kStage = kTileBytes + kOperand;
    static constexpr int kStages = RT == 4 ? 2 : 4;
    // Sums that the steps go to in turn: the tensor core cuts where it adds, so short runs of additions keep more bits
    // (rank 16, 1024 rows in a chunk: dB 8.4e-7 off with one, 4e-7 with four).
    static constexpr int kSets = RT == 1 ? 4 : RT == 2 ? 2 : 1, kTmem = 256;
    static constexpr int kSmem = 1024 + kStages * kStage + kTcChunkSteps * kTcStepRows * 4 + 256;
};

// ------------------------------------------------------------------ the second operand
// A block makes a step's: for each rank and part a row of 64 values of K in 128 bytes, swizzled as tcgen05.mma reads it
// from shared memory, where it goes as it is.
template <int RT>
__global__ void __launch_bounds__(128) adapter_operand_kernel(const AdapterGradArgs a)
{
    constexpr int kRanks = 16 * RT;
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int step = blockIdx.x;
    if (step >= a.step_starts[a.adapters]) return;
    const AdapterTile tile = a.steps[step];
    const float *const small = blockIdx.y ? a.dhidden : a.hidden;
    uint4 *const to = a.operands + ((long long)blockIdx.y * a.most_steps + step) * (TcSizes<RT>::kOperand / 16);
#pragma unroll
    for (int q = 0; q < RT; ++q) {
        const int rank = ((int)threadIdx.x + 128 * q) % kRanks, piece = ((int)threadIdx.x + 128 * q) / kRanks;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = 8 * piece + i;
            v[i] = p < tile.count && rank < a.rank ? __ldg(small + (long long)a.order[tile.first + p] * a.rank + rank) : 0.0f;
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
                // What is left; of infinities and NaN nothing, as their difference with themselves is NaN.
                const float top = __int_as_float(0x7f800000);
                v[2 * i] = fabsf(v[2 * i]) < top ? v[2 * i] - __uint_as_float(w[i] << 16) : 0.0f;
                v[2 * i + 1] = fabsf(v[2 * i + 1]) < top ? v[2 * i + 1] - __uint_as_float(w[i] & 0xffff0000u) : 0.0f;
            }
            const int n = part * kRanks + rank;
            to[n * 8 + (piece ^ (n & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------------------------ the products
__device__ __forceinline__ void give_up(unsigned int bit, volatile int *abort_flag)
{
    atomicOr(&g_adapters_error, bit);
    *abort_flag = 1;
}

// Four rows of the map's box width, from column c on, one after another in shared memory; rows beyond the map are zeros.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *tm, uint32_t bar, int c, int r0, int r1, int r2, int r3)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(c), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
        : "memory");
}

// x and dy: a row of 64 columns a box, which four-row gathers take, and 64 rows.
struct TcMaps {
    CUtensorMap row[2], rows[2];
};

// The adapter of step `at`, from `adapter` on: the first whose steps end behind it.  By a whole warp.
__device__ __forceinline__ int adapter_at(const AdapterGradArgs &a, int adapter, int at)
{
    const int lane = threadIdx.x % 32;
    for (;; adapter += 32) {
        const unsigned behind = __ballot_sync(0xffffffffu, adapter + lane >= a.adapters || a.step_starts[adapter + lane + 1] > at);
        if (behind) return adapter + __ffs((int)behind) - 1;
    }
}

template <int RT>
__global__ void __launch_bounds__(kTcThreads)
    adapter_tc_weights_kernel(const __grid_constant__ TcMaps maps, const AdapterGradArgs a)
{
    using S = TcSizes<RT>;
    constexpr int kStages = S::kStages, kRanks = S::kRanks;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    int *const rows = reinterpret_cast<int *>(smem + kStages * S::kStage);
    uint64_t *const loaded = reinterpret_cast<uint64_t *>(rows + kTcChunkSteps * kTcStepRows);  // [kStages] each
    uint64_t *const empty = loaded + kStages, *const finished = empty + kStages, *const taken = finished + 1,
             *const drain = taken + 1;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            dev::mbar_init(dev::smem_u32(loaded + i), 1);
            dev::mbar_init(dev::smem_u32(empty + i), 1);
        }
        dev::mbar_init(dev::smem_u32(finished), 1);
        dev::mbar_init(dev::smem_u32(taken), 4);
        dev::mbar_init(dev::smem_u32(drain), 1);
        *abort_flag = 0;
        dev::fence_mbarrier_init();
    }
    if (warp == 1) {
        dev::tmem_alloc(dev::smem_u32(tmem_slot), S::kTmem);
        dev::tmem_relinquish_alloc_permit();
    }
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int x_strips = (a.k + 127) / 128;
    const bool of_x = (int)blockIdx.x < x_strips;
    const int column0 = ((int)blockIdx.x - (of_x ? 0 : x_strips)) * 128, width = of_x ? a.k : a.n;
    const int chunk_from = (int)blockIdx.y * a.chunk_rows, all = a.step_starts[a.adapters];
    const int stop = chunk_from + a.chunk_rows < all ? chunk_from + a.chunk_rows : all;
    for (int i = threadIdx.x; i < (stop - chunk_from) * kTcStepRows; i += kTcThreads) {
        const AdapterTile tile = a.steps[chunk_from + i / kTcStepRows];
        rows[i] = i % kTcStepRows < tile.count ? a.order[tile.first + i % kTcStepRows] : a.rows;  // one beyond the last: zeros
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    dev::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot, stages = dev::smem_u32(smem);

    if (warp == 0) {
        // ---------------------------------------------------------- loads: a lane four rows of half the columns
        const CUtensorMap *const row_map = &maps.row[of_x ? 0 : 1], *const rows_map = &maps.rows[of_x ? 0 : 1];
        const uint4 *const operands = a.operands + (of_x ? (long long)a.most_steps * (S::kOperand / 16) : 0);
        const int box = lane / 16, group = lane % 16;
        int issued = 0;
        for (int step = chunk_from; step < stop; ++step, ++issued) {
            const int s = issued % kStages;
            if (!__all_sync(0xffffffffu, wait_bounded(dev::smem_u32(empty + s), ((uint32_t)(issued / kStages) & 1u) ^ 1u, abort_flag, kWaitNs))) {
                if (lane == 0 && !*abort_flag) give_up(kErrTimeoutProducer, abort_flag);
                break;
            }
            const uint32_t to = stages + s * S::kStage, bar = dev::smem_u32(loaded + s);
            if (lane == 0) {
                dev::mbar_arrive_expect_tx(bar, S::kStage);
                dev::bulk_load(to + kTileBytes, operands + (long long)step * (S::kOperand / 16), S::kOperand, bar);
            }
            __syncwarp();
            const int *const r = rows + (step - chunk_from) * kTcStepRows + 4 * group;
            const int r0 = r[0], r1 = r[1], r2 = r[2], r3 = r[3], top = rows[(step - chunk_from) * kTcStepRows];
            // Rows of one request mostly lie one after another: then two loads do, where gathers, at some 25 ns each on an
            // SM, set the pace (8192x4096x4096 of rank 16 49 us).
            if (__all_sync(0xffffffffu, r0 == top + 4 * group && r1 == r0 + 1 && r2 == r0 + 2 && r3 == r0 + 3 && r3 < a.rows)) {
                if (lane < 2) dev::tma_load_2d(to + lane * (kTileBytes / 2), rows_map, bar, (column0 + 64 * lane) / 2, top);
            } else {
                tma_gather4(to + box * (kTileBytes / 2) + group * 512, row_map, bar, (column0 + 64 * box) / 2, r0, r1, r2, r3);
            }
        }
        // Every load has to land before the CTA may leave.
        for (int i = issued < kStages ? 0 : issued - kStages; i < issued; ++i)
            if (!dev::mbar_wait_bounded(dev::smem_u32(loaded + i % kStages), (uint32_t)(i / kStages) & 1u, nullptr, kWaitNs)) {
                give_up(kErrTimeoutDrain, abort_flag);
                break;
            }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs
        const bool issuer = elect_one();
        // M along memory for the first operand (bit 15): 64 columns to a row of 128 bytes, 8 rows to a swizzle atom; the
        // next 8 rows behind it (stride), the next 64 columns a box further (leading).
        constexpr uint32_t idesc = dev::idesc_bf16_f32(128, S::kN) | (1u << 15);
        const uint64_t desc_a = (dev::smem_desc_kmajor(stages, 128) & ~((uint64_t)0x3fff << 16)) | ((uint64_t)(kTileBytes / 2 >> 4) << 16);
        const uint64_t desc_b = dev::smem_desc_kmajor(stages + kTileBytes, 128);
        bool ok = true;
        int run = 0, adapter = 0, done = 0;
        for (int at = chunk_from; at < stop && ok; ++run) {
            adapter = adapter_at(a, adapter, at);
            const int last = a.step_starts[adapter + 1], end = last < stop ? last : stop;
            ok = __all_sync(0xffffffffu, wait_bounded(dev::smem_u32(taken), ((uint32_t)run & 1u) ^ 1u, abort_flag, kWaitNs));
            dev::tc_fence_after_sync();
            for (int step = at; step < end && ok; ++step, ++done) {
                const int s = done % kStages;
                ok = __all_sync(0xffffffffu, wait_bounded(dev::smem_u32(loaded + s), (uint32_t)(done / kStages) & 1u, abort_flag, kWaitNs));
                if (!ok) break;
                dev::tc_fence_after_sync();
                if (issuer) {
                    const uint64_t da = desc_a + (uint64_t)(s * (S::kStage >> 4)), db = desc_b + (uint64_t)(s * (S::kStage >> 4));
                    const uint32_t d = tmem + (uint32_t)((step - at) % S::kSets * S::kN);
#pragma unroll
                    for (int kk = 0; kk < kTcStepRows / 16; ++kk)  // 16 rows: two atoms on, and 32 bytes along K
                        dev::tc_mma_bf16(d, da + (uint64_t)(128 * kk), db + (uint64_t)(2 * kk), idesc, step >= at + S::kSets || kk > 0 ? 1u : 0u);
                    dev::tc_commit(dev::smem_u32(empty + s));
                    if (step + 1 == end) dev::tc_commit(dev::smem_u32(finished));
                }
                __syncwarp();
            }
            if (!ok && lane == 0 && !*abort_flag) give_up(kErrTimeoutMma, abort_flag);
            at = end;
        }
        // Every MMA must have finished before tensor memory is freed.
        if (issuer) {
            dev::tc_commit(dev::smem_u32(drain));
            if (!dev::mbar_wait_bounded(dev::smem_u32(drain), 0, nullptr, kWaitNs)) give_up(kErrTimeoutDrain, abort_flag);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- the sums
        const int quarter = warp & 3;
        int run = 0, adapter = 0;
        for (int at = chunk_from; at < stop; ++run) {
            adapter = adapter_at(a, adapter, at);
            const int first = a.step_starts[adapter], last = a.step_starts[adapter + 1], end = last < stop ? last : stop;
            if (!__all_sync(0xffffffffu, wait_bounded(dev::smem_u32(finished), (uint32_t)run & 1u, abort_flag, kWaitNs))) {
                if (lane == 0 && !*abort_flag) give_up(kErrTimeoutEpilogue, abort_flag);
                break;
            }
            dev::tc_fence_after_sync();
            float sum[kRanks];
#pragma unroll
            for (int r = 0; r < kRanks; ++r) sum[r] = 0.0f;
            const int sets = end - at < S::kSets ? end - at : S::kSets;
#pragma unroll
            for (int part = 2; part >= 0; --part)
                for (int set = 0; set < sets; ++set)
#pragma unroll
                    for (int c = 0; c < kRanks; c += 16) {
                        uint32_t u[16];
                        dev::tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * quarter) << 16) + set * S::kN + part * kRanks + c, u);
                        dev::tmem_ld_wait();
                        dev::reg_fence16(u);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(u[i]);
                    }
            dev::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(dev::smem_u32(taken));
            const float scale = a.scale ? a.scale[adapter] : 1.0f;
            float *out = of_x ? a.da + (long long)adapter * a.rank * a.k : a.db + (long long)adapter * a.rank * a.n;
            if (first < chunk_from || last > stop) {
                out = a.partial + (2LL * blockIdx.y + (first >= chunk_from)) * a.rank * ((long long)a.k + a.n);
                if (!of_x) out += (long long)a.rank * a.k;
            }
            const int column = column0 + 32 * quarter + lane;
            if (column < width) {
#pragma unroll
                for (int r = 0; r < kRanks; ++r)
                    if (r < a.rank) out[of_x ? (long long)r * a.k + column : (long long)column * a.rank + r] = scale * sum[r];
            }
            at = end;
        }
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        dev::tc_fence_after_sync();
        dev::tmem_dealloc(tmem, S::kTmem);
    }
}

template <int RT>
cudaError_t tc_weights_launch(const AdapterGradArgs &a, const TcMaps &maps, cudaStream_t stream)
{
    static bool allowed[kMaxDevices] = {};
    const cudaError_t e = allow_dynamic_smem(adapter_tc_weights_kernel<RT>, TcSizes<RT>::kSmem, allowed);
    if (e != cudaSuccess) return e;
    const cudaError_t made = launch_overlapped(adapter_operand_kernel<RT>, dim3((unsigned)a.most_steps, 2), dim3(128), 0, stream, 1, a);
    if (made != cudaSuccess) return made;
    const dim3 grid((unsigned)((a.k + 127) / 128 + (a.n + 127) / 128), (unsigned)a.chunks);
    return launch_overlapped(adapter_tc_weights_kernel<RT>, grid, dim3(kTcThreads), TcSizes<RT>::kSmem, stream, 1, maps, a);
}

}  // namespace

cudaError_t adapter_tc_weights_launch(const AdapterGradArgs &a, cudaStream_t stream)
{
    TcMaps maps;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
        const void *data = i ? a.dy : a.x;
        const int width = i ? a.n : a.k;
        const long long stride = i ? a.dy_stride : a.x_stride;
        e = encode_bytes_map(data, a.rows, width * 2, stride * 2, 1, 128, &maps.row[i]);
        if (e == cudaSuccess) e = encode_bytes_map(data, a.rows, width * 2, stride * 2, kTcStepRows, 128, &maps.rows[i]);
    }
    if (e != cudaSuccess) return e;
    g_launched.store(true, std::memory_order_relaxed);
    switch (adapter_rank_tiles(a.rank)) {
    case 1: return tc_weights_launch<1>(a, maps, stream);
    case 2: return tc_weights_launch<2>(a, maps, stream);
    default: return tc_weights_launch<4>(a, maps, stream);
    }
}

cudaError_t adapters_read_and_clear_error(cudaStream_t stream, unsigned int *out)
{
    *out = 0;
    return g_launched.load(std::memory_order_relaxed) ? read_and_clear_word(g_adapters_error, stream, out) : cudaSuccess;
}

}  // namespace cbs
