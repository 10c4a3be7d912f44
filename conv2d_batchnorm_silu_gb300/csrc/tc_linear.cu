// tc_linear.cu -- the int8 linear layer on the fifth-generation tensor cores.
//
// This part's tensor cores are fast at 16-bit floats (2.25 PFLOP/s nominal) and slow at 8-bit
// integers.  An int8 is exact in f16, the product of two (up to 2^14) and sums up to 2^24 are
// exact in the fp32 accumulator, so the product runs as an f16 one: a first kernel widens the
// rows and weights to f16 in the workspace (K padded with zeros to whole steps, so every size,
// stride and alignment of the inputs reaches the second kernel as aligned tiles), and a
// persistent GEMM multiplies them with the scales, bias, activation and residual in its epilogue.
//
// Measured, both kernels: 8192x16384x4096 623 us (1,760 TOP/s; the tensor cores' rate, and 58 us of widening),
// 4096x4096x4096 96 us, 25600x1024x256 24 us, where the epilogue sets the pace (a 256 x 256
// tile's takes 3,600 of 5,000 clocks, its MMAs 2,048).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "cbs_internal.h"
#include "linear_device.cuh"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

__device__ unsigned int g_linear_error = 0;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far beyond any legitimate wait

// ------------------------------------------------------------------ widening to f16
struct WidenMatrix {
    const int8_t *src;
    __half *dst;
    long long stride;
    int aligned;  // 16-byte aligned rows: whole pieces load at once
};
struct WidenArgs {
    WidenMatrix a, w;
    long long m, rows;  // rows of a, of both
    int k, kp;
    int lanes_log2;     // threads of a block that share a row
};

__global__ void __launch_bounds__(256) widen_kernel(const WidenArgs args)
{
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int per_block = 256 >> args.lanes_log2, lanes = 1 << args.lanes_log2;
    const long long step = (long long)gridDim.x * per_block;
    for (long long r = (long long)blockIdx.x * per_block + (threadIdx.x >> args.lanes_log2); r < args.rows; r += step) {
        const bool first = r < args.m;
        const long long row = first ? r : r - args.m;
        const int8_t *src = first ? args.a.src + row * args.a.stride : args.w.src + row * args.w.stride;
        __half *dst = (first ? args.a.dst : args.w.dst) + row * args.kp;
        const int aligned = first ? args.a.aligned : args.w.aligned;
        for (int k0 = (threadIdx.x & (lanes - 1)) * 16; k0 < args.kp; k0 += lanes * 16) {
            uint4 v;
            if (aligned) {
                v = load_or_zero(src + k0, k0 < args.k);
            } else {
                v = shifted(load_raw(src, k0, args.k), src, k0);
            }
            if (k0 + 16 > args.k) v = within(v, k0, args.k);
            const uint2 p0 = widen4(v.x), p1 = widen4(v.y), p2 = widen4(v.z), p3 = widen4(v.w);
            uint4 *out = reinterpret_cast<uint4 *>(dst + k0);
            out[0] = make_uint4(p0.x, p0.y, p1.x, p1.y);
            out[1] = make_uint4(p2.x, p2.y, p3.x, p3.y);
        }
    }
}

// ------------------------------------------------------------------ GEMM
constexpr int kBlockK = 64;  // f16 elements per step: one 128-byte swizzle span
constexpr int kBlockM = 128; // rows per CTA
constexpr int kEpiPerQuarter = 3;  // epilogue warps per TMEM lane quarter; they take its 32-column blocks in turn
constexpr int kEpiWarps = 4 * kEpiPerQuarter;
constexpr int kThreads = 128 + 32 * kEpiWarps;

// BN output channels per tile.  PAIR: two CTAs of a cluster work as one on 256 rows, each
// holding its 128 rows and half of the weight tile.
// SIZE: bytes of an output element.
template <int BN, bool PAIR, int SIZE>
struct GemmCfg {
    static constexpr int B_ROWS = PAIR ? BN / 2 : BN;
    static constexpr int A_BYTES = kBlockM * kBlockK * 2;
    static constexpr int B_BYTES = B_ROWS * kBlockK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STG_BLOCK = 32 * 32 * SIZE;              // an epilogue warp's block on its way out
    static constexpr int BLOCKS = BN / 32, MOST = (BLOCKS + kEpiPerQuarter - 1) / kEpiPerQuarter;  // per warp
    static constexpr int STG_WARP = STG_BLOCK + MOST * 256;  // and the scales and biases of its columns
    static constexpr int STG = kEpiWarps * STG_WARP;
    static constexpr int FIT = (232448 - 1024 - 512 - STG) / STAGE;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int SMEM = 1024 + STAGES * STAGE + STG + 512;
    static constexpr int TMEM_COLS = 2 * BN;
    static_assert(STAGES >= 4, "pipeline depth");
};

struct GemmArgs {
    LinearEpilogue e;
    int k_iters;
    int m_tiles, n_tiles;  // of (PAIR ? 256 : 128) rows x BN channels
    int tiles;
};

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *tm, uint32_t bar_cluster, int c0,
                                                 int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar_cluster), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void give_up(unsigned int bit, volatile int *abort_flag)
{
    atomicOr(&g_linear_error, bit);
    *abort_flag = 1;
}

// Arrival on a barrier of the pair, which only orders the tensor memory reads fenced before it: without
// cluster scope, which would wait for the warp's earlier stores to global memory.
__device__ __forceinline__ void arrive_remote(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// Tile t in bands of eight row tiles, channel tiles within a band, row tiles fastest: the tiles in
// flight at one time share both operands in L2.
__device__ __forceinline__ void tile_at(const GemmArgs &a, int t, int &mt, int &nt)
{
    const int band = t / (8 * a.n_tiles), within = t - band * 8 * a.n_tiles;
    const int high = a.m_tiles - band * 8;
    nt = high >= 8 ? within >> 3 : within / high;
    mt = band * 8 + within - nt * (high < 8 ? high : 8);
}

template <typename T, int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                       const GemmArgs a)
{
    using C = GemmCfg<BN, PAIR, sizeof(T)>;
    constexpr int CG = PAIR ? 2 : 1, STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *sm_a = smem, *sm_b = smem + STAGES * C::A_BYTES, *sm_stg = smem + STAGES * C::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm_stg + C::STG);
    uint64_t *empty = full + STAGES, *tfull = empty + STAGES, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)dev::cluster_ctarank() : 0;
    const int vb = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x, vg = PAIR ? (int)gridDim.x >> 1 : (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            dev::mbar_init(dev::smem_u32(&full[i]), 2);  // the two loading warps
            dev::mbar_init(dev::smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            dev::mbar_init(dev::smem_u32(&tfull[i]), 1);
            dev::mbar_init(dev::smem_u32(&tempty[i]), CG * kEpiWarps);
        }
        dev::mbar_init(dev::smem_u32(drain), 1);
        *abort_flag = 0;
        dev::fence_mbarrier_init();
    }
    if (threadIdx.x == 32) {
        dev::prefetch_tensormap(&tm_a);
        dev::prefetch_tensormap(&tm_w);
    }
    if (warp == 1) {
        dev::tmem_alloc<CG>(dev::smem_u32(tmem_slot), C::TMEM_COLS);
        dev::tmem_relinquish_alloc_permit<CG>();
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) dev::cluster_sync();
    dev::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t full0 = PAIR ? dev::mapa_cluster(dev::smem_u32(full), 0) : 0u;
    const uint32_t tempty0 = PAIR ? dev::mapa_cluster(dev::smem_u32(tempty), 0) : 0u;
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();

    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------- loads: warp 0 rows, warp 2 weights
        const bool weights = warp == 2;
        const CUtensorMap *tm = weights ? &tm_w : &tm_a;
        const uint32_t dst0 = dev::smem_u32(weights ? sm_b : sm_a);
        const uint32_t bytes = weights ? C::B_BYTES : C::A_BYTES;
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = true;
            for (int t = vb; t < a.tiles && ok && !*abort_flag; t += vg) {
                int mt, nt;
                tile_at(a, t, mt, nt);
                const int row = weights ? nt * BN + rank * C::B_ROWS : (mt * CG + rank) * kBlockM;
                for (int it = 0; it < a.k_iters; ++it) {
                    if (!wait_bounded(dev::smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitNs)) {
                        if (!*abort_flag) give_up(kErrTimeoutProducer, abort_flag);
                        ok = false;
                        break;
                    }
                    const uint32_t dst = dst0 + (uint32_t)stage * bytes;
                    if constexpr (PAIR) {
                        // Both CTAs' bytes complete on the even CTA's barrier.
                        if (rank == 0) dev::mbar_arrive_expect_tx(dev::smem_u32(&full[stage]), 2 * bytes);
                        tma_load_2d_pair(dst, tm, full0 + (uint32_t)(stage * 8), it * kBlockK, row);
                    } else {
                        dev::mbar_arrive_expect_tx(dev::smem_u32(&full[stage]), bytes);
                        dev::tma_load_2d(dst, tm, dev::smem_u32(&full[stage]), it * kBlockK, row);
                    }
                    issued |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
            }
            // Every load must have landed before the CTA may leave; the odd CTA sees that by the
            // release of the stage by the MMAs that read it.
            for (int i = 0; i < STAGES; ++i)
                if ((issued >> i) & 1u) {
                    const uint32_t bar = dev::smem_u32(PAIR && rank != 0 ? &empty[i] : &full[i]);
                    if (!dev::mbar_wait_bounded(bar, (issued_parity >> i) & 1u, nullptr, kWaitNs)) {
                        give_up(kErrTimeoutDrain, abort_flag);
                        break;
                    }
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs
        // The whole warp runs the loop and one elected lane issues: with the control flow uniform, descriptors
        // are computed and held in uniform registers, which an MMA takes as they are.
        if (rank == 0) {
            const bool issuer = elect_one();
            constexpr uint32_t idesc = idesc_f16(CG * kBlockM, BN);
            const uint64_t desc_a = dev::smem_desc_kmajor(dev::smem_u32(sm_a), 128);
            const uint64_t desc_b = dev::smem_desc_kmajor(dev::smem_u32(sm_b), 128);
            int stage = 0, lt = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = vb; t < a.tiles && ok; t += vg, ++lt) {
                const int buf = lt & 1;
                ok = __all_sync(0xffffffffu, wait_bounded(dev::smem_u32(&tempty[buf]), ((uint32_t)(lt >> 1) & 1u) ^ 1u,
                                                          abort_flag, kWaitNs));
                dev::tc_fence_after_sync();
                const uint32_t d = tmem + (uint32_t)(buf * BN);
                for (int it = 0; it < a.k_iters && ok; ++it) {
                    ok = __all_sync(0xffffffffu, wait_bounded(dev::smem_u32(&full[stage]), phase, abort_flag, kWaitNs));
                    if (!ok) break;
                    dev::tc_fence_after_sync();
                    const uint64_t da = desc_a + (uint64_t)(stage * (C::A_BYTES >> 4));
                    const uint64_t db = desc_b + (uint64_t)(stage * (C::B_BYTES >> 4));
                    if (issuer) {
#pragma unroll
                        for (int kk = 0; kk < kBlockK / 16; ++kk)
                            dev::tc_mma_bf16<CG>(d, da + (uint64_t)(2 * kk), db + (uint64_t)(2 * kk), idesc,
                                                 it > 0 || kk > 0 ? 1u : 0u);
                        if constexpr (PAIR)
                            dev::tc_commit_multicast<CG>(dev::smem_u32(&empty[stage]), (uint16_t)0x3);
                        else
                            dev::tc_commit<CG>(dev::smem_u32(&empty[stage]));
                        if (it + 1 == a.k_iters) {
                            if constexpr (PAIR)
                                dev::tc_commit_multicast<CG>(dev::smem_u32(&tfull[buf]), (uint16_t)0x3);
                            else
                                dev::tc_commit<CG>(dev::smem_u32(&tfull[buf]));
                        }
                    }
                    __syncwarp();
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
                if (!ok && issuer && !*abort_flag) give_up(kErrTimeoutMma, abort_flag);
            }
            // Every MMA must have finished before tensor memory is freed.
            if (issuer) {
                dev::tc_commit<CG>(dev::smem_u32(drain));
                if (!dev::mbar_wait_bounded(dev::smem_u32(drain), 0, nullptr, kWaitNs))
                    give_up(kErrTimeoutDrain, abort_flag);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------- epilogue
        const int quarter = warp & 3, turn = (warp - 4) >> 2;
        const uint32_t stg = dev::smem_u32(sm_stg + (warp - 4) * C::STG_WARP), params = stg + C::STG_BLOCK;
        int lt = 0;
        // A tile's place, scales and biases are found while the tile before it is finished (25600x1024x256
        // 24.0 us, with SiLU 29.4; at the tile's own start 24.8 and 30.9).
        int next_mt = 0, next_nt = 0;
        float next_scale[C::MOST], next_bias[C::MOST], next_row[4];
        auto look_ahead = [&](int t) {
            if (t >= a.tiles) return;
            tile_at(a, t, next_mt, next_nt);
#pragma unroll
            for (int i = 0; i < C::MOST; ++i) {
                const int c = next_nt * BN + (turn + i * kEpiPerQuarter) * 32 + lane;
                const bool in = turn + i * kEpiPerQuarter < C::BLOCKS && c < a.e.n;
                next_scale[i] = in ? __ldg(a.e.w_scale + c) : 0.0f;
                next_bias[i] = in && a.e.bias ? __ldg(a.e.bias + c) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (next_mt * CG + rank) * kBlockM + quarter * 32 + 8 * i + (lane >> 2);
                next_row[i] = row < a.e.m ? __ldg(a.e.a_scale + row) : 0.0f;
            }
        };
        look_ahead(vb);
        for (int t = vb; t < a.tiles; t += vg, ++lt) {
            const int mt = next_mt, nt = next_nt;
            const int buf = lt & 1;
            const long long row0 = (long long)(mt * CG + rank) * kBlockM + quarter * 32;
            float row_scale[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) row_scale[i] = next_row[i];
#pragma unroll
            for (int i = 0; i < C::MOST; ++i) {
                dev::sts_u32(params + 256 * i + 4 * lane, __float_as_uint(next_scale[i]));
                dev::sts_u32(params + 256 * i + 128 + 4 * lane, __float_as_uint(next_bias[i]));
            }
            __syncwarp();
            look_ahead(t + vg);
            int ok = 1;
            if (lane == 0)
                ok = wait_bounded(dev::smem_u32(&tfull[buf]), (uint32_t)(lt >> 1) & 1u, abort_flag, kWaitNs);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                if (lane == 0 && !*abort_flag) give_up(kErrTimeoutEpilogue, abort_flag);
                break;
            }
            dev::tc_fence_after_sync();
            auto hand_back = [&]() {
                dev::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        arrive_remote(tempty0 + (uint32_t)(buf * 8));
                    else
                        dev::mbar_arrive(dev::smem_u32(&tempty[buf]));
                }
            };
            if (turn >= C::BLOCKS) hand_back();  // a warp without a block
            const uint32_t taddr = tmem + (uint32_t)(buf * BN) + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
            for (int j = turn, i = 0; j < C::BLOCKS; j += kEpiPerQuarter, ++i) {
                const int cj = j * 32, col0 = nt * BN + cj;
                uint32_t v[32];
                load_block(taddr, (uint32_t)cj, v);
                dev::tmem_ld_wait();
                dev::reg_fence16(v);
                dev::reg_fence16(v + 16);
                if (j + kEpiPerQuarter >= C::BLOCKS) hand_back();  // the warp's last read, before its stores
                if (col0 < a.e.n && row0 < a.e.m)
                    finish_block<T>(a.e, v, params + 256 * i, row_scale, row0, col0, stg, lane);
            }
        }
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) dev::cluster_sync();
    if (warp == 1) {
        dev::tc_fence_after_sync();
        dev::tmem_dealloc<CG>(tmem, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_status = cudaSuccess;

cudaError_t load_encoder()
{
    std::call_once(g_encode_once, [] {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f) {
            g_encode_status = e != cudaSuccess ? e : cudaErrorNotSupported;
            return;
        }
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return g_encode_status;
}

// f16 [rows][kp] in boxes of one step by box_rows rows.
cudaError_t encode_f16(const void *base, long long rows, int kp, int box_rows, CUtensorMap *out)
{
    cuuint64_t dims[2] = {(cuuint64_t)kp, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)kp * 2};
    cuuint32_t box[2] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = g_encode(out, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int padded_k(int k) { return k > 0 ? (k + kBlockK - 1) / kBlockK * kBlockK : kBlockK; }

template <typename T, int BN, bool PAIR>
cudaError_t gemm_launch(const LinearProblem &p, const __half *a16, const __half *w16, int kp, int sm_count,
                        cudaStream_t stream)
{
    using C = GemmCfg<BN, PAIR, sizeof(T)>;
    static bool allowed[kMaxDevices] = {};
    cudaError_t e = allow_dynamic_smem(linear_gemm_kernel<T, BN, PAIR>, C::SMEM, allowed);
    if (e != cudaSuccess) return e;
    CUtensorMap ta, tw;
    e = encode_f16(a16, p.m, kp, kBlockM, &ta);
    if (e == cudaSuccess) e = encode_f16(w16, p.n, kp, C::B_ROWS, &tw);
    if (e != cudaSuccess) return e;
    GemmArgs a{};
    a.e = linear_epilogue_of(p);
    a.k_iters = kp / kBlockK;
    constexpr int kRows = PAIR ? 256 : 128;
    a.m_tiles = (int)((p.m + kRows - 1) / kRows);
    a.n_tiles = (p.n + BN - 1) / BN;
    a.tiles = a.m_tiles * a.n_tiles;
    const int workers = PAIR ? sm_count / 2 : sm_count;
    const int grid = (a.tiles < workers ? a.tiles : workers) * (PAIR ? 2 : 1);
    return launch_overlapped(linear_gemm_kernel<T, BN, PAIR>, dim3((unsigned)grid), dim3(kThreads), (size_t)C::SMEM,
                             stream, PAIR ? 2 : 1, ta, tw, a);
}

// The three tiles: 256 x 256 and 256 x 128 by CTA pairs, 128 x 64 by single CTAs.  Their time is modelled by
// what they measured (us): a step of 64 K elements, the least time of a tile, which its epilogue sets, and
// what a launch takes besides.  Small tiles pay where the large ones would leave SMs idle:
// 1024x1024x4096 22.6 / 16.0 / 18.3, 512x512x512 8.0 / 6.1 / 5.2, 4096x4096x4096 74 / 86 / 213.
struct TileCost {
    int rows, channels, ctas;
    float step, least, launch;
};
constexpr TileCost kTiles[3] = {{256, 256, 2, 0.30f, 3.4f, 4.8f}, {256, 128, 2, 0.205f, 2.1f, 4.0f}, {128, 64, 1, 0.24f, 1.2f, 3.2f}};

float tile_time(const TileCost &c, long long m, int n, int kp, int sm_count)
{
    const long long tiles = ((m + c.rows - 1) / c.rows) * ((n + c.channels - 1) / c.channels);
    const int workers = sm_count / c.ctas;
    const float steps = c.step * (float)(kp / kBlockK);
    return (float)((tiles + workers - 1) / workers) * (steps > c.least ? steps : c.least) + c.launch;
}

int best_tile(long long m, int n, int kp, int sm_count)
{
    int best = 0;
    for (int i = 1; i < 3; ++i)
        if (tile_time(kTiles[i], m, n, kp, sm_count) < tile_time(kTiles[best], m, n, kp, sm_count)) best = i;
    return best;
}

template <typename T>
cudaError_t gemm_launch_t(const LinearProblem &p, const __half *a16, const __half *w16, int kp, int sm_count,
                          cudaStream_t stream)
{
    switch (best_tile(p.m, p.n, kp, sm_count)) {
    case 0: return gemm_launch<T, 256, true>(p, a16, w16, kp, sm_count, stream);
    case 1: return gemm_launch<T, 128, true>(p, a16, w16, kp, sm_count, stream);
    default: return gemm_launch<T, 64, false>(p, a16, w16, kp, sm_count, stream);
    }
}

}  // namespace

cudaError_t encode_bytes_map(const void *base, long long rows, int k, long long stride, int box_rows, int box_k,
                             CUtensorMap *out)
{
    const cudaError_t e = load_encoder();
    if (e != cudaSuccess) return e;
    cuuint64_t dims[2] = {(cuuint64_t)k / 4, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride};
    cuuint32_t box[2] = {(cuuint32_t)box_k / 4, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = g_encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

float tc_linear_time(long long m, int n, int k, int sm_count)
{
    // Widening reads a byte and writes two for each element, at 5 TB/s.
    const int kp = padded_k(k);
    return 2.5f + 3.0f * (float)(m + n) * (float)kp / 5.0e6f + tile_time(kTiles[best_tile(m, n, kp, sm_count)], m, n, kp, sm_count);
}

void tc_linear_plan(long long m, int n, int k, int sm_count, LinearPlan *plan)
{
    const TileCost &c = kTiles[best_tile(m, n, padded_k(k), sm_count)];
    plan->kernel = CBS_LINEAR_GEMM;
    plan->tile_rows = c.rows;
    plan->tile_channels = c.channels;
    plan->k_steps = padded_k(k) / kBlockK;
    plan->tiles = (int)(((m + c.rows - 1) / c.rows) * ((n + c.channels - 1) / c.channels));
    plan->workers = plan->tiles < sm_count / c.ctas ? plan->tiles : sm_count / c.ctas;
}

long long tc_linear_workspace_bytes(long long m, int n, int k)
{
    const long long kp = padded_k(k);
    return (m * kp * 2 + 255) / 256 * 256 + (long long)n * kp * 2;
}

cudaError_t tc_linear_launch(const LinearProblem &p, int sm_count, cudaStream_t stream)
{
    cudaError_t e = load_encoder();
    if (e != cudaSuccess) return e;
    const int kp = padded_k(p.k);
    __half *a16 = static_cast<__half *>(p.workspace);
    __half *w16 = a16 + (p.m * kp * 2 + 255) / 256 * 256 / 2;
    auto matrix = [](const Rows &r, __half *dst) {
        return WidenMatrix{static_cast<const int8_t *>(r.data), dst, r.stride,
                           reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.stride % 16 == 0};
    };
    WidenArgs wa{matrix(p.a, a16), matrix(p.w, w16), p.m, p.m + p.n, p.k, kp, 0};
    while (wa.lanes_log2 < 8 && (16 << wa.lanes_log2) < kp) ++wa.lanes_log2;
    const long long per_block = 256 >> wa.lanes_log2;
    const long long blocks = (wa.rows + per_block - 1) / per_block, most = 16LL * sm_count;
    e = launch_overlapped(widen_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, stream, 1, wa);
    if (e != cudaSuccess) return e;
    switch (p.out_dtype) {
    case kF32: return gemm_launch_t<float>(p, a16, w16, kp, sm_count, stream);
    case kBf16: return gemm_launch_t<__nv_bfloat16>(p, a16, w16, kp, sm_count, stream);
    default: return gemm_launch_t<__half>(p, a16, w16, kp, sm_count, stream);
    }
}

cudaError_t tc_linear_read_and_clear_error(cudaStream_t stream, unsigned int *out)
{
    return read_and_clear_word(g_linear_error, stream, out);
}

}  // namespace cbs
