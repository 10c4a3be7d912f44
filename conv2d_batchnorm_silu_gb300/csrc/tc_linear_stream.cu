// tc_linear_stream.cu -- the int8 linear layer for tens to hundreds of rows, where the weights' bytes
// count: they are read once as int8 and widened to f16 between global and shared memory.
//
// D[channel][row] = W * A^T with 128 channels on the tensor core's M side and NT rows on its N side.
// Sixteen warps hold the int8 of the coming steps in registers (kAhead steps of 128 K elements, 48 KB of
// weights per SM in flight, whole 128-byte lines of each row), widen a step of weights and rows at a time into
// swizzled f16 tiles, and hand them to the issuing warp.  Rows that start at multiples of 4 bytes only are loaded
// in words, and rows that start anywhere in one word more (64x8192x8192 21 us, x8196 26, x8193 43; widened before
// the product 75).  Every CTA takes an equal run of the (channel tile, row tile, K step) sequence, so that all SMs
// read the same share of the weights, and leaves its tiles as fp32 partial sums in the workspace, which a second
// kernel adds in K order and finishes.
//
// Bound by the widening: with loads in words a step of 128 K elements takes 1,400 clocks with 64 rows, of which
// its bytes need some 700 at the memory's rate and its MMAs 500.
#include <cuda.h>
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
constexpr int kPrefetch = 1024;  // bytes of each weights row that the start of a run brings into L2
constexpr int kWidenWarps = 16;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (kWidenWarps + kEpiWarps + 1);

template <int NT>
struct StreamCfg {
    static constexpr int A_BYTES = kChannels * kStep * 2;
    static constexpr int B_BYTES = NT * kStep * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = NT <= 64 ? 4 : (NT <= 128 ? 3 : 2);
    static constexpr int SMEM = 1024 + STAGES * STAGE + 256;
    static constexpr int ROW_LOADS = (NT + 63) / 64;  // 16-byte pieces of rows per thread and step
    static constexpr int kAhead = NT <= 64 ? 3 : 2;  // steps held in registers
    static constexpr int TMEM_COLS = 2 * NT;
};

struct StreamArgs {
    LinearEpilogue e;
    // The operands, channels on the tensor core's M side and rows on its N side: the weights and the rows of the
    // layer or, where its weights are few, the other way round (its rows streamed as channels).
    const int8_t *a, *w;
    long long a_stride, w_stride;
    int rows, channels;
    int k, k_steps;
    int row_tiles, tiles;      // tile = channel tile * row_tiles + row tile
    int steps;                 // tiles * k_steps
    int workers;               // CTAs that share them: run_base steps each, and one more for the first run_extra
    int run_base, run_extra;
    float *partial;            // [workers + tiles][NT][kChannels]
};

__device__ __forceinline__ void give_up(unsigned int bit, volatile int *abort_flag)
{
    atomicOr(&g_stream_error, bit);
    *abort_flag = 1;
}

// What rows of a hold past k.
__device__ const uint4 g_zeros = {0, 0, 0, 0};

// Predicated loads straight into their registers, which otherwise keep what they hold.
__device__ __forceinline__ void load_if(uint32_t &v, const int8_t *p, bool yes)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "@p ld.global.nc.b32 %0, [%1];\n\t}"
        : "+r"(v)
        : "l"(p), "r"((int)yes));
}
__device__ __forceinline__ void load_if(uint4 &v, const int8_t *p, bool yes)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"((int)yes));
}
// 16 bytes of a row, of which the row has `left`: in one load, in four words, or in the five words that hold them
// where rows start anywhere, which are put in place when they are used.  Of weights what is past the row may be
// anything; of rows it has to be zeros, and is but for the bytes of a last word, which are masked when it is used.
template <int ALIGN>
struct Held {
    uint4 v;
    uint32_t more;
    __device__ __forceinline__ void load_weights(const int8_t *p, int left)
    {
        if constexpr (ALIGN == 16) {
            load_if(v, p, left > 0);
        } else {
            const int off = ALIGN == 1 ? (int)(reinterpret_cast<uintptr_t>(p) & 3) : 0;
            load_if(v.x, p - off, left > 0);
            load_if(v.y, p - off + 4, left > 4 - off);
            load_if(v.z, p - off + 8, left > 8 - off);
            load_if(v.w, p - off + 12, left > 12 - off);
            if constexpr (ALIGN == 1) load_if(more, p - off + 16, off > 0 && left > 16 - off);
        }
    }
    __device__ __forceinline__ void load_row(const int8_t *p, int left)
    {
        const int8_t *zeros = reinterpret_cast<const int8_t *>(&g_zeros);
        if constexpr (ALIGN == 16) {
            load_if(v, left > 0 ? p : zeros, true);
        } else {
            const int off = ALIGN == 1 ? (int)(reinterpret_cast<uintptr_t>(p) & 3) : 0;
            load_if(v.x, left > 0 ? p - off : zeros, true);
            load_if(v.y, left > 4 - off ? p - off + 4 : zeros, true);
            load_if(v.z, left > 8 - off ? p - off + 8 : zeros, true);
            load_if(v.w, left > 12 - off ? p - off + 12 : zeros, true);
            if constexpr (ALIGN == 1) load_if(more, off > 0 && left > 16 - off ? p - off + 16 : zeros, true);
        }
    }
    __device__ __forceinline__ uint4 get(uint32_t off) const
    {
        if constexpr (ALIGN != 1) return v;
        const uint32_t bits = off * 8;
        return make_uint4(__funnelshift_r(v.x, v.y, bits), __funnelshift_r(v.y, v.z, bits), __funnelshift_r(v.z, v.w, bits),
                          __funnelshift_r(v.w, more, bits));
    }
};

// As sts_v4, at a constant distance from a base.
template <int OFFSET>
__device__ __forceinline__ void sts_v4_at(uint32_t base, const uint2 &lo, const uint2 &hi)
{
    asm volatile("st.shared.v4.b32 [%0+%5], {%1, %2, %3, %4};" ::"r"(base), "r"(lo.x), "r"(lo.y), "r"(hi.x), "r"(hi.y),
                 "n"(OFFSET)
                 : "memory");
}

template <int OFFSET>
__device__ __forceinline__ void widen_to(uint32_t at0, uint32_t at1, const uint4 &v)
{
    sts_v4_at<OFFSET>(at0, widen4(v.x), widen4(v.y));
    sts_v4_at<OFFSET>(at1, widen4(v.z), widen4(v.w));
}

// First step of worker b's run, and the worker that has step g.
__device__ __forceinline__ int run_start(const StreamArgs &a, int b) { return b * a.run_base + min(b, a.run_extra); }
__device__ __forceinline__ int worker_of(const StreamArgs &a, int g)
{
    const int longer = a.run_extra * (a.run_base + 1);  // steps of the longer runs
    return g < longer ? g / (a.run_base + 1) : a.run_extra + (g - longer) / a.run_base;
}

// The sums of a run's tiles to the workspace: lane = channel, column = row of a.  This code runs once or twice a
// launch and is bound by fetching itself: it only stores the sums.  (With the epilogue's arithmetic here for tiles
// of one CTA, 64x512x512 took 8.9 us against 6.0 us with the join.)
template <int NT>
__device__ __forceinline__ void store_sums(const StreamArgs &a, int g0, int steps, uint32_t tmem, int warp, int lane,
                                           uint64_t *tfull, uint64_t *tempty, volatile int *abort_flag)
{
    const int quarter = warp & 3;
    int tile = g0 / a.k_steps, ks = g0 - tile * a.k_steps;
    for (int piece = 0, left = steps; left > 0; ++piece, ++tile, ks = 0) {
        const int take = min(left, a.k_steps - ks), buf = piece & 1;
        left -= take;
        const int rows = min(NT, a.rows - tile % a.row_tiles * NT);
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
        float *out = a.partial + ((long long)(blockIdx.x + tile) * NT) * kChannels + quarter * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < rows; c += 16) {
            uint32_t v[16];
            dev::tmem_ld_32x32b_x16(taddr + (uint32_t)c, v);
            dev::tmem_ld_wait();
            dev::reg_fence16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) out[(c + i) * kChannels] = __uint_as_float(v[i]);  // within NT rows
        }
        dev::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&tempty[buf]));
    }
}

// ALIGN: rows of both operands start at multiples of it, and k is one.
template <int NT, int ALIGN>
__global__ void __launch_bounds__(kThreads, 1) linear_stream_kernel(const StreamArgs a)
{
    using C = StreamCfg<NT>;
    constexpr int STAGES = C::STAGES, AHEAD = C::kAhead, LOADS = 2 + C::ROW_LOADS;
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
    const int g0 = run_start(a, blockIdx.x), steps = run_start(a, blockIdx.x + 1) - g0;
    if (threadIdx.x < kChannels) {
        // The weights of the run's first steps.
        const int tile = g0 / a.k_steps, k0 = (g0 - tile * a.k_steps) * kStep;
        const int n = min(tile / a.row_tiles * kChannels + (int)threadIdx.x, a.channels - 1);
        if constexpr (ALIGN == 16) prefetch_l2(a.w + (long long)n * a.w_stride + k0, (uint32_t)min(a.k - k0, kPrefetch));
    }
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();

    if (warp < kWidenWarps) {
        // ---------------------------------------------------------- loads and widening
        // Piece j of this thread: 16 bytes of K from 16 * (tid % 8) of weights rows tid / 8 + 64 j for
        // j < 2, then of rows of a.  Rows past the end read the last one: nothing stores what they give.
        // Past k rows of a are zeros and the weights any values; past the run, too.
        const int tid = threadIdx.x, q = tid & 7, r8 = tid >> 3;
        int tile = g0 / a.k_steps, ks = g0 - tile * a.k_steps, unloaded = steps;  // of the next load
        const bool has_row = NT >= 64 || r8 < NT;
        const int last_left = a.k - (a.k_steps - 1) * kStep - q * 16;  // of a last step, from this thread's part on
        const int8_t *src[LOADS];
        auto rows_of_tile = [&]() {
            const int ct = tile / a.row_tiles, rt = tile - ct * a.row_tiles, k0 = ks * kStep + q * 16;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                src[j] = a.w + (long long)min(ct * kChannels + j * 64 + r8, a.channels - 1) * a.w_stride + k0;
#pragma unroll
            for (int j = 0; j < C::ROW_LOADS; ++j)
                src[2 + j] = a.a + (long long)min(rt * NT + j * 64 + r8, a.rows - 1) * a.a_stride + k0;
        };
        rows_of_tile();
        Held<ALIGN> held[AHEAD][LOADS];
        uint32_t offs[AHEAD];  // where the pieces of each start in a word, two bits for each; bit 31: a last step
        auto load = [&](Held<ALIGN> (&to)[LOADS], uint32_t &off) {
            if (unloaded <= 0) return;  // what is held is not used again
            --unloaded;
            const int left = ks == a.k_steps - 1 ? last_left : 16;
            if constexpr (ALIGN == 1) {
                off = ks == a.k_steps - 1 ? 1u << 31 : 0u;
#pragma unroll
                for (int j = 0; j < LOADS; ++j) off |= ((uint32_t)reinterpret_cast<uintptr_t>(src[j]) & 3u) << (2 * j);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                to[j].load_weights(src[j], left);
                src[j] += kStep;
            }
            if (has_row)
#pragma unroll
                for (int j = 0; j < C::ROW_LOADS; ++j) {
                    to[2 + j].load_row(src[2 + j], left);
                    src[2 + j] += kStep;
                }
            if (++ks == a.k_steps) {
                ks = 0;
                ++tile;
                rows_of_tile();
            }
        };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) held[d][j].v = make_uint4(0, 0, 0, 0), held[d][j].more = 0;
            offs[d] = 0;
            load(held[d], offs[d]);
        }
        // Bytes 16 q .. 16 q + 15 become two f16 pieces of the row's 256 bytes, in the first span (q < 4) or
        // the second.  The second span holds each two pieces in the other order, for weights and rows alike:
        // the sum is the same, and eight lanes of a row meet eight different banks.
        const uint32_t span = (uint32_t)q >> 2, pair = ((uint32_t)q & 3u) * 2, turn = (uint32_t)r8 & 7u;
        const uint32_t o0 = (uint32_t)r8 * 128 + (((pair + span) ^ turn) << 4);
        const uint32_t o1 = (uint32_t)r8 * 128 + (((pair + (span ^ 1u)) ^ turn) << 4);
        const uint32_t ta0 = dev::smem_u32(sm_a) + span * (C::A_BYTES / 2), tb0 = dev::smem_u32(sm_b) + span * (C::B_BYTES / 2);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int left = steps; left > 0 && ok; left -= AHEAD) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                if (d >= left) break;
                ok = __all_sync(0xffffffffu, wait_bounded(dev::smem_u32(&empty[stage]), phase ^ 1u,
                                                                    abort_flag, kWaitNs));
                if (!ok) {
                    if (lane == 0 && !*abort_flag) give_up(kErrTimeoutProducer, abort_flag);
                    break;
                }
                const uint32_t ta = ta0 + (uint32_t)(stage * C::A_BYTES), tb = tb0 + (uint32_t)(stage * C::B_BYTES);
                auto weights = [&](int j) { return held[d][j].get(offs[d] >> (2 * j) & 3u); };
                auto row = [&](int j) {
                    const uint4 v = held[d][2 + j].get(offs[d] >> (2 * j + 4) & 3u);
                    return ALIGN == 1 && (int)offs[d] < 0 ? within(v, 0, max(last_left, 0)) : v;
                };
                widen_to<0>(ta + o0, ta + o1, weights(0));
                widen_to<64 * 128>(ta + o0, ta + o1, weights(1));
                if (has_row) {
                    widen_to<0>(tb + o0, tb + o1, row(0));
                    if constexpr (C::ROW_LOADS > 1) widen_to<64 * 128>(tb + o0, tb + o1, row(1));
                    if constexpr (C::ROW_LOADS > 2) {
                        widen_to<128 * 128>(tb + o0, tb + o1, row(2));
                        widen_to<192 * 128>(tb + o0, tb + o1, row(3));
                    }
                }
                dev::fence_proxy_async_shared();  // the tensor core reads through the async proxy
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(dev::smem_u32(&full[stage]));
                load(held[d], offs[d]);
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMAs
        // The whole warp runs the loop and one elected lane issues: with the control flow uniform, descriptors
        // are computed and held in uniform registers, which an MMA takes as they are (49 clocks an MMA among
        // busy warps, against 71 issued behind `lane == 0`).
        const bool issuer = elect_one();
        constexpr uint32_t idesc = idesc_f16(kChannels, NT);
        const uint64_t desc_a = dev::smem_desc_kmajor(dev::smem_u32(sm_a), 128);
        const uint64_t desc_b = dev::smem_desc_kmajor(dev::smem_u32(sm_b), 128);
        int stage = 0, piece = 0, ks = g0 % a.k_steps;
        uint32_t phase = 0, accumulate = 0;
        for (int g = 0; g < steps; ++g) {
            const int buf = piece & 1;
            bool ok = true;
            if (accumulate == 0)
                ok = wait_bounded(dev::smem_u32(&tempty[buf]), ((uint32_t)(piece >> 1) & 1u) ^ 1u, abort_flag, kWaitNs);
            ok = ok && wait_bounded(dev::smem_u32(&full[stage]), phase, abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                if (issuer && !*abort_flag) give_up(kErrTimeoutMma, abort_flag);
                break;
            }
            dev::tc_fence_after_sync();
            const uint64_t da = desc_a + (uint64_t)(stage * (C::A_BYTES >> 4));
            const uint64_t db = desc_b + (uint64_t)(stage * (C::B_BYTES >> 4));
            const uint32_t d = tmem + (uint32_t)(buf * NT);
            const bool last = ++ks == a.k_steps || g + 1 == steps;
            if (issuer) {
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk) {
                    const uint64_t span = (uint64_t)(kk / 4), in = (uint64_t)(2 * (kk % 4));
                    dev::tc_mma_bf16<1>(d, da + span * (C::A_BYTES / 2 >> 4) + in, db + span * (C::B_BYTES / 2 >> 4) + in,
                                        idesc, kk > 0 ? 1u : accumulate);
                }
                dev::tc_commit<1>(dev::smem_u32(&empty[stage]));
                if (last) dev::tc_commit<1>(dev::smem_u32(&tfull[buf]));
            }
            __syncwarp();
            if (++stage == STAGES) stage = 0, phase ^= 1u;
            accumulate = 1;
            if (last) {
                ks = 0;
                ++piece;
                accumulate = 0;
            }
        }
        // Every MMA must have finished before tensor memory is freed.
        if (issuer) {
            dev::tc_commit<1>(dev::smem_u32(drain));
            if (!dev::mbar_wait_bounded(dev::smem_u32(drain), 0, nullptr, kWaitNs)) give_up(kErrTimeoutDrain, abort_flag);
        }
        __syncwarp();
    } else {
        store_sums<NT>(a, g0, steps, tmem, warp, lane, tfull, tempty, abort_flag);
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        dev::tc_fence_after_sync();
        dev::tmem_dealloc<1>(tmem, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ the same with the weights in tensor memory
// Where both operands' rows are 16-byte aligned and a tile has at most 128 rows.  In linear_stream_kernel shared
// memory takes the widened weights and gives them to the tensor core again, four bytes for each one of memory, and
// each of its loads costs instructions.  Here the bytes of both operands come through TMA rings (96 to 140 KB in
// flight), two groups of eight warps widen the weights of alternate steps from there into tensor memory, where the
// tensor core finds its first operand (lane = channel), and four more widen the rows into shared memory.
//
// 8192x8192 weights: 32 rows 19.7 us (21.1 in linear_stream_kernel), 64 rows 21.5 (23.2), 128 rows 27.1 (30.2);
// turned 25984x40x4800 37 (41).  A step takes 1,000 clocks with 32 rows, hot in L2 or not: what
// 152 SMs draw from L2, weights at 4.8 TB/s and rows beside them; the first step comes 5,000 clocks after the start.
// Tried and slower: prefetching each row's next 1 KB into L2 (32 us), loads in bursts of three steps (23.0).
template <int NT>
struct RingCfg {
    static constexpr int W_RAW = kChannels * kStep, R_RAW = NT * kStep, RAW = W_RAW + R_RAW;
    static constexpr int RAWS = NT == 128 ? 4 : (NT == 64 ? 6 : 7);  // steps of bytes in flight
    static constexpr int B_BYTES = NT * kStep * 2;
    static constexpr int STAGES = NT == 128 ? 3 : 4;  // widened steps
    static constexpr int A_COLS = kStep / 2;          // of tensor memory, for each of them
    static constexpr int WIDEN_WARPS = 8 + 4;         // of a step, for weights and rows; two such groups take turns
    static constexpr int WARPS = 4 + 2 * WIDEN_WARPS + 4;  // TMA, MMA, two without work, widening, epilogue
    static constexpr int SMEM = 1024 + RAWS * RAW + STAGES * B_BYTES + 256;
    static_assert(2 * NT + STAGES * A_COLS <= 512 && SMEM <= 232448, "fits");
};

__device__ __forceinline__ void tc_mma_tmem_a(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 words of each lane to 32 columns of its warp's quarter of tensor memory.
__device__ __forceinline__ void tmem_st_32(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
        " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
        " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int NT>
__global__ void __launch_bounds__(32 * RingCfg<NT>::WARPS, 1)
    linear_ring_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_r, const StreamArgs a)
{
    using C = RingCfg<NT>;
    constexpr int STAGES = C::STAGES, RAWS = C::RAWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sm_raw = dev::smem_u32(smem), sm_b = sm_raw + RAWS * C::RAW;
    uint64_t *rfull = reinterpret_cast<uint64_t *>(smem + RAWS * C::RAW + STAGES * C::B_BYTES);
    uint64_t *rempty = rfull + RAWS, *full = rempty + RAWS, *empty = full + STAGES, *tfull = empty + STAGES;
    uint64_t *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < RAWS; ++i) {
            dev::mbar_init(dev::smem_u32(&rfull[i]), 1);
            dev::mbar_init(dev::smem_u32(&rempty[i]), C::WIDEN_WARPS);
        }
        for (int i = 0; i < STAGES; ++i) {
            dev::mbar_init(dev::smem_u32(&full[i]), C::WIDEN_WARPS);
            dev::mbar_init(dev::smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            dev::mbar_init(dev::smem_u32(&tfull[i]), 1);
            dev::mbar_init(dev::smem_u32(&tempty[i]), kEpiWarps);
        }
        dev::mbar_init(dev::smem_u32(drain), 1);
        *abort_flag = 0;
        dev::fence_mbarrier_init();
        dev::prefetch_tensormap(&tm_w);
        dev::prefetch_tensormap(&tm_r);
    }
    if (warp == 1) {
        dev::tmem_alloc<1>(dev::smem_u32(tmem_slot), 512);
        dev::tmem_relinquish_alloc_permit<1>();
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    dev::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot, tmem_a = tmem + 2 * NT;
    const int g0 = run_start(a, blockIdx.x), steps = run_start(a, blockIdx.x + 1) - g0;
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();

    if (warp == 0) {
        // ---------------------------------------------------------- loads
        int tile = g0 / a.k_steps, ks = g0 - tile * a.k_steps, stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        for (int g = 0; g < steps; ++g) {
            bool ok = true;
            if (lane == 0) {
                ok = wait_bounded(dev::smem_u32(&rempty[stage]), phase ^ 1u, abort_flag, kWaitNs);
                if (!ok && !*abort_flag) give_up(kErrTimeoutProducer, abort_flag);
                if (ok) {
                    const int ct = tile / a.row_tiles, rt = tile - ct * a.row_tiles;
                    const uint32_t bar = dev::smem_u32(&rfull[stage]), dst = sm_raw + (uint32_t)(stage * C::RAW);
                    dev::mbar_arrive_expect_tx(bar, C::RAW);
                    dev::tma_load_2d(dst, &tm_w, bar, ks * (kStep / 4), ct * kChannels);
                    dev::tma_load_2d(dst + C::W_RAW, &tm_r, bar, ks * (kStep / 4), rt * NT);
                    issued |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                }
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            if (++stage == RAWS) stage = 0, phase ^= 1u;
            if (++ks == a.k_steps) ks = 0, ++tile;
        }
        // Every load must have landed before the CTA may leave.
        if (lane == 0)
            for (int i = 0; i < RAWS; ++i)
                if ((issued >> i) & 1u)
                    if (!dev::mbar_wait_bounded(dev::smem_u32(&rfull[i]), (issued_parity >> i) & 1u, nullptr, kWaitNs)) {
                        give_up(kErrTimeoutDrain, abort_flag);
                        break;
                    }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs, as in linear_stream_kernel
        const bool issuer = elect_one();
        constexpr uint32_t idesc = idesc_f16(kChannels, NT);
        const uint64_t desc_b = dev::smem_desc_kmajor(sm_b, 128);
        int stage = 0, piece = 0, ks = g0 % a.k_steps;
        uint32_t phase = 0, accumulate = 0;
        for (int g = 0; g < steps; ++g) {
            const int buf = piece & 1;
            bool ok = true;
            if (accumulate == 0)
                ok = wait_bounded(dev::smem_u32(&tempty[buf]), ((uint32_t)(piece >> 1) & 1u) ^ 1u, abort_flag, kWaitNs);
            ok = ok && wait_bounded(dev::smem_u32(&full[stage]), phase, abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                if (issuer && !*abort_flag) give_up(kErrTimeoutMma, abort_flag);
                break;
            }
            dev::tc_fence_after_sync();
            const uint32_t ta = tmem_a + (uint32_t)(stage * C::A_COLS), d = tmem + (uint32_t)(buf * NT);
            const uint64_t db = desc_b + (uint64_t)(stage * (C::B_BYTES >> 4));
            const bool last = ++ks == a.k_steps || g + 1 == steps;
            if (issuer) {
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk)
                    tc_mma_tmem_a(d, ta + (uint32_t)(8 * kk), db + (uint64_t)(kk / 4 * (C::B_BYTES / 2 >> 4) + 2 * (kk % 4)),
                                  idesc, kk > 0 ? 1u : accumulate);
                dev::tc_commit<1>(dev::smem_u32(&empty[stage]));
                if (last) dev::tc_commit<1>(dev::smem_u32(&tfull[buf]));
            }
            __syncwarp();
            if (++stage == STAGES) stage = 0, phase ^= 1u;
            accumulate = 1;
            if (last) {
                ks = 0;
                ++piece;
                accumulate = 0;
            }
        }
        // Every MMA must have finished before tensor memory is freed.
        if (issuer) {
            dev::tc_commit<1>(dev::smem_u32(drain));
            if (!dev::mbar_wait_bounded(dev::smem_u32(drain), 0, nullptr, kWaitNs)) give_up(kErrTimeoutDrain, abort_flag);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 4 + 2 * C::WIDEN_WARPS) {
        // ---------------------------------------------------------- widening
        // Weights: a lane has its channel's 64 bytes of a step.  Rows: pieces of 16 bytes, as linear_stream_kernel
        // places them; the second span's pieces hold their halves in the other order, here and there.
        const int group = warp >= 4 + C::WIDEN_WARPS, mine = warp - 4 - group * C::WIDEN_WARPS;
        const bool weights = mine < 8;
        const int half = mine >> 2, channel = (warp & 3) * 32 + lane;
        const int tid = (mine - 8) * 32 + lane, q = tid & 7, r8 = tid >> 3;
        constexpr int kRowsAtOnce = 4 * (C::WIDEN_WARPS - 8);
        const uint32_t span = (uint32_t)q >> 2, pair = ((uint32_t)q & 3u) * 2, turn = (uint32_t)r8 & 7u;
        const uint32_t o0 = span * (C::B_BYTES / 2) + (uint32_t)r8 * 128 + (((pair + span) ^ turn) << 4);
        const uint32_t o1 = span * (C::B_BYTES / 2) + (uint32_t)r8 * 128 + (((pair + (span ^ 1u)) ^ turn) << 4);
        int raw = group, stage = group;
        uint32_t raw_phase = 0, phase = 0;
        for (int g = group; g < steps; g += 2) {
            bool ok = wait_bounded(dev::smem_u32(&rfull[raw]), raw_phase, abort_flag, kWaitNs) &&
                      wait_bounded(dev::smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0 && !*abort_flag) give_up(kErrTimeoutProducer, abort_flag);
                break;
            }
            const uint32_t from = sm_raw + (uint32_t)(raw * C::RAW);
            if (weights) {
                dev::tc_fence_after_sync();
                uint32_t v[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 b = dev::lds_v4(from + (uint32_t)channel * 128 + ((uint32_t)((4 * half + c) ^ (channel & 7)) << 4));
                    const uint2 x = widen4(half ? b.z : b.x), y = widen4(half ? b.w : b.y);
                    const uint2 z = widen4(half ? b.x : b.z), w = widen4(half ? b.y : b.w);
                    v[8 * c] = x.x, v[8 * c + 1] = x.y, v[8 * c + 2] = y.x, v[8 * c + 3] = y.y;
                    v[8 * c + 4] = z.x, v[8 * c + 5] = z.y, v[8 * c + 6] = w.x, v[8 * c + 7] = w.y;
                }
                tmem_st_32(tmem_a + (uint32_t)(stage * C::A_COLS + 32 * half) + ((uint32_t)((warp & 3) * 32) << 16), v);
                dev::tc_fence_before_sync();
            } else {
                const uint32_t to = sm_b + (uint32_t)(stage * C::B_BYTES);
#pragma unroll
                for (int r = 0; r < NT; r += kRowsAtOnce) {
                    const uint4 b = dev::lds_v4(from + C::W_RAW + (uint32_t)(r + r8) * 128 + (((uint32_t)q ^ turn) << 4));
                    const uint2 x = widen4(b.x), y = widen4(b.y), z = widen4(b.z), w = widen4(b.w);
                    dev::sts_v4(to + o0 + (uint32_t)r * 128, x.x, x.y, y.x, y.y);
                    dev::sts_v4(to + o1 + (uint32_t)r * 128, z.x, z.y, w.x, w.y);
                }
                dev::fence_proxy_async_shared();  // the tensor core reads through the async proxy
            }
            __syncwarp();
            if (lane == 0) {
                dev::mbar_arrive(dev::smem_u32(&full[stage]));
                dev::mbar_arrive(dev::smem_u32(&rempty[raw]));
            }
            if ((raw += 2) >= RAWS) raw -= RAWS, raw_phase ^= 1u;
            if ((stage += 2) >= STAGES) stage -= STAGES, phase ^= 1u;
        }
    } else if (warp >= 4) {
        store_sums<NT>(a, g0, steps, tmem, warp, lane, tfull, tempty, abort_flag);
    }
    dev::tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        dev::tc_fence_after_sync();
        dev::tmem_dealloc<1>(tmem, 512);
    }
}

// The partial sums of four channels of a tile's row from workers b0 to b1, added in K order; eight load at a time.
template <int NT>
__device__ __forceinline__ void add_partial(const StreamArgs &a, int tile, int b0, int b1, int row, int channel, float *s)
{
    const float *from = a.partial + ((long long)(b0 + tile) * NT + row) * kChannels + channel;
    s[0] = s[1] = s[2] = s[3] = 0.0f;
    for (int b = b0; b <= b1; b += 8) {
        float4 v[8];
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (b + t <= b1) v[t] = *reinterpret_cast<const float4 *>(from + (long long)(b - b0 + t) * NT * kChannels);
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (b + t <= b1) s[0] += v[t].x, s[1] += v[t].y, s[2] += v[t].z, s[3] += v[t].w;
    }
}

// The workers' partial sums of a tile joined and finished.  A thread takes four channels of a row.
constexpr int kJoinRows = 4;
template <typename T, int NT>
__global__ void __launch_bounds__(32 * kJoinRows) linear_join_kernel(const StreamArgs a)
{
    const int tile = blockIdx.x, g = tile * a.k_steps;
    const int b0 = worker_of(a, g), b1 = worker_of(a, g + a.k_steps - 1);
    const int ct = tile / a.row_tiles, rt = tile - ct * a.row_tiles;
    const int i = blockIdx.y * kJoinRows + threadIdx.y, n = ct * kChannels + threadIdx.x * 4;
    const long long m = (long long)rt * NT + i;
    const bool mine = i < NT && m < a.e.m;
    // Nothing is read before the wait, scales and biases neither: the kernel before has waited for what wrote them, but
    // only this kernel's own wait makes that visible here (64x8192x8192 21.7 us; read before it, 21.5).
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    if (!mine) return;
    // On their way together with the first partial sums: without branches, at which the thread would wait for them.
    const float *biases = a.e.bias ? a.e.bias : a.e.w_scale;
    float scale[4], bias[4];
    const float row_scale = __ldg(a.e.a_scale + m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        scale[j] = __ldg(a.e.w_scale + min(n + j, a.e.n - 1));
        bias[j] = __ldg(biases + min(n + j, a.e.n - 1));
    }
    float s[4];
    add_partial<NT>(a, tile, b0, b1, i, threadIdx.x * 4, s);
    const T *res = a.e.residual ? static_cast<const T *>(a.e.residual) + m * a.e.residual_stride + n : nullptr;
    T *y = static_cast<T *>(a.e.y) + m * a.e.y_stride + n;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < a.e.n) {
            float z = activated<T>(fmaf(s[j], row_scale * scale[j], a.e.bias ? bias[j] : 0.0f), a.e.activation);
            if (res) z += to_float(res[j]);
            from_float(z, y + j);
        }
}

// The same where the channels are the layer's rows: 32 columns of 128 rows turned round in shared memory, so that
// each warp finishes 32 columns of a row of y at a time.
constexpr int kTurnWarps = 8;
template <typename T, int NT>
__global__ void __launch_bounds__(32 * kTurnWarps) linear_join_turned_kernel(const StreamArgs a)
{
    __shared__ float turned[32][kChannels + 1];
    const int tile = blockIdx.x, g = tile * a.k_steps, lane = threadIdx.x, warp = threadIdx.y;
    const int b0 = worker_of(a, g), b1 = worker_of(a, g + a.k_steps - 1);
    const int ct = tile / a.row_tiles, c0 = blockIdx.y * 32, n0 = (tile - ct * a.row_tiles) * NT + c0;
    const long long m0 = (long long)ct * kChannels;
    const int n = n0 + lane;
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    float scale = 0.0f, bias = 0.0f, row_scale[kChannels / kTurnWarps];
    if (n < a.e.n) {
        scale = __ldg(a.e.w_scale + n);
        if (a.e.bias) bias = __ldg(a.e.bias + n);
    }
#pragma unroll
    for (int j = 0; j < kChannels / kTurnWarps; ++j)
        row_scale[j] = m0 + j * kTurnWarps + warp < a.e.m ? __ldg(a.e.a_scale + m0 + j * kTurnWarps + warp) : 0.0f;
#pragma unroll
    for (int j = 0; j < 32 / kTurnWarps; ++j) {
        const int c = j * kTurnWarps + warp;
        if (n0 + c >= a.e.n) continue;
        float s[4];
        add_partial<NT>(a, tile, b0, b1, c0 + c, lane * 4, s);
        for (int t = 0; t < 4; ++t) turned[c][lane * 4 + t] = s[t];
    }
    __syncthreads();
    if (n >= a.e.n) return;
#pragma unroll
    for (int j = 0; j < kChannels / kTurnWarps; ++j) {
        const long long m = m0 + j * kTurnWarps + warp;
        if (m >= a.e.m) break;
        float z = activated<T>(fmaf(turned[lane][j * kTurnWarps + warp], row_scale[j] * scale, bias), a.e.activation);
        if (a.e.residual) z += to_float(static_cast<const T *>(a.e.residual)[m * a.e.residual_stride + n]);
        from_float(z, static_cast<T *>(a.e.y) + m * a.e.y_stride + n);
    }
}

// Row tile for m rows: the smallest that holds them.
int row_tile_of(long long m) { return m <= 32 ? 32 : (m <= 64 ? 64 : (m <= 128 ? 128 : 256)); }

struct StreamPlan {
    int nt, k_steps, row_tiles, tiles, workers;
    int steps;
};

StreamPlan plan_of(long long m, int n, int k, int sm_count)
{
    StreamPlan p{};
    p.nt = row_tile_of(m);
    p.k_steps = k > 0 ? (k + kStep - 1) / kStep : 1;
    p.row_tiles = (int)((m + p.nt - 1) / p.nt);
    p.tiles = (n + kChannels - 1) / kChannels * p.row_tiles;
    p.steps = p.tiles * p.k_steps;
    // All SMs, but at least two steps a run, and at most some sixteen runs a tile for the join.
    const int fewest = p.k_steps > 32 ? (p.k_steps + 15) / 16 : 2;
    const int most = p.steps / fewest > 0 ? p.steps / fewest : 1;
    p.workers = most < sm_count ? most : sm_count;
    return p;
}

template <int NT>
cudaError_t ring_launch(const StreamArgs &a, cudaStream_t stream)
{
    using C = RingCfg<NT>;
    static bool allowed[kMaxDevices] = {};
    cudaError_t e = allow_dynamic_smem(linear_ring_kernel<NT>, C::SMEM, allowed);
    CUtensorMap tw, tr;
    if (e == cudaSuccess) e = encode_bytes_map(a.w, a.channels, a.k, a.w_stride, kChannels, kStep, &tw);
    if (e == cudaSuccess) e = encode_bytes_map(a.a, a.rows, a.k, a.a_stride, NT, kStep, &tr);
    return e != cudaSuccess ? e
                            : launch_overlapped(linear_ring_kernel<NT>, dim3((unsigned)a.workers), dim3(32 * C::WARPS),
                                                (size_t)C::SMEM, stream, 1, tw, tr, a);
}

// Where linear_ring_kernel is the one that runs, but for rows without a tensor map.
constexpr bool ring_runs(int nt, int align) { return align == 16 && nt <= 128; }

template <int NT, int ALIGN>
cudaError_t sums_launch(const StreamArgs &a, cudaStream_t stream)
{
    if constexpr (ring_runs(NT, ALIGN)) {
        // Rows that overlap (as where all are the same) or lie 2^40 bytes apart have no tensor map.
        auto mapped = [&](long long stride) { return stride >= a.k && stride < 1LL << 40; };
        return mapped(a.a_stride) && mapped(a.w_stride) ? ring_launch<NT>(a, stream) : sums_launch<NT, 4>(a, stream);
    } else {
        using C = StreamCfg<NT>;
        static bool allowed[kMaxDevices] = {};
        const cudaError_t e = allow_dynamic_smem(linear_stream_kernel<NT, ALIGN>, C::SMEM, allowed);
        return e != cudaSuccess ? e
                                : launch_overlapped(linear_stream_kernel<NT, ALIGN>, dim3((unsigned)a.workers),
                                                    dim3(kThreads), (size_t)C::SMEM, stream, 1, a);
    }
}

template <typename T, int NT>
cudaError_t stream_launch(const StreamArgs &a, int align, bool turned, cudaStream_t stream)
{
    cudaError_t e = align == 16  ? sums_launch<NT, 16>(a, stream)
                    : align == 4 ? sums_launch<NT, 4>(a, stream)
                                 : sums_launch<NT, 1>(a, stream);
    if (e != cudaSuccess) return e;
    const int rows = a.rows < NT ? a.rows : NT;
    if (turned)
        return launch_overlapped(linear_join_turned_kernel<T, NT>, dim3((unsigned)a.tiles, (unsigned)((rows + 31) / 32)),
                                 dim3(32, kTurnWarps), 0, stream, 1, a);
    return launch_overlapped(linear_join_kernel<T, NT>, dim3((unsigned)a.tiles, (unsigned)((rows + kJoinRows - 1) / kJoinRows)),
                             dim3(32, kJoinRows), 0, stream, 1, a);
}

template <typename T>
cudaError_t stream_launch_t(const StreamArgs &a, int nt, int align, bool turned, cudaStream_t stream)
{
    switch (nt) {
    case 32: return stream_launch<T, 32>(a, align, turned, stream);
    case 64: return stream_launch<T, 64>(a, align, turned, stream);
    case 128: return stream_launch<T, 128>(a, align, turned, stream);
    default: return stream_launch<T, 256>(a, align, turned, stream);
    }
}

}  // namespace

float tc_stream_time(long long rows, int channels, int k, int align, bool turned, int sm_count)
{
    // A step of 128 K elements as measured for each row tile, both launches, and the sums' way through L2 (at
    // 5.5 TB/s, with a slower second launch, where they are turned round).
    const StreamPlan p = plan_of(rows, channels, k, sm_count);
    const float loaded = p.nt == 32 ? 0.60f : (p.nt == 64 ? 0.67f : (p.nt == 128 ? 0.91f : 1.50f));
    const float ringed = p.nt == 32 ? 0.52f : (p.nt == 64 ? 0.56f : (p.nt == 128 ? 0.71f : 1.50f));
    const float words = p.nt <= 128 ? 1.2f : 1.4f, anywhere = p.nt == 128 ? 1.6f : 2.0f;
    const float step = align == 16 ? ringed : loaded * (align == 4 ? words : anywhere);
    return (turned ? 6.5f : 5.0f) + step * (float)((p.steps + p.workers - 1) / p.workers) +
           (float)(p.workers + p.tiles) * (float)p.nt * kChannels * 8.0f / (turned ? 5.5e6f : 8.0e6f);
}

int tc_stream_align(const LinearProblem &p)
{
    auto rows_at = [&](const Rows &r, int bytes) {
        return reinterpret_cast<uintptr_t>(r.data) % bytes == 0 && r.stride % bytes == 0 && p.k % bytes == 0;
    };
    auto both_at = [&](int bytes) { return p.k > 0 && rows_at(p.a, bytes) && rows_at(p.w, bytes); };
    return both_at(16) ? 16 : (both_at(4) ? 4 : (p.k > 0 ? 1 : 0));
}

long long tc_stream_workspace_bytes(long long rows, int channels, int k, int sm_count)
{
    const StreamPlan p = plan_of(rows, channels, k, sm_count);
    return ((long long)p.workers + p.tiles) * p.nt * kChannels * 4;
}

void tc_stream_plan(long long rows, int channels, int k, int align, bool turned, int sm_count, LinearPlan *plan)
{
    const StreamPlan p = plan_of(rows, channels, k, sm_count);
    plan->kernel = ring_runs(p.nt, align) ? CBS_LINEAR_RING : CBS_LINEAR_STREAM;
    plan->turned = turned;
    plan->tile_rows = turned ? kChannels : p.nt;
    plan->tile_channels = turned ? p.nt : kChannels;
    plan->align = align;
    plan->k_steps = p.k_steps;
    plan->tiles = p.tiles;
    plan->workers = p.workers;
}

cudaError_t tc_stream_launch(const LinearProblem &p, bool turned, int sm_count, cudaStream_t stream)
{
    const int align = tc_stream_align(p);
    if (align == 0) return cudaErrorInvalidValue;
    StreamArgs a{};
    a.e = linear_epilogue_of(p);
    a.rows = turned ? p.n : (int)p.m;
    a.channels = turned ? (int)p.m : p.n;
    const Rows &rows = turned ? p.w : p.a, &channels = turned ? p.a : p.w;
    a.a = static_cast<const int8_t *>(rows.data);
    a.a_stride = rows.stride;
    a.w = static_cast<const int8_t *>(channels.data);
    a.w_stride = channels.stride;
    const StreamPlan plan = plan_of(a.rows, a.channels, p.k, sm_count);
    a.k = p.k;
    a.k_steps = plan.k_steps;
    a.row_tiles = plan.row_tiles;
    a.tiles = plan.tiles;
    a.steps = plan.steps;
    a.workers = plan.workers;
    a.run_base = plan.steps / plan.workers;
    a.run_extra = plan.steps % plan.workers;
    a.partial = static_cast<float *>(p.workspace);
    switch (p.out_dtype) {
    case kF32: return stream_launch_t<float>(a, plan.nt, align, turned, stream);
    case kBf16: return stream_launch_t<__nv_bfloat16>(a, plan.nt, align, turned, stream);
    default: return stream_launch_t<__half>(a, plan.nt, align, turned, stream);
    }
}

cudaError_t tc_stream_read_and_clear_error(cudaStream_t stream, unsigned int *out)
{
    return read_and_clear_word(g_stream_error, stream, out);
}

}  // namespace cbs
