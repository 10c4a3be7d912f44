// adapters.cu -- low-rank adapters of many requests beside a linear layer, and their gradients.
//
// Row i has adapter g = index[i], or none where index[i] is outside [0, adapters):
//
//   hidden_i = A_g x_i,  y_i = base_i + s_g B_g hidden_i        (y_i = base_i without an adapter)
//
// and with the gradient dy of y,
//
//   dhidden_i = B_g^T dy_i,  dx_i = base_i + s_g A_g^T dhidden_i,
//   dA_g = s_g sum_i dhidden_i x_i^T,  dB_g = s_g sum_i dy_i hidden_i^T  over the rows of g.
//
// y and dx are the same two products after one another, the second with the transposed weights.  Rows are taken by
// adapter, in an order that this file's first kernel finds: any order of rows costs the same, and the sums of the
// weights' gradients are over the rows as they come.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "adapters.h"
#include "cbs_internal.h"
#include "ptx.cuh"
#include "token_ops.h"

namespace cbs {
namespace {

// ------------------------------------------------------------------ rows by adapter
// Each block takes a window of 1024 rows and sorts them by adapter; where an adapter's rows go in all, it finds by
// counting the whole index itself, so that no block waits for another.  The counts are sums of integers: their order
// does not matter.  Rows without an adapter come last, as those of an adapter more.  777 rows 4.8 us, 8192 6.3 (cold),
// by its barriers and trips to memory.  Every block counts every row, so that many rows cost their square: 65536 24 us,
// 262144 154 (of 1189 with the products of 4096x4096, rank 16), 2^20 2065 (of 6016).
constexpr int kWindow = 1024, kFewBins = 96;

struct OrderArgs {
    const int *index;
    int *order, *starts, *tile_count;
    AdapterTile *tiles;
    AdapterTile *steps;  // nullable: tiles of kTcStepRows rows, and where each adapter's begin
    int *step_starts;
    int m, adapters, tile_rows;
};

__global__ void __launch_bounds__(kWindow) adapter_order_kernel(const OrderArgs a)
{
    extern __shared__ int order_bins[];  // [6][bins], and for few [32][kFewBins]
    __shared__ unsigned keys[kWindow];
    __shared__ unsigned long long warp_sums[32];
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const int bins = a.adapters + 1, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int *total = order_bins, *before = total + bins, *head = before + bins, *base = head + bins, *tile_base = base + bins,
        *step_base = tile_base + bins;
    for (int i = tid; i < bins; i += kWindow) total[i] = before[i] = 0;
    __syncthreads();
    auto of = [&](int i) {
        const int v = a.index[i];
        return v < 0 || v >= a.adapters ? a.adapters : v;
    };
    const int start = (int)blockIdx.x * kWindow;
    const bool few = bins <= kFewBins;
    bool here = start + tid < a.m;
    int mine = here ? of(start + tid) : -1, row = start + tid, local;  // local: rows of the adapter before it in the window
    if (!few || a.m > kWindow) {
        constexpr int kAhead = 4;
        for (int i0 = 0; i0 < a.m; i0 += kAhead * kWindow) {
            int v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) v[j] = i0 + j * kWindow + tid < a.m ? of(i0 + j * kWindow + tid) : -1;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const unsigned same = __match_any_sync(0xffffffffu, v[j]);
                if (v[j] >= 0 && lane == __ffs((int)same) - 1) {
                    atomicAdd(total + v[j], __popc(same));
                    if (i0 + j * kWindow < start) atomicAdd(before + v[j], __popc(same));
                }
            }
        }
    }
    if (few) {
        // Of few adapters: each warp's counts side by side, added up over the warps before.
        int(*const counts)[kFewBins] = reinterpret_cast<int(*)[kFewBins]>(step_base + bins);
        for (int b = lane; b < bins; b += 32) counts[warp][b] = 0;
        __syncwarp();
        const unsigned same = __match_any_sync(0xffffffffu, mine);
        local = __popc(same & ((1u << lane) - 1));
        if (here && local == 0) counts[warp][mine] = __popc(same);
        __syncthreads();
        if (tid < bins) {
            int c[32], sum = 0;
#pragma unroll
            for (int w = 0; w < 32; ++w) c[w] = counts[w][tid];
#pragma unroll
            for (int w = 0; w < 32; ++w) {
                counts[w][tid] = sum;
                sum += c[w];
            }
            if (a.m <= kWindow) total[tid] = sum;  // the window is all there is
        }
        __syncthreads();
        if (here) local += counts[warp][mine];
    } else {
        // The window's rows sorted by adapter, and among one adapter's in their order.
        unsigned key = here ? (unsigned)mine << 10 | (unsigned)tid : 0xffffffffu;
        for (int k = 2; k <= kWindow; k <<= 1)
            for (int j = k / 2; j > 0; j >>= 1) {
                unsigned other;
                if (j >= 32) {
                    __syncthreads();
                    keys[tid] = key;
                    __syncthreads();
                    other = keys[tid ^ j];
                } else {
                    other = __shfl_xor_sync(0xffffffffu, key, j);
                }
                const bool smaller = ((tid & j) == 0) == ((tid & k) == 0);
                key = (key < other) == smaller ? key : other;
            }
        __syncthreads();
        keys[tid] = key;
        __syncthreads();
        here = key != 0xffffffffu;
        mine = (int)(key >> 10);
        row = start + (int)(key & 1023u);
        if (here && (tid == 0 || (int)(keys[tid - 1] >> 10) != mine)) head[mine] = tid;
        __syncthreads();
        local = here ? tid - head[mine] : 0;
    }
    // Exclusive sums of rows (21 bits), tiles and steps (21 each) over the adapters before.
    const int each = (bins + kWindow - 1) / kWindow;
    auto amount = [&](int b) {
        const unsigned rows = (unsigned)total[b];
        return (unsigned long long)((rows + kTcStepRows - 1) / kTcStepRows) << 42 |
               (unsigned long long)((rows + a.tile_rows - 1) / a.tile_rows) << 21 | rows;
    };
    constexpr unsigned kField = (1u << 21) - 1;
    unsigned long long sum = 0;
    for (int b = tid * each; b < (tid + 1) * each && b < bins; ++b) sum += amount(b);
    unsigned long long scan = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        unsigned long long v = warp_sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        warp_sums[lane] = v;
    }
    __syncthreads();
    unsigned long long run = scan - sum + (warp ? warp_sums[warp - 1] : 0ull);
    for (int b = tid * each; b < (tid + 1) * each && b < bins; ++b) {
        base[b] = (int)((unsigned)run & kField);
        tile_base[b] = (int)((unsigned)(run >> 21) & kField);
        step_base[b] = (int)(run >> 42);
        if (blockIdx.x == 0) a.starts[b] = base[b];
        if (blockIdx.x == 0 && a.steps) a.step_starts[b] = step_base[b];
        run += amount(b);
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[bins] = a.m;
        *a.tile_count = (int)((unsigned)(warp_sums[31] >> 21) & kField);
    }
    __syncthreads();
    if (!here) return;
    const int rank = before[mine] + local, at = base[mine] + rank;
    a.order[at] = row;
    if (rank % a.tile_rows == 0) {
        const int left = total[mine] - rank;
        a.tiles[tile_base[mine] + rank / a.tile_rows] = AdapterTile{mine, at, left < a.tile_rows ? left : a.tile_rows, 0};
    }
    if (a.steps && rank % kTcStepRows == 0 && mine < a.adapters) {
        const int left = total[mine] - rank;
        a.steps[step_base[mine] + rank / kTcStepRows] = AdapterTile{mine, at, left < kTcStepRows ? left : kTcStepRows, 0};
    }
}

cudaError_t order_launch(const OrderArgs &a, cudaStream_t stream)
{
    const int smem = 6 * 4 * (a.adapters + 1) + (a.adapters < kFewBins ? 32 * kFewBins * 4 : 0);
    static bool allowed[kMaxDevices] = {};
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_dynamic_smem(adapter_order_kernel, 6 * 4 * (kMostAdapters + 1), allowed);
        if (e != cudaSuccess) return e;
    }
    return launch_overlapped(adapter_order_kernel, dim3((unsigned)((a.m + kWindow - 1) / kWindow)), dim3(kWindow), smem, stream, 1, a);
}

// ------------------------------------------------------------------ the weights' gradients, joined
// Adapters whose rows reach over several chunks: the partial sums of the first (its second row), then of the others
// (their first rows), in order.  Those without rows get zeros.
__global__ void __launch_bounds__(kAdapterThreads) adapter_join_kernel(const AdapterGradArgs a)
{
    dev::grid_dependency_wait();
    dev::grid_dependents_launch();
    const long long of_a = (long long)a.rank * a.k, all = of_a + (long long)a.rank * a.n;
    for (int adapter = blockIdx.y; adapter < a.adapters; adapter += gridDim.y) {
        const int first = a.starts[adapter], last = a.starts[adapter + 1];
        const int c0 = first / a.chunk_rows, c1 = (last - 1) / a.chunk_rows;
        if (first < last && c0 == c1) continue;
        for (long long i = (long long)blockIdx.x * kAdapterThreads + threadIdx.x; i < all; i += (long long)gridDim.x * kAdapterThreads) {
            float v = 0.0f;
            if (first < last) {
                v = a.partial[(2LL * c0 + 1) * all + i];
                // Eight loads at once, added in their order.
                for (int c = c0 + 1; c <= c1; c += 8) {
                    float u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] = c + j <= c1 ? a.partial[2LL * (c + j) * all + i] : 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) v += u[j];
                }
            }
            if (i < of_a)
                a.da[adapter * of_a + i] = v;
            else
                a.db[adapter * (all - of_a) + i - of_a] = v;
        }
    }
}

// ------------------------------------------------------------------ what a call launches
struct Layout {
    bool few;      // each cluster finds its rows itself
    bool counted;  // by counting all of them
    bool many;     // tiles of kAdapterManyRows
    int tile_rows, tiles;  // tiles at most
    int clusters, size;
};

// Rows that one call of adapter_products_kernel's clusters looks at by itself.
constexpr int kFew = kAdapterThreads;

// Rows whose tiles a CTA finds by counting all of them: an order by adapter first takes a launch more (777x1001x515 f32
// 11.9 / 9.5 us), and a cluster for each row more clusters than there are tiles, which counts where there are four times
// as many (4096x4096, rank 16, 256 rows of 4 adapters 9.6 / 8.1 us, of 64 adapters 10.5 / 12.3).  From 820 rows of rank 64
// and 456 of 128 on neither is the faster throughout, and rows are ordered (ordered / counted: rank 128, 1000 rows of 4
// adapters 33.8 / 31.5 us, of 64 97 / 106).
bool counted(const AdapterProblem &p)
{
    return p.m <= kCountedRows && p.adapters < kCountedBins && (long long)p.m * (adapter_rank_tiles(p.rank) + 1) < 4096 &&
           (p.m > kFew || (p.m > 64 && 4 * (p.m / kAdapterFewRows + p.adapters) < p.m));
}

Layout layout_of(const AdapterProblem &p, bool ordered, int k, int n, int sm_count)
{
    Layout l{};
    l.counted = !ordered && counted(p);
    l.few = l.counted || (!ordered && p.m <= kFew);
    // Tiles of 128 rows read an adapter's weights an eighth as often, which pays once the tiles of 16 come to several an SM,
    // the later the fewer ranks they multiply with (bf16, 4096x4096 of 4 adapters, 16 / 128 rows a tile: rank 16 with 1600
    // rows 17.3 / 20.5 us, with 1800 28.7 / 22.2; rank 32 with 1100 17.5 / 23.8, with 1366 32.4 / 23.6; rank 64 22.4 / 32.4 and
    // 43.4 / 32.4; rank 128 34.4 / 48.8 and 86.5 / 48.8); where an adapter has few rows, on average over all there are,
    // most of such a tile's warps would have none.
    l.many = p.m >= (adapter_rank_tiles(p.rank) == 1 ? 1700 : 1200) && p.m >= 24LL * p.adapters;
    l.tile_rows = l.many ? kAdapterManyRows : kAdapterFewRows;
    const int full = (p.m + l.tile_rows - 1) / l.tile_rows;
    l.tiles = full + (p.adapters + 1 < p.m ? p.adapters + 1 : p.m);
    l.clusters = l.few && !l.counted ? p.m : l.tiles;
    // CTAs a tile, while each has some steps of 32 elements for its warps: of few rows, what takes the fewest rounds of
    // CTAs for its part of a tile (128 rows of 64 adapters, 4096x4096: 4 CTAs 9.8 us, 8 12.8; one row: 4 CTAs 7.3, 8 6.1);
    // of many, what leaves the fullest SM, busy from so many CTAs on, the least (1 / 2 / 4 / 8 CTAs: 8192x4096x16384 of rank 64
    // 311 / 170 / 156 / 193 us, 8192x4096x4096 of rank 16 76 / 51 / 46 / 57; it misses by a tenth where little is left to
    // share: 32768x64x4096 121 / 114 / 127 / 167).  The fewest of those that do.
    const int ranks = adapter_rank_tiles(p.rank);
    const long long resident = l.many ? (ranks <= 4 && p.dtype != kF32 ? 2 : 1) : ranks == 1 ? 3 : ranks == 2 || (ranks == 4 && p.dtype != kF32) ? 2 : 1;
    const long long about = full + (l.many ? 0 : p.adapters < p.m ? p.adapters : p.m);  // tiles
    auto rounds_of = [&](int size) {
        const long long per_sm = (about * size + sm_count - 1) / sm_count;
        return l.many ? (per_sm > resident ? per_sm : resident) : (about * size + resident * sm_count - 1) / (resident * sm_count);
    };
    const int steps = ((k > n ? k : n) + 31) / 32;
    l.size = 1;
    for (int size = 2; size <= 8 && steps >= 8 * size; size *= 2)
        if (rounds_of(size) * l.size < rounds_of(l.size) * size) l.size = size;
    return l;
}

constexpr long long up16(long long v) { return (v + 15) / 16 * 16; }

struct Workspace {
    long long starts, order, tiles, step_starts, steps, operands, dhidden, partial, bytes;
    int chunks, chunk_rows, most_steps;
};

// Chunks of `units` rows or steps for the weights' gradients: so many CTAs in all, `least` units each at least, and `most`
// at most, which also keeps the runs of additions in the matrix instruction's accumulators short.
void chunks_of(const AdapterProblem &p, int columns, int ctas, long long units, int least, int most, int *chunks, int *chunk_units)
{
    const long long strips = (p.k + columns - 1) / columns + (p.n + columns - 1) / columns;
    long long c = (ctas + strips - 1) / strips;
    if (c > (units + least - 1) / least) c = (units + least - 1) / least;
    if (c < (units + most - 1) / most) c = (units + most - 1) / most;
    if (c < 1) c = 1;
    *chunk_units = (int)((units + c - 1) / c);
    *chunks = (int)((units + *chunk_units - 1) / *chunk_units);
}

// Sizes that adapter_tc_weights_kernel takes, if type and boundaries allow it: where an adapter has few rows on average,
// most of a step's 64 would be none.
bool tc_sizes(const AdapterProblem &p)
{
    return p.k % 8 == 0 && p.n % 8 == 0 && adapter_rank_tiles(p.rank) <= 4 && p.m >= 1024 && p.m >= 128LL * p.adapters;
}

// `tc`: with the chunks of adapter_tc_weights_kernel; the bytes are enough for any kernel that the sizes allow.
Workspace workspace_of(const AdapterProblem &p, bool gradient, bool tc, int sm_count)
{
    Workspace w{};
    const long long rows = p.m;
    w.starts = 16;
    w.order = w.starts + up16(4LL * (p.adapters + 2));
    w.tiles = w.order + up16(4 * rows);
    w.step_starts = w.tiles + 16LL * ((rows + kAdapterFewRows - 1) / kAdapterFewRows + p.adapters + 1);
    w.bytes = w.step_starts;
    if (gradient && rows > 0) {
        int chunks[2], chunk_rows[2];
        w.most_steps = (int)(rows / kTcStepRows + (p.adapters < rows ? p.adapters : rows));
        // A step of 16 rows at least, or as many as an adapter has on average, since a CTA takes one adapter after the other.
        // (bf16, rank 12 to 16, k and n 4096, least 4 rows / 16 / that many: 18 rows of 64 adapters 89 / 114 / 61 us, 200 of 64
        // 116 / 159 / 114, 64 of 8 42 / 36 / 38; f32, 160 of 8 49 / 38 / 38, 200 of 32 81 / 72 / 81.)
        const long long each = (rows + p.adapters - 1) / p.adapters;
        chunks_of(p, adapter_columns(p.rank), 3 * sm_count, rows, each < 16 ? (int)each : 16, kAdapterChunkRows, &chunks[0], &chunk_rows[0]);
        const bool steps = tc_sizes(p);
        chunks[1] = chunk_rows[1] = 0;
        if (steps) chunks_of(p, 128, 2 * sm_count, w.most_steps, 1, kTcChunkSteps, &chunks[1], &chunk_rows[1]);
        w.chunks = chunks[tc];
        w.chunk_rows = chunk_rows[tc];
        w.steps = w.step_starts + up16(4LL * (p.adapters + 1));
        w.operands = (w.steps + (steps ? 16LL * w.most_steps : 0) + 127) / 128 * 128;
        w.dhidden = w.operands + (steps ? 2LL * w.most_steps * adapter_tc_operand(p.rank) : 0);
        w.partial = w.dhidden + up16(4 * rows * p.rank);
        w.bytes = w.partial + 8LL * (chunks[0] > chunks[1] ? chunks[0] : chunks[1]) * p.rank * ((long long)p.k + p.n);
    }
    return w;
}

bool on_boundary(const void *p, long long stride, int element)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * element % 16 == 0;
}

cudaError_t products(const AdapterArgs &a, int dtype, bool transposed, const Layout &l, cudaStream_t stream)
{
    switch (dtype) {
    case kF32: return adapter_products_launch<float>(a, transposed, l.many, l.clusters, l.size, stream);
    case kBf16: return adapter_products_launch<__nv_bfloat16>(a, transposed, l.many, l.clusters, l.size, stream);
    default: return adapter_products_launch<__half>(a, transposed, l.many, l.clusters, l.size, stream);
    }
}

OrderArgs order_args(const AdapterProblem &p, const Workspace &w, const Layout &l, char *work)
{
    OrderArgs o{};
    o.index = p.index;
    o.tile_count = reinterpret_cast<int *>(work);
    o.starts = reinterpret_cast<int *>(work + w.starts);
    o.order = reinterpret_cast<int *>(work + w.order);
    o.tiles = reinterpret_cast<AdapterTile *>(work + w.tiles);
    o.m = p.m;
    o.adapters = p.adapters;
    o.tile_rows = l.tile_rows;
    return o;
}

}  // namespace

long long adapters_workspace_bytes(const AdapterProblem &p, bool gradient, int sm_count)
{
    if (!gradient && (p.m <= kFew || counted(p))) return 0;
    return workspace_of(p, gradient, false, sm_count).bytes;
}

cudaError_t adapters_launch(const AdapterProblem &p, int sm_count, cudaStream_t stream)
{
    const int size = dtype_size(p.dtype);
    const Layout l = layout_of(p, false, p.k, p.n, sm_count);
    AdapterArgs a{};
    a.x = p.x.data;
    a.x_stride = p.x.stride;
    a.base = p.base.data;
    a.base_stride = p.base.stride;
    a.y = p.y.data;
    a.y_stride = p.y.stride;
    a.hidden = p.hidden_out;
    a.w1 = p.a;
    a.w2 = p.b;
    a.scale = p.scale;
    a.index = p.index;
    a.m = p.m;
    a.k = p.k;
    a.n = p.n;
    a.rank = p.rank;
    a.adapters = p.adapters;
    a.x_wide = p.k % 8 == 0 && on_boundary(p.x.data, p.x.stride, size);
    a.w1_wide = p.k % 8 == 0 && on_boundary(p.a, 0, size);
    // Ranks that a lane loads at once in the second product.
    const int near = l.many && size == 2 && adapter_rank_tiles(p.rank) > 1 ? 8 : 4;
    a.w2_wide = p.rank % near == 0 && on_boundary(p.b, 0, size);
    a.w1_pieces = p.k * size % 16 == 0 && on_boundary(p.a, 0, size);
    a.y_wide = p.n % 8 == 0 && on_boundary(p.y.data, p.y.stride, size) && on_boundary(p.base.data, p.base.stride, size);
    a.counted = l.counted;
    if (!l.few) {
        const Workspace w = workspace_of(p, false, false, sm_count);
        const OrderArgs o = order_args(p, w, l, static_cast<char *>(p.workspace));
        const cudaError_t e = order_launch(o, stream);
        if (e != cudaSuccess) return e;
        a.order = o.order;
        a.tiles = o.tiles;
        a.tile_count = o.tile_count;
    }
    return products(a, p.dtype, false, l, stream);
}

cudaError_t adapters_grad_launch(const AdapterProblem &p, int sm_count, cudaStream_t stream)
{
    const int size = dtype_size(p.dtype);
    const Layout l = layout_of(p, true, p.n, p.k, sm_count);
    const bool x_wide = p.k % 8 == 0 && on_boundary(p.x.data, p.x.stride, size), dy_wide = p.n % 8 == 0 && on_boundary(p.dy.data, p.dy.stride, size);
    // A tensor map's rows are less than 2^40 bytes apart.
    const bool tc = p.dtype == kBf16 && tc_sizes(p) && x_wide && dy_wide && p.x.stride >= p.k && p.dy.stride >= p.n &&
                    p.x.stride < (1LL << 39) && p.dy.stride < (1LL << 39);
    const Workspace w = workspace_of(p, true, tc, sm_count);
    char *work = static_cast<char *>(p.workspace);
    OrderArgs o = order_args(p, w, l, work);
    if (tc) {
        o.steps = reinterpret_cast<AdapterTile *>(work + w.steps);
        o.step_starts = reinterpret_cast<int *>(work + w.step_starts);
    }
    cudaError_t e = order_launch(o, stream);
    if (e != cudaSuccess) return e;
    // dhidden and dx: the two products with dy, B and A.
    float *dhidden = reinterpret_cast<float *>(work + w.dhidden);
    AdapterArgs a{};
    a.x = p.dy.data;
    a.x_stride = p.dy.stride;
    a.base = p.base.data;
    a.base_stride = p.base.stride;
    a.y = p.y.data;
    a.y_stride = p.y.stride;
    a.hidden = dhidden;
    a.w1 = p.b;
    a.w2 = p.a;
    a.scale = p.scale;
    a.index = p.index;
    a.order = o.order;
    a.tiles = o.tiles;
    a.tile_count = o.tile_count;
    a.m = p.m;
    a.k = p.n;
    a.n = p.k;
    a.rank = p.rank;
    a.adapters = p.adapters;
    const int near = adapter_rank_tiles(p.rank) < 4 ? 2 * adapter_rank_tiles(p.rank) : 8;  // ranks a lane loads at once
    a.x_wide = p.n % 8 == 0 && on_boundary(p.dy.data, p.dy.stride, size);
    a.w1_wide = p.rank % near == 0 && on_boundary(p.b, 0, size);
    a.w2_wide = p.k % (l.many ? 8 : 4) == 0 && on_boundary(p.a, 0, size);
    a.w1_pieces = p.rank * size % 16 == 0 && on_boundary(p.b, 0, size);
    a.y_wide = p.k % 8 == 0 && on_boundary(p.y.data, p.y.stride, size) && on_boundary(p.base.data, p.base.stride, size);
    e = products(a, p.dtype, true, l, stream);
    if (e != cudaSuccess) return e;
    AdapterGradArgs g{};
    g.x = p.x.data;
    g.x_stride = p.x.stride;
    g.dy = p.dy.data;
    g.dy_stride = p.dy.stride;
    g.hidden = p.hidden;
    g.dhidden = dhidden;
    g.scale = p.scale;
    g.order = o.order;
    g.starts = o.starts;
    g.steps = o.steps;
    g.step_starts = o.step_starts;
    g.operands = reinterpret_cast<uint4 *>(work + w.operands);
    g.most_steps = w.most_steps;
    g.da = p.da;
    g.db = p.db;
    g.partial = reinterpret_cast<float *>(work + w.partial);
    g.rows = p.m;
    g.k = p.k;
    g.n = p.n;
    g.rank = p.rank;
    g.adapters = p.adapters;
    g.chunks = w.chunks;
    g.chunk_rows = w.chunk_rows;
    g.x_wide = x_wide;
    g.dy_wide = dy_wide;
    if (tc) e = adapter_tc_weights_launch(g, stream);
    else switch (p.dtype) {
    case kF32: e = adapter_weights_launch<float>(g, stream); break;
    case kBf16: e = adapter_weights_launch<__nv_bfloat16>(g, stream); break;
    default: e = adapter_weights_launch<__half>(g, stream); break;
    }
    if (e != cudaSuccess) return e;
    if (tc) g.starts = g.step_starts;
    const long long blocks = ((long long)p.rank * ((long long)p.k + p.n) + kAdapterThreads - 1) / kAdapterThreads;
    return launch_overlapped(adapter_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096), (unsigned)p.adapters),
                             dim3(kAdapterThreads), 0, stream, 1, g);
}

}  // namespace cbs
