// adapters.h -- what the translation units of the low-rank adapters share (adapters.cu has the formulas).
// Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "token_ops.h"

namespace cbs {

// Rows of one adapter that a group of CTAs takes: `count` positions from `first` on in the order by adapter.
struct AdapterTile {
    int adapter, first, count, unused;
};

// Two products after one another for each row, y = base + s (x W1) W2, W1 and W2 those of the row's adapter: forward
// with x, A and B, and for the gradient of x with dy, B and A, whose memory is then the transposed one.
struct AdapterArgs {
    const void *x, *base;
    void *y;
    float *hidden;          // nullable [m][rank]: x W1
    const void *w1, *w2;
    const float *scale;     // nullable [adapters]
    const int *index;       // [m]
    const int *order;       // nullable: rows by adapter, with tiles and tile_count
    const AdapterTile *tiles;
    const int *tile_count;
    long long x_stride, base_stride, y_stride;
    int m, k, n, rank, adapters;
    bool counted;           // without an order: tiles found by counting, else by their first rows
    bool x_wide, w1_wide, w2_wide, y_wide;  // rows on the boundaries of wide loads and stores, and as long as they are
    bool w1_pieces;                         // the first weights' rows in whole pieces of 16 bytes
};

// Gradients of the adapters' weights: sums over the rows of each adapter.
struct AdapterGradArgs {
    const void *x, *dy;
    const float *hidden, *dhidden;  // [m][rank]
    const float *scale;             // nullable
    const int *order, *starts;      // starts [adapters + 2]: where each adapter's rows begin in the order
    // adapter_tc_weights_kernel: steps of 64 rows of one adapter, where each adapter's begin, and the steps' second
    // operands [2][most_steps], hidden's and dhidden's.  The join's starts are then step_starts, its chunks of steps.
    const AdapterTile *steps;
    const int *step_starts;
    uint4 *operands;
    int most_steps;
    float *da, *db;                 // [adapters][rank][k], [adapters][n][rank]
    float *partial;                 // [2 * chunks][rank * (k + n)]
    long long x_stride, dy_stride;
    int rows, k, n, rank, adapters;
    int chunks, chunk_rows;
    bool x_wide, dy_wide;
};

constexpr int kAdapterThreads = 256;
constexpr int kCountedRows = 4 * kAdapterThreads, kCountedBins = 96;  // of tiles found by counting: rows, adapters and one
constexpr int kAdapterFewRows = 16, kAdapterManyRows = 128;  // of a tile
constexpr int kAdapterColumns = 512;                        // of a weight gradient's CTA, half for ranks above 32
constexpr int kAdapterChunkRows = 1024;                     // of its chunk at most

constexpr int kTcStepRows = 64, kTcChunkSteps = 16;          // of adapter_tc_weights_kernel's steps and chunks
// Bytes of a step's second operand: three parts of each rank, 64 rows.
inline long long adapter_tc_operand(int rank) { return 3LL * 16 * (rank <= 16 ? 1 : rank <= 32 ? 2 : 4) * 128; }

inline int adapter_rank_tiles(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }
inline int adapter_columns(int rank) { return rank <= 32 ? kAdapterColumns : kAdapterColumns / 2; }

// By element type (adapters_*.cu).  `many`: tiles of 128 rows, else of 16.
template <typename T>
cudaError_t adapter_products_launch(const AdapterArgs &a, bool transposed, bool many, int clusters, int cluster_size,
                                    cudaStream_t stream);
template <typename T>
cudaError_t adapter_weights_launch(const AdapterGradArgs &a, cudaStream_t stream);

// On the tensor cores' own memory (tc_adapters.cu): bf16, wide rows at least their width apart, ranks up to 64.
cudaError_t adapter_tc_weights_launch(const AdapterGradArgs &a, cudaStream_t stream);

}  // namespace cbs
