// token_ops.h -- host-side types of the token-wise operators, shared by the C
// ABI (capi.cu) and their translation units.  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace cbs {

// Element types of activations (the values of cbs_dtype).
enum DType : int { kF32 = 0, kBf16 = 1, kF16 = 2 };

inline int dtype_size(int t) { return t == kF32 ? 4 : 2; }

// Rows of one matrix: element (r, c) is at data[r * stride + c].
struct Rows {
    void *data;
    long long stride;  // in elements
};

struct NormProblem {
    Rows x;              // input, `dtype`
    Rows y;              // normalised output, `dtype` (q.data == nullptr)
    Rows q;              // int8 output instead of y, with row_scale
    float *row_scale;    // [rows], with q only
    float *stats;        // nullable [2][rows]: mean, then 1/sqrt(var + eps)
    const float *gamma;  // nullable [c]
    const float *beta;   // nullable [c]
    float eps;
    int normalise;       // 0: quantise x itself (q only)
    long long rows;
    int c;
    int dtype;
};

struct NormGradProblem {
    Rows dy, x, dx;      // `dtype`
    const float *gamma;  // nullable [c]
    const float *stats;  // [2][rows]
    float *dgamma;       // [c]
    float *dbeta;        // [c]
    float *partial;      // workspace: [partial_rows][2][c]
    int partial_rows;    // from norm_grad_partial_rows
    long long rows;
    int c;
    int dtype;
};

struct RmsNormProblem {
    Rows x;              // input, `dtype`
    Rows residual;       // nullable, added to x
    Rows total;          // their sum, with residual only; may be residual itself
    Rows y;              // normalised output, `dtype`; nullable with q
    Rows q;              // nullable int8 output, with row_scale
    float *row_scale;    // [rows], with q only
    float *rstd;         // nullable [rows]: 1/sqrt(mean square + eps)
    const float *gamma;  // nullable [c]
    float eps;
    long long rows;
    int c;
    int dtype;
};

struct RmsNormGradProblem {
    Rows dy, x, dx;      // `dtype`; x is what was normalised
    Rows residual;       // nullable, added to dx; may be dx itself
    const float *gamma;  // nullable [c]
    const float *rstd;   // [rows]
    float *dgamma;       // [c]
    float *partial;      // workspace: [partial_rows][c]
    int partial_rows;    // from rms_grad_partial_rows
    long long rows;
    int c;
    int dtype;
};

// Low-rank adapters and their gradients.
struct AdapterProblem {
    Rows x;             // `dtype` [m][k]
    Rows base;          // nullable [m][n], or for the gradient [m][k]; may be y itself
    Rows y;             // [m][n]; for the gradient dx [m][k]
    Rows dy;            // gradient only: [m][n]
    const int *index;   // [m]
    const void *a, *b;  // `dtype` [adapters][rank][k], [adapters][n][rank]
    const float *scale; // nullable [adapters]
    float *hidden_out;  // nullable [m][rank], forward only
    const float *hidden;// gradient only
    float *da, *db;     // gradient only: as a and b
    int m, k, n, rank, adapters;
    int dtype;
    void *workspace;    // adapters_workspace_bytes
};
constexpr int kMostAdapters = 4096, kMostRank = 128, kMostAdapterRows = 1 << 20;

// One tensor of an AdamW step: fp32 moments, or e4m3 ones (v's square root) with a scale for each 256 elements.
struct AdamWTensor {
    void *p;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    long long n;
    int p_type, g_type;  // DType
};

// The step's numbers; those with an address are read there, on the device.
struct AdamWScalars {
    const float *lr_at, *grad_scale_at;
    const long long *step_at;
    float lr, grad_scale;
    float beta1, beta2, rest1, rest2;  // rest: 1 - beta
    float ln_beta1, ln_beta2;
    float c1, root_c2;                 // 1 - beta1^step, sqrt(1 - beta2^step)
    float eps, decay;
    long long step;
};

struct LinearProblem {
    Rows a;                // int8 [m][k]
    Rows w;                // int8 [n][k]
    Rows residual;         // nullable `out_dtype` [m][n]
    Rows y;                // `out_dtype` [m][n]
    const float *a_scale;  // [m]
    const float *w_scale;  // [n]
    const float *bias;     // nullable [n]
    long long m;
    int n, k;
    int out_dtype;
    int activation;        // cbs_activation
    void *workspace;       // linear_workspace_bytes
};

// Shared memory above 48 KB, allowed once per kernel and device; `done` is the kernel's own record.
constexpr int kMaxDevices = 64;
template <typename Kernel>
cudaError_t allow_dynamic_smem(Kernel kernel, int bytes, bool (&done)[kMaxDevices])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && __atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < kMaxDevices) __atomic_store_n(&done[dev], true, __ATOMIC_RELEASE);
    return e;
}

// A kernel translation unit's error word: read and cleared in stream order.
template <typename Symbol>
cudaError_t read_and_clear_word(const Symbol &word, cudaStream_t stream, unsigned int *out)
{
    unsigned int host = 0;
    cudaError_t st = cudaMemcpyFromSymbolAsync(&host, word, sizeof host, 0, cudaMemcpyDeviceToHost, stream);
    if (st == cudaSuccess) st = cudaStreamSynchronize(stream);
    if (st == cudaSuccess && host != 0) {
        const unsigned int zero = 0;
        st = cudaMemcpyToSymbolAsync(word, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
        if (st == cudaSuccess) st = cudaStreamSynchronize(stream);
    }
    *out = host;
    return st;
}

cudaError_t norm_launch(const NormProblem &p, int sm_count, cudaStream_t stream);
int norm_grad_partial_rows(long long rows, int sm_count);  // of partial sums, each [2][c]
cudaError_t norm_grad_launch(const NormGradProblem &p, int sm_count, cudaStream_t stream);

cudaError_t rms_norm_launch(const RmsNormProblem &p, int sm_count, cudaStream_t stream);
int rms_grad_partial_rows(long long rows, int sm_count);  // of partial sums, each [c]
cudaError_t rms_norm_grad_launch(const RmsNormGradProblem &p, int sm_count, cudaStream_t stream);

long long adapters_workspace_bytes(const AdapterProblem &p, bool gradient, int sm_count);
cudaError_t adapters_launch(const AdapterProblem &p, int sm_count, cudaStream_t stream);
cudaError_t adapters_read_and_clear_error(cudaStream_t stream, unsigned int *out);
cudaError_t adapters_grad_launch(const AdapterProblem &p, int sm_count, cudaStream_t stream);

constexpr int kAdamWBlock = 256;  // elements that share a scale
cudaError_t adamw_launch(const AdamWTensor *tensors, int count, const AdamWScalars &s, bool eight, cudaStream_t stream);

// What linear_launch runs (the fields of cbs_linear_plan but for the workspace).
struct LinearPlan {
    int kernel;  // cbs_linear_kernel
    int turned;
    int tile_rows, tile_channels;
    int align;
    int k_steps, tiles, workers;
};
LinearPlan linear_plan(long long m, int n, int k, int align, int sm_count);

// Bytes linear_launch may need for these sizes, whatever the pointers and strides.
long long linear_workspace_bytes(long long m, int n, int k, int sm_count);
cudaError_t linear_launch(const LinearProblem &p, int sm_count, cudaStream_t stream);

// The linear layer on the tensor cores (tc_linear.cu); k == 0 counts as a step of zeros.
long long tc_linear_workspace_bytes(long long m, int n, int k);
float tc_linear_time(long long m, int n, int k, int sm_count);  // modelled, us
void tc_linear_plan(long long m, int n, int k, int sm_count, LinearPlan *plan);
cudaError_t tc_linear_launch(const LinearProblem &p, int sm_count, cudaStream_t stream);
cudaError_t tc_linear_read_and_clear_error(cudaStream_t stream, unsigned int *out);

// Bytes [rows][k] at a distance of `stride` (all multiples of 16 but k) in boxes of box_rows rows of box_k bytes,
// 128-byte swizzled; zeros past the ends.
cudaError_t encode_bytes_map(const void *base, long long rows, int k, long long stride, int box_rows, int box_k,
                             CUtensorMap *out);

// The linear layer with the weights widened on their way to the tensor cores, and turned, with its rows in the
// weights' place (tc_linear_stream.cu): rows and channels are then n and m.
int tc_stream_align(const LinearProblem &p);  // 16, 4 or 1: all rows start at multiples of it, and k is one; 0: k is 0
long long tc_stream_workspace_bytes(long long rows, int channels, int k, int sm_count);
float tc_stream_time(long long rows, int channels, int k, int align, bool turned, int sm_count);  // modelled, us
void tc_stream_plan(long long rows, int channels, int k, int align, bool turned, int sm_count, LinearPlan *plan);
cudaError_t tc_stream_launch(const LinearProblem &p, bool turned, int sm_count, cudaStream_t stream);
cudaError_t tc_stream_read_and_clear_error(cudaStream_t stream, unsigned int *out);

// The linear layer in one launch, for small products (linear_tile.cu).
float linear_tile_time(long long m, int n, int k, int sm_count);  // modelled, us
bool linear_tile_supported(long long m, int n);
void linear_tile_plan(long long m, int n, int k, LinearPlan *plan);
cudaError_t linear_tile_launch(const LinearProblem &p, cudaStream_t stream);

// What any of the linear layer's kernels recorded.
cudaError_t linear_read_and_clear_error(cudaStream_t stream, unsigned int *out);

}  // namespace cbs
