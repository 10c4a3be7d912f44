// capi.cu -- the extern "C" boundary declared in include/conv_bn_silu.h:
// argument validation, output sizes, kernel choice and launch, error words.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <vector>

#include "conv_bn_silu.h"
#include "cbs_internal.h"
#include "token_ops.h"

namespace {

thread_local int t_last_cuda_error = 0;

int cuda_fail(cudaError_t e)
{
    t_last_cuda_error = (int)e;
    return CBS_ERR_CUDA;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int dims_from(int h, int w_in, int r, int s, int sh, int sw, int ph, int pw, int *ho, int *wo)
{
    if (h < 1 || w_in < 1 || r < 1 || s < 1 || sh < 1 || sw < 1 || ph < 0 || pw < 0)
        return CBS_ERR_INVALID_ARG;
    const long long hp = (long long)h + 2LL * ph, wp = (long long)w_in + 2LL * pw;
    if (hp < r || wp < s) return CBS_ERR_INVALID_ARG;
    const long long oh = (hp - r) / sh + 1, ow = (wp - s) / sw + 1;
    if (oh < 1 || ow < 1 || oh > 0x7fffffffLL || ow > 0x7fffffffLL) return CBS_ERR_INVALID_ARG;
    *ho = (int)oh;
    *wo = (int)ow;
    return CBS_OK;
}

// Shape checks shared by forward and plan.  Fills everything but the pointers.
int make_problem(int n, int h, int w_in, int c, int c_out, int r, int s, int sh, int sw, int ph, int pw,
                 cbs::ConvProblem *p)
{
    if (n < 0 || c < 1 || c_out < 0) return CBS_ERR_INVALID_ARG;
    int ho = 0, wo = 0;
    const int st = dims_from(h, w_in, r, s, sh, sw, ph, pw, &ho, &wo);
    if (st != CBS_OK) return st;
    p->n = n;
    p->h = h;
    p->w_in = w_in;
    p->c = c;
    p->c_out = c_out;
    p->r = r;
    p->s = s;
    p->stride_h = sh;
    p->stride_w = sw;
    p->pad_h = ph;
    p->pad_w = pw;
    p->ho = ho;
    p->wo = wo;
    p->m = (long long)n * ho * wo;
    // Keep every tensor's element count within 2^62 so byte offsets never overflow.
    const long long xe = (long long)n * h * w_in;
    if (xe > (1LL << 40) / (c > 0 ? c : 1) || p->m > (1LL << 40) / (c_out > 0 ? c_out : 1) ||
        (long long)r * s * c > (1LL << 31) - 1)
        return CBS_ERR_INVALID_ARG;
    return CBS_OK;
}

int select_algo(const cbs::ConvProblem &p, int algo)
{
    if (algo != CBS_ALGO_AUTO) return algo;
    return cbs::tc_supported(p) || cbs::gather_supported(p) ? CBS_ALGO_TCGEN05 : CBS_ALGO_DIRECT;
}

int sm_count_current_device(int *count)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    static std::mutex mu;
    static std::vector<int> cache;
    {
        std::lock_guard<std::mutex> lock(mu);
        if ((int)cache.size() > dev && cache[dev] > 0) {
            *count = cache[dev];
            return CBS_OK;
        }
    }
    int v = 0;
    e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e);
    std::lock_guard<std::mutex> lock(mu);
    if ((int)cache.size() <= dev) cache.resize(dev + 1, 0);
    cache[dev] = v;
    *count = v;
    return CBS_OK;
}

// A request's tcgen05 overrides, or nullptr when it leaves every choice to the planner.
bool has_overrides(const cbs::PlanRequest *rq)
{
    return rq && (rq->swap_ab >= 0 || rq->stream_k >= 0 || rq->pair >= 0 || rq->block_n != 0 ||
                  rq->balanced >= 0 || rq->wres >= 0 || rq->row_boxes >= 0);
}

// Validated problem (pointers set) -> the chosen kernel's launch on `strm`.
int launch_forward(const cbs::ConvProblem &p, int algo, cudaStream_t strm, const cbs::PlanRequest *rq = nullptr)
{
    const int chosen = select_algo(p, algo);
    if (chosen == CBS_ALGO_TCGEN05) {
        if (!cbs::tc_supported(p) && !cbs::gather_supported(p)) return CBS_ERR_UNSUPPORTED;
        int sms = 0;
        const int st = sm_count_current_device(&sms);
        if (st != CBS_OK) return st;
        if (!cbs::tc_supported(p)) {
            if (has_overrides(rq)) return CBS_ERR_UNSUPPORTED;  // the thin-input kernel has no such choices
            cudaError_t e = cbs::gather_launch(p, sms, strm);
            return e == cudaSuccess ? CBS_OK : cuda_fail(e);
        }
        cbs::TcPlan plan{};
        if (cbs::tc_make_plan_request(p, sms, rq, &plan) != 0) return CBS_ERR_UNSUPPORTED;
        // A stream-K plan needs the library-held workspace of this (device, stream).
        if (plan.stream_k && !cbs::tc_workspace_reserve(strm)) return CBS_ERR_UNSUPPORTED;
        cudaError_t e = cbs::tc_launch(p, plan, strm);
        return e == cudaSuccess ? CBS_OK : cuda_fail(e);
    }
    if (has_overrides(rq)) return CBS_ERR_UNSUPPORTED;
    cudaError_t e = cbs::direct_launch(p, strm);
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

// cbs_plan_request -> checked algorithm and planner overrides.
int read_request(const cbs_plan_request *req, int *algo, cbs::PlanRequest *rq)
{
    if (!req) return CBS_ERR_INVALID_ARG;
    if (req->wait_timeout_ns < 0) return CBS_ERR_INVALID_ARG;
    if (req->algo < CBS_ALGO_AUTO || req->algo > CBS_ALGO_DIRECT) return CBS_ERR_INVALID_ARG;
    for (int v : {req->swap_ab, req->stream_k, req->pair, req->balanced, req->weights_resident, req->row_boxes})
        if (v < -1 || v > 1) return CBS_ERR_INVALID_ARG;
    if (req->block_n != 0 && req->block_n != 16 && req->block_n != 32 && req->block_n != 64 &&
        req->block_n != 128 && req->block_n != 256)
        return CBS_ERR_INVALID_ARG;
    *algo = req->algo;
    *rq = cbs::PlanRequest{req->swap_ab, req->stream_k, req->pair, req->block_n, req->balanced,
                           req->weights_resident, req->row_boxes};
    return CBS_OK;
}

// ------------------------------------------------------------------ allocation-free forward
// Scratch for conv_bn_silu_forward_noalloc: the stream-K partial tiles and ready
// flags live in this fixed device array instead of library-allocated memory.
// It is zero-initialised when the module loads; every GPU that loads the
// library holds it until the process exits.  In host code the symbol is only a
// stand-in: its device address comes from cudaGetSymbolAddress below.
constexpr size_t kNoAllocScratchBytes = 20u << 20;  // 20 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of g_noalloc_scratch on the current device, looked up once per
// device (on that device's first call) and cached.
int noalloc_scratch_address(void **out)
{
    static std::mutex mu;
    static void *addr[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= 64) return CBS_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    if (addr[dev] == nullptr) {
        void *p = nullptr;
        e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
        if (e != cudaSuccess) return cuda_fail(e);
        addr[dev] = p;
    }
    *out = addr[dev];
    return CBS_OK;
}

// ------------------------------------------------------------------ token-wise operators
bool aligned_to(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

// Keeps every byte offset of a matrix within 2^62.
bool rows_in_range(long long rows, long long stride) { return stride <= (1LL << 40) && (rows == 0 || stride <= (1LL << 60) / rows); }

// A matrix argument: pointer, alignment to the element, and a row distance an input may have
// (any from 0) or an output (its width at least; a single row has no distance).
int check_rows(const void *p, long long rows, long long c, long long stride, int element, bool output)
{
    if (stride < 0 || !rows_in_range(rows, stride)) return CBS_ERR_INVALID_ARG;
    if (output && rows > 1 && stride < c) return CBS_ERR_INVALID_ARG;
    if (!p) return CBS_ERR_INVALID_ARG;
    return aligned_to(p, element) ? CBS_OK : CBS_ERR_MISALIGNED;
}

bool norm_sizes_ok(long long rows, int c, int dtype)
{
    // The kernels count columns, up to 2 c of them and a block beyond, in 32-bit integers.
    return rows >= 0 && rows <= (1LL << 40) && c >= 1 && c <= (1 << 29) && dtype >= CBS_DTYPE_F32 && dtype <= CBS_DTYPE_F16;
}

int norm_call(const void *x, long long x_stride, const float *gamma, const float *beta, float eps, void *y,
              long long y_stride, void *q, long long q_stride, float *row_scale, float *stats, int normalise,
              long long rows, int c, int dtype, void *stream)
{
    if (!norm_sizes_ok(rows, c, dtype) || !(eps >= 0.0f) || eps > 3.0e38f) return CBS_ERR_INVALID_ARG;
    if (rows == 0) return CBS_OK;
    const int size = cbs::dtype_size(dtype);
    int st = check_rows(x, rows, c, x_stride, size, false);
    if (st != CBS_OK) return st;
    st = q ? check_rows(q, rows, c, q_stride, 1, true) : check_rows(y, rows, c, y_stride, size, true);
    if (st != CBS_OK) return st;
    if (q && !row_scale) return CBS_ERR_INVALID_ARG;
    if (!aligned_to(gamma, 4) || !aligned_to(beta, 4) || !aligned_to(stats, 4) || !aligned_to(row_scale, 4))
        return CBS_ERR_MISALIGNED;
    cbs::NormProblem p{};
    p.x = cbs::Rows{const_cast<void *>(x), x_stride};
    p.y = cbs::Rows{y, y_stride};
    p.q = cbs::Rows{q, q_stride};
    p.row_scale = row_scale;
    p.stats = stats;
    p.gamma = gamma;
    p.beta = beta;
    p.eps = eps;
    p.normalise = normalise;
    p.rows = rows;
    p.c = c;
    p.dtype = dtype;
    int sms = 0;
    st = sm_count_current_device(&sms);
    if (st != CBS_OK) return st;
    cudaError_t e = cbs::norm_launch(p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

bool linear_sizes_ok(long long m, int n, int k)
{
    // Sums of k products of -128 * -128 fit 32-bit integers; tile counts fit 32 bits.
    return m >= 0 && m < (1LL << 31) && n >= 0 && n <= (1 << 22) && k >= 0 && k <= 131071 &&
           ((m + 127) / 128) * ((n + 63LL) / 64) < (1LL << 30);
}

}  // namespace

extern "C" {

int conv_bn_silu_forward_noalloc(const void *x, const void *w, const float *scale, const float *bias,
                                 void *y, int n, int h, int w_in, int c, int c_out, int r, int s,
                                 int stride_h, int stride_w, int pad_h, int pad_w, void *stream)
{
    cbs::ConvProblem p{};
    int st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    if (p.m == 0 || c_out == 0) return CBS_OK;
    if (!x || !w || !scale || !bias || !y) return CBS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(scale) || !aligned16(bias) || !aligned16(y))
        return CBS_ERR_MISALIGNED;
    p.x = x;
    p.w = w;
    p.scale = scale;
    p.bias = bias;
    p.y = y;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    // Set-up, on the first call on each device: the scratch array's device address.
    void *scratch = nullptr;
    st = noalloc_scratch_address(&scratch);
    if (st != CBS_OK) return st;
    int sms = 0;
    if (!cbs::tc_supported(p)) {  // neither of these kernels needs scratch
        cudaError_t e;
        if (cbs::gather_supported(p)) {
            st = sm_count_current_device(&sms);
            if (st != CBS_OK) return st;
            e = cbs::gather_launch(p, sms, strm);
        } else {
            e = cbs::direct_launch(p, strm);
        }
        return e == cudaSuccess ? CBS_OK : cuda_fail(e);
    }
    st = sm_count_current_device(&sms);
    if (st != CBS_OK) return st;
    cbs::TcPlan plan = cbs::tc_make_plan(p, sms);
    if (plan.stream_k && plan.workspace_bytes > (long long)kNoAllocScratchBytes) {
        // The split would not fit the array (a GPU with many more SMs than GB300's 152):
        // whole tiles per CTA instead, which need no scratch.
        const cbs::PlanRequest whole{-1, 0, 0, 0, -1, -1, -1};
        if (cbs::tc_make_plan_request(p, sms, &whole, &plan) != 0) return CBS_ERR_UNSUPPORTED;
    }
    if (plan.stream_k) {
        // The ready flags must start at zero; a previous call that gave up may have left some set.
        cudaError_t e = cudaMemsetAsync(scratch, 0, (size_t)plan.flag_bytes, strm);
        if (e != cudaSuccess) return cuda_fail(e);
    } else {
        scratch = nullptr;
    }
    cudaError_t e = cbs::tc_launch_with_workspace(p, plan, strm, scratch);
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

int conv_bn_silu_fold(const float *gamma, const float *beta, const float *mean, const float *var,
                      float eps, int c_out, float *scale, float *bias, void *stream)
{
    if (c_out < 0 || !(eps >= 0.0f) || eps > 3.0e38f) return CBS_ERR_INVALID_ARG;
    if (c_out == 0) return CBS_OK;
    if (!gamma || !beta || !mean || !var || !scale || !bias) return CBS_ERR_INVALID_ARG;
    if (!aligned16(gamma) || !aligned16(beta) || !aligned16(mean) || !aligned16(var) ||
        !aligned16(scale) || !aligned16(bias))
        return CBS_ERR_MISALIGNED;
    cudaError_t e = cbs::fold_launch(gamma, beta, mean, var, eps, c_out, scale, bias,
                                     static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

int conv_bn_silu_fold_batch(const cbs_fold_layer *layers, int n_layers, void *stream)
{
    if (n_layers < 0 || (n_layers > 0 && !layers)) return CBS_ERR_INVALID_ARG;
    std::vector<cbs::FoldLayer> v;
    v.reserve((size_t)n_layers);
    for (int i = 0; i < n_layers; ++i) {
        const cbs_fold_layer &L = layers[i];
        if (L.c_out < 0 || !(L.eps >= 0.0f) || L.eps > 3.0e38f) return CBS_ERR_INVALID_ARG;
        if (L.c_out == 0) continue;
        if (!L.gamma || !L.beta || !L.mean || !L.var || !L.scale || !L.bias) return CBS_ERR_INVALID_ARG;
        if (!aligned16(L.gamma) || !aligned16(L.beta) || !aligned16(L.mean) || !aligned16(L.var) ||
            !aligned16(L.scale) || !aligned16(L.bias))
            return CBS_ERR_MISALIGNED;
        v.push_back(cbs::FoldLayer{L.gamma, L.beta, L.mean, L.var, L.eps, L.c_out, L.scale, L.bias});
    }
    if (v.empty()) return CBS_OK;
    cudaError_t e = cbs::fold_batch_launch(v.data(), (int)v.size(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

int conv_bn_silu_forward_algo(const void *x, const void *w, const float *scale, const float *bias,
                              void *y, int n, int h, int w_in, int c, int c_out, int r, int s,
                              int stride_h, int stride_w, int pad_h, int pad_w, int algo, void *stream)
{
    if (algo < CBS_ALGO_AUTO || algo > CBS_ALGO_DIRECT) return CBS_ERR_INVALID_ARG;
    cbs::ConvProblem p{};
    int st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    if (p.m == 0 || c_out == 0) return CBS_OK;
    if (!x || !w || !scale || !bias || !y) return CBS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(scale) || !aligned16(bias) || !aligned16(y))
        return CBS_ERR_MISALIGNED;
    p.x = x;
    p.w = w;
    p.scale = scale;
    p.bias = bias;
    p.y = y;
    return launch_forward(p, algo, static_cast<cudaStream_t>(stream));
}

int conv_bn_act_forward(const void *x, const void *w, const float *scale, const float *bias,
                        const void *residual, void *y, int n, int h, int w_in, int c, int c_out, int r,
                        int s, int stride_h, int stride_w, int pad_h, int pad_w, int activation,
                        void *stream)
{
    int mode;
    switch (activation) {
    case CBS_ACT_SILU: mode = cbs::kEpiSilu; break;
    case CBS_ACT_IDENTITY: mode = cbs::kEpiBn; break;
    case CBS_ACT_RELU: mode = cbs::kEpiRelu; break;
    default: return CBS_ERR_INVALID_ARG;
    }
    cbs::ConvProblem p{};
    int st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    if (p.m == 0 || c_out == 0) return CBS_OK;
    if (!x || !w || !scale || !bias || !y) return CBS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(scale) || !aligned16(bias) || !aligned16(y) ||
        (residual && !aligned16(residual)))
        return CBS_ERR_MISALIGNED;
    p.x = x;
    p.w = w;
    p.scale = scale;
    p.bias = bias;
    p.y = y;
    p.epi_mode = mode;
    p.residual = residual;
    return launch_forward(p, CBS_ALGO_AUTO, static_cast<cudaStream_t>(stream));
}

int conv_bn_act_forward_fp8(const void *x, const void *w, const float *scale, const float *bias, void *y,
                            int n, int h, int w_in, int c, int c_out, int r, int s, int stride_h, int stride_w,
                            int pad_h, int pad_w, int activation, void *stream)
{
    int mode;
    switch (activation) {
    case CBS_ACT_SILU: mode = cbs::kEpiSilu; break;
    case CBS_ACT_IDENTITY: mode = cbs::kEpiBn; break;
    case CBS_ACT_RELU: mode = cbs::kEpiRelu; break;
    default: return CBS_ERR_INVALID_ARG;
    }
    cbs::ConvProblem p{};
    int st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    if (p.m == 0 || c_out == 0) return CBS_OK;
    if (!x || !w || !scale || !bias || !y) return CBS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(scale) || !aligned16(bias) || !aligned16(y))
        return CBS_ERR_MISALIGNED;
    p.x = x;
    p.w = w;
    p.scale = scale;
    p.bias = bias;
    p.y = y;
    p.epi_mode = mode;
    p.out_fp8 = 1;
    return launch_forward(p, CBS_ALGO_AUTO, static_cast<cudaStream_t>(stream));
}

int conv_bn_silu_forward_unfused(const void *x, const void *w, const float *scale, const float *bias,
                                 void *t1, void *t2, void *y, int n, int h, int w_in, int c, int c_out,
                                 int r, int s, int stride_h, int stride_w, int pad_h, int pad_w,
                                 void *stream)
{
    cbs::ConvProblem p{};
    int st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    if (p.m == 0 || c_out == 0) return CBS_OK;
    if (!x || !w || !scale || !bias || !t1 || !t2 || !y) return CBS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(scale) || !aligned16(bias) || !aligned16(t1) ||
        !aligned16(t2) || !aligned16(y))
        return CBS_ERR_MISALIGNED;
    p.x = x;
    p.w = w;
    p.scale = scale;
    p.bias = bias;
    p.y = t1;
    p.epi_mode = cbs::kEpiConvOnly;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    st = launch_forward(p, CBS_ALGO_AUTO, strm);
    if (st != CBS_OK) return st;
    const long long count = p.m * c_out;
    cudaError_t e = cbs::bn_apply_launch(t1, scale, bias, t2, count, c_out, strm);
    if (e != cudaSuccess) return cuda_fail(e);
    e = cbs::silu_apply_launch(t2, y, count, strm);
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

int conv_bn_silu_bn_apply(const void *t1, const float *scale, const float *bias, void *t2,
                          long long count, int c_out, void *stream)
{
    if (count < 0 || c_out < 1 || count % c_out != 0) return CBS_ERR_INVALID_ARG;
    if (count > (1LL << 40)) return CBS_ERR_INVALID_ARG;
    if (count == 0) return CBS_OK;
    if (!t1 || !scale || !bias || !t2) return CBS_ERR_INVALID_ARG;
    if (!aligned16(t1) || !aligned16(scale) || !aligned16(bias) || !aligned16(t2)) return CBS_ERR_MISALIGNED;
    cudaError_t e = cbs::bn_apply_launch(t1, scale, bias, t2, count, c_out, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

int conv_bn_silu_silu_apply(const void *t2, void *y, long long count, void *stream)
{
    if (count < 0 || count > (1LL << 40)) return CBS_ERR_INVALID_ARG;
    if (count == 0) return CBS_OK;
    if (!t2 || !y) return CBS_ERR_INVALID_ARG;
    if (!aligned16(t2) || !aligned16(y)) return CBS_ERR_MISALIGNED;
    cudaError_t e = cbs::silu_apply_launch(t2, y, count, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

int conv_bn_silu_forward(const void *x, const void *w, const float *scale, const float *bias, void *y,
                         int n, int h, int w_in, int c, int c_out, int r, int s, int stride_h,
                         int stride_w, int pad_h, int pad_w, void *stream)
{
    return conv_bn_silu_forward_algo(x, w, scale, bias, y, n, h, w_in, c, c_out, r, s, stride_h,
                                     stride_w, pad_h, pad_w, CBS_ALGO_AUTO, stream);
}

int conv_bn_silu_output_dims(int h, int w_in, int r, int s, int stride_h, int stride_w, int pad_h,
                             int pad_w, int *ho, int *wo)
{
    if (!ho || !wo) return CBS_ERR_INVALID_ARG;
    return dims_from(h, w_in, r, s, stride_h, stride_w, pad_h, pad_w, ho, wo);
}

static int fill_plan(const cbs::ConvProblem &p, int algo, int sm_count, const cbs::PlanRequest *rq,
                     cbs_plan_info *info)
{
    const int n = p.n, c = p.c, c_out = p.c_out, r = p.r, s = p.s;
    (void)n;
    const int chosen = select_algo(p, algo);
    cbs_plan_info out{};
    out.algo = chosen;
    if (chosen == CBS_ALGO_TCGEN05 && !cbs::tc_supported(p)) {
        // Thin-input kernel: 128-pixel tiles, K zero-padded to 32 or 64, each CTA an equal
        // range of pixels whose input rows it stages in shared memory.
        cbs::GatherPlan g{};
        if (has_overrides(rq) || !cbs::gather_plan(p, sm_count, &g)) return CBS_ERR_UNSUPPORTED;
        out.block_m = 128;
        out.block_n = g.block_n;
        out.block_k = g.block_k;
        out.stages = g.stages;
        out.tiles = g.tiles;
        out.grid = g.grid;
        out.threads = cbs::kGatherBlockThreads;
        out.smem_bytes = g.smem_bytes;
        out.k_iters = 1;
        out.cluster = 1;
    } else if (chosen == CBS_ALGO_TCGEN05) {
        cbs::TcPlan t{};
        if (cbs::tc_make_plan_request(p, sm_count, rq, &t) != 0) return CBS_ERR_UNSUPPORTED;
        out.block_m = t.cmajor ? t.cm_unit_px : (t.swap_ab ? t.block_n : cbs::kTcBlockM);  // output pixels per tile
        out.block_n = t.swap_ab ? cbs::kTcBlockM : t.block_n;  // output channels per tile
        out.block_k = t.block_k;
        out.stages = t.stages;
        out.tiles = t.m_tiles * t.n_tiles;
        out.grid = t.grid;
        out.threads = t.cmajor ? cbs::kCmThreads : cbs::tc_threads(t.block_n, t.pair != 0);
        out.smem_bytes = t.smem_bytes;
        out.k_iters = t.k_iters;
        out.stream_k = t.stream_k;
        out.swap_ab = t.swap_ab;
        out.cluster = t.pair ? 2 : 1;
        out.workspace_bytes = t.workspace_bytes;
        out.balanced = t.balanced;
        out.weights_resident = t.cmajor ? t.cm_wres : 0;
        out.row_boxes = t.cmajor && t.cm_xmode != 0 ? 1 : 0;
    } else {
        if (has_overrides(rq)) return CBS_ERR_UNSUPPORTED;  // the direct kernel has no tilings to choose
        const long long bx = (p.m + cbs::kDirectThreads - 1) / cbs::kDirectThreads;
        const int by = (c_out + cbs::kDirectBlockN - 1) / cbs::kDirectBlockN;
        out.block_m = cbs::kDirectThreads;
        out.block_n = cbs::kDirectBlockN;
        out.block_k = 1;
        out.stages = 0;
        out.tiles = (int)(bx * by);
        out.grid = out.tiles;
        out.threads = cbs::kDirectThreads;
        out.smem_bytes = 0;
        out.k_iters = r * s * c;
    }
    *info = out;
    return CBS_OK;
}

int conv_bn_silu_plan(int n, int h, int w_in, int c, int c_out, int r, int s, int stride_h, int stride_w,
                      int pad_h, int pad_w, int algo, int sm_count, cbs_plan_info *info)
{
    if (!info || sm_count < 1 || algo < CBS_ALGO_AUTO || algo > CBS_ALGO_DIRECT)
        return CBS_ERR_INVALID_ARG;
    cbs::ConvProblem p{};
    const int st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    return fill_plan(p, algo, sm_count, nullptr, info);
}

int conv_bn_silu_plan_request(int n, int h, int w_in, int c, int c_out, int r, int s, int stride_h,
                              int stride_w, int pad_h, int pad_w, const cbs_plan_request *req, int sm_count,
                              cbs_plan_info *info)
{
    if (!info || sm_count < 1) return CBS_ERR_INVALID_ARG;
    int algo = 0;
    cbs::PlanRequest rq{};
    int st = read_request(req, &algo, &rq);
    if (st != CBS_OK) return st;
    cbs::ConvProblem p{};
    st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    return fill_plan(p, algo, sm_count, &rq, info);
}

int conv_bn_silu_forward_request(const void *x, const void *w, const float *scale, const float *bias,
                                 void *y, int n, int h, int w_in, int c, int c_out, int r, int s,
                                 int stride_h, int stride_w, int pad_h, int pad_w, const cbs_plan_request *req,
                                 void *stream)
{
    int algo = 0;
    cbs::PlanRequest rq{};
    int st = read_request(req, &algo, &rq);
    if (st != CBS_OK) return st;
    cbs::ConvProblem p{};
    st = make_problem(n, h, w_in, c, c_out, r, s, stride_h, stride_w, pad_h, pad_w, &p);
    if (st != CBS_OK) return st;
    if (p.m == 0 || c_out == 0) return CBS_OK;
    if (!x || !w || !scale || !bias || !y) return CBS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(scale) || !aligned16(bias) || !aligned16(y))
        return CBS_ERR_MISALIGNED;
    p.x = x;
    p.w = w;
    p.scale = scale;
    p.bias = bias;
    p.y = y;
    p.wait_timeout_ns = req->wait_timeout_ns;
    return launch_forward(p, algo, static_cast<cudaStream_t>(stream), &rq);
}

int conv_bn_silu_layer_norm(const void *x, long long x_stride, const float *gamma, const float *beta, float eps,
                            void *y, long long y_stride, float *stats, long long rows, int c, int dtype,
                            void *stream)
{
    return norm_call(x, x_stride, gamma, beta, eps, y, y_stride, nullptr, 0, nullptr, stats, 1, rows, c, dtype, stream);
}

int conv_bn_silu_quantize_rows(const void *x, long long x_stride, void *q, long long q_stride, float *row_scale,
                               long long rows, int c, int dtype, void *stream)
{
    if (!q && rows != 0) return CBS_ERR_INVALID_ARG;
    return norm_call(x, x_stride, nullptr, nullptr, 0.0f, nullptr, 0, q, q_stride, row_scale, nullptr, 0, rows, c,
                     dtype, stream);
}

int conv_bn_silu_layer_norm_quantize(const void *x, long long x_stride, const float *gamma, const float *beta,
                                     float eps, void *q, long long q_stride, float *row_scale, long long rows,
                                     int c, int dtype, void *stream)
{
    if (!q && rows != 0) return CBS_ERR_INVALID_ARG;
    return norm_call(x, x_stride, gamma, beta, eps, nullptr, 0, q, q_stride, row_scale, nullptr, 1, rows, c, dtype,
                     stream);
}

long long conv_bn_silu_layer_norm_backward_workspace(long long rows, int c)
{
    if (!norm_sizes_ok(rows, c, CBS_DTYPE_F32)) return -1;
    int sms = 0;
    if (sm_count_current_device(&sms) != CBS_OK) return -1;
    return 8LL * c * cbs::norm_grad_partial_rows(rows, sms);
}

int conv_bn_silu_layer_norm_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                     const float *gamma, const float *stats, void *dx, long long dx_stride,
                                     float *dgamma, float *dbeta, long long rows, int c, int dtype,
                                     void *workspace, long long workspace_bytes, void *stream)
{
    if (!norm_sizes_ok(rows, c, dtype)) return CBS_ERR_INVALID_ARG;
    if (!dgamma || !dbeta) return CBS_ERR_INVALID_ARG;
    if (!aligned_to(gamma, 4) || !aligned_to(stats, 4) || !aligned_to(dgamma, 4) || !aligned_to(dbeta, 4))
        return CBS_ERR_MISALIGNED;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        cudaError_t e = cudaMemsetAsync(dgamma, 0, 4 * (size_t)c, strm);
        if (e == cudaSuccess) e = cudaMemsetAsync(dbeta, 0, 4 * (size_t)c, strm);
        return e == cudaSuccess ? CBS_OK : cuda_fail(e);
    }
    const int size = cbs::dtype_size(dtype);
    int st = check_rows(dy, rows, c, dy_stride, size, false);
    if (st == CBS_OK) st = check_rows(x, rows, c, x_stride, size, false);
    if (st == CBS_OK) st = check_rows(dx, rows, c, dx_stride, size, true);
    if (st != CBS_OK) return st;
    if (!stats || !workspace) return CBS_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return CBS_ERR_MISALIGNED;
    int sms = 0;
    st = sm_count_current_device(&sms);
    if (st != CBS_OK) return st;
    cbs::NormGradProblem p{};
    p.partial_rows = cbs::norm_grad_partial_rows(rows, sms);
    if (workspace_bytes < 8LL * c * p.partial_rows) return CBS_ERR_INVALID_ARG;
    p.dy = cbs::Rows{const_cast<void *>(dy), dy_stride};
    p.x = cbs::Rows{const_cast<void *>(x), x_stride};
    p.dx = cbs::Rows{dx, dx_stride};
    p.gamma = gamma;
    p.stats = stats;
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    p.partial = static_cast<float *>(workspace);
    p.rows = rows;
    p.c = c;
    p.dtype = dtype;
    cudaError_t e = cbs::norm_grad_launch(p, sms, strm);
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

long long conv_bn_silu_linear_int8_workspace(long long m, int n, int k)
{
    if (!linear_sizes_ok(m, n, k)) return -1;
    int sms = 0;
    if (sm_count_current_device(&sms) != CBS_OK) return -1;
    return cbs::linear_workspace_bytes(m, n, k, sms);
}

int conv_bn_silu_linear_int8_plan(long long m, int n, int k, int align, int sm_count, cbs_linear_plan *plan)
{
    if (!plan || sm_count < 1 || !linear_sizes_ok(m, n, k) || (align != 16 && align != 4 && align != 1))
        return CBS_ERR_INVALID_ARG;
    const cbs::LinearPlan p = cbs::linear_plan(m, n, k, align, sm_count);
    *plan = cbs_linear_plan{p.kernel, p.turned, p.tile_rows, p.tile_channels, p.align, p.k_steps, p.tiles, p.workers};
    return CBS_OK;
}

int conv_bn_silu_linear_int8(const void *a, long long a_stride, const void *w, long long w_stride,
                             const float *a_scale, const float *w_scale, const float *bias, const void *residual,
                             long long residual_stride, void *y, long long y_stride, long long m, int n, int k,
                             int activation, int out_dtype, void *workspace, long long workspace_bytes,
                             void *stream)
{
    if (!linear_sizes_ok(m, n, k)) return CBS_ERR_INVALID_ARG;
    if (activation < CBS_ACT_SILU || activation > CBS_ACT_RELU) return CBS_ERR_INVALID_ARG;
    if (out_dtype < CBS_DTYPE_F32 || out_dtype > CBS_DTYPE_F16) return CBS_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return CBS_OK;
    const int size = cbs::dtype_size(out_dtype);
    int st = check_rows(y, m, n, y_stride, size, true);
    if (st == CBS_OK && k > 0) st = check_rows(a, m, k, a_stride, 1, false);
    if (st == CBS_OK && k > 0) st = check_rows(w, n, k, w_stride, 1, false);
    if (st == CBS_OK && residual) st = check_rows(residual, m, n, residual_stride, size, false);
    if (st != CBS_OK) return st;
    if (!a_scale || !w_scale) return CBS_ERR_INVALID_ARG;
    if (!aligned_to(a_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(bias, 4) || !aligned16(workspace))
        return CBS_ERR_MISALIGNED;
    int sms = 0;
    st = sm_count_current_device(&sms);
    if (st != CBS_OK) return st;
    if (workspace_bytes < cbs::linear_workspace_bytes(m, n, k, sms)) return CBS_ERR_INVALID_ARG;
    if (!workspace && workspace_bytes > 0) return CBS_ERR_INVALID_ARG;
    cbs::LinearProblem p{};
    p.a = cbs::Rows{const_cast<void *>(a), a_stride};
    p.w = cbs::Rows{const_cast<void *>(w), w_stride};
    p.residual = cbs::Rows{const_cast<void *>(residual), residual_stride};
    p.y = cbs::Rows{y, y_stride};
    p.a_scale = a_scale;
    p.w_scale = w_scale;
    p.bias = bias;
    p.m = m;
    p.n = n;
    p.k = k;
    p.out_dtype = out_dtype;
    p.activation = activation;
    p.workspace = workspace;
    cudaError_t e = cbs::linear_launch(p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBS_OK : cuda_fail(e);
}

int conv_bn_silu_check(void *stream)
{
    unsigned int word = 0;
    cudaError_t e = cbs::tc_read_and_clear_error(static_cast<cudaStream_t>(stream), &word);
    if (e != cudaSuccess) return cuda_fail(e);
    unsigned int gword = 0;
    e = cbs::gather_read_and_clear_error(static_cast<cudaStream_t>(stream), &gword);
    if (e != cudaSuccess) return cuda_fail(e);
    unsigned int wword = 0;
    e = cbs::cmajor_read_and_clear_error(static_cast<cudaStream_t>(stream), &wword);
    if (e != cudaSuccess) return cuda_fail(e);
    unsigned int lword = 0;
    e = cbs::linear_read_and_clear_error(static_cast<cudaStream_t>(stream), &lword);
    if (e != cudaSuccess) return cuda_fail(e);
    if ((gword != 0 || wword != 0 || lword != 0) && word == 0) return CBS_ERR_TIMEOUT;
    if (word == 0) return CBS_OK;
    // A kernel gave up mid-way: stream-K ready flags may be left raised.
    e = cbs::tc_reset_workspaces();
    if (e != cudaSuccess) return cuda_fail(e);
    return CBS_ERR_TIMEOUT;
}

const char *conv_bn_silu_status_string(int status)
{
    switch (status) {
    case CBS_OK: return "ok";
    case CBS_ERR_INVALID_ARG: return "invalid argument";
    case CBS_ERR_MISALIGNED: return "device pointer not 16-byte aligned";
    case CBS_ERR_UNSUPPORTED: return "shape not supported by the requested kernel";
    case CBS_ERR_CUDA: return "CUDA error";
    case CBS_ERR_TIMEOUT: return "kernel pipeline wait timed out";
    default: return "unknown status";
    }
}

int conv_bn_silu_last_cuda_error(void) { return t_last_cuda_error; }

}  // extern "C"
