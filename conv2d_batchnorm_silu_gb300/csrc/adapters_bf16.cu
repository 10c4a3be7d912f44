// adapters_bf16.cu -- the low-rank adapters' kernels for bf16 activations (adapters.cu has the formulas).
#include "adapters_device.cuh"

namespace cbs {
template cudaError_t adapter_products_launch<__nv_bfloat16>(const AdapterArgs &, bool, bool, int, int, cudaStream_t);
template cudaError_t adapter_weights_launch<__nv_bfloat16>(const AdapterGradArgs &, cudaStream_t);
}  // namespace cbs
