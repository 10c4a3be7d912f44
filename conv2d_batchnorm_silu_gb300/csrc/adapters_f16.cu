// adapters_f16.cu -- the low-rank adapters' kernels for f16 activations (adapters.cu has the formulas).
#include "adapters_device.cuh"

namespace cbs {
template cudaError_t adapter_products_launch<__half>(const AdapterArgs &, bool, bool, int, int, cudaStream_t);
template cudaError_t adapter_weights_launch<__half>(const AdapterGradArgs &, cudaStream_t);
}  // namespace cbs
