// adapters_f32.cu -- the low-rank adapters' kernels for f32 activations (adapters.cu has the formulas).
#include "adapters_device.cuh"

namespace cbs {
template cudaError_t adapter_products_launch<float>(const AdapterArgs &, bool, bool, int, int, cudaStream_t);
template cudaError_t adapter_weights_launch<float>(const AdapterGradArgs &, cudaStream_t);
}  // namespace cbs
