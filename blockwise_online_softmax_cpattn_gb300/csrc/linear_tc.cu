#include "layer.cuh"
namespace cpattn {
bool linear_tc_supported(const Ring&) { return false; }
cudaError_t launch_linear_tc(const Linear&, cudaStream_t, bool) { return cudaErrorNotSupported; }
}
