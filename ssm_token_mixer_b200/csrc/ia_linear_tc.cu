#include "ia_linear.h"
namespace ia {
bool lin_tc_supported(const ia_linear_shape_t&) { return false; }
cudaError_t launch_lin_tc(const LinArgs&, bool, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace ia
