#include "retention.cuh"
namespace linattn {
bool ret_tc_supported(const RetArgs &, Dtype) { return false; }
int ret_parts_tc(const RetArgs &) { return 1; }
cudaError_t launch_retention_tc(const RetArgs &, int, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace linattn
