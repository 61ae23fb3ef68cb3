// Stand-ins for the kernel launchers of include/hq_train.h, for the host-only sanitizer build of
// its C-ABI layer (hq_train_api.cpp): argument checks only, no launcher is ever reached.
#include "../../hadamard_rotated_precision_amd/csrc/hq_train_internal.hpp"

namespace hq {

hipError_t block_quant_pass(const BlockQuantPass&, hipStream_t) { return hipErrorInvalidValue; }
size_t block_gemm_ws(int64_t, int64_t, int64_t) { return 0; }
hipError_t block_gemm_pass(const BlockGemmPass&, hipStream_t) { return hipErrorInvalidValue; }
bool block_gemv_fused_ok(int64_t, int64_t) { return false; }
hipError_t block_gemv_pass(const BlockGemmPass&, const void*, int, bool, hipStream_t) {
  return hipErrorInvalidValue;
}
hipError_t adamw_pass(const hq_adamw_tensor*, int, const hq_adamw_config&, const hq_adamw_scalars&,
                      const hq_adamw_scalars*, hipStream_t) {
  return hipErrorInvalidValue;
}

}  // namespace hq
