// Stand-ins for the kernel launchers of include/hq_mx.h, for the host-only sanitizer build of its
// C-ABI layer (hq_mx_api.cpp): argument checks only, no launcher is ever reached.
#include "../../hadamard_rotated_precision_amd/csrc/hq_mx_internal.hpp"

namespace hq {

hipError_t mx_quant_pass(const MxQuantPass&, hipStream_t) { return hipErrorInvalidValue; }
hipError_t mx_dequant_pass(const MxOperand&, int64_t, int64_t, int, void*, int, hipStream_t) { return hipErrorInvalidValue; }
size_t mx_gemm_ws(int64_t, int64_t, int64_t) { return 0; }
hipError_t mx_gemm_pass(const MxGemmPass&, hipStream_t) { return hipErrorInvalidValue; }
bool mx_gemv_fused_ok(int64_t, int64_t) { return false; }
hipError_t mx_gemv_pass(const MxGemmPass&, const void*, int, int, hipStream_t) { return hipErrorInvalidValue; }
hipError_t kv_append_pass(const KvAppendPass&, hipStream_t) { return hipErrorInvalidValue; }
hipError_t kv_read_pass(const KvReadPass&, hipStream_t) { return hipErrorInvalidValue; }
size_t kv_attention_ws(const hq_kv_cache&, const hq_kv_batch& b) { return b.seqs > 0 && b.max_len > 64 ? 1024 : 0; }
hipError_t kv_attention_pass(const KvAttentionPass&, hipStream_t) { return hipErrorInvalidValue; }

}  // namespace hq
