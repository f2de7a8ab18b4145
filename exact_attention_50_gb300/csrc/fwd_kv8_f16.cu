// fwd_kv8_f16.cu -- fp16 instantiations of the tcgen05 forward over an expanded 8-bit cache, and the
// dtype switch.
#include "fwd_tc.cuh"

namespace attn {
cudaError_t launch_fwd_kv8_bf16(const FwdMaps& maps, const FwdParams& p, bool causal, cudaStream_t stream);

cudaError_t launch_fwd_kv8(const FwdMaps& maps, const FwdParams& p, attn_dtype_t dtype, bool causal, cudaStream_t stream) {
  if (dtype == ATTN_BF16) return launch_fwd_kv8_bf16(maps, p, causal, stream);
  return launch_fwd_kv8_dtype<__half>(maps, p, causal, stream);
}
}  // namespace attn
