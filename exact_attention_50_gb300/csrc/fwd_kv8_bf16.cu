// fwd_kv8_bf16.cu -- bf16 instantiations of the tcgen05 forward over an expanded 8-bit cache.
#include "fwd_tc.cuh"

namespace attn {
cudaError_t launch_fwd_kv8_bf16(const FwdMaps& maps, const FwdParams& p, bool causal, cudaStream_t stream) {
  return launch_fwd_kv8_dtype<__nv_bfloat16>(maps, p, causal, stream);
}
}  // namespace attn
