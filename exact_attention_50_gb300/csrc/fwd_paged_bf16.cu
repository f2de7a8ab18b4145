// fwd_paged_bf16.cu -- bf16 instantiations of the tcgen05 forward over a KV cache in pages.
#include "fwd_tc.cuh"

namespace attn {
cudaError_t launch_fwd_paged_bf16(const FwdMaps& maps, const FwdParams& p, bool causal, cudaStream_t stream) {
  return launch_fwd_mode<__nv_bfloat16, kModePaged>(maps, p, causal, stream);
}
}  // namespace attn
