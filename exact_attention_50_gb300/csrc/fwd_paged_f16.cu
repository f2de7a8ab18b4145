// fwd_paged_f16.cu -- fp16 instantiations of the tcgen05 forward over a KV cache in pages,
// and the dtype switch.
#include "fwd_tc.cuh"

namespace attn {
cudaError_t launch_fwd_paged_bf16(const FwdMaps& maps, const FwdParams& p, bool causal, cudaStream_t stream);

cudaError_t launch_fwd_paged(const FwdMaps& maps, const FwdParams& p, attn_dtype_t dtype, bool causal, cudaStream_t stream) {
  if (dtype == ATTN_BF16) return launch_fwd_paged_bf16(maps, p, causal, stream);
  return launch_fwd_mode<__half, kModePaged>(maps, p, causal, stream);
}
}  // namespace attn
