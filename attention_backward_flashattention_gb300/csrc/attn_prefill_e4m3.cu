// attn_prefill_e4m3.cu — prefill over an e4m3 cache (attn_prefill.cuh).
#include "attn_prefill.cuh"

namespace attn {

cudaError_t launch_prefill_e4m3(const PrefillLaunch& L) {
  if (L.dqk == 64) return launch_prefill_sized<64, 64, true>(L);
  if (L.dqk == 128) return launch_prefill_sized<128, 128, true>(L);
  if (L.dqk == 192) return launch_prefill_sized<192, 128, true>(L);
  return cudaErrorInvalidValue;
}

}  // namespace attn
