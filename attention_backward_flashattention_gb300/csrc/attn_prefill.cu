// attn_prefill.cu — prefill over a bf16 cache (attn_prefill.cuh).
#include "attn_prefill.cuh"

namespace attn {

cudaError_t launch_prefill(const PrefillLaunch& L) {
  if (L.cache.e4m3) return launch_prefill_e4m3(L);
  if (L.dqk == 64) return launch_prefill_sized<64, 64, false>(L);
  if (L.dqk == 128) return launch_prefill_sized<128, 128, false>(L);
  if (L.dqk == 192) return launch_prefill_sized<192, 128, false>(L);
  return cudaErrorInvalidValue;
}

}  // namespace attn
