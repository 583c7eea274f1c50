// attn_decode.cu — the decode over bf16 caches, and which cache it is.
#include "attn_decode.cuh"

namespace attn {

cudaError_t launch_decode(const DecodeLaunch& L) {
  return L.cache.e4m3 ? launch_decode_e4m3(L) : launch_cache<false>(L);
}

}  // namespace attn
