// attn_decode_e4m3.cu — the decode over e4m3 caches (a file of its own: the two
// compile side by side).
#include "attn_decode.cuh"

namespace attn {

cudaError_t launch_decode_e4m3(const DecodeLaunch& L) { return launch_cache<true>(L); }

}  // namespace attn
