// attn_status.cu — reading a sticky status word of the kernels and clearing it in
// one step.  Kernels on other streams may set the word at any time: with a copy
// and a memset, what is set between the two is lost.
#include <atomic>
#include <thread>

#include "../../include/attn.h"
#include "attn_internal.h"

namespace attn {

namespace {

constexpr int kTakers = 64;  // reads under way at once (others wait for one to end)
__device__ int g_taken[kTakers];

__global__ void take_kernel(int* status, int slot) { g_taken[slot] = atomicExch(status, 0); }

// A slot of g_taken that no other read uses.
class Slot {
 public:
  Slot() {
    unsigned long long used = mask().load();
    for (;;) {
      if (~used == 0) {
        std::this_thread::yield();
        used = mask().load();
        continue;
      }
      index = __builtin_ctzll(~used);
      if (mask().compare_exchange_weak(used, used | 1ull << index)) return;
    }
  }
  ~Slot() { mask().fetch_and(~(1ull << index)); }
  Slot(const Slot&) = delete;
  Slot& operator=(const Slot&) = delete;
  int index;

 private:
  static std::atomic<unsigned long long>& mask() {
    static std::atomic<unsigned long long> m{0};
    return m;
  }
};

}  // namespace

int take_status(int* status, cudaStream_t stream) {
  if (status == nullptr) return ATTN_ERR_CUDA;
  void* taken = nullptr;
  if (cudaGetSymbolAddress(&taken, g_taken) != cudaSuccess) return ATTN_ERR_CUDA;
  Slot slot;
  int st = 0;
  take_kernel<<<1, 1, 0, stream>>>(status, slot.index);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (cudaMemcpyAsync(&st, static_cast<int*>(taken) + slot.index, sizeof(int),
                      cudaMemcpyDeviceToHost, stream) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ATTN_ERR_CUDA;
  return st;
}

}  // namespace attn
