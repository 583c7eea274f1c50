// Check of clc_drop_rest (ptx.cuh), compiled and run by tests/test_gpu_give_up.py: a launch of many
// more CTAs than fit, each of which gives up at once, in one of four ways:
//   0  returns: every CTA of the launch starts
//   1  takes the others over first: only those start that were running together
//   2  the same, after one question whose answer it has read
//   3  the same, after one question without having waited for the answer
#include <cstdio>
#include <cstdlib>

#include "../attention_backward_flashattention_gb300/csrc/ptx.cuh"

using namespace attn;

__global__ void give_up(int* started, int mode) {
  __shared__ uint64_t bar_word;
  __shared__ __align__(16) uint64_t answer_words[2];
  if (threadIdx.x != 0) return;
  atomicAdd(started, 1);
  const uint32_t bar = smem_u32(&bar_word), answer = smem_u32(answer_words);
  mbar_init(bar, 1);
  fence_barrier_init();
  const uint64_t t0 = globaltimer();  // (until all of those that fit are there: 200 us)
  while (globaltimer() - t0 < 200000) {
  }
  if (mode == 0) return;
  uint32_t asked = 0;
  if (mode >= 2) {
    mbar_arrive_expect_tx(bar, 16);
    clc_ask(answer, bar);
    asked = 1;
    int x;
    if (mode == 2 && (!mbar_wait_drain(bar, 0) || !clc_read(answer, &x))) return;
  }
  clc_drop_rest(answer, bar, asked, gridDim.x);
}

#define OK(x)                                                                   \
  do {                                                                          \
    cudaError_t e = (x);                                                        \
    if (e != cudaSuccess) {                                                     \
      std::printf("%s: %s\n", #x, cudaGetErrorString(e));                       \
      return 1;                                                                 \
    }                                                                           \
  } while (0)

int main() {
  int sms = 0, *started = nullptr, n = 0;
  OK(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, 0));
  OK(cudaMalloc(&started, sizeof(int)));
  constexpr int kSmem = 200 * 1024;  // (one CTA an SM)
  OK(cudaFuncSetAttribute(give_up, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  for (int mode = 0; mode < 4; ++mode)
    for (int grid : {1, sms, sms + 1, 8 * sms}) {
      OK(cudaMemset(started, 0, sizeof(int)));
      give_up<<<grid, 32, kSmem>>>(started, mode);
      OK(cudaGetLastError());
      OK(cudaDeviceSynchronize());
      OK(cudaMemcpy(&n, started, sizeof(int), cudaMemcpyDeviceToHost));
      std::printf("%d %d %d %d\n", mode, grid, sms, n);
    }
  return 0;
}
