// spa_errors.cu - reads and clears the error words of several translation units at once.
#include "spa_errors.h"

#include <mutex>

namespace spa {

namespace {

constexpr int kMaxDevices = 64;
constexpr int kWords = 6;
struct Words {
  int* at[kWords];
};

static __device__ int g_collected;

__global__ void collect_kernel(const Words w) {
  int v = 0;
  for (int i = 0; i < kWords; ++i) v |= atomicExch(w.at[i], 0);
  g_collected = v;
}

std::mutex g_mu;               // (one collection at a time: they share g_collected)
Words g_words[kMaxDevices];
bool g_known[kMaxDevices];

}  // namespace

cudaError_t collect_error_words(int* value) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_known[dev]) {
    int i = 0;
    for (cudaError_t (*word)(int**) : {indexer_error_word, latent_cache_error_word,
                                       latent_decode_error_word, latent_prefill_error_word,
                                       latent_tree_error_word, rotary_error_word}) {
      e = word(&g_words[dev].at[i++]);
      if (e != cudaSuccess) return e;
    }
    g_known[dev] = true;
  }
  // On the legacy stream, as the copy after it and the copies of the other words.  (The launch's own status: the
  // last error may be one that somebody else left.)
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(1);
  c.blockDim = dim3(1);
  e = cudaLaunchKernelEx(&c, collect_kernel, g_words[dev]);
  if (e != cudaSuccess) return e;
  return cudaMemcpyFromSymbol(value, g_collected, sizeof(int));
}

}  // namespace spa
