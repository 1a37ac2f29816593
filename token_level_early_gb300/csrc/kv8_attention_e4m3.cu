// Attention over the 8-bit K/V cache: the e4m3 kernels (see kv8_attention.cuh).
#include "kv8_attention.cuh"

namespace rv {
namespace kv8a {

cudaError_t launch_e4m3(const Kv8AttnArgs &a, int nt, int n_sm, cudaStream_t s, int pdl) {
  return launch_fmt<RV_KV8_E4M3>(a, nt, n_sm, s, pdl);
}

}  // namespace kv8a
}  // namespace rv
