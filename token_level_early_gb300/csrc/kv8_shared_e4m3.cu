// Attention over a shared prefix: the e4m3 kernels (see kv8_shared.cuh).
#include "kv8_shared.cuh"

namespace rv {
namespace kv8s {

cudaError_t launch_prefix_e4m3(const SharedArgs &a, int n_sm, cudaStream_t s) { return launch_prefix_fmt<RV_KV8_E4M3>(a, n_sm, s); }

}  // namespace kv8s
}  // namespace rv
