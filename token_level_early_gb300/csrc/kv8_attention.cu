// Attention over the 8-bit K/V cache: the int8 kernels and the choice of row
// groups (kernels in kv8_attention.cuh; e4m3 in kv8_attention_e4m3.cu).
#include "kv8_attention.cuh"

namespace rv {

namespace kv8a {

constexpr int kMaxNt = 3;

// Columns of 8 query rows per pass over a KV head's cache: as few passes as
// kMaxNt allows, evenly filled.
int pick_nt(int rows) {
  const int cols = (rows + 7) / 8, passes = (cols + kMaxNt - 1) / kMaxNt;
  return (cols + passes - 1) / passes;
}

cudaError_t launch_int8(const Kv8AttnArgs &a, int nt, int n_sm, cudaStream_t s, int pdl) {
  return launch_fmt<RV_KV8_INT8>(a, nt, n_sm, s, pdl);
}

}  // namespace kv8a

size_t kv8_attention_work(const Kv8 &c, int, int T, int H, int n_sm) {
  // a smaller T may run fewer columns (and then more blocks): the largest need
  const int cols = (T * (H / c.Hkv) + 7) / 8;
  size_t most = 0;
  for (int nt = 1; nt <= kv8a::kMaxNt && nt <= cols; ++nt) {
    const size_t n = kv8a::work_bytes(c.hd, nt, kv8a::blocks_per_sm(c.hd, nt) * n_sm);
    if (n > most) most = n;
  }
  return most;
}

cudaError_t launch_kv8_attention(const Kv8AttnArgs &a, int n_sm, cudaStream_t s, int pdl) {
  const int nt = kv8a::pick_nt(a.T * (a.H / a.c.Hkv));
  return a.c.fmt == RV_KV8_INT8 ? kv8a::launch_int8(a, nt, n_sm, s, pdl) : kv8a::launch_e4m3(a, nt, n_sm, s, pdl);
}

}  // namespace rv
