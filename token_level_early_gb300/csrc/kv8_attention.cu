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

// The cluster plan for short contexts: enough blocks for two tiles each while
// the units' clusters fit one block per SM, more (two per SM) where a block
// would have over 16 tiles; the line where it still has.  Measured in
// microseconds, line / clusters of 1 / 2 / 4 / 8 (bf16, head_dim 128, one row
// of 8 KV heads): 256 positions 9.7 / 6.9 / 5.8 / 5.2 / 5.4, 1024: 10.1 / 11.2
// / 8.1 / 6.7 / 6.0, 4096: 11.3 / 28 / 17 / 11.0 / 8.1, 8192: 12.9 / - / - /
// 16.5 / 11.0; 16 such rows: 256: 17.9 / 6.8 / 6.3 / 11.3 / 22, 1024: 11.9 /
// 11.1 / 9.3 / 13.8 / 23, 2048: 13.6 / 16.8 / 13.5 / 16 / 25, 4096: 20.4 / 30 /
// 21 / 24 / 33; one KV head: 2048: 7.7 / 17 / 11 / 8.2 / 6.7, 4096: 7.7 / 29 /
// 17 / 11 / 8.1.  Where the rule is not the faster one: it leaves clusters of 8
// for the line above 16 tiles a block, although 8 KV heads at 8192 positions
// are 1.9 us faster on them, and stays with them for one KV head at 4096, which
// costs 0.4.  `most` is the cache's max_seq in rv_kv8_attention, which cannot
// see the rows' lengths on the device, and the longest row in the model.
int kv8_attention_cluster(const Kv8 &c, int B, int T, int H, int n_sm, int most) {
  const int rows = T * (H / c.Hkv), nt = kv8a::pick_nt(rows);
  const int64_t tiles = (most + kv8a::tile_len(c.hd) - 1) / kv8a::tile_len(c.hd);
  const int64_t units = (int64_t)B * c.Hkv * ((rows + 8 * nt - 1) / (8 * nt));
  int cs = 1;
  while (cs < 8 && tiles > 2 * cs && units * cs * 2 <= n_sm) cs *= 2;
  while (cs < 8 && tiles > 16 * cs && units * cs * 2 <= 2 * n_sm) cs *= 2;
  return tiles <= 16 * cs && units <= INT32_MAX / 8 ? cs : 0;
}

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
