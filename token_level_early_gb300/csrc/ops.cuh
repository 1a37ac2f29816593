// Shared pieces of the stand-alone operators (rope.cu, kv8.cu, kv8_attention.cu):
// tensor descriptors as the kernels see them, host checks, and the internal
// launchers that the model's own paths call.
#pragma once

#include <stddef.h>

#include "../../include/rv.h"
#include "common.cuh"
#include "kernels.cuh"

namespace rv {

// Every kernel of these operators waits for its predecessor's end before it
// touches memory (griddepcontrol.wait), so all of them may be launched with
// programmatic dependence on whatever is before them in the stream: the
// launch then overlaps the predecessor's tail.  So what the predecessor writes
// is written during their lifetime, and none of them reads memory through the
// read-only path (__ldg), which holds only for data that no one writes while
// the kernel lives.

// Records the message and returns the code.
int op_fail(int code, const char *fmt, ...);

// A [B][T][heads][head_dim] tensor (strides in elements).
struct Heads {
  void *p;
  int64_t sb, st, sh;
};
inline Heads heads_of(const rv_heads *h) { return h ? Heads{h->data, h->stride_b, h->stride_t, h->stride_h} : Heads{}; }

// Unsigned division by a run-time constant: q = (x * m) >> 32 with m =
// floor(2^32 / d) + 1 is exact for x * d < 2^32 (the error x / 2^32 * (m d -
// 2^32) / d stays below 1 / d).
struct FastDiv {
  uint32_t d, m;
};
inline FastDiv fast_div(uint32_t d) { return FastDiv{d, d == 1 ? 0u : (uint32_t)((1ull << 32) / d + 1)}; }
__device__ __forceinline__ uint32_t div_by(uint32_t x, FastDiv f) { return f.d == 1 ? x : __umulhi(x, f.m); }

// Two floats rounded to a 16-bit pair (lo in the low half).
__device__ __forceinline__ uint32_t pack_act2(float lo, float hi, int act) {
  uint32_t r;
  if (act) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 operations in one instruction (each half rounded as the scalar one;
// the compiler may fuse f2_mul into an f2_add of its result).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// A row's token count and first position (see the conventions in rv.h).
__device__ __forceinline__ int row_count(const int32_t *count, int b, int T) {
  return count ? min(max(count[b], 0), T) : T;
}
__device__ __forceinline__ int row_pos(const int32_t *pos, int b) { return pos ? pos[b] : 0; }

constexpr int kKv8ErrPos = 64;  // bit 6 of *d_err: a position outside the cache

// Checks one tensor: pointer, dtype, head count, 16-byte rows; for outputs,
// that no two rows overlap.  Returns RV_OK or RV_EINVAL with the message set.
int check_heads(const char *what, const rv_heads *h, int B, int T, int head_dim, bool output);
int check_batch(int B, int T);
// RV_EINVAL if p is not device (or managed) memory of the current device.
int check_device(const char *what, const void *p);

// Rotary positions.
struct RopeArgs {
  Heads in[2], out[2];  // q, k
  int H[2];
  int B, T;
  const int32_t *pos, *count;
  int inverse;
};
cudaError_t launch_rope(const rv_rope_plan &plan, const RopeArgs &a, int in_dtype, int out_dtype, cudaStream_t s, int pdl = 0);
// (cos, sin) of positions 0..T-1 x head_dim/2 pairs, times the attention factor.
cudaError_t launch_rope_table(const rv_rope_plan &plan, float2 *cs, int T, cudaStream_t s);

// 8-bit K/V cache.
struct Kv8 {
  uint8_t *codes[2];
  float *scale[2];
  uint16_t *tail[2];
  int B, Hkv, hd, T, N, block, fmt, act;  // T = max_seq, N = T rounded up to a block
};
Kv8 kv8_of(const rv_kv8 *c);
struct Kv8Io {
  Heads k, v;
  int B, T;
  const int32_t *pos, *count;
  int32_t *err;
};
cudaError_t launch_kv8_append(const Kv8 &c, const Kv8Io &io, int in_dtype, cudaStream_t s, int pdl = 0);
cudaError_t launch_kv8_read(const Kv8 &c, const Kv8Io &io, int out_dtype, cudaStream_t s, int pdl = 0);

struct Kv8AttnArgs {
  Kv8 c;
  Heads q, out;
  int H, B, T;
  int q_f32, out_dtype;
  int round_out;  // RV_F32 output rounded to act_dtype (the model's activations)
  float scale;
  const int32_t *pos, *count;
  float *lse;
  void *work;
  int cluster;  // blocks of a cluster (short contexts: a cluster per unit), or 0 (the cut line)
};
// Kv8AttnArgs::cluster for rows that see up to `most` positions.
int kv8_attention_cluster(const Kv8 &c, int B, int T, int H, int n_sm, int most);
size_t kv8_attention_work(const Kv8 &c, int B, int T, int H, int n_sm);
cudaError_t launch_kv8_attention(const Kv8AttnArgs &a, int n_sm, cudaStream_t s, int pdl = 0);

}  // namespace rv
