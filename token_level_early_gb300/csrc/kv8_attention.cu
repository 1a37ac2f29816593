// Attention of a few new tokens per row over the 8-bit K/V cache.
//
// out = sum_p w_p v_p / sum_p w_p with w_p = exp(scale q.k_p - m), one pass
// over the visible positions with a running maximum m, sum and weighted sum.
// k_p = code * s_block, so q.k_p = s_block (q.code).
#include <cuda_fp8.h>

#include "ops.cuh"

namespace rv {
namespace {

constexpr int kWarps = 8;

template <int FMT>
__device__ __forceinline__ float code_value(uint8_t q) {
  return FMT == RV_KV8_INT8 ? (float)(int8_t)q : __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
}

// One block per (query token, query head, row): its warps take the visible
// positions in turn, a lane holds HD / 32 elements; the warps' states are
// joined through shared memory.
template <int FMT, int HD>
__global__ void __launch_bounds__(kWarps * 32) k_attn8(Kv8AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int PER = HD / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][HD];
  const int t = blockIdx.x % a.T, b = blockIdx.x / a.T, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (t >= row_count(a.count, b, a.T)) return;
  const Kv8 &c = a.c;
  const int64_t see = (int64_t)row_pos(a.pos, b) + t + 1;
  const int n = (int)(see < 0 ? 0 : see > c.T ? c.T : see);
  const int64_t row = (int64_t)b * c.Hkv + h / (a.H / c.Hkv);
  float q[PER];
  const int64_t qo = b * a.q.sb + t * a.q.st + h * a.q.sh + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    q[i] = a.q_f32 ? round_act(static_cast<const float *>(a.q.p)[qo + i], c.act)
                   : act_to_f(static_cast<const uint16_t *>(a.q.p)[qo + i], c.act);
  float m = -INFINITY, l = 0.f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  const float *ks = c.scale[0] + row * (c.N / c.block), *vs = c.scale[1] + row * (c.N / c.block);
  for (int p = warp; p < n; p += kWarps) {
    const uint8_t *kc = c.codes[0] + (row * c.N + p) * HD + lane * PER, *vc = c.codes[1] + (row * c.N + p) * HD + lane * PER;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) x = fmaf(q[i], code_value<FMT>(kc[i]), x);
    x = warp_sum(x) * ks[p / c.block] * a.scale;
    const float mn = fmaxf(m, x), sv = vs[p / c.block];
    const float f = m == mn ? 1.f : expf(m - mn), w = x == mn ? 1.f : expf(x - mn);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] * f + w * (sv * code_value<FMT>(vc[i]));
    m = mn;
    if (x != x) l = x;
  }
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
  for (int i = 0; i < PER; ++i) so[warp][lane * PER + i] = o[i];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
  for (int w = 0; w < kWarps; ++w) ll += sm[w] == -INFINITY && sl[w] == 0.f ? 0.f : sl[w] * (sm[w] == mm ? 1.f : expf(sm[w] - mm));
  for (int d = threadIdx.x; d < HD; d += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (sm[w] != -INFINITY || sl[w] != 0.f) x += so[w][d] * (sm[w] == mm ? 1.f : expf(sm[w] - mm));
    x = n ? x / ll : 0.f;
    const int64_t oo = b * a.out.sb + t * a.out.st + h * a.out.sh + d;
    if (a.out_dtype == RV_F32) static_cast<float *>(a.out.p)[oo] = a.round_out ? round_act(x, c.act) : x;
    else static_cast<uint16_t *>(a.out.p)[oo] = f_to_act(x, c.act);
  }
  if (a.lse && threadIdx.x == 0) a.lse[((int64_t)b * a.T + t) * a.H + h] = n ? mm + logf(ll) : -INFINITY;
}

}  // namespace

size_t kv8_attention_work(const Kv8 &, int, int, int, int) { return 0; }

cudaError_t launch_kv8_attention(const Kv8AttnArgs &a, int n_sm, cudaStream_t s, int pdl) {
  (void)n_sm;
  auto fn = a.c.fmt == RV_KV8_INT8 ? (a.c.hd == 64 ? k_attn8<RV_KV8_INT8, 64> : k_attn8<RV_KV8_INT8, 128>)
                                   : (a.c.hd == 64 ? k_attn8<RV_KV8_E4M3, 64> : k_attn8<RV_KV8_E4M3, 128>);
  return launch_k(fn, dim3(a.B * a.T, a.H), dim3(kWarps * 32), 0, s, pdl, a);
}

}  // namespace rv
