// Rotary positions of query and key heads, and the table that the model's own
// kernels read.
//
// y = a R(p f_i) x on pairs (x0, x1): y0 = a (x0 cos - x1 sin),
// y1 = a (x0 sin + x1 cos).  The angle is kept in turns as a 64-bit binary
// fraction: p x turns in unsigned 64-bit arithmetic wraps exactly at whole
// turns, so the range reduction that a far position needs costs one integer
// multiplication and loses nothing; the top 32 bits, read as a signed
// fraction of a half turn, go to sincospif.
//
// The work is a copy with a few operations per element, bound by memory: each
// element is read and written once (16 bytes a thread and access), the sines
// and cosines of a token are made once per block and serve all of its heads.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "ops.cuh"

namespace rv {

int op_fail(int code, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_error_message(buf);
  return code;
}

int check_batch(int B, int T) {
  if (B < 1 || T < 1) return op_fail(RV_EINVAL, "B and T must be at least 1");
  if ((int64_t)B * T > INT32_MAX / 2) return op_fail(RV_EINVAL, "B x T above 2^30");
  return RV_OK;
}

int check_heads(const char *what, const rv_heads *h, int B, int T, int head_dim, bool output) {
  if (!h || !h->data) return op_fail(RV_EINVAL, "%s: null pointer", what);
  if (h->dtype != RV_F16 && h->dtype != RV_BF16 && h->dtype != RV_F32)
    return op_fail(RV_EINVAL, "%s: unknown dtype %d", what, h->dtype);
  if (h->heads < 1 || h->heads > 65535) return op_fail(RV_EINVAL, "%s: heads must be in 1..65535", what);
  const int64_t align = h->dtype == RV_F32 ? 4 : 8;  // elements of 16 bytes
  const int64_t n[3] = {B, T, h->heads}, st[3] = {h->stride_b, h->stride_t, h->stride_h};
  if (reinterpret_cast<uintptr_t>(h->data) & 15u) return op_fail(RV_EINVAL, "%s: data not 16-byte aligned", what);
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1) {
      if (st[i] % align) return op_fail(RV_EINVAL, "%s: rows not 16-byte aligned (stride %lld)", what, (long long)st[i]);
      if (st[i] < 0 || st[i] > (INT64_MAX >> 4) / n[i]) return op_fail(RV_EINVAL, "%s: stride out of range", what);
    }
  if (output) {
    // rows overlap unless, by rising stride, each dimension steps over all
    // that the smaller ones span
    int o[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (st[o[j]] > st[o[j + 1]]) { const int t = o[j]; o[j] = o[j + 1]; o[j + 1] = t; }
    int64_t span = head_dim;
    for (int i = 0; i < 3; ++i)
      if (n[o[i]] > 1) {
        if (st[o[i]] < span) return op_fail(RV_EINVAL, "%s: output rows overlap", what);
        span += (n[o[i]] - 1) * st[o[i]];
      }
  }
  return RV_OK;
}

int check_device(const char *what, const void *p) {
  if (!p) return RV_OK;
  cudaPointerAttributes at;
  cudaError_t e = cudaPointerGetAttributes(&at, p);
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return op_fail(RV_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  }
  if (at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == dev)) return RV_OK;
  return op_fail(RV_EINVAL, "%s: not memory of the current device", what);
}

// ------------------------------------------------------------------ kernel

namespace {

constexpr int kThreads = 256;

// 8 elements of a row as they lie in memory, and as floats.
template <int DT>
struct Raw8 {
  uint4 v[DT == RV_F32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void *base, int64_t off) {
  Raw8<DT> r;
  if (DT == RV_F32) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off);
    r.v[0] = p[0];
    r.v[DT == RV_F32] = p[DT == RV_F32];
  } else {
    r.v[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off);
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void floats8(const Raw8<DT> &r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
  if (DT == RV_F32) {
    const uint4 h = r.v[DT == RV_F32];
    const uint32_t y[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __uint_as_float(w[i]);
      x[4 + i] = __uint_as_float(y[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = act_to_f((uint16_t)w[i], DT);
      x[2 * i + 1] = act_to_f((uint16_t)(w[i] >> 16), DT);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void *base, int64_t off, const float (&x)[8]) {
  if (DT == RV_F32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + off);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + off) =
        make_uint4(pack_act2(x[0], x[1], DT), pack_act2(x[2], x[3], DT), pack_act2(x[4], x[5], DT), pack_act2(x[6], x[7], DT));
  }
}

// cos and sin of position p's turn of pair frequency `turns`.
__device__ __forceinline__ float2 cos_sin(int64_t p, uint64_t turns) {
  const uint64_t phase = (uint64_t)p * turns;
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

struct RopeGrid {
  int tokens_per_block;
  FastDiv items, chunks, pairs, row;  // items of a token, 16-element chunks of a head, pairs, tokens of a row
};

// One item: 16 elements (8 pairs) of one head of one token.
struct Item {
  bool ok, rot;
  int which, cs;             // q or k; first of its 8 pairs in the block's table
  int64_t src, dst;
  int lo, hi;                // the two runs of 8 elements
};

// A block takes a run of tokens: its threads ask for their first kItems items,
// make the tokens' sines and cosines while these are on the way, then turn
// and store them.
template <int IN, int OUT, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ rv_rope_plan plan, const __grid_constant__ RopeArgs a, RopeGrid g) {
  pdl_wait();
  pdl_trigger();
  constexpr int kItems = IN == RV_F32 ? 2 : 4;
  extern __shared__ float2 cs[];  // [tokens_per_block][pairs]
  const int pairs = plan.rotary_dim / 2, tok0 = blockIdx.x * g.tokens_per_block;
  const int ntok = min(g.tokens_per_block, a.B * a.T - tok0), b0 = tok0 / a.T, at0 = tok0 - b0 * a.T;
  const int per = g.items.d, total = ntok * per;
  // row and token of the block's token tk (the quotient is exact below 2^16; above, at most one row ends)
  auto place = [&](int tk, int &b, int &t) {
    const int x = at0 + tk, q = a.T < 32768 ? (int)div_by(x, g.row) : x >= a.T;
    b = b0 + q;
    t = x - q * a.T;
  };
  auto item = [&](int it) {
    Item m;
    const int tk = div_by(it, g.items), r = it - tk * per;
    const int hh = div_by(r, g.chunks), j = r - hh * (int)g.chunks.d;
    int b, t;
    place(tk, b, t);
    m.ok = it < total && t < row_count(a.count, b, a.T);
    m.which = hh >= a.H[0];
    const int h = hh - (m.which ? a.H[0] : 0);
    m.rot = 16 * j < plan.rotary_dim;
    m.cs = tk * pairs + 8 * j;
    m.lo = m.rot && HALF ? 8 * j : 16 * j;
    m.hi = m.rot && HALF ? m.lo + pairs : m.lo + 8;
    const Heads &in = a.in[m.which], &out = a.out[m.which];
    m.src = b * in.sb + t * in.st + h * in.sh;
    m.dst = b * out.sb + t * out.st + h * out.sh;
    return m;
  };
  auto turn = [&](const Item &m, const Raw8<IN> &rx, const Raw8<IN> &ry) {
    float x[8], y[8];
    floats8<IN>(rx, x);
    floats8<IN>(ry, y);
    if (m.rot) {
      float2 c[8];
      const float4 *p = reinterpret_cast<const float4 *>(cs + m.cs);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = p[i];
        c[2 * i] = make_float2(v.x, v.y);
        c[2 * i + 1] = make_float2(v.z, v.w);
      }
      auto pair = [](float &x0, float &x1, float2 c) {
        const float u = x0 * c.x - x1 * c.y, v = x0 * c.y + x1 * c.x;
        x0 = u;
        x1 = v;
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (HALF) pair(x[i], y[i], c[i]);
        else if (i < 4) pair(x[2 * i], x[2 * i + 1], c[i]);
        else pair(y[2 * i - 8], y[2 * i - 7], c[i]);
      }
    }
    store8<OUT>(a.out[m.which].p, m.dst + m.lo, x);
    store8<OUT>(a.out[m.which].p, m.dst + m.hi, y);
  };

  Item m[kItems];
  Raw8<IN> x[kItems], y[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    m[k] = item(threadIdx.x + k * kThreads);
    if (m[k].ok) {
      x[k] = load8<IN>(a.in[m[k].which].p, m[k].src + m[k].lo);
      y[k] = load8<IN>(a.in[m[k].which].p, m[k].src + m[k].hi);
    }
  }
  for (int u = threadIdx.x; u < ntok * pairs; u += kThreads) {
    const int tk = div_by(u, g.pairs), i = u - tk * pairs;
    int b, t;
    place(tk, b, t);
    float2 v = cos_sin((int64_t)row_pos(a.pos, b) + t, plan.turns[i]);
    v.x *= plan.attention_factor;
    v.y *= a.inverse ? -plan.attention_factor : plan.attention_factor;
    cs[u] = v;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kItems; ++k)
    if (m[k].ok) turn(m[k], x[k], y[k]);
  for (int it = threadIdx.x + kItems * kThreads; it < total; it += kThreads) {  // heads beyond a block's items
    const Item n = item(it);
    if (n.ok) turn(n, load8<IN>(a.in[n.which].p, n.src + n.lo), load8<IN>(a.in[n.which].p, n.src + n.hi));
  }
}

template <int IN, int OUT>
cudaError_t launch_io(const rv_rope_plan &plan, const RopeArgs &a, cudaStream_t s, int pdl) {
  const int chunks = plan.head_dim / 16, items = (a.H[0] + a.H[1]) * chunks, pairs = plan.rotary_dim / 2, tokens = a.B * a.T;
  RopeGrid g;
  // as many tokens as the threads' first items cover, but enough blocks to fill the GPU
  int tpb = kThreads * (IN == RV_F32 ? 2 : 4) / items;
  if (tpb > tokens / 608) tpb = tokens / 608;
  if (tpb > 4096 / pairs) tpb = 4096 / pairs;  // 32 KB of sines and cosines
  if (tpb < 1) tpb = 1;
  g.tokens_per_block = tpb;
  g.items = fast_div(items);
  g.chunks = fast_div(chunks);
  g.pairs = fast_div(pairs);
  g.row = fast_div(a.T);
  const int grid = (tokens + tpb - 1) / tpb;
  const size_t smem = sizeof(float2) * pairs * tpb;
  auto fn = plan.layout == RV_ROPE_HALF ? k_rope<IN, OUT, true> : k_rope<IN, OUT, false>;
  return launch_k(fn, dim3(grid), dim3(kThreads), smem, s, pdl, plan, a, g);
}

__global__ void k_rope_plan_table(const __grid_constant__ rv_rope_plan plan, float2 *cs, int T) {
  const int pairs = plan.rotary_dim / 2;
  for (size_t u = blockIdx.x * (size_t)blockDim.x + threadIdx.x; u < (size_t)T * pairs; u += (size_t)gridDim.x * blockDim.x) {
    const float2 v = cos_sin((int64_t)(u / pairs), plan.turns[u % pairs]);
    cs[u] = make_float2(v.x * plan.attention_factor, v.y * plan.attention_factor);
  }
}

}  // namespace

cudaError_t launch_rope(const rv_rope_plan &plan, const RopeArgs &a, int in_dtype, int out_dtype, cudaStream_t s, int pdl) {
  if (in_dtype == RV_F32) {
    if (out_dtype == RV_F32) return launch_io<RV_F32, RV_F32>(plan, a, s, pdl);
    return out_dtype == RV_F16 ? launch_io<RV_F32, RV_F16>(plan, a, s, pdl) : launch_io<RV_F32, RV_BF16>(plan, a, s, pdl);
  }
  return in_dtype == RV_F16 ? launch_io<RV_F16, RV_F16>(plan, a, s, pdl) : launch_io<RV_BF16, RV_BF16>(plan, a, s, pdl);
}

cudaError_t launch_rope_table(const rv_rope_plan &plan, float2 *cs, int T, cudaStream_t s) {
  const size_t n = (size_t)T * (plan.rotary_dim / 2);
  const size_t grid = (n + 255) / 256;
  k_rope_plan_table<<<(unsigned)(grid < 4096 ? grid : 4096), 256, 0, s>>>(plan, cs, T);
  return cudaGetLastError();
}

}  // namespace rv

// ==================================================================== C ABI

using namespace rv;

extern "C" int rv_rope_init(const rv_rope_config *cfg, rv_rope_plan *plan) {
  set_error_message("");
  if (!cfg || !plan) return op_fail(RV_EINVAL, "null pointer");
  const rv_rope_config &c = *cfg;
  const double two_pi = 6.283185307179586476925;
  const int r = c.rotary_dim;
  if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 16) return op_fail(RV_EINVAL, "head_dim must be a multiple of 16 in 16..256");
  if (r < 16 || r > c.head_dim || r % 16) return op_fail(RV_EINVAL, "rotary_dim must be a multiple of 16 in 16..head_dim");
  if (c.layout != RV_ROPE_HALF && c.layout != RV_ROPE_INTERLEAVED) return op_fail(RV_EINVAL, "unknown layout %d", c.layout);
  if (c.scaling < RV_ROPE_PLAIN || c.scaling > RV_ROPE_RAMP) return op_fail(RV_EINVAL, "unknown scaling %d", c.scaling);
  if (!(c.theta > 1.0) || !isfinite(c.theta)) return op_fail(RV_EINVAL, "theta must be finite and above 1");
  if (c.scaling != RV_ROPE_PLAIN && (!(c.factor > 0.0) || !isfinite(c.factor))) return op_fail(RV_EINVAL, "factor must be finite and above 0");
  if ((c.scaling == RV_ROPE_BANDS || c.scaling == RV_ROPE_RAMP) && c.original_max_position < 1)
    return op_fail(RV_EINVAL, "original_max_position must be at least 1");
  if (c.scaling == RV_ROPE_BANDS && (!(c.low_freq_factor > 0.0) || !(c.high_freq_factor > c.low_freq_factor) || !isfinite(c.high_freq_factor)))
    return op_fail(RV_EINVAL, "needs 0 < low_freq_factor < high_freq_factor");
  if (c.scaling == RV_ROPE_RAMP && (!(c.beta_slow > 0.0) || !(c.beta_fast > c.beta_slow) || !isfinite(c.beta_fast)))
    return op_fail(RV_EINVAL, "needs beta_fast > beta_slow > 0");
  if (!isfinite(c.attention_factor) || c.attention_factor < 0.0) return op_fail(RV_EINVAL, "attention_factor must be finite and not negative");
  rv_rope_plan p{};
  p.head_dim = c.head_dim;
  p.rotary_dim = r;
  p.layout = c.layout;
  double att = c.attention_factor;
  if (att == 0.0) att = c.scaling == RV_ROPE_RAMP && c.factor > 1.0 ? 0.1 * log(c.factor) + 1.0 : 1.0;
  if (!(att <= 3.402823466e38)) return op_fail(RV_EINVAL, "attention_factor is out of fp32's range");
  p.attention_factor = (float)att;
  const double base = c.scaling == RV_ROPE_BASE ? c.theta * pow(c.factor, r / (r - 2.0)) : c.theta;
  if (!(base > 0.0) || !isfinite(base)) return op_fail(RV_EINVAL, "factor moves theta out of range");
  double lo = 0.0, hi = 1.0;
  if (c.scaling == RV_ROPE_RAMP) {
    const double k = r / (2.0 * log(c.theta));
    lo = fmin(fmax(floor(k * log(c.original_max_position / (two_pi * c.beta_fast))), 0.0), r - 1.0);
    hi = fmin(fmax(ceil(k * log(c.original_max_position / (two_pi * c.beta_slow))), 0.0), r - 1.0);
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < r / 2; ++i) {
    const double f0 = pow(base, -2.0 * i / r);
    double f = f0;
    if (c.scaling == RV_ROPE_LINEAR) {
      f = f0 / c.factor;
    } else if (c.scaling == RV_ROPE_BANDS) {
      const double k = fmin(fmax((c.original_max_position * f0 / two_pi - c.low_freq_factor) / (c.high_freq_factor - c.low_freq_factor), 0.0), 1.0);
      f = k * f0 + (1.0 - k) * f0 / c.factor;
    } else if (c.scaling == RV_ROPE_RAMP) {
      const double u = fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
      f = (1.0 - u) * f0 + u * f0 / c.factor;
    }
    const double turns = f / two_pi;  // whole turns per position make no difference
    if (!(turns < 1e9)) return op_fail(RV_EINVAL, "a frequency is out of range");
    p.turns[i] = (uint64_t)ldexp(turns - floor(turns), 64);  // below 2^64: the fraction is at most 1 - 2^-53
  }
  *plan = p;
  return RV_OK;
}

extern "C" int rv_rope(const rv_rope_plan *plan, const rv_heads *q_in, const rv_heads *q_out, const rv_heads *k_in,
                       const rv_heads *k_out, int B, int T, const int32_t *d_pos, const int32_t *d_count, int inverse,
                       void *stream) {
  set_error_message("");
  if (!plan) return op_fail(RV_EINVAL, "null pointer");
  const int hd = plan->head_dim, r = plan->rotary_dim;
  if (hd < 16 || hd > 256 || hd % 16 || r < 16 || r > hd || r % 16 ||
      (plan->layout != RV_ROPE_HALF && plan->layout != RV_ROPE_INTERLEAVED))
    return op_fail(RV_EINVAL, "the plan was not made by rv_rope_init");
  if (check_batch(B, T)) return RV_EINVAL;
  if ((k_in == nullptr) != (k_out == nullptr)) return op_fail(RV_EINVAL, "k_in and k_out: both or neither");
  if (check_heads("q_in", q_in, B, T, hd, false) || check_heads("q_out", q_out, B, T, hd, true)) return RV_EINVAL;
  if (k_in && (check_heads("k_in", k_in, B, T, hd, false) || check_heads("k_out", k_out, B, T, hd, true))) return RV_EINVAL;
  if (q_in->heads != q_out->heads || (k_in && k_in->heads != k_out->heads)) return op_fail(RV_EINVAL, "in and out differ in heads");
  if (k_in && (k_in->dtype != q_in->dtype || k_out->dtype != q_out->dtype)) return op_fail(RV_EINVAL, "q and k differ in dtype");
  // the kernel's quotients of a token's 16-element chunks are exact up to here
  if ((int64_t)(q_in->heads + (k_in ? k_in->heads : 0)) * (hd / 16) > 32768)
    return op_fail(RV_EINVAL, "query and key heads x head_dim above 2^19 elements a token");
  if (q_in->dtype != q_out->dtype && q_in->dtype != RV_F32) return op_fail(RV_EINVAL, "a 16-bit input keeps its dtype");
  if (q_in->data == q_out->data && q_in->dtype != q_out->dtype) return op_fail(RV_EINVAL, "in place needs one dtype");
  if (k_in && k_in->data == k_out->data && k_in->dtype != k_out->dtype) return op_fail(RV_EINVAL, "in place needs one dtype");
  if ((reinterpret_cast<uintptr_t>(d_pos) | reinterpret_cast<uintptr_t>(d_count)) & 3u)
    return op_fail(RV_EINVAL, "d_pos or d_count not 4-byte aligned");
  if (int rc = check_device("q_in", q_in->data)) return rc;
  if (int rc = check_device("q_out", q_out->data)) return rc;
  if (k_in) {
    if (int rc = check_device("k_in", k_in->data)) return rc;
    if (int rc = check_device("k_out", k_out->data)) return rc;
  }
  if (int rc = check_device("d_pos", d_pos)) return rc;
  if (int rc = check_device("d_count", d_count)) return rc;
  RopeArgs a{};
  a.in[0] = heads_of(q_in);
  a.out[0] = heads_of(q_out);
  a.in[1] = heads_of(k_in);
  a.out[1] = heads_of(k_out);
  a.H[0] = q_in->heads;
  a.H[1] = k_in ? k_in->heads : 0;
  a.B = B; a.T = T;
  a.pos = d_pos; a.count = d_count;
  a.inverse = inverse != 0;
  const cudaError_t e = launch_rope(*plan, a, q_in->dtype, q_out->dtype, static_cast<cudaStream_t>(stream), 1);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return op_fail(RV_ECUDA, "rv_rope: %s", cudaGetErrorString(e));
  }
  return RV_OK;
}
