// The 8-bit K/V cache: quantising new tokens as they are appended and reading
// the cache back.
//
// A block is `block` positions of one row and one KV head.  Its scale is
// s = max(up8(amax / Q), 2^-100) and a code is x / s rounded to the nearest
// code, ties to even.  amax comes from the 16-bit originals by integer
// comparison (magnitude bits order like the values, infinities and NaNs
// above all), so it is exact; s has 8 significant bits and x at most 11, so
// x / s is either a midpoint between codes exactly or at least 2^-20 away
// from one in relative terms, and the correctly rounded fp32 quotient rounds
// to the same code as the real one.
//
// Both are copies with little arithmetic: memory bounds them.
#include <cuda_fp8.h>

#include "ops.cuh"

namespace rv {
namespace {

constexpr float kScaleMin = 0x1p-100f;

// Magnitude bits from which a 16-bit value is infinite or NaN.
template <int ACT>
__device__ __forceinline__ constexpr uint32_t inf_bits() { return ACT == RV_BF16 ? 0x7f80u : 0x7c00u; }

// Largest magnitude bits of the two 16-bit halves of a and b.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7fff7fffu); }

// Scale of a block whose largest magnitude bits are m.
template <int ACT, int FMT>
__device__ __forceinline__ float block_scale(uint32_t m) {
  if (m >= inf_bits<ACT>()) return __int_as_float(0x7fc00000);
  const float t = act_to_f((uint16_t)m, ACT) / (FMT == RV_KV8_INT8 ? 127.f : 448.f);
  const float up = __uint_as_float((__float_as_uint(t) + 0xffffu) & 0xffff0000u);
  return fmaxf(up, kScaleMin);
}

// Two codes of a 16-bit pair (low half first), in the low 16 bits.
template <int ACT, int FMT>
__device__ __forceinline__ uint32_t code2(uint32_t v, float s) {
  const float x0 = act_to_f((uint16_t)v, ACT) / s, x1 = act_to_f((uint16_t)(v >> 16), ACT) / s;
  if (FMT == RV_KV8_INT8) return (uint32_t)(__float2int_rn(x0) & 0xff) | (uint32_t)(__float2int_rn(x1) & 0xff) << 8;
  return __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
}

// 8 values of an input row as 16-bit pairs (RV_F32 rows are rounded).
template <int ACT, bool F32>
__device__ __forceinline__ uint4 load_row8(const void *base, int64_t off) {
  if (!F32) return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off);
  const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off);
  const float4 a = p[0], b = p[1];
  auto two = [](float x, float y) { return f_to_act(x, ACT) | (uint32_t)f_to_act(y, ACT) << 16; };
  return make_uint4(two(a.x, a.y), two(a.z, a.w), two(b.x, b.y), two(b.z, b.w));
}

// ------------------------------------------------------------------ append

struct AppendGrid {
  int threads_per_unit, units_per_block;  // a unit is one cache block
  int blocks_per_row;                     // cache blocks that T tokens can touch
  int64_t units;
};

// A unit (threads_per_unit threads, 4 vectors of 8 values each) takes one
// cache block: originals before the row's first new position come from the
// tail, the others from the input; their largest magnitude gives the scale,
// and the codes of the block's present positions are written.  The unit of a
// row's first block also copies the row's last 2 x block new originals into
// the tail, after it has read what it needs from there: no other unit reads
// the tail.
template <int ACT, int FMT, bool F32, int HD>
__global__ void k_append(Kv8 c, Kv8Io io, AppendGrid g) {
  pdl_wait();
  pdl_trigger();
  constexpr int VR = HD / 8;  // vectors of a row
  __shared__ uint32_t red[16];
  const int grp = threadIdx.x / g.threads_per_unit, tid = threadIdx.x - grp * g.threads_per_unit;
  const int64_t unit = (int64_t)blockIdx.x * g.units_per_block + grp;
  bool live = unit < g.units;
  int b = 0, h = 0, kv = 0, blk = 0, p0 = 0, end = 0, pos = 0;
  if (live) {
    const int i = (int)(unit % g.blocks_per_row);
    int64_t r = unit / g.blocks_per_row;
    kv = (int)(r & 1);
    r >>= 1;
    h = (int)(r % c.Hkv);
    b = (int)(r / c.Hkv);
    pos = row_pos(io.pos, b);
    const int n = row_count(io.count, b, io.T);
    if (n == 0) {
      live = false;
    } else if (pos < 0 || pos >= c.T) {
      live = false;
      if (io.err && i == 0 && tid == 0) atomicOr(io.err, kKv8ErrPos);
    } else {
      end = (int)min((int64_t)pos + n, (int64_t)c.T);
      if (io.err && i == 0 && tid == 0 && end - pos < n) atomicOr(io.err, kKv8ErrPos);
      blk = pos / c.block + i;
      p0 = blk * c.block;
      live = p0 < end;
    }
  }
  const Heads &in = kv ? io.v : io.k;
  const int64_t row = (int64_t)b * c.Hkv + h;
  uint16_t *tail = c.tail[kv] + row * 2 * c.block * HD;
  const int64_t src = b * in.sb + h * in.sh;
  uint4 v[4];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int u = tid + k * g.threads_per_unit, p = p0 + u / VR, d = (u % VR) * 8;
    v[k] = make_uint4(0, 0, 0, 0);
    if (live && p < end)
      v[k] = p < pos ? *reinterpret_cast<const uint4 *>(tail + (p % (2 * c.block)) * HD + d)
                     : load_row8<ACT, F32>(in.p, src + (p - pos) * in.st + d);
    m = max_abs2(max_abs2(max_abs2(max_abs2(m, v[k].x), v[k].y), v[k].z), v[k].w);
  }
  m = max(m & 0xffffu, m >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  const int warp = threadIdx.x >> 5, nw = g.threads_per_unit >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = m;
  __syncthreads();
  for (int i = 0; i < nw; ++i) m = max(m, red[grp * nw + i]);
  if (!live) return;
  const float s = block_scale<ACT, FMT>(m);
  const bool bad = !(s == s);
  uint8_t *codes = c.codes[kv] + (row * c.N + p0) * HD;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int u = tid + k * g.threads_per_unit;
    if (p0 + u / VR >= end) continue;
    uint2 o = make_uint2(0, 0);
    if (!bad) {
      o.x = code2<ACT, FMT>(v[k].x, s) | code2<ACT, FMT>(v[k].y, s) << 16;
      o.y = code2<ACT, FMT>(v[k].z, s) | code2<ACT, FMT>(v[k].w, s) << 16;
    }
    *reinterpret_cast<uint2 *>(codes + (int64_t)u * 8) = o;
  }
  if (tid == 0) c.scale[kv][row * (c.N / c.block) + blk] = s;
  if (p0 <= pos) {
    const int from = max(pos, end - 2 * c.block);
    for (int u = tid; u < (end - from) * VR; u += g.threads_per_unit) {
      const int p = from + u / VR, d = (u % VR) * 8;
      *reinterpret_cast<uint4 *>(tail + (p % (2 * c.block)) * HD + d) = load_row8<ACT, F32>(in.p, src + (int64_t)(p - pos) * in.st + d);
    }
  }
}

template <int ACT, int FMT, bool F32, int HD>
cudaError_t append_t(const Kv8 &c, const Kv8Io &io, cudaStream_t s, int pdl) {
  AppendGrid g;
  g.threads_per_unit = c.block * HD / 32;
  const int threads = g.threads_per_unit < 128 ? 128 : g.threads_per_unit;
  g.units_per_block = threads / g.threads_per_unit;
  g.blocks_per_row = (io.T + c.block - 2) / c.block + 1;
  g.units = (int64_t)g.blocks_per_row * 2 * c.Hkv * io.B;
  const int64_t grid = (g.units + g.units_per_block - 1) / g.units_per_block;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_k(k_append<ACT, FMT, F32, HD>, dim3((unsigned)grid), dim3(threads), 0, s, pdl, c, io, g);
}

// ------------------------------------------------------------------ read

// One thread reads 8 codes of a row and writes their values.
template <int OUT, int FMT, int HD>
__global__ void __launch_bounds__(256) k_read(Kv8 c, Kv8Io io, int64_t total) {
  constexpr int VR = HD / 8;
  for (int64_t u = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; u < total; u += (int64_t)gridDim.x * blockDim.x) {
    const int d = (int)(u % VR) * 8;
    int64_t r = u / VR;
    const int h = (int)(r % c.Hkv);
    r /= c.Hkv;
    const int t = (int)(r % io.T);
    r /= io.T;
    const int b = (int)(r % io.B), kv = (int)(r / io.B);
    const Heads &out = kv ? io.v : io.k;
    if (!out.p || t >= row_count(io.count, b, io.T)) continue;
    const int64_t p = (int64_t)row_pos(io.pos, b) + t;
    if (p < 0 || p >= c.T) {
      if (io.err) atomicOr(io.err, kKv8ErrPos);
      continue;
    }
    const int64_t row = (int64_t)b * c.Hkv + h;
    const uint2 w = *reinterpret_cast<const uint2 *>(c.codes[kv] + (row * c.N + p) * HD + d);
    const float s = c.scale[kv][row * (c.N / c.block) + p / c.block];
    const uint32_t cw[2] = {w.x, w.y};
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint8_t q = (uint8_t)(cw[i >> 2] >> (8 * (i & 3)));
      x[i] = FMT == RV_KV8_INT8 ? (float)(int8_t)q : __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
      x[i] *= s;
    }
    const int64_t dst = b * out.sb + t * out.st + h * out.sh + d;
    if (OUT == RV_F32) {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out.p) + dst);
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      const float top = OUT == RV_F16 ? 65504.f : __uint_as_float(0x7f7f0000u);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (x[i] == x[i]) x[i] = fminf(fmaxf(x[i], -top), top);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = f_to_act(x[2 * i], OUT) | (uint32_t)f_to_act(x[2 * i + 1], OUT) << 16;
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out.p) + dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int OUT, int FMT>
cudaError_t read_t(const Kv8 &c, const Kv8Io &io, cudaStream_t s) {
  const int64_t total = (int64_t)2 * io.B * io.T * c.Hkv * (c.hd / 8);
  const int64_t grid = (total + 255) / 256;
  auto fn = c.hd == 64 ? k_read<OUT, FMT, 64> : k_read<OUT, FMT, 128>;
  fn<<<(unsigned)(grid < 152 * 64 ? grid : 152 * 64), 256, 0, s>>>(c, io, total);
  return cudaGetLastError();
}

}  // namespace

Kv8 kv8_of(const rv_kv8 *p) {
  Kv8 c{};
  c.codes[0] = static_cast<uint8_t *>(p->k_codes);
  c.codes[1] = static_cast<uint8_t *>(p->v_codes);
  c.scale[0] = p->k_scale;
  c.scale[1] = p->v_scale;
  c.tail[0] = static_cast<uint16_t *>(p->k_tail);
  c.tail[1] = static_cast<uint16_t *>(p->v_tail);
  c.B = p->max_batch; c.Hkv = p->n_kv_heads; c.hd = p->head_dim; c.T = p->max_seq;
  c.block = p->block; c.fmt = p->format; c.act = p->act_dtype;
  c.N = (c.T + c.block - 1) / c.block * c.block;
  return c;
}

cudaError_t launch_kv8_append(const Kv8 &c, const Kv8Io &io, int in_dtype, cudaStream_t s, int pdl) {
#define RV_A(ACT_, FMT_)                                                                        \
  if (c.act == ACT_ && c.fmt == FMT_) {                                                         \
    if (in_dtype == RV_F32)                                                                     \
      return c.hd == 64 ? append_t<ACT_, FMT_, true, 64>(c, io, s, pdl) : append_t<ACT_, FMT_, true, 128>(c, io, s, pdl); \
    return c.hd == 64 ? append_t<ACT_, FMT_, false, 64>(c, io, s, pdl) : append_t<ACT_, FMT_, false, 128>(c, io, s, pdl); \
  }
  RV_A(RV_F16, RV_KV8_INT8) RV_A(RV_F16, RV_KV8_E4M3) RV_A(RV_BF16, RV_KV8_INT8) RV_A(RV_BF16, RV_KV8_E4M3)
#undef RV_A
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv8_read(const Kv8 &c, const Kv8Io &io, int out_dtype, cudaStream_t s) {
#define RV_R(OUT_) \
  if (out_dtype == OUT_) return c.fmt == RV_KV8_INT8 ? read_t<OUT_, RV_KV8_INT8>(c, io, s) : read_t<OUT_, RV_KV8_E4M3>(c, io, s);
  RV_R(RV_F16) RV_R(RV_BF16) RV_R(RV_F32)
#undef RV_R
  return cudaErrorInvalidValue;
}

}  // namespace rv

// ==================================================================== C ABI

using namespace rv;

namespace {

int check_cache(const rv_kv8 *c, bool pointers) {
  if (!c) return op_fail(RV_EINVAL, "null pointer");
  if (c->max_batch < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 65535 || c->max_seq < 1)
    return op_fail(RV_EINVAL, "cache: max_batch, n_kv_heads and max_seq must be positive");
  if (c->max_seq > INT32_MAX - 256) return op_fail(RV_EINVAL, "cache: max_seq too large");
  if (c->head_dim != 64 && c->head_dim != 128) return op_fail(RV_EINVAL, "cache: head_dim must be 64 or 128");
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return op_fail(RV_EINVAL, "cache: block must be 16, 32, 64 or 128");
  if (c->format != RV_KV8_INT8 && c->format != RV_KV8_E4M3) return op_fail(RV_EINVAL, "cache: unknown format %d", c->format);
  if (c->act_dtype != RV_F16 && c->act_dtype != RV_BF16) return op_fail(RV_EINVAL, "cache: act_dtype must be RV_F16 or RV_BF16");
  if (!pointers) return RV_OK;
  const void *p[6] = {c->k_codes, c->v_codes, c->k_scale, c->v_scale, c->k_tail, c->v_tail};
  for (const void *q : p) {
    if (!q) return op_fail(RV_EINVAL, "cache: null pointer");
    if (reinterpret_cast<uintptr_t>(q) & 15u) return op_fail(RV_EINVAL, "cache: memory not 16-byte aligned");
  }
  return RV_OK;
}

int check_rows(const rv_kv8 *c, int B, int T) {
  if (check_batch(B, T)) return RV_EINVAL;
  if (B > c->max_batch) return op_fail(RV_EINVAL, "B above the cache's max_batch");
  return RV_OK;
}

int check_kv(const rv_kv8 *c, const char *what, const rv_heads *h, int B, int T, bool output) {
  if (int rc = check_heads(what, h, B, T, c->head_dim, output)) return rc;
  if (h->heads != c->n_kv_heads) return op_fail(RV_EINVAL, "%s: heads differ from the cache's n_kv_heads", what);
  return RV_OK;
}

int check_index(const int32_t *pos, const int32_t *count, const int32_t *err) {
  if ((reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(count) | reinterpret_cast<uintptr_t>(err)) & 3u)
    return op_fail(RV_EINVAL, "d_pos, d_count or d_err not 4-byte aligned");
  return RV_OK;
}

// Where every pointer of a call lives (after the checks that need no GPU).
int check_memory(const rv_kv8 *c, const void *x, const void *y, const int32_t *pos, const int32_t *count,
                 const void *more) {
  const void *p[] = {c->k_codes, c->v_codes, c->k_scale, c->v_scale, c->k_tail, c->v_tail};
  for (const void *q : p)
    if (int rc = check_device("cache", q)) return rc;
  if (int rc = check_device("data", x)) return rc;
  if (int rc = check_device("data", y)) return rc;
  if (int rc = check_device("d_pos", pos)) return rc;
  if (int rc = check_device("d_count", count)) return rc;
  return check_device("d_err, d_lse or workspace", more);
}

int launched(const char *what, cudaError_t e) {
  if (e == cudaSuccess) return RV_OK;
  cudaGetLastError();
  return op_fail(RV_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

int sm_count(int *n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return launched("device query", e);
}

}  // namespace

extern "C" int rv_kv8_append(const rv_kv8 *cache, const rv_heads *k, const rv_heads *v, int B, int T,
                             const int32_t *d_pos, const int32_t *d_count, int32_t *d_err, void *stream) {
  set_error_message("");
  if (int rc = check_cache(cache, true)) return rc;
  if (int rc = check_rows(cache, B, T)) return rc;
  if (int rc = check_kv(cache, "k", k, B, T, false)) return rc;
  if (int rc = check_kv(cache, "v", v, B, T, false)) return rc;
  if (k->dtype != v->dtype) return op_fail(RV_EINVAL, "k and v differ in dtype");
  if (k->dtype != RV_F32 && k->dtype != cache->act_dtype) return op_fail(RV_EINVAL, "k and v must be act_dtype or RV_F32");
  if (int rc = check_index(d_pos, d_count, d_err)) return rc;
  if (int rc = check_memory(cache, k->data, v->data, d_pos, d_count, d_err)) return rc;
  Kv8Io io{heads_of(k), heads_of(v), B, T, d_pos, d_count, d_err};
  return launched("rv_kv8_append", launch_kv8_append(kv8_of(cache), io, k->dtype, static_cast<cudaStream_t>(stream)));
}

extern "C" int rv_kv8_read(const rv_kv8 *cache, const rv_heads *k_out, const rv_heads *v_out, int B, int T,
                           const int32_t *d_pos, const int32_t *d_count, int32_t *d_err, void *stream) {
  set_error_message("");
  if (int rc = check_cache(cache, true)) return rc;
  if (int rc = check_rows(cache, B, T)) return rc;
  if (!k_out && !v_out) return op_fail(RV_EINVAL, "null pointer");
  if (k_out)
    if (int rc = check_kv(cache, "k_out", k_out, B, T, true)) return rc;
  if (v_out)
    if (int rc = check_kv(cache, "v_out", v_out, B, T, true)) return rc;
  if (k_out && v_out && k_out->dtype != v_out->dtype) return op_fail(RV_EINVAL, "k_out and v_out differ in dtype");
  if (int rc = check_index(d_pos, d_count, d_err)) return rc;
  if (int rc = check_memory(cache, k_out ? k_out->data : nullptr, v_out ? v_out->data : nullptr, d_pos, d_count, d_err)) return rc;
  Kv8Io io{heads_of(k_out), heads_of(v_out), B, T, d_pos, d_count, d_err};
  return launched("rv_kv8_read", launch_kv8_read(kv8_of(cache), io, (k_out ? k_out : v_out)->dtype, static_cast<cudaStream_t>(stream)));
}

namespace {
int check_attention(const rv_kv8 *cache, int B, int T, int heads, bool pointers) {
  if (int rc = check_cache(cache, pointers)) return rc;
  if (int rc = check_rows(cache, B, T)) return rc;
  if (T > 16) return op_fail(RV_EINVAL, "T must be in 1..16");
  if (heads < 1 || heads > 65535 || heads % cache->n_kv_heads) return op_fail(RV_EINVAL, "query heads must be a multiple of n_kv_heads");
  return RV_OK;
}
}  // namespace

extern "C" size_t rv_kv8_attention_workspace(const rv_kv8 *cache, int B, int T, int n_heads) {
  set_error_message("");
  int n_sm = 0;
  if (check_attention(cache, B, T, n_heads, false) || sm_count(&n_sm)) return 0;
  return kv8_attention_work(kv8_of(cache), B, T, n_heads, n_sm);
}

extern "C" int rv_kv8_attention(const rv_kv8 *cache, const rv_heads *q, const rv_heads *out, int B, int T, float scale,
                                const int32_t *d_pos, const int32_t *d_count, float *d_lse, void *workspace,
                                size_t workspace_bytes, void *stream) {
  set_error_message("");
  if (int rc = check_cache(cache, true)) return rc;
  if (int rc = check_heads("q", q, B > 0 ? B : 1, T > 0 ? T : 1, cache->head_dim, false)) return rc;
  if (int rc = check_attention(cache, B, T, q->heads, false)) return rc;
  if (int rc = check_heads("out", out, B, T, cache->head_dim, true)) return rc;
  if (out->heads != q->heads) return op_fail(RV_EINVAL, "q and out differ in heads");
  if (q->dtype != cache->act_dtype && q->dtype != RV_F32) return op_fail(RV_EINVAL, "q must be act_dtype or RV_F32");
  if (out->dtype != cache->act_dtype && out->dtype != RV_F32) return op_fail(RV_EINVAL, "out must be act_dtype or RV_F32");
  if (!(scale - scale == 0.f)) return op_fail(RV_EINVAL, "scale must be finite");
  if (int rc = check_index(d_pos, d_count, reinterpret_cast<const int32_t *>(d_lse))) return rc;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return op_fail(RV_EINVAL, "workspace not 16-byte aligned");
  if (int rc = check_memory(cache, q->data, out->data, d_pos, d_count, d_lse)) return rc;
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  const Kv8 c = kv8_of(cache);
  const size_t need = kv8_attention_work(c, B, T, q->heads, n_sm);
  if (workspace_bytes < need) return op_fail(RV_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (need && !workspace) return op_fail(RV_EINVAL, "workspace: null pointer");
  if (int rc = check_device("workspace", workspace)) return rc;
  Kv8AttnArgs a{};
  a.c = c;
  a.q = heads_of(q);
  a.out = heads_of(out);
  a.H = q->heads; a.B = B; a.T = T;
  a.q_f32 = q->dtype == RV_F32;
  a.out_dtype = out->dtype;
  a.scale = scale;
  a.pos = d_pos; a.count = d_count;
  a.lse = d_lse;
  a.work = workspace;
  return launched("rv_kv8_attention", launch_kv8_attention(a, n_sm, static_cast<cudaStream_t>(stream)));
}
