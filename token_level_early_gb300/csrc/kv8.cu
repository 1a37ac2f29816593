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
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
  return r;
}

// Scale of a block whose largest magnitude bits are m.
template <int ACT, int FMT>
__device__ __forceinline__ float block_scale(uint32_t m) {
  if (m >= inf_bits<ACT>()) return __int_as_float(0x7fc00000);
  const float t = act_to_f((uint16_t)m, ACT) / (FMT == RV_KV8_INT8 ? 127.f : 448.f);
  const float up = __uint_as_float((__float_as_uint(t) + 0xffffu) & 0xffff0000u);
  return fmaxf(up, kScaleMin);
}

// Four codes of two 16-bit pairs.  The quotient x / s is x * inv (inv = 1 / s)
// with one step of residual correction (Markstein): r = x - t s is exact where
// x / s is representable, as midpoints between codes are, and t + r inv then
// rounds to it; elsewhere the result is within a unit in the last place, far
// from any midpoint.  int8: adding 1.5 2^23 rounds to the nearest integer,
// ties to even, and leaves it in the low byte.
template <int ACT, int FMT>
__device__ __forceinline__ uint32_t code4(uint32_t v0, uint32_t v1, F2 neg_s, F2 inv) {
  float2 y[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? v1 : v0;
    const F2 x = f2(act_to_f((uint16_t)w, ACT), act_to_f((uint16_t)(w >> 16), ACT)), t = f2_mul(x, inv);
    F2 q = f2_fma(f2_fma(t, neg_s, x), inv, t);
    if (FMT == RV_KV8_INT8) q = f2_add(q, f2(12582912.f, 12582912.f));
    y[i] = f2_split(q);
  }
  if (FMT == RV_KV8_INT8) {
    const uint32_t a = __byte_perm(__float_as_uint(y[0].x), __float_as_uint(y[0].y), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(y[1].x), __float_as_uint(y[1].y), 0x0040);
    return __byte_perm(a, b, 0x5410);
  }
  return (uint32_t)__nv_cvt_float2_to_fp8x2(y[0], __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(y[1], __NV_SATFINITE, __NV_E4M3) << 16;
}

// 8 values of an input row as 16-bit pairs (RV_F32 rows are rounded).
template <int ACT, bool F32>
__device__ __forceinline__ uint4 load_row8(const void *base, int64_t off) {
  if (!F32) return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off);
  const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off);
  const float4 a = p[0], b = p[1];
  return make_uint4(pack_act2(a.x, a.y, ACT), pack_act2(a.z, a.w, ACT), pack_act2(b.x, b.y, ACT), pack_act2(b.z, b.w, ACT));
}

// ------------------------------------------------------------------ append

// A block of threads takes one cache block of one row, KV head and K or V: NV
// vectors of 8 values a thread, so block x head_dim / (8 NV) threads.  Originals
// before the row's first new position come from the tail, the others from the
// input; their largest magnitude gives the scale, and the codes of the block's
// present positions are written.  The threads of a row's first block also copy
// the row's last 2 x block new originals into the tail, after they have read
// what they need from there: no others read the tail.
template <int ACT, int FMT, bool F32, int HD, int NV>
__global__ void __launch_bounds__(512) k_append(Kv8 c, Kv8Io io, int log_block) {
  pdl_wait();
  pdl_trigger();
  constexpr int VR = HD / 8;  // vectors of a row
  __shared__ uint32_t red[16];
  const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y >> 1, kv = blockIdx.y & 1, block = 1 << log_block;
  const int pos = row_pos(io.pos, b), n = row_count(io.count, b, io.T);
  if (n == 0) return;
  const int end = (int)min((int64_t)pos + n, (int64_t)c.T);
  if (pos < 0 || end - pos < n) {  // not a position of the cache, or some tokens are not
    if (io.err && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) atomicOr(io.err, kKv8ErrPos);
    if (pos < 0 || pos >= c.T) return;
  }
  const int blk = (pos >> log_block) + blockIdx.x, p0 = blk << log_block;
  if (p0 >= end) return;
  const Heads &in = kv ? io.v : io.k;
  const int64_t row = (int64_t)b * c.Hkv + h;
  const int d = (tid % VR) * 8, p = p0 + tid / VR, step = block / NV;  // a thread's vectors are `step` positions apart
  uint16_t *tail = c.tail[kv] + row * (2 << log_block) * HD + d;
  const int64_t src = b * in.sb + h * in.sh + d;
  const int wrap = 2 * block - 1;
  const int64_t src_step = (int64_t)step * in.st;
  const bool all = p0 + block <= end;
  uint4 v[NV];
  if (p0 >= pos && all) {
    int64_t o = src + (int64_t)(p - pos) * in.st;
#pragma unroll
    for (int k = 0; k < NV; ++k, o += src_step) v[k] = load_row8<ACT, F32>(in.p, o);
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int q = p + k * step;
      v[k] = make_uint4(0, 0, 0, 0);
      if (q < pos) v[k] = *reinterpret_cast<const uint4 *>(tail + (q & wrap) * HD);
      else if (q < end) v[k] = load_row8<ACT, F32>(in.p, src + (int64_t)(q - pos) * in.st);
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) m = max_abs2(max_abs2(max_abs2(max_abs2(m, v[k].x), v[k].y), v[k].z), v[k].w);
  m = max(m & 0xffffu, m >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  if (blockDim.x > 32) {
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, red[(tid & 31) & ((blockDim.x >> 5) - 1)]);
  }
  const float s = block_scale<ACT, FMT>(m), inv = 1.f / s;
  const bool bad = !(s == s);
  const F2 ns2 = f2(-s, -s), inv2 = f2(inv, inv);
  uint8_t *codes = c.codes[kv] + (row * c.N + p) * HD + d;
#pragma unroll
  for (int k = 0; k < NV; ++k, codes += step * HD) {
    if (!all && p + k * step >= end) continue;
    uint2 o = make_uint2(code4<ACT, FMT>(v[k].x, v[k].y, ns2, inv2), code4<ACT, FMT>(v[k].z, v[k].w, ns2, inv2));
    if (bad) o = make_uint2(0, 0);
    *reinterpret_cast<uint2 *>(codes) = o;
  }
  if (tid == 0) c.scale[kv][row * (c.N >> log_block) + blk] = s;
  if (blockIdx.x == 0) {
    const int from = max(pos, end - 2 * block);
    for (int q = from + tid / VR; q < end; q += step)
      *reinterpret_cast<uint4 *>(tail + (q & wrap) * HD) = load_row8<ACT, F32>(in.p, src + (int64_t)(q - pos) * in.st);
  }
}

template <int ACT, int FMT, bool F32, int HD>
cudaError_t append_t(const Kv8 &c, const Kv8Io &io, cudaStream_t s, int pdl) {
  int log_block = 4;
  while (1 << log_block < c.block) ++log_block;
  const dim3 grid((io.T + c.block - 2) / c.block + 1, 2 * c.Hkv, io.B);  // blocks that T positions can touch
  // 4 vectors a thread where a call is short and its latency counts (or a
  // block has no more), 8 where it is long and a thread's fixed work counts
  if (io.T > 2 * c.block && c.block * HD >= 2048)
    return launch_k(k_append<ACT, FMT, F32, HD, 8>, grid, dim3(c.block * HD / 64), 0, s, pdl, c, io, log_block);
  return launch_k(k_append<ACT, FMT, F32, HD, 4>, grid, dim3(c.block * HD / 32), 0, s, pdl, c, io, log_block);
}

// ------------------------------------------------------------------ read

// 32 bytes in one store where they lie on a 32-byte boundary: two 16-byte
// stores of a warp would each write half sectors.
__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    uint4 *d = static_cast<uint4 *>(p);
    d[0] = make_uint4(v[0], v[1], v[2], v[3]);
    d[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// 16 codes -> values of the output type, rounded once.  A block whose largest
// possible value passes the type's range is limited to it.
template <int OUT, int FMT>
__device__ __forceinline__ void read16(uint4 w, float s, void *out, int64_t dst, bool wide) {
  const uint32_t cw[4] = {w.x, w.y, w.z, w.w};
  float x[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 lo, hi;
    if (FMT == RV_KV8_INT8) {  // byte ^ 0x80 = code + 128 under the exponent of 1024 is 1152 + code
      const uint32_t u = cw[i] ^ 0x80808080u, a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
      const __half2 bias = __half2half2(__ushort_as_half(0x6480));
      lo = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
      hi = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
    } else {
      lo = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)cw[i], __NV_E4M3));
      hi = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(cw[i] >> 16), __NV_E4M3));
    }
    const float2 f = __half22float2(lo), g = __half22float2(hi);
    const float2 u = f2_split(f2_mul(f2(f.x, f.y), f2(s, s))), v = f2_split(f2_mul(f2(g.x, g.y), f2(s, s)));
    x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = v.x; x[4 * i + 3] = v.y;
  }
  if (OUT == RV_F32) {
    uint32_t o[2][8];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i >> 3][i & 7] = __float_as_uint(x[i]);
    store32(static_cast<float *>(out) + dst, o[0], wide);
    store32(static_cast<float *>(out) + dst + 8, o[1], wide);
  } else {
    const float top = OUT == RV_F16 ? 65504.f : __uint_as_float(0x7f7f0000u);
    if (s * (FMT == RV_KV8_INT8 ? 127.f : 448.f) > top) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -top), top);
    }
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = pack_act2(x[2 * i], x[2 * i + 1], OUT);
    store32(static_cast<uint16_t *>(out) + dst, o, wide);
  }
}

// A block takes a run of one row's tokens and up to 256 / (HD / 16) heads of
// K or V; a thread keeps its 16 elements of one head and goes from token to
// token, four loads in flight.
constexpr int kReadItems = 4;
struct ReadGrid {
  int heads, groups;  // heads of a block, blocks of all heads
  bool wide;          // output rows on 32-byte boundaries
};
template <int OUT, int FMT, int HD>
__global__ void __launch_bounds__(256) k_read(Kv8 c, Kv8Io io, ReadGrid g) {
  pdl_wait();
  pdl_trigger();
  constexpr int CH = HD / 16;
  const int kv = blockIdx.y & 1, per = g.heads * CH, pass = blockDim.x / per, b = blockIdx.z;  // tokens of a pass
  const Heads &out = kv ? io.v : io.k;
  const int t0 = blockIdx.x * pass * kReadItems, t1 = min(row_count(io.count, b, io.T), t0 + pass * kReadItems);
  if (!out.p || t0 >= t1) return;
  const int pos = row_pos(io.pos, b), shift = __ffs(c.block) - 1;
  if (io.err && threadIdx.x == 0 && ((int64_t)pos + t0 < 0 || (int64_t)pos + t1 > c.T)) atomicOr(io.err, kKv8ErrPos);
  const int tl = threadIdx.x / per, r = threadIdx.x - tl * per, h = (blockIdx.y >> 1) * g.heads + r / CH, d = r % CH * 16;
  if (h >= c.Hkv) return;
  const int64_t row = (int64_t)b * c.Hkv + h, p0 = (int64_t)pos + t0 + tl;
  const uint8_t *src = c.codes[kv] + (row * c.N + p0) * HD + d;
  const float *scale = c.scale[kv] + row * (c.N >> shift);
  const int64_t dst = b * out.sb + (int64_t)(t0 + tl) * out.st + h * out.sh + d, step = pass * out.st;
  uint4 w[kReadItems];
  float s[kReadItems];
  bool ok[kReadItems];
#pragma unroll
  for (int k = 0; k < kReadItems; ++k) {
    const int64_t p = p0 + k * pass;
    ok[k] = t0 + tl + k * pass < t1 && p >= 0 && p < c.T;
    if (ok[k]) {
      w[k] = *reinterpret_cast<const uint4 *>(src + k * pass * HD);
      s[k] = scale[p >> shift];
    }
  }
#pragma unroll
  for (int k = 0; k < kReadItems; ++k)
    if (ok[k]) read16<OUT, FMT>(w[k], s[k], out.p, dst + k * step, g.wide);
}

template <int OUT, int FMT>
cudaError_t read_t(const Kv8 &c, const Kv8Io &io, cudaStream_t s, int pdl) {
  const int chunks = c.hd / 16, most = 256 / chunks;
  ReadGrid g;
  g.heads = c.Hkv < most ? c.Hkv : most;
  g.groups = (c.Hkv + g.heads - 1) / g.heads;
  g.wide = true;
  for (const Heads *h : {&io.k, &io.v})
    if (((reinterpret_cast<uintptr_t>(h->p) | (uintptr_t)h->sb * (OUT == RV_F32 ? 4 : 2) | (uintptr_t)h->st * (OUT == RV_F32 ? 4 : 2) |
          (uintptr_t)h->sh * (OUT == RV_F32 ? 4 : 2)) & 31u))
      g.wide = false;
  const int per = g.heads * chunks, pass = 256 / per, tokens = pass * kReadItems;
  auto fn = c.hd == 64 ? k_read<OUT, FMT, 64> : k_read<OUT, FMT, 128>;
  return launch_k(fn, dim3((io.T + tokens - 1) / tokens, 2 * g.groups, io.B), dim3(pass * per), 0, s, pdl, c, io, g);
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

cudaError_t launch_kv8_read(const Kv8 &c, const Kv8Io &io, int out_dtype, cudaStream_t s, int pdl) {
#define RV_R(OUT_) \
  if (out_dtype == OUT_) return c.fmt == RV_KV8_INT8 ? read_t<OUT_, RV_KV8_INT8>(c, io, s, pdl) : read_t<OUT_, RV_KV8_E4M3>(c, io, s, pdl);
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
  if (c->max_batch < 1 || c->max_batch > 65535 || c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->max_seq < 1)
    return op_fail(RV_EINVAL, "cache: max_batch in 1..65535, n_kv_heads in 1..1024 and max_seq > 0 are needed");
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
  // what the launches count in 32 bits: 16-token blocks of both K and V of every head
  if (((int64_t)T / 16 + 2) * B * 2 * c->n_kv_heads > INT32_MAX) return op_fail(RV_EINVAL, "B x T x n_kv_heads too large");
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
  return launched("rv_kv8_append", launch_kv8_append(kv8_of(cache), io, k->dtype, static_cast<cudaStream_t>(stream), 1));
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
  return launched("rv_kv8_read", launch_kv8_read(kv8_of(cache), io, (k_out ? k_out : v_out)->dtype, static_cast<cudaStream_t>(stream), 1));
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
  a.cluster = kv8_attention_cluster(c, B, T, a.H, n_sm, c.T);
  return launched("rv_kv8_attention", launch_kv8_attention(a, n_sm, static_cast<cudaStream_t>(stream), 1));
}
