// Attention of new tokens over a prefix that several rows share and over each
// row's own positions.
//
// out = (sum over the prefix + sum over the own positions) of w v / sum of w:
// three kernels leave states (reference m, sum l, weighted sum O) and join them.
// The own positions are the cache attention's (kv8_attention.cuh), which here
// leaves its rows' states; the prefix, whose fan x T x (H / Hkv) query rows of a KV
// head are taken together, is kv8_shared.cuh's.  That one needs no result of the
// first and may begin while it runs (it waits for the first at its end, so that the
// join, which waits for it, has both).  The cluster plan of the own positions lets
// it at once; the cut line's kernel as its last states are joined, and its join
// waits before it lets on, so there the two follow one another.  The plan goes by
// the own cache's room (kv8_attention.cu): 64 rows of 400 positions, 8 KV heads of
// 128, 70 us of the whole with room for 401, 74 to 75 with room for 1,024 to 16,384
// (line); 128 rows of up to 300, heads of 64, 56 with room up to 1,024, 73 from
// 4,096 on; 4 rows of 30 12.4 to 12.8 with room up to 1,024, 17.4 at 4,096, 18.7 at
// 16,384; 32 rows of 5 tokens, on the line throughout, 103.
#include "kv8_shared.cuh"

namespace rv {
namespace kv8s {

// ------------------------------------------------------------------ join

// A warp an output row: the prefix's parts, kJoin of them on their way at once,
// and the own positions' state.  (Measured with 5 and 10 at once, and with 2 or
// 4 warps a row: 72.7, 71.9, 73.3 and 73.5 us of the whole for 64 rows behind
// 32K positions, 55.2, 56.0, 58.7 and 60.1 for 16 prompts of 8 rows.)
constexpr int kJoin = 8;
template <int PER>
__device__ __forceinline__ void load_part(float (&x)[PER], const float *from) {
  if (PER == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(from);
    x[0] = v.x; x[1] = v.y; x[PER - 2] = v.z; x[PER - 1] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2 *>(from);
    x[0] = v.x; x[1] = v.y;
  }
}
template <int HD>
__global__ void __launch_bounds__(256) k_shared_join(const __grid_constant__ SharedArgs a, const __grid_constant__ Kv8AttnArgs f, const float *own,
                                                     const float2 *raw) {
  constexpr int PER = HD / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), bt = row / a.H, h = row - bt * a.H, b = bt / a.T, t = bt - b * a.T;
  if (row >= a.B * a.T * a.H || t >= row_count(a.count, b, a.T)) return;
  const int grp = a.H / a.c.Hkv, p = b / a.fan, g = h / grp, i = ((b - p * a.fan) * a.T + t) * grp + h - g * grp, group = i / kRows, rr = i - group * kRows;
  const int tiles = prefix_tiles(a, p), piece = a.line[a.P], begin = a.line[p] + (g * a.groups + group) * tiles;
  const float2 s0 = raw[row];
  float mm = s0.y == 0.f ? -INFINITY : s0.x, ll = s0.y, x[PER];
  load_part(x, own + (int64_t)row * HD + lane * PER);
  const int c0 = begin / piece, c1 = tiles ? (begin + tiles - 1) / piece : -1;
  const float *slots = a.slots + (size_t)((p * a.c.Hkv + g) * a.groups + group) * slot_floats(a.slot_rows, HD);
  for (int c = c0; c <= c1; c += kJoin) {
    float2 v[kJoin];
    float y[kJoin][PER], top = mm;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      v[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int d = 0; d < PER; ++d) y[j][d] = 0.f;
      if (c + j <= c1) {
        const float *s = slots + (size_t)(c + j) * slot_floats(a.slot_rows, HD);
        v[j] = *reinterpret_cast<const float2 *>(s + (size_t)a.slot_rows * HD + 2 * rr);
        load_part(y[j], s + (size_t)rr * HD + lane * PER);
      }
    }
#pragma unroll
    for (int j = 0; j < kJoin; ++j) top = fmaxf(top, v[j].x);
    const float base = top == -INFINITY ? 0.f : top, old = ex2(mm - base);
    ll *= old;
#pragma unroll
    for (int d = 0; d < PER; ++d) x[d] *= old;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const float e = ex2(v[j].x - base);
      ll = fmaf(v[j].y, e, ll);
#pragma unroll
      for (int d = 0; d < PER; ++d) x[d] = fmaf(y[j][d], e, x[d]);
    }
    mm = top;
  }
  float4 v;
  if (PER == 4) v = make_float4(x[0], x[1], x[PER - 2], x[PER - 1]);
  else v = make_float4(x[0], x[1], __shfl_down_sync(0xffffffffu, x[0], 1), __shfl_down_sync(0xffffffffu, x[1], 1));
  if (PER == 4 || !(lane & 1)) kv8a::write_out(f, b, t, h, lane * PER, v, mm, ll);
}
template <int HD>
cudaError_t launch_join(const SharedArgs &a, const Kv8AttnArgs &f, const float *own, const float2 *raw, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.T * a.H;
  return launch_k(k_shared_join<HD>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, 1, a, f, own, raw);
}

struct Plan {
  int P, rows, groups, slot_rows;
  int64_t units;
  size_t own_work, own_out, raw, line, slots, bytes;  // offsets
};
Plan plan_of(const Kv8 &cache, int B, int T, int fan, int H, int n_sm) {
  Plan s;
  if (fan > B) fan = B;
  s.P = (B + fan - 1) / fan;
  s.rows = fan * T * (H / cache.Hkv);
  s.groups = (s.rows + kRows - 1) / kRows;
  s.slot_rows = s.rows < kRows ? s.rows : kRows;
  s.units = (int64_t)s.P * cache.Hkv * s.groups;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  size_t at = 0;
  s.own_work = at; at += up(kv8_attention_work(cache, B, T, H, n_sm));
  s.own_out = at; at += up((size_t)B * T * H * cache.hd * 4);
  s.raw = at; at += up((size_t)B * T * H * 8);
  s.line = at; at += up((size_t)(s.P + 1) * 4);
  s.slots = at; at += up((size_t)(n_sm + s.units) * slot_floats(s.slot_rows, cache.hd) * 4);
  s.bytes = at + 240;  // the parts begin on 256-byte boundaries of a 16-byte aligned workspace
  return s;
}

cudaError_t launch_prefix_int8(const SharedArgs &a, int n_sm, cudaStream_t s) { return launch_prefix_fmt<RV_KV8_INT8>(a, n_sm, s); }

int check_shared(const rv_kv8 *prefix, const rv_kv8 *cache, int B, int T, int fan, int heads, bool pointers) {
  if (int rc = check_cache(prefix, pointers)) return rc;
  if (int rc = check_cache(cache, pointers)) return rc;
  if (prefix->n_kv_heads != cache->n_kv_heads || prefix->head_dim != cache->head_dim || prefix->act_dtype != cache->act_dtype)
    return op_fail(RV_EINVAL, "prefix and cache differ in n_kv_heads, head_dim or act_dtype");
  if (int rc = check_rows(cache, B, T)) return rc;
  if (T > 16) return op_fail(RV_EINVAL, "T must be in 1..16");
  if (fan < 1) return op_fail(RV_EINVAL, "fan must be at least 1");
  if ((B + (int64_t)fan - 1) / fan > prefix->max_batch) return op_fail(RV_EINVAL, "B / fan above the prefix's max_batch");
  if (heads < 1 || heads > 65535 || heads % cache->n_kv_heads) return op_fail(RV_EINVAL, "query heads must be a multiple of n_kv_heads");
  if ((int64_t)B * T * heads > INT32_MAX / 8) return op_fail(RV_EINVAL, "B x T x heads above 2^28");
  // what the kernels count in 32 bits: tiles of all units
  const int64_t f = fan < B ? fan : B, rows = f * T * (heads / cache->n_kv_heads), tiles = ((int64_t)prefix->max_seq + kTile - 1) / kTile;
  if ((B + f - 1) / f * cache->n_kv_heads * ((rows + kRows - 1) / kRows) * tiles > INT32_MAX / 2)
    return op_fail(RV_EINVAL, "B / fan x n_kv_heads x the prefix's max_seq too large");
  return RV_OK;
}

}  // namespace kv8s
}  // namespace rv

// ==================================================================== C ABI

using namespace rv;

extern "C" size_t rv_kv8_attention_shared_workspace(const rv_kv8 *prefix, const rv_kv8 *cache, int B, int T, int fan, int n_heads) {
  set_error_message("");
  int n_sm = 0;
  if (kv8s::check_shared(prefix, cache, B, T, fan, n_heads, false) || sm_count(&n_sm)) return 0;
  return kv8s::plan_of(kv8_of(cache), B, T, fan, n_heads, n_sm).bytes;
}

extern "C" int rv_kv8_attention_shared(const rv_kv8 *prefix, const rv_kv8 *cache, const rv_heads *q, const rv_heads *out, int B, int T, int fan,
                                       float scale, const int32_t *d_prefix_len, const int32_t *d_pos, const int32_t *d_count, float *d_lse,
                                       int32_t *d_err, void *workspace, size_t workspace_bytes, void *stream) {
  set_error_message("");
  if (int rc = check_cache(cache, true)) return rc;
  if (int rc = check_heads("q", q, B > 0 ? B : 1, T > 0 ? T : 1, cache->head_dim, false)) return rc;
  if (int rc = kv8s::check_shared(prefix, cache, B, T, fan, q->heads, true)) return rc;
  if (int rc = check_heads("out", out, B, T, cache->head_dim, true)) return rc;
  if (out->heads != q->heads) return op_fail(RV_EINVAL, "q and out differ in heads");
  if (q->dtype != cache->act_dtype && q->dtype != RV_F32) return op_fail(RV_EINVAL, "q must be act_dtype or RV_F32");
  if (out->dtype != cache->act_dtype && out->dtype != RV_F32) return op_fail(RV_EINVAL, "out must be act_dtype or RV_F32");
  if (!(scale - scale == 0.f)) return op_fail(RV_EINVAL, "scale must be finite");
  if (int rc = check_index(d_pos, d_count, reinterpret_cast<const int32_t *>(d_lse))) return rc;
  if (int rc = check_index(d_prefix_len, nullptr, d_err)) return rc;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return op_fail(RV_EINVAL, "workspace not 16-byte aligned");
  if (int rc = check_memory(cache, q->data, out->data, d_pos, d_count, d_lse)) return rc;
  if (int rc = check_memory(prefix, nullptr, nullptr, d_prefix_len, nullptr, d_err)) return rc;
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  const Kv8 c = kv8_of(cache);
  const kv8s::Plan plan = kv8s::plan_of(c, B, T, fan, q->heads, n_sm);
  if (workspace_bytes < plan.bytes) return op_fail(RV_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, plan.bytes);
  if (!workspace) return op_fail(RV_EINVAL, "workspace: null pointer");
  if (int rc = check_device("workspace", workspace)) return rc;
  char *work = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~(uintptr_t)255);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the own positions
  Kv8AttnArgs own{};
  own.c = c;
  own.q = heads_of(q);
  own.out = Heads{work + plan.own_out, (int64_t)T * q->heads * c.hd, (int64_t)q->heads * c.hd, c.hd};
  own.H = q->heads; own.B = B; own.T = T;
  own.q_f32 = q->dtype == RV_F32;
  own.out_dtype = RV_F32;
  own.round_out = out->dtype != RV_F32;
  own.scale = scale;
  own.pos = d_pos; own.count = d_count;
  own.raw = reinterpret_cast<float2 *>(work + plan.raw);
  own.work = work + plan.own_work;
  own.cluster = kv8_attention_cluster(c, B, T, own.H, n_sm, c.T);
  if (int rc = launched("rv_kv8_attention_shared", launch_kv8_attention(own, n_sm, s, 1))) return rc;
  // the prefix
  kv8s::SharedArgs a{};
  a.c = kv8_of(prefix);
  a.q = heads_of(q);
  a.q_f32 = own.q_f32;
  a.H = own.H; a.B = B; a.T = T; a.fan = fan < B ? fan : B; a.P = plan.P;
  a.rows = plan.rows; a.groups = plan.groups; a.slot_rows = plan.slot_rows;
  a.scale = scale;
  a.plen = d_prefix_len; a.count = d_count; a.err = d_err;
  a.line = reinterpret_cast<int32_t *>(work + plan.line);
  a.slots = reinterpret_cast<float *>(work + plan.slots);
  a.lo = c.act == RV_F16 || out->dtype == RV_F32;
  const cudaError_t e = a.c.fmt == RV_KV8_INT8 ? kv8s::launch_prefix_int8(a, n_sm, s) : kv8s::launch_prefix_e4m3(a, n_sm, s);
  if (int rc = launched("rv_kv8_attention_shared", e)) return rc;
  // the join
  Kv8AttnArgs f = own;
  f.out = heads_of(out);
  f.out_dtype = out->dtype;
  f.round_out = 0;
  f.raw = nullptr;
  f.lse = d_lse;
  const float *own_out = static_cast<const float *>(own.out.p);
  return launched("rv_kv8_attention_shared", c.hd == 64 ? kv8s::launch_join<64>(a, f, own_out, own.raw, s) : kv8s::launch_join<128>(a, f, own_out, own.raw, s));
}
