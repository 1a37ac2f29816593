// Rows of the 8-bit K/V cache copied to other rows: a prompt forked to the rows
// that go on from it, beams put into a new order, finished rows closed up.
//
// All copies of a call happen at once, as if every source were read before any
// destination is written: the work is cut across the rows, not along them.  An
// item is one range of bytes of one KV head's codes (or tail, or scales) in
// ALL pairs' rows: a block brings the range of every source into shared memory
// and only then writes the destinations, so pairs may exchange rows in place,
// and a source that several pairs name is read once.
//
// Memory bounds it.  Bulk copies do the moving (each thread issues those of its
// pairs), two buffers keep an item's loads on their way while the one before it
// is written.  Measured: 16 forks of 32,768 positions of 8 KV heads of 128 (1.15 GB)
// in 193 us, 5.95 TB/s, 88% of a copy's rate; 48 ragged rows in a new order (123
// MB) in 29 us, 62%: a short kernel, whose blocks begin with three dependent
// loads and end with their last items' stores.
#include "async.cuh"
#include "ops.cuh"

namespace rv {
namespace {

constexpr int kThreads = 64, kMaxPairs = 1024;
constexpr uint32_t kFree = 0xffffffffu;

struct CopyArgs {
  Kv8 src, dst;
  int n;
  const int32_t *from, *to, *len;
  int32_t *err;
  int chunk;  // bytes of an item in each row, a multiple of 16
  int table;  // slots of the hash tables, a power of two above n
};

// What a thread knows of a pair: lives in shared memory.
struct Pair {
  int from, to, bytes, lead;  // codes' bytes of a head; the pair whose buffer holds the source's
};

// The slot of `key` in a table of keys (open addressing; it holds more slots than keys).
__device__ __forceinline__ int slot_of(uint32_t *keys, int mask, uint32_t key) {
  int s = (int)((key * 2654435761u) >> 16) & mask;
  for (int i = 0; i <= mask; ++i) {
    const uint32_t old = atomicCAS(&keys[s], kFree, key);
    if (old == kFree || old == key) break;
    s = (s + 1) & mask;
  }
  return s;
}

__global__ void __launch_bounds__(kThreads) k_copy(const __grid_constant__ CopyArgs a) {
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ __align__(8) uint64_t full[2];
  __shared__ int s_most;
  pdl_wait();
  fence_async_global();  // what earlier kernels wrote with ordinary stores is read by bulk copies
  const int tid = threadIdx.x, hd = a.dst.hd, mask = a.table - 1;
  const size_t buffer = (size_t)a.n * a.chunk;
  Pair *pairs = reinterpret_cast<Pair *>(sm + 2 * buffer);
  uint32_t *keys = reinterpret_cast<uint32_t *>(pairs + a.n);
  int *value = reinterpret_cast<int *>(keys + a.table);

  // ---- the pairs: of several with one destination the last counts; the
  // longest of those with one source leads (it loads for all)
  if (tid == 0) {
    bar_init(&full[0], kThreads);
    bar_init(&full[1], kThreads);
    bar_init_done();
    s_most = 0;
  }
  const int most = min(a.src.T, a.dst.T);
  int bad = 0;
  for (int i = tid; i < a.n; i += kThreads) {
    int from = a.from[i], to = a.to[i], len = a.len ? a.len[i] : most;
    if (from >= a.src.B || to >= a.dst.B || len > most) bad = 1;
    if (from < 0 || to < 0 || from >= a.src.B || to >= a.dst.B) from = to = -1;
    len = min(max(len, 0), most);
    pairs[i] = Pair{from, to, len * hd, i};
  }
  if (bad && a.err && blockIdx.x == 0) atomicOr(a.err, kKv8ErrPos);
  for (int i = tid; i < a.table; i += kThreads) { keys[i] = kFree; value[i] = -1; }
  __syncthreads();
  for (int i = tid; i < a.n; i += kThreads)
    if (pairs[i].to >= 0) {
      const int s = slot_of(keys, mask, pairs[i].to);
      pairs[i].lead = s;
      atomicMax(&value[s], i);
    }
  __syncthreads();
  for (int i = tid; i < a.n; i += kThreads)
    if (pairs[i].to >= 0 && value[pairs[i].lead] != i) pairs[i].to = -1;
  __syncthreads();
  for (int i = tid; i < a.table; i += kThreads) { keys[i] = kFree; value[i] = -1; }
  __syncthreads();
  // longest first, the lower index among equals: (bytes, n - i) in one number (bytes < 2^38 / 2^6 in units of 64)
  unsigned long long *best = reinterpret_cast<unsigned long long *>(value + a.table);
  for (int i = tid; i < a.table; i += kThreads) best[i] = 0;
  __syncthreads();
  for (int i = tid; i < a.n; i += kThreads)
    if (pairs[i].to >= 0) {
      const int s = slot_of(keys, mask, pairs[i].from);
      pairs[i].lead = s;
      atomicMax(&best[s], (unsigned long long)pairs[i].bytes << 12 | (unsigned)(a.n - i));
      atomicMax(&s_most, pairs[i].bytes);
    }
  __syncthreads();
  for (int i = tid; i < a.n; i += kThreads)
    if (pairs[i].to >= 0) pairs[i].lead = a.n - (int)(best[pairs[i].lead] & 0xfff);
  __syncthreads();

  // ---- items: [codes | tail | scales], each for K and V and every head
  const int lb = __ffs(a.dst.block) - 1, log_hd = hd == 64 ? 6 : 7, heads = 2 * a.dst.Hkv;
  const int tail_bytes = 4 * a.dst.block * hd, scale_bytes = (((s_most >> log_hd) + a.dst.block - 1) >> lb) * 4;
  const int n_codes = (s_most + a.chunk - 1) / a.chunk, n_tail = (tail_bytes + a.chunk - 1) / a.chunk;
  const int n_scale = (scale_bytes + a.chunk - 1) / a.chunk;
  const int64_t end = (int64_t)heads * (n_codes + n_tail + n_scale);

  struct Item {
    int kind, kv, h, off;  // 0 codes, 1 tail, 2 scales; byte offset in a head's range
  };
  auto item = [&](int64_t i) {
    Item t;
    const int64_t c = (int64_t)heads * n_codes, d = c + (int64_t)heads * n_tail;
    t.kind = i < c ? 0 : i < d ? 1 : 2;
    const int per = t.kind == 0 ? n_codes : t.kind == 1 ? n_tail : n_scale;
    const int64_t j = i - (t.kind == 0 ? 0 : t.kind == 1 ? c : d), head = j / per;
    t.kv = (int)(head & 1);
    t.h = (int)(head >> 1);
    t.off = (int)(j - head * per) * a.chunk;
    return t;
  };
  // where a row's bytes of the item begin, and how many of them pair p copies
  auto place = [&](const Kv8 &c, const Item &t, int row) {
    const int64_t r = (int64_t)row * c.Hkv + t.h;
    if (t.kind == 0) return c.codes[t.kv] + r * c.N * hd + t.off;
    if (t.kind == 1) return reinterpret_cast<uint8_t *>(c.tail[t.kv]) + r * tail_bytes + t.off;
    return reinterpret_cast<uint8_t *>(c.scale[t.kv] + r * (c.N >> lb)) + t.off;
  };
  auto bytes_of = [&](const Item &t, const Pair &p) {
    const int all = t.kind == 0 ? p.bytes : t.kind == 1 ? tail_bytes : (((p.bytes >> log_hd) + a.dst.block - 1) >> lb) * 4;
    return p.to < 0 ? 0 : min(max(all - t.off, 0), a.chunk);
  };
  auto load = [&](const Item &t, int buf) {
    unsigned char *to = sm + buf * buffer;
    uint32_t total = 0;
    if (t.kind < 2)
      for (int i = tid; i < a.n; i += kThreads)
        if (pairs[i].lead == i) total += bytes_of(t, pairs[i]);
    bar_arrive_tx(&full[buf], total);
    for (int i = tid; i < a.n; i += kThreads) {
      const Pair p = pairs[i];
      const int n = p.lead == i ? bytes_of(t, p) : 0;
      if (n == 0) continue;
      const uint8_t *from = place(a.src, t, p.from);
      if (t.kind < 2) bulk_load(to + (size_t)i * a.chunk, from, n, &full[buf]);
      else  // scales begin on 4-byte boundaries
        for (int k = 0; k < n; k += 4) *reinterpret_cast<uint32_t *>(to + (size_t)i * a.chunk + k) = *reinterpret_cast<const uint32_t *>(from + k);
    }
  };

  int64_t at = blockIdx.x;
  if (at >= end) return;
  Item cur = item(at);
  load(cur, 0);
  bool ok = true;
  for (int k = 0;; ++k) {
    const int buf = k & 1;
    const int64_t next = at + gridDim.x;
    const bool more = next < end;
    Item nxt = cur;
    if (more) {
      nxt = item(next);
      bulk_wait_read<0>();  // the other buffer's stores have left it
      __syncthreads();
      load(nxt, buf ^ 1);
    }
    if (!bar_wait(&full[buf], (k >> 1) & 1)) {
      ok = false;
      bar_wait(&full[buf], (k >> 1) & 1);
      if (more) bar_wait(&full[buf ^ 1], ((k + 1) >> 1) & 1);
    }
    if (__syncthreads_or(!ok)) break;  // (also: every thread's scales are in place)
    for (int i = tid; i < a.n; i += kThreads) {
      const Pair p = pairs[i];
      const int n = bytes_of(cur, p);
      if (n == 0) continue;
      uint8_t *to = place(a.dst, cur, p.to);
      const unsigned char *from = sm + buf * buffer + (size_t)p.lead * a.chunk;
      if (cur.kind < 2) bulk_store(to, from, n);
      else
        for (int j = 0; j < n; j += 4) *reinterpret_cast<uint32_t *>(to + j) = *reinterpret_cast<const uint32_t *>(from + j);
    }
    bulk_commit();
    if (!more) break;
    at = next;
    cur = nxt;
  }
  if (!ok && a.err) atomicOr(a.err, kErrWait);
  pdl_trigger();
  bulk_wait<0>();
}

int table_slots(int n) {
  int t = 4;
  while (t < 2 * n) t *= 2;
  return t;
}
size_t copy_smem(int n, int chunk) { return 2 * (size_t)n * chunk + (size_t)n * sizeof(Pair) + (size_t)table_slots(n) * 16; }

}  // namespace

// The bytes of an item in each row: as much as brings 8 to 16 KB with all pairs,
// 512 bytes at least while two blocks of it find room in an SM, and so little
// that the blocks have a few items each.  (16 forks of 32K positions, 48 rows in
// a new order: 1 KB and 512 bytes 197.7 and 29.2 us with 128 threads, 193.2 and
// 29.3 with 64, 204.8 and 30.0 with 256; 2 KB and 512 bytes 214.7; 1 KB and 256
// bytes 196.7 and 42.7; 512 and 128 bytes 220.4 and 42.9; 4 blocks in an SM 197.7,
// 3 250.5, 5 207.0.)
int kv8_copy_chunk(int n, int64_t row_bytes, int n_sm) {
  int chunk = 64;
  while (chunk < 8192 && (chunk < 512 ? copy_smem(n, 2 * chunk) <= 110000 : 2 * chunk * n <= 16384)) chunk *= 2;
  while (chunk > 1024 && row_bytes / chunk < 4 * n_sm) chunk /= 2;
  return chunk;
}

cudaError_t launch_kv8_copy(const Kv8 &src, const Kv8 &dst, int n, const int32_t *from, const int32_t *to, const int32_t *len, int32_t *err,
                            int n_sm, cudaStream_t s, int pdl) {
  CopyArgs a{src, dst, n, from, to, len, err, 0, table_slots(n)};
  const int64_t row = (int64_t)2 * dst.Hkv * (src.N < dst.N ? src.N : dst.N) * dst.hd;
  a.chunk = kv8_copy_chunk(n, row, n_sm);
  const size_t smem = copy_smem(n, a.chunk);
  cudaError_t e = cudaFuncSetAttribute(k_copy, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int per_sm = smem > 100000 ? 1 : smem > 70000 ? 2 : smem > 52000 ? 3 : 4;
  const int64_t items = row / a.chunk + 6 * dst.Hkv + 2 * dst.Hkv * (4 * dst.block * dst.hd / a.chunk + 1), most = (int64_t)per_sm * n_sm;
  return launch_k(k_copy, dim3((unsigned)(items < most ? items : most)), dim3(kThreads), smem, s, pdl, a);
}

}  // namespace rv

// ==================================================================== C ABI

using namespace rv;

extern "C" int rv_kv8_copy(const rv_kv8 *src, const rv_kv8 *dst, int n, const int32_t *d_from, const int32_t *d_to, const int32_t *d_len,
                           int32_t *d_err, void *stream) {
  set_error_message("");
  if (int rc = check_cache(src, true)) return rc;
  if (int rc = check_cache(dst, true)) return rc;
  if (src->n_kv_heads != dst->n_kv_heads || src->head_dim != dst->head_dim || src->block != dst->block || src->format != dst->format ||
      src->act_dtype != dst->act_dtype)
    return op_fail(RV_EINVAL, "src and dst differ in n_kv_heads, head_dim, block, format or act_dtype");
  if (n < 1 || n > kMaxPairs) return op_fail(RV_EINVAL, "n must be in 1..%d", kMaxPairs);
  if (!d_from || !d_to) return op_fail(RV_EINVAL, "d_from or d_to: null pointer");
  if (int rc = check_index(d_from, d_to, d_err)) return rc;
  if (int rc = check_index(d_len, nullptr, nullptr)) return rc;
  const int alike = (src->k_codes == dst->k_codes) + (src->v_codes == dst->v_codes) + (src->k_scale == dst->k_scale) +
                    (src->v_scale == dst->v_scale) + (src->k_tail == dst->k_tail) + (src->v_tail == dst->v_tail);
  if (alike != 0 && (alike != 6 || src->max_seq != dst->max_seq || src->max_batch != dst->max_batch))
    return op_fail(RV_EINVAL, "src and dst share a part of their memory");
  if ((int64_t)(src->max_seq < dst->max_seq ? src->max_seq : dst->max_seq) * dst->head_dim > INT32_MAX - 8192)
    return op_fail(RV_EINVAL, "max_seq x head_dim of both above 2^31");
  if (int rc = check_memory(src, nullptr, nullptr, d_from, d_to, d_len)) return rc;
  if (int rc = check_memory(dst, nullptr, nullptr, nullptr, nullptr, d_err)) return rc;
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  return launched("rv_kv8_copy",
                  launch_kv8_copy(kv8_of(src), kv8_of(dst), n, d_from, d_to, d_len, d_err, n_sm, static_cast<cudaStream_t>(stream), 1));
}
