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
// is written.  Scales begin on 4-byte boundaries only and go through registers:
// all threads share the words of an item, 8 loads each on their way, and an item
// has few of them (a thread a pair, as it was: 3 rows of up to 45,380 positions
// with 709 scales a head 50 us instead of 18.6).  Measured: 16 forks of 32,768
// positions of 8 KV heads of 128 (1.15 GB) in 185 us, 6.2 TB/s, 92% of a copy's
// rate; 48 ragged rows in a new order (123 MB) in 24.4 to 24.9 us, 73%: a short kernel,
// whose blocks begin with three dependent loads and end with their last items'
// stores; 3 rows of up to 45,380 positions (108 MB, some of it still in L2) in 15.3 us.
#include "async.cuh"
#include "ops.cuh"

namespace rv {
namespace {

constexpr int kThreads = 128, kMaxPairs = 1024;
constexpr uint32_t kFree = 0xffffffffu;

struct CopyArgs {
  Kv8 src, dst;
  int n;
  const int32_t *from, *to, *len;
  int32_t *err;
  int chunk;  // bytes of an item in each row, a multiple of 16
  int words;  // log2 of the 32-bit words of a scale item in each row
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
  // longest first, the lower index among equals: bytes (below 2^31) x 2^12 + n - i (at most 1024)
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

  // ---- items: [scales | tail | codes], each for K and V and every head (scales go
  // through registers, which takes its time: not at the end)
  const int lb = __ffs(a.dst.block) - 1, log_hd = hd == 64 ? 6 : 7, heads = 2 * a.dst.Hkv;
  const int tail_bytes = 4 * a.dst.block * hd, scale_bytes = (((s_most >> log_hd) + a.dst.block - 1) >> lb) * 4;
  const int n_codes = (s_most + a.chunk - 1) / a.chunk, n_tail = (tail_bytes + a.chunk - 1) / a.chunk;
  const int n_scale = (scale_bytes + (4 << a.words) - 1) / (4 << a.words);
  const int64_t end = (int64_t)heads * (n_codes + n_tail + n_scale);

  struct Item {
    int kind, kv, h, off;  // 0 scales, 1 tail, 2 codes; byte offset in a head's range
  };
  auto item = [&](int64_t i) {
    Item t;
    const int64_t c = (int64_t)heads * n_scale, d = c + (int64_t)heads * n_tail;
    t.kind = i < c ? 0 : i < d ? 1 : 2;
    const int per = t.kind == 0 ? n_scale : t.kind == 1 ? n_tail : n_codes;
    const int64_t j = i - (t.kind == 0 ? 0 : t.kind == 1 ? c : d), head = j / per;
    t.kv = (int)(head & 1);
    t.h = (int)(head >> 1);
    t.off = (int)(j - head * per) * (t.kind ? a.chunk : 4 << a.words);
    return t;
  };
  // where a row's bytes of the item begin, and how many of them pair p copies
  auto place = [&](const Kv8 &c, const Item &t, int row) {
    const int64_t r = (int64_t)row * c.Hkv + t.h;
    if (t.kind == 2) return c.codes[t.kv] + r * c.N * hd + t.off;
    if (t.kind == 1) return reinterpret_cast<uint8_t *>(c.tail[t.kv]) + r * tail_bytes + t.off;
    return reinterpret_cast<uint8_t *>(c.scale[t.kv] + r * (c.N >> lb)) + t.off;
  };
  auto bytes_of = [&](const Item &t, const Pair &p) {
    const int all = t.kind == 2 ? p.bytes : t.kind == 1 ? tail_bytes : (((p.bytes >> log_hd) + a.dst.block - 1) >> lb) * 4;
    return p.to < 0 ? 0 : min(max(all - t.off, 0), t.kind ? a.chunk : 4 << a.words);
  };
  auto load = [&](const Item &t, int buf) {
    unsigned char *to = sm + buf * buffer;
    uint32_t total = 0;
    if (t.kind)
      for (int i = tid; i < a.n; i += kThreads)
        if (pairs[i].lead == i) total += bytes_of(t, pairs[i]);
    bar_arrive_tx(&full[buf], total);
    if (t.kind) {
      for (int i = tid; i < a.n; i += kThreads) {
        const Pair p = pairs[i];
        const int n = p.lead == i ? bytes_of(t, p) : 0;
        if (n) bulk_load(to + (size_t)i * a.chunk, place(a.src, t, p.from), n, &full[buf]);
      }
    } else {  // scales begin on 4-byte boundaries: all threads, with some loads each on their way
      const int all = a.n << a.words, within = (1 << a.words) - 1;
      for (int k0 = tid; k0 < all; k0 += 8 * kThreads) {
        uint32_t v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int k = k0 + u * kThreads, i = k >> a.words, off = (k & within) * 4;
          v[u] = 0;
          if (k < all && pairs[i].lead == i && off < bytes_of(t, pairs[i])) v[u] = *reinterpret_cast<const uint32_t *>(place(a.src, t, pairs[i].from) + off);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int k = k0 + u * kThreads;
          if (k < all) *reinterpret_cast<uint32_t *>(to + (size_t)(k >> a.words) * a.chunk + (k & within) * 4) = v[u];
        }
      }
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
    const unsigned char *from = sm + buf * buffer;
    if (cur.kind) {
      for (int i = tid; i < a.n; i += kThreads) {
        const Pair p = pairs[i];
        const int n = bytes_of(cur, p);
        if (n) bulk_store(place(a.dst, cur, p.to), from + (size_t)p.lead * a.chunk, n);
      }
    } else {
      for (int k = tid; k < a.n << a.words; k += kThreads) {
        const int i = k >> a.words, off = (k - (i << a.words)) * 4;
        const Pair p = pairs[i];
        if (off < bytes_of(cur, p)) *reinterpret_cast<uint32_t *>(place(a.dst, cur, p.to) + off) = *reinterpret_cast<const uint32_t *>(from + (size_t)p.lead * a.chunk + off);
      }
      fence_async_smem();  // bulk copies take the buffer next
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
// (the kernel's limit is the same for every call: calls of several threads may come between one's setting of it and its launch)
constexpr int kMostSmem = 226 * 1024;
size_t copy_smem(int n, int chunk) { return 2 * (size_t)n * chunk + (size_t)n * sizeof(Pair) + (size_t)table_slots(n) * 16; }

}  // namespace

// The bytes of an item in each row: as much as brings 8 to 16 KB with all pairs,
// 512 bytes at least while two blocks of it find room in an SM, and so little
// that the blocks have a few items each.  (Blocks of 128 threads, 4 in an SM, 512
// bytes, 1, 2 and 4 KB: 16 forks of 32K positions 356, 185, 204, - us (2 in an SM
// at 2 KB); 8 rows in a new order 150, 78, 56, 55; 5 forks of 19K - , 83, 48, 46; 3
// rows in a new order - , 48, 27, 18.6.  48 rows in a new order, 256 and 512 bytes:
// 42.7 and 29.3 before scales had all threads, 24.4 at 512 since.  Blocks of 64
// threads: 183 us for the 16 forks, 26.1 for the 48 rows, 19.9 for the 3; of 256:
// 210, 25.2, 21.1.)
int kv8_copy_chunk(int n, int64_t row_bytes, int n_sm) {
  int chunk = 64;
  while (chunk < 8192 && (chunk < 512 ? copy_smem(n, 2 * chunk) <= 110000 : 2 * chunk * n <= 16384)) chunk *= 2;
  while (chunk > 1024 && row_bytes / chunk < 4 * n_sm) chunk /= 2;
  return chunk;
}

cudaError_t launch_kv8_copy(const Kv8 &src, const Kv8 &dst, int n, const int32_t *from, const int32_t *to, const int32_t *len, int32_t *err,
                            int n_sm, cudaStream_t s, int pdl) {
  CopyArgs a{src, dst, n, from, to, len, err, 0, 4, table_slots(n)};
  const int64_t row = (int64_t)2 * dst.Hkv * (src.N < dst.N ? src.N : dst.N) * dst.hd;
  a.chunk = kv8_copy_chunk(n, row, n_sm);
  while (4 << (a.words + 1) <= a.chunk && n << (a.words + 1) <= 1024) ++a.words;
  const size_t smem = copy_smem(n, a.chunk);
  cudaError_t e = cudaFuncSetAttribute(k_copy, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (e != cudaSuccess) return e;
  // (8 blocks in an SM instead of 4: one to four rows of 3 to 45K positions 18.6 -> 15.3, 17.7 -> 17.6, 6.5 -> 5.6 and
  // 6.9 -> 6.1 us; rows written at more places: 8 rows in a new order 55.9 -> 59.4, 16 forks 185 -> 198)
  const int room = smem > 100000 ? 1 : smem > 70000 ? 2 : smem > 52000 ? 3 : 4;
  const int per_sm = n <= 4 ? (int)(200000 / smem < 8 ? 200000 / smem : 8) : room;
  const int64_t items = row / a.chunk + 6 * dst.Hkv + 2 * dst.Hkv * (4 * dst.block * dst.hd / a.chunk + 1), most = (int64_t)per_sm * n_sm;
  return launch_k(k_copy, dim3((unsigned)(items < most ? items : most)), dim3(kThreads), smem, s, pdl, a);
}

}  // namespace rv

// ==================================================================== C ABI

using namespace rv;

namespace {

// The memory of a cache's six arrays; an end behind the last address is the last address.
struct Spans {
  uintptr_t from[6], to[6];
};
Spans spans_of(const rv_kv8 *c) {
  const void *p[6] = {c->k_codes, c->v_codes, c->k_scale, c->v_scale, c->k_tail, c->v_tail};
  const uint64_t rows = (uint64_t)c->max_batch * c->n_kv_heads, blocks = ((uint64_t)c->max_seq + c->block - 1) / c->block;
  const uint64_t row[3] = {blocks * c->block * c->head_dim, blocks * 4, (uint64_t)4 * c->block * c->head_dim};  // codes, scales, tail
  Spans s;
  for (int i = 0; i < 6; ++i) {
    s.from[i] = reinterpret_cast<uintptr_t>(p[i]);
    s.to[i] = rows > (UINTPTR_MAX - s.from[i]) / row[i / 2] ? UINTPTR_MAX : s.from[i] + rows * row[i / 2];
  }
  return s;
}
bool share_memory(const rv_kv8 *a, const rv_kv8 *b) {
  const Spans x = spans_of(a), y = spans_of(b);
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < 6; ++j)
      if (x.from[i] < y.to[j] && y.from[j] < x.to[i]) return true;
  return false;
}

}  // namespace

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
  const bool one = alike == 6 && src->max_seq == dst->max_seq && src->max_batch == dst->max_batch;
  if (!one && share_memory(src, dst))
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
