// Drawing the next token of each row from its logits.
//
// Weights are whole numbers, w = round(2^40 2^((x - max) log2(e) / temperature)):
// sums of them are exact in any order, so the draw is one function of the
// logits, the row's settings and the random number, however the work is cut.
// Everything below is counting on integers; only the weights are computed
// numbers, to some 2^-30 of themselves (see `weight`).
//
// A cluster of 1 to 8 blocks takes a row and keeps it in shared memory: logits
// are read once.  The order that top-k and top-p cut (descending logits, equal
// ones by index) is never made.  `select` finds the element at which a running
// count (top-k) or weight (top-p) reaches its target: a histogram of the keys'
// range over 2048 bins, the bin that the target falls into, a histogram of that
// bin's range, and so on down to one key; among elements of that one key the
// index decides, found by `locate`, the same search along the index that draws
// the token in the end.
#include <math.h>

#include "ops.cuh"

namespace rv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 2048, kLimbs = 3, kLimbBits = 14;
constexpr int kMaxVocab = 1 << 18, kMaxCluster = 8;
constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;

typedef unsigned long long u64;

// round(2^31 2^(i / 256)).
struct Pow2 {
  uint32_t t[256];
};

struct SampleArgs {
  const void *x;
  int64_t stride;  // of a row, in elements
  int B, V;
  int granules;  // 16-byte pieces of a block's share of a row
  int words;     // 32-bit words of a thread's share, odd
  const float *temperature, *top_p, *min_p, *u;
  const int32_t *top_k;
  int32_t *ids;
  float *logprob;
};

__device__ __forceinline__ unsigned cluster_size() {
  unsigned n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned n;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the cluster's block k's copy of a shared variable.
__device__ __forceinline__ uint32_t at_rank(const void *p, int k) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(k));
  return r;
}
__device__ __forceinline__ uint32_t load_rank(const uint32_t *p, int k) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at_rank(p, k)) : "memory");
  return v;
}
__device__ __forceinline__ u64 load_rank(const u64 *p, int k) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at_rank(p, k)) : "memory");
  return v;
}

// Keys ascend as logits descend; -infinity and NaN have none.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 is 0
  return b & 0x80000000u ? b : 0x7fffffffu - b;
}

// What a row's weights need: the largest logit and log2(e) / temperature in two
// parts.
struct Scale {
  float top, hi, lo;
  float least;  // logits below weigh nothing
};

// round(2^40 2^z), z = (x - top) c <= 0.  The difference is taken with its
// rounding error (two-sum), the product with its own (fma); z is cut into a
// multiple of 2^-8 and f, |f| <= 2^-9, and 2^z = 2^n T[i] 2^f with the table of
// 2^(i / 256) (Tang's method): 2^f - 1 below 2^-9.5 needs two terms of its
// series, the third is below 2^-31, and is added as a multiple of 2^-31.
__device__ __forceinline__ u64 weight(float x, const Scale &s, const uint32_t *table) {
  if (x == s.top) return 1ull << 40;  // also where both are infinite
  const float d = x - s.top, b = d - x, e = (x - (d - b)) - (s.top + b);
  const float p = d * s.hi, r = fmaf(d, s.lo, fmaf(e, s.hi, fmaf(d, s.hi, -p)));
  if (!(p > -42.f)) return 0;
  const float t = p + 49152.f;  // 1.5 2^15: the last bit is 2^-8
  const float f = (p - (t - 49152.f)) + r;
  const int zi = (int)(__float_as_uint(t) - 0x47400000u);  // 256 z, rounded
  const float g = f * fmaf(f, fmaf(f, 0.0555041087f, 0.240226507f), 0.693147181f);
  const int gi = (int)(__float_as_uint(g + 0.005859375f) - 0x3bc00000u);  // 1.5 2^-8: the last bit is 2^-31
  const uint32_t ti = table[zi & 255];
  const uint32_t w = ti + (uint32_t)(((long long)(int)(ti >> 1) * (2 * (long long)gi)) >> 31);
  const int n = zi >> 8;  // <= 0
  return ((((u64)w << 10) >> -n) + 1) >> 1;
}

struct alignas(16) Shared {  // the row's share follows, in 16-byte pieces
  uint32_t table[256];
  uint32_t hist[kLimbs][kBins];
  u64 warp[kWarps];
  u64 total[2];      // of this block, for the others to read; two, used in turn
  u64 before[2];     // results that one thread finds
  uint32_t found[4];
  float top;
  uint32_t least_index;
};

template <int DT>
struct Row {
  static constexpr int PER = DT == RV_F32 ? 1 : 2;  // elements of a word
  Shared *sh;
  const uint32_t *data;  // this block's share, as 32-bit words
  int words, n_words;    // of a thread, of the block
  int shift;             // index of the share's first element (may be negative: before the row)
  int rank, ranks, phase;

  __device__ __forceinline__ float value(uint32_t w, int i) const {
    if (DT == RV_F32) return __uint_as_float(w);
    return act_to_f((uint16_t)(w >> (16 * i)), DT == RV_BF16);
  }
  // f(x, index) for a thread's elements, in the order of the index.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int w0 = threadIdx.x * words, w1 = min(w0 + words, n_words);
    for (int w = w0; w < w1; ++w) {
      const uint32_t v = data[w];
#pragma unroll
      for (int i = 0; i < PER; ++i) f(value(v, i), w * PER + i + shift);
    }
  }

  // Sum over the block, before this thread and in all; every thread calls.
  __device__ __forceinline__ u64 scan(u64 mine, u64 &all) {
    u64 x = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh->warp[warp] = x;
    __syncthreads();
    u64 before = x - mine;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const u64 y = sh->warp[w];
      if (w < warp) before += y;
      all += y;
    }
    return before;
  }
  // The same over the cluster.
  __device__ __forceinline__ u64 scan_cluster(u64 mine, u64 &all) {
    u64 block;
    u64 before = scan(mine, block);
    if (ranks == 1) {
      all = block;
      return before;
    }
    phase ^= 1;
    if (threadIdx.x == 0) sh->total[phase] = block;
    cluster_sync();
    all = 0;
    for (int k = 0; k < ranks; ++k) {
      const u64 y = load_rank(&sh->total[phase], k);
      if (k < rank) before += y;
      all += y;
    }
    return before;
  }

  // The first element, by index, at which the running sum of measure(x, index)
  // reaches goal(sum of all): its index (by the block that has it: others
  // return -1), its measure and the sum of all.
  template <typename M, typename G>
  __device__ int locate(M measure, G goal, u64 &own, u64 &all) {
    u64 mine = 0;
    each([&](float x, int i) { mine += measure(x, i); });
    u64 before = scan_cluster(mine, all);
    const u64 to = goal(all);
    int got = -1;
    const bool here = before < to && to <= before + mine;
    const unsigned vote = __ballot_sync(0xffffffffu, here);
    if (vote) {  // this warp: its lanes share the elements of the thread that has it
      const int src = __ffs(vote) - 1, lane = threadIdx.x & 31;
      before = __shfl_sync(0xffffffffu, before, src);
      const int w0 = ((threadIdx.x & ~31) + src) * words, w1 = min(w0 + words, n_words);
      for (int w = w0; w < w1; w += 32) {
        u64 m[PER], sum = 0;
        const uint32_t v = w + lane < w1 ? data[w + lane] : 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          m[i] = w + lane < w1 ? measure(value(v, i), (w + lane) * PER + i + shift) : 0;
          sum += m[i];
        }
        u64 x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        u64 at = before + x - sum;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (at < to && to <= at + m[i]) {
            sh->found[0] = (w + lane) * PER + i;
            sh->before[0] = m[i];
          }
          at += m[i];
        }
        before = __shfl_sync(0xffffffffu, before + x, 31);
      }
      __syncwarp();
      got = (int)sh->found[0] + shift;
      own = sh->before[0];
    }
    return got;
  }

  // Cuts the order (ascending keys, then indices) at the first element at which
  // the running sum of measure(x, index) reaches goal(sum of all): elements
  // beyond it have key > key, or key == key and index > last.
  // Keys lie in [lo, hi].  MASS: measures up to 2^41, else 0 or 1.
  template <bool MASS, typename M, typename G>
  __device__ void select(uint32_t lo, uint32_t hi, M measure, G goal, uint32_t &key, int &last) {
    constexpr int L = MASS ? kLimbs : 1;
    u64 base = 0, to = 0;
    bool first = true;
    last = INT32_MAX;
    for (int round = 0; round < 4; ++round) {  // 3 at most: 11 bits of a key each
      const int sh_bits = max(0, 32 - __clz(hi - lo) - 11);  // (hi - lo) >> sh_bits < kBins
      __syncthreads();
      for (int i = threadIdx.x; i < L * kBins; i += kThreads) sh->hist[0][i] = 0;
      __syncthreads();
      each([&](float x, int i) {
        const uint32_t k = key_of(x);
        if (k < lo || k > hi) return;
        const u64 m = measure(x, i);
        const uint32_t bin = (k - lo) >> sh_bits;
#pragma unroll
        for (int l = 0; l < L; ++l) {
          const uint32_t part = L == 1 ? (uint32_t)m : (uint32_t)(m >> (kLimbBits * l)) & ((1u << kLimbBits) - 1);
          if (part) atomicAdd(&sh->hist[l][bin], part);
        }
      });
      if (ranks > 1) cluster_sync();
      else __syncthreads();
      // a block takes a run of the bins, a thread a run of those
      const int per_block = kBins / ranks, per = max(1, per_block / kThreads), b0 = rank * per_block + threadIdx.x * per;
      const bool live = threadIdx.x * per < per_block;
      u64 sums[kBins / kThreads], mine = 0;
#pragma unroll
      for (int j = 0; j < kBins / kThreads; ++j) {
        sums[j] = 0;
        if (j < per && live) {
          for (int k = 0; k < ranks; ++k)
#pragma unroll
            for (int l = 0; l < L; ++l) {
              const uint32_t *p = &sh->hist[l][b0 + j];
              sums[j] += (u64)(ranks > 1 ? load_rank(p, k) : *p) << (kLimbBits * l);
            }
        }
        mine += sums[j];
      }
      u64 all;
      u64 before = base + scan_cluster(mine, all);
      if (first) {
        to = goal(all);
        first = false;
        if (to > all) {  // nothing is cut (a goal above the sum: all stay)
          key = hi;
          return;
        }
      }
#pragma unroll
      for (int j = 0; j < kBins / kThreads; ++j) {
        if (j < per && live && before < to && to <= before + sums[j])
          for (int k = 0; k < ranks; ++k) {  // tell every block
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_rank(&sh->found[1], k)), "r"(b0 + j) : "memory");
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at_rank(&sh->before[1], k)), "l"(before) : "memory");
          }
        before += sums[j];
      }
      if (ranks > 1) cluster_sync();
      else __syncthreads();
      const uint32_t bin = sh->found[1];
      base = sh->before[1];
      lo += bin << sh_bits;
      hi = min(hi, lo + ((1u << sh_bits) - 1));
      if (lo >= hi) break;
    }
    key = lo;
    // several elements of this key: the index decides
    u64 own = 0, all;
    const int at = locate([&](float x, int i) { return key_of(x) == lo ? (u64)measure(x, i) : 0ull; }, [&](u64) { return to - base; }, own, all);
    if (at >= 0 && own)
      for (int k = 0; k < ranks; ++k)
        if ((threadIdx.x & 31) == 0) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_rank(&sh->found[2], k)), "r"(at) : "memory");
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    last = (int)sh->found[2];
  }
};

// floor(f x n), f in [0, 1] of at most 24 significant bits.
__device__ __forceinline__ u64 part_of(float f, u64 n, bool &exact) {
  const uint32_t b = __float_as_uint(f);
  const int e = (int)(b >> 23);
  const u64 m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int down = 150 - max(e, 1);  // f = m 2^-down
  const u64 lo = m * n, hi = __umul64hi(m, n);
  if (down >= 88) {  // m n < 2^88
    exact = lo == 0 && hi == 0;
    return 0;
  }
  if (down >= 64) {
    const int s = down - 64;
    exact = lo == 0 && (hi & ((1ull << s) - 1)) == 0;
    return hi >> s;
  }
  exact = (lo & ((1ull << down) - 1)) == 0;
  return (lo >> down) | (down ? hi << (64 - down) : 0);
}

// Smallest float not below d.
__device__ __forceinline__ float up32(double d) { return __double2float_ru(d); }

template <int DT>
__global__ void __launch_bounds__(kThreads) k_sample(const __grid_constant__ SampleArgs a, const __grid_constant__ Pow2 pow2) {
  extern __shared__ __align__(16) unsigned char sm[];
  Shared *sh = reinterpret_cast<Shared *>(sm);
  uint4 *data = reinterpret_cast<uint4 *>(sm + sizeof(Shared));
  constexpr int SIZE = DT == RV_F32 ? 4 : 2, EPG = 16 / SIZE;
  const int tid = threadIdx.x, ranks = (int)cluster_size(), rank = (int)cluster_rank(), b = blockIdx.x / ranks;
  for (int i = tid; i < 256; i += kThreads) sh->table[i] = pow2.t[i];
  pdl_wait();

  // ---- this block's share of the row: whole 16-byte pieces of memory; elements
  // beside the row are -infinity
  const char *row = static_cast<const char *>(a.x) + b * a.stride * SIZE;
  const char *base = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15);
  const int lead = (int)(row - base) / SIZE, g0 = rank * a.granules, total = (lead + a.V + EPG - 1) / EPG;
  const int mine = max(0, min(a.granules, total - g0));
  float top = -INFINITY;
  Row<DT> r{sh, reinterpret_cast<const uint32_t *>(data), a.words, mine * 4, g0 * EPG - lead, rank, ranks, 0};
  auto take = [&](uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < Row<DT>::PER; ++j) top = fmaxf(top, r.value(w[i], j));  // (fmaxf passes over NaN)
  };
  auto whole = [&](int g) { return (g0 + g) * EPG - lead >= 0 && (g0 + g + 1) * EPG - lead <= a.V; };
  constexpr int FLY = 8;
  for (int g = tid; g < mine; g += FLY * kThreads) {
    uint4 v[FLY];
#pragma unroll
    for (int k = 0; k < FLY; ++k) {
      const int q = g + k * kThreads;
      if (q < mine && whole(q)) v[k] = reinterpret_cast<const uint4 *>(base)[g0 + q];
    }
#pragma unroll
    for (int k = 0; k < FLY; ++k) {
      const int q = g + k * kThreads;
      if (q >= mine) continue;
      if (!whole(q)) {
        uint32_t w[4] = {};
        for (int e = 0; e < EPG; ++e) {
          const int i = (g0 + q) * EPG + e - lead;
          const uint32_t low = DT == RV_F32 ? 0xff800000u : DT == RV_BF16 ? 0xff80u : 0xfc00u;
          uint32_t x = low;
          if (i >= 0 && i < a.V) x = DT == RV_F32 ? reinterpret_cast<const uint32_t *>(row)[i] : reinterpret_cast<const uint16_t *>(row)[i];
          w[e * SIZE / 4] |= x << (8 * (e * SIZE % 4));
        }
        v[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      data[q] = v[k];
      take(v[k]);
    }
  }
  const float tau = a.temperature ? a.temperature[b] : 1.f, draw = a.u[b];
  const float p = a.top_p ? a.top_p[b] : 1.f, lowest = a.min_p ? a.min_p[b] : 0.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  // ---- the largest logit
  top = warp_max(top);
  if ((tid & 31) == 0) sh->warp[tid >> 5] = __float_as_uint(top);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, __uint_as_float((uint32_t)sh->warp[w]));
  if (ranks > 1) {
    if (tid == 0) sh->top = top;
    cluster_sync();
    for (int i = 0; i < ranks; ++i) top = fmaxf(top, __uint_as_float(load_rank(reinterpret_cast<const uint32_t *>(&sh->top), i)));
  }
  pdl_trigger();
  if (top == -INFINITY) {  // (the same in every block of the cluster)
    if (rank == 0 && tid == 0) {
      a.ids[b] = -1;
      if (a.logprob) a.logprob[b] = -INFINITY;
    }
    if (ranks > 1) cluster_sync();
    return;
  }

  // ---- the draw
  const bool greedy = !(tau > 0.f);
  Scale s;
  s.top = top;
  const double c = greedy ? 0.0 : fmin(kLog2e / (double)tau, 0x1p100);
  s.hi = (float)c;
  s.lo = (float)(c - (double)s.hi);
  s.least = -INFINITY;
  uint32_t key = 0xffffffffu;   // elements beyond are cut
  int last = INT32_MAX;         // at `key`, those of a higher index
  if (greedy || isinf(top)) s.least = top;
  else {
    // weights below half a unit are zero (a margin of a unit more)
    s.least = up32((double)top - 41.5 / c);
    if (lowest > 0.f) s.least = fmaxf(s.least, up32((double)top + (double)tau * log(fmin((double)lowest, 1.0))));
  }
  const float least = s.least;
  const float bottom = greedy || isinf(top) ? top : up32((double)top - 41.5 / c);  // of the order that top-k and top-p cut
  const uint32_t k_top = key_of(top), k_bottom = key_of(fmaxf(bottom, -3.402823466e38f));
  auto kept = [&](float x, int i) {
    const uint32_t q = key_of(x);
    return x >= bottom && (q < key || (q == key && i <= last));
  };
  const uint32_t *table = sh->table;
  if (greedy) {
    key = k_top;
    u64 own, all;
    const int at = r.locate([&](float x, int) { return x == top ? 1ull : 0ull; }, [](u64) { return 1ull; }, own, all);
    if (at >= 0 && (tid & 31) == 0) {
      a.ids[b] = at;
      if (a.logprob) a.logprob[b] = 0.f;
    }
    if (ranks > 1) cluster_sync();
    return;
  }
  if (k > 0 && k < a.V) {
    uint32_t kk;
    int kl;
    r.template select<false>(k_top, k_bottom, [&](float x, int) { return x >= bottom ? 1ull : 0ull; }, [&](u64) { return (u64)k; }, kk, kl);
    key = kk;
    last = kl;
  }
  if (p < 1.f) {
    const uint32_t key0 = key;
    const int last0 = last;
    uint32_t kk;
    int kl;
    r.template select<true>(
        k_top, min(k_bottom, key0),
        [&](float x, int i) {
          const uint32_t q = key_of(x);
          return x >= bottom && (q < key0 || (q == key0 && i <= last0)) ? weight(x, s, table) : 0ull;
        },
        [&](u64 all) {
          bool exact;
          const u64 n = part_of(fmaxf(p, 0.f), all, exact);
          return max(exact ? n : n + 1, 1ull);
        },
        kk, kl);
    if (kk < key || (kk == key && kl < last)) {
      key = kk;
      last = kl;
    }
  }
  u64 own = 0, all;
  const float f = draw >= 1.f ? 0x1.fffffep-1f : draw > 0.f ? draw : 0.f;
  const int at = r.locate([&](float x, int i) { return x >= least && kept(x, i) ? weight(x, s, table) : 0ull; },
                          [&](u64 n) {
                            bool exact;
                            return part_of(f, n, exact) + 1;
                          },
                          own, all);
  if (at >= 0 && (tid & 31) == 0) {
    a.ids[b] = at;
    if (a.logprob) a.logprob[b] = (float)(log((double)own) - log((double)all));
  }
  if (ranks > 1) cluster_sync();  // no block leaves while another reads its shared memory
}

template <int DT>
cudaError_t launch_t(const SampleArgs &a, const Pow2 &t, int ranks, cudaStream_t s, int pdl) {
  const size_t smem = sizeof(Shared) + (size_t)a.granules * 16;
  auto fn = k_sample<DT>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, fn, a, t);
  return e != cudaSuccess ? e : cudaGetLastError();
}

const Pow2 &pow2_table() {
  static const Pow2 table = [] {
    Pow2 t;
    for (int i = 0; i < 256; ++i) t.t[i] = (uint32_t)llrint(ldexp(exp2(i / 256.0), 31));
    return t;
  }();
  return table;
}

static_assert(sizeof(Shared) % 16 == 0, "the row's share is aligned");

}  // namespace

// Blocks of a row's cluster: as many as its logits need in shared memory, and
// more while the rows alone do not fill the GPU and a block keeps 8 KB.
int sample_cluster(int B, int64_t row_bytes, int n_sm) {
  int ranks = 1;
  while (ranks < kMaxCluster && row_bytes > (int64_t)ranks * 180000) ranks *= 2;
  while (ranks < kMaxCluster && (int64_t)B * ranks * 2 <= n_sm && row_bytes >= (int64_t)ranks * 16384) ranks *= 2;
  return ranks;
}

}  // namespace rv

// ==================================================================== C ABI

using namespace rv;

extern "C" int rv_sample(const void *d_logits, int dtype, int64_t stride, int B, int vocab, const float *d_temperature, const int32_t *d_top_k,
                         const float *d_top_p, const float *d_min_p, const float *d_u, int32_t *d_ids, float *d_logprob, void *stream) {
  set_error_message("");
  if (!d_logits || !d_u || !d_ids) return op_fail(RV_EINVAL, "d_logits, d_u or d_ids: null pointer");
  if (dtype != RV_F16 && dtype != RV_BF16 && dtype != RV_F32) return op_fail(RV_EINVAL, "logits: unknown dtype %d", dtype);
  if (B < 1 || B > 65535) return op_fail(RV_EINVAL, "B must be in 1..65535");
  if (vocab < 1 || vocab > kMaxVocab) return op_fail(RV_EINVAL, "vocab must be in 1..%d", kMaxVocab);
  if (stride < 0 || stride > (INT64_MAX >> 4) / B) return op_fail(RV_EINVAL, "stride out of range");
  const int size = dtype == RV_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(d_logits) & (size - 1)) return op_fail(RV_EINVAL, "logits not aligned to their type");
  const void *words[] = {d_temperature, d_top_k, d_top_p, d_min_p, d_u, d_ids, d_logprob};
  const char *names[] = {"d_temperature", "d_top_k", "d_top_p", "d_min_p", "d_u", "d_ids", "d_logprob"};
  for (int i = 0; i < 7; ++i)
    if (reinterpret_cast<uintptr_t>(words[i]) & 3u) return op_fail(RV_EINVAL, "%s not 4-byte aligned", names[i]);
  if (int rc = check_device("logits", d_logits)) return rc;
  for (int i = 0; i < 7; ++i)
    if (int rc = check_device(names[i], words[i])) return rc;
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  const int ranks = sample_cluster(B, (int64_t)vocab * size, n_sm);
  SampleArgs a{};
  a.x = d_logits; a.stride = stride; a.B = B; a.V = vocab;
  const int total = (vocab * size + 14) / 16 + 1;  // 16-byte pieces that a row can touch
  a.granules = (total + ranks - 1) / ranks;
  a.words = ((a.granules * 4 + kThreads - 1) / kThreads) | 1;
  a.temperature = d_temperature; a.top_k = d_top_k; a.top_p = d_top_p; a.min_p = d_min_p; a.u = d_u;
  a.ids = d_ids; a.logprob = d_logprob;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Pow2 &t = pow2_table();
  return launched("rv_sample", dtype == RV_F32    ? launch_t<RV_F32>(a, t, ranks, s, 1)
                               : dtype == RV_BF16 ? launch_t<RV_BF16>(a, t, ranks, s, 1)
                                                  : launch_t<RV_F16>(a, t, ranks, s, 1));
}
