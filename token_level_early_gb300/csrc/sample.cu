// Drawing the next token of each row from its logits.
//
// Weights are whole numbers, w = round(2^40 2^((x - max) log2(e) / temperature)):
// sums of them are exact in any order, so the draw is one function of the
// logits, the row's settings and the random number, however the work is cut.
// Everything below is counting on integers; only the weights are computed
// numbers, to some 2^-29 of themselves (see `weight`).
//
// A cluster of 1 to 8 blocks takes a row and keeps it in shared memory: logits
// are read once.  The order that top-k and top-p cut (descending logits, equal
// ones by index) is never made.  bf16 has few values: counting them gives the
// weight up to each exactly, the border is a value, and elements that have it stay
// by index (`by_values`).  Other types: a count of the logits in 4096 steps of
// their distance to the largest gives the step of top-k's border; with the sum of
// their places inside the step it gives bounds of each step's weight, to 10^-4,
// and so the step or two that top-p's border can lie in.  One pass then sums the
// exact weights of the steps before (and behind, for the total) and lists the
// elements inside, some few, which one block ranks (`resolve`).  Where the list
// would be too long, as with many equal logits, `select` finds the border among
// all: a histogram over their keys' range, then over the bin that holds the
// border, down to one key, where the index decides.  The draw itself is a prefix
// sum along the index (`locate`).
//
// What bounds it: instructions (a weight is some 25), shared-memory atomics and
// the cluster's barriers, not memory.  64 rows of 128,256 fp32 with settings of
// their own: 58 to 71 us by the settings (33 MB: 0.5 TB/s); of a block's 50,000 cycles, two in an SM,
// loading takes 5,000, counts 9,000, bounds 13,000 in five barriers, exact weights
// 5,500, the border 8,000, the draw 4,000.  256 rows of bf16 under top-p: 169 to 188 us by the rows;
// counting takes a third of it (14.7 cycles a warp's 32 atomics, banks at random;
// two copies of the counts: 198 us instead of 195, with blocks of 512).  200 rows
// of 50,257 fp16 with a temperature alone: 37 us; of 80 warp instructions for 32
// elements the weight (one for each, the draw adds those of a thread or so) is
// some 25, the rest loading, the maximum, the loops and the cut's tests, which are
// made although nothing is cut.  One row of 32,000: 16 to 18 us, eight blocks and
// nine barriers.
#include <math.h>

#include "ops.cuh"

namespace rv {
namespace {

constexpr int kBins = 2048, kLimbs = 3, kLimbBits = 14;
constexpr int kSteps = 4096, kList = 1024;  // steps of the first count; elements that are listed at most
constexpr float kOctaves = 41.9f;          // below the largest: weights beyond are zero
constexpr int kMaxVocab = 1 << 18, kMaxCluster = 8;
constexpr double kLog2e = 1.4426950408889634074;

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
// The two halves of the first one: that all blocks have begun.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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
__device__ __forceinline__ int add_rank(const int *p, int k, int v) {
  int old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(old) : "r"(at_rank(p, k)), "r"(v) : "memory");
  return old;
}

// Keys ascend as logits descend; -infinity and NaN have none.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 is 0
  return b & 0x80000000u ? b : 0x7fffffffu - b;
}

// x c cut into a multiple of 2^-8 (its bits, from the rounding constant on) and
// a rest: c = hi + lo.
struct Parts {
  int n;
  float f;
};
__device__ __forceinline__ Parts parts_of(float x, float hi, float lo) {
  const float t = fmaf(x, hi, 49152.f);  // 1.5 2^15: the last bit is 2^-8
  return Parts{(int)__float_as_uint(t), fmaf(x, lo, fmaf(x, hi, 49152.f - t))};
}
// What a row's weights need: the largest logit, c = log2(e) / temperature in two
// parts, and the parts of top c.
struct Scale {
  float top, hi, lo;
  Parts at;
};
__device__ __forceinline__ Scale scale_of(float top, float tau) {
  constexpr float L = 0x1.715476p+0f, LL = 0x1.4ae0cp-26f;  // log2(e) = L + LL to 2^-52
  Scale s;
  s.top = top;
  s.hi = __fdiv_rn(L, tau);
  s.lo = __fdiv_rn(fmaf(-s.hi, tau, L) + LL, tau);
  s.at = parts_of(top, s.hi, s.lo);
  return s;
}

// round(2^40 2^z), z = (x - top) c <= 0.  x c is cut into a multiple of 2^-8,
// taken off exactly by fma, and a rest; with top's the rest is f, |f| <= 2^-8,
// and 2^z = 2^n T[i] 2^f with the table of 2^(i / 256) (Tang's method): 2^f - 1
// by three terms of its series, the fourth is below 2^-38, as a multiple of
// 2^-30.  |x c| is below 2^13 (`fits`), else the plain form.
__device__ __forceinline__ u64 weight(float x, const Scale &s, const uint32_t *table) {
  const Parts q = parts_of(x, s.hi, s.lo);
  const float f = q.f - s.at.f;
  const int zi = q.n - s.at.n;  // 256 z, nearly
  const float g = fmaf(f, fmaf(f, fmaf(f, 0.0555041087f, 0.240226507f), 0.693147181f), 0.01171875f);
  const int gi = (int)(__float_as_uint(g) - 0x3c400000u);  // 1.5 2^-7: the last bit is 2^-30
  const uint32_t ti = table[zi & 255];
  const u64 w = ti + (u64)(((long long)(int)(ti >> 1) * gi) >> 29);  // (f = 2^-8 behind the last T: 2^32)
  const int down = min(max(-(zi >> 8), 0), 63);
  return x == s.top ? 1ull << 40 : (((w << 10) >> down) + 1) >> 1;
}
__device__ __forceinline__ bool fits(float top, float tau) { return tau > 0x1p-20f && tau < 0x1p20f && fabsf(top) < 5000.f * tau; }
// The same for any finite or infinite numbers, in 64 bits.
__device__ __noinline__ u64 weight_plain(float x, float top, float tau) {
  if (x == top) return 1ull << 40;
  const double z = ((double)x - (double)top) * (kLog2e / (double)tau);
  return z > -42.0 ? (u64)rint(exp2(z + 40.0)) : 0;  // (NaN: 0)
}

template <int NT>  // threads of a block
struct alignas(16) Shared {  // the row's share follows, in 16-byte pieces
  uint32_t table[256];
  union {
    uint32_t hist[2 * kSteps];  // of the first count: elements, and their places; of `select`: kLimbs x kBins
    u64 value[kSteps];          // bf16: the weights of its values
    struct {
      u64 order[kList], weight[kList];  // in the first block: all listed elements (the counts have been read by then)
    };
  };
  uint32_t list[kList];
  u64 add[NT];
  u64 warp[4 * NT / 32];
  u64 total[2][32];  // of all blocks, 8 for each sum; two, used in turn
  u64 small;         // bf16: the weight of the small values, in the block that has their place
  u64 before[4];     // results that one thread finds
  uint32_t found[8];
  float least;
  int listed, gathered;
};
static_assert(kLimbs * kBins <= 2 * kSteps, "select's bins fit");
static_assert(sizeof(Shared<512>) + 66032 <= 113 * 1024, "two blocks in an SM");
static_assert(sizeof(Shared<1024>) + 132032 <= 227 * 1024, "one block in an SM");
static_assert(sizeof(Shared<512>) % 16 == 0 && sizeof(Shared<1024>) % 16 == 0, "the row's share is aligned");

// Sums, and places in them, over a block.
template <typename T, int N, int NT>
__device__ __forceinline__ void block_scan(Shared<NT> *sh, const T (&mine)[N], T (&before)[N], T (&all)[N]) {
  constexpr int W = NT / 32;
  static_assert(N <= 4 && sizeof(T) <= 8, "room for the warps' sums");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    T x = mine[n];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    before[n] = x - mine[n];
    if (lane == 31) reinterpret_cast<T *>(&sh->warp[n * W])[warp] = x;
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {  // every warp adds the warps' sums up for itself
    T x = lane < W ? reinterpret_cast<T *>(&sh->warp[n * W])[lane] : T(0);
    const T own = x;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    before[n] += __shfl_sync(0xffffffffu, x - own, warp);
    all[n] = __shfl_sync(0xffffffffu, x, W - 1);
  }
}

template <int DT, int NT>
struct Row {
  static constexpr int PER = DT == RV_F32 ? 1 : 2;  // elements of a word
  Shared<NT> *sh;
  const uint32_t *data;  // this block's share, as 32-bit words
  int words, n_words;    // of a thread, of the block
  int shift;             // index of the share's first element (may be negative: before the row)
  int rank, ranks, phase;

  __device__ __forceinline__ float value(uint32_t w, int i) const {
    if (DT == RV_F32) return __uint_as_float(w);
    return act_to_f((uint16_t)(w >> (16 * i)), DT == RV_BF16);
  }
  // f(bits, element) for a thread's 16-bit elements.
  template <typename F>
  __device__ __forceinline__ void each_bits(F f) const {
    const int w0 = threadIdx.x * words, w1 = min(w0 + words, n_words);
#pragma unroll 2
    for (int w = w0; w < w1; ++w) {
      const uint32_t v = data[w];
      f((uint16_t)v, 2 * w);
      f((uint16_t)(v >> 16), 2 * w + 1);
    }
  }
  __device__ __forceinline__ float at(int e) const { return value(data[e / PER], e % PER); }
  // f(x, element) for a thread's elements, in the order of the index; an element's index is its number + shift.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int w0 = threadIdx.x * words, w1 = min(w0 + words, n_words);
#pragma unroll 2
    for (int w = w0; w < w1; ++w) {
      const uint32_t v = data[w];
#pragma unroll
      for (int i = 0; i < PER; ++i) f(value(v, i), w * PER + i);
    }
  }
  __device__ __forceinline__ void sync() const {
    if (ranks > 1) cluster_sync();
    else __syncthreads();
  }
  // Every block of the cluster gets v in its found[i].
  __device__ __forceinline__ void tell(int i, uint32_t v) const {
    for (int k = 0; k < ranks; ++k) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_rank(&sh->found[i], k)), "r"(v) : "memory");
  }
  // Every block's found[i] becomes the smallest of what it is told.
  __device__ __forceinline__ void least(int i, uint32_t v) const {
    for (int k = 0; k < ranks; ++k)
      asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(at_rank(&sh->found[i], k)), "r"(v) : "memory");
  }
  __device__ __forceinline__ void tell(int i, u64 v) const {
    for (int k = 0; k < ranks; ++k) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at_rank(&sh->before[i], k)), "l"(v) : "memory");
  }

  // N sums over the cluster, each before this thread and in all; every thread calls.
  template <typename T, int N>
  __device__ __forceinline__ void scan(const T (&mine)[N], T (&before)[N], T (&all)[N]) {
    block_scan(sh, mine, before, all);
    if (ranks == 1) return;
    // a lane a block and sum, 8 lanes of blocks for each: the first warp tells every block, then all read their own
    phase ^= 1;
    const int n = (threadIdx.x & 31) >> 3, k = threadIdx.x & 7;
    if (threadIdx.x < 8 * N && k < ranks) {
      u64 bits = 0;
#pragma unroll
      for (int m = 0; m < N; ++m)
        if (m == n) *reinterpret_cast<T *>(&bits) = all[m];
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at_rank(&sh->total[phase][8 * n + rank], k)), "l"(bits) : "memory");
    }
    cluster_sync();
    u64 bits = n < N && k < ranks ? sh->total[phase][8 * n + k] : 0;
    T x = *reinterpret_cast<T *>(&bits), y = k < rank ? x : T(0);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
    }
#pragma unroll
    for (int m = 0; m < N; ++m) {
      all[m] = __shfl_sync(0xffffffffu, x, 8 * m);
      before[m] += __shfl_sync(0xffffffffu, y, 8 * m);
    }
  }
  __device__ __forceinline__ u64 scan(u64 mine, u64 &all) {
    u64 m[1] = {mine}, b[1], t[1];
    scan(m, b, t);
    all = t[0];
    return b[0];
  }

  // The first element, by index, at which the running sum of measure(x, element)
  // reaches goal(sum of all), a thread's own elements having `mine` in all: its
  // index (in the warp that has it: others return -1), its measure and the sum
  // of all.
  template <typename M, typename G>
  __device__ int locate(u64 mine, M measure, G goal, u64 &own, u64 &all) {
    u64 before = scan(mine, all);
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
          m[i] = w + lane < w1 ? measure(value(v, i), (w + lane) * PER + i) : 0;
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
  template <typename M>
  __device__ __forceinline__ u64 sum(M measure) const {
    u64 mine = 0;
    each([&](float x, int e) { mine += measure(x, e); });
    return mine;
  }

  // Cuts the order (ascending keys, then indices) at the first element at which
  // the running sum of measure(x, element) reaches `to`: elements beyond it have
  // key > key, or key == key and element > last (of this block).  Keys lie in
  // [lo, hi].  WIDE: measures of up to 41 bits, else 0 or 1.  False: the sum does
  // not reach it.
  template <bool WIDE, typename M>
  __device__ __noinline__ bool select(uint32_t lo, uint32_t hi, u64 to, const M &measure, uint32_t &key, int &last) {
    constexpr int L = WIDE ? kLimbs : 1;
    u64 base = 0, of_key = 0;
    for (int round = 0; round < 4; ++round) {  // 3 at most: 11 bits of a key each
      const int down = max(0, 32 - __clz(hi - lo) - 11);  // (hi - lo) >> down < kBins
      __syncthreads();
      for (int i = threadIdx.x; i < L * kBins; i += NT) sh->hist[i] = 0;
      __syncthreads();
      each([&](float x, int e) {
        const uint32_t k = key_of(x);
        if (k < lo || k > hi) return;
        const u64 m = measure(x, e);
        const uint32_t bin = (k - lo) >> down;
#pragma unroll
        for (int l = 0; l < L; ++l) {
          const uint32_t part = L == 1 ? (uint32_t)m : (uint32_t)(m >> (kLimbBits * l)) & ((1u << kLimbBits) - 1);
          if (part) atomicAdd(&sh->hist[l * kBins + bin], part);
        }
      });
      sync();
      // a block takes a run of the bins, a thread a run of those
      const int per_block = kBins / ranks, per = max(1, per_block / NT), b0 = rank * per_block + threadIdx.x * per;
      const bool live = threadIdx.x * per < per_block;
      u64 sums[kBins / NT], mine = 0;
#pragma unroll
      for (int j = 0; j < kBins / NT; ++j) {
        sums[j] = 0;
        if (j < per && live) {
          for (int k = 0; k < ranks; ++k)
#pragma unroll
            for (int l = 0; l < L; ++l) {
              const uint32_t *p = &sh->hist[l * kBins + b0 + j];
              sums[j] += (u64)(ranks > 1 ? load_rank(p, k) : *p) << (kLimbBits * l);
            }
        }
        mine += sums[j];
      }
      u64 all;
      u64 before = base + scan(mine, all);
      if (round == 0 && (to > all || to == 0)) return false;
#pragma unroll
      for (int j = 0; j < kBins / NT; ++j) {
        if (j < per && live && before < to && to <= before + sums[j]) {
          tell(1, (uint32_t)(b0 + j));
          tell(1, before);
          tell(2, sums[j]);
        }
        before += sums[j];
      }
      sync();
      base = sh->before[1];
      of_key = sh->before[2];
      lo += sh->found[1] << down;
      hi = min(hi, lo + ((1u << down) - 1));
      if (lo >= hi) break;
    }
    key = lo;
    last = INT32_MAX;
    // elements of this key weigh the same: where not all of them stay, the index decides
    u64 one = 1;
    if constexpr (WIDE) one = measure.of(__uint_as_float(lo & 0x80000000u ? lo : 0x7fffffffu - lo));
    if (to + one > base + of_key) return true;
    u64 own = 0, all;
    const auto tie = [&](float x, int e) { return key_of(x) == lo ? measure(x, e) : 0ull; };
    const int at = locate(sum(tie), tie, [&](u64) { return to - base; }, own, all);
    // (a block before the one that has it keeps all of its own, one behind none)
    if (at >= 0 && (threadIdx.x & 31) == 0) tell(2, (uint32_t)at);
    sync();
    last = (int)sh->found[2] - shift;
    return true;
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

// What stays: logits from `bottom` on (others weigh nothing), of the order that
// ends at (key, last).
struct Cut {
  float bottom;
  uint32_t key;
  int last;
  __device__ __forceinline__ bool keeps(float x, int e) const {
    const uint32_t k = key_of(x);
    return x >= bottom && (k < key || (k == key && e <= last));
  }
};
// Weights of what a cut keeps.
struct Kept {
  Cut cut;
  Scale s;
  float tau;
  const uint32_t *table;
  bool fast;
  __device__ __forceinline__ u64 of(float x) const { return fast ? weight(x, s, table) : weight_plain(x, s.top, tau); }
  __device__ __forceinline__ u64 operator()(float x, int e) const { return cut.keeps(x, e) ? of(x) : 0ull; }
};
struct Counted {
  float bottom;
  __device__ __forceinline__ u64 operator()(float x, int) const { return x >= bottom ? 1ull : 0ull; }
};

// A logit's distance to the largest in 256ths of a step; a step is kOctaves /
// (kSteps - 2).  Monotone, and the same wherever it is asked; off by less than
// 0.007 of a step.  What lies below bottom, -infinity and NaN among it, gives
// kSteps x 256 or more.
struct Steps {
  float top, scale;
  __device__ __forceinline__ Steps(float top, float tau) : top(top), scale(1.44269504f / tau * ((float)(kSteps - 2) / kOctaves)) {}
  __device__ __forceinline__ uint32_t operator()(float x) const {
    return __float_as_uint(fmaf(top - x, scale, 49152.f)) - 0x47400000u;  // 1.5 2^15: the last bit is 2^-8
  }
};

// The running weight that top-p's last element reaches.
__device__ __forceinline__ u64 goal_of(float p, u64 all) {
  bool exact;
  const u64 n = part_of(fmaxf(p, 0.f), all, exact);
  return max(exact ? n : n + 1, 1ull);
}

// The last element that stays of `all` listed ones (order, weight), by one
// block: of those with bit 63 of the weight top-k keeps the first k (0: no
// top-k); p < 1: with `before` ahead of all of them and `rest` behind those in
// question in the weight that top-p takes its part of.
template <int NT>
__device__ __noinline__ u64 resolve(Shared<NT> *sh, int all, u64 k, float p, u64 before, u64 rest) {
  constexpr u64 EDGE = 1ull << 63;
  const int tid = threadIdx.x;
  u64 cut = ~0ull;
  __syncthreads();
  if (all <= 128) {  // a thread an element: what lies at or before it
    const u64 o = tid < all ? sh->order[tid] : ~0ull, v = tid < all ? sh->weight[tid] : 0;
    if (k) {
      if (v & EDGE) {
        u64 n = 0;
        for (int i = 0; i < all; ++i) n += sh->weight[i] >> 63 && sh->order[i] <= o;
        if (n == k) sh->before[1] = o;
      }
      __syncthreads();
      cut = sh->before[1];
    }
    if (p < 1.f) {
      if (tid < all && o <= cut) {
        u64 run = 0, kept = 0;
        for (int i = 0; i < all; ++i) {
          const u64 oi = sh->order[i], w = oi <= cut ? sh->weight[i] & ~EDGE : 0;
          kept += w;
          if (oi <= o) run += w;
        }
        const u64 goal = goal_of(p, before + rest + kept) - before;  // (above 0, as the bounds say)
        if (run - (v & ~EDGE) < goal && goal <= run) sh->before[2] = o;
      }
      __syncthreads();
      cut = sh->before[2];
    }
    return cut;
  }
  // sorted (Batcher's bitonic network), then prefix sums
  int most = 256;
  while (most < all) most *= 2;
  for (int i = all + tid; i < most; i += NT) {
    sh->order[i] = ~0ull;
    sh->weight[i] = 0;
  }
  for (int size = 2; size <= most; size *= 2)
    for (int by = size / 2; by > 0; by /= 2) {
      __syncthreads();
      if (tid < most / 2) {
        const int i = 2 * tid - (tid & (by - 1)), j = i + by;
        const u64 x = sh->order[i], y = sh->order[j];
        if ((x > y) == ((i & size) == 0)) {
          sh->order[i] = y;
          sh->order[j] = x;
          const u64 w = sh->weight[i];
          sh->weight[i] = sh->weight[j];
          sh->weight[j] = w;
        }
      }
    }
  __syncthreads();
  const bool in = 2 * tid < most;
  const u64 o0 = in ? sh->order[2 * tid] : ~0ull, o1 = in ? sh->order[2 * tid + 1] : ~0ull;
  const u64 v0 = in ? sh->weight[2 * tid] : 0, v1 = in ? sh->weight[2 * tid + 1] : 0;
  u64 b[1], t[1];
  if (k) {
    const u64 m[1] = {(v0 >> 63) + (v1 >> 63)};
    block_scan(sh, m, b, t);
    if (v0 >> 63 && b[0] + 1 == k) sh->before[1] = o0;
    if (v1 >> 63 && b[0] + m[0] == k) sh->before[1] = o1;
    __syncthreads();
    cut = sh->before[1];
  }
  if (p < 1.f) {
    const u64 w0 = o0 <= cut ? v0 & ~EDGE : 0, w1 = o1 <= cut ? v1 & ~EDGE : 0, m[1] = {w0 + w1};
    block_scan(sh, m, b, t);
    const u64 goal = goal_of(p, before + rest + t[0]) - before;
    if (b[0] < goal && goal <= b[0] + w0) sh->before[2] = o0;
    else if (b[0] + w0 < goal && goal <= b[0] + m[0]) sh->before[2] = o1;
    __syncthreads();
    cut = sh->before[2];
  }
  return cut;
}

// bf16 has few values: from the largest logit down to 2^-7, and from -2^-7 to
// the bottom, each has a place of its own, in descending order; the small ones
// between share one (`mid`).
struct Values {
  uint32_t top;  // magnitude bits of the largest logit
  int low;       // place of the negative magnitude m: m - low
  int mid;
  bool fit;
  static constexpr uint32_t kLow = 0x3c00;  // 2^-7
  __device__ __forceinline__ Values(float t, float bottom) {
    const uint32_t bits = __float_as_uint(t) >> 16;
    top = bits & 0x7fff;
    if (bits & 0x8000) {
      low = (int)top;
      mid = -1;
    } else {
      mid = (int)top - (int)kLow + 1;
      low = (int)kLow - (mid + 1);
    }
    fit = top >= kLow && place((uint16_t)(__float_as_uint(bottom) >> 16)) < (uint32_t)kSteps;
  }
  __device__ __forceinline__ uint32_t place(uint16_t bits) const {
    const int m = bits & 0x7fff;
    const int at = bits & 0x8000 ? m - low : (int)top - m;
    return (uint32_t)(m < (int)kLow && mid >= 0 ? mid : at);
  }
  __device__ __forceinline__ float value(int place) const {  // (not of mid)
    const uint32_t bits = mid < 0 || place > mid ? (uint32_t)(place + low) | 0x8000u : top - (uint32_t)place;
    return __uint_as_float(bits << 16);
  }
};

// Top-k and top-p by the counts of values: sums of a value's weights are its
// count times its weight, so the border is a value, with so many of the elements
// that have it, by index.  `sum` becomes the weight of this thread's elements
// that stay.  False: the border lies among the small ones.
template <int DT, int NT>
__device__ __noinline__ bool by_values(Row<DT, NT> &r, Kept &kept, const Values values, u64 k, float p, float least, u64 &sum) {
  Shared<NT> *sh = r.sh;
  const int tid = threadIdx.x;
  const float bottom = kept.cut.bottom;
  constexpr int MOST = kSteps / NT;
  const int per_block = kSteps / r.ranks, per = max(1, per_block / NT), q0 = r.rank * per_block + tid * per, run = tid * per < per_block ? per : 0;
  u64 small = 0;
  r.each_bits([&](uint16_t bits, int) {
    const uint32_t q = values.place(bits);
    if (q >= (uint32_t)kSteps) return;
    atomicAdd(&sh->hist[q], 1u);
    if ((int)q == values.mid) small += weight(__uint_as_float((uint32_t)bits << 16), kept.s, kept.table);
  });
  if (small)  // to the block that has the place
    asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(at_rank(&sh->small, values.mid / per_block)), "l"(small) : "memory");
  r.sync();
  uint32_t n[MOST];
  u64 one[MOST], mine[2] = {0, 0}, at[2], all[2];  // weight of an element of a place; of mid: of all its elements
  const auto mass = [&](int j) { return q0 + j == values.mid ? one[j] : n[j] * one[j]; };
#pragma unroll
  for (int j = 0; j < MOST; ++j) {
    n[j] = 0;
    one[j] = 0;
    if (j < run) {
      uint32_t x[kMaxCluster];
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) x[i] = i < r.ranks ? load_rank(&sh->hist[q0 + j], i) : 0;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) n[j] += x[i];
      const float v = values.value(q0 + j);
      if (n[j]) one[j] = q0 + j == values.mid ? sh->small : v >= bottom ? weight(v, kept.s, kept.table) : 0;
    }
    mine[0] += n[j];
    mine[1] += mass(j);
  }
  r.scan(mine, at, all);
  // the border: a value's place, how many of its elements stay, whether all do
  uint32_t edge = kSteps;
  u64 stay = 0;
  bool every = true;
  u64 total = all[1];
  if (k && k < all[0]) {
    u64 c = at[0], b = at[1];
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      if (c < k && k <= c + n[j]) {
        const u64 left = k - c;
        r.tell(1, (uint32_t)(q0 + j));
        r.tell(2, (uint32_t)(left == n[j]));
        r.tell(0, left);
        r.tell(1, b + left * one[j]);
      }
      c += n[j];
      b += mass(j);
    }
    r.sync();
    edge = sh->found[1];
    every = sh->found[2] != 0;
    stay = sh->before[0];
    total = sh->before[1];
    if ((int)edge == values.mid) return false;  // (its weights differ)
  }
  if (p < 1.f) {
    const u64 goal = goal_of(p, total);
    u64 b = at[1];
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      const uint32_t q = q0 + j;
      const u64 here = q < edge ? mass(j) : q == edge ? one[j] * (every ? (u64)n[j] : stay) : 0;
      if (b < goal && goal <= b + here) {
        const u64 left = (goal - b + one[j] - 1) / one[j];
        r.tell(3, q);
        r.tell(4, (uint32_t)(left == n[j]));
        r.tell(2, left);
      }
      b += mass(j);
    }
    r.sync();
    edge = sh->found[3];
    every = sh->found[4] != 0;
    stay = sh->before[2];
    if ((int)edge == values.mid) return false;
  }
  // ---- a weight for each place; elements at the border count in units of 2^52
  constexpr u64 TIE = 1ull << 52;
  const float border = edge < kSteps ? values.value((int)edge) : 0.f;
  for (int q = tid; q < kSteps; q += NT) {
    const float v = values.value(q);
    sh->value[q] = q == values.mid || q > (int)edge || !(v >= least) ? 0 : q == (int)edge ? TIE : weight(v, kept.s, kept.table);
  }
  __syncthreads();
  const bool small_stay = values.mid >= 0 && values.mid < (int)edge;
  const uint32_t last = min(edge, (uint32_t)kSteps - 1);
  u64 mixed = 0;
  r.each_bits([&](uint16_t bits, int) {
    const uint32_t q = values.place(bits);
    if (q > last) return;
    mixed += sh->value[q];
    if ((int)q == values.mid && small_stay) {
      const float x = __uint_as_float((uint32_t)bits << 16);
      if (x >= least) mixed += weight(x, kept.s, kept.table);
    }
  });
  sum = mixed & (TIE - 1);
  const u64 ties = mixed >> 52;
  kept.cut.key = edge < kSteps ? key_of(border) : 0xffffffffu;
  kept.cut.last = INT32_MAX;
  if (edge < kSteps && border >= least) {
    const u64 one = weight(border, kept.s, kept.table);
    if (every) {
      sum += ties * one;
    } else {  // the first `stay` of them, by index
      u64 sum_all;
      const u64 before = r.scan(ties, sum_all);
      const u64 mine_stay = before >= stay ? 0 : min(ties, stay - before);
      sum += mine_stay * one;
      if (before < stay && stay <= before + ties) {  // this thread has the last one
        u64 left = stay - before;
        r.each([&](float x, int e) {
          if (x == border && --left == 0) r.tell(5, (uint32_t)(e + r.shift));
        });
      }
      r.sync();
      kept.cut.last = (int)sh->found[5] - r.shift;
    }
  }
  return true;
}

template <int DT, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_sample(const __grid_constant__ SampleArgs a, const __grid_constant__ Pow2 pow2) {
  extern __shared__ __align__(16) unsigned char sm[];
  Shared<NT> *sh = reinterpret_cast<Shared<NT> *>(sm);
  uint4 *data = reinterpret_cast<uint4 *>(sm + sizeof(Shared<NT>));
  constexpr int SIZE = DT == RV_F32 ? 4 : 2, EPG = 16 / SIZE;
  const int tid = threadIdx.x, ranks = (int)cluster_size(), rank = (int)cluster_rank(), b = blockIdx.x / ranks;
  for (int i = tid; i < 256; i += NT) sh->table[i] = pow2.t[i];
  for (int i = tid; i < 2 * kSteps; i += NT) sh->hist[i] = 0;
  if (tid == 0) {
    sh->listed = sh->gathered = 0;
    sh->small = 0;
  }
  if (tid < 8) sh->found[tid] = 0xffffffffu;
  sh->add[tid] = 0;
  if (ranks > 1) cluster_arrive();
  pdl_wait();

  // ---- this block's share of the row: whole 16-byte pieces of memory; elements
  // beside the row are -infinity
  const char *row = static_cast<const char *>(a.x) + b * a.stride * SIZE;
  const char *base = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15);
  const int lead = (int)(row - base) / SIZE, g0 = rank * a.granules, total = (lead + a.V + EPG - 1) / EPG;
  const int mine = max(0, min(a.granules, total - g0));
  float top = -INFINITY;
  Row<DT, NT> r{sh, reinterpret_cast<const uint32_t *>(data), a.words, mine * 4, g0 * EPG - lead, rank, ranks, 0};
  const float tau = a.temperature ? a.temperature[b] : 1.f, draw = a.u[b];
  const float p = a.top_p ? a.top_p[b] : 1.f, lowest = a.min_p ? a.min_p[b] : 0.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  auto take = [&](uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < Row<DT, NT>::PER; ++j) top = fmaxf(top, r.value(w[i], j));  // (fmaxf passes over NaN)
  };
  auto whole = [&](int g) { return (g0 + g) * EPG - lead >= 0 && (g0 + g + 1) * EPG - lead <= a.V; };
  constexpr int FLY = 6;
  for (int g = tid; g < mine; g += FLY * NT) {
    uint4 v[FLY];
#pragma unroll
    for (int q = 0; q < FLY; ++q)
      if (g + q * NT < mine && whole(g + q * NT)) v[q] = reinterpret_cast<const uint4 *>(base)[g0 + g + q * NT];
#pragma unroll
    for (int q = 0; q < FLY; ++q) {
      const int at = g + q * NT;
      if (at >= mine) continue;
      if (!whole(at)) {
        uint32_t w[4] = {};
        for (int e = 0; e < EPG; ++e) {
          const int i = (g0 + at) * EPG + e - lead;
          uint32_t x = DT == RV_F32 ? 0xff800000u : DT == RV_BF16 ? 0xff80u : 0xfc00u;
          if (i >= 0 && i < a.V) x = DT == RV_F32 ? reinterpret_cast<const uint32_t *>(row)[i] : reinterpret_cast<const uint16_t *>(row)[i];
          w[e * SIZE / 4] |= x << (8 * (e * SIZE % 4));
        }
        v[q] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      data[at] = v[q];
      take(v[q]);
    }
  }
  // ---- the largest logit
  top = warp_max(top);
  if ((tid & 31) == 0) sh->warp[tid >> 5] = __float_as_uint(top);
  __syncthreads();
  top = warp_max((tid & 31) < NT / 32 ? __uint_as_float((uint32_t)sh->warp[tid & 31]) : -INFINITY);
  if (ranks > 1) {
    cluster_wait();
    if (tid < ranks)  // (the first scan uses the other one)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at_rank(&sh->total[0][rank], tid)), "l"((u64)__float_as_uint(top)) : "memory");
    cluster_sync();
    top = warp_max((tid & 31) < ranks ? __uint_as_float((uint32_t)sh->total[0][tid & 31]) : -INFINITY);
  }
  pdl_trigger();
  if (top == -INFINITY) {  // (the same in every block of the cluster)
    if (rank == 0 && tid == 0) {
      a.ids[b] = -1;
      if (a.logprob) a.logprob[b] = -INFINITY;
    }
    return;
  }
  if (!(tau > 0.f)) {  // the first of the largest
    u64 own, all;
    const auto is = [&](float x, int) { return x == top ? 1ull : 0ull; };
    const int at = r.locate(r.sum(is), is, [](u64) { return 1ull; }, own, all);
    if (at >= 0 && (tid & 31) == 0) {
      a.ids[b] = at;
      if (a.logprob) a.logprob[b] = 0.f;
    }
    return;
  }

  // ---- the draw
  Kept kept;
  kept.tau = tau;
  kept.table = sh->table;
  kept.fast = fits(top, tau);
  kept.s = scale_of(top, kept.fast ? tau : 1.f);
  const bool floor = lowest > 0.f && !isinf(top);
  if (floor) {  // (64-bit operations are slow: one thread's)
    if (tid == 0) sh->least = up32((double)top + (double)tau * log(fmin((double)lowest, 1.0)));
    __syncthreads();
  }
  // weights below half a unit are zero (a margin of some tenths of an octave)
  const float bottom = isinf(top) ? top : fmaxf(top - kOctaves * 0.693147181f * tau, -3.402823466e38f);
  const float least = floor ? fmaxf(bottom, sh->least) : bottom;
  kept.cut = Cut{bottom, 0xffffffffu, INT32_MAX};
  const uint32_t k_top = key_of(top), k_bottom = key_of(bottom);
  bool by_k = k > 0 && k < a.V, by_p = p < 1.f;
  u64 sum = 0;  // of this thread's elements that stay
  bool done = false;
  if constexpr (DT == RV_BF16) {
    const Values values(top, bottom);
    if (kept.fast && (by_k || by_p) && values.fit) {
      done = by_values(r, kept, values, by_k ? (u64)k : 0, p, least, sum);
      if (!done) {  // as it was at first
        kept.cut = Cut{bottom, 0xffffffffu, INT32_MAX};
        sum = 0;
        __syncthreads();
        for (int i = tid; i < 2 * kSteps; i += NT) sh->hist[i] = 0;
        if (tid < 8) sh->found[tid] = 0xffffffffu;
        __syncthreads();
      }
    }
  }
  if (!done && kept.fast && (by_k || by_p)) {
    // ---- elements a step, and the sum of their places in it
    const Steps step(top, tau);
    uint32_t *counts = sh->hist, *places = sh->hist + kSteps;
    r.each([&](float x, int) {
      const uint32_t q = step(x);
      if (q < kSteps * 256u) {
        atomicAdd(&counts[q >> 8], 1u);
        if (by_p) atomicAdd(&places[q >> 8], q & 255u);
      }
    });
    r.sync();
    // ---- a block takes a run of the steps, a thread a run of those.  Bounds of each step's weight, of the largest: with A =
    // ln 2 x a step in octaves, a place f of 256 weighs (1 - A f / 256 + [0, 2.6 10^-5]) 2^(-step); places are off by 0.007
    // of a step at most (5 10^-5 of the weight), whole numbers by half a unit of 2^-40, the sums below by 2^-18
    const int per_block = kSteps / ranks, per = max(1, per_block / NT), q0 = rank * per_block + tid * per, run = tid * per < per_block ? per : 0;
    constexpr int MOST = kSteps / NT;
    constexpr float OCT = kOctaves / (kSteps - 2), A = 0.693147181f * OCT;
    float n[MOST], low[MOST], high[MOST], mine[3] = {0.f, 0.f, 0.f}, at[3], sums[3];  // counts are below 2^24: exact
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      n[j] = low[j] = high[j] = 0.f;
      if (j < run) {
        uint32_t x[kMaxCluster], y[kMaxCluster], count = 0, place = 0;  // (all on their way at once)
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
          x[i] = i < ranks ? load_rank(&counts[q0 + j], i) : 0;
          y[i] = i < ranks && by_p ? load_rank(&places[q0 + j], i) : 0;
        }
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
          count += x[i];
          place += y[i];
        }
        n[j] = (float)count;
        if (by_p && count) {
          const float w = exp2f(-OCT * (float)(q0 + j)) * (n[j] - A / 256.f * (float)place), half = n[j] * 0x1p-41f;
          low[j] = fmaxf(w * 0.9999f - half, 0.f);
          high[j] = w * 1.0001f + half;
        }
      }
      mine[0] += n[j];
      mine[1] += low[j];
      mine[2] += high[j];
    }
    r.scan(mine, at, sums);
    uint32_t edge = kSteps, ahead = 0;  // the step of top-k's border; before it `ahead` elements
    by_k = by_k && (float)k < sums[0];
    if (by_k) {
      float before = at[0], lo = at[1], hi = at[2];
#pragma unroll
      for (int j = 0; j < MOST; ++j) {
        if (before < (float)k && (float)k <= before + n[j]) {
          const float left = (float)k - before, w = exp2f(-OCT * (float)(q0 + j)) * left, half = left * 0x1p-41f;
          r.tell(1, (uint32_t)(q0 + j));
          r.tell(2, (uint32_t)before);
          r.tell(5, __float_as_uint(lo + fmaxf(w * (1.f - 2.f * A) - half, 0.f)));
          r.tell(6, __float_as_uint(hi + w * 1.0001f + half));
        }
        before += n[j];
        lo += low[j];
        hi += high[j];
      }
      r.sync();
      edge = sh->found[1];
      ahead = sh->found[2];
      sums[1] = __uint_as_float(sh->found[5]);
      sums[2] = __uint_as_float(sh->found[6]);
    }
    uint32_t z0 = edge, z1 = edge;  // the steps that top-p's border can lie in
    if (by_p) {
      // z0: the first step that the upper bounds reach the lower goal with; z1: that the lower ones reach the upper goal with
      const float goal_lo = p * sums[1] * (1.f - 0x1p-17f), goal_hi = fmaxf(p, 0.f) * sums[2] * (1.f + 0x1p-17f);
      uint32_t first_lo = kSteps, first_hi = kSteps;
#pragma unroll
      for (int j = 0; j < MOST; ++j) {
        at[1] += low[j];
        at[2] += high[j];
        if (j < run && at[2] * (1.f + 0x1p-18f) >= goal_lo) first_lo = min(first_lo, (uint32_t)(q0 + j));
        if (j < run && at[1] * (1.f - 0x1p-18f) >= goal_hi) first_hi = min(first_hi, (uint32_t)(q0 + j));
      }
      first_lo = __reduce_min_sync(0xffffffffu, first_lo);
      first_hi = __reduce_min_sync(0xffffffffu, first_hi);
      if ((tid & 31) == 0) {
        if (first_lo < kSteps) r.least(3, first_lo);
        if (first_hi < kSteps) r.least(4, first_hi);
      }
      r.sync();
      z0 = min(sh->found[3], edge);
      z1 = max(z0, min(min(sh->found[4], edge), (uint32_t)kSteps - 1));
    }
    // ---- exact weights: of the steps before z0 (`sum`: of at least min-p), of those between z1 and the edge (`rest`); the
    // elements between are listed: here, and with their place in the order (key, index) and their weights in the first block
    u64 before = 0, rest = 0;
    r.each([&](float x, int e) {
      const uint32_t q = step(x) >> 8;
      if (q > edge || q >= kSteps || (q > z1 && q != edge && !by_p)) return;
      const u64 w = x >= bottom ? weight(x, kept.s, kept.table) : 0;
      if ((q >= z0 && q <= z1) || q == edge) {
        const int here = atomicAdd(&sh->listed, 1);
        if (here < kList) {
          sh->list[here] = (uint32_t)e;
          const int at = add_rank(&sh->gathered, 0, 1);
          if (at < kList) {
            const u64 o = (u64)key_of(x) << 32 | (uint32_t)(e + r.shift), v = w | (by_k && q == edge ? 1ull << 63 : 0);  // (bit 63: top-k counts it)
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at_rank(&sh->order[at], 0)), "l"(o) : "memory");
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at_rank(&sh->weight[at], 0)), "l"(v) : "memory");
          }
        } else if (here == kList) {
          add_rank(&sh->gathered, 0, kList + 1);  // too many
        }
      } else if (q > z1) {
        rest += w;
      } else {
        before += w;
        if (!floor || x >= least) sum += w;
      }
    });
    const u64 exact[2] = {before, rest};
    u64 exact_at[2], exact_all[2];
    r.scan(exact, exact_at, exact_all);
    if (rank == 0) {
      const int all = sh->gathered;
      if (all <= kList) {
        const u64 cut = resolve(sh, all, by_k ? (u64)k - ahead : 0, by_p ? p : 1.f, exact_all[0], exact_all[1]);
        if (tid == 0) r.tell(3, cut);
      }
      if (tid == 0) r.tell(7, (uint32_t)(all <= kList));
    }
    r.sync();
    done = sh->found[7] != 0;
    if (done) {
      const u64 cut = sh->before[3];
      kept.cut.key = (uint32_t)(cut >> 32);
      kept.cut.last = (int)(uint32_t)cut - r.shift;
      // listed elements that stay belong to the threads whose elements they are
      for (int i = tid; i < sh->listed; i += NT) {
        const int e = (int)sh->list[i];
        const float x = r.at(e);
        const u64 w = x >= least ? kept(x, e) : 0;
        if (w) atomicAdd(&sh->add[e / Row<DT, NT>::PER / a.words], w);
      }
      __syncthreads();
      sum += sh->add[tid];
    }
  }
  if (!done) {
    uint32_t key;
    int last;
    if (by_k && r.template select<false>(k_top, k_bottom, (u64)k, Counted{bottom}, key, last)) kept.cut = Cut{bottom, key, last};
    if (by_p) {
      u64 all;
      r.scan(r.sum(kept), all);
      if (r.template select<true>(k_top, k_bottom, goal_of(p, all), kept, key, last))
        kept.cut = Cut{bottom, key, key == kept.cut.key ? min(last, kept.cut.last) : last};
    }
    kept.cut.bottom = least;
    sum = r.sum(kept);
  }
  kept.cut.bottom = least;
  u64 own = 0, all;
  const float f = draw >= 1.f ? 0x1.fffffep-1f : draw > 0.f ? draw : 0.f;
  const int at = r.locate(sum, kept,
                          [&](u64 n) {
                            bool exact;
                            return part_of(f, n, exact) + 1;
                          },
                          own, all);
  if (at >= 0 && (tid & 31) == 0) {
    a.ids[b] = at;
    if (a.logprob) a.logprob[b] = (float)log((double)own / (double)all);
  }
  // (what a block reads or writes of another's shared memory lies before a barrier that the other one passes later)
}

template <int DT, int NT>
cudaError_t launch_t(SampleArgs a, const Pow2 &t, int ranks, cudaStream_t s, int pdl) {
  a.words = ((a.granules * 4 + NT - 1) / NT) | 1;
  const size_t smem = sizeof(Shared<NT>) + (size_t)a.granules * 16;
  auto fn = k_sample<DT, NT>;
  // (one limit for every call: calls of several threads may come between one's setting of it and its launch)
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * ranks);
  cfg.blockDim = dim3(NT);
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

}  // namespace

// Threads of a block: 1024 and an SM for itself for bf16, whose 4096 values are
// gone through three times whatever the row's length; 512 and two blocks in an SM
// for the others, and where there are more short rows than SMs.  (512 / 1024, us,
// the better cluster of each.  bf16 under top-p: one row of 1,000 16.3 / 14.3, of
// 24,000 21.8 / 19.6, 100 of 8,000 23.1 / 19.6, 150 of 50,257 45.9 / 34.0, 70 of
// 128,256 59.5 / 50.3, 256 of them 195 / 169; 300 of 8,000 29.9 / 36.9, 300 of
// 24,000 46.7 / 50.0, 512 of 32,000 102 / 100.  fp32: one row of 32,000 16.5 / 19.1,
// 64 of 128,256 58.0 / 59.3, 472 of 422 27.1 / 47.6; fp16: 148 of 10,487 20.9 /
// 21.3, 200 of 50,257 37.6 / 43.9.)
int sample_threads(int B, int vocab, bool bf16, int n_sm) { return bf16 && (B <= n_sm || vocab >= 32768) ? 1024 : 512; }

// Blocks of a row's cluster: as many as its share of an SM's shared memory asks
// for, and more while there is an SM for each and a thread keeps 16 bytes.
// (1 / 2 / 4 / 8 blocks, us: 148 rows of 10,487 fp16 under top-p 20.9 / 27.9 /
// 47.7 / 91, 100 of 20,000 bf16 32.1 / 33.8 / 46.8 / 71, 30 of 50,257 bf16 - /
// 37.7 / 28.5 / 29.6, 64 of 32,000 fp32 - / 36.7 / 36.3 / 51.5, one of 32,000 - /
// 26.2 / 19.2 / 16.7, 8 of 4,000 13.4 / 15.1 / 15.0 / 14.4.  With 512 threads.)
int sample_cluster(int B, int64_t row_bytes, int n_sm, int threads) {
  int ranks = 1;
  while (ranks < kMaxCluster && row_bytes > (int64_t)ranks * (threads / 512) * 66000) ranks *= 2;
  while (ranks < kMaxCluster && (int64_t)B * ranks * 2 <= n_sm && row_bytes >= (int64_t)ranks * (threads / 512) * 16384) ranks *= 2;
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
  const int threads = sample_threads(B, vocab, dtype == RV_BF16, n_sm);
  const int ranks = sample_cluster(B, (int64_t)vocab * size, n_sm, threads);
  SampleArgs a{};
  a.x = d_logits; a.stride = stride; a.B = B; a.V = vocab;
  const int total = (vocab * size + 14) / 16 + 1;  // 16-byte pieces that a row can touch
  a.granules = (total + ranks - 1) / ranks;
  a.temperature = d_temperature; a.top_k = d_top_k; a.top_p = d_top_p; a.min_p = d_min_p; a.u = d_u;
  a.ids = d_ids; a.logprob = d_logprob;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Pow2 &t = pow2_table();
  return launched("rv_sample", dtype == RV_F32    ? launch_t<RV_F32, 512>(a, t, ranks, s, 1)
                               : dtype == RV_F16  ? launch_t<RV_F16, 512>(a, t, ranks, s, 1)
                               : threads == 512   ? launch_t<RV_BF16, 512>(a, t, ranks, s, 1)
                                                  : launch_t<RV_BF16, 1024>(a, t, ranks, s, 1));
}
