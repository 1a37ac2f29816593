// The part of a shared prefix in the attention of kv8_shared.cu.
//
// The fan x T x (H / Hkv) query rows that share a KV head of a prefix row make
// it a dense product, so it runs on the 5th-generation tensor cores: S = Q K^T
// with 128 query rows by 128 positions an item, softmax weights with a thread a
// row, O += P V.  K and V codes become fp16 (exact) in shared memory, once for up
// to 256 query rows; a K block's scale multiplies its scores, a V block's scale
// (over a power of two that the rows keep) its weights, which enter the product
// as fp16 (two terms for fp16 caches and fp32 outputs) from tensor memory, where
// they take their scores' place.  O stays in tensor memory.
//
// A block per SM: 4 warps turn codes to fp16, one thread issues the products, 8
// warps in two streams do the softmax, so that one's products run under the
// other's weights.  Up to 128 query rows, the streams take every other tile of
// positions and are joined at the end; with more, each has its 128 rows.
#pragma once

#include "async.cuh"
#include "kv8_attention.cuh"
#include "ops.cuh"

namespace rv {
namespace kv8s {


using kv8a::ex2;
using kv8a::kLog2e;
using kv8a::kOutUnit;

constexpr int kTile = 128;   // positions of a tile
constexpr int kRows = 256;   // query rows of a unit at most

// A unit is one prefix row, KV head and group of up to kRows query rows; its
// tiles lie in one line with all others, which is cut evenly over the blocks.
// Block c that takes a part of unit u leaves its state in slot c + u (both rise
// along the line, so no two parts share one).
struct SharedArgs {
  Kv8 c;  // the prefix
  Heads q;
  int q_f32;
  int H, B, T, fan, P;
  int rows, groups, slot_rows;  // query rows of a prefix row and KV head, units of them, rows of a slot
  float scale;
  const int32_t *plen, *count;
  int32_t *err;
  int64_t *line;  // [P + 2]: where each prefix row's units begin in the line, its end, the length of a piece
  float *slots;   // [blocks + units][slot_rows][hd + 2]
  int lo;         // weights as two fp16 terms
};

// (slots begin on 32-byte boundaries)
__host__ __device__ __forceinline__ size_t slot_floats(int slot_rows, int hd) { return ((size_t)slot_rows * (hd + 2) + 7) / 8 * 8; }

__device__ __forceinline__ int prefix_len(const SharedArgs &a, int p) {
  const int n = a.plen ? a.plen[p] : a.c.T;
  return min(max(n, 0), a.c.T);
}
__device__ __forceinline__ int prefix_tiles(const SharedArgs &a, int p) { return (prefix_len(a, p) + kTile - 1) / kTile; }

// Query row i of prefix row p: token i / grp of its rows' tokens, head i % grp.
struct QueryRow {
  int b, t;
  bool live;
};
__device__ __forceinline__ QueryRow query_row(const SharedArgs &a, int p, int i, int grp) {
  QueryRow r;
  const int k = i / grp, f = k / a.T;
  r.b = p * a.fan + f;
  r.t = k - f * a.T;
  r.live = i < a.rows && r.b < a.B;
  if (r.live) r.live = r.t < row_count(a.count, r.b, a.T);
  return r;
}

// The line: this block's piece, and the prefix row that it begins in.  Every
// block computes it; block 0 leaves it for the join.
constexpr int kMinTiles = 2;  // of a piece
struct Piece {
  int64_t begin, end, off;  // off: into row p
  int p;
};
template <int THREADS>
__device__ Piece cut_line(const SharedArgs &a, int64_t *scratch /* THREADS + 2 */) {
  const int tid = threadIdx.x, per = (a.P + THREADS - 1) / THREADS, p0 = min(a.P, tid * per), p1 = min(a.P, p0 + per);
  int64_t mine = 0;
  const int64_t units = (int64_t)a.c.Hkv * a.groups;
  for (int p = p0; p < p1; ++p) mine += units * prefix_tiles(a, p);
  scratch[tid] = mine;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int i = 0; i < min(THREADS, a.P); ++i) {  // (the others have none)
    const int64_t x = scratch[i];
    if (i < tid) before += x;
    total += x;
  }
  const int64_t piece = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kMinTiles);
  Piece w;
  w.begin = piece * blockIdx.x;
  w.end = min(total, w.begin + piece);
  int64_t at = before;
  for (int p = p0; p < p1; ++p) {
    const int64_t n = units * prefix_tiles(a, p);
    if (blockIdx.x == 0) a.line[p] = at;
    if (w.begin >= at && w.begin < at + n) {
      scratch[THREADS] = p;
      scratch[THREADS + 1] = w.begin - at;
    }
    at += n;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.line[a.P] = total;
    a.line[a.P + 1] = piece;
  }
  __syncthreads();
  w.p = (int)scratch[THREADS];
  w.off = scratch[THREADS + 1];
  return w;
}

// ------------------------------------------------------------------ the prefix

constexpr int kSoftWarps = 8, kCodeWarps = 4, kThreads = 32 * (kSoftWarps + kCodeWarps + 1);
constexpr int kHalf = 16384;  // 128 rows of 64 fp16
__host__ __device__ constexpr int tile_bytes(int hd) { return hd / 64 * kHalf; }
struct Bars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];  // stages of K and V
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];  // streams
  uint64_t exchange, drained;
};
// What the block's threads share beside the operands.
struct Side {
  Bars bar;
  float m[2][128], l[2][128];  // the streams' rows, for their join
  int e[2][4];
  int64_t scratch[kThreads + 2];
  uint32_t tmem;
  int dead;  // a wait ran out: everyone leaves
};
__host__ __device__ constexpr int prefix_smem(int hd) { return 1024 + 6 * tile_bytes(hd) + (int)sizeof(Side); }

// A part of a unit.
struct Part {
  int p, g, group, t0, t1, n, rows;  // tiles [t0, t1) of the prefix row's n positions; query rows of the unit
  int64_t kv, slot;                  // KV row; slot of the state
};
struct Walk {
  int64_t at, end, off;
  int p;
  __device__ __forceinline__ bool next(const SharedArgs &a, Part &s) {
    while (at < end && p < a.P) {  // (p: only if the lengths changed under the kernel)
      const int n = prefix_len(a, p), tiles = (n + kTile - 1) / kTile;
      const int64_t in_row = (int64_t)a.c.Hkv * a.groups * tiles;
      if (off >= in_row) { off -= in_row; ++p; continue; }
      const int unit = (int)(off / tiles), t0 = (int)(off - (int64_t)unit * tiles), take = (int)min((int64_t)(tiles - t0), end - at);
      s.p = p;
      s.g = unit / a.groups;
      s.group = unit - s.g * a.groups;
      s.t0 = t0;
      s.t1 = t0 + take;
      s.n = n;
      s.rows = min(kRows, a.rows - s.group * kRows);
      s.kv = (int64_t)p * a.c.Hkv + s.g;
      s.slot = blockIdx.x + s.kv * a.groups + s.group;
      at += take;
      off += take;
      return true;
    }
    return false;
  }
};

// 4 codes as fp16 (kv8.cu's read-back takes them the same way).
template <int FMT>
__device__ __forceinline__ uint2 codes4(uint32_t w) {
  if (FMT == RV_KV8_INT8) {  // byte ^ 0x80 = code + 128 under the exponent of 1024 is 1152 + code
    const uint32_t u = w ^ 0x80808080u, lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 bias = kv8a::bits_h2(0x64806480u);
    return make_uint2(kv8a::h2_bits(__hsub2(kv8a::bits_h2(lo), bias)), kv8a::h2_bits(__hsub2(kv8a::bits_h2(hi), bias)));
  }
  uint2 r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(r.x), "=r"(r.y) : "r"(w));
  return r;
}

template <int FMT, int HD, bool LO>
__global__ void __launch_bounds__(kThreads, 1) k_prefix(const __grid_constant__ SharedArgs a) {
  extern __shared__ unsigned char raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  constexpr int TB = tile_bytes(HD);
  unsigned char *sq = sm, *sk = sm + 2 * TB, *sv = sm + 4 * TB;
  Side &side = *reinterpret_cast<Side *>(sm + 6 * TB);
  Bars &bar = side.bar;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kSoftWarps + kCodeWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&side.tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&bar.k_full[i], kCodeWarps);
      bar_init(&bar.k_free[i], 1);
      bar_init(&bar.v_full[i], kCodeWarps);
      bar_init(&bar.v_free[i], 1);
      bar_init(&bar.q_full[i], 4);
      bar_init(&bar.s_full[i], 1);
      bar_init(&bar.p_full[i], 4);
      bar_init(&bar.o_full[i], 1);
    }
    bar_init(&bar.exchange, kSoftWarps);
    bar_init(&bar.drained, 1);
    bar_init_done();
    side.dead = 0;
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = side.tmem;
  pdl_wait();
  const Piece piece = cut_line<kThreads>(a, side.scratch);
  Walk walk{piece.begin, piece.end, piece.off, piece.p};
  const Kv8 &c = a.c;
  const int grp = a.H / c.Hkv, lb = __ffs(c.block) - 1;
  volatile int *dead = &side.dead;
  auto wait = [&](uint64_t *b, uint32_t parity) {
    if (bar_wait(b, parity, dead)) return true;
    if (!*dead && a.err) atomicOr(a.err, kErrWait);
    *dead = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
  // Tensor memory: the streams' scores (and weights), then their O.
  auto at_s = [&](int s) { return tmem + 128 * s; };
  auto at_o = [&](int s) { return tmem + 256 + HD * s; };
  Part part;
  // Items of a part: (stream, tile) = (i & 1, i) where the streams share the rows, (i & 1, i >> 1) where each has its own.

  if (warp >= kSoftWarps && warp < kSoftWarps + kCodeWarps) {
    // ================================================ codes to fp16
    // Thread: 16 codes of position 32 j + 8 w + lane / 4 of the tile, and 64 codes on; a phase of 8 lanes
    // reads 64 bytes of two positions and stores 16-byte pieces that meet all banks.
    constexpr int NC = HD / 16;  // 16-byte loads of a thread, tile and operand
    const int w = warp - kSoftWarps, p_in = 8 * w + (lane >> 2), col = (lane & 3) * 16;
    uint4 buf[2][NC];
    auto load = [&](int which, const Part &s, int t) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int half = HD == 128 ? j & 1 : 0, pos = t * kTile + 32 * (HD == 128 ? j >> 1 : j) + p_in;
        buf[which][j] = make_uint4(0, 0, 0, 0);
        if (pos < s.n) buf[which][j] = *reinterpret_cast<const uint4 *>(c.codes[which] + (s.kv * c.N + pos) * HD + half * 64 + col);
      }
    };
    auto store = [&](int which, unsigned char *to) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int half = HD == 128 ? j & 1 : 0, pos = 32 * (HD == 128 ? j >> 1 : j) + p_in;
        unsigned char *row = to + half * kHalf + pos * 128;
        const int piece = (lane & 3) * 2, x = pos & 7;
        const uint4 v = buf[which][j];
        const uint2 y0 = codes4<FMT>(v.x), y1 = codes4<FMT>(v.y), y2 = codes4<FMT>(v.z), y3 = codes4<FMT>(v.w);
        *reinterpret_cast<uint4 *>(row + ((piece ^ x) << 4)) = make_uint4(y0.x, y0.y, y1.x, y1.y);
        *reinterpret_cast<uint4 *>(row + (((piece + 1) ^ x) << 4)) = make_uint4(y2.x, y2.y, y3.x, y3.y);
      }
      fence_async_smem();
      __syncwarp();
    };
    bool more = walk.next(a, part);
    if (more) { load(0, part, part.t0); load(1, part, part.t0); }
    int t = part.t0;
    for (uint32_t k = 0; more; ++k) {
      const uint32_t st = k & 1, parity = ((k >> 1) & 1) ^ 1;
      Part then = part;
      int tn = t + 1;
      if (tn == part.t1) { more = walk.next(a, then); tn = then.t0; }
      if (!wait_warp(&bar.k_free[st], parity)) break;
      store(0, sk + st * TB);
      if (lane == 0) bar_arrive(&bar.k_full[st]);
      if (more) load(0, then, tn);
      if (!wait_warp(&bar.v_free[st], parity)) break;
      store(1, sv + st * TB);
      if (lane == 0) bar_arrive(&bar.v_full[st]);
      if (more) load(1, then, tn);
      part = then;
      t = tn;
    }
  } else if (warp == kSoftWarps + kCodeWarps) {
    // ================================================ products
    if (lane == 0) {
      constexpr uint32_t KIND = 1u << 4 | (uint32_t)(kTile >> 4) << 24;  // fp16, fp32 sums, 128 rows
      constexpr uint32_t KIND_S = KIND | (uint32_t)(kTile >> 3) << 17, KIND_O = KIND | (uint32_t)(HD >> 3) << 17 | 1u << 16;  // V: elements contiguous
      uint32_t tiles = 0, parts = 0, items[2] = {0, 0};
      bool ok = true;
      while (ok && walk.next(a, part)) {
        const int per = part.rows > 128 ? 2 : 1, n = (part.t1 - part.t0) * per;
        for (int s = 0; ok && s < 2; ++s) ok = wait(&bar.q_full[s], parts & 1);
        auto scores = [&](int i) {
          const int s = i & 1;
          const uint32_t k = tiles + (per == 2 ? i >> 1 : i), st = k & 1;
          ok = ok && wait(&bar.k_full[st], (k >> 1) & 1);
          if (!ok) return;
          tmem_fence_after();
          const uint64_t q = mma_operand(smem_addr(sq + s * TB), 16), kk = mma_operand(smem_addr(sk + st * TB), 16);
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            const uint32_t at = ((j >> 2) * kHalf + (j & 3) * 32) >> 4;
            mma_ss(at_s(s), q + at, kk + at, KIND_S, j != 0);
          }
          mma_commit(&bar.s_full[s]);
          if (per == 1 || s == 1) mma_commit(&bar.k_free[st]);
        };
        for (int i = 0; i < 2 && i < n; ++i) scores(i);
        for (int i = 0; ok && i < n; ++i) {
          const int s = i & 1;
          const uint32_t k = tiles + (per == 2 ? i >> 1 : i), st = k & 1;
          ok = wait(&bar.v_full[st], (k >> 1) & 1) && wait(&bar.p_full[s], items[s] & 1);
          if (!ok) break;
          ++items[s];
          tmem_fence_after();
          const uint64_t v = mma_operand(smem_addr(sv + st * TB), kHalf);
#pragma unroll
          for (int j = 0; j < kTile / 16; ++j) {
            const uint32_t p = at_s(s) + 32 * (j >> 1) + 8 * (j & 1);
            mma_ts(at_o(s), p, v + j * (2048 >> 4), KIND_O, i >= 2 || j != 0);
            if (LO) mma_ts(at_o(s), p + 16, v + j * (2048 >> 4), KIND_O, true);
          }
          if (per == 1 || s == 1) mma_commit(&bar.v_free[st]);
          if (i + 2 >= n) mma_commit(&bar.o_full[s]);
          if (i + 2 < n) scores(i + 2);
        }
        tiles += part.t1 - part.t0;
        ++parts;
      }
      if (!ok) {  // what was issued is done before the block leaves
        mma_commit(&bar.drained);
        bar_wait(&bar.drained, 0);
      }
    }
    __syncwarp();
  } else {
    // ================================================ softmax: a thread a row of its stream
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's first lane, in an address
    const uint32_t my_s = at_s(s) + lanes, my_o = at_o(s) + lanes;
    uint32_t items = 0, outs = 0, exchanges = 0;
    bool ok = true;
    while (ok && walk.next(a, part)) {
      const bool two = part.rows > 128;
      const int per = two ? 2 : 1, n_items = (part.t1 - part.t0) * per;
      // ---- the row's query, scaled by a power of two into fp16's range
      const int i_row = part.group * kRows + (two ? 128 * s : 0) + r;
      const bool inside = i_row < part.group * kRows + part.rows;
      const QueryRow qr = query_row(a, part.p, i_row, grp);
      const bool live = inside && qr.live;
      float rf = 0.f;
      {
        uint32_t x[HD / 2];
        float mx = 0.f;
        const int h = part.g * grp + i_row % grp;
        const int64_t o = qr.b * a.q.sb + qr.t * a.q.st + h * a.q.sh;
#pragma unroll
        for (int d = 0; d < HD; d += 8) {
          uint4 y = make_uint4(0, 0, 0, 0);
          if (live) {
            if (a.q_f32) {
              const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q.p) + o + d);
              const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q.p) + o + d + 4);
              y = make_uint4(pack_act2(u.x, u.y, c.act), pack_act2(u.z, u.w, c.act), pack_act2(v.x, v.y, c.act), pack_act2(v.z, v.w, c.act));
            } else {
              y = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q.p) + o + d);
            }
          }
          x[d / 2] = y.x; x[d / 2 + 1] = y.y; x[d / 2 + 2] = y.z; x[d / 2 + 3] = y.w;
        }
#pragma unroll
        for (int d = 0; d < HD / 2; ++d)
          mx = fmaxf(mx, fmaxf(fabsf(act_to_f((uint16_t)x[d], c.act)), fabsf(act_to_f((uint16_t)(x[d] >> 16), c.act))));
        constexpr int QE = 4;  // the largest element in [2^4, 2^5): both exponents below stay those of normal numbers
        const int e = max(min((int)(__float_as_uint(mx) >> 23), 254) - 127, QE - 126);
        const float down = copysignf(__uint_as_float((uint32_t)(127 + QE - e) << 23), a.scale);  // the scale's sign goes to the query
        rf = __uint_as_float((uint32_t)(127 + e - QE) << 23) * fabsf(a.scale) * kLog2e;
        if (mx == INFINITY) rf = __int_as_float(0x7fc00000);
        unsigned char *row = sq + s * TB + r * 128;
#pragma unroll
        for (int d = 0; d < HD / 2; d += 4) {
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = kv8a::pack_h2(act_to_f((uint16_t)x[d + k], c.act) * down, act_to_f((uint16_t)(x[d + k] >> 16), c.act) * down);
          const int piece = d / 4;
          *reinterpret_cast<uint4 *>(row + (piece >> 3) * kHalf + (((piece & 7) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(&bar.q_full[s]);
      // ---- items
      const bool some = __any_sync(0xffffffffu, live);  // rows that no one asks for need no weights
      const int nb = kTile >> lb;                       // blocks of a tile: their K scales in lanes 0.., their V scales in lanes 8..
      float m = kv8a::kUnseen, l = 0.f, scales = 0.f;
      int e = -200;  // V scales are taken in units of 2^e
      auto fetch = [&](int i) {
        const int t = part.t0 + (two ? i >> 1 : i), at = t * kTile + ((lane & 7) << lb);
        scales = 0.f;
        if (i < n_items && lane < 16 && (lane & 7) < nb && at < part.n) scales = c.scale[lane >> 3][part.kv * (c.N >> lb) + (at >> lb)];
      };
      fetch(s);
      bool any = false;
      for (int i = s; i < n_items; i += 2) {
        const int edge = part.n - (part.t0 + (two ? i >> 1 : i)) * kTile;  // positions of the tile that there are
        const float sc = scales;
        fetch(i + 2);
        ok = wait_warp(&bar.s_full[s], items & 1);
        ++items;
        if (!ok) break;
        tmem_fence_after();
        if (some) {
          auto factor = [&](int col) { return __fmul_rn(__shfl_sync(0xffffffffu, sc, col >> lb), rf); };
          // the row's largest score
          float top = -INFINITY;
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t x[32];
            tmem_load32(my_s + 32 * ch, x);
            tmem_wait_load(x);
            if (32 * ch + 32 > edge) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (32 * ch + k >= edge) x[k] = 0xff800000u;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float y = __uint_as_float(x[16 * h]);
#pragma unroll
              for (int k = 1; k < 15; k += 2) y = kv8a::max3(y, __uint_as_float(x[16 * h + k]), __uint_as_float(x[16 * h + k + 1]));
              y = fmaxf(y, __uint_as_float(x[16 * h + 15]));
              top = fmaxf(top, __fmul_rn(y, factor(32 * ch + 16 * h)));  // (a NaN, of a block that is not seen or is one, is passed over)
            }
          }
          // the references: scores', a power of two above the V scales
          int ve = lane >= 8 && lane < 16 ? (int)(__float_as_uint(sc) >> 23) - 126 : -200;
          if (ve > 128) ve = -200;  // NaN
          ve = __reduce_max_sync(0xffffffffu, ve);
          if (__any_sync(0xffffffffu, top - m > kv8a::kLag) || ve > e) {
            const float to = top - m > kv8a::kLag ? top - kv8a::kTop : m, al = ex2(m - to);
            const int en = max(e, ve);
            l *= al;
            if (any) {
              const float f = al * ex2((float)max(e - en, -200));
#pragma unroll
              for (int ch = 0; ch < HD / 32; ++ch) {
                uint32_t x[32];
                tmem_load32(my_o + 32 * ch, x);
                tmem_wait_load(x);
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                tmem_store32(my_o + 32 * ch, x);
              }
            }
            m = to;
            e = en;
          }
          const float unit = __uint_as_float((uint32_t)min(max(127 - e, 1), 254) << 23);  // 2^-e
          // weights
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t x[32], y[16], z[16];
            tmem_load32(my_s + 32 * ch, x);
            tmem_wait_load(x);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = factor(32 * ch + 16 * h), vr = __shfl_sync(0xffffffffu, sc, 8 + ((32 * ch + 16 * h) >> lb)) * unit;
#pragma unroll
              for (int k = 16 * h; k < 16 * h + 16; ++k)  // the score is rounded before the reference is taken off (kv8_attention.cuh)
                x[k] = __float_as_uint(ex2(__fadd_rn(__fmul_rn(__uint_as_float(x[k]), f), -m)));
              if (32 * ch + 16 * h + 16 > edge) {  // what is not there weighs nothing, whatever its scale
#pragma unroll
                for (int k = 16 * h; k < 16 * h + 16; ++k)
                  if (32 * ch + k >= edge) x[k] = 0;
              }
#pragma unroll
              for (int k = 16 * h; k < 16 * h + 16; ++k) {
                l += __uint_as_float(x[k]);
                x[k] = __float_as_uint(__uint_as_float(x[k]) * vr);
              }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float u = __uint_as_float(x[2 * k]), v = __uint_as_float(x[2 * k + 1]);
              y[k] = kv8a::pack_h2(u, v);
              if (LO) {
                const float2 hi = __half22float2(kv8a::bits_h2(y[k]));
                z[k] = kv8a::pack_h2(u - hi.x, v - hi.y);
              }
            }
            tmem_store16(my_s + 32 * ch, y);
            if (LO) tmem_store16(my_s + 32 * ch + 16, z);
          }
          tmem_wait_store();
        }
        any = true;
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar.p_full[s]);
      }
      // ---- the part's state
      if (ok && any) ok = wait_warp(&bar.o_full[s], outs++ & 1);
      if (!ok) break;
      tmem_fence_after();
      if (!any) m = -INFINITY;
      float *slot = a.slots + part.slot * slot_floats(a.slot_rows, HD);
      float *ml = slot + (size_t)a.slot_rows * HD;
      e = max(e, -126);
      auto put = [&](float *to, const uint32_t (&x)[32]) {
#pragma unroll
        for (int k = 0; k < 32; k += 8)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + k), "r"(x[k]), "r"(x[k + 1]), "r"(x[k + 2]), "r"(x[k + 3]),
                       "r"(x[k + 4]), "r"(x[k + 5]), "r"(x[k + 6]), "r"(x[k + 7])
                       : "memory");
      };
      auto power = [&](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };
      if (two) {
        const int rr = 128 * s + r;
        const float f = power(e);
#pragma unroll
        for (int ch = 0; ch < HD / 32; ++ch) {
          uint32_t x[32];
          tmem_load32(my_o + 32 * ch, x);
          tmem_wait_load(x);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * (1.f / kOutUnit) * f);
          if (live) put(slot + (size_t)rr * HD + 32 * ch, x);
          __syncwarp();
        }
        if (live) *reinterpret_cast<float2 *>(ml + 2 * rr) = make_float2(m, l);
      } else {  // the streams' rows are the same: each joins half of the elements
        side.m[s][r] = m;
        side.l[s][r] = l;
        if (lane == 0) side.e[s][warp & 3] = e;
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar.exchange);
        ok = wait_warp(&bar.exchange, exchanges++ & 1);
        if (!ok) break;
        tmem_fence_after();
        const float m0 = side.m[0][r], m1 = side.m[1][r], mm = fmaxf(m0, m1), f0 = ex2(m0 - mm), f1 = ex2(m1 - mm);
        const float g0 = f0 * power(side.e[0][warp & 3]), g1 = f1 * power(side.e[1][warp & 3]);
#pragma unroll
        for (int ch = 0; ch < HD / 64; ++ch) {
          const int at = 32 * (s * (HD / 64) + ch);
          uint32_t x[32];
          tmem_load32(at_o(0) + lanes + at, x);
          tmem_wait_load(x);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * (1.f / kOutUnit) * g0);
          if (n_items > 1) {
            uint32_t y[32];
            tmem_load32(at_o(1) + lanes + at, y);
            tmem_wait_load(y);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(fmaf(__uint_as_float(y[k]) * (1.f / kOutUnit), g1, __uint_as_float(x[k])));
          }
          if (live) put(slot + (size_t)r * HD + at, x);
          __syncwarp();
        }
        if (live && s == 0) *reinterpret_cast<float2 *>(ml + 2 * r) = make_float2(mm, side.l[0][r] * f0 + side.l[1][r] * f1);
      }
      tmem_fence_before();  // (the next part's products write what was read here)
    }
  }
  pdl_trigger();
  tmem_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kCodeWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <int FMT, int HD, bool LO>
cudaError_t launch_prefix_t(const SharedArgs &a, int n_sm, cudaStream_t s) {
  auto fn = k_prefix<FMT, HD, LO>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, prefix_smem(HD));
  if (e != cudaSuccess) return e;
  return launch_k(fn, dim3(n_sm), dim3(kThreads), prefix_smem(HD), s, 1, a);
}
template <int FMT>
cudaError_t launch_prefix_fmt(const SharedArgs &a, int n_sm, cudaStream_t s) {
  if (a.c.hd == 64) return a.lo ? launch_prefix_t<FMT, 64, true>(a, n_sm, s) : launch_prefix_t<FMT, 64, false>(a, n_sm, s);
  return a.lo ? launch_prefix_t<FMT, 128, true>(a, n_sm, s) : launch_prefix_t<FMT, 128, false>(a, n_sm, s);
}
cudaError_t launch_prefix_int8(const SharedArgs &a, int n_sm, cudaStream_t s);
cudaError_t launch_prefix_e4m3(const SharedArgs &a, int n_sm, cudaStream_t s);

}  // namespace kv8s
}  // namespace rv
