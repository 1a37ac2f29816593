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
// A block per SM: 4 or 8 warps turn codes to fp16, one thread issues the
// products, 8 warps in two streams do the softmax, so that one's products run
// under the other's weights.  Up to 128 query rows, the streams take every other
// tile of positions and are joined at the end; with more, each has its 128 rows.
// With 32 or 64 rows at most, the rows are there four times or twice, each time
// for another part of a tile's positions (the others' weights are zero): the
// products would take as long with empty rows, and so all warps share the
// weights (16 prompts of 8 rows 60 -> 52 us with the rest; 52 to 57 from run to run).
//
// What bounds it: the chain S, weights, O of a stream.  For 256 query rows behind
// 32,768 positions of 8 KV heads of 128 (a piece of 13.5 tiles for each SM) a
// tile takes some 4,800 cycles, 2 x 1,040 of them products back to back (which is
// what they take alone); of a stream's 4,800, 2,300 are softmax (max 620, weights
// 1,500: 276 cycles per 32 positions alone, 380 here) and the rest products and
// hand-overs (a wait on an mbarrier takes 200 cycles, done or not).  Measured and
// dropped: two warps a row quarter, each half of the positions (72 registers, no
// faster: 81.8 against 80.9 us then); a warp for each stream's products, taking
// turns or not (the streams fall in step: 82.1 and 79.3 against 73.4 us); one lane
// that asks for its warp (95.5); the next scores under way during the weights
// (spills); hints of time with the waits, naps between tries (no change).  The
// beginning takes 6 us (codes, queries and instructions come from far), the
// states' way out 4: 152 blocks leave 256 rows of 512 bytes each.
#pragma once

#include <type_traits>

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
  int32_t *line;  // [P + 1]: where each prefix row's units begin in the line, the length of a piece
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
constexpr int kMinTiles = 1;  // of a piece (2: 13.1 us instead of 12.1 behind 200 positions; 4: 20.8)
struct Piece {
  int begin, end, off, p, n;  // off: into row p; n: its length, if known (else -1)
};
template <int THREADS>
__device__ __forceinline__ Piece cut_line(const SharedArgs &a, int *scratch /* THREADS + 2 */) {
  const int tid = threadIdx.x, units = a.c.Hkv * a.groups;
  Piece w{0, 0, 0, 0, -1};
  if (a.P == 1) {
    w.n = prefix_len(a, 0);
    const int total = units * ((w.n + kTile - 1) / kTile), piece = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinTiles);
    w.begin = w.off = min(total, piece * (int)blockIdx.x);
    w.end = min(total, w.begin + piece);
    if (blockIdx.x == 0 && tid == 0) {
      a.line[0] = 0;
      a.line[1] = piece;
    }
    return w;
  }
  const int per = (a.P + THREADS - 1) / THREADS, p0 = min(a.P, tid * per), p1 = min(a.P, p0 + per);
  int mine = 0;
  for (int p = p0; p < p1; ++p) mine += units * prefix_tiles(a, p);
  scratch[tid] = mine;
  __syncthreads();
  int before = 0, total = 0;
  for (int i = 0; i < min(THREADS, a.P); ++i) {  // (the others have none)
    const int x = scratch[i];
    if (i < tid) before += x;
    total += x;
  }
  const int piece = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinTiles);
  w.begin = min(total, piece * (int)blockIdx.x);
  w.end = min(total, w.begin + piece);
  int at = before;
  for (int p = p0; p < p1; ++p) {
    const int n = units * prefix_tiles(a, p);
    if (blockIdx.x == 0) a.line[p] = at;
    if (w.begin >= at && w.begin < at + n) {
      scratch[THREADS] = p;
      scratch[THREADS + 1] = w.begin - at;
    }
    at += n;
  }
  if (blockIdx.x == 0 && tid == 0) a.line[a.P] = piece;
  __syncthreads();
  w.p = scratch[THREADS];
  w.off = scratch[THREADS + 1];
  return w;
}

// ------------------------------------------------------------------ the prefix

constexpr int kSoftWarps = 8;
// Warps that turn codes to fp16: 4 for K and V, or 4 for each where tiles are
// short and follow one another sooner.  (4 / 8, with 128 / 96 registers a thread:
// head_dim 128, 64 rows behind 32K positions 69.5 / 73.4 us; 64, 16 prompts of 8
// rows 57.3 / 51.7, each in one run: see above.)
__host__ __device__ constexpr int code_warps(int hd) { return hd == 128 ? 4 : 8; }
__host__ __device__ constexpr int threads_of(int hd) { return 32 * (kSoftWarps + code_warps(hd) + 1); }
constexpr int kHalf = 16384;  // 128 rows of 64 fp16
__host__ __device__ constexpr int tile_bytes(int hd) { return hd / 64 * kHalf; }
struct Bars {
  uint64_t full[2][2], free[2][2];                      // stages of K and of V
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];  // streams
  uint64_t exchange, drained;
};
// What the streams' warps tell each other of a part: rows by stream.
struct Told {
  float m[2][128], l[2][128];
  int e[2][4];
};
// What the block's threads share beside the operands.
struct Side {
  Bars bar;
  Told told[2];  // by turns: a stream without items in a part writes its own before the other is through with the part before
  int scratch[threads_of(64) + 2];
  uint32_t tmem;
  int dead;  // a wait ran out: everyone leaves
};
__host__ __device__ constexpr int prefix_smem(int hd) { return 1024 + 6 * tile_bytes(hd) + (int)sizeof(Side); }

// A part of a unit.
struct Part {
  int p, g, group, t0, t1, n, rows;  // tiles [t0, t1) of the prefix row's n positions; query rows of the unit
  int kv, slot;                      // KV row; slot of the state
};
struct Walk {
  int at, end, off, p, n = -1;  // n: positions of row p, if known
  __device__ __forceinline__ bool next(const SharedArgs &a, Part &s) {
    while (at < end && p < a.P) {  // (p: only if the lengths changed under the kernel)
      if (n < 0) n = prefix_len(a, p);
      const int tiles = (n + kTile - 1) / kTile, in_row = a.c.Hkv * a.groups * tiles;
      if (off >= in_row) { off -= in_row; ++p; n = -1; continue; }
      const int unit = off / tiles, t0 = off - unit * tiles, take = min(tiles - t0, end - at);
      s.p = p;
      s.g = unit / a.groups;
      s.group = unit - s.g * a.groups;
      s.t0 = t0;
      s.t1 = t0 + take;
      s.n = n;
      s.rows = min(kRows, a.rows - s.group * kRows);
      s.kv = p * a.c.Hkv + s.g;
      s.slot = (int)blockIdx.x + s.kv * a.groups + s.group;
      at += take;
      off += take;
      return true;
    }
    return false;
  }
};

// Largest magnitude bits of two 16-bit halves.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
  return r;
}

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
__global__ void __launch_bounds__(threads_of(HD), 1) k_prefix(const __grid_constant__ SharedArgs a) {
  extern __shared__ unsigned char raw[];
  unsigned char *sm = raw + (-smem_addr(raw) & 1023);  // (as an offset, so that the compiler knows it for shared memory)
  constexpr int TB = tile_bytes(HD), kCodeWarps = code_warps(HD);
  constexpr bool APART = kCodeWarps == 8;  // K's and V's warps
  unsigned char *sq = sm, *sk = sm + 2 * TB, *sv = sm + 4 * TB;
  Side &side = *reinterpret_cast<Side *>(sm + 6 * TB);
  Bars &bar = side.bar;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // (the warp's number in a uniform register)
  if (warp == kSoftWarps + kCodeWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&side.tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&bar.full[0][i], 4);
      bar_init(&bar.free[0][i], 1);
      bar_init(&bar.full[1][i], 4);
      bar_init(&bar.free[1][i], 1);
      bar_init(&bar.q_full[i], kSoftWarps / 2);
      bar_init(&bar.s_full[i], 1);
      bar_init(&bar.p_full[i], kSoftWarps / 2);
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, side.tmem, 0);
  // No wait for the kernel before: it reads other positions, and all that this one reads or overwrites was done before it
  // began, since every block of that one has waited for it (the condition that this puts on it: ops.cuh).  Lines of before
  // that may be in this SM are given up (0.4 us).
  __threadfence();
  const Piece piece = cut_line<threads_of(HD)>(a, side.scratch);
  Walk walk{piece.begin, piece.end, piece.off, piece.p, piece.n};
  const Kv8 &c = a.c;
  const int lb = __ffs(c.block) - 1;
  volatile int *dead = &side.dead;
  // Waits are for whole warps.
  auto waited = [&](bool mine) {
    const bool ok = __all_sync(0xffffffffu, mine);
    if (!ok) {
      if (!*dead && a.err) atomicOr(a.err, kErrWait);
      *dead = 1;
    }
    __syncwarp();
    return ok;
  };
  auto wait = [&](uint64_t *b, uint32_t parity) { return waited(bar_wait(b, parity, dead)); };
  // Tensor memory: the streams' scores (and weights), then their O.
  auto at_s = [&](int s) { return tmem + 128 * s; };
  auto at_o = [&](int s) { return tmem + 256 + HD * s; };
  Part part;
  // Items of a part: (stream, tile) = (i & 1, i) where the streams share the rows, (i & 1, i >> 1) where each has its own.

  if (warp >= kSoftWarps && warp < kSoftWarps + kCodeWarps) {
    // ================================================ codes to fp16
    // Thread: 16 codes of position 32 j + 8 w + lane / 4 of the tile, and 64 codes on; a phase of 8 lanes
    // reads 64 bytes of two positions and stores 16-byte pieces that meet all banks.
    constexpr int NC = HD / 16;  // 16-byte loads of a thread and tile
    const int w = warp & 3, p_in = 8 * w + (lane >> 2);
    const int x = p_in & 7, piece = (lane & 3) * 2;
    unsigned char *to0 = sk + p_in * 128 + ((piece ^ x) << 4), *to1 = sk + p_in * 128 + (((piece + 1) ^ x) << 4);
    constexpr int OPS = APART ? 1 : 2;  // K and V, or one of them
    auto which_of = [&](int o) { return APART ? (warp - kSoftWarps) >> 2 : o; };
    uint4 buf[OPS][NC];
    auto load = [&](int o, const Part &s, int t) {
      const int p0 = t * kTile + p_in;
      const uint8_t *from = c.codes[which_of(o)] + ((int64_t)s.kv * c.N + p0) * HD + (lane & 3) * 16;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int half = HD == 128 ? j & 1 : 0, at = 32 * (HD == 128 ? j >> 1 : j);
        buf[o][j] = make_uint4(0, 0, 0, 0);
        if (p0 + at < s.n) buf[o][j] = *reinterpret_cast<const uint4 *>(from + at * HD + half * 64);
      }
    };
    bool more = walk.next(a, part), ok = true;
    if (more)
#pragma unroll
      for (int o = 0; o < OPS; ++o) load(o, part, part.t0);
    int t = part.t0;
    for (uint32_t k = 0; ok && more; ++k) {
      const uint32_t st = k & 1;
      if (++t == part.t1) {
        more = walk.next(a, part);
        t = part.t0;
      }
#pragma unroll
      for (int o = 0; o < OPS; ++o) {
        const int which = which_of(o);
        ok = ok && waited(bar_wait<100>(&bar.free[which][st], ((k >> 1) & 1) ^ 1, dead));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const int off = which * 2 * TB + st * TB + (HD == 128 ? j & 1 : 0) * kHalf + 32 * 128 * (HD == 128 ? j >> 1 : j);
          const uint4 b = buf[o][j];
          const uint2 y0 = codes4<FMT>(b.x), y1 = codes4<FMT>(b.y), y2 = codes4<FMT>(b.z), y3 = codes4<FMT>(b.w);
          *reinterpret_cast<uint4 *>(to0 + off) = make_uint4(y0.x, y0.y, y1.x, y1.y);
          *reinterpret_cast<uint4 *>(to1 + off) = make_uint4(y2.x, y2.y, y3.x, y3.y);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar.full[which][st]);
        if (more) load(o, part, t);
      }
    }
  } else if (warp == kSoftWarps + kCodeWarps) {
    // ================================================ products
    constexpr uint32_t KIND = 1u << 4 | (uint32_t)(kTile >> 4) << 24;  // fp16, fp32 sums, 128 rows
    constexpr uint32_t KIND_S = KIND | (uint32_t)(kTile >> 3) << 17, KIND_O = KIND | (uint32_t)(HD >> 3) << 17 | 1u << 16;  // V: elements contiguous
    const uint64_t q_op = mma_operand(smem_addr(sq), 16), k_op = mma_operand(smem_addr(sk), 16), v_op = mma_operand(smem_addr(sv), kHalf);
    uint32_t tiles = 0, parts = 0, items = 0;  // items: of the streams, a bit each (the parity)
    bool ok = true;
    while (ok && walk.next(a, part)) {
      const int per = part.rows > 128 ? 2 : 1, n = (part.t1 - part.t0) * per;
      for (int s = 0; ok && s < 2; ++s) ok = wait(&bar.q_full[s], parts & 1);
      auto tile_of = [&](int i) { return tiles + (per == 2 ? i >> 1 : i); };
      auto there = [&](int which, int i) { return wait(&bar.full[which][tile_of(i) & 1], (tile_of(i) >> 1) & 1); };
      auto scores = [&](int i) {
        const int s = i & 1;
        const uint32_t st = tile_of(i) & 1;
        const uint64_t q = q_op + s * (TB >> 4), kk = k_op + st * (TB >> 4);
        const uint32_t d = at_s(s);
#pragma unroll
        for (int j = 0; j < HD / 16; ++j) mma_ss(d, q + (((j >> 2) * kHalf + (j & 3) * 32) >> 4), kk + (((j >> 2) * kHalf + (j & 3) * 32) >> 4), KIND_S, j != 0);
        mma_commit(&bar.s_full[s]);
        if (per == 1 || s == 1) mma_commit(&bar.free[0][st]);
      };
      for (int i = 0; ok && i < 2 && i < n; ++i) {
        ok = there(0, i);
        if (!ok) break;
        tmem_fence_after();
        if (elect_one()) scores(i);
        __syncwarp();
      }
      for (int i = 0; ok && i < n; ++i) {
        const int s = i & 1;
        const uint32_t st = tile_of(i) & 1;
        // (what is waited for last is what comes last: a wait takes some 200 cycles, done or not, and none lies between the two products)
        ok = there(1, i) && (i + 2 >= n || there(0, i + 2)) && wait(&bar.p_full[s], (items >> s) & 1);
        if (!ok) break;
        items ^= 1u << s;
        tmem_fence_after();
        const uint64_t v = v_op + st * (TB >> 4);
        const uint32_t d = at_o(s), p = at_s(s);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kTile / 16; ++j) {
            mma_ts(d, p + 32 * (j >> 1) + 8 * (j & 1), v + j * (2048 >> 4), KIND_O, i >= 2 || j != 0);
            if (LO) mma_ts(d, p + 32 * (j >> 1) + 8 * (j & 1) + 16, v + j * (2048 >> 4), KIND_O, true);
          }
          if (per == 1 || s == 1) mma_commit(&bar.free[1][st]);
          if (i + 2 >= n) mma_commit(&bar.o_full[s]);
          else scores(i + 2);
        }
        __syncwarp();
      }
      tiles += part.t1 - part.t0;
      ++parts;
    }
    if (!ok) {  // what was issued is done before the block leaves
      if (elect_one()) mma_commit(&bar.drained);
      __syncwarp();
      bar_wait(&bar.drained, 0);
    }
  } else {
    // ================================================ softmax: a thread a row of its stream
    const int s = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)quarter << 21;  // the warp's first lane, in an address
    const uint32_t my_s = at_s(s) + lanes, my_o = at_o(s) + lanes;
    const int grp = a.H / c.Hkv, nb = kTile >> lb;  // blocks of a tile: their K scales in lanes 0.., their V scales in lanes 8..
    uint32_t items = 0, outs = 0, exchanges = 0, turn = 0;
    bool ok = true;
    while (ok && walk.next(a, part)) {
      const bool two = part.rows > 128;
      const int per = two ? 1 : 2, tiles = part.t1 - part.t0;  // tiles from one item of the stream to its next
      // ---- queries, scaled by a power of two into fp16's range
      const int times = two || part.rows > 64 ? 1 : part.rows > 32 ? 2 : 4, span = kTile / times;  // copies of the rows, positions of each
      const int i_row = r & (span - 1), copy = r / span, row0 = part.group * kRows + (two ? 128 * s : 0), end = part.group * kRows + part.rows;
      const QueryRow qr = query_row(a, part.p, row0 + i_row, grp);
      const bool live = row0 + i_row < end && qr.live;
      const int64_t my_q = live ? qr.b * a.q.sb + qr.t * a.q.st + (part.g * grp + (row0 + i_row) % grp) * a.q.sh : -1;
      auto q_piece = [&](int row, int k) { return reinterpret_cast<uint4 *>(sq + s * TB + row * 128 + (k >> 3) * kHalf + (((k & 7) ^ (row & 7)) << 4)); };
      float rf;
      {
        // the warp's rows as they are into their place, whole rows at a time; then each thread turns its own
        constexpr int LR = HD / 8, RI = 32 / LR, NI = 32 / RI;  // lanes of a row, rows of a turn, turns
        const int piece = lane % LR;
        if (a.q_f32) {
#pragma unroll 4
          for (int k = 0; k < NI; ++k) {
            const int64_t o = __shfl_sync(0xffffffffu, my_q, k * RI + lane / LR);
            float4 u = make_float4(0, 0, 0, 0), v = u;
            if (o >= 0) {
              u = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q.p) + o + 8 * piece);
              v = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q.p) + o + 8 * piece + 4);
            }
            *q_piece(quarter * 32 + k * RI + lane / LR, piece) =
                make_uint4(pack_act2(u.x, u.y, c.act), pack_act2(u.z, u.w, c.act), pack_act2(v.x, v.y, c.act), pack_act2(v.z, v.w, c.act));
          }
        } else {
          uint4 y[NI];  // all on their way at once: behind the first tiles' codes, which every block asks for now, each turn would wait some 2 us
#pragma unroll
          for (int k = 0; k < NI; ++k) {
            const int64_t o = __shfl_sync(0xffffffffu, my_q, k * RI + lane / LR);
            y[k] = make_uint4(0, 0, 0, 0);
            if (o >= 0) y[k] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q.p) + o + 8 * piece);
          }
#pragma unroll
          for (int k = 0; k < NI; ++k) *q_piece(quarter * 32 + k * RI + lane / LR, piece) = y[k];
        }
        __syncwarp();
        uint32_t top = 0;
#pragma unroll 4
        for (int k = 0; k < HD / 8; ++k) {
          const uint4 y = *q_piece(r, k);
          top = max_magnitude(max_magnitude(max_magnitude(max_magnitude(top, y.x), y.y), y.z), y.w);
        }
        top = max(top & 0xffffu, top >> 16);
        const float mx = act_to_f((uint16_t)top, c.act);
        constexpr int QE = 4;  // the largest element in [2^4, 2^5): both exponents below stay those of normal numbers
        const int e = max(min((int)(__float_as_uint(mx) >> 23), 254) - 127, QE - 126);
        const float down = copysignf(__uint_as_float((uint32_t)(127 + QE - e) << 23), a.scale);  // the scale's sign goes to the query
        rf = mx < INFINITY ? __uint_as_float((uint32_t)(127 + e - QE) << 23) * fabsf(a.scale) * kLog2e : __int_as_float(0x7fc00000);
        auto turn = [&](auto bf16) {
#pragma unroll 4
          for (int k = 0; k < HD / 8; ++k) {
            const uint4 y = *q_piece(r, k);
            auto scaled = [&](uint32_t w) {
              if (decltype(bf16)::value) return kv8a::pack_h2(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down);
              const float2 v = __half22float2(kv8a::bits_h2(w));
              return kv8a::pack_h2(v.x * down, v.y * down);
            };
            *q_piece(r, k) = make_uint4(scaled(y.x), scaled(y.y), scaled(y.z), scaled(y.w));
          }
        };
        if (c.act == RV_BF16) turn(std::true_type{});
        else turn(std::false_type{});
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(&bar.q_full[s]);
      // ---- items
      const int from = copy * span, to = from + span;   // this row's positions of a tile
      const bool some = __any_sync(0xffffffffu, live);  // rows that no one asks for need no weights
      float m = kv8a::kUnseen, scales = 0.f;
      F2 l[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
      int e = -200;  // V scales are taken in units of 2^e
      int t = two ? 0 : s, edge = part.n - (part.t0 + t) * kTile;  // the item's tile, from t0; positions of it that there are
      // this lane's scale of the next item: block lane & 7 of the tile
      const float *scale_at = c.scale[(lane >> 3) & 1] + (int64_t)part.kv * (c.N >> lb) + ((part.t0 + t) * nb + (lane & 7));
      const int scale_from = (lane & 7) << lb;
      const bool scale_lane = lane < 16 && (lane & 7) < nb;
      auto fetch = [&](int t, int edge) {
        scales = 0.f;
        if (scale_lane && t < tiles && scale_from < edge) scales = *scale_at;
        scale_at += per * nb;
      };
      fetch(t, edge);
      bool any = false;
      for (; t < tiles; t += per, edge -= per * kTile) {
        const float sc = scales;
        fetch(t + per, edge - per * kTile);
        ok = wait(&bar.s_full[s], items & 1);
        ++items;
        if (!ok) break;
        tmem_fence_after();
        if (some) {
          auto factor = [&](int col) { return __fmul_rn(__shfl_sync(0xffffffffu, sc, col >> lb), rf); };
          // the row's largest score
          float top = -INFINITY;
#pragma unroll 1
          for (int ch = from; ch < to; ch += 32) {
            uint32_t x[32];
            tmem_load32(my_s + ch, x);
            tmem_wait_load(x);
#pragma unroll 1
            for (int turn = ch + 32 > edge; turn > 0; --turn) {  // (a loop of one turn or none stays a branch: predicated, it would cost every tile)
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (ch + k >= edge) x[k] = 0xff800000u;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t *v = x + 16 * h;
              float y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[k] = kv8a::max3(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]), fmaxf(__uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3])));
              top = fmaxf(top, __fmul_rn(kv8a::max3(y[0], y[1], fmaxf(y[2], y[3])), factor(ch + 16 * h)));  // (a NaN is passed over)
            }
          }
          // the references: scores', and a power of two above the V scales
          int ve = (lane & 24) == 8 ? (int)(__float_as_uint(sc) >> 23) - 126 : -200;
          if (ve > 128) ve = -200;  // NaN
          ve = __reduce_max_sync(0xffffffffu, ve);
          if (__any_sync(0xffffffffu, top - m > kv8a::kLag) || ve > e) {
            const float next = top - m > kv8a::kLag ? top - kv8a::kTop : m, al = ex2(m - next);
            const int en = max(e, ve);
            l[0] = f2_mul(l[0], f2(al, al));
            l[1] = f2_mul(l[1], f2(al, al));
            if (any) {
              const float g = al * ex2((float)max(e - en, -200));
#pragma unroll 1
              for (int ch = 0; ch < HD / 32; ++ch) {
                uint32_t x[32];
                tmem_load32(my_o + 32 * ch, x);
                tmem_wait_load(x);
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * g);
                tmem_store32(my_o + 32 * ch, x);
              }
            }
            m = next;
            e = en;
          }
          const float unit = __uint_as_float((uint32_t)min(max(127 - e, 1), 254) << 23);  // 2^-e
          const F2 neg = f2(-m, -m);
          // Weights.  Scores are taken by their factor and off the reference in one step; where they are so large that
          // the reference's own rounding would be more than a quarter, the product is rounded first, as the reference was.
          const bool large = __any_sync(0xffffffffu, fabsf(m) > 4194304.f);
          // a chunk of 32 positions: its scores, scaled by f and off the reference, become weights
          auto weigh = [&](int ch, uint32_t (&v)[32], const F2 (&f)[2], int have) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int k = 16 * h; k < 16 * h + 16; k += 2) {
                const float2 w = f2_split(f2_fma(f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), f[h], neg));
                v[k] = __float_as_uint(ex2(w.x));
                v[k + 1] = __float_as_uint(ex2(w.y));
                if (have < 32) {  // what is not there weighs nothing, whatever its scale
                  if (k >= have) v[k] = 0;
                  if (k + 1 >= have) v[k + 1] = 0;
                }
              }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float vr = __shfl_sync(0xffffffffu, sc, 8 + ((ch + 16 * h) >> lb)) * unit;
              const F2 vv = f2(vr, vr);
              uint32_t y[8], z[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const F2 w = f2(__uint_as_float(v[16 * h + 2 * k]), __uint_as_float(v[16 * h + 2 * k + 1]));
                l[k & 1] = f2_add(l[k & 1], w);
                const float2 u = f2_split(f2_mul(w, vv));
                y[k] = kv8a::pack_h2(u.x, u.y);
                if (LO) {
                  const float2 hi = __half22float2(kv8a::bits_h2(y[k]));
                  z[k] = kv8a::pack_h2(u.x - hi.x, u.y - hi.y);
                }
              }
              tmem_store8(my_s + ch + 8 * h, y);
              if (LO) tmem_store8(my_s + ch + 16 + 8 * h, z);
            }
          };
          if (times > 1) {  // other copies' positions
            const uint32_t none[8] = {};
            for (int ch = 0; ch < kTile; ch += 32)
              if (ch < from || ch >= to) {
                tmem_store8(my_s + ch, none);
                tmem_store8(my_s + ch + 8, none);
                if (LO) {
                  tmem_store8(my_s + ch + 16, none);
                  tmem_store8(my_s + ch + 24, none);
                }
              }
          }
          if (edge >= kTile && !large) {
#pragma unroll 1
            for (int ch = from; ch < to; ch += 32) {
              uint32_t v[32];
              tmem_load32(my_s + ch, v);
              const float f0 = factor(ch), f1 = factor(ch + 16);
              const F2 f[2] = {f2(f0, f0), f2(f1, f1)};
              tmem_wait_load(v);
              weigh(ch, v, f, 32);
            }
          } else {  // (apart: branches inside would keep the exponentials and the rest from running side by side, 364 cycles a chunk against 276)
#pragma unroll 1
            for (int ch = from; ch < to; ch += 32) {
              uint32_t v[32];
              tmem_load32(my_s + ch, v);
              float f0 = factor(ch), f1 = factor(ch + 16);
              tmem_wait_load(v);
              if (large) {
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__fmul_rn(__uint_as_float(v[k]), k < 16 ? f0 : f1));
                f0 = f1 = 1.f;
              }
              const F2 f[2] = {f2(f0, f0), f2(f1, f1)};
              weigh(ch, v, f, edge - ch);
            }
          }
          tmem_wait_store();
        }
        any = true;
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar.p_full[s]);
      }
      if (!ok) break;
      // ---- the part's state
      if (any) ok = wait(&bar.o_full[s], outs++ & 1);
      if (!ok) break;
      if (!any) m = -INFINITY;
      Told &told = side.told[turn];
      turn ^= 1;
      const float2 l2 = f2_split(f2_add(l[0], l[1]));
      told.l[s][r] = l2.x + l2.y;
      told.m[s][r] = m;
      if (lane == 0) told.e[s][quarter] = max(e, -126);
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&bar.exchange);
      ok = wait(&bar.exchange, exchanges++ & 1);
      if (!ok) break;
      tmem_fence_after();
      float *slot = a.slots + part.slot * slot_floats(a.slot_rows, HD);
      float *ml = slot + (size_t)a.slot_rows * HD;
      auto power = [&](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };
      // O in units of 2^40 and of m's reference: the stream's own rows, or half of the elements of both streams' rows
      const int other = two ? s : s ^ 1, rr = two ? 128 * s + r : i_row;
      float mm = fmaxf(told.m[s][r], told.m[other][r]);
      for (int k = 0; k < times; ++k) mm = fmaxf(mm, fmaxf(told.m[s][k * span + i_row], told.m[other][k * span + i_row]));
      const float g0 = ex2(told.m[s][r] - mm) * power(told.e[s][quarter]), g1 = ex2(told.m[other][r] - mm) * power(told.e[other][quarter]);
      const bool others = !two && (s == 1 || tiles > 1);
      const int c0 = two ? 0 : s * (HD / 2), c1 = two ? HD : c0 + HD / 2;
      // with copies: through the queries' place (a row HD / 2 numbers, 16-byte pieces by piece ^ (row mod 8)), and summed
      auto put = [&](int row, int k) { return reinterpret_cast<float4 *>(sq + s * TB + row * (HD * 2) + ((k ^ (row & 7)) << 4)); };
#pragma unroll 1
      for (int at = c0; at < c1; at += 32) {
        uint32_t x[32];
        if (any) {
          tmem_load32(my_o + at, x);
          tmem_wait_load(x);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * (1.f / kOutUnit) * g0);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = 0;
        }
        if (others) {
          uint32_t y[32];
          tmem_load32(at_o(other) + lanes + at, y);
          tmem_wait_load(y);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(fmaf(__uint_as_float(y[k]) * (1.f / kOutUnit), g1, __uint_as_float(x[k])));
        }
        if (times > 1) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *put(r, (at - c0 + k) / 4) = make_float4(__uint_as_float(x[k]), __uint_as_float(x[k + 1]), __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
        } else if (live) {
          float *to = slot + (size_t)rr * HD + at;
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + k), "r"(x[k]), "r"(x[k + 1]), "r"(x[k + 2]), "r"(x[k + 3]),
                         "r"(x[k + 4]), "r"(x[k + 5]), "r"(x[k + 6]), "r"(x[k + 7])
                         : "memory");
        }
        __syncwarp();
      }
      if (live && copy == 0 && (two || s == 0)) {
        float sum = 0.f;
        for (int k = 0; k < times; ++k) {
          sum = fmaf(told.l[s][k * span + i_row], ex2(told.m[s][k * span + i_row] - mm), sum);
          if (!two) sum = fmaf(told.l[1][k * span + i_row], ex2(told.m[1][k * span + i_row] - mm), sum);
        }
        *reinterpret_cast<float2 *>(ml + 2 * rr) = make_float2(mm, sum);
      }
      if (times > 1) {
        if (lane == 0) bar_arrive(&bar.exchange);
        ok = wait(&bar.exchange, exchanges++ & 1);
        if (!ok) break;
        for (int k = r; k < part.rows * (HD / 8); k += 128) {
          const int row = k / (HD / 8), piece = k % (HD / 8);
          float4 x = *put(row, piece);
          for (int t = 1; t < times; ++t) {
            const float4 y = *put(t * span + row, piece);
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
          }
          *reinterpret_cast<float4 *>(slot + (size_t)row * HD + c0 + 4 * piece) = x;  // (rows that no one asks for too: of the slot, and not read)
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&bar.exchange);
        ok = wait(&bar.exchange, exchanges++ & 1);  // before the next queries take the place
        if (!ok) break;
      }
      tmem_fence_before();  // (the next part's products write what was read here)
    }
  }
  pdl_trigger();
  tmem_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kCodeWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  pdl_wait();  // the join, which waits for this kernel, needs the one before too
}

template <int FMT, int HD, bool LO>
cudaError_t launch_prefix_t(const SharedArgs &a, int n_sm, cudaStream_t s) {
  auto fn = k_prefix<FMT, HD, LO>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, prefix_smem(HD));
  if (e != cudaSuccess) return e;
  return launch_k(fn, dim3(n_sm), dim3(threads_of(HD)), prefix_smem(HD), s, 1, a);
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
