// Attention of a few new tokens per row over the 8-bit K/V cache.
//
// out = sum_p w_p v_p / sum_p w_p, w_p = exp(scale q.k_p - m), in one pass over
// the visible positions with a running maximum m, sum and weighted sum (all
// fp32, exponents in base 2).  k_p = s_block x code, so a score is
// (s_block scale) (q.code): codes go to the tensor pipe as exact fp16 values
// and the block's scale multiplies the fp32 scores; the V scale multiplies
// the block's fp32 partial product.  A query row is scaled by a power of two
// (from its largest magnitude), so bf16 rows fit fp16's range; the power
// returns with the scale.
//
// The products are taken transposed: S^T = K Q^T (16 positions x 8 query rows
// per mma.m16n8k16), O^T = V^T P^T (16 elements x 8 rows).  With 4 to 8 query
// rows per KV head an mma with the queries as its 16 rows would be half
// empty; here a KV head's T x (H / Hkv) rows fill columns of 8 (NT of them),
// and every K and V code is unpacked once for all of them.  P^T moves from
// accumulator to operand layout by movmatrix.  The contraction's order of the
// head elements is free, so a thread takes 16 consecutive bytes of a
// position's K row as its part of four k-steps, and 16 (head_dim 128) or 8
// consecutive bytes of four V rows as its part of two positions' pairs.
//
// Memory bounds it: 2 head_dim bytes per position and KV head, read once.
// Each warp streams its own tiles of 8 KB (32 positions at head_dim 128, 64 at
// 64) through a private ring in shared memory (cp.async, no barriers inside a
// segment).  The (row, KV head, row group) units with their tiles form one
// line that is cut evenly over the resident blocks, whatever the rows'
// lengths: a block computes its own piece of the line from d_pos, finishes
// the units that lie in it and leaves the state (m, l, O) of at most two cut
// ones, which a second kernel, chained by programmatic dependent launch,
// joins.  Short contexts take a cluster per unit instead, which joins through
// distributed shared memory.  fp16 caches and fp32 outputs split each weight
// into a high and a low fp16 term.
//
// Measured on a GB300 (graph of passes, inputs larger than L2): one row of
// 131,000 positions, 8 KV heads of 128: 46.6 us = 5.8 TB/s, 86% of a copy's
// rate (a kernel that only reads the same bytes through the same rings takes
// 41 us; the joining kernel is 3 to 4 of the difference); 64 ragged rows of the
// 1B shape: 54.7 us = 5.7 TB/s.  16 rows of 24 query rows per KV head take 50.6
// us for 149 MB, and no unit is full (DRAM 33%, tensor pipe 36%, issue 36%):
// 255 registers leave two warps per scheduler, and of the 5.5 cycles between a
// warp's instructions 1.6 go to fixed latencies (products that add to one sum,
// transposes), 0.8 to instruction fetch, 0.5 to the full tensor pipe's queue
// and 0.5 to shared and global loads: latency that two warps do not hide.
#pragma once

#include <cuda_fp8.h>

#include "ops.cuh"

namespace rv {
namespace kv8a {

constexpr int kWarps = 4;  // warps of a block
// Positions of a tile: 4 KB of K and 4 KB of V.
__host__ __device__ constexpr int tile_len(int hd) { return hd == 128 ? 32 : 64; }
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Smallest piece of the line a block takes: one tile for each of its warps
// (a unit where units are shorter: short ones side by side, not in a row).
constexpr int kMinTiles = kWarps;
// What beginning a unit costs a block, in tiles (its queries' operands, the
// join of the warps): the line counts it, where pieces are long enough.
// Measured with 0 / 4 / 8 / 12 / 16: 131K positions 55.6 / 48.5 / 47.5 / 48.2 /
// 49.1 us (one column of rows); 24 rows 78 / 56.4 / 53.1 / 51.6 / 53.6, 16 rows
// - / 45.3 / 41.2 / 38.8 / 38.1.
__host__ __device__ constexpr int unit_tiles(int nt) { return nt == 1 ? 8 : 12; }
// Blocks per SM, as many as the registers leave room for; tiles of a warp's
// ring (K and V have their own slots: with one tile a half of it is on its way
// while the other is worked on); query operands in shared memory or in
// registers.  Measured, blocks / ring / operands: up to 8 rows, head_dim 64,
// ragged batch of 64: 3/1/shared 56.8 us, 3/2/registers 59.9, 4/1/shared 59.3;
// head_dim 128, 131K positions: 2/1/registers 50.1 us, 2/2/registers 51.7,
// 3/1/shared 51.8, 4/1/shared 61.6 (spills); 16 rows of 9000 positions: 2/1
// 41.9 us, 2/2 45.0; 24 rows: 2/1 45.8, 2/2 47.8.  Blocks of 8 warps, half as
// many: 54.6 and 58.0 us there; of 2 warps, twice as many: 42.8 and 49.2.
__host__ __device__ constexpr int blocks_per_sm(int hd, int nt) { return nt == 1 && hd == 64 ? 3 : 2; }
constexpr int kStages = 1;
__host__ __device__ constexpr bool query_smem(int hd, int nt) { return nt > 1 || hd == 64; }
// A stage: K rows, V rows, a K and a V scale for each 16 positions.
__host__ __device__ constexpr int stage_bytes(int hd) { return 2 * tile_len(hd) * hd + 32; }
__host__ __device__ constexpr int ring_bytes(int hd) { return kWarps * kStages * stage_bytes(hd); }
// The warps' O at a unit's end, in two halves where a whole one is too large.
__host__ __device__ constexpr int halves(int hd, int nt) { return hd * nt > 256 ? 2 : 1; }
__host__ __device__ constexpr int state_bytes(int hd, int nt) { return kWarps * 8 * nt * (hd / halves(hd, nt)) * 4; }
__host__ __device__ constexpr int query_bytes(int hd, int nt) { return query_smem(hd, nt) ? nt * (hd / 16) * 32 * 8 : 0; }
__host__ __device__ constexpr int smem_bytes(int hd, int nt) { return ring_bytes(hd) + state_bytes(hd, nt) + query_bytes(hd, nt); }
// The reference that a row's weights are taken against, exp2(x - m), is set to
// kTop below its scores' maximum and follows it only when that is ahead by more
// than kLag: weights up to 2^kLag are as good in fp16 (whose largest value is
// just below 2^16) and in fp32, and a tile that raises no maximum needs no
// reduction over the warp and no rescaling.  kTop puts the largest weight at
// 2^7 or above, so that fp16 holds weights down to 2^-31 of it, and down to
// 2^-21 with all bits: behind a first token that takes nearly all, as trained
// models have, the rest still counts.  kUnseen: nothing seen yet (finite, so
// that -m stays an ordinary addend).
constexpr float kTop = 7.f, kLag = 15.f, kUnseen = -3.402823466e38f;
// One cut unit's state: O [rows][hd], then m and l [rows].
__host__ __device__ constexpr size_t slot_floats(int hd, int nt) { return (size_t)8 * nt * (hd + 2); }

// A unit that the cut of the line went through: it begins in piece c0 (its
// state in slot 2 c0 + slot) and goes on to piece `last` (slots 2 c).  last =
// 0: not cut.  Kept by unit, or where there are more units than pieces by the
// piece that it begins in.
struct Cut {
  int b, g, row0, c0, last, slot, pad[2];
};
// Workspace: a cut for each piece, then two slots for each.
__host__ __device__ constexpr size_t work_bytes(int hd, int nt, int blocks) {
  return blocks * (sizeof(Cut) + 2 * sizeof(float) * slot_floats(hd, nt));
}

// ------------------------------------------------------------------ the line

struct Row {
  int n, count, groups, tiles;  // visible positions of its last token, tokens, row groups, tiles of a unit
};
template <int HD>
__device__ __forceinline__ Row row_of(const Kv8AttnArgs &a, int b, int rows_per_group) {
  Row r;
  r.count = row_count(a.count, b, a.T);
  const int64_t n = (int64_t)row_pos(a.pos, b) + r.count;
  r.n = (int)(n < 0 ? 0 : n > a.c.T ? a.c.T : n);
  r.groups = (r.count * (a.H / a.c.Hkv) + rows_per_group - 1) / rows_per_group;
  r.tiles = r.groups ? (r.n + tile_len(HD) - 1) / tile_len(HD) : 0;
  return r;
}
__device__ __forceinline__ int row_units(const Kv8AttnArgs &a, const Row &r) { return r.tiles ? a.c.Hkv * r.groups : 0; }

// ------------------------------------------------------------------ operands

__device__ __forceinline__ __half2 bits_h2(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }
__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

// K: 4 codes of a word as two fp16 pairs, exact; int8 in units of 2^-24 and
// biased: byte ^ 0x80 = code + 128 under a zero exponent is the subnormal
// (code + 128) 2^-24, which costs no conversion.  The products' sums begin at
// -128 2^-24 x the query's sum, and the score's factors make up for 2^24.  The
// tensor pipe cuts a sum's terms at the last bit that the largest exponent
// leaves them, and a subnormal's exponent is that of 2^-14: a score is off by
// some 2^-22 of the largest it could be.  K takes bytes 0, 2 and 1, 3 (the
// order of the head elements is free).
// V: an output may be much smaller than its block's largest values, and the
// same cut would show in it (2.5 x 10^-4 of outputs over 75K positions).  So its
// codes are taken without bias and as normal numbers: byte ^ 0x80 under the
// exponent of 1024 is 1152 + code, less 1152 by one subtraction a pair (below
// 2 x 10^-6; 24 rows 52.1 -> 50.6 us, since the products that summed the
// weights for the bias are gone, 1K positions 5.8 -> 5.9).
//
// The running O is kept in units of 2^40: a sum of 2^24 weights of up to 2^15
// times values at the end of bf16's range stays finite, and at V scales of
// 2^-100, the smallest, fp32's subnormals still hold 16 bits of a block's
// largest.
constexpr float kOutUnit = 0x1p40f;
// No factor of a score passes fp32's range before the score does.  Query rows
// stand at 2^15 (int8: the top of fp16's range) or 2^4 instead of 2^0, which
// keeps the row's factor, with int8 2^12 of K's 2^24 in it, finite for every
// |scale q| below 2^130; the other 2^12 meets the product of the block's scale
// and the row's factor.
template <int FMT>
constexpr int kQueryExp = FMT == RV_KV8_INT8 ? 15 : 4;
template <int FMT>
constexpr int kRowExp = FMT == RV_KV8_INT8 ? 12 : 0;
template <int FMT>
__device__ __forceinline__ float score_factor(float key_scale, float row) {
  const float f = __fmul_rn(key_scale, row);
  return FMT == RV_KV8_INT8 ? f * 0x1p12f : f;
}
constexpr float kBias = 128.f * 0x1p-24f;
// (x & mask) ^ flip in one operation: both constants in registers.
struct I8Const {
  uint32_t mask, flip;
};
__device__ __forceinline__ I8Const i8_const() {
  I8Const c;
  asm volatile("mov.b32 %0, 0x00ff00ff; mov.b32 %1, 0x00800080;" : "=r"(c.mask), "=r"(c.flip));
  return c;
}
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t mask, uint32_t flip) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(x), "r"(mask), "r"(flip));
  return y;
}
template <int FMT>
__device__ __forceinline__ void unpack_k(uint32_t w, uint32_t &lo, uint32_t &hi, I8Const c) {
  if (FMT == RV_KV8_INT8) {
    lo = and_xor(w, c.mask, c.flip);
    hi = and_xor(w >> 8, c.mask, c.flip);
  } else {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(lo), "=r"(hi) : "r"(w));
  }
}
// Byte i of two words (two positions' codes of one element) for i = 0..3.
template <int FMT>
__device__ __forceinline__ void unpack_v(uint32_t w0, uint32_t w1, uint32_t (&x)[4], I8Const c) {
  if (FMT == RV_KV8_INT8) {
    constexpr uint32_t k1152 = 0x64806480u;  // the pair of fp16 1152; also the exponent of 1024 and the flip of a byte's sign
    x[0] = prmt(w0, w1, 0x5410);
    x[1] = prmt(w0, w1, 0x6521);
    x[2] = prmt(w0, w1, 0x7632);
    x[3] = prmt(w0, w1, 0x4703);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = h2_bits(__hsub2(bits_h2(and_xor(x[i], c.mask, k1152)), bits_h2(k1152)));
  } else {
    const uint32_t a = prmt(w0, w1, 0x5140), b = prmt(w0, w1, 0x7362);
    unpack_k<FMT>(a, x[0], x[1], c);
    unpack_k<FMT>(b, x[2], x[3], c);
  }
}

__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same into d from a starting value per column pair.
__device__ __forceinline__ void mma16_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  return h2_bits(__floats2half2_rn(lo, hi));
}

__device__ __forceinline__ void cp16z(unsigned dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4z(unsigned dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Byte offset of 16-byte chunk c of position p's row inside a tile, swizzled
// so that the 8 lanes of a 16-byte access phase meet different banks: K is
// read by (8 positions x 4 consecutive chunks), V by (positions 2 apart x 2
// chunks at head_dim 128, x 4 half chunks at 64).
template <int HD>
__device__ __forceinline__ int k_off(int p, int c) {
  if (HD == 128) return p * 128 + ((c ^ ((p & 1) << 2)) << 4);
  return p * 64 + (c << 4);
}
template <int HD>
__device__ __forceinline__ int v_off(int p, int c) {
  if (HD == 128) return p * 128 + ((c ^ (((p >> 1) & 3) << 1)) << 4);
  return (p >> 1) * 128 + (((((p & 1) << 2) | c) ^ (((p >> 1) & 3) << 1)) << 4);
}

// ------------------------------------------------------------------ main kernel

__device__ __forceinline__ unsigned cluster_blocks() {
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
// Shared memory of the cluster's block k at the address that `at` is here.
__device__ __forceinline__ unsigned map_cluster(unsigned at, int k) {
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(k));
  return r;
}
__device__ __forceinline__ float ld_cluster(unsigned at, int k) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(map_cluster(at, k)) : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(unsigned at, int k) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(map_cluster(at, k))
               : "memory");
  return x;
}

// 4 elements of an output row from its joined state (x = weighted sum in units
// of kOutUnit, mm = reference in base 2, ll = sum).
__device__ __forceinline__ void write_out(const Kv8AttnArgs &a, int b, int t, int h, int d, float4 x, float mm, float ll) {
  if (a.raw) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out.p) + b * a.out.sb + t * a.out.st + h * a.out.sh + d) = x;
    if (d == 0) a.raw[((int64_t)b * a.T + t) * a.H + h] = make_float2(mm, ll);
    return;
  }
  const float f = ll == 0.f ? 0.f : kOutUnit / ll;  // nothing seen: zeros
  x.x *= f; x.y *= f; x.z *= f; x.w *= f;
  const int act = a.c.act;
  const int64_t o = b * a.out.sb + t * a.out.st + h * a.out.sh + d;
  if (a.out_dtype == RV_F32) {
    if (a.round_out) x = make_float4(round_act(x.x, act), round_act(x.y, act), round_act(x.z, act), round_act(x.w, act));
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out.p) + o) = x;
  } else {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out.p) + o) =
        make_uint2(pack_act2(x.x, x.y, act), pack_act2(x.z, x.w, act));
  }
  if (a.lse && d == 0) a.lse[((int64_t)b * a.T + t) * a.H + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// Query rows of a unit are T x (H / Hkv), token-major: row i is token i / grp,
// head g grp + i % grp; a row group is 8 NT of them.
// A segment of the line: tiles [t0, t1) of one unit.
struct Segment {
  int b, g, row0, t0, t1;
  int n, count, tiles;  // the row's visible positions and tokens, the unit's tiles
  int64_t last;         // where the unit ends in the line (its last tile)
  int64_t rows;         // KV row: b Hkv + g
};

// GS: 16-position steps of a tile that share a scale (the smaller of block and
// tile).  LO: the weights enter as two fp16 terms (high and low part).
// CL: short contexts; a cluster takes one unit, its blocks cut the unit's
// tiles evenly and join through distributed shared memory: no workspace and
// no second kernel.
template <int FMT, int HD, int NT, int GS, bool LO, bool CL>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(HD, NT)) k_attn8(const __grid_constant__ Kv8AttnArgs a, int by_unit) {
  constexpr int KS = HD / 16, MD = HD / 16, ROWS = 8 * NT, ST = kStages, SB = stage_bytes(HD);
  constexpr int TL = tile_len(HD), TM = TL / 16, NG = TM / GS;
  constexpr bool QS = query_smem(HD, NT);
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS], s_rs[ROWS], s_qb[ROWS];
  __shared__ int s_see[ROWS];
  __shared__ int64_t s_tiles[kWarps], s_units[kWarps], s_off;
  __shared__ int s_row;
  pdl_wait();  // (first of all: with `raw` the kernel behind rests on it, see ops.cuh)
  if (CL && a.raw) pdl_trigger();  // what comes next does not need this one's results before its end
  const Kv8 &c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int grp = a.H / c.Hkv, groups = (a.T * grp + ROWS - 1) / ROWS;
  Cut *cuts = static_cast<Cut *>(a.work);
  float *slots = reinterpret_cast<float *>(cuts + gridDim.x) + (size_t)2 * blockIdx.x * slot_floats(HD, NT);
  if (!CL && tid == 0 && !by_unit) cuts[blockIdx.x].last = 0;
  // rows that see nothing have no tiles: zeros
  for (int i = blockIdx.x; i < a.B; i += gridDim.x) {
    const Row r = row_of<HD>(a, i, ROWS);
    if (!CL && by_unit)
      for (int u = tid; u < c.Hkv * groups; u += kWarps * 32)
        if (!r.tiles || u % groups >= r.groups) cuts[(int64_t)i * c.Hkv * groups + u].last = 0;
    if (r.n) continue;
    for (int u = tid; u < r.count * a.H * (HD / 4); u += kWarps * 32) {
      const int d = (u % (HD / 4)) * 4, h = u / (HD / 4) % a.H, tt = u / (HD / 4) / a.H;
      write_out(a, i, tt, h, d, make_float4(0, 0, 0, 0), 0.f, 0.f);
    }
  }

  // ---- this block's piece [begin, end) of the line, and where it begins:
  // `off` into row `b`.  A unit takes `extra` + its tiles of the line.
  int64_t total = 0, piece = 1, begin = 0, end = 0, off = 0;
  int b = 0, extra = 0;
  const int ranks = CL ? (int)cluster_blocks() : 1, rank = CL ? (int)cluster_rank() : 0;
  if (!CL) {
    // each thread sums a run of rows; the one whose run holds `begin` finds the row
    const int per = (a.B + kWarps * 32 - 1) / (kWarps * 32), r0 = min(a.B, tid * per), r1 = min(a.B, r0 + per);
    int64_t tiles = 0, units = 0, all_tiles = 0, all_units = 0, tiles_before = 0, units_before = 0;
    if (a.B == 1) {
      const Row r = row_of<HD>(a, 0, ROWS);
      all_units = row_units(a, r);
      all_tiles = all_units * r.tiles;
    } else {
      for (int i = r0; i < r1; ++i) {
        const Row r = row_of<HD>(a, i, ROWS);
        units += row_units(a, r);
        tiles += (int64_t)row_units(a, r) * r.tiles;
      }
      int64_t it = tiles, iu = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, it, o), y = __shfl_up_sync(0xffffffffu, iu, o);
        if (lane >= o) { it += x; iu += y; }
      }
      if (lane == 31) { s_tiles[warp] = it; s_units[warp] = iu; }
      __syncthreads();
      tiles_before = it - tiles;
      units_before = iu - units;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) { tiles_before += s_tiles[w]; units_before += s_units[w]; }
        all_tiles += s_tiles[w];
        all_units += s_units[w];
      }
    }
    extra = all_tiles >= (int64_t)gridDim.x * 2 * kWarps ? unit_tiles(NT) : 0;
    total = all_tiles + extra * all_units;
    piece = (total + gridDim.x - 1) / gridDim.x;
    if (piece < kMinTiles && all_units) piece = max(piece, min((int64_t)kMinTiles, (all_tiles + all_units - 1) / all_units));
    begin = piece * blockIdx.x;
    if (begin >= total) return;
    end = min(total, begin + piece);
    if (a.B == 1) {
      off = begin;
    } else {
      int64_t at = tiles_before + extra * units_before;
      if (begin >= at && begin < at + tiles + extra * units)
        for (int i = r0; i < r1; ++i) {
          const Row r = row_of<HD>(a, i, ROWS);
          const int64_t n = (int64_t)row_units(a, r) * (r.tiles + extra);
          if (begin < at + n) {
            s_row = i;
            s_off = begin - at;
            break;
          }
          at += n;
        }
      __syncthreads();
      b = s_row;
      off = s_off;
    }
  }

  // ---- segments, one ahead of the one that is worked on
  int64_t left = end - begin;
  if (CL) b = blockIdx.x / ranks / (c.Hkv * groups);
  Row r = row_of<HD>(a, b, ROWS);
  auto next_segment = [&](Segment &s) {
    if (CL) {  // one segment: this block's share of the cluster's unit (it may be empty)
      const int unit = blockIdx.x / ranks - b * c.Hkv * groups, per = (r.tiles + ranks - 1) / ranks;
      s.b = b;
      s.g = unit / groups;
      s.row0 = (unit - s.g * groups) * ROWS;
      s.t0 = min(r.tiles, rank * per);
      s.t1 = min(r.tiles, s.t0 + per);
      s.n = r.n;
      s.count = r.count;
      s.tiles = r.tiles;
      s.rows = (int64_t)b * c.Hkv + s.g;
      left = 0;
      return r.tiles > 0 && unit - s.g * groups < r.groups;
    }
    for (;;) {
      if (left <= 0) return false;
      const int64_t in_row = (int64_t)row_units(a, r) * (r.tiles + extra);
      if (off >= in_row) {  // rows without tiles, or the row is done
        off -= in_row;
        if (++b >= a.B) return false;  // only if d_pos changed under the kernel
        r = row_of<HD>(a, b, ROWS);
        continue;
      }
      const unsigned len = r.tiles + extra;
      const int unit = off >> 32 ? (int)(off / len) : (int)((unsigned)off / len), rem = (int)(off - (int64_t)unit * len);
      s.last = end - left - rem + len - 1;
      const int take = (int)min((int64_t)(r.tiles + extra - rem), left);
      s.t0 = max(0, rem - extra);
      s.t1 = max(0, rem + take - extra);
      off += take;
      left -= take;
      if (s.t1 <= s.t0) continue;
      s.b = b;
      s.g = unit / r.groups;
      s.row0 = (unit - s.g * r.groups) * ROWS;
      s.n = r.n;
      s.count = r.count;
      s.tiles = r.tiles;
      s.rows = (int64_t)b * c.Hkv + s.g;
      return true;
    }
  };

  const I8Const ic = i8_const();
  const int lb = __ffs(c.block) - 1;
  constexpr int CH = HD / 16, NC = TL * CH / 32;  // 16-byte chunks of a row, copies of a lane and tile
  const unsigned ring = (unsigned)__cvta_generic_to_shared(sm) + warp * ST * SB;
  const unsigned char *ringp = sm + warp * ST * SB;
  float *so = reinterpret_cast<float *>(sm + ring_bytes(HD));
  uint2 *sq = reinterpret_cast<uint2 *>(sm + ring_bytes(HD) + state_bytes(HD, NT));
  const unsigned ko = k_off<HD>(lane / CH, lane % CH), vo = v_off<HD>(lane / CH, lane % CH);

  // A warp's tiles run through the segments in order: index i of the current
  // one, then the next one's.  Every step commits a K and a V group, empty if
  // there is nothing to copy, so that waiting for all but the last 2 ST - 1
  // groups always covers the tile at hand.
  Segment cur, nxt;
  if (!next_segment(cur)) return;
  bool more = !CL && next_segment(nxt);
  auto tiles_of = [&](const Segment &s) { return (s.t1 - s.t0 - warp + kWarps - 1) / kWarps; };  // >= 0: -3 / 4 = 0
  int cnt = tiles_of(cur), ncnt = more ? tiles_of(nxt) : 0;
  int filled[2] = {0, 0}, fill[2] = {0, 0}, head = 0;  // [K, V]: tiles asked for from the current segment on, and the slot of the next
  // Asks for the next tile's K (which = 0) or V rows and scales.
  auto step = [&](int which) {
    const int i = filled[which];
    if (i < cnt + ncnt) {
      const bool here = i < cnt;
      const int p0 = ((here ? cur.t0 + i * kWarps : nxt.t0 + (i - cnt) * kWarps) + warp) * TL, n = here ? cur.n : nxt.n;
      const int64_t rows = here ? cur.rows : nxt.rows;
      const unsigned slot = ring + fill[which] * SB, st = slot + which * TL * HD;
      const uint8_t *src = c.codes[which] + (rows * c.N + p0) * HD + lane * 16;
      if (p0 + TL <= n) {
        // copy i is 512 bytes on; at head_dim 128 the swizzle of V's rows alternates
        const unsigned d0 = st + (which ? vo : ko), d1 = st + (which ? (HD == 128 ? vo ^ 64 : vo) : ko);
#pragma unroll
        for (int k = 0; k < NC; ++k) cp16s((k & 1 ? d1 : d0) + k * 512, src + k * 512);
      } else {  // the unit's last tile: zeros behind the last position
#pragma unroll 1
        for (int k = 0; k < NC; ++k) {
          const int q = k * (32 / CH) + lane / CH, bytes = p0 + q < n ? 16 : 0;
          cp16z(st + (which ? v_off<HD>(q, lane % CH) : k_off<HD>(q, lane % CH)), bytes ? src + k * 512 : c.codes[0], bytes);
        }
      }
      if (lane < TM) {
        const int q = p0 + lane * 16, bytes = q < n ? 4 : 0;
        cp4z(slot + 2 * TL * HD + (which * TM + lane) * 4, c.scale[which] + rows * (c.N >> lb) + (bytes ? q >> lb : 0), bytes);
      }
      ++filled[which];
      fill[which] = fill[which] + 1 == ST ? 0 : fill[which] + 1;
    }
    cp_commit();
  };
  for (int i = 0; i < ST; ++i) { step(0); step(1); }

  for (bool first = true;; first = false) {
    // ---- query operands: column gq of n-tile nt is query row row0 + 8 nt + gq
    uint32_t qf[QS ? 1 : NT][QS ? 1 : KS][2];
    // of rows 2 tq, 2 tq + 1: score factor (not negative), where their scores'
    // sums begin, positions they see; with QS in shared memory too
    float rs_[QS ? 1 : NT][2], qb_[QS ? 1 : NT][2];
    int see_[QS ? 1 : NT][2];
    auto rs = [&](int nt) { return QS ? *reinterpret_cast<const float2 *>(s_rs + 8 * nt + 2 * tq) : make_float2(rs_[QS ? 0 : nt][0], rs_[QS ? 0 : nt][1]); };
    auto qb = [&](int nt) { return QS ? *reinterpret_cast<const float2 *>(s_qb + 8 * nt + 2 * tq) : make_float2(qb_[QS ? 0 : nt][0], qb_[QS ? 0 : nt][1]); };
    auto see = [&](int nt) { return QS ? *reinterpret_cast<const int2 *>(s_see + 8 * nt + 2 * tq) : make_int2(see_[QS ? 0 : nt][0], see_[QS ? 0 : nt][1]); };
    auto sees = [&](int row) {  // rows that do not exist see zeros
      const int64_t n = (int64_t)row_pos(a.pos, cur.b) + row / grp + 1;
      return row < cur.count * grp ? (int)(n < 0 ? 0 : n > cur.n ? cur.n : n) : cur.n;
    };
    const int nrows = cur.count * grp;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float up, qsum = 0.f;
      if (!QS || nt % kWarps == warp) {
        const int row = cur.row0 + 8 * nt + gq;
        float x[HD / 4];
        float mx = 0.f;
        const bool ok = row < nrows;
        const int t = row / grp, h = cur.g * grp + row - t * grp;
        const int64_t o = cur.b * a.q.sb + t * a.q.st + h * a.q.sh;
#pragma unroll
        for (int j = 0; j < HD / 64; ++j) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int64_t od = o + 64 * j + 16 * tq + 8 * v;
            if (a.q_f32) {
              float4 y0 = make_float4(0, 0, 0, 0), y1 = y0;
              if (ok) {
                y0 = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q.p) + od);
                y1 = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q.p) + od + 4);
              }
              const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
              for (int i = 0; i < 8; ++i) x[16 * j + 8 * v + i] = round_act(y[i], c.act);
            } else {
              uint4 y = make_uint4(0, 0, 0, 0);
              if (ok) y = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q.p) + od);
              const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int i = 0; i < 8; ++i) x[16 * j + 8 * v + i] = act_to_f((uint16_t)(w[i >> 1] >> (16 * (i & 1))), c.act);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < HD / 4; ++i) mx = fmaxf(mx, fabsf(x[i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int e = min((int)(__float_as_uint(mx) >> 23), 254) - 127;
        constexpr int QE = kQueryExp<FMT>, RE = kRowExp<FMT>;  // both exponents below stay those of normal numbers
        e = max(e, QE - 126);
        const float down = copysignf(__uint_as_float((uint32_t)(127 + QE - e) << 23), a.scale);  // the scale's sign goes to the query
        up = __uint_as_float((uint32_t)(127 + e - QE + RE) << 23) * fabsf(a.scale) * kLog2e;
        if (mx == INFINITY) up = __int_as_float(0x7fc00000);  // also where all its scores would be -infinity
#pragma unroll
        for (int j = 0; j < HD / 64; ++j)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const float *y = x + 16 * j + 4 * s;
            constexpr int E = FMT == RV_KV8_INT8 ? 2 : 1;  // the second element of unpack_k's first pair
            const uint32_t q0 = pack_h2(y[0] * down, y[E] * down), q1 = pack_h2(y[3 - E] * down, y[3] * down);
            if (QS) sq[(nt * KS + 4 * j + s) * 32 + lane] = make_uint2(q0, q1);
            else { qf[QS ? 0 : nt][QS ? 0 : 4 * j + s][0] = q0; qf[QS ? 0 : nt][QS ? 0 : 4 * j + s][1] = q1; }
            if (FMT == RV_KV8_INT8) {
              const float2 u = __half22float2(bits_h2(q0)), v = __half22float2(bits_h2(q1));
              qsum += (u.x + u.y) + (v.x + v.y);
            }
          }
        if (FMT == RV_KV8_INT8) {
          qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
          qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
        }
        if (QS && tq == 0) {
          s_rs[8 * nt + gq] = up;
          s_qb[8 * nt + gq] = -kBias * qsum;
        }
      }
      if (!QS) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          rs_[QS ? 0 : nt][k] = __shfl_sync(0xffffffffu, up, (2 * tq + k) * 4);
          qb_[QS ? 0 : nt][k] = -kBias * __shfl_sync(0xffffffffu, qsum, (2 * tq + k) * 4);
          see_[QS ? 0 : nt][k] = sees(cur.row0 + 8 * nt + 2 * tq + k);
        }
      }
    }
    if (QS) {
      if (tid < ROWS) s_see[tid] = sees(cur.row0 + tid);
      __syncthreads();
    }
    int see_all = cur.n;  // positions that every row of the group sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int2 n = see(nt);
      see_all = min(see_all, min(n.x, n.y));
    }
    see_all = __reduce_min_sync(0xffffffffu, see_all);

    F2 o[MD][NT][2];  // [16-element tile][n-tile][element 2 i, 2 i + 1]: columns 2 tq, 2 tq + 1
    float m[NT][2];
    F2 l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kUnseen;
      l[nt] = f2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < MD; ++i) o[i][nt][0] = o[i][nt][1] = f2(0.f, 0.f);
    }

    for (int ti = 0; ti < cnt; ++ti) {
      const unsigned char *kt = ringp + head * SB, *vt = kt + TL * HD;
      const float *fs = reinterpret_cast<const float *>(kt + 2 * TL * HD);
      const int p0 = (cur.t0 + warp + ti * kWarps) * TL;
      cp_wait<2 * ST - 1>();
      __syncwarp();
      // (products in an order that keeps those into one sum apart: an mma waits
      // for the one before it only if it adds to its result)
      float s[TM][NT][4];
#pragma unroll
      for (int j = 0; j < HD / 64; ++j) {
        uint4 w[TM][2];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) w[i][k] = *reinterpret_cast<const uint4 *>(kt + k_off<HD>(16 * i + gq + 8 * k, 4 * j + tq));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint2 q[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (QS) q[nt] = sq[(nt * KS + 4 * j + k) * 32 + lane];
            else q[nt] = make_uint2(qf[QS ? 0 : nt][QS ? 0 : 4 * j + k][0], qf[QS ? 0 : nt][QS ? 0 : 4 * j + k][1]);
          }
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const uint32_t x0[4] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w}, x1[4] = {w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
            uint32_t f[4];
            unpack_k<FMT>(x0[k], f[0], f[2], ic);
            unpack_k<FMT>(x1[k], f[1], f[3], ic);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (j == 0 && k == 0) mma16_from(s[i][nt], f, q[nt].x, q[nt].y, qb(nt).x, qb(nt).y);
              else mma16(s[i][nt], f, q[nt].x, q[nt].y);
            }
          }
        }
      }
      float ks[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) ks[i] = fs[i * GS];
      __syncwarp();  // every lane is done with the tile's K: its slot takes the next copy
      step(0);
      // ---- mask, reference, weights (column 2 tq + k of n-tile nt); factors
      // are not negative, so a block's maximum is its scores' times the factor
      // (the loops of one or no turn keep the masks a branch: as predicated
      // operations they would cost every tile)
      // The scaled score is rounded before the reference is taken off: the
      // reference is such a rounded score itself, and a fused product minus it
      // would leave up to half a step of the score, which from 2^28 on is more
      // than an fp16 weight's range.  __fmul_rn, because a packed product
      // before a packed sum is fused all the same (24 rows 51.5 -> 52.0 us,
      // 1K positions 5.8 -> 5.9; the long cases do not change).
      const int edge = p0 + TL > see_all;
      uint32_t pb[TM][NT][2], pl[TM][NT][2];
      float top[NT][2];
      bool ahead = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll 1
        for (int e = edge; e > 0; --e) {
          const int2 sn = see(nt);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int n = (k ? sn.y : sn.x) - p0 - gq;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
              if (n <= 16 * i) s[i][nt][k] = -INFINITY;
              if (n <= 16 * i + 8) s[i][nt][2 + k] = -INFINITY;
            }
          }
        }
        const float2 rr = rs(nt);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[nt][k] = -INFINITY;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float y = fmaxf(s[g * GS][nt][k], s[g * GS][nt][2 + k]);
#pragma unroll
            for (int i = 1; i < GS; ++i) y = max3(y, s[g * GS + i][nt][k], s[g * GS + i][nt][2 + k]);
            // -infinity x 0 of an unseen block: a NaN, which fmaxf passes over
            top[nt][k] = fmaxf(top[nt][k], __fmul_rn(y, score_factor<FMT>(ks[g], k ? rr.y : rr.x)));
          }
          ahead |= top[nt][k] - m[nt][k] > kLag;  // (the difference, which is exact where it decides)
        }
      }
      if (__any_sync(0xffffffffu, ahead)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float al[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = top[nt][k];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fmaxf(x - kTop, m[nt][k]);
            al[k] = ex2(m[nt][k] - x);
            m[nt][k] = x;
          }
          const F2 al2 = f2(al[0], al[1]);
          l[nt] = f2_mul(l[nt], al2);
#pragma unroll
          for (int i = 0; i < MD; ++i) {
            o[i][nt][0] = f2_mul(o[i][nt][0], al2);
            o[i][nt][1] = f2_mul(o[i][nt][1], al2);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 rr = rs(nt);
        const F2 neg = f2(-m[nt][0], -m[nt][1]);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const float2 ff = make_float2(score_factor<FMT>(ks[i / GS], rr.x), score_factor<FMT>(ks[i / GS], rr.y));
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 x = f2_split(f2_add(f2(__fmul_rn(s[i][nt][2 * q], ff.x), __fmul_rn(s[i][nt][2 * q + 1], ff.y)), neg));
            s[i][nt][2 * q] = ex2(x.x);
            s[i][nt][2 * q + 1] = ex2(x.y);
          }
        }
#pragma unroll 1
        for (int e = edge; e > 0; --e) {  // what is not seen weighs nothing, whatever its block's scale
          const int2 sn = see(nt);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int n = (k ? sn.y : sn.x) - p0 - gq;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
              if (n <= 16 * i) s[i][nt][k] = 0.f;
              if (n <= 16 * i + 8) s[i][nt][2 + k] = 0.f;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float x = s[i][nt][2 * q], y = s[i][nt][2 * q + 1];
            l[nt] = f2_add(l[nt], f2(x, y));
            const uint32_t hi = pack_h2(x, y);
            pb[i][nt][q] = transpose8(hi);
            if (LO) {
              const float2 h = __half22float2(bits_h2(hi));
              pl[i][nt][q] = transpose8(pack_h2(x - h.x, y - h.y));
            }
          }
      }
      cp_wait<2 * ST - 1>();
      __syncwarp();
      F2 vs[NG][NT];
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float x = fs[TM + i * GS] * (1.f / kOutUnit);
          vs[i][nt] = f2(x, x);
        }
#pragma unroll 1
      for (int e = edge; e > 0; --e) {  // a block that a row sees nothing of adds nothing, whatever its scale
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 x = f2_split(vs[i][nt]);
            const int2 sn = see(nt);
            vs[i][nt] = f2(sn.x <= p0 + 16 * GS * i ? 0.f : x.x, sn.y <= p0 + 16 * GS * i ? 0.f : x.y);
          }
      }
      // ---- O^T += vs (V^T P^T)
      // (words of a V row that a thread takes: all at once, or where registers
      // are short a pair at a time)
      constexpr int VP = HD == 128 && NT >= 2 ? 2 : 1, VW = HD / 32 / VP;
#pragma unroll
      for (int vp = 0; vp < VP; ++vp) {
      uint32_t vw[TM][2][2][VW];  // [k-step][8 positions][position][word]
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int p = 16 * i + 8 * hb + 2 * tq + k;
            const unsigned char *row = HD == 128 ? vt + v_off<HD>(p, gq) + 8 * vp : vt + v_off<HD>(p, gq >> 1) + 8 * (gq & 1);
            if (VW == 4) {
              const uint4 w = *reinterpret_cast<const uint4 *>(row);
              vw[i][hb][k][0] = w.x; vw[i][hb][k][1] = w.y; vw[i][hb][k][VW - 2] = w.z; vw[i][hb][k][VW - 1] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2 *>(row);
              vw[i][hb][k][0] = w.x; vw[i][hb][k][1] = w.y;
            }
          }
      if (vp == VP - 1) {
        __syncwarp();
        step(1);
      }
#pragma unroll
      for (int wq = 0; wq < VW; ++wq) {  // a word of each V row: two 16-element tiles of O^T
        uint32_t f[TM][2][4];            // [k-step][tile][operand]
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            uint32_t x[4];
            unpack_v<FMT>(vw[i][hb][0][wq], vw[i][hb][1][wq], x, ic);
            f[i][0][2 * hb] = x[0];
            f[i][0][2 * hb + 1] = x[1];
            f[i][1][2 * hb] = x[2];
            f[i][1][2 * hb + 1] = x[3];
          }
        constexpr int HH = NT == 1 ? 2 : 1;  // tiles whose sums run side by side
#pragma unroll
        for (int h0 = 0; h0 < 2; h0 += HH)
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            float acc[HH][NT][4];
#pragma unroll
            for (int j = 0; j < GS; ++j) {
              const int st = i * GS + j;
#pragma unroll
              for (int h = 0; h < HH; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if (j == 0) mma16_from(acc[h][nt], f[st][h0 + h], pb[st][nt][0], pb[st][nt][1], 0.f, 0.f);
                  else mma16(acc[h][nt], f[st][h0 + h], pb[st][nt][0], pb[st][nt][1]);
                }
              if (LO) {
#pragma unroll
                for (int h = 0; h < HH; ++h)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma16(acc[h][nt], f[st][h0 + h], pl[st][nt][0], pl[st][nt][1]);
              }
            }
#pragma unroll
            for (int h = 0; h < HH; ++h)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                F2(&oo)[2] = o[2 * (vp * VW + wq) + h0 + h][nt];
                oo[0] = f2_fma(f2(acc[h][nt][0], acc[h][nt][1]), vs[i][nt], oo[0]);
                oo[1] = f2_fma(f2(acc[h][nt][2], acc[h][nt][3]), vs[i][nt], oo[1]);
              }
          }
      }
      }
      head = head + 1 == ST ? 0 : head + 1;
    }

    // ---- join the warps' states
    if (!more) pdl_trigger();  // the next kernel's blocks come up while the last states are joined
    if (CL) cp_wait<0>();
    __syncthreads();  // the states of the segment before have been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 x = f2_split(l[nt]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float y = k ? x.y : x.x;
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (gq == 0) {
          s_m[warp][8 * nt + 2 * tq + k] = m[nt][k] == kUnseen ? -INFINITY : m[nt][k];
          s_l[warp][8 * nt + 2 * tq + k] = y;
        }
      }
    }
    static_assert(slot_floats(HD, NT) * 4 <= ring_bytes(HD), "a cluster block's state fits the rings");
    const bool whole = !CL && cur.t0 == 0 && cur.t1 == cur.tiles;
    float *slotp = slots + (first ? 0 : slot_floats(HD, NT));
    if (!CL && tid == 0 && cur.t0 == 0 && (by_unit || !whole)) {  // the unit begins here; cut: it goes on in the next piece
      const int64_t at = by_unit ? cur.rows * groups + cur.row0 / ROWS : blockIdx.x;
      cuts[at] = Cut{cur.b, cur.g, cur.row0, (int)blockIdx.x, whole ? 0 : (int)(cur.last / piece), first ? 0 : 1, {0, 0}};
    }
    constexpr int HV = halves(HD, NT), HE = HD / HV, HP = HD / 8 / HV;  // elements of a half; of a thread and half
#pragma unroll
    for (int hv = 0; hv < HV; ++hv) {
      if (hv) __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float *d = so + (warp * ROWS + 8 * nt + 2 * tq) * HE + gq * HP;
#pragma unroll
        for (int i = 0; i < MD / HV; i += 2) {
          const float2 w0 = f2_split(o[hv * (MD / HV) + i][nt][0]), w1 = f2_split(o[hv * (MD / HV) + i][nt][1]);
          const float2 w2 = f2_split(o[hv * (MD / HV) + i + 1][nt][0]), w3 = f2_split(o[hv * (MD / HV) + i + 1][nt][1]);
          *reinterpret_cast<float4 *>(d + 2 * i) = make_float4(w0.x, w1.x, w2.x, w3.x);
          *reinterpret_cast<float4 *>(d + HE + 2 * i) = make_float4(w0.y, w1.y, w2.y, w3.y);
        }
      }
      __syncthreads();
      for (int u = tid; u < ROWS * (HE / 4); u += kWarps * 32) {
        const int rr = u / (HE / 4), e = (u - rr * (HE / 4)) * 4, d = e / HP * (HD / 8) + hv * HP + e % HP, row = cur.row0 + rr;
        if (row >= nrows) break;
        float mm = s_m[0][rr];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][rr]);
        const float base = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 x = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(s_m[w][rr] - base);
          const float4 y = *reinterpret_cast<const float4 *>(so + (w * ROWS + rr) * HE + e);
          ll = fmaf(s_l[w][rr], f, ll);
          x.x = fmaf(y.x, f, x.x); x.y = fmaf(y.y, f, x.y); x.z = fmaf(y.z, f, x.z); x.w = fmaf(y.w, f, x.w);
        }
        if (CL) slotp = reinterpret_cast<float *>(sm);  // the rings are idle
        if (!whole) {
          *reinterpret_cast<float4 *>(slotp + rr * HD + d) = x;
          if (d == 0) {
            slotp[ROWS * HD + rr] = mm;
            slotp[ROWS * HD + ROWS + rr] = ll;
          }
        } else {
          const int t = row / grp, h = cur.g * grp + row - t * grp;
          write_out(a, cur.b, t, h, d, x, mm, ll);
        }
      }
    }
    if (CL) {
      // every block of the cluster has left its state in shared memory: each
      // joins a part of the elements
      cluster_sync();
      for (int u = rank * kWarps * 32 + tid; u < ROWS * (HD / 4); u += ranks * kWarps * 32) {
        const int rr = u / (HD / 4), d = (u - rr * (HD / 4)) * 4, row = cur.row0 + rr;
        if (row >= nrows) break;
        const unsigned at = (unsigned)__cvta_generic_to_shared(sm);
        float mm = -INFINITY, ll = 0.f;
        float4 x = make_float4(0, 0, 0, 0);
        for (int k = 0; k < ranks; ++k) mm = fmaxf(mm, ld_cluster(at + 4 * (ROWS * HD + rr), k));
        const float base = mm == -INFINITY ? 0.f : mm;
        for (int k = 0; k < ranks; ++k) {
          const float f = ex2(ld_cluster(at + 4 * (ROWS * HD + rr), k) - base);
          const float4 y = ld_cluster4(at + 4 * (rr * HD + d), k);
          ll = fmaf(ld_cluster(at + 4 * (ROWS * HD + ROWS + rr), k), f, ll);
          x.x = fmaf(y.x, f, x.x); x.y = fmaf(y.y, f, x.y); x.z = fmaf(y.z, f, x.z); x.w = fmaf(y.w, f, x.w);
        }
        const int t = row / grp, h = cur.g * grp + row - t * grp;
        write_out(a, cur.b, t, h, d, x, mm, ll);
      }
      cluster_sync();  // no block leaves while another reads its state
      break;
    }
    if (!more) break;
    // ---- on to the next segment, part of whose tiles are on their way
    filled[0] -= cnt;
    filled[1] -= cnt;
    cur = nxt;
    cnt = ncnt;
    more = next_segment(nxt);
    ncnt = more ? tiles_of(nxt) : 0;
    for (int i = filled[0]; i < ST; ++i) { step(0); step(1); }
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------ join

// Joins the states of the units that the cut of the line went through: block
// x takes cut x of `pieces`.  WPR warps take one query row, each a run of its
// states with up to kJoin of them on their way at once: what this kernel
// takes is the latency of its dependent loads.
constexpr int kJoin = 6;
template <int HD, int NT, int WPR>
__global__ void __launch_bounds__(256) k_attn8_join(const __grid_constant__ Kv8AttnArgs a, int pieces) {
  constexpr int ROWS = 8 * NT, PER = HD / 32, RPB = 8 / WPR;
  __shared__ float s_x[8][HD], s_m[8], s_l[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = a.H / a.c.Hkv;
  pdl_wait();  // (as in k_attn8)
  pdl_trigger();
  const Cut *cuts = static_cast<const Cut *>(a.work);
  const float *work = reinterpret_cast<const float *>(cuts + pieces);
  union {
    int4 v[2];
    Cut cut;
  } u;
  u.v[0] = __ldcg(reinterpret_cast<const int4 *>(cuts + blockIdx.x));
  u.v[1] = __ldcg(reinterpret_cast<const int4 *>(cuts + blockIdx.x) + 1);
  const Cut cut = u.cut;
  const int b = cut.b, c0 = cut.c0, c1 = cut.last;
  if (c1 == 0) return;
  const int rr = blockIdx.y * RPB + warp / WPR, row = cut.row0 + rr, sub = warp % WPR;
  const bool live = rr < ROWS && row < row_count(a.count, b, a.T) * grp;
  const int t = row / grp, h = cut.g * grp + row - t * grp;
  float mm = -INFINITY, ll = 0.f, x[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = 0.f;
  if (live) {
    for (int c = c0 + sub; c <= c1; c += WPR * kJoin) {
      float sm[kJoin], sl[kJoin], y[kJoin][PER], top = mm;
#pragma unroll
      for (int j = 0; j < kJoin; ++j) {
        const int cc = c + j * WPR;
        sm[j] = -INFINITY;
        sl[j] = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) y[j][i] = 0.f;
        if (cc <= c1) {
          const float *s = work + (size_t)(2 * cc + (cc == c0 ? cut.slot : 0)) * slot_floats(HD, NT);
          sm[j] = __ldcg(s + ROWS * HD + rr);
          sl[j] = __ldcg(s + ROWS * HD + ROWS + rr);
          if (PER == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(s + rr * HD) + lane);
            y[j][0] = v.x; y[j][1] = v.y; y[j][PER - 2] = v.z; y[j][PER - 1] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2 *>(s + rr * HD) + lane);
            y[j][0] = v.x; y[j][1] = v.y;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kJoin; ++j) top = fmaxf(top, sm[j]);
      const float base = top == -INFINITY ? 0.f : top, old = ex2(mm - base);
      ll *= old;
#pragma unroll
      for (int i = 0; i < PER; ++i) x[i] *= old;
#pragma unroll
      for (int j = 0; j < kJoin; ++j) {
        const float f = ex2(sm[j] - base);
        ll = fmaf(sl[j], f, ll);
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = fmaf(y[j][i], f, x[i]);
      }
      mm = top;
    }
  }
  // through shared memory: the warps of a row, and 4 elements to a thread
#pragma unroll
  for (int i = 0; i < PER; ++i) s_x[warp][lane * PER + i] = x[i];
  if (lane == 0) {
    s_m[warp] = mm;
    s_l[warp] = ll;
  }
  if (WPR > 1) __syncthreads();
  else __syncwarp();
  if (!live || sub || lane >= HD / 4) return;
#pragma unroll
  for (int w = 1; w < WPR; ++w) mm = fmaxf(mm, s_m[warp + w]);
  const float base = mm == -INFINITY ? 0.f : mm;
  float4 v = make_float4(0, 0, 0, 0);
  ll = 0.f;
#pragma unroll
  for (int w = 0; w < WPR; ++w) {
    const float4 y = *reinterpret_cast<const float4 *>(&s_x[warp + w][4 * lane]);
    const float f = ex2(s_m[warp + w] - base);
    v.x = fmaf(y.x, f, v.x); v.y = fmaf(y.y, f, v.y); v.z = fmaf(y.z, f, v.z); v.w = fmaf(y.w, f, v.w);
    ll = fmaf(s_l[warp + w], f, ll);
  }
  write_out(a, b, t, h, 4 * lane, v, mm, ll);
}

template <int FMT, int HD, int NT, int GS, bool LO>
cudaError_t launch_t(const Kv8AttnArgs &a, int n_sm, cudaStream_t s, int pdl) {
  const int rows = a.T * (a.H / a.c.Hkv);
  const int64_t units = (int64_t)a.B * a.c.Hkv * ((rows + 8 * NT - 1) / (8 * NT));
  if (a.cluster) {
    auto fn = k_attn8<FMT, HD, NT, GS, LO, true>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(HD, NT));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * a.cluster));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem_bytes(HD, NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, fn, a, 0);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  auto fn = k_attn8<FMT, HD, NT, GS, LO, false>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(HD, NT));
  if (e != cudaSuccess) return e;
  const int pieces = blocks_per_sm(HD, NT) * n_sm;
  const int by_unit = units <= pieces, cuts = by_unit ? (int)units : pieces;
  e = launch_k(fn, dim3(pieces), dim3(kWarps * 32), smem_bytes(HD, NT), s, pdl, a, by_unit);
  if (e != cudaSuccess) return e;
  // few units are cut into many pieces: eight warps join a row; else one
  const int per_unit = rows < 8 * NT ? rows : 8 * NT;
  if (units * 4 <= pieces) return launch_k(k_attn8_join<HD, NT, 8>, dim3(cuts, per_unit), dim3(256), 0, s, 1, a, pieces);
  return launch_k(k_attn8_join<HD, NT, 1>, dim3(cuts, (per_unit + 7) / 8), dim3(256), 0, s, 1, a, pieces);
}

template <int FMT, int HD, int NT, bool LO>
cudaError_t launch_lo(const Kv8AttnArgs &a, int n_sm, cudaStream_t s, int pdl) {
  if (a.c.block == 16) return launch_t<FMT, HD, NT, 1, LO>(a, n_sm, s, pdl);
  if (a.c.block == 32 || HD == 128) return launch_t<FMT, HD, NT, 2, LO>(a, n_sm, s, pdl);
  return launch_t<FMT, HD, NT, HD == 128 ? 2 : 4, LO>(a, n_sm, s, pdl);
}

template <int FMT, int HD, int NT>
cudaError_t launch_nt(const Kv8AttnArgs &a, int n_sm, cudaStream_t s, int pdl) {
  // fp16 outputs have 11 bits and fp32 ones 24: weights rounded to 11 would show in them
  return a.c.act == RV_F16 || (a.out_dtype == RV_F32 && !a.round_out) ? launch_lo<FMT, HD, NT, true>(a, n_sm, s, pdl) : launch_lo<FMT, HD, NT, false>(a, n_sm, s, pdl);
}

template <int FMT>
cudaError_t launch_fmt(const Kv8AttnArgs &a, int nt, int n_sm, cudaStream_t s, int pdl) {
  if (a.c.hd == 64) {
    if (nt == 1) return launch_nt<FMT, 64, 1>(a, n_sm, s, pdl);
    return nt == 2 ? launch_nt<FMT, 64, 2>(a, n_sm, s, pdl) : launch_nt<FMT, 64, 3>(a, n_sm, s, pdl);
  }
  if (nt == 1) return launch_nt<FMT, 128, 1>(a, n_sm, s, pdl);
  return nt == 2 ? launch_nt<FMT, 128, 2>(a, n_sm, s, pdl) : launch_nt<FMT, 128, 3>(a, n_sm, s, pdl);
}

cudaError_t launch_int8(const Kv8AttnArgs &a, int nt, int n_sm, cudaStream_t s, int pdl);
cudaError_t launch_e4m3(const Kv8AttnArgs &a, int nt, int n_sm, cudaStream_t s, int pdl);

}  // namespace kv8a
}  // namespace rv
