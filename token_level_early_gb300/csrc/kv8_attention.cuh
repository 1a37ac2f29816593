// Attention of a few new tokens per row over the 8-bit K/V cache.
//
// out = sum_p w_p v_p / sum_p w_p, w_p = exp(scale q.k_p - m), in one pass over
// the visible positions with a running maximum m, sum and weighted sum (all
// fp32, exponents in base 2).  k_p = s_block x code, so a score is
// (s_block scale) (q.code): codes go to the tensor pipe as exact fp16 values
// and the block's scale multiplies the fp32 scores; the V scale multiplies
// the block's fp32 partial product.  A query row is divided by a power of two
// (its largest magnitude's), so bf16 rows fit fp16's range; the power returns
// with the scale.
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
// Each warp streams its own tiles of 32 positions (8 KB at head_dim 128)
// through a private ring in shared memory (cp.async, no barriers inside a
// segment).  The (row, KV head, row group) units with their tiles form one
// line that is cut evenly over the resident blocks, whatever the rows'
// lengths: a block computes its own piece of the line from d_pos, finishes
// the units that lie in it and leaves the state (m, l, O) of at most two cut
// ones, which a second kernel, chained by programmatic dependent launch,
// joins.  fp16 caches split each weight into a high and a low fp16 term.
#pragma once

#include <cuda_fp8.h>

#include "ops.cuh"

namespace rv {
namespace kv8a {

constexpr int kWarps = 4;  // warps of a block
// Positions of a tile: 4 KB of K and 4 KB of V.
__host__ __device__ constexpr int tile_len(int hd) { return hd == 128 ? 32 : 64; }
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Smallest piece of the line a block takes: one tile for each of its warps.
constexpr int kMinTiles = kWarps;

// Blocks per SM: as many as the registers leave room for.
__host__ __device__ constexpr int blocks_per_sm(int hd, int nt) { return nt == 1 && hd == 64 ? 3 : 2; }
// Tiles of a warp's ring: what the blocks of an SM fit into 227 KB.
__host__ __device__ constexpr int stages(int nt) { return nt == 1 ? 2 : 3; }
// A stage: K rows, V rows, a K and a V scale for each 16 positions.
__host__ __device__ constexpr int stage_bytes(int hd) { return 2 * tile_len(hd) * hd + 32; }
__host__ __device__ constexpr int smem_bytes(int hd, int nt) { return kWarps * stages(nt) * stage_bytes(hd); }
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
__device__ __forceinline__ int64_t line_tiles(const Kv8AttnArgs &a, const Row &r) { return (int64_t)a.c.Hkv * r.groups * r.tiles; }
__device__ __forceinline__ int64_t piece_of(int64_t total, int blocks) {
  const int64_t p = (total + blocks - 1) / blocks;
  return p < kMinTiles ? kMinTiles : p;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------ operands

__device__ __forceinline__ __half2 bits_h2(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }
__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

// 4 codes of a word as two fp16 pairs, exact; int8 in units of 2^-24 and
// biased: byte ^ 0x80 = code + 128 under a zero exponent is the subnormal
// (code + 128) 2^-24, which costs no conversion.  The products' sums begin at
// -128 2^-24 x the other operand's sum, and 2^24 joins the scale.  K takes
// bytes 0, 2 and 1, 3 (the order of the head elements is free).
template <int FMT>
__device__ __forceinline__ float code_unit() { return FMT == RV_KV8_INT8 ? 0x1p24f : 1.f; }
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
__device__ __forceinline__ uint32_t and_xor(uint32_t x, I8Const c) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(x), "r"(c.mask), "r"(c.flip));
  return y;
}
template <int FMT>
__device__ __forceinline__ void unpack_k(uint32_t w, uint32_t &lo, uint32_t &hi, I8Const c) {
  if (FMT == RV_KV8_INT8) {
    lo = and_xor(w, c);
    hi = and_xor(w >> 8, c);
  } else {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(lo), "=r"(hi) : "r"(w));
  }
}
// Byte i of two words (two positions' codes of one element) for i = 0..3.
template <int FMT>
__device__ __forceinline__ void unpack_v(uint32_t w0, uint32_t w1, uint32_t (&x)[4], I8Const c) {
  if (FMT == RV_KV8_INT8) {
    x[0] = and_xor(prmt(w0, w1, 0x5410), c);
    x[1] = and_xor(prmt(w0, w1, 0x6521), c);
    x[2] = and_xor(prmt(w0, w1, 0x7632), c);
    x[3] = and_xor(prmt(w0, w1, 0x4703), c);
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

// 4 elements of an output row from its joined state (x = weighted sum, mm =
// maximum in base 2, ll = sum).
__device__ __forceinline__ void write_out(const Kv8AttnArgs &a, int b, int t, int h, int d, float4 x, float mm, float ll) {
  const float f = ll == 0.f ? 0.f : 1.f / ll;  // nothing seen: zeros
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
// GS: 16-position steps of a tile that share a scale (the smaller of block and
// tile).  LO: the weights enter as two fp16 terms (high and low part).
template <int FMT, int HD, int NT, int GS, bool LO>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(HD, NT)) k_attn8(const __grid_constant__ Kv8AttnArgs a, int by_unit) {
  constexpr int KS = HD / 16, MD = HD / 16, ROWS = 8 * NT, ST = stages(NT), SB = stage_bytes(HD);
  constexpr int TL = tile_len(HD), TM = TL / 16, NG = TM / GS;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ int64_t s_scan[kWarps + 1];
  __shared__ int s_row;
  __shared__ int64_t s_at;
  pdl_wait();
  pdl_trigger();  // after the wait: the joining kernel may read d_pos at once
  const Kv8 &c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int grp = a.H / c.Hkv;
  Cut *cuts = static_cast<Cut *>(a.work);
  float *slots = reinterpret_cast<float *>(cuts + gridDim.x) + (size_t)2 * blockIdx.x * slot_floats(HD, NT);
  const int groups = (a.T * grp + ROWS - 1) / ROWS;
  if (tid == 0 && !by_unit) cuts[blockIdx.x].last = 0;
  // rows that see nothing have no tiles: zeros
  for (int i = blockIdx.x; i < a.B; i += gridDim.x) {
    const Row r = row_of<HD>(a, i, ROWS);
    if (by_unit)
      for (int u = tid; u < c.Hkv * groups; u += kWarps * 32)
        if (!r.tiles || u % groups >= r.groups) cuts[(int64_t)i * c.Hkv * groups + u].last = 0;
    if (r.n) continue;
    for (int u = tid; u < r.count * a.H * (HD / 4); u += kWarps * 32) {
      const int d = (u % (HD / 4)) * 4, h = u / (HD / 4) % a.H, tt = u / (HD / 4) / a.H;
      write_out(a, i, tt, h, d, make_float4(0, 0, 0, 0), 0.f, 0.f);
    }
  }

  // ---- this block's piece of the line
  int64_t total, piece, begin, end;
  int b;
  int64_t off;  // tiles of row b that lie before the piece
  if (a.B == 1) {
    total = line_tiles(a, row_of<HD>(a, 0, ROWS));
    piece = piece_of(total, gridDim.x);
    begin = piece * blockIdx.x;
    if (begin >= total) return;
    end = min(total, begin + piece);
    b = 0;
    off = begin;
  } else {
    // each thread sums a run of rows; the thread whose run holds the piece's
    // begin finds the row
    const int per = (a.B + kWarps * 32 - 1) / (kWarps * 32), r0 = min(a.B, tid * per), r1 = min(a.B, r0 + per);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += line_tiles(a, row_of<HD>(a, r, ROWS));
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    total = 0;
    int64_t before = inc - mine;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    piece = piece_of(total, gridDim.x);
    begin = piece * blockIdx.x;
    if (begin >= total) return;
    end = min(total, begin + piece);
    if (begin >= before && begin < before + mine) {
      for (int r = r0; r < r1; ++r) {
        const int64_t n = line_tiles(a, row_of<HD>(a, r, ROWS));
        if (begin < before + n) {
          s_row = r;
          s_at = begin - before;
          break;
        }
        before += n;
      }
    }
    __syncthreads();
    b = s_row;
    off = s_at;
  }

  const I8Const ic = i8_const();
  const unsigned ring = (unsigned)__cvta_generic_to_shared(sm) + warp * ST * SB;
  unsigned char *ringp = sm + warp * ST * SB;
  bool first = true;
  for (int64_t left = end - begin; left > 0;) {
    // ---- next segment
    Row r = row_of<HD>(a, b, ROWS);
    int64_t in_row = line_tiles(a, r);
    while (off >= in_row) {  // rows without tiles, or the row is done
      off -= in_row;
      if (++b >= a.B) return;  // only if d_pos changed under the kernel
      r = row_of<HD>(a, b, ROWS);
      in_row = line_tiles(a, r);
    }
    const int unit = (int)(off / r.tiles), t0 = (int)(off - (int64_t)unit * r.tiles);
    const int t1 = (int)min((int64_t)r.tiles, t0 + left);
    const int g = unit / r.groups, row0 = (unit - g * r.groups) * ROWS;
    const int64_t kvrow = (int64_t)b * c.Hkv + g;
    const uint8_t *kc = c.codes[0] + kvrow * c.N * HD, *vc = c.codes[1] + kvrow * c.N * HD;
    const float *ksc = c.scale[0] + kvrow * (c.N / c.block), *vsc = c.scale[1] + kvrow * (c.N / c.block);

    // One tile's K (which = 0) or V rows and scales into ring slot `slot`.
    auto issue = [&](int which, int tile, int slot) {
      if (tile < t1) {
        constexpr int CH = HD / 16, N = TL * CH / 32;  // 16-byte chunks of a row, copies of a lane
        const int p0 = tile * TL, p = lane / CH, ch = lane % CH;
        const unsigned st = ring + slot * SB + which * TL * HD;
        const uint8_t *src = (which ? vc : kc) + (size_t)p0 * HD + lane * 16;
        if (p0 + TL <= r.n) {
          // copy i is 512 bytes on; at head_dim 128 the swizzle of V's rows alternates
          const unsigned o = which ? v_off<HD>(p, ch) : k_off<HD>(p, ch), d0 = st + o;
          const unsigned d1 = st + (which && HD == 128 ? o ^ 64 : o);
#pragma unroll
          for (int i = 0; i < N; ++i) cp16s((i & 1 ? d1 : d0) + i * 512, src + i * 512);
        } else {  // the unit's last tile: zeros behind the last position
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int q = i * (32 / CH) + p, bytes = p0 + q < r.n ? 16 : 0;
            cp16z(st + (which ? v_off<HD>(q, ch) : k_off<HD>(q, ch)), bytes ? src + i * 512 : kc, bytes);
          }
        }
        if (lane < TM) {
          const int q = p0 + lane * 16, bytes = q < r.n ? 4 : 0;
          cp4z(ring + slot * SB + 2 * TL * HD + (which * TM + lane) * 4, (which ? vsc : ksc) + (bytes ? q / c.block : 0), bytes);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      issue(0, t0 + warp + i * kWarps, i);
      issue(1, t0 + warp + i * kWarps, i);
    }

    // ---- query operands: column gq of n-tile nt is query row row0 + 8 nt + gq
    uint32_t qf[NT][KS][2];
    float rs[NT][2];   // score factor of rows 2 tq, 2 tq + 1
    float qb[NT][2];   // where their scores' sums begin
    int see[NT][2];    // positions they see
    const int nrows = r.count * grp;
    const float sl2 = a.scale * kLog2e;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + 8 * nt + gq;
      float x[HD / 4];
      float mx = 0.f;
      const bool ok = row < nrows;
      const int t = row / grp, h = g * grp + row - t * grp;
      const int64_t o = b * a.q.sb + t * a.q.st + h * a.q.sh;
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
      int e = (int)(__float_as_uint(mx) >> 23) - 127;
      e = min(max(e, -126), 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23) * (sl2 * code_unit<FMT>());
      float qsum = 0.f;
#pragma unroll
      for (int j = 0; j < HD / 64; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float *y = x + 16 * j + 4 * s;
          constexpr int E = FMT == RV_KV8_INT8 ? 2 : 1;  // the second element of unpack_k's first pair
          qf[nt][4 * j + s][0] = pack_h2(y[0] * down, y[E] * down);
          qf[nt][4 * j + s][1] = pack_h2(y[3 - E] * down, y[3] * down);
          if (FMT == RV_KV8_INT8) {
            const float2 u = __half22float2(bits_h2(qf[nt][4 * j + s][0])), v = __half22float2(bits_h2(qf[nt][4 * j + s][1]));
            qsum += (u.x + u.y) + (v.x + v.y);
          }
        }
      if (FMT == RV_KV8_INT8) {
        qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
        qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        rs[nt][k] = __shfl_sync(0xffffffffu, up, (2 * tq + k) * 4);
        qb[nt][k] = -kBias * __shfl_sync(0xffffffffu, qsum, (2 * tq + k) * 4);
        const int rr = row0 + 8 * nt + 2 * tq + k;
        const int64_t n = (int64_t)row_pos(a.pos, b) + rr / grp + 1;
        see[nt][k] = rr < nrows ? (int)(n < 0 ? 0 : n > r.n ? r.n : n) : r.n;  // rows that do not exist see zeros
      }
    }
    int see_all = r.n;  // positions that every row of the group sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) see_all = min(see_all, min(see[nt][0], see[nt][1]));
    see_all = __reduce_min_sync(0xffffffffu, see_all);

    float o[MD][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MD; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    }

    int slot = 0;
    for (int tile = t0 + warp; tile < t1; tile += kWarps) {
      const unsigned char *kt = ringp + slot * SB, *vt = kt + TL * HD;
      const float *fs = reinterpret_cast<const float *>(kt + 2 * TL * HD);
      const int p0 = tile * TL;
      cp_wait<2 * ST - 1>();
      __syncwarp();
      float s[TM][NT][4];
#pragma unroll
      for (int j = 0; j < HD / 64; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const uint4 w0 = *reinterpret_cast<const uint4 *>(kt + k_off<HD>(16 * i + gq, 4 * j + tq));
          const uint4 w1 = *reinterpret_cast<const uint4 *>(kt + k_off<HD>(16 * i + gq + 8, 4 * j + tq));
          const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t f[4];
            unpack_k<FMT>(x0[k], f[0], f[2], ic);
            unpack_k<FMT>(x1[k], f[1], f[3], ic);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (j == 0 && k == 0) mma16_from(s[i][nt], f, qf[nt][0][0], qf[nt][0][1], qb[nt][0], qb[nt][1]);
              else mma16(s[i][nt], f, qf[nt][4 * j + k][0], qf[nt][4 * j + k][1]);
            }
          }
        }
      float ks[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) ks[i] = fs[i * GS];
      __syncwarp();  // every lane is done with the tile's K: its slot takes the next copy
      issue(0, tile + ST * kWarps, slot);
      // ---- scale, mask, running maximum (column 2 tq + k of n-tile nt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const float f = ks[i / GS] * rs[nt][k];
            s[i][nt][k] *= f;
            s[i][nt][2 + k] *= f;
          }
      const bool edge = p0 + TL > see_all;
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int n = see[nt][k] - p0 - gq;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
              if (n <= 16 * i) s[i][nt][k] = -INFINITY;
              if (n <= 16 * i + 8) s[i][nt][2 + k] = -INFINITY;
            }
          }
      }
      uint32_t pb[TM][NT][2], pl[TM][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mn[2], al[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = fmaxf(s[0][nt][k], s[0][nt][2 + k]);
#pragma unroll
          for (int i = 1; i < TM; ++i) x = fmaxf(x, fmaxf(s[i][nt][k], s[i][nt][2 + k]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mo = m[nt][k];
          m[nt][k] = fmaxf(mo, x);
          mn[k] = m[nt][k] == -INFINITY ? 0.f : m[nt][k];
          al[k] = ex2(mo - mn[k]);
          l[nt][k] *= al[k];
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
          for (int q = 0; q < 4; ++q) s[i][nt][q] = ex2(s[i][nt][q] - mn[q & 1]);
          l[nt][0] += s[i][nt][0] + s[i][nt][2];
          l[nt][1] += s[i][nt][1] + s[i][nt][3];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t hi = pack_h2(s[i][nt][2 * k], s[i][nt][2 * k + 1]);
            pb[i][nt][k] = transpose8(hi);
            if (LO) {
              const float2 h = __half22float2(bits_h2(hi));
              pl[i][nt][k] = transpose8(pack_h2(s[i][nt][2 * k] - h.x, s[i][nt][2 * k + 1] - h.y));
            }
          }
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < MD; ++i) {
            o[i][nt][0] *= al[0]; o[i][nt][1] *= al[1]; o[i][nt][2] *= al[0]; o[i][nt][3] *= al[1];
          }
        }
      }
      cp_wait<2 * ST - 1>();
      __syncwarp();
      float vs[NG][NT][2];
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            vs[i][nt][k] = fs[TM + i * GS] * code_unit<FMT>();
            // a block that the row sees nothing of adds nothing, whatever its scale
            if (edge && see[nt][k] <= p0 + 16 * GS * i) vs[i][nt][k] = 0.f;
          }
      float bias[NG][NT][2];  // where the products' sums begin
      if (FMT == RV_KV8_INT8) {
        const uint32_t one[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4];
#pragma unroll
            for (int j = 0; j < GS; ++j) {
              if (j == 0) mma16_from(x, one, pb[i * GS][nt][0], pb[i * GS][nt][1], 0.f, 0.f);
              else mma16(x, one, pb[i * GS + j][nt][0], pb[i * GS + j][nt][1]);
              if (LO) mma16(x, one, pl[i * GS + j][nt][0], pl[i * GS + j][nt][1]);
            }
            bias[i][nt][0] = -kBias * x[0];
            bias[i][nt][1] = -kBias * x[1];
          }
      }
      // ---- O^T += vs (V^T P^T)
      constexpr int VW = HD / 32;  // words of a V row that a thread takes
      uint32_t vw[TM][2][2][VW];   // [k-step][8 positions][position][word]
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int p = 16 * i + 8 * hb + 2 * tq + k;
            if (HD == 128) {
              const uint4 w = *reinterpret_cast<const uint4 *>(vt + v_off<HD>(p, gq));
              vw[i][hb][k][0] = w.x; vw[i][hb][k][1] = w.y; vw[i][hb][k][VW - 2] = w.z; vw[i][hb][k][VW - 1] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2 *>(vt + v_off<HD>(p, gq >> 1) + 8 * (gq & 1));
              vw[i][hb][k][0] = w.x; vw[i][hb][k][1] = w.y;
            }
          }
      __syncwarp();
      issue(1, tile + ST * kWarps, slot);
#pragma unroll
      for (int wq = 0; wq < VW; ++wq) {  // a word of each V row: two 16-element tiles of O^T
        uint32_t f[TM][2][4];            // [k-step][tile][operand]
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            const uint32_t w0 = vw[i][hb][0][wq], w1 = vw[i][hb][1][wq];
            uint32_t x[4];
            unpack_v<FMT>(w0, w1, x, ic);
            f[i][0][2 * hb] = x[0];
            f[i][0][2 * hb + 1] = x[1];
            f[i][1][2 * hb] = x[2];
            f[i][1][2 * hb + 1] = x[3];
          }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float(&oo)[4] = o[2 * wq + h][nt];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
              float acc[4];
              constexpr bool I8 = FMT == RV_KV8_INT8;
              mma16_from(acc, f[i * GS][h], pb[i * GS][nt][0], pb[i * GS][nt][1], I8 ? bias[i][nt][0] : 0.f, I8 ? bias[i][nt][1] : 0.f);
              if (LO) mma16(acc, f[i * GS][h], pl[i * GS][nt][0], pl[i * GS][nt][1]);
#pragma unroll
              for (int j = 1; j < GS; ++j) {
                mma16(acc, f[i * GS + j][h], pb[i * GS + j][nt][0], pb[i * GS + j][nt][1]);
                if (LO) mma16(acc, f[i * GS + j][h], pl[i * GS + j][nt][0], pl[i * GS + j][nt][1]);
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) oo[q] = fmaf(acc[q], vs[i][nt][q & 1], oo[q]);
            }
          }
      }
      slot = slot + 1 == ST ? 0 : slot + 1;
    }
    cp_wait<0>();

    // ---- join the warps' states
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = l[nt][k];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (gq == 0) {
          s_m[warp][8 * nt + 2 * tq + k] = m[nt][k];
          s_l[warp][8 * nt + 2 * tq + k] = x;
        }
      }
    __syncthreads();  // every warp is done with its ring: the states reuse it
    float *so = reinterpret_cast<float *>(sm);
    static_assert(kWarps * ROWS * HD * 4 <= smem_bytes(HD, NT), "the joined states fit the rings");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float *d = so + ((warp * ROWS) + 8 * nt + 2 * tq + k) * HD + gq * (HD / 8);
#pragma unroll
        for (int i = 0; i < MD; i += 2)
          *reinterpret_cast<float4 *>(d + 2 * i) = make_float4(o[i][nt][k], o[i][nt][2 + k], o[i + 1][nt][k], o[i + 1][nt][2 + k]);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == r.tiles;
    float *slotp = slots + (first ? 0 : slot_floats(HD, NT));
    if (tid == 0 && t0 == 0 && (by_unit || !whole)) {  // the unit begins here; cut: it goes on in the next piece
      const int64_t at = by_unit ? (int64_t)(b * c.Hkv + g) * groups + row0 / ROWS : blockIdx.x;
      cuts[at] = Cut{b, g, row0, (int)blockIdx.x, whole ? 0 : (int)((end - left + r.tiles - 1) / piece), first ? 0 : 1, {0, 0}};
    }
    for (int u = tid; u < ROWS * (HD / 4); u += kWarps * 32) {
      const int rr = u / (HD / 4), d = (u - rr * (HD / 4)) * 4, row = row0 + rr;
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
        const float4 y = *reinterpret_cast<const float4 *>(so + (w * ROWS + rr) * HD + d);
        ll = fmaf(s_l[w][rr], f, ll);
        x.x = fmaf(y.x, f, x.x); x.y = fmaf(y.y, f, x.y); x.z = fmaf(y.z, f, x.z); x.w = fmaf(y.w, f, x.w);
      }
      if (!whole) {
        *reinterpret_cast<float4 *>(slotp + rr * HD + d) = x;
        if (d == 0) {
          slotp[ROWS * HD + rr] = mm;
          slotp[ROWS * HD + ROWS + rr] = ll;
        }
      } else {
        const int t = row / grp, h = g * grp + row - t * grp;
        write_out(a, b, t, h, d, x, mm, ll);
      }
    }
    __syncthreads();  // the next segment's copies reuse the rings
    first = false;
    left -= t1 - t0;
    off += t1 - t0;
  }
}

// ------------------------------------------------------------------ join

// Joins the states of the units that the cut of the line went through: block
// x takes cut x of `pieces`.  WPR warps take one query row.
template <int HD, int NT, int WPR>
__global__ void __launch_bounds__(256) k_attn8_join(const __grid_constant__ Kv8AttnArgs a, int pieces) {
  constexpr int ROWS = 8 * NT, PER = HD / 32, RPB = 8 / WPR;
  __shared__ float s_x[8][HD], s_l[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = a.H / a.c.Hkv;
  pdl_wait();
  const Cut *cuts = static_cast<const Cut *>(a.work);
  const float *work = reinterpret_cast<const float *>(cuts + pieces);
  const Cut cut = cuts[blockIdx.x];
  const int b = cut.b, c0 = cut.c0, c1 = cut.last;
  if (c1 == 0) return;
  const int rr = blockIdx.y * RPB + warp / WPR, row = cut.row0 + rr, sub = warp % WPR;
  const bool live = rr < ROWS && row < row_count(a.count, b, a.T) * grp;
  const int t = row / grp, h = cut.g * grp + row - t * grp;
  float mm = -INFINITY, ll = 0.f, x[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = 0.f;
  if (live) {
    auto slot = [&](int c) { return work + (size_t)(2 * c + (c == c0 ? cut.slot : 0)) * slot_floats(HD, NT); };
    for (int c = c0 + lane; c <= c1; c += 32) mm = fmaxf(mm, __ldcg(slot(c) + ROWS * HD + rr));
    mm = warp_max(mm);
    const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
    for (int c = c0 + sub; c <= c1; c += WPR) {
      const float *s = slot(c);
      const float f = ex2(__ldcg(s + ROWS * HD + rr) - base);
      ll = fmaf(__ldcg(s + ROWS * HD + ROWS + rr), f, ll);
      float y[PER];
      if (PER == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(s + rr * HD) + lane);
        y[0] = v.x; y[1] = v.y; y[PER - 2] = v.z; y[PER - 1] = v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(s + rr * HD) + lane);
        y[0] = v.x; y[1] = v.y;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) x[i] = fmaf(y[i], f, x[i]);
    }
  }
  // through shared memory: the warps of a row, and 4 elements to a thread
#pragma unroll
  for (int i = 0; i < PER; ++i) s_x[warp][lane * PER + i] = x[i];
  if (lane == 0) s_l[warp] = ll;
  if (WPR > 1) __syncthreads();
  else __syncwarp();
  if (!live || sub || lane >= HD / 4) return;
  float4 v = make_float4(0, 0, 0, 0);
  ll = 0.f;
#pragma unroll
  for (int w = 0; w < WPR; ++w) {
    const float4 y = *reinterpret_cast<const float4 *>(&s_x[warp + w][4 * lane]);
    v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    ll += s_l[warp + w];
  }
  write_out(a, b, t, h, 4 * lane, v, mm, ll);
}

template <int FMT, int HD, int NT, int GS, bool LO>
cudaError_t launch_t(const Kv8AttnArgs &a, int n_sm, cudaStream_t s, int pdl) {
  auto fn = k_attn8<FMT, HD, NT, GS, LO>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(HD, NT));
  if (e != cudaSuccess) return e;
  const int pieces = blocks_per_sm(HD, NT) * n_sm, rows = a.T * (a.H / a.c.Hkv);
  const int64_t units = (int64_t)a.B * a.c.Hkv * ((rows + 8 * NT - 1) / (8 * NT));
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
  // fp16 outputs have 11 bits: weights rounded to as many would show in them
  return a.c.act == RV_F16 ? launch_lo<FMT, HD, NT, true>(a, n_sm, s, pdl) : launch_lo<FMT, HD, NT, false>(a, n_sm, s, pdl);
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
