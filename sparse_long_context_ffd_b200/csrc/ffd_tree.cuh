// ffd_tree.cuh -- what the kernels of drafted-token attention share: a CTA's
// part of the work, the e4m3 parts of a weight, the end of a segment.
#pragma once

#include <cuda_bf16.h>

#include "ffd_ptx.cuh"
#include "ffd_serve.h"
#include "ffd_tcgen05.cuh"

namespace ffd {
namespace {

constexpr int kTile = kTreeTile;
constexpr float kScoreScale = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)

__device__ __forceinline__ float bf16_f(uint32_t b) { return __uint_as_float(b << 16); }

// A running reference in units of log 2.  Weights are 2^(s - m), s exact and m a
// score rounded to fp32: all of a row's are off by the factor that m is, which its
// sum shares.  In bf16 that may be 2^64, at 2^30.  In e4m3 it must stay within the
// 7% between 448, where m moves, and 480, which is NaN's code; at 2^19 the score's
// and the border's roundings make 2% of it.  A row beyond that is NaN, not a
// number that is wrong.
template <bool kByte>
__device__ __forceinline__ float in_range(float m) {
  return fabsf(m) > (kByte ? 0x1p19f : 0x1p30f) && m != -INFINITY ? __uint_as_float(0x7FFFFFFFu) : m;
}

__device__ __forceinline__ float exp2_f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in one 64-bit register: one instruction does both.
__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void one_each(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 2^z of two values on the multiply-add pipe, for a part of a tile's weights:
// the exponential unit gives 16 a clock and multiprocessor, and would set the
// pace alone.  z is taken apart into the nearest whole number n (adding 1.5 2^23
// rounds to it) and f in [-0.5, 0.5]; 2^f is a polynomial of degree 4, of least
// relative error 2.6e-6 (found by Remez's exchange; a weight is rounded to 2^-9);
// 2^n is made of its bits.  z up to 127; below -126 it gives 2^-126, and NaN
// stays NaN.
__device__ __forceinline__ void exp2_poly2(uint64_t z, float &a, float &b) {
  float z0, z1;
  one_each(z, z0, z1);
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(z0));  // -126
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(z1));
  z = two(z0, z1);
  constexpr float kRound = 12582912.0f;
  const uint64_t n = add2(z, two(kRound, kRound));
  const uint64_t f = fma2(add2(n, two(-kRound, -kRound)), two(-1.0f, -1.0f), z);
  uint64_t y = fma2(f, two(0.009570102207362652f, 0.009570102207362652f), two(0.05591785907745361f, 0.05591785907745361f));
  y = fma2(y, f, two(0.240247443318367f, 0.240247443318367f));
  y = fma2(y, f, two(0.6931217908859253f, 0.6931217908859253f));
  y = fma2(y, f, two(0.9999992847442627f, 0.9999992847442627f));
  float n0, n1;
  one_each(n, n0, n1);
  y = mul2(y, two(__uint_as_float((__float_as_uint(n0) << 23) + 0x3F800000u),
                  __uint_as_float((__float_as_uint(n1) << 23) + 0x3F800000u)));
  one_each(y, a, b);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Four values in [0, 448] as e4m3 parts, a byte each: `hi` cut off to 4
// significant bits, `lo` what is left, rounded to 4.  Times 2^-120 a value's
// e4m3 code is bits 20 to 27 of its fp32 code, subnormals included, so cutting
// off is a mask and rounding an addition; the conversion instructions run at a
// quarter of these ones' rate.  NaN becomes e4m3's NaN.
// The second part is kept times 2^kLo, where products of the two parts are
// summed apart: kLo 3 takes values below 512.
template <int kLo = 0>
__device__ __forceinline__ void split4(float w0, float w1, float w2, float w3, uint32_t &hi, uint32_t &lo) {
  uint32_t h[4], l[4];
  const float w[4] = {w0, w1, w2, w3};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float t = w[e] * 0x1p-120f;
    const uint32_t bits = __float_as_uint(t);
    h[e] = bits << 4;
    float rest = t - __uint_as_float(bits & 0xFFF00000u);
    // (the intrinsic: of a plain product by 2^kLo whose bits are used like this,
    // nvcc 12.9 shifted the bits, which is another number)
    if (kLo > 0) rest = __fmul_rn(rest, static_cast<float>(1 << kLo));
    l[e] = __float_as_uint(rest) * 16u + 0x00800000u;
  }
  hi = __byte_perm(__byte_perm(h[0], h[1], 0x0073), __byte_perm(h[2], h[3], 0x0073), 0x5410);
  lo = __byte_perm(__byte_perm(l[0], l[1], 0x0073), __byte_perm(l[2], l[3], 0x0073), 0x5410);
}

// The same of values of either sign.
template <int kLo = 0>
__device__ __forceinline__ void split4_signed(float w0, float w1, float w2, float w3, uint32_t &hi, uint32_t &lo) {
  split4<kLo>(fabsf(w0), fabsf(w1), fabsf(w2), fabsf(w3), hi, lo);
  const uint32_t signs = __byte_perm(__byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x0073),
                                     __byte_perm(__float_as_uint(w2), __float_as_uint(w3), 0x0073), 0x5410) &
                         0x80808080u;
  hi |= signs;
  lo |= signs;
}

// ------------------------------------------------------------------ waits --

// A CTA's waits, in shared memory.  After one of them ran out nobody waits any more:
// copies and matrix instructions stop, and the softmax threads, whose barriers count
// on one another, go through the rest of their work on whatever is there.
struct Waits {
  volatile int dead;  // a wait was given up
  uint32_t *err;
  uint64_t limit_ns;
};

#ifdef FFD_DEBUG
constexpr uint32_t kAttempts = 1;
#else
constexpr uint32_t kAttempts = 4096;  // a few milliseconds at most
#endif

// Whether to go on; else the CTA's waits are over.
__device__ __forceinline__ bool keep_waiting(Waits *w, uint64_t start) {
  if (w->dead == 0 && global_timer_ns() - start > w->limit_ns) {
    w->dead = 1;
    atomicOr(w->err, kFlagTimeout);
  }
  return w->dead == 0;
}

// A wait whose first attempts were in vain.  (Apart: inlined at every wait, one token
// over 4 x 32768 in 8 bits took 63 us instead of 62.)
__device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, Waits *w) {
  const uint64_t start = global_timer_ns();
  while (keep_waiting(w, start))
    if (mbar_wait_short<kAttempts>(bar, parity)) return true;
  return false;
}

// ------------------------------------------------------------------- work --

struct Sequence {
  int len, size;
  bool good;
  __device__ __forceinline__ Sequence(const TreeParams &p, int b) {
    len = p.lengths[b];
    size = p.sizes != nullptr ? p.sizes[b] : p.nodes;
    good = len >= 0 && len <= p.capacity && size >= 0 && size <= p.nodes && size <= len;
  }
  // tiles of each of its units
  __device__ __forceinline__ int tiles() const { return good && size > 0 ? (len + kTile - 1) / kTile : 0; }
};

struct Segment {
  int b, unit, tile0, tiles, all;  // tiles of the unit in this CTA, and in all
  int len, size;
};

// A CTA's part of the tile list, segment by segment.
struct Walk {
  int b, off, left;
  __device__ __forceinline__ bool next(const TreeParams &p, Segment &g) {
    if (left == 0) return false;
    const int units = p.kv_heads * p.units_a_head;
    for (; b < p.batch; ++b, off = 0) {
      const Sequence q(p, b);
      const int each = q.tiles();
      if (off >= each * units) continue;
      g.b = b;
      g.unit = off / each;
      g.tile0 = off - g.unit * each;
      g.all = each;
      g.tiles = min(each - g.tile0, left);
      g.len = q.len;
      g.size = q.size;
      off += g.tiles;
      left -= g.tiles;
      return true;
    }
    return false;
  }
};

// A part of a unit in the workspace: its rows' O, 32 channels after another as
// [row][32], a row's eight 16-byte vectors in the order c ^ (row & 7) (as they
// are staged in shared memory, free of bank conflicts), then (m, l) of the rows.
__host__ __device__ constexpr size_t part_floats(int rows) { return (static_cast<size_t>(rows) * 130 + 3) / 4 * 4; }

__device__ __forceinline__ size_t part_vector(int rows, int row, int vector) {  // of 32, four channels each
  return (static_cast<size_t>(vector >> 3) * rows + row) * 32 + 4 * ((vector & 7) ^ (row & 7));
}

__device__ __forceinline__ size_t part_sums(int rows, int row) { return static_cast<size_t>(rows) * 128 + 2 * row; }

// CTA c of the grid holds tiles part_begin(c) to part_begin(c + 1) of `total`;
// of as many CTAs as there are tiles every one has one.
__device__ __forceinline__ int part_begin(int total, int c) {
  const int ctas = min(static_cast<int>(gridDim.x), total), each = total / ctas;
  return c * each + min(c, total - each * ctas);
}

__device__ __forceinline__ int part_of(int total, int tile) {
  const int ctas = min(static_cast<int>(gridDim.x), total), each = total / ctas, longer = total - each * ctas;
  const int split = longer * (each + 1);
  return tile < split ? tile / (each + 1) : longer + (tile - split) / each;
}

// This CTA's part of the tiles: thread t adds up the sequences of its chunk.
// start: the first sequence, the tile among its units', tiles, all tiles, and (or
// 0) the CTAs of its unit (CTA-wide after the next __syncthreads).
//
// A CTA that goes on to a second unit ends the first and begins the next at a
// cost of about four tiles (5 us; 64 nodes over 3 ragged contexts of up to 16K:
// such CTAs took 65 us, the others 54).  So where there are no more than 32
// sequences, and fewer units than CTAs, every unit is cut into equal pieces of
// at most L tiles, one a CTA, with the smallest L for which there are CTAs
// enough; unless L is more than kSegmentTiles above the equal share (4 x 8 units
// of 256 tiles: 64 against 56).
constexpr int kSegmentTiles = 4;

template <int kThreads>
__device__ __forceinline__ void find_part(const TreeParams &p, int *sum_s, int *start) {
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) start[0] = start[1] = start[2] = start[4] = 0;
  const int chunk = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, tid * chunk), b1 = min(p.batch, b0 + chunk);
  const int units = p.kv_heads * p.units_a_head;
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += Sequence(p, b).tiles() * units;
  int upto = sum;
  for (int d = 1; d < 32; d <<= 1) {
    const int other = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if ((tid & 31) >= d) upto += other;
  }
  if ((tid & 31) == 31) sum_s[warp] = upto;
  __syncthreads();
  int total = 0, before = upto - sum;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sum_s[w];
    total += sum_s[w];
  }
  int begin = 0, end = 0;
  if (static_cast<int>(blockIdx.x) < total) {
    begin = part_begin(total, blockIdx.x);
    end = part_begin(total, blockIdx.x + 1);
  }
  if (begin >= before && begin < before + sum && end > begin) {
    int off = begin - before, b = b0;
    for (; b < b1; ++b) {
      const int n = chunk == 1 ? sum : Sequence(p, b).tiles() * units;
      if (off < n) break;
      off -= n;
    }
    start[0] = b;
    start[1] = off;
    start[2] = end - begin;
  }
  if (tid == 0) start[3] = total;
  if (warp == 0 && p.batch <= 32 && total > static_cast<int>(gridDim.x)) {
    __syncwarp();
    const int ctas = gridDim.x, t = sum / units;  // (chunk is 1)
    if (static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, t > 0 ? units : 0)) <= ctas) {
      const int share = (total + ctas - 1) / ctas;
      int lo = share + kSegmentTiles + 1;
#pragma unroll
      for (int more = kSegmentTiles; more >= 0; --more) {
        const int pieces = units * ((t + share + more - 1) / (share + more));
        if (static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, pieces)) <= ctas) lo = share + more;
      }
      if (lo <= share + kSegmentTiles) {
        const int pieces = (t + lo - 1) / lo, mine = units * pieces;
        int to = mine;
        for (int d = 1; d < 32; d <<= 1) {
          const int other = __shfl_up_sync(0xFFFFFFFFu, to, d);
          if (tid >= d) to += other;
        }
        const int c = blockIdx.x, at = c - (to - mine), all = __shfl_sync(0xFFFFFFFFu, to, 31);
        if (tid == 0) start[2] = 0;
        __syncwarp();
        if (at >= 0 && at < mine && c < all) {
          const int unit = at / pieces, k = at - unit * pieces, each = t / pieces, longer = t - each * pieces;
          start[0] = tid;
          start[1] = unit * t + k * each + min(k, longer);
          start[2] = each + (k < longer ? 1 : 0);
          start[4] = pieces;
        }
      }
    }
  }
}

// Where merge_tree_kernel finds the parts of a unit whose first tile is here.
__device__ __forceinline__ void note_unit(const TreeParams &p, const Segment &g, const Walk &walk, const int *start,
                                          bool starts) {
  int2 *entry = p.table + static_cast<size_t>(g.b) * p.kv_heads * p.units_a_head + g.unit;
  if (start[4] > 0) {
    *entry = make_int2(2 * static_cast<int>(blockIdx.x), start[4]);
    return;
  }
  const int total = start[3];
  const int here = part_begin(total, blockIdx.x) + start[2] - walk.left - g.tiles;  // the unit's first tile
  const int c1 = part_of(total, here + g.all - 1);
  *entry =
      make_int2(2 * static_cast<int>(blockIdx.x) + (starts ? 0 : 1), c1 - static_cast<int>(blockIdx.x) + 1);
}

// The nodes of its tree that node i sees, of those that are there.
__device__ __forceinline__ uint64_t seen_nodes(const TreeParams &p, const Segment &g, int i) {
  if (i >= g.size) return 0;
  const uint64_t in_tree = g.size >= 64 ? ~0ull : (1ull << g.size) - 1ull;
  return (p.mask != nullptr ? p.mask[static_cast<size_t>(g.b) * p.nodes + i] : (2ull << i) - 1ull) & in_tree;
}

// What the values of drafted tokens that are not finite, taken out of the
// products, add to channel `channel` of a row that sees `bits`.
template <bool kByte>
__device__ __noinline__ float odd_values(const TreeParams &p, const Segment &g, int bh, uint64_t bits, int channel) {
  float y = 0.0f;
  for (; bits != 0; bits &= bits - 1) {
    const size_t row = static_cast<size_t>(bh) * p.capacity + (g.len - g.size) + __ffsll(static_cast<long long>(bits)) - 1;
    if constexpr (kByte) {
      if ((p.v[row * kHeadDim + channel] & 0x7Fu) == 0x7Fu || (p.v_scales[row] & 0x7F80u) == 0x7F80u)
        y = __uint_as_float(0x7FFFFFFFu);
    } else {
      const uint32_t x = reinterpret_cast<const uint16_t *>(p.v)[row * kHeadDim + channel];
      if ((x & 0x7F80u) == 0x7F80u) y += bf16_f(x);
    }
  }
  return y;
}

// A weight of zero must not meet a value that is not finite.  Of token t's row
// in a tile of V in shared memory, vectors [c0, c1): past the sequence the row
// may hold anything and is cleared; a drafted token's may hold infinities or NaN
// that some nodes see: they are taken out, and true is returned.
template <bool kByte>
__device__ __noinline__ bool clean_values(uint8_t *tile, int t, bool past, int c0, int c1) {
  uint4 *v = reinterpret_cast<uint4 *>(tile + t * 128);
  bool bad = false;
  for (int c = c0; c < c1; ++c) {
    uint4 &y = v[(c >> 3) * 1024 + ((c + t) & 7)];
    if (past) {
      y = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint32_t x[4] = {y.x, y.y, y.z, y.w};
    bool changed = false;
    constexpr uint32_t kTop = kByte ? 0x7Fu : 0x7F80u, kAll = kByte ? 0xFFu : 0xFFFFu;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int h = 0; h < 32; h += kByte ? 8 : 16)
        if (((x[e] >> h) & kTop) == kTop) {
          x[e] &= ~(kAll << h);
          changed = true;
        }
    if (changed) {
      y = make_uint4(x[0], x[1], x[2], x[3]);
      bad = true;
    }
  }
  return bad;
}

}  // namespace
}  // namespace ffd
