// rows.cu -- rotary positions, the cache write of several tokens a sequence,
// and the 8-bit cache read back.
//
// All three pass once over rows of 128 channels.  At small counts they are the
// launch and the host's call (16 tokens: 7 us a call back to back; a kernel may start
// while the one before it ends, 0.8 us more without).  At large ones rotation and
// read-back are near HBM's rate (8191 tokens x 40 heads, half of the channels,
// interleaved: 32 us, 5.3 TB/s, all of them in halves: 38; read-back 5.4 to 5.8), as is
// the bf16 write (32K tokens: 150 us, 5.4 TB/s).  The 8-bit write is slowed by
// instruction issue (173 us, 4.3 TB/s, 65% of issue slots taken): each of a row's 16
// threads does the row's division and reciprocal again.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ffd_serve.h"

namespace ffd {
namespace {

constexpr int kThreads = 256;
constexpr int kRowLanes = 16;                     // threads of a row, 8 channels (16 bytes) each
constexpr int kRowsAtOnce = kThreads / kRowLanes;  // rows a block handles at a time
constexpr int kMaxTokens = 8;                      // tokens of a block

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  x[0] = lo_f(w.x); x[1] = hi_f(w.x);
  x[2] = lo_f(w.y); x[3] = hi_f(w.y);
  x[4] = lo_f(w.z); x[5] = hi_f(w.z);
  x[6] = lo_f(w.w); x[7] = hi_f(w.w);
}

// Where a token goes: its cache slot, or -1 if it is not written.
__device__ __forceinline__ int token_slot(const RowsParams &p, int b, int i) {
  const int len = p.lengths[b];
  const int count = p.counts != nullptr ? p.counts[b] : p.new_tokens;
  if (len < 0 || len > p.capacity || count < 0 || count > p.new_tokens || count > len || i >= count) return -1;
  return len - count + i;
}

// A block takes `tokens_a_block` tokens and the row chunk blockIdx.y of each, at
// most kTableRows rows.
//
// The angles come first: thread t finds (cos, sin) of one pair of one token
// and leaves them in shared memory, since every head of the token needs them.
// position * turns wraps at whole turns in 64 bits; its top 32 bits, signed,
// are the angle in turns to 2^-32, which fp32 rounds by up to 2^-26 of a turn, and
// sincospif takes it from there.  Where a row comes from and goes to is found by one
// thread instead of 16.
//
// Then 16 threads take rows of one token, kInFlight before the first is used (a
// block has 16 KB on its way from HBM), each with the angles of its channels in
// registers: read from shared memory at every row, they were 88% of its
// bandwidth and set the pace.  Where the pairs' halves fall on whole
// threads (rotary_dim a multiple of 16, or interleaved) the partner channels
// come by shuffle; else each partner is loaded on its own.
constexpr int kInFlight = 4;
constexpr int kTableRows = kThreads;

struct RowPlace {
  const uint16_t *src;
  uint8_t *dst;       // null: not written
};

template <bool kAppend, bool kByte>
__global__ void __launch_bounds__(kThreads, kByte ? 4 : 5) rows_kernel(const __grid_constant__ RowsParams p, int tokens_a_block,
                                                        int rows_a_block) {
  extern __shared__ float2 turn_s[];  // [tokens_a_block][half]
  __shared__ RowPlace place_s[kTableRows];
  __shared__ uint16_t *scale_s[kByte ? kTableRows : 1];
  __shared__ uint8_t kind_s[kTableRows];  // 0 query, 1 key, 2 value
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int half = p.rotary_dim >> 1;
  const int token0 = blockIdx.x * tokens_a_block;
  const int tokens_here = min(tokens_a_block, p.tokens - token0);
  const int kv_rows = p.k != nullptr ? p.kv_heads : 0;
  const int q_rows = p.q != nullptr ? p.q_heads : 0;
  const int rows = q_rows + kv_rows + (kAppend ? kv_rows : 0);
  const int row_begin = blockIdx.y * rows_a_block;
  const int width = min(rows, row_begin + rows_a_block) - row_begin;
  const int todo = tokens_here * width;
  for (int r = threadIdx.x; r < todo; r += kThreads) {
    const int tl = r / width, row = row_begin + r - tl * width;
    const int token = token0 + tl;
    const int kind = row < q_rows ? 0 : row < q_rows + kv_rows ? 1 : 2;
    const int head = kind == 0 ? row : (row - q_rows) - (kind == 2 ? kv_rows : 0);
    RowPlace at;
    at.src = kind == 0 ? p.q + (static_cast<size_t>(token) * q_rows + head) * kHeadDim
                       : (kind == 1 ? p.k : p.v) + (static_cast<size_t>(token) * kv_rows + head) * kHeadDim;
    int slot = 0, b = 0;
    if (kAppend) {
      b = token / p.new_tokens;
      slot = token_slot(p, b, token - b * p.new_tokens);
    }
    if (kind == 0) {
      at.dst = reinterpret_cast<uint8_t *>(p.q_out + (static_cast<size_t>(token) * q_rows + head) * kHeadDim);
    } else if (kAppend) {
      const size_t to = (static_cast<size_t>(b) * p.kv_heads + head) * p.capacity + slot;
      at.dst = static_cast<uint8_t *>(kind == 1 ? p.k_out : p.v_out) + to * (kByte ? kByteRow : 2 * kHeadDim);
      if (kByte) scale_s[r] = (kind == 1 ? p.k_scales : p.v_scales) + to;
    } else {
      at.dst = static_cast<uint8_t *>(p.k_out) + (static_cast<size_t>(token) * kv_rows + head) * (2 * kHeadDim);
    }
    if (slot < 0) at.dst = nullptr;
    place_s[r] = at;
    kind_s[r] = static_cast<uint8_t>(kind);
  }
  for (int t = threadIdx.x; t < tokens_here * half; t += kThreads) {
    const int tl = t / half, token = token0 + tl;
    int position;
    if (p.positions != nullptr) {
      position = p.positions[token];
    } else {
      const int b = token / p.new_tokens;
      position = token_slot(p, b, token - b * p.new_tokens);
    }
    const uint64_t wrapped = static_cast<uint64_t>(static_cast<int64_t>(position)) * p.turns[t - tl * half];
    float sine, cosine;
    sincospif(static_cast<float>(static_cast<int32_t>(wrapped >> 32)) * 0x1p-31f, &sine, &cosine);
    turn_s[t] = make_float2(cosine * p.amplitude, sine * p.amplitude * p.sign);
  }
  __syncthreads();

  const int lane = threadIdx.x & (kRowLanes - 1);
  const int c0 = 8 * lane;
  const int mine_token = (threadIdx.x / kRowLanes) % tokens_a_block;  // tokens_a_block: a power of two up to 8
  const int first_row = threadIdx.x / kRowLanes / tokens_a_block, row_step = kRowsAtOnce / tokens_a_block;
  const float2 *cs = turn_s + mine_token * half;
  // the pairs of this thread's channels: 8 of them, or (interleaved) 4
  const int step = half >> 3;  // half layout: threads between a pair's halves
  const bool first = lane < step, second = !first && lane < 2 * step;
  float2 turn[8];
  if (mine_token < tokens_here) {
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((c0 >> 1) + e < half) turn[e] = cs[(c0 >> 1) + e];
    } else if ((half & 7) == 0 && (first || second)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        turn[e] = cs[(first ? c0 : c0 - half) + e];
        if (first) turn[e].y = -turn[e].y;
      }
    }
  }
  // (every thread of a warp runs the same number of rounds: the shuffles need both halves)
  for (int at = 0; at < width; at += kInFlight * row_step) {
    uint4 loaded[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int row = at + u * row_step + first_row, mine = mine_token * width + row;
      loaded[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row < width && mine < todo && place_s[mine].dst != nullptr)
        loaded[u] = *reinterpret_cast<const uint4 *>(place_s[mine].src + c0);
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      if (at + u * row_step >= width) break;
      const int row = at + u * row_step + first_row, mine = mine_token * width + row;
      const bool there = row < width && mine < todo;
      const RowPlace place = place_s[there ? mine : 0];
      const int kind = kind_s[there ? mine : 0];
      const bool live = there && place.dst != nullptr;
      const uint4 w = loaded[u];
      float x[8];
      unpack8(w, x);
      if (half > 0 && p.interleaved) {
        if (kind != 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((c0 >> 1) + e < half) {
              const float a = x[2 * e], b = x[2 * e + 1];
              x[2 * e] = a * turn[e].x - b * turn[e].y;
              x[2 * e + 1] = b * turn[e].x + a * turn[e].y;
            }
          }
        }
      } else if (half > 0 && (half & 7) == 0) {
        const int from = first ? lane + step : second ? lane - step : lane;
        uint4 o;
        o.x = __shfl_sync(0xFFFFFFFFu, w.x, from, kRowLanes);
        o.y = __shfl_sync(0xFFFFFFFFu, w.y, from, kRowLanes);
        o.z = __shfl_sync(0xFFFFFFFFu, w.z, from, kRowLanes);
        o.w = __shfl_sync(0xFFFFFFFFu, w.w, from, kRowLanes);
        if (kind != 2 && (first || second)) {
          float y[8];
          unpack8(o, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * turn[e].x + y[e] * turn[e].y;
        }
      } else if (half > 0 && kind != 2 && live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c0 + e;
          if (c < half) {
            x[e] = x[e] * cs[c].x - lo_f(place.src[c + half]) * cs[c].y;
          } else if (c < 2 * half) {
            x[e] = x[e] * cs[c - half].x + lo_f(place.src[c - half]) * cs[c - half].y;
          }
        }
      }
      __syncwarp();  // (an output may be its input: every partner is read before any store)
      if (live && (!kByte || kind == 0))
        *reinterpret_cast<uint4 *>(place.dst + 2 * c0) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
      if (kByte) {
        if (__all_sync(0xFFFFFFFFu, kind == 0)) continue;
        float top = 0.0f;  // (the maximum of a row with a NaN in it is NaN)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[e]));
#pragma unroll
        for (int d = kRowLanes / 2; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d, kRowLanes));
        if (live && kind != 0) {
          const __nv_bfloat16 s16 = __float2bfloat16_rn(__fdiv_rn(top, 448.0f));
          const float s = __bfloat162float(s16);
          uint16_t s_bits = __bfloat16_as_ushort(s16);
          uint32_t codes[2] = {0u, 0u};
          if (!(top < INFINITY)) {
            s_bits = 0x7FFFu;
            codes[0] = codes[1] = 0x7F7F7F7Fu;
          } else if (s != 0.0f) {
            // x / s correctly rounded, by Markstein's theorem (IBM J. Res. Dev. 34,
            // 1990): with inv the correctly rounded 1 / s, q = x inv and the exact
            // remainder x - q s, q + remainder inv is the rounded quotient, as long
            // as nothing underflows.  (A quotient below 2^-11 has code 0 anyway.)
            const float inv = __frcp_rn(s);
            float y[8];
            if (s >= 0x1p-80f) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float q = __fmul_rn(x[e], inv);
                y[e] = __fmaf_rn(__fmaf_rn(-q, s, x[e]), inv, q);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], s);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              codes[e >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(y[2 * e], y[2 * e + 1]),
                                                                              __NV_SATFINITE, __NV_E4M3))
                               << (16 * (e & 1));
          }
          *reinterpret_cast<uint2 *>(place.dst + c0) = make_uint2(codes[0], codes[1]);
          if (lane == 0) *scale_s[mine] = s_bits;
        }
      }
    }
  }
}

// Sixteen codes (16 bytes in, 32 out) a thread; code * scale is exact in fp32 (4
// and 8 significant bits), so the only rounding is the one to bf16.  Bound by HBM
// (4 x 8 x 32768 tokens: 139 to 149 us, 5.4 to 5.8 TB/s; 18 MB: 5.8 us).  One row a thread and
// more blocks beat several rows in flight a thread: 2, 4 and 8 of them took 141,
// 144 and 154 us, and of the 18 MB 8.1, 8.2 and 9.0 us where one took 7.2.
constexpr int kReadLanes = 8;  // threads of a row
constexpr int kReadAtOnce = kThreads / kReadLanes;

__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const bool values = blockIdx.y != 0;
  uint16_t *out = values ? p.out[1] : p.out[0];
  const uint8_t *codes = values ? p.codes[1] : p.codes[0];
  const uint16_t *scales = values ? p.scales[1] : p.scales[0];
  if (out == nullptr) return;
  const int chunks = (p.count + kReadAtOnce - 1) / kReadAtOnce;
  const int bh = blockIdx.x / chunks;
  const int len = p.lengths[bh / p.kv_heads];
  if (len < 0 || len > p.capacity) return;
  const int rows = min(p.count, len - p.begin);
  const int lane = threadIdx.x & (kReadLanes - 1);
  const int t = (blockIdx.x - bh * chunks) * kReadAtOnce + threadIdx.x / kReadLanes;
  if (t >= rows) return;
  const size_t in0 = static_cast<size_t>(bh) * p.capacity + p.begin;
  const size_t out0 = static_cast<size_t>(bh) * p.count;
  const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(codes + (in0 + t) * kByteRow) + lane);
  const float s = lo_f(scales[in0 + t]);
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  uint32_t y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __nv_fp8x2_storage_t pair = static_cast<__nv_fp8x2_storage_t>(words[e >> 1] >> (16 * (e & 1)));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    y[e] = pack_bf16(f.x * s, f.y * s);
  }
  uint4 *dst = reinterpret_cast<uint4 *>(out + (out0 + t) * kHeadDim) + 2 * lane;
  __stcs(dst, make_uint4(y[0], y[1], y[2], y[3]));
  __stcs(dst + 1, make_uint4(y[4], y[5], y[6], y[7]));
}

template <bool kAppend, bool kByte>
cudaError_t launch_rows_as(const RowsParams &p, cudaStream_t stream) {
  const int rows = (p.q != nullptr ? p.q_heads : 0) + (p.k != nullptr ? (kAppend ? 2 : 1) * p.kv_heads : 0);
  // Few tokens: as many blocks as there are sixteens of rows, for the latency.
  // Many: whole tokens, whose angles are then found once.
  int tokens_a_block = 1, rows_a_block = kRowsAtOnce;
  if (p.tokens >= 2048) {
    rows_a_block = rows < kTableRows ? rows : kTableRows;
    while (tokens_a_block < kMaxTokens && 2 * tokens_a_block * rows_a_block <= kTableRows) tokens_a_block *= 2;
  }
  const dim3 grid(static_cast<unsigned>((p.tokens + tokens_a_block - 1) / tokens_a_block),
                  static_cast<unsigned>((rows + rows_a_block - 1) / rows_a_block));
  const size_t smem = static_cast<size_t>(tokens_a_block) * (p.rotary_dim / 2) * sizeof(float2);
  return launch_early(rows_kernel<kAppend, kByte>, grid, kThreads, smem, stream, p, tokens_a_block, rows_a_block);
}

}  // namespace

cudaError_t launch_rows(const RowsParams &p, bool append, int format, cudaStream_t stream) {
  if (!append) return launch_rows_as<false, false>(p, stream);
  return format == FFD_CACHE_BYTE ? launch_rows_as<true, true>(p, stream) : launch_rows_as<true, false>(p, stream);
}

cudaError_t launch_read(const ReadParams &p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.count + kReadAtOnce - 1) / kReadAtOnce) * static_cast<unsigned>(p.batch * p.kv_heads), 2);
  return launch_early(read_kernel, grid, kThreads, 0, stream, p);
}

}  // namespace ffd
