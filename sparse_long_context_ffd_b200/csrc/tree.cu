// tree.cu -- attention of drafted tokens over the cache: the plain kernel.
//
// One CTA of 128 threads per (node, query head, sequence).  128 tokens at a
// time: thread t scores token t, the tile joins the running maximum and sum
// (fp32), then thread c adds the tile's weighted values of channel c.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ffd_ptx.cuh"
#include "ffd_serve.h"

namespace ffd {
namespace {

constexpr int kTile = 128;

__device__ __forceinline__ float e4m3_f(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half *>(&h));
}

__device__ __forceinline__ float bf16_f(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

template <bool kByte>
__global__ void __launch_bounds__(kTile) tree_kernel(const TreeParams p) {
  __shared__ float q_s[kHeadDim], w_s[kTile], red[4];
  const int i = blockIdx.x, head = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  const int heads = p.kv_heads * p.group;
  uint16_t *out = p.out + ((static_cast<size_t>(b) * p.nodes + i) * heads + head) * kHeadDim;
  const int len = p.lengths[b], size = p.sizes != nullptr ? p.sizes[b] : p.nodes;
  if (len < 0 || len > p.capacity || size < 0 || size > p.nodes || size > len) {
    if (t == 0) atomicOr(p.err, kFlagBadLength);
    out[t] = 0;
    return;
  }
  if (i >= size) return;
  const size_t row0 = (static_cast<size_t>(b) * p.kv_heads + head / p.group) * p.capacity;
  const int first = len - size;
  const uint64_t seen = p.mask != nullptr ? p.mask[static_cast<size_t>(b) * p.nodes + i] : (2ull << i) - 1ull;
  q_s[t] = bf16_f(p.q[((static_cast<size_t>(b) * p.nodes + i) * heads + head) * kHeadDim + t]) *
           (0.08838834764831845f * 1.4426950408889634f);
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int t0 = 0; t0 < len; t0 += kTile) {
    __syncthreads();
    const int token = t0 + t;
    const bool see = token < first || (token < len && ((seen >> (token - first)) & 1ull));
    float s = -INFINITY;
    if (see) {
      s = 0.0f;
      if (kByte) {
        const uint8_t *k = p.k + (row0 + token) * kByteRow;
        for (int c = 0; c < kHeadDim; ++c) s += q_s[c] * e4m3_f(k[c]);
        s *= bf16_f(p.k_scales[row0 + token]);
      } else {
        const uint16_t *k = reinterpret_cast<const uint16_t *>(p.k) + (row0 + token) * kHeadDim;
        for (int c = 0; c < kHeadDim; ++c) s += q_s[c] * bf16_f(k[c]);
      }
    }
    float top = s;
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if ((t & 31) == 0) red[t >> 5] = top;
    __syncthreads();
    const float m_new = fmaxf(fmaxf(m, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
    const float ref = m_new == -INFINITY ? 0.0f : m_new;
    const float w = see ? exp2f(s - ref) : 0.0f;
    w_s[t] = w;
    const float fade = exp2f(m - ref);
    m = m_new;
    o *= fade;
    l *= fade;
    __syncthreads();
    const int n = min(kTile, len - t0);
    for (int j = 0; j < n; ++j) {
      const int tok = t0 + j;
      if (tok >= first && !((seen >> (tok - first)) & 1ull)) continue;
      l += w_s[j];
      const float v = kByte ? e4m3_f(p.v[(row0 + tok) * kByteRow + t]) * bf16_f(p.v_scales[row0 + tok])
                            : bf16_f(reinterpret_cast<const uint16_t *>(p.v)[(row0 + tok) * kHeadDim + t]);
      o += w_s[j] * v;
    }
  }
  const float y = l == 0.0f ? 0.0f : o / l;
  out[t] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

}  // namespace

TreeLayout tree_layout(int32_t, int32_t, int32_t, int32_t) { return TreeLayout{256, 256}; }

cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.nodes), static_cast<unsigned>(p.kv_heads * p.group),
                  static_cast<unsigned>(p.batch));
  if (p.format == FFD_CACHE_BYTE)
    tree_kernel<true><<<grid, kTile, 0, stream>>>(p);
  else
    tree_kernel<false><<<grid, kTile, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ffd
