// ffd_serve.h -- parameter blocks and launchers of the multi-token operators:
// rotary positions, the cache write, the 8-bit cache's read-back (rows.cu) and
// attention of drafted tokens over the cache (tree.cu).
#pragma once

#include "ffd_internal.h"

namespace ffd {

constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kByteRow = kHeadDim;  // bytes of an e4m3 cache row

// ffd_rotate and ffd_append_tokens.  A token's rows are its query heads, key
// heads and (append only) value heads, in that order.
struct RowsParams {
  uint64_t turns[kMaxPairs];  // f / 2pi of each rotated pair, a 64-bit binary fraction
  float amplitude, sign;      // sign -1: the opposite angle
  int32_t rotary_dim, interleaved;
  const uint16_t *q, *k, *v;    // null: no such rows
  uint16_t *q_out;
  void *k_out, *v_out;          // rotate: like the input; append: the cache
  uint16_t *k_scales, *v_scales;
  const int32_t *positions;     // null: the slot (append)
  const int32_t *lengths, *counts;
  int32_t tokens;               // rotate: tokens; append: batch * new_tokens
  int32_t q_heads, kv_heads, new_tokens, capacity;
};

struct ReadParams {
  const uint8_t *codes[2];      // k, v
  const uint16_t *scales[2];
  uint16_t *out[2];             // null: not wanted
  const int32_t *lengths;
  int32_t batch, kv_heads, capacity, begin, count;
};

// A launch that may start while the kernel before it in the stream ends, and
// waits for it on the GPU (griddepcontrol.wait, before it reads or writes anything
// of the stream's; a call's second kernel may read what its first has waited for): 14.3 -> 12.1 us for 5 nodes over 4096 tokens back to back.
template <class Kernel, class... Args>
inline cudaError_t launch_early(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                const Args &...args) {
  cudaLaunchAttribute attribute{};
  attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attribute.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(static_cast<unsigned>(threads));
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &attribute;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

// append: write k and v into the cache of the given format; else rotate only.
cudaError_t launch_rows(const RowsParams &p, bool append, int format, cudaStream_t stream);
cudaError_t launch_read(const ReadParams &p, cudaStream_t stream);

constexpr int kTreeTile = 128;        // tokens of a tile
constexpr int kTreeCtas = 148;        // one a multiprocessor
constexpr int kTreeRows = 256;        // query rows of a unit: two accumulators of 128

// A unit: up to kTreeRows query rows (node, head of the group) of one kv-head
// of one sequence, over all the sequence's tiles.
struct TreeParams {
  const uint16_t *q;            // bf16 [B][n][Hq][D]
  const uint16_t *k_scales, *v_scales;
  const uint8_t *k, *v;
  const int32_t *lengths, *sizes;
  const uint64_t *mask;
  uint16_t *out;
  uint32_t *err;
  int2 *table;                  // [B][kv_heads][units a head]: first CTA * 2 + its slot, CTAs
  float *partials;              // [ctas][2][part_floats(rows)]
  int32_t batch, kv_heads, group_log2, nodes, capacity, format;
  int32_t units_a_head, rows, ctas;
  uint64_t wait_limit_ns;
};

struct TreeLayout {
  size_t table, partials, total;
  int32_t units_a_head, rows, ctas;
};

TreeLayout tree_layout(int32_t batch, int32_t kv_heads, int32_t group, int32_t nodes, int32_t capacity);
cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream);
cudaError_t launch_tree_narrow(const TreeParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v,
                               cudaStream_t stream);  // at most 16 rows; without the merge

}  // namespace ffd
