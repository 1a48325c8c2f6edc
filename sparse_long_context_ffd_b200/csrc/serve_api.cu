// serve_api.cu -- entry points of the multi-token operators (include/ffd.h,
// "Several new tokens a sequence"): host checks, the rotary plan, parameter
// blocks.  No call allocates, synchronises or keeps state.
#include <cmath>
#include <cstring>

#include "ffd.h"
#include "ffd_serve.h"

using namespace ffd;

namespace {

constexpr size_t kErrBytes = 256;  // the error word at the head of a workspace

// The limit of ffd_decode_tree's waits on the device; the debug library can shorten it.
#ifdef FFD_DEBUG
uint64_t g_wait_limit_ns = kWaitLimitNs;
#else
constexpr uint64_t g_wait_limit_ns = kWaitLimitNs;
#endif

struct Range {
  const void *p;
  size_t bytes;
};

bool overlap(const Range &a, const Range &b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool rope_ok(const ffd_rope *r) {
  return r->rotary_dim >= 2 && r->rotary_dim <= kHeadDim && r->rotary_dim % 2 == 0 &&
         (r->layout == FFD_ROPE_HALF || r->layout == FFD_ROPE_INTERLEAVED) && std::isfinite(r->amplitude) &&
         r->amplitude > 0.0f;
}

void set_rope(RowsParams *p, const ffd_rope *r, bool inverse) {
  p->amplitude = 1.0f;
  p->sign = inverse ? -1.0f : 1.0f;
  if (r == nullptr) return;
  std::memcpy(p->turns, r->turns, sizeof(p->turns));
  p->amplitude = r->amplitude;
  p->rotary_dim = r->rotary_dim;
  p->interleaved = r->layout == FFD_ROPE_INTERLEAVED;
}

bool positive(double x) { return std::isfinite(x) && x > 0.0; }

// Tensors of the cache: null, alignment and format checks.
ffd_status check_cache(const ffd_cache *c) {
  if (c == nullptr || c->reserved != 0 || (c->format != FFD_CACHE_BF16 && c->format != FFD_CACHE_BYTE))
    return FFD_ERR_INVALID_ARG;
  if (c->k == nullptr || c->v == nullptr || !aligned16(c->k) || !aligned16(c->v)) return FFD_ERR_INVALID_ARG;
  if (c->format == FFD_CACHE_BYTE &&
      (c->k_scales == nullptr || c->v_scales == nullptr || !aligned16(c->k_scales) || !aligned16(c->v_scales)))
    return FFD_ERR_INVALID_ARG;
  return FFD_OK;
}

}  // namespace

extern "C" {

ffd_status ffd_rope_init(const ffd_rope_options *o, ffd_rope *rope) {
  if (o == nullptr || rope == nullptr) return FFD_ERR_INVALID_ARG;
  if (o->reserved != 0 || o->rotary_dim < 2 || o->rotary_dim > kHeadDim || o->rotary_dim % 2 != 0 ||
      (o->layout != FFD_ROPE_HALF && o->layout != FFD_ROPE_INTERLEAVED) ||
      o->scaling < FFD_ROPE_SCALE_NONE || o->scaling > FFD_ROPE_SCALE_BY_PARTS || !positive(o->base) ||
      !positive(o->amplitude) || !std::isfinite(static_cast<float>(o->amplitude)) ||
      static_cast<float>(o->amplitude) == 0.0f)
    return FFD_ERR_INVALID_ARG;
  if (o->scaling != FFD_ROPE_SCALE_NONE && !positive(o->factor)) return FFD_ERR_INVALID_ARG;
  if (o->scaling == FFD_ROPE_SCALE_BY_PARTS &&
      (!positive(o->original_length) || !std::isfinite(o->low) || !std::isfinite(o->high) || o->low < 0.0 ||
       !(o->high > o->low)))
    return FFD_ERR_INVALID_ARG;
  // 64-bit mantissas (long double), so that the fractions are exact to far
  // below the 2^-32 of a turn that the kernel uses at any 32-bit position
  const long double two_pi = 2.0L * acosl(-1.0L);
  const int d = o->rotary_dim;
  long double base = o->base;
  if (o->scaling == FFD_ROPE_SCALE_BASE && d > 2)
    base *= powl(static_cast<long double>(o->factor), static_cast<long double>(d) / (d - 2));
  ffd_rope r{};
  for (int i = 0; i < d / 2; ++i) {
    long double f = powl(base, -2.0L * i / d);
    if (o->scaling == FFD_ROPE_SCALE_LINEAR) f /= o->factor;
    if (o->scaling == FFD_ROPE_SCALE_BY_PARTS) {
      const long double turns = o->original_length * f / two_pi;
      const long double g = fminl(fmaxl((turns - o->low) / (static_cast<long double>(o->high) - o->low), 0.0L), 1.0L);
      f = (1.0L - g) * f / o->factor + g * f;
    }
    if (!std::isfinite(f)) return FFD_ERR_INVALID_ARG;
    long double whole;
    const long double part = modfl(f / two_pi, &whole);  // whole turns do not matter: positions are integers
    r.turns[i] = static_cast<uint64_t>(ldexpl(part, 64));
  }
  r.amplitude = static_cast<float>(o->amplitude);
  r.rotary_dim = d;
  r.layout = o->layout;
  *rope = r;
  return FFD_OK;
}

ffd_status ffd_rotate(const ffd_rope *rope, int64_t tokens, const int32_t *d_positions, int32_t inverse,
                      int32_t num_q_heads, const void *q_bf16, void *q_out_bf16, int32_t num_k_heads,
                      const void *k_bf16, void *k_out_bf16, void *cuda_stream) {
  if (rope == nullptr || !rope_ok(rope) || tokens < 0 || (inverse != 0 && inverse != 1) || num_q_heads < 1)
    return FFD_ERR_INVALID_ARG;
  const bool with_k = k_bf16 != nullptr || k_out_bf16 != nullptr;
  if (with_k && num_k_heads < 1) return FFD_ERR_INVALID_ARG;
  if (tokens >= (int64_t{1} << 31) || num_q_heads > 65535 || (with_k && num_k_heads > 65535))
    return FFD_ERR_UNSUPPORTED;
  if (tokens == 0) return FFD_OK;
  if (q_bf16 == nullptr || q_out_bf16 == nullptr || d_positions == nullptr || !aligned4(d_positions) ||
      !aligned16(q_bf16) || !aligned16(q_out_bf16))
    return FFD_ERR_INVALID_ARG;
  if (with_k && (k_bf16 == nullptr || k_out_bf16 == nullptr || !aligned16(k_bf16) || !aligned16(k_out_bf16)))
    return FFD_ERR_INVALID_ARG;
  const size_t q_bytes = static_cast<size_t>(tokens) * num_q_heads * kHeadDim * 2;
  const size_t k_bytes = with_k ? static_cast<size_t>(tokens) * num_k_heads * kHeadDim * 2 : 0;
  const Range q{q_bf16, q_bytes}, qo{q_out_bf16, q_bytes}, k{k_bf16, k_bytes}, ko{k_out_bf16, k_bytes};
  const Range at{d_positions, static_cast<size_t>(tokens) * 4};
  if ((q.p != qo.p && overlap(q, qo)) || (k.p != ko.p && overlap(k, ko)) || overlap(q, ko) || overlap(k, qo) ||
      overlap(qo, ko) || overlap(at, qo) || overlap(at, ko))
    return FFD_ERR_INVALID_ARG;
  RowsParams p{};
  set_rope(&p, rope, inverse == 1);
  p.q = static_cast<const uint16_t *>(q_bf16);
  p.q_out = static_cast<uint16_t *>(q_out_bf16);
  p.q_heads = num_q_heads;
  if (with_k) {
    p.k = static_cast<const uint16_t *>(k_bf16);
    p.k_out = k_out_bf16;
    p.kv_heads = num_k_heads;
  }
  p.positions = d_positions;
  p.tokens = static_cast<int32_t>(tokens);
  return launch_rows(p, false, FFD_CACHE_BF16, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? FFD_OK
                                                                                                     : FFD_ERR_CUDA;
}

ffd_status ffd_append_tokens(const ffd_shape *s, const ffd_cache *c, const ffd_rope *rope, int32_t new_tokens,
                             const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16,
                             const int32_t *d_positions, const int32_t *d_lengths, const int32_t *d_new_lengths,
                             void *q_out_bf16, void *cuda_stream) {
  ffd_status st = check_shape(s);
  if (st != FFD_OK) return st;
  if (new_tokens < 0 || (rope != nullptr && !rope_ok(rope))) return FFD_ERR_INVALID_ARG;
  if ((q_bf16 == nullptr) != (q_out_bf16 == nullptr)) return FFD_ERR_INVALID_ARG;
  if (new_tokens > s->capacity) return FFD_ERR_INVALID_ARG;
  if (s->batch == 0 || new_tokens == 0) return FFD_OK;
  st = check_cache(c);
  if (st != FFD_OK) return st;
  if (k_new_bf16 == nullptr || v_new_bf16 == nullptr || d_lengths == nullptr || !aligned16(k_new_bf16) ||
      !aligned16(v_new_bf16) || !aligned16(q_bf16) || !aligned16(q_out_bf16) || !aligned4(d_lengths) ||
      !aligned4(d_new_lengths) || !aligned4(d_positions))
    return FFD_ERR_INVALID_ARG;
  const bool byte = c->format == FFD_CACHE_BYTE;
  const size_t tokens = static_cast<size_t>(s->batch) * new_tokens;
  const size_t rows = static_cast<size_t>(s->batch) * s->num_kv_heads * s->capacity;
  const Range in[6] = {{q_bf16, tokens * s->num_q_heads * kHeadDim * 2},
                       {k_new_bf16, tokens * s->num_kv_heads * kHeadDim * 2},
                       {v_new_bf16, tokens * s->num_kv_heads * kHeadDim * 2},
                       {d_positions, tokens * 4},
                       {d_lengths, static_cast<size_t>(s->batch) * 4},
                       {d_new_lengths, static_cast<size_t>(s->batch) * 4}};
  const Range out[5] = {{q_out_bf16, in[0].bytes},
                        {c->k, rows * (byte ? kByteRow : 2 * kHeadDim)},
                        {c->v, rows * (byte ? kByteRow : 2 * kHeadDim)},
                        {byte ? c->k_scales : nullptr, rows * 2},
                        {byte ? c->v_scales : nullptr, rows * 2}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 6; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j == 0 && out[0].p == in[0].p)) return FFD_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return FFD_ERR_INVALID_ARG;
  }
  RowsParams p{};
  set_rope(&p, rope, false);
  p.q = static_cast<const uint16_t *>(q_bf16);
  p.q_out = static_cast<uint16_t *>(q_out_bf16);
  p.k = static_cast<const uint16_t *>(k_new_bf16);
  p.v = static_cast<const uint16_t *>(v_new_bf16);
  p.k_out = c->k;
  p.v_out = c->v;
  p.k_scales = static_cast<uint16_t *>(c->k_scales);
  p.v_scales = static_cast<uint16_t *>(c->v_scales);
  p.positions = d_positions;
  p.lengths = d_lengths;
  p.counts = d_new_lengths;
  p.tokens = static_cast<int32_t>(tokens);  // at most batch * capacity, below 2^31 (check_shape)
  p.q_heads = s->num_q_heads;
  p.kv_heads = s->num_kv_heads;
  p.new_tokens = new_tokens;
  p.capacity = s->capacity;
  return launch_rows(p, true, c->format, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? FFD_OK
                                                                                               : FFD_ERR_CUDA;
}

ffd_status ffd_read_cache(const ffd_shape *s, const ffd_cache *c, const int32_t *d_lengths, int32_t token_begin,
                          int32_t token_count, void *k_out_bf16, void *v_out_bf16, void *cuda_stream) {
  ffd_status st = check_shape(s);
  if (st != FFD_OK) return st;
  if (token_begin < 0 || token_count < 0 || token_begin > s->capacity || token_count > s->capacity - token_begin)
    return FFD_ERR_INVALID_ARG;
  if (s->batch == 0 || token_count == 0) return FFD_OK;
  st = check_cache(c);
  if (st != FFD_OK) return st;
  if (c->format != FFD_CACHE_BYTE) return FFD_ERR_INVALID_ARG;
  if (d_lengths == nullptr || !aligned4(d_lengths) || (k_out_bf16 == nullptr && v_out_bf16 == nullptr) ||
      !aligned16(k_out_bf16) || !aligned16(v_out_bf16))
    return FFD_ERR_INVALID_ARG;
  const size_t bh = static_cast<size_t>(s->batch) * s->num_kv_heads, rows = bh * s->capacity;
  const size_t out_bytes = bh * token_count * kHeadDim * 2;
  const Range out[2] = {{k_out_bf16, out_bytes}, {v_out_bf16, out_bytes}};
  const Range in[5] = {{c->k, rows * kByteRow}, {c->v, rows * kByteRow}, {c->k_scales, rows * 2},
                       {c->v_scales, rows * 2}, {d_lengths, static_cast<size_t>(s->batch) * 4}};
  for (const Range &o : out)
    for (const Range &i : in)
      if (overlap(o, i)) return FFD_ERR_INVALID_ARG;
  if (overlap(out[0], out[1])) return FFD_ERR_INVALID_ARG;
  ReadParams p{};
  p.codes[0] = static_cast<const uint8_t *>(c->k);
  p.codes[1] = static_cast<const uint8_t *>(c->v);
  p.scales[0] = static_cast<const uint16_t *>(c->k_scales);
  p.scales[1] = static_cast<const uint16_t *>(c->v_scales);
  p.out[0] = static_cast<uint16_t *>(k_out_bf16);
  p.out[1] = static_cast<uint16_t *>(v_out_bf16);
  p.lengths = d_lengths;
  p.batch = s->batch;
  p.kv_heads = s->num_kv_heads;
  p.capacity = s->capacity;
  p.begin = token_begin;
  p.count = token_count;
  return launch_read(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? FFD_OK : FFD_ERR_CUDA;
}

#ifdef FFD_DEBUG
// Debug library only (not in the public header): the limit of the following calls'
// waits.
void ffd_debug_tree_wait_limit(uint64_t ns) { g_wait_limit_ns = ns; }
#endif

size_t ffd_decode_tree_workspace_bytes(const ffd_shape *s, int32_t num_nodes) {
  if (check_shape(s) != FFD_OK || num_nodes < 1 || num_nodes > FFD_MAX_TREE_NODES) return 0;
  return tree_layout(s->batch, s->num_kv_heads, s->num_q_heads / s->num_kv_heads, num_nodes, s->capacity).total;
}

ffd_status ffd_decode_tree_workspace_init(const ffd_shape *s, int32_t num_nodes, void *workspace,
                                          size_t workspace_bytes, void *cuda_stream) {
  const ffd_status st = check_shape(s);
  if (st != FFD_OK) return st;
  if (num_nodes < 1 || num_nodes > FFD_MAX_TREE_NODES) return FFD_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < ffd_decode_tree_workspace_bytes(s, num_nodes))
    return FFD_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FFD_ERR_INVALID_ARG;
  return cudaMemsetAsync(workspace, 0, kErrBytes, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? FFD_OK
                                                                                                       : FFD_ERR_CUDA;
}

ffd_status ffd_decode_tree(const ffd_shape *s, const ffd_cache *c, int32_t num_nodes, const void *q_bf16,
                           const int32_t *d_lengths, const int32_t *d_tree_sizes, const uint64_t *d_tree_mask,
                           void *out_bf16, void *workspace, size_t workspace_bytes, void *cuda_stream) {
  ffd_status st = check_shape(s);
  if (st != FFD_OK) return st;
  if (num_nodes < 1 || num_nodes > FFD_MAX_TREE_NODES) return FFD_ERR_INVALID_ARG;
  if (s->batch == 0) return FFD_OK;
  // one block of the merge a row
  if (static_cast<int64_t>(s->batch) * num_nodes * s->num_q_heads >= (int64_t{1} << 31)) return FFD_ERR_UNSUPPORTED;
  const int group = s->num_q_heads / s->num_kv_heads;
  const TreeLayout L = tree_layout(s->batch, s->num_kv_heads, group, num_nodes, s->capacity);
  if (workspace == nullptr || workspace_bytes < L.total) return FFD_ERR_WORKSPACE;
  if (s->capacity > 0) {
    st = check_cache(c);
    if (st != FFD_OK) return st;
  } else if (c == nullptr || c->reserved != 0 || (c->format != FFD_CACHE_BF16 && c->format != FFD_CACHE_BYTE)) {
    return FFD_ERR_INVALID_ARG;
  }
  if (q_bf16 == nullptr || d_lengths == nullptr || out_bf16 == nullptr || !aligned16(q_bf16) ||
      !aligned16(out_bf16) || !aligned16(workspace) || !aligned4(d_lengths) || !aligned4(d_tree_sizes) ||
      (reinterpret_cast<uintptr_t>(d_tree_mask) & 7u) != 0)
    return FFD_ERR_INVALID_ARG;
  const bool byte = c->format == FFD_CACHE_BYTE;
  const size_t nodes = static_cast<size_t>(s->batch) * num_nodes;
  const size_t rows = static_cast<size_t>(s->batch) * s->num_kv_heads * s->capacity;
  const size_t io = nodes * s->num_q_heads * kHeadDim * 2, row_bytes = byte ? kByteRow : 2 * kHeadDim;
  const Range out[2] = {{out_bf16, io}, {workspace, L.total}};
  const Range in[8] = {{q_bf16, io}, {c->k, rows * row_bytes}, {c->v, rows * row_bytes},
                       {byte ? c->k_scales : nullptr, rows * 2}, {byte ? c->v_scales : nullptr, rows * 2},
                       {d_lengths, static_cast<size_t>(s->batch) * 4},
                       {d_tree_sizes, static_cast<size_t>(s->batch) * 4}, {d_tree_mask, nodes * 8}};
  for (const Range &o : out)
    for (const Range &i : in)
      if (overlap(o, i)) return FFD_ERR_INVALID_ARG;
  if (overlap(out[0], out[1])) return FFD_ERR_INVALID_ARG;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  TreeParams p{};
  p.q = static_cast<const uint16_t *>(q_bf16);
  p.k = static_cast<const uint8_t *>(c->k);
  p.v = static_cast<const uint8_t *>(c->v);
  p.k_scales = static_cast<const uint16_t *>(c->k_scales);
  p.v_scales = static_cast<const uint16_t *>(c->v_scales);
  p.lengths = d_lengths;
  p.sizes = d_tree_sizes;
  p.mask = d_tree_mask;
  p.out = static_cast<uint16_t *>(out_bf16);
  p.err = reinterpret_cast<uint32_t *>(ws);
  p.table = reinterpret_cast<int2 *>(ws + L.table);
  p.partials = reinterpret_cast<float *>(ws + L.partials);
  p.units_a_head = L.units_a_head;
  p.rows = L.rows;
  p.ctas = L.ctas;
  p.batch = s->batch;
  p.kv_heads = s->num_kv_heads;
  p.group_log2 = group == 8 ? 3 : group == 4 ? 2 : group == 2 ? 1 : 0;
  p.nodes = num_nodes;
  p.capacity = s->capacity;
  p.format = c->format;
  p.wait_limit_ns = g_wait_limit_ns;
  return launch_tree(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? FFD_OK : FFD_ERR_CUDA;
}

}  // extern "C"
