// tree_narrow.cu -- drafted-token attention with up to 16 query rows a kv-head.
//
// Tokens are the 128 lanes of an accumulator and query rows its columns, S^T =
// K Q^T and O^T += V^T P^T: a matrix instruction's time goes with its columns,
// so few rows cost little (with rows as lanes 128 of them are paid for), and a
// thread has one token, whose scale and visibility it keeps in registers.  The
// weights' reference m of a row is the same for all tokens; whether any score
// passes it is one vote a tile, and only then are maxima taken over the lanes.
//
// e4m3: the two parts of a query row are two columns' worth of S^T, added in
// fp32, and those of a weight two columns of O^T, added at the end: K and V
// pass through the tensor cores once.
//
// Groups of 128 threads take the tiles in turn, with an S and an O each.
//
// One token of 4 sequences x 32K over e4m3 (4 rows): 62 us, 4.4 TB/s, where the
// kernel with rows as lanes took 80.  48 of them are the tiles, 64 in each of the 128
// CTAs that the 32 units are cut for, at 0.75 us (1340 clocks, 5.7 TB/s); start, parts
// and merge take the others.  With 32 and 64 rows this form was slower than the other
// (190 us where it took 146: every weight of every column passes one thread's
// arithmetic).
#include <atomic>

#include "ffd_tree.cuh"

namespace ffd {
namespace {

constexpr int kGroup = 128;      // threads of a group
constexpr int kRowBytes = 32;     // of a token's weights: 16 rows in bf16, or two e4m3 parts
constexpr int kSmemMax = 232448;
// second parts of query rows are kept times 2^4, those of weights times 2^3
constexpr int kQLo = 4, kWLo = 3;
constexpr float kNever = -3.0e38f;  // the reference of a row that has seen nothing

constexpr int kRows = 16;

template <bool kByte>
struct Narrow {
  // More groups hide more of a tile's latency, which a tile of bf16, twice as
  // long in coming, hides with two.  A K that waits for its turn behind kGroups
  // V's must find a slot: 2 kGroups of them at least.
  static constexpr int kGroups = kByte ? 4 : 2;
  static constexpr int kThreads = (kGroups + 1) * kGroup;   // the last four warps copy and multiply
  static constexpr int kN = kByte ? 2 * kRows : kRows;      // columns of S and O
  static constexpr int kTmem = kByte ? 256 : 128;
  static constexpr int kSlot = kByte ? 16384 : 32768;       // bytes of K or V of a tile
  static constexpr int kQ = 4096;                           // the query rows
  static constexpr int kWeights = kQ;                       // [group][128 tokens][kRowBytes]
  static constexpr int kRing = kWeights + kGroups * 128 * kRowBytes;
  static constexpr int kSlots = kByte ? 10 : 6;
  static constexpr int kScales = kRing + kSlots * kSlot;    // [slot][128] bf16
  static constexpr int kRef = kScales + (kByte ? kSlots * 256 : 0);  // [group][kRows] m
  static constexpr int kFade = kRef + kGroups * kRows * 4;  // [group][kRows]
  static constexpr int kWarpRow = kFade + kGroups * kRows * 4;  // [group][4 warps][kRows]
  static constexpr int kSeen = kWarpRow + kGroups * 4 * kRows * 4;  // [kRows]
  static constexpr int kTot = kSeen + kRows * 8;            // [kRows] (m, sum); before, scales of the query rows
  static constexpr int kBars = kTot + kRows * 8;
  static constexpr int kNumBars = 2 * kSlots + 3 * kGroups + 2;
  static constexpr int kWords = kBars + kNumBars * 8;
  static constexpr int kTotal = kWords + 32 + sizeof(Waits);
  static_assert(kTotal <= kSmemMax, "shared memory");
  // (even: a slot then holds K's only or V's only, as `idle` below needs)
  static_assert(kSlots >= 2 * kGroups && kSlots % 2 == 0, "the ring would stop");
  static_assert(kRing % 1024 == 0 && 2 * kGroups * kN <= kTmem, "layout");
};

// For each of 16 rows the 32 lanes' v[row] joined (sum, or largest): lane t has
// row t / 2, in v[0].
template <bool kMax>
__device__ __forceinline__ void join_lanes(float *v, int lane) {
  auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int n = 8; n > 0; n >>= 1) {
    const bool up = lane & (2 * n);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = join(keep, __shfl_xor_sync(0xFFFFFFFFu, send, 2 * n));
    }
  }
  v[0] = join(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
}

template <bool kByte>
__global__ void __launch_bounds__(Narrow<kByte>::kThreads, 1)
    tree_narrow_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const TreeParams p) {
  using L = Narrow<kByte>;
  constexpr int kGroups = L::kGroups, kN = L::kN, kSlots = L::kSlots;
  constexpr int kSteps = kByte ? 4 : 8;  // matrix instructions of a product
  constexpr uint32_t kIdescS = instr_desc(kByte ? 0 : 1, kN, false, false);
  constexpr uint32_t kIdescO = instr_desc(kByte ? 0 : 1, kN, true, true);
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *full = bars, *empty = bars + kSlots, *bar_s = empty + kSlots, *bar_p = bar_s + kGroups,
           *bar_f = bar_p + kGroups, *bar_q = bar_f + kGroups, *bar_end = bar_q + 1;
  float *ref_s = reinterpret_cast<float *>(smem + L::kRef);
  float *fade_s = reinterpret_cast<float *>(smem + L::kFade);
  float *warp_row_s = reinterpret_cast<float *>(smem + L::kWarpRow);
  float2 *tot_s = reinterpret_cast<float2 *>(smem + L::kTot);
  float *row_scale_s = reinterpret_cast<float *>(tot_s);  // of the query rows, until a segment's end (e4m3)
  uint64_t *seen_s = reinterpret_cast<uint64_t *>(smem + L::kSeen);
  Waits *waits = reinterpret_cast<Waits *>(smem + L::kWords + 32);
  volatile int *words = reinterpret_cast<volatile int *>(smem + L::kWords);
  volatile int *odd = words + 1;       // a value in a drafted token's row is not finite
  int *start_s = const_cast<int *>(words) + 2;  // b, offset, tiles, all tiles
  constexpr int kMatrixWarp = kGroups * kGroup / 32, kCopyWarp = kMatrixWarp + 1;

  if (warp == kMatrixWarp) tmem_alloc(reinterpret_cast<uint32_t *>(smem + L::kWords), L::kTmem);
  if (tid == kCopyWarp * 32) {  // (warp 0 divides the work meanwhile)
    for (int i = 0; i < 2 * kSlots; ++i) mbar_init(bars + i, 1);
    for (int s = 0; s < kGroups; ++s) {
      mbar_init(bar_s + s, 1);
      mbar_init(bar_p + s, kGroup);
      mbar_init(bar_f + s, 1);
    }
    mbar_init(bar_q, kGroups * kGroup);
    mbar_init(bar_end, 1);
    fence_mbar_init();
    waits->dead = 0;
    waits->err = p.err;
    waits->limit_ns = p.wait_limit_ns;
    *odd = 0;
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  // (nothing of the stream's earlier work is read or written before this; the
  // merge may start then, and reads lengths and sizes at once)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  find_part<L::kThreads>(p, reinterpret_cast<int *>(warp_row_s), start_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(words[0]);
  Walk walk{start_s[0], start_s[1], start_s[2]};
  Segment g;

  // A warp's answer to its lanes' waits: the same in every lane, which stand
  // together again (they leave a wait one by one, and elect_one and the
  // instructions under it are for a converged warp).
  auto all = [](bool b) { return __all_sync(0xFFFFFFFFu, b) != 0; };
  bool alive = true;  // no wait of this thread was given up
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (alive && !mbar_wait_short<kAttempts>(bar, parity)) alive = wait_on(bar, parity, waits);
    return alive;
  };

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------- copies --
    // (the whole warp walks and waits, one lane issues)
    uint32_t i = 0;  // K of tile n is copy 2n, V copy 2n + 1
    while (alive && walk.next(p, g)) {
      const int bh = g.b * p.kv_heads + g.unit;
      for (int j = 0; alive && j < 2 * g.tiles; ++j, ++i) {
        const uint32_t slot = i % kSlots, round = i / kSlots;
        // (a slot given back by a thread that waits no more may still be filling)
        if (round > 0) alive = all(wait(empty + slot, (round - 1) & 1) && waits->dead == 0);
        if (!alive) break;
        const int t0 = (g.tile0 + (j >> 1)) * kTile;
        const int row = bh * p.capacity + t0;
        uint64_t *landed = full + slot;
        uint8_t *dst = smem + L::kRing + slot * L::kSlot;
        const void *map = (j & 1) ? &tmap_v : &tmap_k;
        if (!elect_one()) continue;
        if constexpr (kByte) {
          // (each copy brings its scales)
          const uint32_t scale_bytes = 2u * static_cast<uint32_t>(min(kTile, p.capacity - t0));
          mbar_arrive_expect_tx(landed, L::kSlot + scale_bytes);
          tma_load_2d(dst, map, 0, row, landed);
          bulk_g2s(smem + L::kScales + slot * 256, ((j & 1) ? p.v_scales : p.k_scales) + row, scale_bytes, landed);
        } else {
          mbar_arrive_expect_tx(landed, L::kSlot);
          tma_load_3d(dst, map, 0, row, 0, landed);
        }
      }
    }
    __syncwarp();
    // what is in flight lands before the CTA ends, whoever gave up
    for (uint32_t s = 0; s < static_cast<uint32_t>(kSlots) && s < i; ++s)
      mbar_wait(full + s, ((i - 1 - s) / kSlots) & 1, kWaitLimitNs);
  } else if (warp == kMatrixWarp) {
    // ------------------------------------------------------------ matrices --
    // Tile i of a segment is group i % kGroups'.  S of a tile goes out when its K
    // is there and the group has read its last S, O += of one when V and the
    // weights are there, whichever is first: neither holds up the other's slot.
    // A commit holds the thread until what the last one stands for is done, and
    // until the next issue the tensor cores stand still: so the commits come last,
    // and four lanes ask the four barriers at once.
    uint32_t n = 0, segments = 0, p_phases = 0, f_phases = (1u << kGroups) - 1u;
    // (lane 0's copy: known to be the same in every lane, such values stay in
    // uniform registers)
    auto uniform = [](uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
    const uint32_t q = uniform(smem_addr(smem)), ring = q + L::kRing, tm = uniform(tmem);
    while (alive && walk.next(p, g)) {
      alive = all(wait(bar_q, segments & 1));
      ++segments;
      int si = 0, oi = 0;  // tiles whose S, whose O have gone out
      uint32_t spin = 0;
      uint64_t since = 0;
#pragma unroll 1
      while (alive && oi < g.tiles) {
        const uint32_t sg = uniform(si % kGroups), og = uniform(oi % kGroups);
        const uint32_t ka = 2 * (n + si), va = 2 * (n + oi) + 1;
        const uint32_t k_slot = uniform(ka % kSlots), v_slot = uniform(va % kSlots);
        uint64_t *bar = (lane & 2) ? ((lane & 1) ? bar_p + og : full + v_slot) : ((lane & 1) ? bar_f + sg : full + k_slot);
        const uint32_t parity = (lane & 2) ? ((lane & 1) ? p_phases >> og : va / kSlots) : ((lane & 1) ? f_phases >> sg : ka / kSlots);
        const uint32_t yes = __ballot_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity & 1));
        __syncwarp();  // (what the asking lanes have seen, the issuing one has)
        const bool do_s = (yes & 3u) == 3u && si < g.tiles, do_o = (yes & 12u) == 12u && oi < si;
        if (!do_s && !do_o) {
          if ((++spin & (kAttempts - 1)) != 0) continue;
          if (spin == kAttempts) since = global_timer_ns();
          alive = all(keep_waiting(waits, since));
          continue;
        }
        spin = 0;
        tc_fence_after();
        const uint32_t add = uniform(oi < kGroups ? 0 : 1), v = ring + v_slot * L::kSlot, k = ring + k_slot * L::kSlot;
        const uint32_t o = tm + (kGroups + og) * kN, w = q + L::kWeights + og * 128 * kRowBytes, d = tm + sg * kN;
        if (elect_one()) {
          if (do_o) {
#pragma unroll
            for (int c = 0; c < kSteps; ++c)  // bf16: 16 tokens a step; e4m3: 32
              mma_ss<kByte>(o, smem_desc(v + c * (kByte ? 4096 : 2048), 16384),
                            smem_desc<kRowBytes>(w + c * (kByte ? 32 : 16) * kRowBytes), kIdescO, c > 0 || add != 0);
          }
          if (do_s) {
#pragma unroll
            for (int c = 0; c < kSteps; ++c)  // bf16: 16 channels a step, four a 128-byte half; e4m3: 32
              mma_ss<kByte>(d, smem_desc(k + (c >> 2) * 16384 + (c & 3) * 32),
                            smem_desc(q + (c >> 2) * kN * 128 + (c & 3) * 32), kIdescS, c > 0);
            mma_commit(bar_s + sg);
          }
          if (do_o) mma_commit(empty + v_slot);
        }
        if (do_o) {
          p_phases ^= 1u << og;
          ++oi;
        }
        if (do_s) {
          f_phases ^= 1u << sg;
          ++si;
        }
        __syncwarp();
      }
      n += g.tiles;
    }
    // what was issued is done before tensor memory is given back, whoever gave up
    if (elect_one()) mma_commit(bar_end);
    __syncwarp();
    mbar_wait(bar_end, 0, kWaitLimitNs);
  } else if (warp < kMatrixWarp) {
    // ------------------------------------------------------------- softmax --
    const int s = warp >> 2, w = warp & 3;       // group; which 32 lanes of an accumulator
    const int t = tid & 127;                     // token of a tile; channel of O
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const uint32_t tm_s = tmem + lanes + s * kN, tm_o = tmem + lanes + (kGroups + s) * kN;
    const uint32_t bar_group = 1 + s, bar_all = 5;
    float *ref = ref_s + s * kRows;
    float *fade = fade_s + s * kRows;
    // The weights of a group are read and its O is idle when V's slot is empty
    // again.  (The slot's next V belongs to a later tile, whose product comes
    // after the one that this group has still to ask for.)
    auto idle = [&](uint32_t v) { return wait(empty + v % kSlots, (v / kSlots) & 1); };
    uint32_t last_v = 0;                         // copy of V of the group's last tile
    uint32_t count = 0, n = 0;                   // tiles of this group so far; of the CTA
    bool starts = true;                          // the CTA's first segment
    while (walk.next(p, g)) {
      const int head = g.unit;
      const int first = g.len - g.size;
      const int bh = g.b * p.kv_heads + head;
      // ---- the query rows: 16 threads a row, all loads before the first use ----
      // e4m3: each row is scaled by a power of two, its largest magnitude into [128, 256).
      {
        const int c = tid & 15, r = tid >> 4, i = r >> p.group_log2;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < kRows && i < g.size)
          x = __ldg(reinterpret_cast<const uint4 *>(
                        p.q + (((static_cast<size_t>(g.b) * p.nodes + i) * p.kv_heads + head) << p.group_log2) * kHeadDim +
                        (r & ((1 << p.group_log2) - 1)) * kHeadDim) + c);
        if (tid < kRows) seen_s[tid] = seen_nodes(p, g, tid >> p.group_log2);
        if (tid < kGroups * kRows) ref_s[tid] = kNever;
        if constexpr (kByte) {
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(v[e] & 0x7FFFu, (v[e] >> 16) & 0x7FFFu));
#pragma unroll
          for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
          const int exponent = top == 0 ? 0 : min(100, 134 - static_cast<int>(top >> 7));
          const float by = __uint_as_float(static_cast<uint32_t>(127 + exponent) << 23);
          const float down = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            split4_signed<kQLo>(bf16_f(v[2 * e] & 0xFFFFu) * by, __uint_as_float(v[2 * e] & 0xFFFF0000u) * by,
                                bf16_f(v[2 * e + 1] & 0xFFFFu) * by, __uint_as_float(v[2 * e + 1] & 0xFFFF0000u) * by, hi[e], lo[e]);
          if (r < kRows) {  // first parts are rows 0 on, second parts kRows on
            uint8_t *dst = smem + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
            *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(dst + kRows * 128) = make_uint2(lo[0], lo[1]);
            // (an infinity spoils its row)
            if (c == 0) row_scale_s[r] = top < 0x7F80u ? kScoreScale * down : __uint_as_float(0x7FFFFFFFu);
          }
        } else {
          *reinterpret_cast<uint4 *>(smem + r * 128 + (c >> 3) * kRows * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bar_q);
      named_barrier(bar_all, kGroups * kGroup);

      // ---- the tiles ----
      float l[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) l[r] = 0.0f;
      uint32_t here = 0;                         // of this segment's
      for (int j = s; j < g.tiles; j += kGroups, ++here) {
        const int t0 = (g.tile0 + j) * kTile, token = t0 + t;
        const bool masked = t0 + kTile > first;
        const uint32_t vi = 2 * (n + j) + 1, v_slot = vi % kSlots, k_slot = (vi - 1) % kSlots;
        float ks = kScoreScale, vs = 1.0f, lv = 0.0f;
        if constexpr (kByte) {
          wait(full + k_slot, ((vi - 1) / kSlots) & 1);
          ks = bf16_f(reinterpret_cast<const uint16_t *>(smem + L::kScales + k_slot * 256)[t]);
        }
        wait(bar_s + s, count & 1);
        tc_fence_after();
        if constexpr (kByte) {
          wait(full + v_slot, (vi / kSlots) & 1);
          vs = bf16_f(reinterpret_cast<const uint16_t *>(smem + L::kScales + v_slot * 256)[t]);
          if (masked && token >= first) {
            // (a weight of zero must not meet a scale that is not finite: as for values, below)
            if (token >= g.len) {
              vs = 0.0f;
            } else if (!(fabsf(vs) < INFINITY)) {
              vs = 0.0f;
              *odd = 1;
            }
          }
          lv = __log2f(fabsf(vs));
          lv = lv < -60.0f ? -60.0f : lv;  // (a zero scale: far below any other, but not infinitely far)
        }
        // the token's scores, in units of log 2, above m of `below`
        auto load = [&](float *x, auto below) {
          tmem_ld<16>(tm_s, x);
          if constexpr (kByte) {
            float x2[16];
            tmem_ld<16>(tm_s + kRows, x2);
            tmem_wait_ld<16>(x);
            tmem_wait_ld<16, false>(x2);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = fmaf(x2[e], 1.0f / (1 << kQLo), x[e]);
          } else {
            tmem_wait_ld<16>(x);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 m = below(e);
            if constexpr (kByte) {
              const float4 rs = *reinterpret_cast<const float4 *>(row_scale_s + e);
              x[e] = fmaf(x[e] * ks, rs.x, -m.x);
              x[e + 1] = fmaf(x[e + 1] * ks, rs.y, -m.y);
              x[e + 2] = fmaf(x[e + 2] * ks, rs.z, -m.z);
              x[e + 3] = fmaf(x[e + 3] * ks, rs.w, -m.w);
            } else {
              x[e] = fmaf(x[e], ks, -m.x);
              x[e + 1] = fmaf(x[e + 1], ks, -m.y);
              x[e + 2] = fmaf(x[e + 2], ks, -m.z);
              x[e + 3] = fmaf(x[e + 3], ks, -m.w);
            }
          }
          if (masked && token >= first) {
            const int at = token - first;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (at >= 64 || !((seen_s[e] >> (at & 63)) & 1ull)) x[e] = -INFINITY;
          }
        };
        auto above_m = [&](int r) { return *reinterpret_cast<const float4 *>(ref + r); };
        // The reference m of a row moves only when weights would leave their
        // range: in bf16 past 2^8; in e4m3 past 448 (2^8.8), from 2^4 at the last
        // move, so that small weights keep their bits.
        constexpr float kRoom = kByte ? 8.8f : 8.0f, kAbove = kByte ? 4.0f : 0.0f;
        float z[kRows], top = -INFINITY;
        load(z, above_m);
#pragma unroll
        for (int r = 0; r < kRows; ++r) top = fmaxf(top, z[r]);
        if (here > 0) idle(last_v);
        last_v = vi;
        tc_fence_before();
        const bool move = named_barrier_any(bar_group, kGroup, top > kRoom - lv);
        const bool speaks = (tid & (kGroup - 1)) == 0;
        if (speaks) mbar_arrive(empty + k_slot);  // K and its scales are read
        if (move) {
          float v[kRows];
          load(v, [&](int) { return make_float4(-lv, -lv, -lv, -lv); });
          join_lanes<true>(v, lane);
          if ((lane & 1) == 0) warp_row_s[(4 * s + w) * kRows + (lane >> 1)] = v[0];
          named_barrier(bar_group, kGroup);
          const int r = tid & (kGroup - 1);
          if (r < kRows) {
            const float *of = warp_row_s + 4 * s * kRows + r;
            const float high = fmaxf(fmaxf(of[0], of[kRows]), fmaxf(of[2 * kRows], of[3 * kRows]));
            const float m = ref[r], next = high > m + kRoom ? in_range<kByte>(high - kAbove) : m;
            ref[r] = next;
            fade[r] = next == m ? 1.0f : exp2_f(m - next);
          }
          named_barrier(bar_group, kGroup);
          load(z, above_m);
#pragma unroll
          for (int e = 0; e < kRows; ++e) l[e] *= fade[e];
          if (here > 0) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kN; c += kRows) {
              float o[kRows];
              tmem_ld<kRows>(tm_o + c, o);
              tmem_wait_ld<kRows>(o);
#pragma unroll
              for (int e = 0; e < kRows; ++e) o[e] *= fade[e];
              tmem_st<kRows>(tm_o + c, reinterpret_cast<const uint32_t *>(o));
            }
            tmem_wait_st();
          }
          tc_fence_before();
          named_barrier(bar_group, kGroup);
        }
        if (speaks) mbar_arrive(bar_f + s);  // S is read
        // ---- weights ----
        uint8_t *mine = smem + L::kWeights + (s * 128 + t) * kRowBytes;
        // 16-byte vector c of a token's row under the swizzle of its span
        auto swizzle = [&](int c) { return (c ^ ((t >> 2) & 1)) << 4; };
#pragma unroll
        for (int r = 0; r < kRows; r += kByte ? 16 : 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < (kByte ? 16 : 8); e += 4) {
            const float p0 = exp2_f(z[r + e]), p1 = exp2_f(z[r + e + 1]);
            const float p2 = exp2_f(z[r + e + 2]), p3 = exp2_f(z[r + e + 3]);
            l[r + e] += p0;
            l[r + e + 1] += p1;
            l[r + e + 2] += p2;
            l[r + e + 3] += p3;
            if constexpr (kByte) {
              split4<kWLo>(p0 * vs, p1 * vs, p2 * vs, p3 * vs, hi[e >> 2], lo[e >> 2]);
            } else {
              hi[e >> 1] = pack_bf16(p0, p1);
              hi[(e >> 1) + 1] = pack_bf16(p2, p3);
            }
          }
          if constexpr (kByte) {
            *reinterpret_cast<uint4 *>(mine + swizzle(0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(mine + swizzle(1)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
            *reinterpret_cast<uint4 *>(mine + swizzle(r >> 3)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          }
        }
        if (masked) {
          wait(full + v_slot, (vi / kSlots) & 1);
          if (token >= first &&
              clean_values<kByte>(smem + L::kRing + v_slot * L::kSlot, t, token >= g.len, 0, kByte ? 8 : 16))
            *odd = 1;
        }
        ++count;
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar_p + s);
      }
      n += g.tiles;

      // ---- the end of a segment: the groups' sums and O together ----
      if (here > 0) idle(last_v);
      join_lanes<false>(l, lane);
      if ((lane & 1) == 0) warp_row_s[(4 * s + w) * kRows + (lane >> 1)] = l[0];
      tc_fence_after();
      named_barrier(bar_all, kGroups * kGroup);
      const bool whole = g.tiles == g.all;
      const bool any_odd = *odd != 0;
      const int used = min(g.tiles, kGroups);  // groups that have an O
      if (tid < kRows) {  // a row's reference and sum, and what its O's are multiplied with
        float m = kNever, sum = 0.0f;
        for (int u = 0; u < used; ++u) m = fmaxf(m, ref_s[u * kRows + tid]);
        for (int u = 0; u < used; ++u) {
          const float *of = warp_row_s + 4 * u * kRows + tid;
          const float f = exp2_f(ref_s[u * kRows + tid] - m);
          fade_s[u * kRows + tid] = f;
          sum += ((of[0] + of[kRows]) + (of[2 * kRows] + of[3 * kRows])) * f;
        }
        tot_s[tid] = make_float2(m, sum);
        warp_row_s[tid] = 1.0f / sum;
      }
      named_barrier(bar_all, kGroups * kGroup);
      // four rows at a time, 32 channels a warp, one a lane
      constexpr int kMine = kRows / kGroups;
      float *part_out = p.partials + static_cast<size_t>(2 * blockIdx.x + (starts ? 0 : 1)) * part_floats(p.rows);
#pragma unroll 1
      for (int r0 = s * kMine; r0 < (s + 1) * kMine && (r0 >> p.group_log2) < g.size; r0 += 4) {
        float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int u = 0; u < used; ++u) {
          float v[4], v2[4];
          tmem_ld<4>(tmem + lanes + (kGroups + u) * kN + r0, v);
          if constexpr (kByte) tmem_ld<4>(tmem + lanes + (kGroups + u) * kN + kRows + r0, v2);
          tmem_wait_ld<4>(v);
          if constexpr (kByte) {
            tmem_wait_ld<4, false>(v2);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(v2[e], 1.0f / (1 << kWLo), v[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = fmaf(v[e], fade_s[u * kRows + r0 + e], o[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + e, i = r >> p.group_log2;
          if (i < g.size) {
            if (any_odd) o[e] += odd_values<kByte>(p, g, bh, seen_s[r], t);
            if (whole) {
              const float y = tot_s[r].y == 0.0f && o[e] == 0.0f ? 0.0f : o[e] * warp_row_s[r];
              p.out[((((static_cast<size_t>(g.b) * p.nodes + i) * p.kv_heads + head) << p.group_log2) +
                     (r & ((1 << p.group_log2) - 1))) * kHeadDim + t] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
            } else {
              part_out[part_vector(p.rows, r, t >> 2) + (t & 3)] = o[e];
              if (t == 0) *reinterpret_cast<float2 *>(part_out + part_sums(p.rows, r)) = tot_s[r];
            }
          }
        }
      }
      if (tid == 0 && g.tile0 == 0) note_unit(p, g, walk, start_s, starts);
      starts = false;
      tc_fence_before();
      named_barrier(bar_all, kGroups * kGroup);
      if (tid == 0) *odd = 0;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMatrixWarp) {
    tc_fence_after();
    tmem_free(tmem, L::kTmem);
  }
}

template <bool kByte>
cudaError_t launch_as(const TreeParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v, cudaStream_t stream) {
  using L = Narrow<kByte>;
  static std::atomic<uint64_t> configured{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(tree_narrow_kernel<kByte>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  return launch_early(tree_narrow_kernel<kByte>, p.ctas, L::kThreads, L::kTotal, stream, map_k, map_v, p);
}

}  // namespace

cudaError_t launch_tree_narrow(const TreeParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v,
                               cudaStream_t stream) {
  return p.format == FFD_CACHE_BYTE ? launch_as<true>(p, map_k, map_v, stream)
                                    : launch_as<false>(p, map_k, map_v, stream);
}

}  // namespace ffd
