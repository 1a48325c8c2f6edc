// tree.cu -- attention of drafted tokens over the cache (ffd_decode_tree).
//
// Query rows (node, head of the group) are the 128 lanes of a tensor-memory
// accumulator, tokens its columns: S = Q K^T, P = 2^(S c - m), O += P V, one
// pass over K and V with a running maximum m and sum l a row (fp32).  Few rows
// are replicated over the lanes, a copy for each part of the tile's tokens, so
// that every thread has work and no sum crosses lanes inside the pass.
//
// The work of a call is one list of 128-token tiles, (sequence, kv-head, rows)
// after another, cut into equal parts, one for each CTA: long sequences are
// split, short ones share a CTA, whatever the lengths are (or, see find_part,
// each unit into its own).  Parts of a unit are joined by merge_tree_kernel, in
// the order of the CTAs.
//
// A CTA: two groups of 128 softmax threads, one thread that issues the copies
// and one that issues the matrix instructions.  Up to 128 rows, the groups
// take alternate tiles with an accumulator each; more, they take 128 rows each
// of the same tiles.  Either way the tensor cores work for one group while the
// other does its exponentials.
//
// What bounds it.  A tile's time is the difference between 32 tiles a CTA and 8,
// every multiprocessor busy.  64 rows over bf16: 1.3 us (2200 clocks), 7.4 TB/s, the
// copies.  52 rows over e4m3 (13 nodes, group 4): 2250 clocks, where the bytes would
// take 1290 at the copies' rate; a group, which has every other tile, needs twice that
// for its chain of scales, maxima, exponentials and the split of each weight, and two
// products of each kind in turn with the other group's.  2 x 128 rows: 3600 a pair of
// tiles, of which the tensor cores work 2048, and 7900 over e4m3.  The rest of a call is
// its start, the parts and the merge: of 16 nodes over 128K tokens (104 us) 74 are
// the 56 tiles of a CTA, of 64 nodes over 3 sequences of up to 16K (58 us) 26 are its
// 14 pairs, of 13 nodes over 5 sequences of up to 64K in e4m3 (144 us) 95.  Up to 19
// MB of parts go out and come back, and a merge CTA starts for every row, also where
// no unit was cut (1.1 us a thousand).  One matrix warp for each group, as they please
// or under a lock, was slower (both groups fall into step: 74 and 69 us where one warp
// took 67), and so were two threads a row (95 us).
//
// bf16 cache: P has bf16's 8 significant bits.  8-bit cache: codes enter the
// matrix instructions as they are.  The query row, scaled by a power of two
// into e4m3's range, is the sum of two e4m3 parts (exact for channels down to
// 2^-9 of the row's largest, half of 2^-17 of it off below); the K row's scale
// multiplies the score in fp32; the V row's scale multiplies the weight, which
// is the sum of two e4m3 parts too: 8 significant bits, in units of 2^-16 of
// the largest weight so far, or finer.
#include <atomic>

#include "ffd_tree.cuh"

namespace ffd {
namespace {

constexpr int kGroup = 128;                  // threads of a softmax group
constexpr int kCtaThreads = 3 * kGroup;       // and four warps, of which one copies and one multiplies
constexpr int kSmemMax = 232448;
constexpr int kOutTile = 32768;               // bytes of a Q tile (bf16, or two e4m3 parts)

// ------------------------------------------------------------------ layout --

template <bool kByte, bool kPair>
struct Layout {
  static constexpr int kSlot = kByte ? 16384 : 32768;  // bytes of K or V of a tile
  static constexpr int kQ = (kPair ? 2 : 1) * kOutTile;
  static constexpr int kSlots = kByte ? (kPair ? 8 : 10) : (kPair ? 5 : 6);
  static constexpr int kRing = kQ;
  static constexpr int kScales = kRing + kSlots * kSlot;               // [slot][K, V][128] bf16
  static constexpr int kTokens = kScales + (kByte ? kSlots * 512 : 0);  // [group][2][3][128] fp32
  static constexpr int kRow = kTokens + (kByte ? 2 * 2 * 3 * 512 : 0);  // [2][128] float2
  static constexpr int kScale = kRow + 2 * kGroup * 8;                  // [2][128] fp32, of the query rows
  static constexpr int kBars = kScale + (kByte ? 2 * kGroup * 4 : 0);
  static constexpr int kNumBars = 2 * kSlots + 8;
  static constexpr int kWords = kBars + kNumBars * 8;
  static constexpr int kTotal = kWords + 32 + sizeof(Waits);
  static_assert(kTotal <= kSmemMax, "shared memory");
};

// --------------------------------------------------------------- the kernel --

template <bool kByte, int kCols, bool kPair>
__global__ void __launch_bounds__(kCtaThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                const __grid_constant__ CUtensorMap tmap_q, const TreeParams p) {
  using L = Layout<kByte, kPair>;
  constexpr int kRep = kTile / kCols;        // copies of a row
  constexpr int kRowsHere = kGroup / kRep;   // rows of an accumulator
  constexpr int kSlots = L::kSlots;
  constexpr uint32_t kIdescS = instr_desc(kByte ? 0 : 1, 128, false, false);
  constexpr uint32_t kIdescO = instr_desc(kByte ? 0 : 1, 128, false, true);
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5;
  float2 *row_s = reinterpret_cast<float2 *>(smem + L::kRow);
  float *scale_s = reinterpret_cast<float *>(smem + L::kScale);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *full = bars, *empty = bars + kSlots;
  uint64_t *bar_s = empty + kSlots, *bar_p = bar_s + 2, *bar_o = bar_s + 4, *bar_q = bar_s + 6;
  uint64_t *bar_end = bar_s + 7;
  Waits *waits = reinterpret_cast<Waits *>(smem + L::kWords + 32);
  volatile int *words = reinterpret_cast<volatile int *>(smem + L::kWords);
  // The last segment with a drafted token's value that is not finite.  (Not a flag
  // to be cleared: the groups go on to a next segment without waiting for each other.)
  volatile int *odd = words + 1;
  int *start_s = const_cast<int *>(words) + 2;  // b, offset, tiles, all tiles

  if (warp == 9) tmem_alloc(reinterpret_cast<uint32_t *>(smem + L::kWords), 512);
  if (tid == 8 * 32) {  // (warp 0 divides the work meanwhile)
    for (int i = 0; i < 2 * kSlots; ++i) mbar_init(bars + i, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_s + s, 1);
      mbar_init(bar_p + s, kGroup);
      mbar_init(bar_o + s, 1);
    }
    mbar_init(bar_q, kByte ? 2 * kGroup : 1);
    mbar_init(bar_end, 1);
    fence_mbar_init();
    waits->dead = 0;
    waits->err = p.err;
    waits->limit_ns = p.wait_limit_ns;
    *odd = 0;
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    if (!kByte) prefetch_tmap(&tmap_q);
  }
  // (nothing of the stream's earlier work is read or written before this; the
  // merge may start then, and reads lengths and sizes at once)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  find_part<kCtaThreads>(p, reinterpret_cast<int *>(row_s), start_s);
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

  // bf16: the query rows.  Rows past the tree are whatever lies there: no other
  // row's result has anything of them.
  auto load_query = [&](const Segment &g) {
    constexpr int kTiles = kPair ? 2 : 1;
    const int head = g.unit / p.units_a_head, row0 = (g.unit - head * p.units_a_head) * kTreeRows;
    mbar_arrive_expect_tx(bar_q, kTiles * kOutTile);
#pragma unroll
    for (int i = 0; i < 2 * kTiles * kRep; ++i) {
      const int q_tile = i / (2 * kRep), half = i & 1, copy = (i >> 1) % kRep;
      tma_load_4d(smem + q_tile * kOutTile + half * 16384 + copy * kRowsHere * 128, &tmap_q, half * 64, 0, head,
                  g.b * p.nodes + ((row0 + q_tile * kGroup) >> p.group_log2), bar_q);
    }
  };

  if (warp == 8) {
    // ------------------------------------------------------------- copies --
    // (the whole warp walks and waits, one lane issues)
    uint32_t i = 0;  // K of tile n is copy 2n, V copy 2n + 1
    while (alive && walk.next(p, g)) {
      if (!kByte && i == 0 && elect_one()) load_query(g);
      __syncwarp();
      const int bh = g.b * p.kv_heads + g.unit / p.units_a_head;
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
          const uint32_t scale_bytes = 2u * static_cast<uint32_t>(min(kTile, p.capacity - t0));
          mbar_arrive_expect_tx(landed, L::kSlot + ((j & 1) ? 2 * scale_bytes : 0));
          tma_load_2d(dst, map, 0, row, landed);
          if (j & 1) {
            bulk_g2s(smem + L::kScales + slot * 512, p.k_scales + row, scale_bytes, landed);
            bulk_g2s(smem + L::kScales + slot * 512 + 256, p.v_scales + row, scale_bytes, landed);
          }
        } else {
          mbar_arrive_expect_tx(landed, L::kSlot);
          tma_load_3d(dst, map, 0, row, 0, landed);
        }
      }
    }
    // what is in flight lands before the CTA ends, whoever gave up
    for (uint32_t s = 0; s < static_cast<uint32_t>(kSlots) && s < i; ++s)
      mbar_wait(full + s, ((i - 1 - s) / kSlots) & 1, kWaitLimitNs);
  } else if (warp == 9) {
    // ------------------------------------------------------------ matrices --
    // Item i of a segment is a tile's product pair for group i % 2.  S goes out
    // when its K is there and the group's O += of the item before, over whose
    // weights it is written, has gone out (products of a thread run in the order
    // of their issue), O += when V and the weights are there, whichever is first.
    // A commit holds the thread until what the last one stands for is done, and
    // until the next issue the tensor cores stand still: so the commits come last,
    // and lanes ask the barriers at once.
    uint32_t n = 0, segments = 0, p_phases = 0;
    // (lane 0's copy: known to be the same in every lane, such values stay in
    // uniform registers)
    auto uniform = [](uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
    const uint32_t q0 = uniform(smem_addr(smem)), ring = q0 + L::kRing, tm0 = uniform(tmem);
    const int lane = tid & 31;
    while (alive && walk.next(p, g)) {
      const int items = kPair ? 2 * g.tiles : g.tiles;
      alive = all(wait(bar_q, segments & 1));
      ++segments;
      int si = 0, oi = 0;  // items whose S, whose O have gone out
      uint32_t spin = 0;
      uint64_t since = 0;
#pragma unroll 1
      while (alive && oi < items) {
        const uint32_t sg = uniform(si & 1), og = uniform(oi & 1);
        const uint32_t ka = 2 * (n + (kPair ? si >> 1 : si)), va = 2 * (n + (kPair ? oi >> 1 : oi)) + 1;
        const uint32_t k_slot = uniform(ka % kSlots), v_slot = uniform(va % kSlots);
        uint64_t *bar = (lane & 1) ? full + v_slot : (lane & 2) ? bar_p + og : full + k_slot;
        const uint32_t parity = (lane & 1) ? va / kSlots : (lane & 2) ? p_phases >> og : ka / kSlots;
        const uint32_t yes = __ballot_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity & 1));
        __syncwarp();  // (what the asking lanes have seen, the issuing one has)
        const bool do_o = (yes & 6u) == 6u && oi < si;
        const bool do_s = (yes & 1u) != 0 && si < items && si < oi + (do_o ? 3 : 2);
        if (!do_s && !do_o) {
          if ((++spin & (kAttempts - 1)) != 0) continue;
          if (spin == kAttempts) since = global_timer_ns();
          alive = all(keep_waiting(waits, since));
          continue;
        }
        spin = 0;
        tc_fence_after();
        const uint32_t add = uniform(oi < 2 ? 0 : 1), v = ring + v_slot * L::kSlot, tm_v = tm0 + 128 * og;
        const uint32_t k = ring + k_slot * L::kSlot, q = q0 + (kPair ? sg * kOutTile : 0), tm_k = tm0 + 128 * sg;
        if (elect_one()) {
          if (do_o) {
#pragma unroll
            for (int c = 0; c < 8; ++c)  // bf16: 16 tokens a step; e4m3: 32, first parts, then second
              mma_ts<kByte>(tm_v + 256, tm_v + 8 * c, smem_desc(v + (kByte ? (c & 3) * 4096 : c * 2048), 16384), kIdescO,
                            c > 0 || add != 0);
          }
          if (do_s) {
#pragma unroll
            for (int c = 0; c < 8; ++c)  // bf16: 16 channels a step, four a 128-byte half; e4m3: 32, Q's first part, then its second
              mma_ss<kByte>(tm_k, smem_desc(q + (c >> 2) * 16384 + (c & 3) * 32),
                            smem_desc(k + (kByte ? 0 : (c >> 2) * 16384) + (c & 3) * 32), kIdescS, c > 0);
            mma_commit(bar_s + sg);
          }
          if (do_o) {
            if (!kPair || og == 1) mma_commit(empty + v_slot);
            if (oi >= items - 2) mma_commit(bar_o + og);
          }
        }
        if (do_o) {
          p_phases ^= 1u << og;
          ++oi;
        }
        if (do_s) ++si;
        __syncwarp();
      }
      n += g.tiles;
    }
    // what was issued is done before tensor memory is given back, whoever gave up
    if (elect_one()) mma_commit(bar_end);
    __syncwarp();
    mbar_wait(bar_end, 0, kWaitLimitNs);
  } else if (warp < 8) {
    // ------------------------------------------------------------- softmax --
    const int s = warp >> 2;                     // group
    const int t = tid & (kGroup - 1);            // lane of the accumulator
    const int w = warp & 3;
    const int row = t & (kRowsHere - 1);
    const int part = t / kRowsHere;              // which tokens of a tile: kCols from part * kCols on
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const uint32_t tm_s = tmem + lanes + 128 * s, tm_o = tmem + lanes + 256 + 128 * s;
    uint32_t s_count = 0, o_count = 0, n = 0;
    uint32_t queries = 0;                        // tiles of query rows asked for (bf16; thread 0)
    int segment = 0;                             // of the CTA, from 1
    while (walk.next(p, g)) {
      ++segment;
      const bool starts = segment == 1;
      const int head = g.unit / p.units_a_head;
      const int block = (g.unit - head * p.units_a_head) * kTreeRows + (kPair ? s * kGroup : 0);
      const int first = g.len - g.size;
      const int bh = g.b * p.kv_heads + head;
      // ---- the query rows: 16 threads a row, all loads before the first use ----
      const uint64_t seen = seen_nodes(p, g, (block + row) >> p.group_log2);
      float score_scale = kScoreScale;
      if constexpr (kByte) {
        constexpr int kThreads = kPair ? kGroup : 2 * kGroup, kStep = kThreads / 16, kChunks = kRowsHere / kStep;
        const int at = kPair ? t : tid, c = at & 15, r0 = at >> 4;
        // (kStep is a multiple of the group: a chunk further is whole nodes on)
        const int i0 = (block + r0) >> p.group_log2, step = kStep >> p.group_log2;
        const size_t heads = static_cast<size_t>(p.kv_heads) << p.group_log2;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + ((static_cast<size_t>(g.b) * p.nodes + i0) * heads + (head << p.group_log2) +
                   ((block + r0) & ((1 << p.group_log2) - 1))) * kHeadDim) + c;
        uint4 q[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
          q[k] = i0 + k * step < g.size ? __ldg(src + k * step * heads * 16) : make_uint4(0, 0, 0, 0);
        uint8_t *tile = smem + (kPair ? s * kOutTile : 0);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int r = r0 + k * kStep;
          {
            const uint32_t x[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            // the largest magnitude into [128, 256) (a subnormal one, whose
            // exponent reads as 0, below), by a power of two within fp32's range
            const int exponent = top == 0 ? 0 : min(100, 134 - static_cast<int>(top >> 7));
            const float up = __uint_as_float(static_cast<uint32_t>(127 + exponent) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              split4_signed(bf16_f(x[2 * e] & 0xFFFFu) * up, __uint_as_float(x[2 * e] & 0xFFFF0000u) * up,
                            bf16_f(x[2 * e + 1] & 0xFFFFu) * up, __uint_as_float(x[2 * e + 1] & 0xFFFF0000u) * up, hi[e], lo[e]);
#pragma unroll
            for (int copy = 0; copy < kRep; ++copy) {
              const int rr = r + copy * kRowsHere;
              uint8_t *dst = tile + rr * 128 + (((c >> 1) ^ (rr & 7)) << 4) + (c & 1) * 8;
              *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2 *>(dst + 16384) = make_uint2(lo[0], lo[1]);
            }
            if (c == 0)
              scale_s[(kPair ? s * kGroup : 0) + r] = top < 0x7F80u ? kScoreScale * down : __uint_as_float(0x7FFFFFFFu);
          }
        }
        if constexpr (kPair) named_barrier(2 + s, kGroup); else named_barrier(1, 2 * kGroup);
        score_scale = scale_s[(kPair ? s * kGroup : 0) + row];
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar_q);
      } else if (tid == 0) {  // (the first segment's: the copy warp, before K and V)
        if (!starts && alive) load_query(g);
        if (alive) ++queries;
      }

      // ---- the tiles ----
      float m = -INFINITY, l = 0.0f;
      for (int j = kPair ? 0 : s; j < g.tiles; j += kPair ? 1 : 2) {
        const int t0 = (g.tile0 + j) * kTile;
        const bool masked = t0 + kTile > first;
        const uint32_t vi = 2 * (n + j) + 1, v_slot = vi % kSlots;
        const float4 *tok = nullptr;  // [3][kCols]: K scale, V scale, its log2
        if constexpr (kByte) {
          wait(full + vi % kSlots, (vi / kSlots) & 1);
          const uint16_t *raw = reinterpret_cast<const uint16_t *>(smem + L::kScales + v_slot * 512);
          float *mine = reinterpret_cast<float *>(smem + L::kTokens) + (s * 2 + (s_count & 1)) * 3 * kTile;
          float vs = bf16_f(raw[kTile + t]);
          if (masked && t0 + t >= first) {
            // (a weight of zero must not meet a scale that is not finite: as for values, below)
            if (t0 + t >= g.len) {
              vs = 0.0f;
            } else if (!(fabsf(vs) < INFINITY)) {
              vs = 0.0f;
              *odd = segment;
            }
          }
          mine[t] = bf16_f(raw[t]);
          mine[kTile + t] = vs;
          // (a zero scale: far below any other, but not infinitely far)
          const float lv = log2f(fabsf(vs));
          mine[2 * kTile + t] = lv < -60.0f ? -60.0f : lv;
          named_barrier(2 + s, kGroup);
          tok = reinterpret_cast<const float4 *>(mine + part * kCols);
        }
        wait(bar_s + s, s_count & 1);
        ++s_count;
        tc_fence_after();
        if ((kPair ? s == 1 : true) && t == 0) mbar_arrive(empty + (vi - 1) % kSlots);  // K is read
        // 64 tokens at a time; of 128 the first 64 stay in registers for their
        // weights, the others are read twice.  (All 128 do not fit beside the
        // rest, and what a thread spills passes through the memory that feeds the
        // matrix instructions: with 180 bytes of it a tile took half as long again.)
        constexpr int kPart = kCols < 64 ? kCols : 64;
        auto load = [&](int c0, float (&x)[kPart]) {
#pragma unroll
          for (int c = 0; c < kPart; c += 32) tmem_ld<32>(tm_s + part * kCols + c0 + c, x + c);
          tmem_wait_ld<32>(x);
#pragma unroll
          for (int c = 32; c < kPart; c += 32) tmem_wait_ld<32, false>(x + c);
          if constexpr (kByte) {
#pragma unroll
            for (int c = 0; c < kPart; c += 4) {
              const float4 ks = tok[(c0 + c) >> 2];
              x[c] *= ks.x;
              x[c + 1] *= ks.y;
              x[c + 2] *= ks.z;
              x[c + 3] *= ks.w;
            }
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < kPart; c += 32) {
              const int at = t0 + part * kCols + c0 + c - first;  // the first column's node (below 0: before the tree)
              uint32_t bits;
              if (at <= -32)
                bits = ~0u;
              else if (at < 0)
                bits = static_cast<uint32_t>(seen << -at) | ((1u << -at) - 1u);
              else
                bits = at < 64 ? static_cast<uint32_t>(seen >> at) : 0u;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) x[c + e] = -INFINITY;
            }
          }
        };
        auto highest = [&](int c0, const float (&x)[kPart]) {
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if constexpr (kByte) {
#pragma unroll
            for (int c = 0; c < kPart; c += 4) {
              const float4 lv = tok[(2 * kTile + c0 + c) >> 2];
              top[0] = fmaxf(top[0], fmaf(x[c], score_scale, lv.x));
              top[1] = fmaxf(top[1], fmaf(x[c + 1], score_scale, lv.y));
              top[2] = fmaxf(top[2], fmaf(x[c + 2], score_scale, lv.z));
              top[3] = fmaxf(top[3], fmaf(x[c + 3], score_scale, lv.w));
            }
          } else {
#pragma unroll
            for (int c = 0; c < kPart; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
          }
          return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        };
        float x[kPart], high = -INFINITY;
        if constexpr (kCols > kPart) {
          load(kPart, x);
          high = highest(kPart, x);
        }
        load(0, x);
        high = fmaxf(high, highest(0, x));
        // The reference m moves only when weights would leave their range: in
        // bf16 past 2^8; in e4m3 past 448 (2^8.8), from 2^7 at the last move,
        // so that small weights keep their bits.  O follows, which is idle:
        // the product before the one that made S was the last to add to it.
        constexpr float kRoom = kByte ? 8.8f - 7.0f : 8.0f;
        if constexpr (kByte) high -= 7.0f; else high *= kScoreScale;
        if (j < 2 && (kPair ? j == 0 : true)) {
          m = in_range<kByte>(high);
        } else if (__any_sync(0xFFFFFFFFu, high > m + kRoom)) {
          const float next = in_range<kByte>(fmaxf(m, high));
          const float f = next == m ? 1.0f : exp2_f(m - next);
          m = next;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 16) {
            float o[16];
            tmem_ld<16>(tm_o + c, o);
            tmem_wait_ld<16>(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= f;
            tmem_st<16>(tm_o + c, reinterpret_cast<const uint32_t *>(o));
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        const uint64_t scale2 = two(score_scale, score_scale), ref2 = two(-ref, -ref);
        uint64_t sums[2] = {0, 0};
        // Weights of 64 tokens, into columns of S that have been read.  Of every
        // eight pairs three by polynomial, but not where there are masked ones:
        // their weight has to be 0, which the polynomial does not give.
        auto weigh = [&](int c0, const float (&x)[kPart], bool plain) {
          uint32_t w[kPart / 2];  // bf16 pairs; e4m3: first parts, then second
#pragma unroll
          for (int c = 0; c < kPart; c += 4) {
            float q[4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint64_t z = fma2(two(x[c + e], x[c + e + 1]), scale2, ref2);
              constexpr uint32_t kPoly = kByte ? 0u : 0x52u;
              if (!plain && ((kPoly >> (((c + e) >> 1) & 7)) & 1u)) {
                exp2_poly2(z, q[e], q[e + 1]);
              } else {
                one_each(z, q[e], q[e + 1]);
                q[e] = exp2_f(q[e]);
                q[e + 1] = exp2_f(q[e + 1]);
              }
              sums[e >> 1] = add2(sums[e >> 1], two(q[e], q[e + 1]));
            }
            if constexpr (kByte) {
              const float4 vs = tok[(kTile + c0 + c) >> 2];
              split4(q[0] * vs.x, q[1] * vs.y, q[2] * vs.z, q[3] * vs.w, w[c >> 2], w[kPart / 4 + (c >> 2)]);
            } else {
              w[c >> 1] = pack_bf16(q[0], q[1]);
              w[(c >> 1) + 1] = pack_bf16(q[2], q[3]);
            }
          }
          if constexpr (kByte) {
            tmem_st<kPart / 4>(tm_s + (part * kCols + c0) / 4, w);
            tmem_st<kPart / 4>(tm_s + 32 + (part * kCols + c0) / 4, w + kPart / 4);
          } else {
            tmem_st<kPart / 2>(tm_s + (part * kCols + c0) / 2, w);
          }
        };
        if (kByte || masked || __any_sync(0xFFFFFFFFu, m == -INFINITY)) {
          weigh(0, x, true);
          if constexpr (kCols > kPart) {
            load(kPart, x);
            weigh(kPart, x, true);
          }
        } else {
          weigh(0, x, false);
          if constexpr (kCols > kPart) {
            load(kPart, x);
            weigh(kPart, x, false);
          }
        }
        if constexpr (kRep > 1) {
          // a copy of the row has no weights for the other copies' tokens
          constexpr int kWide = kByte ? kCols / 4 : kCols / 2;
          uint32_t none[kWide];
#pragma unroll
          for (int c = 0; c < kWide; ++c) none[c] = 0u;
#pragma unroll
          for (int r = 1; r < kRep; ++r) {
            const int at = ((part + r) & (kRep - 1)) * kWide;
            tmem_st<kWide>(tm_s + at, none);
            if constexpr (kByte) tmem_st<kWide>(tm_s + 32 + at, none);
          }
        }
        float sum[4];
        one_each(sums[0], sum[0], sum[1]);
        one_each(sums[1], sum[2], sum[3]);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        if (masked) {
          wait(full + v_slot, (vi / kSlots) & 1);
          if (t0 + t >= first &&
              clean_values<kByte>(smem + L::kRing + v_slot * L::kSlot, t, t0 + t >= g.len, 0, kByte ? 8 : 16))
            *odd = segment;
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(bar_p + s);
      }
      n += g.tiles;

      // ---- the end of a segment ----
      const bool both = kPair || g.tiles > 1;  // both accumulators hold something
      if (both || s == 0) {
        wait(bar_o + s, o_count & 1);
        ++o_count;
      }
      row_s[s * kGroup + t] = make_float2(m, l);
      tc_fence_after();
      // (the other group's sums, or only what it found in the drafted tokens' rows)
      if (!kPair || (g.tile0 + g.tiles) * kTile > first) named_barrier(1, 2 * kGroup);
      else named_barrier(2 + s, kGroup);
      const bool whole = g.tiles == g.all;
      const bool any_odd = *odd == segment;
      float f0 = 1.0f, f1 = 0.0f, row_m = m, row_l = l;
      if constexpr (!kPair) {
        row_m = -INFINITY;
#pragma unroll
        for (int r = 0; r < 2 * kRep; ++r)
          row_m = fmaxf(row_m, row_s[(r & 1) * kGroup + (r >> 1) * kRowsHere + row].x);
        const float ref = row_m == -INFINITY ? 0.0f : row_m;
        row_l = 0.0f;
#pragma unroll
        for (int r = 0; r < 2 * kRep; ++r) {
          const float2 v = row_s[(r & 1) * kGroup + (r >> 1) * kRowsHere + row];
          row_l += v.y * exp2_f(v.x - ref);
        }
        f0 = exp2_f(row_s[t].x - ref);
        f1 = exp2_f(row_s[kGroup + t].x - ref);
        named_barrier(1, 2 * kGroup);
        row_s[s * kGroup + t] = make_float2(row_m, row_l);  // every copy of the row the same
      }
      // 32 channels at a time through shared memory (the Q tile's, which no
      // product reads any more): copies of a row are added, and what is left goes
      // out as one copy (a part), or row by row.
      const int block_row = kPair ? s * kGroup : 0;   // of the unit
      float *part_out = p.partials + static_cast<size_t>(2 * blockIdx.x + (starts ? 0 : 1)) * part_floats(p.rows);
      const int rows_out = min(kRowsHere, p.rows - block_row);
      if (!whole && (kPair || s == 0) && t < rows_out)
        *reinterpret_cast<float2 *>(part_out + part_sums(p.rows, block_row + t)) = row_s[s * kGroup + t];
      constexpr int kChannels = kPair ? kHeadDim : kHeadDim / 2;
#pragma unroll 1
      for (int c0 = 0; c0 < kChannels; c0 += 32) {
        const int ch = (kPair ? 0 : s * kChannels) + c0;
        // (two stages where there is room for them)
        float4 *stage = reinterpret_cast<float4 *>(smem + (kPair ? s * kOutTile + (c0 & 32) * 512 : s * (kOutTile / 2)));
        float o[32];
        if constexpr (kPair) {
          tmem_ld<32>(tm_o + ch, o);
          tmem_wait_ld<32>(o);
        } else {
          tmem_ld<32>(tmem + lanes + 256 + ch, o);
          tmem_wait_ld<32>(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f0;
          if (both) {
            float o1[32];
            tmem_ld<32>(tmem + lanes + 384 + ch, o1);
            tmem_wait_ld<32>(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], f1, o[e]);
          }
        }
        if (c0 >= (kPair ? 64 : 32)) {
          if (t == 0) bulk_wait_read<kPair ? 1 : 0>();
          named_barrier(2 + s, kGroup);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          stage[t * 8 + (c ^ (t & 7))] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        if (any_odd && part == 0) {
          float *mine = reinterpret_cast<float *>(stage + t * 8);
#pragma unroll 1
          for (int e = 0; e < 32; ++e)
            mine[4 * ((e >> 2) ^ (t & 7)) + (e & 3)] += odd_values<kByte>(p, g, bh, seen, ch + e);
        }
        fence_proxy_async_smem();
        named_barrier(2 + s, kGroup);
        if constexpr (kRep > 1) {
#pragma unroll 1
          for (int item = t; item < kRowsHere * 8; item += kGroup) {  // (row, place): every copy has the same place
            float4 v = stage[item];
#pragma unroll
            for (int k = 1; k < kRep; ++k) {
              const float4 u = stage[item + k * kRowsHere * 8];
              v.x += u.x;
              v.y += u.y;
              v.z += u.z;
              v.w += u.w;
            }
            stage[item] = v;
          }
          fence_proxy_async_smem();
          named_barrier(2 + s, kGroup);
        }
        if (!whole) {
          if (t == 0 && rows_out > 0) {
            bulk_s2g(part_out + (static_cast<size_t>(ch >> 5) * p.rows + block_row) * 32, stage, rows_out * 128);
            bulk_commit();
          }
          continue;
        }
#pragma unroll 1
        for (int item = t; item < kRowsHere * 8; item += kGroup) {
          const int r = item >> 3, c = item & 7, q_row = block + r, i = q_row >> p.group_log2;
          if (i >= g.size) break;
          float4 v = stage[r * 8 + (c ^ (r & 7))];
          const float sum = row_s[s * kGroup + r].y, inv = sum == 0.0f ? 1.0f : 1.0f / sum;
          v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);  // (a row that saw nothing: 0)
          uint16_t *dst = p.out + (((static_cast<size_t>(g.b) * p.nodes + i) * p.kv_heads + head) << p.group_log2) * kHeadDim +
                          (q_row & ((1 << p.group_log2) - 1)) * kHeadDim + ch + 4 * c;
          *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        }
        named_barrier(2 + s, kGroup);
      }
      if (t == 0) bulk_wait_read<0>();
      if (tid == 0 && g.tile0 == 0) note_unit(p, g, walk, start_s, starts);
      tc_fence_before();
      fence_proxy_async_smem();  // the next Q comes over what was staged
      named_barrier(1, 2 * kGroup);
    }
    if (t == 0) bulk_wait<0>();
    // (the products waited for them, but may have been given up)
    if (queries > 0) mbar_wait(bar_q, (queries - 1) & 1, kWaitLimitNs);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// --------------------------------------------------------------- the merge --

// One CTA a row (sequence, node, head): joins the parts of a unit that several
// CTAs shared, clears the rows of a bad sequence, and has nothing to do
// otherwise.  Four warps take the parts in turn, four channels a lane.
__global__ void __launch_bounds__(128) merge_tree_kernel(const TreeParams p) {
  __shared__ float4 acc_s[4][32];
  __shared__ float2 ml_s[4];
  const int heads = p.kv_heads << p.group_log2;
  const int head = blockIdx.x % heads, bi = blockIdx.x / heads;
  const int b = bi / p.nodes, i = bi - b * p.nodes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint16_t *out = p.out + static_cast<size_t>(blockIdx.x) * kHeadDim;
  asm volatile("griddepcontrol.launch_dependents;");
  // (lengths and sizes are inputs, and the call's kernel before has waited for what
  // wrote them; with an empty cache there is none)
  if (p.ctas == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  const Sequence q(p, b);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!q.good) {
    if (threadIdx.x == 0 && i == 0 && head == 0) atomicOr(p.err, kFlagBadLength);
    out[threadIdx.x] = 0;
    return;
  }
  if (i >= q.size) return;
  const int row = (i << p.group_log2) + (head & ((1 << p.group_log2) - 1));
  const int kv = head >> p.group_log2, block = row / kTreeRows;
  const int2 at = p.table[(static_cast<size_t>(b) * p.kv_heads + kv) * p.units_a_head + block];
  // (every call writes its entries, one that gave up too; no other is followed)
  if (at.y <= 1 || at.y > p.ctas || at.x < 0 || (at.x >> 1) > p.ctas - at.y) return;
  const size_t slot = part_floats(p.rows);
  // part 0 is in the slot that the table names, the others begin their CTAs: slot 0
  const int r0 = row - block * kTreeRows;
  const size_t vector = part_vector(p.rows, r0, lane), sums = part_sums(p.rows, r0);
  const float *part0 = p.partials + at.x * slot, *parts = p.partials + static_cast<size_t>(at.x >> 1) * 2 * slot;
  // four parts' loads in flight a warp, joined on a running maximum
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f, m = -INFINITY;
  for (int k0 = warp; k0 < at.y; k0 += 16) {
    float2 ml[4];
    float4 o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + 4 * u;
      ml[u] = make_float2(-INFINITY, 0.0f);
      o[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (k < at.y) {
        const float *from = k == 0 ? part0 : parts + 2 * k * slot;
        ml[u] = *reinterpret_cast<const float2 *>(from + sums);
        o[u] = *reinterpret_cast<const float4 *>(from + vector);
      }
    }
    const float next = fmaxf(m, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
    const float ref = next == -INFINITY ? 0.0f : next, fade = exp2_f(m - ref);
    m = next;
    acc.x *= fade;
    acc.y *= fade;
    acc.z *= fade;
    acc.w *= fade;
    l *= fade;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = exp2_f(ml[u].x - ref);
      acc.x = fmaf(o[u].x, f, acc.x);
      acc.y = fmaf(o[u].y, f, acc.y);
      acc.z = fmaf(o[u].z, f, acc.z);
      acc.w = fmaf(o[u].w, f, acc.w);
      l = fmaf(ml[u].y, f, l);
    }
  }
  acc_s[warp][lane] = acc;
  if (lane == 0) ml_s[warp] = make_float2(m, l);
  __syncthreads();
  float top = -INFINITY, y = 0.0f, total = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, ml_s[w].x);
  if (top == -INFINITY) top = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = exp2_f(ml_s[w].x - top);
    y = fmaf(reinterpret_cast<const float *>(acc_s[w])[threadIdx.x], f, y);
    total = fmaf(ml_s[w].y, f, total);
  }
  const float r = total == 0.0f && y == 0.0f ? 0.0f : y / total;
  out[threadIdx.x] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
}

// ----------------------------------------------------------------- launches --

bool make_tensor_map(CUtensorMap *map, const void *base, uint64_t rows, bool byte) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  if (byte) {
    const cuuint64_t dims[2] = {kByteRow, rows}, strides[1] = {kByteRow};
    const cuuint32_t box[2] = {kByteRow, kTile}, steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  // a row's two 128-byte halves as the outermost dimension: [half][token][64 channels] in shared memory
  const cuuint64_t dims[3] = {64, rows, 2}, strides[2] = {2 * kHeadDim, 128};
  const cuuint32_t box[3] = {64, kTile, 2}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as [node][kv-head][head of the group][channel]: a box is `rows`
// rows of one kv-head, half of the channels.
bool make_query_map(CUtensorMap *map, const TreeParams &p, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint32_t group = 1u << p.group_log2;
  const cuuint64_t dims[4] = {kHeadDim, group, static_cast<cuuint64_t>(p.kv_heads),
                              static_cast<cuuint64_t>(p.batch) * p.nodes};
  const cuuint64_t strides[3] = {2 * kHeadDim, 2 * kHeadDim * group, 2 * kHeadDim * group * dims[2]};
  const cuuint32_t box[4] = {64, group, 1, static_cast<cuuint32_t>(rows) / group}, steps[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(p.q), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kByte, int kCols, bool kPair>
cudaError_t launch_as(const TreeParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v, cudaStream_t stream) {
  CUtensorMap map_q{};
  if (!kByte && !make_query_map(&map_q, p, kCols)) return cudaErrorInvalidValue;  // (kCols rows, too: 128 / copies)
  using L = Layout<kByte, kPair>;
  static std::atomic<uint64_t> configured{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(tree_kernel<kByte, kCols, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  return launch_early(tree_kernel<kByte, kCols, kPair>, p.ctas, kCtaThreads, L::kTotal, stream, map_k, map_v, map_q, p);
}

cudaError_t launch_rows_of(const TreeParams &p, cudaStream_t stream) {
  const bool byte = p.format == FFD_CACHE_BYTE;
  CUtensorMap map_k, map_v;
  const uint64_t tokens = static_cast<uint64_t>(p.batch) * p.kv_heads * p.capacity;
  if (!make_tensor_map(&map_k, p.k, tokens, byte) || !make_tensor_map(&map_v, p.v, tokens, byte))
    return cudaErrorInvalidValue;
  const int rows = p.nodes << p.group_log2;
  if (rows <= 16) return launch_tree_narrow(p, map_k, map_v, stream);
  if (rows <= 32)
    return byte ? launch_as<true, 32, false>(p, map_k, map_v, stream) : launch_as<false, 32, false>(p, map_k, map_v, stream);
  if (rows <= 64)
    return byte ? launch_as<true, 64, false>(p, map_k, map_v, stream) : launch_as<false, 64, false>(p, map_k, map_v, stream);
  if (rows <= 128)
    return byte ? launch_as<true, 128, false>(p, map_k, map_v, stream) : launch_as<false, 128, false>(p, map_k, map_v, stream);
  return byte ? launch_as<true, 128, true>(p, map_k, map_v, stream) : launch_as<false, 128, true>(p, map_k, map_v, stream);
}

}  // namespace

TreeLayout tree_layout(int32_t batch, int32_t kv_heads, int32_t group, int32_t nodes, int32_t capacity) {
  TreeLayout L{};
  const int rows = group * nodes;
  L.units_a_head = (rows + kTreeRows - 1) / kTreeRows;
  L.rows = rows < kTreeRows ? rows : kTreeRows;
  const int64_t units = static_cast<int64_t>(batch) * kv_heads * L.units_a_head;
  const int64_t tiles = units * ((static_cast<int64_t>(capacity) + kTile - 1) / kTile);
  L.ctas = static_cast<int32_t>(tiles < kTreeCtas ? tiles : kTreeCtas);
  L.table = 256;
  L.partials = L.table + (static_cast<size_t>(units) * 8 + 255) / 256 * 256;
  L.total = (L.partials + static_cast<size_t>(L.ctas) * 2 * part_floats(L.rows) * 4 + 255) / 256 * 256;
  return L;
}

cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream) {
  if (p.ctas > 0) {
    const cudaError_t e = launch_rows_of(p, stream);
    if (e != cudaSuccess) return e;
  }
  const dim3 rows(static_cast<unsigned>(p.batch) * static_cast<unsigned>(p.nodes) *
                  static_cast<unsigned>(p.kv_heads << p.group_log2));
  return launch_early(merge_tree_kernel, rows, 128, 0, stream, p);
}

}  // namespace ffd
