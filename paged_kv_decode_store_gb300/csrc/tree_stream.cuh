// What the tensor-core kernels of drafted trees share (tree_tc.cu: up to two Q
// tiles of 128 rows; tree_few.cu: up to 64 rows): a slice's segments, the copies
// of K, V and Q, and the barriers between them.
#pragma once


#include "common.cuh"
#include "launch.h"
#include "score_mod.cuh"
#include "tc_softmax.cuh"
#include "tcgen05.cuh"
#include "tree_plan.cuh"

namespace pkvd {

constexpr int kTreeThreads = 640;
constexpr int kStreamWarps = 8;           // softmax warps of a stream
constexpr int kKvWarp = 16, kMmaWarp = 17, kQWarp = 18, kMmaWarp1 = 19;
constexpr uint32_t kTmemCols = 512;
enum : int { kCap = 1, kBias = 2 };       // what a call modifies, known when compiled

// mbarriers: five for each stage of K and V; those of a stream take + g, S, P and
// PV + g + 2 half
enum : int {
  kKFull = 0, kKEmpty = 5, kVFull = 10, kVCut = 15, kVEmpty = 20, kQFull = 25, kQEmpty = 27, kItemFull = 29,
  kItemFree = 33, kDrain = 37, kOFree = 39, kJoin = 41, kSFull = 45, kSRead = 49, kPFull = 51, kPVDone = 55, kNumBars = 59
};
constexpr uint32_t kBarBytes = 512, kTmemSlot = 8 * kNumBars;
static_assert(kTmemSlot + 4 <= kBarBytes, "behind the barriers");
constexpr int kTreeFull = kJoin;                  // tree_few.cu, two: a segment's tree_rows (its streams need not join)
constexpr int kTreeBytes = 64 * 8 + 64;            // tree_rows
constexpr int kItemUsers = 3 + 2 * kStreamWarps;   // K/V, two MMA and softmax warps

struct TcTree {
  CUtensorMap tmap_q, tmap_k, tmap_v;
  TreePlan plan;
  void* out;
  const int32_t* tables;
  const int32_t* parents;
  int max_blocks;
  int block_size, block_shift;   // a power of two
  uint32_t block_limit;          // num_blocks, at most 2^31
  int seg_rows;                  // rows per TMA box of the cache: min(block_size, 128)
  int tile_tokens;               // nodes of a Q tile
  uint32_t q_box;                // bytes of one 64-column box of a Q tile
  float scale_log2;
  ScoreMod mod;
  float poly[4], poly_range;     // cap_poly
  const uint16_t* values;        // V of the cache, and its strides in elements
  int64_t block_stride, token_stride, head_stride;
  int wide_out;                  // out is 32-byte aligned: stores of 32 bytes
  int32_t* err;
};

// A segment: n tiles of a (unit, KV head) from tile kt_last down.  n = -1: no more.
struct __align__(16) Item {
  int seq, hk, q0, tokens;       // q0: the unit's first row of q
  int node0, cached, lo, hi;     // node0: its place in the plan's arrays; keys outside [lo, hi] are not read
  int kt_last, n, slot, two;     // two Q tiles?
  int qbuf, late;                // where a single Q tile lies; more than the unit's last tile, and that
  int odd, pad;                  // set by the copies of V: values that are no numbers (tidy_values)
};

__device__ __forceinline__ int window_first(int c, int window) { return (window > 0 && c > window) ? c - window : 0; }

// Which keys no row sees, and which ones perhaps some: drafted ones, and those
// that a window has left behind for some of the rows.
struct Sight {
  int lo, hi, cached, edge;      // keys outside [lo, hi]: no row; cached keys from `edge` on: all rows
  __device__ Sight(const Item& it, int window)
      : lo(it.lo), hi(it.hi), cached(it.cached), edge(window_first(it.hi + 1, window)) {}
  __device__ bool whole(int kbase) const {     // of a tile: all rows see every key
    return kbase >= lo && kbase >= edge && kbase + kTcKeys <= min(cached, hi + 1);
  }
};

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// A V tile (H boxes of 64 dims), by a warp, where not all rows see every key: a
// weight of 0 times an infinity or a NaN would be a NaN.  Rows that no row of Q
// sees become zeros; in those that some see, every element that is no finite
// number does.  Returns whether there was one: the sums get it afterwards, where
// it is seen (odd_keys).
template <typename T, int H>
__device__ __forceinline__ bool tidy_values(uint32_t tile, int kbase, const Sight& s, int lane) {
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
  const int first = max(s.lo - kbase, 0), end = min(s.hi - kbase + 1, kTcKeys);
  bool odd = false;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const uint32_t at = tile + h * kHalf;      // a key: 128 bytes, whose order does not matter here
    for (int i = lane; i < first * 8; i += 32) st_shared_v4(at + i * 16, make_uint4(0u, 0u, 0u, 0u));
    for (int i = end * 8 + lane; i < kTcKeys * 8; i += 32) st_shared_v4(at + i * 16, make_uint4(0u, 0u, 0u, 0u));
    auto look = [&](int from, int to) {
      uint32_t any = 0u;
#pragma unroll 4
      for (int i = from * 8 + lane; i < to * 8; i += 32) {
        const uint4 x = ld_shared_v4(at + i * 16);          // (a carry into the sign: all ones in the exponent)
        any |= ((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne);
      }
      if (!(any & 0x80008000u)) return;
      for (int i = from * 8 + lane; i < to * 8; i += 32) {
        const uint4 x = ld_shared_v4(at + i * 16);
        const uint32_t a = __vcmpeq2(x.x & kExp, kExp), b = __vcmpeq2(x.y & kExp, kExp),
                       c = __vcmpeq2(x.z & kExp, kExp), d = __vcmpeq2(x.w & kExp, kExp);
        if (a | b | c | d) {
          odd = true;
          st_shared_v4(at + i * 16, make_uint4(x.x & ~a, x.y & ~b, x.z & ~c, x.w & ~d));
        }
      }
    };
    look(first, min(s.edge - kbase, end));
    look(max(s.cached - kbase, first), end);
  }
  return __any_sync(FULL_MASK, odd);
}

// The keys of tiles [kt0, kt1] that tidy_values looks at, for sums that miss a
// value (softmax weights are above 0, so an infinity or a NaN goes into them as it
// is): f(key, its row of V).
template <typename F>
__device__ __forceinline__ void odd_keys(const TcTree& p, const Item& it, const Sight& s, int kt0, int kt1, F f) {
  const int k0 = max(s.lo, kt0 * kTcKeys), k1 = min(s.hi, kt1 * kTcKeys + kTcKeys - 1);
#pragma unroll 1
  for (int k = k0; k <= k1; ++k) {
    if (k >= s.edge && k < s.cached) {         // on to the drafted ones
      k = max(k, min(s.cached, k1 + 1) - 1);
      continue;
    }
    const uint32_t b = (uint32_t)__ldg(p.tables + (int64_t)it.seq * p.max_blocks + (k >> p.block_shift));
    if (b >= p.block_limit) continue;
    f(k, p.values + (int64_t)b * p.block_stride + (int64_t)(k & (p.block_size - 1)) * p.token_stride +
             (int64_t)it.hk * p.head_stride);
  }
}
template <typename T>
__device__ __forceinline__ float odd_value(const uint16_t* at) {   // 0 for a finite number
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  const uint16_t x = *at;
  T t;
  memcpy(&t, &x, 2);
  return (x & kExp) == kExp ? DT<T>::to_f(t) : 0.f;
}

// Barriers and what a kernel's layout L says of its arrivals.
template <typename L>
__device__ __forceinline__ void tree_init_barriers(uint64_t* bars) {
  for (int i = 0; i < kNumBars; ++i) {
    int arrivals = 1;
    if ((i >= kPFull && i < kPVDone) || (i >= kSRead && i < kPFull)) arrivals = kStreamWarps;
    if (i >= kOFree && i < kJoin) arrivals = 2 * kStreamWarps + 1;
    if ((i >= kKEmpty && i < kVFull) || (i >= kVEmpty && i < kQFull) || i == kQEmpty || i == kQEmpty + 1) arrivals = 2;
    if (i >= kItemFree && i < kDrain) arrivals = kItemUsers;
    if (i >= kJoin && i < kSFull) arrivals = L::kJoinWarps;
    mbar_init(&bars[i], arrivals);
  }
  fence_mbar_init();
}

// K and V (one warp; the block tables are inputs, read before the wait for the
// kernel before).  Lane s copies segment s of a tile; K runs kAhead tiles
// ahead of V.  A V tile with keys that not every row sees lands on a barrier of
// its own (kVCut) and is released when tidy_values has seen to it.
template <typename T, typename L>
__device__ __forceinline__ void tree_copy_kv(const TcTree& p, uint64_t* bars, uint32_t base, Item* ring_items, int lane) {
  constexpr int H = L::kHalves, kKStages = L::kKStages, kVStages = L::kVStages, kItemRing = L::kItemRing;
  constexpr int kAhead = kKStages - 2;
  const uint32_t box = (uint32_t)p.seg_rows * 128u;
  const int nseg = kTcKeys / p.seg_rows;
  const uint32_t whole = (1u << nseg) - 1u;  // at most 16 segments
  if (lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_v)) : "memory");
  }
  constexpr int kNone = -1;                  // a segment of rows that are not read: nothing to load
  bool ok = true;
  int kstg = 0, vstg = 0, landed = 0;        // next stages; phases of kVCut
  uint32_t kpar = 1, vpar = 1;               // parities of their release (nothing to wait for in the first round)
  auto wait = [&](int bar, uint32_t parity) {
    if (ok) ok = __all_sync(FULL_MASK, wait_bounded(&bars[bar], parity));
  };
  // one operand of a tile into a stage, whose block id is b in lane s
  auto copy = [&](const CUtensorMap* map, uint32_t dst, int bar, int ks, int hk, int b, auto is_read) {
    const bool good = (uint32_t)b < p.block_limit;
    const uint32_t loaded = __ballot_sync(FULL_MASK, good);
    uint32_t bytes = H * kHalf;
    dst += lane * box;
    if (loaded != whole) {
      bytes = (uint32_t)__popc(loaded) * box * H;
      const uint32_t bad = __ballot_sync(FULL_MASK, !good && is_read(ks));
      if (bad) {                             // a bad block id reads as zeros
        if (lane == 0) flag_error(p.err, PKVD_ERR_BLOCK_ID);
        if ((bad >> lane) & 1u) {
          for (int h = 0; h < H; ++h)
            for (uint32_t o = 0; o < box; o += 16) st_shared_v4(dst + h * kHalf + o, make_uint4(0u, 0u, 0u, 0u));
          fence_proxy_async_smem();
        }
        __syncwarp();
      }
    }
    if (lane == 0) mbar_arrive_expect_tx(&bars[bar], bytes);
    __syncwarp();
    if (good) {
#pragma unroll
      for (int h = 0; h < H; ++h) tma_load4(dst + h * kHalf, map, h * 64, hk, ks & (p.block_size - 1), b, &bars[bar]);
    }
  };
  for (int r = 0; ok; ++r) {
    ok = __all_sync(FULL_MASK, wait_item(&bars[kItemFull + r % kItemRing], (r / kItemRing) & 1));
    if (!ok) break;
    Item& cur = ring_items[r % kItemRing];
    if (cur.n < 0) break;
    const int32_t* table = p.tables + (int64_t)cur.seq * p.max_blocks;
    const int n = cur.n, hk = cur.hk, lo = cur.lo, hi = cur.hi, kt_last = cur.kt_last;
    const Sight sight(cur, p.plan.window);
    auto key_of = [&](int t) { return (kt_last - t) * kTcKeys + lane * p.seg_rows; };
    auto is_read = [&](int ks) { return lane < nseg && ks <= hi && ks + p.seg_rows - 1 >= lo; };
    auto fetch = [&](int t) -> int {
      const int ks = key_of(t);
      return t < n && is_read(ks) ? __ldg(table + (ks >> p.block_shift)) : kNone;
    };
    auto copy_k = [&](int t, int b) {
      wait(kKEmpty + kstg, kpar);
      if (!ok) return;
      copy(&p.tmap_k, base + L::kK + kstg * H * kHalf, kKFull + kstg, key_of(t), hk, b, is_read);
      if (++kstg == kKStages) kstg = 0, kpar ^= 1;
    };
    int b[4];                                // block ids of V tile t and the three after it
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = fetch(i);
    if (r == 0) pdl_wait();                  // the cache rows of this step
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < n) copy_k(i, b[i]);
    for (int t = 0; ok && t < n; ++t) {
      if (t + kAhead < n) copy_k(t + kAhead, b[kAhead]);
      wait(kVEmpty + vstg, vpar);
      if (!ok) break;
      const int kbase = (kt_last - t) * kTcKeys;
      const bool cut = !sight.whole(kbase);
      const uint32_t dst = base + L::kV + vstg * H * kHalf;
      copy(&p.tmap_v, dst, (cut ? kVCut : kVFull) + vstg, kbase + lane * p.seg_rows, hk, b[0], is_read);
      if (cut) {
        wait(kVCut + vstg, (landed >> vstg) & 1);
        if (!ok) break;
        landed ^= 1 << vstg;
        if (tidy_values<T, H>(dst, kbase, sight, lane) && lane == 0) cur.odd = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kVFull + vstg]);
      }
      if (++vstg == kVStages) vstg = 0, vpar ^= 1;
      b[0] = b[1];
      b[1] = b[2];
      b[2] = b[3];
      b[3] = fetch(t + 4);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kItemFree + r % kItemRing]);
  }
  if (!ok && lane == 0) {
    // gave up: let the copies still in flight land before the CTA leaves
    flag_error(p.err, PKVD_ERR_TIMEOUT);
    // (a stage's full barrier is behind its release, or one phase ahead of it)
    for (int u = 0; u < kKStages; ++u) wait_bounded(&bars[kKFull + u], (kpar ^ (u < kstg ? 0u : 1u)) ^ 1u);
    for (int u = 0; u < kVStages; ++u) wait_bounded(&bars[kVFull + u], (vpar ^ (u < vstg ? 0u : 1u)) ^ 1u);
    // (a V tile on its way to the cut barrier; without one this runs into its limit, which costs a loop nothing)
    wait_bounded(&bars[kVCut + vstg], (landed >> vstg) & 1);
  }
}

// A tree of at most 64 rows, by a warp: which rows see a node (64 bits), and its
// depth.  Every node (lane's and lane + 32's parents: up) walks up to its root.
__device__ __forceinline__ void tree_rows(const TcTree& p, int n, int (&up)[2], uint32_t* rows, uint8_t* depths, int lane) {
  const TreePlan& pl = p.plan;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = i * 32 + lane;
    if (up[i] < -1 || up[i] >= t) {
      flag_error(p.err, PKVD_ERR_TREE);
      up[i] = -1;
    }
    rows[2 * t] = rows[2 * t + 1] = 0u;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = i * 32 + lane;
    if (i * 32 >= n) break;
    const uint64_t mine = t < n ? (pl.group == 64 ? ~0ull : (1ull << pl.group) - 1ull) << (t * pl.group) : 0ull;
    int u = t < n ? t : -1, depth = -1;
    while (__any_sync(FULL_MASK, u >= 0)) {
      if (u >= 0) {
        ++depth;
        if (pl.window <= 0 || depth < pl.window) {
          if ((uint32_t)mine) atomicOr(rows + 2 * u, (uint32_t)mine);
          if (mine >> 32) atomicOr(rows + 2 * u + 1, (uint32_t)(mine >> 32));
        }
      }
      const int a = __shfl_sync(FULL_MASK, up[0], u & 31), b = __shfl_sync(FULL_MASK, up[1], u & 31);
      if (u >= 0) u = u < 32 ? a : b;
    }
    if (t < n) depths[t] = (uint8_t)depth;
  }
  __syncwarp();
}

// Segments and Q (one warp).  A Q tile's rows are one box per 64 columns (G heads
// of tile_tokens nodes).  Two tiles of a unit fill both buffers; single ones take
// them in turn (L::kQBufs), so the next is loaded while the last is in use.  The
// first segments are there before the wait for the kernel before, where there is no
// plan to wait for.
template <typename L>
__device__ __forceinline__ void tree_segments(const TcTree& p, uint64_t* bars, uint32_t base, uint8_t* gbase, int lane) {
  constexpr int H = L::kHalves, kItemRing = L::kItemRing;
  const TreePlan& pl = p.plan;
  Item* ring_items = reinterpret_cast<Item*>(gbase + L::kItems);
  const bool own = !pl.planned;
  TreeWalk walk;
  bool waited = !own;
  if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_q)) : "memory");
  int64_t total = 0;
  if (own) {
    const OwnStart s(pl, blockIdx.x, lane);
    walk.start(pl, blockIdx.x, s.first);
    total = s.total;
    if (s.bad && blockIdx.x == 0) flag_error(p.err, PKVD_ERR_CONTEXT);
  } else {                                   // (the kernel before, the plan, was waited for)
    walk.start(pl, blockIdx.x, pl.slice[blockIdx.x]);
    total = pl.starts[pl.num_seqs];
  }
  bool ok = true;
  int used[2] = {0, 0}, turn = 0;
  for (int r = 0; ok; ++r) {
    const int slot = r % kItemRing;
    if (r >= kItemRing) ok = __all_sync(FULL_MASK, wait_item(&bars[kItemFree + slot], ((r / kItemRing) - 1) & 1));
    if (!ok) break;
    Item it;
    TreeSegment g;
    it.n = -1;
    if (walk.next(pl, g)) {
      const int tb = g.unit * pl.unit_tokens;
      it.seq = g.seq;
      it.hk = g.head;
      it.q0 = walk.s.q0 + tb;
      it.tokens = min(pl.unit_tokens, walk.s.n - tb);
      it.node0 = g.seq * pl.max_q + tb;
      it.cached = walk.s.cached;
      it.lo = walk.s.lo;
      it.hi = walk.s.klen - 1;
      it.kt_last = walk.s.lo_tile + g.t1 - 1;
      it.n = g.t1 - g.t0;
      it.slot = g.slot;
      it.late = g.t1 == walk.s.tiles && it.n > 1;
      it.odd = 0;
      it.two = it.tokens > p.tile_tokens;
      it.qbuf = turn;
      if (!it.two && L::kQBufs == 2) turn ^= 1;
    }
    if (lane == 0) {
      ring_items[slot] = it;
      mbar_arrive(&bars[kItemFull + slot]);
    }
    __syncwarp();
    if (it.n < 0) {
      if (L::kTree > 0 && lane == 0) mbar_arrive(&bars[kTreeFull + slot]);
      if (r == 0) {
        if (!waited) pdl_wait();
        if (lane == 0) tell_join(pl, walk, g, false, total);
      }
      break;
    }
    int up[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      up[i] = L::kTree > 0 && i * 32 + lane < it.tokens ? p.parents[it.q0 + i * 32 + lane] : -1;
    if (!waited) pdl_wait();
    waited = true;
#pragma unroll
    for (int g2 = 0; g2 < 2; ++g2) {
      if (!ok || !(it.two || it.qbuf == g2)) continue;
      if (used[g2] > 0) ok = __all_sync(FULL_MASK, wait_item(&bars[kQEmpty + g2], (used[g2] - 1) & 1));
      if (!ok) continue;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[kQFull + g2], p.q_box * H);
        for (int h = 0; h < H; ++h)
          tma_load3(base + L::kQ + (g2 * H + h) * L::kQHalf, &p.tmap_q, h * 64, it.hk * pl.group,
                    it.q0 + (it.two ? g2 * p.tile_tokens : 0), &bars[kQFull + g2]);
      }
      ++used[g2];
    }
    if constexpr (L::kTree > 0) {              // the unit is the whole tree
      uint8_t* tree = gbase + L::kTree + slot * kTreeBytes;
      tree_rows(p, it.tokens, up, reinterpret_cast<uint32_t*>(tree), tree + 512, lane);
      if (lane == 0) mbar_arrive(&bars[kTreeFull + slot]);
    }
    if (r == 0 && lane == 0) tell_join(pl, walk, g, true, total);
  }
  if (!ok && lane == 0) flag_error(p.err, PKVD_ERR_TIMEOUT);
  if (lane == 0)
    for (int g2 = 0; g2 < 2; ++g2)             // no copy is in flight when the CTA leaves
      if (used[g2] > 0) wait_bounded(&bars[kQFull + g2], (used[g2] - 1) & 1);
}

// Host: the parameters, without the shape of a Q tile's rows.
inline bool tree_tc_params(const TreeArgs& a, const TreePlan& plan, int tile_tokens, TcTree* prm) {
  const pkvd_cache& c = a.cache;
  prm->plan = plan;
  prm->seg_rows = c.block_size < kTcKeys ? c.block_size : kTcKeys;
  prm->tile_tokens = tile_tokens;
  if (!encode_cache_map(&prm->tmap_k, c.k_base, c, prm->seg_rows) ||
      !encode_cache_map(&prm->tmap_v, c.v_base, c, prm->seg_rows) ||
      !encode_q_map(&prm->tmap_q, a.q, c.dtype, c.head_dim, a.num_q_heads, a.total_q, plan.group, tile_tokens))
    return false;
  prm->values = static_cast<const uint16_t*>(c.v_base);
  prm->block_stride = c.block_stride;
  prm->token_stride = c.token_stride;
  prm->head_stride = c.head_stride;
  prm->out = a.out;
  prm->tables = a.block_tables;
  prm->parents = a.parents;
  prm->max_blocks = a.max_blocks_per_seq;
  prm->block_limit = (uint32_t)(c.num_blocks < 0x80000000ll ? c.num_blocks : 0x80000000ll);
  prm->block_size = c.block_size;
  prm->block_shift = 0;
  while ((1 << prm->block_shift) < c.block_size) ++prm->block_shift;
  prm->q_box = 128u * (uint32_t)(plan.group * tile_tokens);
  prm->scale_log2 = a.scale * 1.4426950408889634f;
  prm->mod = a.mod;
  prm->poly_range = cap_poly(a.mod, prm->poly);
  prm->wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  prm->err = a.err;
  return true;
}

}  // namespace pkvd
