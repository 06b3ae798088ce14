// Attention for trees of drafted tokens on the 5th-generation tensor cores
// (the mathematics: tree.cu; how the work is cut: tree_plan.cuh).
//
// A drafted tree is a handful of query rows over a long cache, so every CTA
// streams an equal share of all keys (one persistent CTA an SM, a slice of the
// batch's list of 128-key tiles), and a (unit, KV head) that is cut leaves records
// that the merge kernel joins.
//
// Rows are (node, query head of the group) pairs, up to 128 a Q tile.  The CTA
// has two streams, each with its S, P and O in tensor memory and eight softmax
// warps (two threads a row):
//   a unit of two Q tiles: stream g takes Q tile g, both use each K/V tile;
//   a unit of one Q tile: both take it, stream g every second K/V tile, and
//   their sums are joined from tensor memory at the end of the segment.
// A stream takes a tile's keys 64 at a time, in two S buffers: the next scores are
// there when a softmax ends, and the product with V and the one after next run
// beside it.  (All 128 at once, weights over their scores, left the tensor pipe
// idle while a softmax ran and the softmax while products did: 4,200 clocks a tile;
// now 2,000 for 64 keys of both Q tiles, tensor pipe 57 % and issue slots 52 % active.
// 16 sequences of 64 nodes, 64 + 8 heads of 128 over 512 to 32,768 tokens: 308 us,
// 0.47 of the bf16 rate (341 so).)
// A row's reference moves only when a score passes it by far (bf16 weights have
// fp32's range), by a vote of the row's two warps.  Keys go from the newest
// backwards; the drafted ones, which are masked by a bit a (row, node), come first.
//
// Warps (20): 0-7 and 8-15 softmax of stream 0 and 1 (warp w of a stream: TMEM
// lanes 32 (w % 4) .., keys 32 (w / 4) .. of 64), 16 copies of K and V, 17 and 19
// the products of stream 0 and 1, 18 the segments and Q.
#include "tree_stream.cuh"

namespace pkvd {

namespace {

// TMEM columns: S of stream g, keys of half h, at [128 g + 64 h, ..), its weights
// over the first 16 of each thread's 32; O at [256 + g D, 256 + g D + D).
constexpr uint32_t kColO = 256;
constexpr int kThreadKeys = 32;           // keys of a softmax thread
constexpr float kLinear = 16384.f;        // largest bias (log2 units) put together from parts

template <int D>
struct Layout {
  static constexpr int kKStages = D == 64 ? 4 : 3, kVStages = D == 64 ? 4 : 2;
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kQ = 0;                                    // 2 Q tiles
  static constexpr uint32_t kK = kQ + 2 * kHalves * kHalf;
  static constexpr uint32_t kV = kK + kKStages * kHalves * kHalf;
  static constexpr uint32_t kBar = kV + kVStages * kHalves * kHalf;
  static constexpr uint32_t kQHalf = kHalf;                            // bytes of a Q tile's 64 columns
  static constexpr int kQBufs = 2, kJoinWarps = 4;                     // kJoin: a quarter of the rows, both streams
  static constexpr uint32_t kX = kBar + kBarBytes;                     // exchange: 1024 bytes a stream
  static constexpr uint32_t kItems = kX + 2048;                        // ring of segments
  static constexpr int kItemRing = 4;
  static constexpr uint32_t kTree = 0;                                 // (the plan's array is read)
  static constexpr uint32_t kGaveUp = kItems + sizeof(Item) * kItemRing;             // one word a pair of softmax warps
  static constexpr uint32_t kEnd = kGaveUp + 32;
  // at least 120 KB so that one CTA (which holds all TMEM) is resident per SM
  static constexpr uint32_t kBytes = kEnd > 122880u ? kEnd : 122880u;
};
static_assert(Layout<128>::kBytes <= 232448, "227 KB of shared memory");

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void st_global_v8(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Which of a thread's 32 keys its row sees, and how many visible nodes lie after
// the last of them.
struct Seen {
  uint32_t word;
  int after;
};

// Keys that reach into the tree: `cut` of them lie before the first node (below 0:
// the first is a later node), the first `first` before the row's window.
__device__ __forceinline__ Seen tree_keys(const uint32_t* anc, int words, int first, int cut) {
  Seen s;
  s.after = 0;
  for (int k = 0; k < words; ++k) {                  // nodes at 32 - cut and later
    const int from = kThreadKeys - cut - 32 * k;
    const uint32_t x = anc[k];
    s.after += __popc(from <= 0 ? x : from >= 32 ? 0u : x >> from);
  }
  uint32_t x = 0u;
  if (cut <= 0) {
    const int k = -cut >> 5;
    const uint32_t lo = k < words ? anc[k] : 0u, hi = k + 1 < words ? anc[k + 1] : 0u;
    x = __funnelshift_r(lo, hi, -cut & 31);
  } else if (cut < 32) {
    x = anc[0] << cut;
  }
  s.word = x | span_bits(first, cut);
  return s;
}

// Everything a row does not see becomes `x`, whatever it was.  Most groups of
// eight keys are visible to the whole warp.
__device__ __forceinline__ void hide(float (&v)[kThreadKeys], uint32_t seen, float x) {
  const uint32_t every = __reduce_and_sync(FULL_MASK, seen);
#pragma unroll
  for (int c8 = 0; c8 < 32; c8 += 8) {
    if (((every >> c8) & 0xffu) == 0xffu) continue;
#pragma unroll
    for (int c = c8; c < c8 + 8; ++c) v[c] = (seen >> c) & 1u ? v[c] : x;
  }
}

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_tc_kernel(const __grid_constant__ TcTree p) {
  using L = Layout<D>;
  constexpr int H = L::kHalves, kKStages = L::kKStages, kVStages = L::kVStages, kItemRing = L::kItemRing;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* gbase = smem_raw;
  const uint32_t base = smem_u32(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + L::kBar);
  const TreePlan& pl = p.plan;
  const int warp = __shfl_sync(FULL_MASK, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // known to be uniform

  if (threadIdx.x == 0) tree_init_barriers<L>(bars);
  if (threadIdx.x < 8) reinterpret_cast<uint32_t*>(gbase + L::kGaveUp)[threadIdx.x] = 0;
  // a Q tile's rows past its G * tile_tokens: no copy writes them, they stay zero
  for (int i = pl.group * p.tile_tokens * 8 + (int)threadIdx.x; i < kTcRows * 8; i += kTreeThreads)
    for (int t = 0; t < 2 * H; ++t) st_shared_v4(base + L::kQ + t * kHalf + i * 16, make_uint4(0u, 0u, 0u, 0u));
  fence_proxy_async_smem();
  if (warp == kMmaWarp) tmem_alloc(base + L::kBar + kTmemSlot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL_MASK, *reinterpret_cast<volatile uint32_t*>(gbase + L::kBar + kTmemSlot), 0);

  // (what the kernels before leave is waited for where it is used)
  Item* ring_items = reinterpret_cast<Item*>(gbase + L::kItems);
  if (pl.planned) pdl_wait();

  // registers: 512 x 104 + 128 x 56 = 60416 of the 61440 that 640 threads start with
  if (warp >= kKvWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == kKvWarp) {
    tree_copy_kv<T, L>(p, bars, base, ring_items, lane);
  } else if (warp == kQWarp) {
    tree_segments<L>(p, bars, base, gbase, lane);
  } else if (warp == kMmaWarp || warp == kMmaWarp1) {
    // ---------------------------------------------------------------- MMA
    // S(n, h) of the stream, n counting all its K tiles, h = 1 (the newer 64
    // keys) before 0: Q and K have landed and PV(n - 1, h), whose weights lie in
    // the same columns, is done.  PV(n, h): the weights, V, and for a segment's
    // first one the O columns of the segment before were read.  A stage of K, V or
    // Q is free when both streams are done with it; one that this stream does not
    // use it waits for all the same, so that no phase of a stage is waited for
    // before the one before it is over.  The whole warp walks through this and one
    // elected thread issues.
    pdl_wait();          // (no bounded wait may run while the kernel before does)
    const bool leader = elect_one();
    const int g = warp == kMmaWarp ? 0 : 1;
    constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    constexpr uint32_t id_s = tc_idesc(fmt, 64, 0), id_pv = tc_idesc(fmt, D, 1), hi = desc_hi(1024);
    const uint32_t s_cols = tmem + g * 128, o_cols = tmem + kColO + g * D;
    bool ok = true;
    auto wait = [&](int bar, uint32_t parity) {
      if (ok) ok = __all_sync(FULL_MASK, wait_bounded(&bars[bar], parity));
    };
    int n = 0, used[2] = {0, 0};                   // this stream's K tiles of all segments; uses of the Q buffers
    int kstg = 0, vstg = 0;                        // next stages and their phases, every tile of every segment
    uint32_t kpar = 0, vpar = 0;
    auto next_k = [&] {
      if (++kstg == kKStages) kstg = 0, kpar ^= 1;
    };
    auto next_v = [&] {
      if (++vstg == kVStages) vstg = 0, vpar ^= 1;
    };
    auto release = [&](int full, int empty, uint32_t parity) {     // of what this stream does not use
      wait(full, parity);
      if (ok && leader) mbar_arrive(&bars[empty]);
    };
    for (int r = 0; ok; ++r) {
      ok = __all_sync(FULL_MASK, wait_item(&bars[kItemFull + r % kItemRing], (r / kItemRing) & 1));
      if (!ok) break;
      const Item& it = ring_items[r % kItemRing];
      const int all = __shfl_sync(FULL_MASK, it.n, 0);
      if (all < 0) break;
      const int two = __shfl_sync(FULL_MASK, it.two, 0), qbuf = two ? g : __shfl_sync(FULL_MASK, it.qbuf, 0);
      const int gn = two ? all : (all + 1 - g) >> 1;
      const uint32_t qd = desc_lo(base + L::kQ + qbuf * H * kHalf, 16);
      int kt = 0, vt = 0;                          // tiles of the segment that the rings have passed
      auto tile = [&](int j) { return two ? j : 2 * j + g; };
      auto to_k = [&](int t) {
        for (; ok && kt < t; ++kt) {
          release(kKFull + kstg, kKEmpty + kstg, kpar);
          next_k();
        }
      };
      auto to_v = [&](int t) {
        for (; ok && vt < t; ++vt) {
          release(kVFull + vstg, kVEmpty + vstg, vpar);
          next_v();
        }
      };
      // S(m, h) of the segment's j-th tile, m its count of all
      auto scores = [&](int m, int j, int h) {
        if (h == 1) {
          to_k(tile(j));
          wait(kKFull + kstg, kpar);
        }
        if (m > 0) wait(kPVDone + g + 2 * h, (m - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t kd = desc_lo(base + L::kK + kstg * H * kHalf, 16) + h * (64 * 128 >> 4), d = s_cols + h * 64;
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
            if (k == 0) mma_ss<false>(d, qd, kd, hi, id_s);
            else mma_ss<true>(d, qd + off, kd + off, hi, id_s);
          }
          tc_commit(&bars[kSFull + g + 2 * h]);
          if (h == 0) {
            tc_commit(&bars[kKEmpty + kstg]);
            if (j == gn - 1) tc_commit(&bars[kQEmpty + qbuf]);
          }
        }
        __syncwarp();
        if (h == 0) next_k(), ++kt;
      };
      // The O columns of the segment before were read.  This warp's own arrival
      // for the segment keeps the softmax warps of a segment in which the stream
      // has no tile from completing a phase that is still to be waited for.
      auto pass_o = [&] {
        if (r > 0) wait(kOFree + g, (r - 1) & 1);
        if (ok && leader) mbar_arrive(&bars[kOFree + g]);
      };
      auto values = [&](int j, int h) {
        if (h == 1) {
          to_v(tile(j));
          wait(kVFull + vstg, vpar);
          if (j == 0) pass_o();
        }
        wait(kPFull + g + 2 * h, n & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t vd = desc_lo(base + L::kV + vstg * H * kHalf, kHalf) + h * 4 * 128;
        if (leader) {
#pragma unroll
          for (int k = 0; k < 4; ++k)                      // 16 keys = 8 packed columns of weights
            mma_ts(o_cols, s_cols + h * 64 + (k >> 1) * kThreadKeys + (k & 1) * 8, vd + k * 128, hi, id_pv,
                   j > 0 || h == 0 || k > 0 ? 1u : 0u);
          tc_commit(&bars[kPVDone + g + 2 * h]);
          if (h == 0) tc_commit(&bars[kVEmpty + vstg]);
        }
        __syncwarp();
        if (h == 0) next_v(), ++vt;
      };
      if (gn > 0) {
        wait(kQFull + qbuf, used[qbuf] & 1);
        scores(n, 0, 1);
        scores(n, 0, 0);
        for (int j = 0; ok && j < gn; ++j, ++n) {
#pragma unroll
          for (int h = 1; h >= 0; --h) {
            values(j, h);
            if (j + 1 < gn) scores(n + 1, j + 1, h);
          }
        }
      } else {
        pass_o();
        release(kQFull + qbuf, kQEmpty + qbuf, used[qbuf] & 1);
      }
      if (two) release(kQFull + (g ^ 1), kQEmpty + (g ^ 1), used[g ^ 1] & 1);
      to_k(all);
      to_v(all);
      if (two) ++used[0], ++used[1];
      else ++used[qbuf];
      __syncwarp();
      if (ok && leader) mbar_arrive(&bars[kItemFree + r % kItemRing]);
    }
    if (!ok && leader) flag_error(p.err, PKVD_ERR_TIMEOUT);
    if (leader) tc_commit(&bars[kDrain + g]);     // every product issued is done when the CTA leaves
    wait_bounded(&bars[kDrain + g], 0);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    pdl_wait();
    pdl_trigger();
    // ------------------------------------------------------------ softmax
    // Every wait is bounded; a warp whose wait gives up leaves (the others'
    // then give up in turn).  The two warps of a quarter of a stream's rows meet
    // at a named barrier, which does not give up, but always brings both: each
    // passes the same ones, a last one when it leaves, where one that gave up asks,
    // so that both learn of it and leave.  The two streams' warps of a
    // quarter meet at an mbarrier (kJoin), whose wait is bounded too.
    const int g = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + g * 128 + half * kThreadKeys;
    const uint32_t o_addr = tmem + lane_base + kColO + g * D + half * (D / 2);
    // what a row's threads tell each other: 256 bytes a quarter of a stream's rows
    float* const x0 = reinterpret_cast<float*>(gbase + L::kX + quarter * 256);
    float* const xch = x0 + g * 256;
    Factors f;
    f.scale = both(p.scale_log2);
#pragma unroll
    for (int k = 0; k < 4; ++k) f.poly[k] = both(p.poly[k]);
    bool ok = true;
    auto wait = [&](int bar, uint32_t parity) {
      if (ok) ok = __all_sync(FULL_MASK, wait_bounded(&bars[bar], parity));
    };
    auto arrive = [&](int bar) {                 // for the warp
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bar]);
    };
    volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(gbase + L::kGaveUp) + g * 4 + quarter;
    bool told = false;
    auto vote = [&](bool mine) -> bool {         // any thread's of the row's two warps?
      uint32_t any;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
          "barrier.cta.red.or.pred p, %2, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(any)
          : "r"((uint32_t)mine), "r"(1 + g * 4 + quarter)
          : "memory");
      return any != 0;
    };
    auto meet = [&] {                            // where nobody asks for anything: one that does gave up
      if (vote(false)) ok = false, told = true;
    };
    int joins = 0;
    auto join = [&] {                            // the same for the row's four warps of both streams
      arrive(kJoin + quarter);
      wait(kJoin + quarter, joins & 1);
      ++joins;
    };
    // How far a score may pass its reference before that moves: tree_few.cu.  f16
    // weights keep their bits down to 2^-21 of the row's largest.
    constexpr bool kNarrow = std::is_same<T, __half>::value;
    constexpr float kLift = kNarrow ? 7.f : 0.f, kLimit = kNarrow ? 15.f : 24.f;
    int n = 0;                                   // this stream's K tiles so far, of all segments
    for (int r = 0; ok; ++r) {
      ok = __all_sync(FULL_MASK, wait_item(&bars[kItemFull + r % kItemRing], (r / kItemRing) & 1));
      if (!ok) break;
      const Item& it = ring_items[r % kItemRing];
      if (it.n < 0) break;
      // (the shuffles: known to be uniform, and so is what the masks make of a tile)
      auto uniform = [](int x) { return __shfl_sync(FULL_MASK, x, 0); };
      const int all = uniform(it.n), two = uniform(it.two), cached = uniform(it.cached), slot = uniform(it.slot);
      const int gn = two ? all : (all + 1 - g) >> 1, tb = two ? g * p.tile_tokens : 0;
      const bool live = row < min(p.tile_tokens, it.tokens - tb) * pl.group;
      const int tt = live ? row / pl.group : 0, gi = live ? row - tt * pl.group : 0;   // padding rows mirror row 0
      const int64_t node = it.node0 + tb + tt;
      const uint32_t* anc = pl.anc + node * pl.words;
      const int pr = cached + ((MODE & kBias) || pl.window > 0 ? pl.depth[node] : 0);
      const int wr = window_first(pr + 1, pl.window);
      const int wr_max = __reduce_max_sync(FULL_MASK, wr);
      const float nslope = bias_slope(p.mod, it.hk * pl.group + gi);
      int near = 0;                              // the first key whose bias may be put together from parts (kLinear)
      if (MODE & kBias) {
        const float steepest = __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(fabsf(nslope))));
        near = uniform(__reduce_max_sync(FULL_MASK, pr) - (int)fminf(kLinear / steepest, 1e9f));
      }
      const float range = live ? p.poly_range : INFINITY;   // padding rows have no say
      float m_ref = -INFINITY, less = 0.f, limit = -3e38f, l = 0.f;   // no reference yet: any visible key asks for one
      const int step_keys = two ? kTcKeys : 2 * kTcKeys;
      int kbase = (uniform(it.kt_last) - (two ? 0 : g)) * kTcKeys + half * kThreadKeys;
      for (int j = 0; j < gn; ++j, ++n, kbase -= step_keys) {
#pragma unroll 1
        for (int h = 1; h >= 0; --h) {
          const int k0 = kbase + h * 64;                   // this thread's first key
          // masks first: their loads run beside the product
          const bool tree = k0 + kThreadKeys > cached;
          const bool whole = !tree && k0 >= wr_max;
          const int cut = min(cached - k0, kThreadKeys);
          Seen seen;
          seen.word = 0xffffffffu;
          seen.after = 0;
          if (tree) seen = tree_keys(anc, pl.words, wr - k0, cut);
          else if (!whole) seen.word = span_bits(wr - k0, 32);
          wait(kSFull + g + 2 * h, n & 1);
          if (!ok) break;
          tc_fence_after();
          float v[kThreadKeys];
          tmem_ld32(s_addr + h * 64, v);
          tmem_ld_wait();
          // raw scores become scores in log2 units, up to a part of a linear bias
          // that is the same for eight keys: key c's is v[c] + bias + (c / 8) step
          const bool linear = (MODE & kBias) && !tree && k0 >= near;
          float kk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) kk[i] = linear ? -nslope * (float)i : 0.f;
          const float bias = linear ? nslope * (float)(pr - k0) : 0.f, step = linear ? -nslope * 8.f : 0.f;
          if (MODE & kCap) {
            // the form is chosen by the scores that count: with what else lies in
            // the stages the last bit would change from run to run
            if (!whole) hide(v, seen.word, 0.f);
            float most = 0.f;            // largest square: the polynomial's range
#pragma unroll
            for (int c = 0; c < kThreadKeys; c += 2)
              odd_poly2<(MODE & kBias) != 0>(v[c], v[c + 1], f.poly, kk[c & 7], kk[(c & 7) + 1], most);
            if (!__all_sync(FULL_MASK, most <= range)) {
              tmem_ld32(s_addr + h * 64, v);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < kThreadKeys; ++c)
                v[c] = fmaf(tanh_fast(v[c] * p.mod.cap_in), p.mod.cap_out_log2, kk[c & 7]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kThreadKeys; c += 2) {
              if (MODE & kBias) scale_add2(v[c], v[c + 1], f.scale, kk[c & 7], kk[(c & 7) + 1]);
              else scale2(v[c], v[c + 1], f.scale);
            }
          }
          if ((MODE & kBias) && !linear) {
            const float first = (float)(pr - k0);
            int after = seen.after;
#pragma unroll
            for (int c = kThreadKeys - 1; c >= 0; --c) {
              float back = first - (float)c;
              if (tree && c >= cut) {    // a node: as far as there are visible ones after it
                back = (float)after;
                after += (seen.word >> c) & 1u;
              }
              v[c] = fmaf(nslope, back, v[c]);
            }
          }
          if (!whole) hide(v, seen.word, -INFINITY);
          // relative to the row's reference
          float top = -INFINITY, shift0 = bias + less, shift1 = shift0;
#pragma unroll
          for (int c = 0; c < kThreadKeys; c += 4) {
            if ((MODE & kBias) && c > 0 && c % 8 == 0) tc_add2(shift0, shift1, step, step);
            tc_add2(v[c], v[c + 1], shift0, shift1);
            tc_add2(v[c + 2], v[c + 3], shift0, shift1);
            top = tc_max3(tc_max3(top, v[c], v[c + 1]), v[c + 2], v[c + 3]);
          }
          const bool rebase = vote(live && top > limit);
          if (rebase && *gave_up) ok = false, told = true;     // (the same word for both)
          if (!ok) break;
          if (rebase) {
            // ---- new references for the rows that passed theirs: the row's two
            // threads agree on the largest score
            xch[half * 32 + lane] = top - less;
            meet();
            if (!ok) break;
            const float most = fmaxf(top - less, xch[(half ^ 1) * 32 + lane]);
            const bool unset = m_ref == -INFINITY;
            const bool moves = unset ? most > -INFINITY : most - m_ref > kLimit;
            const float now = moves ? most - kLift : m_ref, alpha = moves && !unset ? tc_ex2(m_ref - now) : 1.f;
            if (moves) {
              m_ref = now;
              limit = kLimit;
              l *= alpha;
              const float by = -now - less;
              less = -now;
#pragma unroll
              for (int c = 0; c < kThreadKeys; ++c) v[c] += by;
            }
            if (__any_sync(FULL_MASK, alpha != 1.f)) {     // O too, when every product before this one is done
              if (h == 0) wait(kPVDone + g + 2, n & 1);
              else wait(kPVDone + g, (n - 1) & 1);
              if (ok) tc_fence_after();
#pragma unroll 1
              for (int c4 = 0; c4 < D / 64; ++c4) {
                float o[32];
                tmem_ld32(o_addr + c4 * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                tmem_st32(o_addr + c4 * 32, o);
              }
            }
            meet();                 // both have read
            if (!ok) break;
          }
          uint32_t pk[kThreadKeys / 2];
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int c = 0; c < kThreadKeys; c += 4) {
            const float e0 = tc_ex2(v[c]), e1 = tc_ex2(v[c + 1]), e2 = tc_ex2(v[c + 2]), e3 = tc_ex2(v[c + 3]);
            tc_add2(s0, s1, e0, e1);
            tc_add2(s2, s3, e2, e3);
            pk[c / 2] = Mma<T>::pack(e0, e1);
            pk[c / 2 + 1] = Mma<T>::pack(e2, e3);
          }
          l += (s0 + s1) + (s2 + s3);
          tmem_st16(s_addr + h * 64, pk);
          tmem_st_wait();
          tc_fence_before();
          arrive(kPFull + g + 2 * h);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // the last product
      if (gn > 0) wait(kPVDone + g, (n - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      // the row's sum: half 1's part to half 0, the whole and the reference back
      if (half == 1) xch[lane] = l;
      meet();
      if (!ok) break;
      if (half == 0) {
        l += xch[lane];
        xch[lane] = l;
        xch[32 + lane] = m_ref;
      }
      tc_fence_before();
      if (two) meet();
      else join();
      if (!ok) break;
      tc_fence_after();
      // factors of this row's sums in both streams' O (two: of this stream's alone)
      float f0 = 1.f, f1 = 0.f, sum = xch[lane], top = m_ref;
      bool has1 = false;
      if (!two) {
        const float l0 = x0[lane], m0 = x0[32 + lane], l1 = x0[256 + lane], m1 = x0[256 + 32 + lane];
        top = fmaxf(m0, m1);
        const float ref = top == -INFINITY ? 0.f : top;
        f0 = tc_ex2(m0 - ref);
        f1 = tc_ex2(m1 - ref);
        sum = l0 * f0 + l1 * f1;
        has1 = all > 1;
      }
      const bool odd = *static_cast<const volatile int*>(&it.odd);
      const int cols = two ? D / 2 : D / 4, col0 = two ? half * (D / 2) : (2 * g + half) * (D / 4);
      const uint32_t o0 = tmem + lane_base + kColO + (two ? g * D : 0) + col0, o1 = tmem + lane_base + kColO + D + col0;
      const float inv = slot >= 0 ? 1.f : sum > 0.f ? 1.f / sum : 0.f;
      f0 *= inv;
      f1 *= inv;
      const int64_t rec_row = (int64_t)slot * pl.unit_rows + (tb + tt) * pl.group + gi;
      T* dst = static_cast<T*>(p.out) + ((int64_t)(it.q0 + tb + tt) * pl.hq + (int64_t)it.hk * pl.group + gi) * D + col0;
      float* rec = pl.rec + rec_row * D + col0;
#pragma unroll 1
      for (int c = 0; c < cols; c += 16) {
        float o[16];
        tmem_ld16(o0 + c, o);
        if (has1) {
          float y[16];
          tmem_ld16(o1 + c, y);
          tmem_ld_wait();
          // a stream whose keys this row sees none of has zeros there
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = fmaf(y[e], f1, o[e] * f0);
        } else {
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f0;
        }
        if (odd) {
          const int kt_last = it.kt_last;
          odd_keys(p, it, Sight(it, pl.window), kt_last - all + 1, kt_last, [&](int k, const uint16_t* at) {
            const int u = k - cached;
            if (u >= 0 ? !((anc[u >> 5] >> (u & 31)) & 1u) : k < wr) return;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] += odd_value<T>(at + col0 + c + e);
          });
        }
        if (!live) continue;
        if (slot >= 0) {
          st_global_v8(rec + c, reinterpret_cast<const uint32_t*>(o));
          st_global_v8(rec + c + 8, reinterpret_cast<const uint32_t*>(o) + 8);
        } else {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = Mma<T>::pack(o[2 * e], o[2 * e + 1]);
          if (p.wide_out) {
            st_global_v8(dst + c, w);
          } else {
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
      if (slot >= 0 && live && half == 0 && (two || g == 0)) pl.rec_ml[rec_row] = make_float2(top, sum);
      tc_fence_before();
      arrive(kOFree);
      arrive(kOFree + 1);
      arrive(kItemFree + r % kItemRing);
      if (two) meet();                      // the exchanged values are read before the next segment's
      else join();
    }
    if (!told) {
      if (!ok) *gave_up = 1;
      vote(!ok);
    }
    if (!ok && lane == 0) flag_error(p.err, PKVD_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename T, int D, int MODE>
cudaError_t launch_mode(const TcTree& prm, cudaStream_t stream) {
  constexpr int smem = Layout<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<T, D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_tc_kernel<T, D, MODE>, dim3((unsigned)prm.plan.grid), dim3(kTreeThreads), smem, stream, prm);
}

template <typename T, int D>
cudaError_t launch_typed(const TcTree& prm, cudaStream_t stream) {
  const bool cap = prm.mod.cap_in != 0.f, bias = prm.mod.slopes != nullptr;
  if (cap && bias) return launch_mode<T, D, kCap | kBias>(prm, stream);
  if (bias) return launch_mode<T, D, kBias>(prm, stream);
  return cap ? launch_mode<T, D, kCap>(prm, stream) : launch_mode<T, D, 0>(prm, stream);
}

}  // namespace

// What the tensor copies need: the cache's strides nest, rows on 16 bytes.
bool tree_tc_supported(const TreeArgs& a) {
  const pkvd_cache& c = a.cache;
  if (c.dtype != PKVD_F16 && c.dtype != PKVD_BF16) return false;
  if (c.block_size < 8) return false;            // a box fills whole 8-row swizzle atoms
  if ((reinterpret_cast<uintptr_t>(a.out) & 15u) || (reinterpret_cast<uintptr_t>(a.q) & 15u)) return false;
  if (c.head_stride < c.head_dim || c.token_stride < c.head_stride * c.num_kv_heads ||
      c.block_stride < c.token_stride * c.block_size)
    return false;
  CUtensorMap m;
  return encode_cache_map(&m, c.k_base, c, c.block_size < kTcKeys ? c.block_size : kTcKeys);
}

cudaError_t launch_tree_tc(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  TcTree prm;
  if (!tree_tc_params(a, plan, kTcRows / plan.group, &prm)) return cudaErrorInvalidValue;
  const bool wide = a.cache.head_dim == 128;
  if (a.cache.dtype == PKVD_BF16)
    return wide ? launch_typed<__nv_bfloat16, 128>(prm, stream) : launch_typed<__nv_bfloat16, 64>(prm, stream);
  return wide ? launch_typed<__half, 128>(prm, stream) : launch_typed<__half, 64>(prm, stream);
}

}  // namespace pkvd
