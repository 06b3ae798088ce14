// Attention for trees of drafted tokens, units of at most N = 32 or 64 rows, on
// the 5th-generation tensor cores (the mathematics: tree.cu; how the work is cut:
// tree_plan.cuh).
//
// With a Q tile of 128 rows (tree_tc.cu) a small tree leaves most of each
// softmax thread's work to rows that do not exist, and its accumulators fill
// tensor memory, so a stream has one product in flight.  Here the products are
// the other way round: keys are the 128 rows, query rows the N columns,
//   S^T[128 keys x N] = K Q^T,   O^T[D x N] += V^T P^T,
// so that softmax work and accumulators shrink with N, S^T has two buffers (the
// next scores are there before the last weights are done) and one row of tiles
// suffices: no second stream to join.  32 sequences of 8 nodes over 2,048
// tokens, 48 + 8 heads of 128 in bf16: 62 us instead of 71, 275 MB of K and V at 0.65
// of the copy rate (128 sequences: 188 us, 0.86; the rest is start, first and last
// tiles and the merge).  A tile takes the larger of its copies, 2,600 clocks at
// head_dim 128, and the chain from scores to weights, 2,200, which bounds head_dim 64.
//
// A softmax thread has one key and a fourth of the columns.  A column's maximum
// would need a reduction over the tile's 128 threads; instead the weights are
// taken against a reference that moves only when some score passes it by far (a
// vote a tile; the first tile of a segment sets it), and every thread sums its
// own weights, joined at the end of the segment.  Weights go through shared
// memory (one 128-byte row a key, the operand's swizzle); O^T leaves with whole
// rows of D a warp and column.
//
// Warps (20): 0-15 softmax (warp w: keys and lanes 32 (w % 4) .., columns N / 4
// (w / 4) ..), 16 copies of K, 17 the products, 18 the segments and Q, 19 copies
// of V.
#include "tree_stream.cuh"

namespace pkvd {

namespace {

constexpr int kVWarp = 19;
constexpr float kNoRef = 3e38f;           // added to a score: no reference yet, so any visible key asks for one
constexpr uint32_t kFewCols = 256;        // TMEM: S^T at [64 buffer, ..), O^T at [128, ..)
constexpr uint32_t kColO = 128;

template <int D, int N>
struct Layout {
  static constexpr int kKStages = D == 64 ? 5 : 3, kVStages = kKStages;
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kQHalf = N * 128;                          // bytes of a Q tile's 64 columns
  static constexpr int kQBufs = D == 64 ? 2 : 1;
  static constexpr uint32_t kK = 0;                                    // K and V before P: V^T of 64 dims has 128
  static constexpr uint32_t kV = kK + kKStages * kHalves * kHalf;      //   rows all the same, the others unused
  static constexpr uint32_t kP = kV + kVStages * kHalves * kHalf;      // 128 keys x 128 bytes
  static constexpr uint32_t kQ = kP + kHalf;
  static constexpr uint32_t kBar = kQ + kQBufs * kHalves * kQHalf;
  static constexpr uint32_t kRef = kBar + kBarBytes;                   // [64] references (log2 units), -inf: none yet
  static constexpr uint32_t kNeg = kRef + 256;                         // [64] what is added to a score: -reference
  static constexpr uint32_t kPos = kNeg + 256;                         // [64] positions of the columns' rows
  static constexpr uint32_t kSlope = kPos + 256;                       // [64]
  static constexpr uint32_t kItems = kSlope + 256;
  static constexpr int kItemRing = 2;
  static constexpr uint32_t kTree = kItems + sizeof(Item) * kItemRing; // of each segment: which rows see a drafted key
  static constexpr uint32_t kGaveUp = kTree + kTreeBytes * kItemRing;
  static constexpr uint32_t kEnd = kGaveUp + 16;
  // at least 120 KB so that one CTA is resident per SM
  static constexpr uint32_t kBytes = kEnd > 122880u ? kEnd : 122880u;
};
static_assert(Layout<128, 64>::kBytes <= 232448, "227 KB of shared memory");

// C consecutive fp32 columns of this thread's TMEM lane.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[C]) {
  static_assert(C == 8 || C == 16, "");
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  }
}
template <int C>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[C]) {
  static_assert(C == 8 || C == 16, "");
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  if constexpr (C == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  }
}

__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  d0 = a0, d1 = a1;
  tc_add2(d0, d1, b0, b1);
}

// Order-preserving whole numbers of fp32 (for maxima in shared memory).
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

__device__ __forceinline__ void mma_ss_if(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}


// The j-th tile of a segment: from the newest backwards, but the newest one last
// where it ends with the tree (`late`): it has few keys to set references by.
__device__ __forceinline__ int tile_at(int kt_last, int n, int late, int j) {
  return late ? (j == n - 1 ? kt_last : kt_last - 1 - j) : kt_last - j;
}

// K or V of every segment (a warp each): lane s copies 8 to 128 rows of a tile.  A
// V tile with keys that not every row sees lands on a barrier of its own (kVCut)
// and is released when tidy_values has seen to it.
template <typename T, typename L, bool IS_V>
__device__ __forceinline__ void copy_tiles(const TcTree& p, uint64_t* bars, uint32_t base, Item* ring_items, int lane) {
  constexpr int H = L::kHalves, kStages = IS_V ? L::kVStages : L::kKStages, kItemRing = L::kItemRing;
  constexpr int full = IS_V ? kVFull : kKFull, empty = IS_V ? kVEmpty : kKEmpty;
  const CUtensorMap* map = IS_V ? &p.tmap_v : &p.tmap_k;
  const uint32_t ring = base + (IS_V ? L::kV : L::kK), box = (uint32_t)p.seg_rows * 128u;
  const int nseg = kTcKeys / p.seg_rows;
  const uint32_t whole = (1u << nseg) - 1u;    // at most 16 segments
  if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  constexpr int kNone = -1;                    // a segment of rows that are not read: nothing to load
  bool ok = true;
  int stg = 0, landed = 0;                     // next stage; phases of kVCut
  uint32_t par = 1;                            // parity of its release (nothing to wait for in the first round)
  auto wait = [&](int bar, uint32_t parity) {
    if (ok) ok = __all_sync(FULL_MASK, wait_bounded(&bars[bar], parity));
  };
  for (int r = 0; ok; ++r) {
    ok = __all_sync(FULL_MASK, wait_item(&bars[kItemFull + r % kItemRing], (r / kItemRing) & 1));
    if (!ok) break;
    Item& cur = ring_items[r % kItemRing];
    if (cur.n < 0) break;
    const Sight sight(cur, p.plan.window);
    const int32_t* table = p.tables + (int64_t)cur.seq * p.max_blocks;
    const int n = cur.n, hk = cur.hk, lo = cur.lo, hi = cur.hi, kt_last = cur.kt_last, late = cur.late;
    auto is_read = [&](int ks) { return lane < nseg && ks <= hi && ks + p.seg_rows - 1 >= lo; };
    auto fetch = [&](int t) -> int {
      const int ks = tile_at(kt_last, n, late, t) * kTcKeys + lane * p.seg_rows;
      return t < n && is_read(ks) ? __ldg(table + (ks >> p.block_shift)) : kNone;
    };
    int b[4];                                  // block ids of tile t and the three after it
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = fetch(i);
    if (r == 0) pdl_wait();                    // the cache rows of this step
    for (int t = 0; ok && t < n; ++t) {
      wait(empty + stg, par);
      if (!ok) break;
      const int kbase = tile_at(kt_last, n, late, t) * kTcKeys, ks = kbase + lane * p.seg_rows;
      const bool cut = IS_V && !sight.whole(kbase);
      uint64_t* bar = &bars[(cut ? kVCut : full) + stg];
      const uint32_t tile = ring + stg * H * kHalf, dst = tile + lane * box;
      const bool good = (uint32_t)b[0] < p.block_limit;
      const uint32_t loaded = __ballot_sync(FULL_MASK, good);
      uint32_t bytes = H * kHalf;
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
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (good) {
#pragma unroll
        for (int h = 0; h < H; ++h) tma_load4(dst + h * kHalf, map, h * 64, hk, ks & (p.block_size - 1), b[0], bar);
      }
      if (cut) {
        wait(kVCut + stg, (landed >> stg) & 1);
        if (!ok) break;
        landed ^= 1 << stg;
        if (tidy_values<T, H>(tile, kbase, sight, lane) && lane == 0) cur.odd = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kVFull + stg]);
      }
      if (++stg == kStages) stg = 0, par ^= 1;
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
    for (int u = 0; u < kStages; ++u) wait_bounded(&bars[full + u], (par ^ (u < stg ? 0u : 1u)) ^ 1u);
    // (a V tile on its way to the cut barrier; without one this runs into its limit, which costs a loop nothing)
    if (IS_V) wait_bounded(&bars[kVCut + stg], (landed >> stg) & 1);
  }
}

template <typename T, int D, int N, int MODE>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_few_kernel(const __grid_constant__ TcTree p) {
  using L = Layout<D, N>;
  constexpr int H = L::kHalves, kKStages = L::kKStages, kVStages = L::kVStages, kItemRing = L::kItemRing;
  constexpr int kWarps = 16;               // of the softmax
  constexpr int C = N / 4;                 // columns of a softmax thread
  // whole swizzle atoms, at an address known when linked
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* gbase = smem_raw;
  const uint32_t base = smem_u32(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + L::kBar);
  const TreePlan& pl = p.plan;
  const int warp = __shfl_sync(FULL_MASK, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // known to be uniform

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int arrivals = 1;
      if (i >= kSRead && i < kPVDone) arrivals = kWarps;               // S^T read, weights
      if (i == kOFree) arrivals = kWarps;
      if (i >= kItemFree && i < kDrain) arrivals = kWarps + 3;
      mbar_init(&bars[i], arrivals);
    }
    fence_mbar_init();
    *reinterpret_cast<uint32_t*>(gbase + L::kGaveUp) = 0;
  }
  // a Q tile's rows past its G * tile_tokens: no copy writes them, they stay zero
  for (int i = pl.group * p.tile_tokens * 8 + (int)threadIdx.x; i < N * 8; i += kTreeThreads)
    for (int t = 0; t < L::kQBufs * H; ++t) st_shared_v4(base + L::kQ + t * L::kQHalf + i * 16, make_uint4(0u, 0u, 0u, 0u));
  fence_proxy_async_smem();
  if (warp == kMmaWarp) tmem_alloc(base + L::kBar + kTmemSlot, kFewCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL_MASK, *reinterpret_cast<volatile uint32_t*>(gbase + L::kBar + kTmemSlot), 0);

  // (what the kernel before leaves is waited for where it is used)
  Item* ring_items = reinterpret_cast<Item*>(gbase + L::kItems);
  if (pl.planned) pdl_wait();

  // registers: 512 x 104 + 128 x 56 = 60416 of the 61440 that 640 threads start with
  if (warp >= kWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == kKvWarp) {
    copy_tiles<T, L, false>(p, bars, base, ring_items, lane);
  } else if (warp == kVWarp) {
    copy_tiles<T, L, true>(p, bars, base, ring_items, lane);
  } else if (warp == kQWarp) {
    tree_segments<L>(p, bars, base, gbase, lane);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA
    // S^T(n), n counting all tiles: Q and K have landed and S^T(n - 2), in the
    // same columns, was read.  PV(n): the weights, V, and for a segment's first
    // one the O^T of the segment before was read.  The whole warp walks through
    // this and one elected thread issues.
    pdl_wait();          // (no bounded wait may run while the kernel before does)
    const bool leader = elect_one();
    constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    constexpr uint32_t id_s = tc_idesc(fmt, N, 0), id_pv = tc_idesc(fmt, N, 1) | (1u << 15), hi = desc_hi(1024);
    const uint32_t o_cols = tmem + kColO, pd = desc_lo(base + L::kP, kHalf);
    bool ok = true;
    auto wait = [&](int bar, uint32_t parity) {
      if (ok) ok = __all_sync(FULL_MASK, wait_bounded(&bars[bar], parity));
    };
    int n = 0, used[2] = {0, 0};                   // tiles of all segments; uses of the Q buffers
    int kstg = 0, vstg = 0;
    uint32_t kpar = 0, vpar = 0;
    for (int r = 0; ok; ++r) {
      ok = __all_sync(FULL_MASK, wait_item(&bars[kItemFull + r % kItemRing], (r / kItemRing) & 1));
      if (!ok) break;
      const Item& it = ring_items[r % kItemRing];
      const int all = __shfl_sync(FULL_MASK, it.n, 0);
      if (all < 0) break;
      const int qbuf = __shfl_sync(FULL_MASK, it.qbuf, 0);
      const uint32_t qd = desc_lo(base + L::kQ + qbuf * H * L::kQHalf, 16);
      auto scores = [&](int m, bool last) {        // S^T(m)
        wait(kKFull + kstg, kpar);
        if (m > 1) wait(kSRead + (m & 1), ((m >> 1) - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t kd = desc_lo(base + L::kK + kstg * H * kHalf, 16), d = tmem + (m & 1) * 64;
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t ko = ((k >> 2) * kHalf + (k & 3) * 32) >> 4, qo = ((k >> 2) * L::kQHalf + (k & 3) * 32) >> 4;
            if (k == 0) mma_ss<false>(d, kd, qd, hi, id_s);
            else mma_ss<true>(d, kd + ko, qd + qo, hi, id_s);
          }
          tc_commit(&bars[kSFull + (m & 1)]);
          tc_commit(&bars[kKEmpty + kstg]);
          if (last) tc_commit(&bars[kQEmpty + qbuf]);
        }
        __syncwarp();
        if (++kstg == kKStages) kstg = 0, kpar ^= 1;
      };
      wait(kQFull + qbuf, used[qbuf] & 1);
      ++used[qbuf];
      scores(n, all == 1);
      for (int j = 0; ok && j < all; ++j, ++n) {
        if (j + 1 < all) scores(n + 1, j + 2 == all);
        wait(kVFull + vstg, vpar);
        if (j == 0 && r > 0) wait(kOFree, (r - 1) & 1);
        wait(kPFull, n & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t vd = desc_lo(base + L::kV + vstg * H * kHalf, kHalf);
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTcKeys / 16; ++k)           // 16 keys = 2048 bytes of either operand
            mma_ss_if(o_cols, vd + k * 128, pd + k * 128, hi, id_pv, k > 0 ? 1u : (uint32_t)j);
          tc_commit(&bars[kPVDone]);
          tc_commit(&bars[kVEmpty + vstg]);
        }
        __syncwarp();
        if (++vstg == kVStages) vstg = 0, vpar ^= 1;
      }
      __syncwarp();
      if (ok && leader) mbar_arrive(&bars[kItemFree + r % kItemRing]);
    }
    if (!ok && leader) flag_error(p.err, PKVD_ERR_TIMEOUT);
    if (leader) tc_commit(&bars[kDrain]);         // every product issued is done when the CTA leaves
    wait_bounded(&bars[kDrain], 0);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    pdl_wait();
    pdl_trigger();
    // ------------------------------------------------------------ softmax
    // Every wait is bounded.  The warps meet at a named barrier, which does not
    // give up, but always brings all: each passes the same ones, a last one when
    // it leaves, where one that gave up asks, so that all learn of it and leave.
    const int quarter = warp & 3, c0 = (warp >> 2) * C, krow = quarter * 32 + lane, me = threadIdx.x;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + c0, o_addr = s_addr + kColO;
    const uint32_t p_row = base + L::kP;
    float* ref = reinterpret_cast<float*>(gbase + L::kRef);
    float* neg = reinterpret_cast<float*>(gbase + L::kNeg);
    int* pos = reinterpret_cast<int*>(gbase + L::kPos);
    float* slope = reinterpret_cast<float*>(gbase + L::kSlope);
    // while the weights' buffer is free: the largest scores and rescaling factors
    // of a new reference; the sums at the end
    int* most_of = reinterpret_cast<int*>(gbase + L::kP);
    float* alpha_of = reinterpret_cast<float*>(gbase + L::kP + 256);
    float* sums = reinterpret_cast<float*>(gbase + L::kP);                                   // [4][64]
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
    volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(gbase + L::kGaveUp);
    bool told = false;
    auto vote = [&](bool mine) -> bool {         // any thread's?
      uint32_t any;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
          "barrier.cta.red.or.pred p, 1, 512, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(any)
          : "r"((uint32_t)mine)
          : "memory");
      return any != 0;
    };
    auto meet = [&] {                            // where nobody asks for anything: one that does gave up
      if (vote(false)) ok = false, told = true;
    };
    // How far a score may pass its reference before that moves.  bf16 weights
    // have fp32's range: 2^24 times 2^23 keys and values of 2^80 stay within it.
    // f16 ones end at 2^16 and are normal from 2^-14 on: the first tile's
    // reference lies 3 below its largest score (later tiles usually have larger
    // ones), a later one 7, so weights keep their bits down to 2^-17 of the row's
    // largest at least.
    constexpr bool kNarrow = std::is_same<T, __half>::value;
    constexpr float kLift = kNarrow ? 7.f : 0.f, kFirst = kNarrow ? 4.f : 0.f, kLimit = kNarrow ? 15.f : 24.f;
    int n = 0;                                   // tiles so far, of all segments
    for (int r = 0; ok; ++r) {
      ok = __all_sync(FULL_MASK, wait_item(&bars[kTreeFull + r % kItemRing], (r / kItemRing) & 1));
      if (!ok) break;
      const Item& it = ring_items[r % kItemRing];
      if (it.n < 0) break;
      // (the shuffles: known to be uniform, and so is what the masks make of a tile)
      auto uniform = [](int x) { return __shfl_sync(FULL_MASK, x, 0); };
      const int all = uniform(it.n), cached = uniform(it.cached), slot = uniform(it.slot);
      const int lo = uniform(it.lo), hi = uniform(it.hi), live = uniform(it.tokens * pl.group);
      // keys before this one may lie before some row's window (no position is past hi)
      const int wr_most = window_first(hi + 1, pl.window);
      const uint32_t* rows_of = reinterpret_cast<const uint32_t*>(gbase + L::kTree + (r % kItemRing) * kTreeBytes);
      const uint8_t* depth_of = reinterpret_cast<const uint8_t*>(rows_of) + 512;
      if (me < N) {
        const int c = min(me, live - 1), t = c / pl.group;
        ref[me] = -INFINITY;
        neg[me] = me < live ? kNoRef : -kNoRef;                // (no column: its scores never ask)
        most_of[me] = ordered(-INFINITY);
        if ((MODE & kBias) || pl.window > 0) {
          pos[me] = cached + depth_of[t];
          slope[me] = bias_slope(p.mod, it.hk * pl.group + c - t * pl.group);
        }
      }
      meet();
      if (!ok) break;
      const uint32_t mine = span_bits(0, live - c0);           // this thread's columns that are rows
      float l[C], less[C];                 // sums of weights; what is added to a column's scores (neg)
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] = 0.f, less[c] = 0.f;
      const int kt_last = uniform(it.kt_last), late = uniform(it.late);
      for (int j = 0; j < all; ++j, ++n) {
        const int kbase = tile_at(kt_last, all, late, j) * kTcKeys;
        const int buf = n & 1, key = kbase + krow, u = key - cached;
        const bool cut = kbase < lo || kbase + kTcKeys - 1 > hi;             // keys that no row sees
        const bool tree = kbase + kTcKeys > cached;                          // drafted ones among them
        const bool edge = pl.window > 0 && kbase < wr_most;
        const bool seen = !cut || (key >= lo && key <= hi);
        // which of its columns see this thread's key, and the key's position
        uint32_t see = seen ? mine : 0u;
        int at = key;
        if (tree || edge) {
          if (u >= 0 && seen) {
            see &= rows_of[u * 2 + c0 / 32] >> (c0 & 31);
            if ((MODE & kBias) || edge) at = cached + depth_of[u];
          }
          if (edge) {
            const int oldest = at + pl.window;               // of the positions that see it
#pragma unroll
            for (int c = 0; c < C; c += 4) {
              const int4 q = *reinterpret_cast<const int4*>(pos + c0 + c);
              const uint32_t m = (uint32_t)(q.x < oldest) | (uint32_t)(q.y < oldest) << 1 | (uint32_t)(q.z < oldest) << 2 |
                                 (uint32_t)(q.w < oldest) << 3;
              see &= ~(15u << c) | m << c;
            }
          }
        }
        wait(kSFull + buf, (n >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        float v[C];
        tmem_ld<C>(s_addr + buf * 64, v);
        tmem_ld_wait();
        // raw scores become scores in log2 units
        if (MODE & kCap) {
          // the form is chosen by the scores that count: with what else lies in
          // the stages and in other rows the last bit would change from run to run
#pragma unroll
          for (int c = 0; c < C; ++c) v[c] = (see >> c) & 1u ? v[c] : 0.f;
          float most = 0.f;              // largest square: the polynomial's range
#pragma unroll
          for (int c = 0; c < C; c += 2) odd_poly2<false>(v[c], v[c + 1], f.poly, 0.f, 0.f, most);
          if (!__all_sync(FULL_MASK, most <= p.poly_range)) {
            tmem_ld<C>(s_addr + buf * 64, v);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = tanh_fast(v[c] * p.mod.cap_in) * p.mod.cap_out_log2;
          }
        } else {
#pragma unroll
          for (int c = 0; c < C; c += 2) scale2(v[c], v[c + 1], f.scale);
        }
        tc_fence_before();
        arrive(kSRead + buf);
        if (MODE & kBias) {
#pragma unroll
          for (int c = 0; c < C; ++c) v[c] = fmaf(slope[c0 + c], (float)(pos[c0 + c] - at), v[c]);
        }
        if (cut || tree || edge) {
#pragma unroll
          for (int c = 0; c < C; ++c) v[c] = (see >> c) & 1u ? v[c] : -INFINITY;
        }
        // A segment's first tile has no references yet.  Where all rows see all of
        // it they are the largest scores of 32 of its keys, another quarter of the
        // tile for each quarter of the columns; a score far above asks as usual.
        const bool sample = j == 0 && !(cut || tree || edge);
        if (sample) {
          float most = 0.f;              // lane e: of the e-th column of this quarter
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (quarter == s) {
#pragma unroll
              for (int e = 0; e < C / 4; ++e) {
                const float m = unordered(__reduce_max_sync(FULL_MASK, ordered(v[s * (C / 4) + e])));
                most = lane == e ? m : most;
              }
            }
          const int col = c0 + quarter * (C / 4) + lane;
          if (lane < C / 4 && col < live && most > -INFINITY) {
            const float now = most - kLift + kFirst;
            ref[col] = now;
            neg[col] = -now;
          }
          meet();
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 s = *reinterpret_cast<const float4*>(neg + c0 + c);
            less[c] = s.x, less[c + 1] = s.y, less[c + 2] = s.z, less[c + 3] = s.w;
          }
        }
        bool rebase = j == 0 && !sample;
        float x[C];
        if (!rebase) {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            add2(x[c], x[c + 1], v[c], v[c + 1], less[c], less[c + 1]);
            add2(x[c + 2], x[c + 3], v[c + 2], v[c + 3], less[c + 2], less[c + 3]);
            top = tc_max3(tc_max3(top, x[c], x[c + 1]), x[c + 2], x[c + 3]);
          }
          rebase = vote(top > kLimit);
          if (rebase && *gave_up) ok = false, told = true;     // (the same word for all)
          if (!ok) break;
        }
        if (rebase) {
          // ---- new references for the columns that passed theirs
          if (j > 0) {
            wait(kPVDone, (n - 1) & 1);                        // the weights' buffer and O^T are free
            if (ok) tc_fence_after();
            if (me < N) most_of[me] = ordered(-INFINITY);      // (a segment starts with that)
            meet();
            if (!ok) break;
          }
          int most = 0;                  // lane c: of column c (mod C) over the warp's keys
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int m = __reduce_max_sync(FULL_MASK, ordered(v[c]));
            most = lane % C == c ? m : most;
          }
          if (lane < C) atomicMax(&most_of[c0 + lane], most);
          meet();
          if (!ok) break;
          if (me < N) {
            const float before = ref[me], top_of = unordered(most_of[me]);
            float now = before;
            if (me < live && (before == -INFINITY ? top_of > -INFINITY : top_of - before > kLimit))
              now = top_of - kLift + (j == 0 ? kFirst : 0.f);
            alpha_of[me] = before == -INFINITY ? 1.f : tc_ex2(before - now);
            ref[me] = now;
            if (now > -INFINITY) neg[me] = -now;
          }
          meet();
          if (!ok) break;
          if (j > 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) l[c] *= alpha_of[c0 + c];
            float o[C];
            tmem_ld<C>(o_addr, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] *= alpha_of[c0 + c];
            tmem_st<C>(o_addr, o);
            tmem_st_wait();
            meet();                 // the factors are read before the weights take their place
            if (!ok) break;
          }
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 s = *reinterpret_cast<const float4*>(neg + c0 + c);
            less[c] = s.x, less[c + 1] = s.y, less[c + 2] = s.z, less[c + 3] = s.w;
            add2(x[c], x[c + 1], v[c], v[c + 1], s.x, s.y);
            add2(x[c + 2], x[c + 3], v[c + 2], v[c + 3], s.z, s.w);
          }
        }
        uint32_t pk[C / 2];
#pragma unroll
        for (int c = 0; c < C; c += 2) {
          const float e0 = tc_ex2(x[c]), e1 = tc_ex2(x[c + 1]);
          tc_add2(l[c], l[c + 1], e0, e1);
          pk[c / 2] = Mma<T>::pack(e0, e1);
        }
        if (j > 0 && !rebase) wait(kPVDone, (n - 1) & 1);      // the weights' buffer is free
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < C; c += 8)
          st_shared_v4(p_row + swz(krow, (c0 + c) / 8), make_uint4(pk[c / 2], pk[c / 2 + 1], pk[c / 2 + 2], pk[c / 2 + 3]));
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(kPFull);
      }
      if (!ok) break;
      // a column's sum over the warp's 32 keys: lane i ends up with column i (mod C)
#pragma unroll
      for (int s = 16; s >= C; s >>= 1)
#pragma unroll
        for (int c = 0; c < C; ++c) l[c] += __shfl_xor_sync(FULL_MASK, l[c], s);
#pragma unroll
      for (int s = C / 2; s >= 1; s >>= 1)
#pragma unroll
        for (int c = 0; c < s; ++c) {
          const bool up = lane & s;
          const float keep = up ? l[c + s] : l[c], send = up ? l[c] : l[c + s];
          l[c] = keep + __shfl_xor_sync(FULL_MASK, send, s);
        }
      wait(kPVDone, (n - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      if (lane < C) sums[quarter * 64 + c0 + lane] = l[0];     // (the weights were read)
      meet();
      if (!ok) break;
      // a warp: 32 dims of its columns
      float o[C];
      if (quarter * 32 < D) {
        tmem_ld<C>(o_addr, o);
        tmem_ld_wait();
      }
      tc_fence_before();
      arrive(kOFree);
      if (*static_cast<const volatile int*>(&it.odd) && quarter * 32 < D) {
        odd_keys(p, it, Sight(it, pl.window), kt_last - all + 1, kt_last, [&](int k, const uint16_t* v) {
          const float x = odd_value<T>(v + krow);
          uint32_t see = 0u;
          if (k >= cached) see = rows_of[(k - cached) * 2 + c0 / 32] >> (c0 & 31);
#pragma unroll
          for (int c = 0; c < C; ++c)
            if (k >= cached ? (see >> c) & 1u : pos[c0 + c] < k + pl.window) o[c] += x;
        });
      }
      const int64_t rec0 = (int64_t)slot * pl.unit_rows;
      // lane c: the sum of column c (mod C), then one over it
      const int mycol = c0 + lane % C;
      const float sum = (sums[mycol] + sums[64 + mycol]) + (sums[128 + mycol] + sums[192 + mycol]);
      if (slot >= 0 && quarter == 0 && lane < C && mycol < live) pl.rec_ml[rec0 + mycol] = make_float2(ref[mycol], sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      if (quarter * 32 < D && c0 < live) {
        int t = c0 / pl.group, gi = c0 - t * pl.group;
        const int64_t row_stride = (int64_t)pl.hq * D;
        T* dst = static_cast<T*>(p.out) + (int64_t)(it.q0 + t) * row_stride + ((int64_t)it.hk * pl.group + gi) * D + krow;
        float* rec = pl.rec + (rec0 + c0) * D + krow;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int col = c0 + c;
          if (col >= live) break;
          if (slot >= 0) {
            rec[c * D] = o[c];
          } else {
            *dst = DT<T>::from_f(o[c] * __shfl_sync(FULL_MASK, inv, c));
          }
          dst += D;
          if (++gi == pl.group) gi = 0, dst += row_stride - (int64_t)pl.group * D;
        }
      }
      arrive(kItemFree + r % kItemRing);
      meet();                       // the sums and references are read before the next segment's
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
    tmem_dealloc(tmem, kFewCols);
  }
}

template <typename T, int D, int N, int MODE>
cudaError_t launch_mode(const TcTree& prm, cudaStream_t stream) {
  constexpr int smem = Layout<D, N>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(tree_few_kernel<T, D, N, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_few_kernel<T, D, N, MODE>, dim3((unsigned)prm.plan.grid), dim3(kTreeThreads), smem, stream, prm);
}

template <typename T, int D, int N>
cudaError_t launch_typed(const TcTree& prm, cudaStream_t stream) {
  const bool cap = prm.mod.cap_in != 0.f, bias = prm.mod.slopes != nullptr;
  if (cap && bias) return launch_mode<T, D, N, kCap | kBias>(prm, stream);
  if (bias) return launch_mode<T, D, N, kBias>(prm, stream);
  return cap ? launch_mode<T, D, N, kCap>(prm, stream) : launch_mode<T, D, N, 0>(prm, stream);
}

template <typename T>
cudaError_t launch_rows(const TcTree& prm, int head_dim, int rows, cudaStream_t stream) {
  if (head_dim == 128) return rows <= 32 ? launch_typed<T, 128, 32>(prm, stream) : launch_typed<T, 128, 64>(prm, stream);
  return rows <= 32 ? launch_typed<T, 64, 32>(prm, stream) : launch_typed<T, 64, 64>(prm, stream);
}

}  // namespace

// Units of at most kTreeFewRows rows, calls that tree_tc_supported takes.
cudaError_t launch_tree_few(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
  TcTree prm;
  if (!tree_tc_params(a, plan, plan.unit_tokens, &prm)) return cudaErrorInvalidValue;
  return a.cache.dtype == PKVD_BF16 ? launch_rows<__nv_bfloat16>(prm, a.cache.head_dim, plan.unit_rows, stream)
                                    : launch_rows<__half>(prm, a.cache.head_dim, plan.unit_rows, stream);
}

}  // namespace pkvd
