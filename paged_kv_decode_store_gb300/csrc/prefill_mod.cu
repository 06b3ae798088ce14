// Varlen paged prefill attention with modified scores (score_mod.cuh) on the
// 5th-generation tensor cores: the operation of prefill_tc.cu with
//   s = cap * tanh(scale <q, k> / cap) - slope_h |p - j|
// over the causal window of every row and its sequence's prefix; and without
// any of these where the scale is not positive (prefill_tc.cu takes maxima
// before it scales).
//
// What differs from the plain kernel is the softmax, which is three times as
// long here and would set the pace alone.  So
// * sixteen softmax warps instead of eight: two threads share a query row, each
//   with its half of a tile's keys.  They agree on the row's reference maximum
//   through shared memory (their two warps meet once a tile); the sums are
//   joined once, at the end.
// * the CTAs are persistent: one per SM walks (sequence, KV head, pair of Q
//   tiles) items, the longest sequences first.  The grid is one CTA an item;
//   a running CTA takes the next one over from the CTAs still waiting to start
//   (clusterlaunchcontrol.try_cancel), so the SMs finish together.  The Q
//   producer does that near the end of the item before and hands items over in
//   shared memory; K, V and the next Q tile (TMA, one box of G heads a token)
//   arrive while the previous item is finished; barriers count on across items.
// * keys are taken from the newest backwards, so a distance bias has its
//   largest scores first and the running maximum hardly ever moves.
// * a cap's tanh is a polynomial on the FMA pipe, two keys an instruction, as
//   long as all of a warp's scores are within 0.7 of it; a warp with a larger
//   one reads its scores again and takes the exponential form.
// * bf16 weights have fp32's range: with a cap and no slopes every score lies
//   in [-cap, cap], and while 2^(cap log2 e) is far inside that range no
//   reference is needed at all -- no maximum, no exchange, no rescaling (167
//   instead of 130 us for 8 capped prompts of 1024 tokens with one).
// * weights are rounded to the cache's type for the product with V: its two
//   operands have one type, and a second product for the bits below would
//   double that part.  It costs half a step a weight, as in the plain kernel
//   (error of the capped prompts 2.3e-3 of the result, 1.7e-3 of them the
//   output's own rounding).
//
// Measured: 8 prompts of 1024 tokens, 48 + 8 heads of 128, bf16, capped: 130 us
// (794 TFLOP/s of visible pairs; 281 us with the plain kernel's structure).  Four
// chunks of about 1000 tokens after up to 7168, 64 + 8 heads of 64, f16, bias
// and prefix: 415 us (924 TFLOP/s; 709 us).  Bound: not the tensor pipe (active
// 39 % of the time; leaving out nearly all products saved 1 to 2 %).  At
// head_dim 64 the instructions (issue slots 70 % taken; a scheduler has four
// softmax warps and one of the others, and the slowest scheduler sets the
// pace).  At 128 the chain of a half tile: weights, product, next scores; with
// two Q tiles a CTA there is no TMEM for a second S beside 2 O and 2 S, and the
// next S must wait for the weights that lie in it (taking whichever half is ready, by polling, was
// slower: 174 instead of 160 us).
//
// Warps (20): 0-7 and 8-15 softmax of Q tile 0 and 1 (warp w of a tile: TMEM
// lanes 32 (w % 4) .., keys 64 (w / 4) ..), 16 producer of K and V, 17 and 19
// the products of Q tile 0 and 1 (one warp for both, polling, took 700 to 1400
// clocks a round: beside four busy softmax warps it gets an instruction in about
// every thirteenth clock), 18 items and Q.
// Row = token * G + query head of the group, as in the plain kernel.
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "score_mod.cuh"
#include "tc_softmax.cuh"
#include "tcgen05.cuh"

namespace pkvd {

namespace {

constexpr int kThreads = 640;
constexpr int kTileWarps = 8;         // softmax warps per Q tile (two threads per row)
constexpr int kKvWarp = 16, kMmaWarp = 17, kQWarp = 18, kMmaWarp1 = 19;
constexpr uint32_t kTmemCols = 512;
// TMEM columns: S of tile g at [128 g, 128 g + 128), O of tile g at [256 + g D,
// 256 + g D + D).  head_dim 128: a half's weights overwrite the first 32 of its
// own 64 S columns; head_dim 64: they have [384 + 64 g, 448 + 64 g), so the
// next S may be computed while they are in use.
constexpr uint32_t kColO = 256, kColP64 = 384;
// What a call modifies, known when compiled: the 64 keys of a thread fill its
// registers, and every choice left to them costs instructions in each tile.
enum : int {
  kCap = 1,
  kBias = 2,
  kBounded = 4,        // every score is in [-cap, cap] and its exponential in range: no reference
};
constexpr float kRebase = 8.f;        // re-base the running maximum when it grows by > 2^8
// Largest bias (log2 units) that is put together from parts: their sums round
// at the bias's own size, several times and in the maximum otherwise than in
// the weights, so from 2^22 on a weight would pass f16's range (and from 2^30
// on all of a row could vanish).  Up to 2^14 it is at most a few 2^-10.
constexpr float kLinear = 16384.f;

template <int D>
struct Layout {
  static constexpr int kKStages = D == 64 ? 4 : 3, kVStages = D == 64 ? 4 : 2;
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kQ = 0;                                    // 2 Q tiles
  static constexpr uint32_t kK = kQ + 2 * kHalves * kHalf;
  static constexpr uint32_t kV = kK + kKStages * kHalves * kHalf;
  static constexpr uint32_t kBar = kV + kVStages * kHalves * kHalf;
  static constexpr uint32_t kX = kBar + 512;                           // exchange: 1024 bytes a tile and buffer
  static constexpr int kXBufs = D == 64 ? 2 : 1;
  // at least 120 KB so that one CTA (which holds all TMEM) is resident per SM
  static constexpr uint32_t kItems = kX + kXBufs * 2048;               // ring of items
  static constexpr uint32_t kOrder = kItems + 384;                     // sequences, longest first
  static constexpr uint32_t kGaveUp = kOrder + 64;                     // one word a pair of softmax warps
  static constexpr uint32_t kEnd = kGaveUp + 32;
  static constexpr uint32_t kBytes = kEnd > 122880u ? kEnd : 122880u;
};
static_assert(Layout<128>::kBytes <= 232448, "227 KB of shared memory");

// mbarriers; those of a Q tile take + g, S, P and PV + g + 2 half where a tile's
// halves of keys go their own ways.
enum : int {
  kKFull = 0, kKEmpty = 4, kVFull = 8, kVCut = 12, kVEmpty = 16, kQFull = 20, kQEmpty = 22, kSFull = 24, kPFull = 28,
  kPVDone = 32, kSRead = 36, kOFree = 38, kItemFull = 40, kItemFree = 44, kClaim = 48, kDrain = 49,
  kNear = 51, kNumBars = 52
};
constexpr uint32_t kTmemSlot = 8 * kNumBars;        // the TMEM base, then 16 bytes of a claim's answer
constexpr uint32_t kAnswer = (kTmemSlot + 4 + 15) / 16 * 16;
static_assert(kAnswer + 16 <= 512, "behind the barriers");
constexpr int kItemRing = 4;
constexpr int kSorted = 64;           // sequences that are put in order of length
constexpr int kItemUsers = 3 + 2 * kTileWarps;   // K/V, two MMA and softmax warps

struct ModParams {
  CUtensorMap tmap_q, tmap_k, tmap_v;
  void* out;
  const int32_t* tables;
  int max_blocks;
  int block_size, block_shift;   // a power of two
  uint32_t block_limit;  // num_blocks, at most 2^31
  int seg_rows;          // rows per TMA box of the cache: min(block_size, 128)
  const int32_t* cu_q;
  const int32_t* cu_k;
  int total_q, hq, hkv, group, tile_tokens;
  uint32_t q_box;        // bytes of one 64-column box of a Q tile
  int pairs;             // Q-tile pairs per (sequence, KV head)
  int pair;              // tiles of a pair: 2, or 1 (only tile 1)
  int num_seqs, items;
  int waves;             // more items than SMs: they are put in order (418 us; 424 as they come) and taken
                         // over; fewer: neither (10 to 12 us calls 1 to 2 us shorter)
  float scale_log2;
  int window;
  ScoreMod mod;
  // score of a raw product s as s * polynomial in s^2, for s^2 <= poly_range (-1: not used)
  float poly[4], poly_range;
  int wide_out;          // out is 32-byte aligned: stores of 32 bytes (132 us; 142 in 16)
  int32_t* err;
};

// One item: the keys of a pair of Q tiles.  n = 0: nothing to do, -1: no more.
// K/V tiles are counted from the last one backwards: tile t holds keys
// [kt_last - t, ..) * 128, from tile n_main on `gap` tiles less.  Keys that no
// row sees are not read: those outside [lo, hi] and, between the prefix and the
// window, [hole, hole_end).
struct __align__(16) Item {
  int seq, hk, q0, cached, prefix;
  int tb[2], te[2];      // new tokens of Q tile g (0: the earlier one, may be empty)
  int lo, hi, kt_last, n;
  int gf[2], gn[2];      // first K/V tile and number of tiles of Q tile g
  int n_main, gap, hole, hole_end;
  int pad[3];
  __device__ int tile(int t) const { return kt_last - t - (t >= n_main ? gap : 0); }
};
static_assert(sizeof(Item) * kItemRing == 384, "the ring in Layout");

__device__ __forceinline__ int window_first(int c, int window) { return (window > 0 && c > window) ? c - window : 0; }

// Item i: the sequences in `order` (as they come without it), their pairs from
// the end, KV heads fastest.
__device__ __forceinline__ Item item_at(const ModParams& p, const uint8_t* order, int i) {
  Item t;
  t.n = t.gn[0] = t.gn[1] = 0;
  const int nh = p.hkv, rank = i / (p.pairs * nh), rest = i - rank * (p.pairs * nh);
  const int zpair = rest / nh;
  t.hk = rest - zpair * nh;
  t.seq = order ? order[rank] : rank;
  const int q0 = p.cu_q[t.seq], q1 = p.cu_q[t.seq + 1], k0 = p.cu_k[t.seq], k1 = p.cu_k[t.seq + 1];
  const int qlen = q1 - q0, klen = k1 - k0;
  if (q0 < 0 || qlen < 0 || klen < qlen || q1 > p.total_q || (int64_t)klen > (int64_t)p.max_blocks * p.block_size) {
    if (zpair == 0 && t.hk == 0) flag_error(p.err, PKVD_ERR_CONTEXT);
    return t;
  }
  if (zpair == 0 && t.hk == 0 && qlen > p.pair * p.pairs * p.tile_tokens)
    flag_error(p.err, PKVD_ERR_CONTEXT);   // longer than max_seqlen_q: the earliest tokens are not computed
  t.q0 = q0;
  t.cached = klen - qlen;
  t.prefix = prefix_of(p.mod, t.seq, klen);
  int lo_g[2], hi_g[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    t.te[g] = p.pair == 2 ? qlen - (2 * zpair + 1 - g) * p.tile_tokens : g ? qlen - zpair * p.tile_tokens : 0;
    t.tb[g] = max(0, t.te[g] - p.tile_tokens);
    lo_g[g] = window_first(t.cached + t.tb[g] + 1, p.window);
    hi_g[g] = max(t.cached + t.te[g] - 1, t.prefix - 1);
  }
  if (t.te[1] <= 0) return t;                    // past the sequence's last pair
  t.lo = t.te[0] > 0 ? lo_g[0] : lo_g[1];
  t.hi = hi_g[1];
  t.kt_last = t.hi / kTcKeys;
  t.n = t.n_main = t.kt_last - t.lo / kTcKeys + 1;
  t.gap = t.hole = t.hole_end = 0;
  if (t.prefix > 0) {
    t.hole = t.prefix;
    t.hole_end = t.lo;
    const int last = (t.prefix - 1) / kTcKeys;             // the prefix's last tile
    t.gap = max(0, t.lo / kTcKeys - 1 - last);
    t.n = t.kt_last + 1 - t.gap;
    t.lo = 0;
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    t.gf[g] = t.kt_last - hi_g[g] / kTcKeys;
    t.gn[g] = t.te[g] <= 0 ? 0 : t.prefix > 0 ? t.n - t.gf[g] : hi_g[g] / kTcKeys - lo_g[g] / kTcKeys + 1;
  }
  return t;
}

// Ask for a CTA that has not started, in its place: 16 bytes at `dst`, counted
// on `bar`; and its index, -1 if there is none left (then not to be asked
// again).
__device__ __forceinline__ void claim(uint32_t dst, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
      "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ int claimed(uint32_t src) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b64 lo, hi;\n\t"
      "ld.shared.v2.b64 {lo, hi}, [%1];\n\t"
      "mov.b128 h, {lo, hi};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
      : "=r"(x)
      : "r"(src)
      : "memory");
  return x;
}


// A thread's visible columns: [lo, end) of its 64, and those below `prefix`.
struct Visible {
  int lo, end, prefix;
  __device__ uint32_t bits(int word) const {
    return span_bits(lo - 32 * word, end - 32 * word) | span_bits(0, prefix - 32 * word);
  }
  // Everything else becomes `x`, whatever it was (masked keys may hold
  // anything).  Most groups of eight columns are visible to the whole warp,
  // also in a tile that the mask cuts.
  template <int N>
  __device__ void hide(float (&v)[N], float x) const {
#pragma unroll
    for (int w = 0; w < N / 32; ++w) {
      const uint32_t m = bits(w), every = __reduce_and_sync(FULL_MASK, m);
#pragma unroll
      for (int c8 = 0; c8 < 32; c8 += 8) {
        if (((every >> c8) & 0xffu) == 0xffu) continue;
#pragma unroll
        for (int c = c8; c < c8 + 8; ++c) v[32 * w + c] = ((m >> c) & 1u) ? v[32 * w + c] : x;
      }
    }
  }
};

// A thread's 64 raw scores become scores in log2 units, -inf where the mask
// leaves a column out, up to a part of the bias that is the same for eight
// columns: column c's score is v[c] + base + (c / 8) * step.  A bias that
// falls linearly (no key after any of the warp's rows) then costs nothing per
// key: eight multiples of the slope ride on the last product, the rest joins
// the reference that the exponent subtracts anyway.  A large bias (kLinear) is
// added to each score in one rounding instead.  The same for the whole
// warp: `whole`, every row sees every column, and `linear`.  `range`: of the
// polynomial, in squares of the raw score.  `off`: the first column's
// key minus the row's position; `again` reads the raw scores once more (a
// warp with a score past the polynomial's range: it has computed in vain).
template <int MODE, int N, typename Again>
__device__ __forceinline__ void modify(float (&v)[N], const ModParams& p, const Factors& f, const Visible& see,
                                       bool whole, bool linear, float range, float nslope, int off, float& base,
                                       float& step, Again again) {
  const ScoreMod& m = p.mod;
  float k[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) k[i] = (linear ? -nslope : 0.f) * (float)i;
  base = linear ? nslope * (float)-off : 0.f;
  step = linear ? -nslope * 8.f : 0.f;
  if (MODE & kCap) {
    // the form is chosen by the scores that count: with what else lies in the
    // stages and in other rows the last bit would change from run to run
    if (!whole) see.hide(v, 0.f);
    float most = 0.f;                  // largest square: the polynomial's range
#pragma unroll
    for (int c = 0; c < N; c += 2)
      odd_poly2<(MODE & kBias) != 0>(v[c], v[c + 1], f.poly, k[c & 7], k[(c & 7) + 1], most);
    if (!__all_sync(FULL_MASK, most <= range)) {
      again(v);
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = fmaf(tanh_fast(v[c] * m.cap_in), m.cap_out_log2, k[c & 7]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      if (MODE & kBias)
        scale_add2(v[c], v[c + 1], f.scale, k[c & 7], k[(c & 7) + 1]);
      else
        scale2(v[c], v[c + 1], f.scale);
    }
  }
  if ((MODE & kBias) && !linear) {
    const float first = (float)off;
#pragma unroll
    for (int c = 0; c < N; ++c) v[c] = fmaf(nslope, fabsf(first + (float)c), v[c]);
  }
  if (!whole) see.hide(v, -INFINITY);
}

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) prefill_mod_kernel(const __grid_constant__ ModParams p) {
  using L = Layout<D>;
  constexpr int H = L::kHalves, kKStages = L::kKStages, kVStages = L::kVStages;
  constexpr bool kSepP = D == 64;
  // head_dim 128 without a reference: nothing ties the two halves of a tile's
  // keys together, so each has its own S, P and PV and the products of one run
  // beside the softmax of the other (132 us; 142 together).
  constexpr bool kSplit = D == 128 && (MODE & kBounded);
  // whole swizzle atoms; an address known when linked keeps the barriers' out
  // of the loops (rounded up at run time: 475 instead of 468 us for four chunks
  // of 1000 tokens after up to 7168)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* gbase = smem_raw;
  const uint32_t base = smem_u32(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + L::kBar);
  const int warp = __shfl_sync(FULL_MASK, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // known to be uniform

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int arrivals = 1;
      if (i >= kPFull && i < kPVDone) arrivals = kSplit ? kTileWarps / 2 : kTileWarps;
      if (i >= kSRead && i < kItemFull) arrivals = kTileWarps;
      if ((i >= kKEmpty && i < kVFull) || (i >= kVEmpty && i < kQFull)) arrivals = 2;      // both Q tiles
      if (i >= kItemFree && i < kClaim) arrivals = kItemUsers;
      mbar_init(&bars[i], arrivals);
    }
    fence_mbar_init();
  }
  if (threadIdx.x < 8) reinterpret_cast<uint32_t*>(gbase + L::kGaveUp)[threadIdx.x] = 0;
  // a Q tile's rows past its G * tile_tokens: no copy writes them, they stay zero
  for (int i = p.group * p.tile_tokens * 8 + (int)threadIdx.x; i < kTcRows * 8; i += kThreads)
    for (int t = 0; t < 2 * H; ++t) st_shared_v4(base + L::kQ + t * kHalf + i * 16, make_uint4(0u, 0u, 0u, 0u));
  fence_proxy_async_smem();
  if (warp == kMmaWarp) tmem_alloc(base + L::kBar + kTmemSlot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL_MASK, *reinterpret_cast<volatile uint32_t*>(gbase + L::kBar + kTmemSlot), 0);

  pdl_wait();      // the cache rows of this step come from the store kernel
  pdl_trigger();
  Item* ring_items = reinterpret_cast<Item*>(gbase + L::kItems);

  // registers: 512 x 104 + 128 x 56 = 60416 of the 61440 that 640 threads start with
  if (warp >= kKvWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == kKvWarp) {
    // ------------------------------------------------------- K and V producer
    // Lane s copies segment s of a tile; K runs kAhead tiles ahead of V.  A V
    // tile with rows that are not read lands on a barrier of its own (kVCut)
    // and is released with those rows zeroed, so that they never weigh in.
    // Every instruction here is one that the softmax warps of the same
    // scheduler do not get, and they set the pace (with divisions, a barrier and
    // some votes more a tile: 500 instead of 445 us for the four chunks).
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
      wait(kItemFull + r % kItemRing, (r / kItemRing) & 1);
      if (!ok) break;
      const Item& cur = ring_items[r % kItemRing];
      if (cur.n < 0) break;
      const int32_t* table = p.tables + (int64_t)cur.seq * p.max_blocks;
      const int n = cur.n, hk = cur.hk, lo = cur.lo, hi = cur.hi, hole = cur.hole, hole_end = cur.hole_end;
      const int kt_last = cur.kt_last, n_main = cur.n_main, gap = cur.gap, near = max(0, n - 1 - kAhead);
      auto tile_of = [&](int t) { return kt_last - t - (t >= n_main ? gap : 0); };
      auto key_of = [&](int t) { return tile_of(t) * kTcKeys + lane * p.seg_rows; };
      auto is_read = [&](int ks) {
        return lane < nseg && ks <= hi && ks + p.seg_rows - 1 >= lo && !(ks >= hole && ks + p.seg_rows <= hole_end);
      };
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
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < n) copy_k(i, b[i]);
      for (int t = 0; ok && t < n; ++t) {
        if (t + kAhead < n) copy_k(t + kAhead, b[kAhead]);
        if (lane == 0 && t == near) mbar_arrive(&bars[kNear]);
        wait(kVEmpty + vstg, vpar);
        if (!ok) break;
        const int kbase = tile_of(t) * kTcKeys;
        const bool cut = kbase < lo || kbase + kTcKeys - 1 > hi || max(kbase, hole) < min(kbase + kTcKeys, hole_end);
        const uint32_t dst = base + L::kV + vstg * H * kHalf;
        copy(&p.tmap_v, dst, (cut ? kVCut : kVFull) + vstg, kbase + lane * p.seg_rows, hk, b[0], is_read);
        if (cut) {
          wait(kVCut + vstg, (landed >> vstg) & 1);
          if (!ok) break;
          landed ^= 1 << vstg;
          for (int rr = lane; rr < kTcKeys; rr += 32) {
            const int kp = kbase + rr;
            if (kp >= lo && kp <= hi && !(kp >= hole && kp < hole_end)) continue;
            for (int h = 0; h < H; ++h)
              for (int c = 0; c < 8; ++c) st_shared_v4(dst + h * kHalf + rr * 128 + c * 16, make_uint4(0u, 0u, 0u, 0u));
          }
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
  } else if (warp == kQWarp) {
    // ------------------------------------------------- items and Q producer
    // The next item is claimed once the K/V producer comes to the end of the
    // one before (earlier it would wait behind the rest of this CTA's item while
    // another CTA runs out of them: 160 instead of 154 us for 1600 items of one
    // to eight tiles); empty ones are left out, -1 ends the list.  A tile's rows are one box per 64 columns (G heads of
    // tile_tokens tokens), loaded once the tensor cores are done with the item
    // before.
    uint8_t* order = p.waves && p.num_seqs <= kSorted ? gbase + L::kOrder : nullptr;
    if (order) {                                 // a sequence's place: how many are longer, or as long and before it
      for (int i = lane; i < p.num_seqs; i += 32) {
        const int len = p.cu_k[i + 1] - p.cu_k[i];
        int before = 0;
        for (int j = 0; j < p.num_seqs; ++j) {
          const int other = p.cu_k[j + 1] - p.cu_k[j];
          before += other > len || (other == len && j < i);
        }
        order[before] = (uint8_t)i;
      }
      __syncwarp();
    }
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_q)) : "memory");
      bool ok = true, own = true;                // first the CTA's own item
      int made = 0, asked = 0, used[2] = {0, 0}, next = blockIdx.x;
      auto make = [&] {                          // the next item into the ring
        const int slot = made % kItemRing;
        if (made > 0) ok = wait_item(&bars[kNear], (made - 1) & 1);
        if (made >= kItemRing) ok = ok && wait_bounded(&bars[kItemFree + slot], ((made / kItemRing) - 1) & 1);
        Item it;
        it.n = 0;
        while (ok && it.n == 0) {
          if (!own && !p.waves) {
            next = -1;
          } else if (!own) {
            fence_proxy_async_smem();            // the last answer has been read
            mbar_arrive_expect_tx(&bars[kClaim], 16);
            claim(base + L::kBar + kAnswer, &bars[kClaim]);
            ok = wait_bounded(&bars[kClaim], asked & 1);
            ++asked;
            if (!ok) break;
            next = claimed(base + L::kBar + kAnswer);
          }
          own = false;
          if (next < 0) it.n = -1;
          else it = item_at(p, order, next);
        }
        if (!ok) return;
        ring_items[slot] = it;
        mbar_arrive(&bars[kItemFull + slot]);
        ++made;
      };
      for (int r = 0; ok; ++r) {
        make();
        if (!ok) break;
        const Item it = ring_items[r % kItemRing];
        if (it.n < 0) break;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!ok || it.gn[g] == 0) continue;
          if (used[g] > 0) ok = wait_bounded(&bars[kQEmpty + g], (used[g] - 1) & 1);
          if (!ok) continue;
          mbar_arrive_expect_tx(&bars[kQFull + g], p.q_box * H);
          for (int h = 0; h < H; ++h)
            tma_load3(base + L::kQ + (g * H + h) * kHalf, &p.tmap_q, h * 64, it.hk * p.group, it.q0 + it.tb[g],
                      &bars[kQFull + g]);
          ++used[g];
        }
      }
      if (!ok) flag_error(p.err, PKVD_ERR_TIMEOUT);
      for (int g = 0; g < 2; ++g)                // no copy is in flight when the CTA leaves
        if (used[g] > 0) wait_bounded(&bars[kQFull + g], (used[g] - 1) & 1);
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp1) {
    // ---------------------------------------------------------------- MMA
    // S(n) of the Q tile, n counting all its K tiles: Q and K have landed and
    // its S columns are free (head_dim 64: S(n - 1) was read; 128: PV(n - 1)
    // is done, its weights lie there).  PV(n): the weights, V, and for an
    // item's first one the O columns of the item before were read.  A K or V
    // stage is free when both Q tiles are done with it; a tile that this one
    // does not use it waits for all the same, so that no phase of a stage is
    // waited for before the one before it is over.
    //
    // The whole warp walks through this and one elected thread issues: a
    // product takes its operands from uniform registers, which the compiler
    // fills directly where everything is known to be the same in all lanes
    // (hence the shuffles).  In a branch of one lane every operand was moved
    // there for every product, 200 to 300 clocks each.
    {
      const bool leader = elect_one();
      const int g = warp == kMmaWarp ? 0 : 1;
      constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t id_s = tc_idesc(fmt, kSplit ? kCols : kTcKeys, 0), id_pv = tc_idesc(fmt, D, 1), hi = desc_hi(1024);
      const uint32_t qd = desc_lo(base + L::kQ + g * H * kHalf, 16);
      const uint32_t s_cols = tmem + g * kTcKeys, o_cols = tmem + kColO + g * D;
      const uint32_t p_cols = kSepP ? tmem + kColP64 + g * 64 : s_cols;
      constexpr int kParts = kSplit ? 2 : 1;
      bool ok = true;
      auto wait = [&](int bar, uint32_t parity) {
        if (ok) ok = __all_sync(FULL_MASK, wait_bounded(&bars[bar], parity));
      };
      int n = 0, used = 0;                          // this tile's K tiles of all items, its items
      int kstg = 0, vstg = 0;                       // next stages and their phases, every tile of every item
      uint32_t kpar = 0, vpar = 0;
      auto next_k = [&] {
        if (++kstg == kKStages) kstg = 0, kpar ^= 1;
      };
      auto next_v = [&] {
        if (++vstg == kVStages) vstg = 0, vpar ^= 1;
      };
      auto skip = [&](int tiles) {                  // that this Q tile does not use
        for (int t = 0; t < tiles; ++t) {
          wait(kKFull + kstg, kpar);
          if (ok && leader) mbar_arrive(&bars[kKEmpty + kstg]);
          next_k();
          wait(kVFull + vstg, vpar);
          if (ok && leader) mbar_arrive(&bars[kVEmpty + vstg]);
          next_v();
        }
      };
      // S of the next K stage: half h or all (0) of its keys
      auto issue_s = [&](int h, bool last) {
        tc_fence_after();
        const uint32_t kd = desc_lo(base + L::kK + kstg * H * kHalf, 16) + h * (kCols * 128 >> 4), d = s_cols + h * kCols;
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
            if (k == 0) mma_ss<false>(d, qd, kd, hi, id_s);
            else mma_ss<true>(d, qd + off, kd + off, hi, id_s);
          }
          tc_commit(&bars[kSFull + g + 2 * h]);
          if (h == kParts - 1) {
            tc_commit(&bars[kKEmpty + kstg]);
            if (last) tc_commit(&bars[kQEmpty + g]);
          }
        }
        __syncwarp();
        if (h == kParts - 1) next_k();
      };
      auto issue_pv = [&](int h, uint32_t add) {    // half h or all of the next V stage
        tc_fence_after();
        const uint32_t vd = desc_lo(base + L::kV + vstg * H * kHalf, kHalf);
        if (leader) {
#pragma unroll
          for (int i = 0; i < kTcKeys / 16 / kParts; ++i) {        // 16 keys = 8 packed columns of weights
            const int k = h * (kTcKeys / 32) + i;
            const uint32_t col = kSepP ? k * 8 : (k >> 2) * kCols + (k & 3) * 8;
            mma_ts(o_cols, p_cols + col, vd + k * 128, hi, id_pv, k > 0 ? 1u : add);
          }
          tc_commit(&bars[kPVDone + g + 2 * h]);
          if (h == kParts - 1) tc_commit(&bars[kVEmpty + vstg]);
        }
        __syncwarp();
        if (h == kParts - 1) next_v();
      };
      for (int r = 0; ok; ++r) {
        wait(kItemFull + r % kItemRing, (r / kItemRing) & 1);
        if (!ok) break;
        const Item& it = ring_items[r % kItemRing];
        const int all = __shfl_sync(FULL_MASK, it.n, 0);
        if (all < 0) break;
        const int gn = __shfl_sync(FULL_MASK, it.gn[g], 0), before = __shfl_sync(FULL_MASK, it.gf[g], 0);
        skip(gn > 0 ? before : all);
        if (gn > 0) {
          // what arrives last (the softmax warps' part) is waited for last
          wait(kQFull + g, used & 1);
          wait(kKFull + kstg, kpar);
#pragma unroll
          for (int h = 0; h < kParts; ++h) {
            if (n > 0) wait((kSepP ? kSRead : kPVDone) + g + 2 * h, (n - 1) & 1);
            if (ok) issue_s(h, gn == 1);
          }
          for (int j = 0; ok && j < gn; ++j, ++n) {
            const bool more = j + 1 < gn;
            if (more) wait(kKFull + kstg, kpar);
            if (kSepP && more) {
              wait(kSRead + g, n & 1);
              if (ok) issue_s(0, j + 2 == gn);
            }
            wait(kVFull + vstg, vpar);
            if (j == 0 && used > 0) wait(kOFree + g, (used - 1) & 1);
#pragma unroll
            for (int h = 0; h < kParts; ++h) {
              wait(kPFull + g + 2 * h, n & 1);
              if (ok) issue_pv(h, j);
              if (!kSepP && more) {
                wait(kPVDone + g + 2 * h, n & 1);
                if (ok) issue_s(h, j + 2 == gn);
              }
            }
          }
          ++used;
          skip(all - before - gn);
        }
        __syncwarp();
        if (leader) mbar_arrive(&bars[kItemFree + r % kItemRing]);
      }
      if (!ok && leader) flag_error(p.err, PKVD_ERR_TIMEOUT);
      if (leader) tc_commit(&bars[kDrain + g]);   // every product issued is done when the CTA leaves
      wait_bounded(&bars[kDrain + g], 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ------------------------------------------------------------ softmax
    // Every wait is bounded; a warp whose wait gives up leaves (the others'
    // then give up in turn).  The two warps of a quarter of the rows meet at a
    // named barrier, which does not give up, but always brings both: each passes
    // the same ones, a last one when it leaves, and one that gave up says so at
    // their next meeting, where both leave.  (An mbarrier, with its arrival and
    // its wait, took 435 instead of 420 us for the four chunks.)
    const int g = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int sub = g + (kSplit ? 2 * half : 0);   // which S, P and PV
    const uint32_t s_addr = tmem + lane_base + g * kTcKeys + half * kCols;
    const uint32_t p_addr = kSepP ? tmem + lane_base + kColP64 + g * 64 + half * 32 : s_addr;
    const uint32_t o_addr = tmem + lane_base + kColO + g * D + half * (D / 2);
    // what a row's two threads tell each other: 256 bytes a quarter of the rows
    float* xch = reinterpret_cast<float*>(gbase + L::kX + g * 1024 + quarter * 256);
    float* xsum = xch;
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
    auto exchange = [&] {                        // what the row's two warps wrote is readable by both
      asm volatile("bar.sync %0, 64;" ::"r"(1 + g * 4 + quarter) : "memory");
      if (*gave_up) ok = false, told = true;     // the same word in every lane
    };
    int n = 0;                                   // this tile's K tiles so far, of all items
    for (int r = 0; ok; ++r) {
      ok = __all_sync(FULL_MASK, wait_item(&bars[kItemFull + r % kItemRing], (r / kItemRing) & 1));
      if (!ok) break;
      const Item& it = ring_items[r % kItemRing];
      if (it.n < 0) break;
      // (the shuffles: known to be uniform, and so is what the masks make of a tile)
      auto uniform = [](int x) { return __shfl_sync(FULL_MASK, x, 0); };
      const int tb = uniform(it.tb[g]), te = uniform(it.te[g]), gf = uniform(it.gf[g]), gn = uniform(it.gn[g]);
      if (gn == 0) {
        arrive(kItemFree + r % kItemRing);
        continue;
      }
      const int prefix = uniform(it.prefix);
      const bool live = row < (te - tb) * p.group;
      const int tt = live ? row / p.group : 0, gi = live ? row - tt * p.group : 0;
      const int pr = it.cached + tb + tt;        // padding rows mirror row 0
      const int wr = window_first(pr + 1, p.window);
      const int pr_min = __reduce_min_sync(FULL_MASK, pr), wr_max = __reduce_max_sync(FULL_MASK, wr);
      const int pr_max = __reduce_max_sync(FULL_MASK, pr), wr_min = __reduce_min_sync(FULL_MASK, wr);
      const float nslope = bias_slope(p.mod, it.hk * p.group + gi);
      int near = 0;                              // the first key whose bias may be put together from parts (kLinear)
      if (MODE & kBias) {
        const float steepest = __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(fabsf(nslope))));
        near = uniform(pr_max - (int)fminf(kLinear / steepest, 1e9f));
      }
      const float range = live ? p.poly_range : INFINITY;   // padding rows have no say
      float m_ref = (MODE & kBounded) ? 0.f : -INFINITY, l = 0.f;
      int kbase = uniform(it.tile(gf)) * kTcKeys + half * kCols;
      const int jump = uniform(it.n_main) - gf, gap = uniform(it.gap) * kTcKeys;
      for (int j = 0; j < gn; ++j, ++n, kbase -= kTcKeys) {
        if (j == jump && j > 0) kbase -= gap;     // (a first tile behind the gap: tile() knows)
        wait(kSFull + sub, n & 1);
        if (!ok) break;
        tc_fence_after();
        if constexpr ((MODE & kBounded) != 0) {
          // nothing is needed of the whole row before its weights: 32 keys at a
          // time, in a loop of half the code
#pragma unroll 1
          for (int c0 = 0; c0 < kCols; c0 += 32) {
            uint32_t pk[16];
            const int k0 = kbase + c0;
            if ((k0 > pr_max || k0 + 31 < wr_min) && k0 >= prefix) {       // no row sees any
#pragma unroll
              for (int c = 0; c < 16; ++c) pk[c] = 0u;
            } else {
              float v[32], bias, step, s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
              auto read = [&](float (&x)[32]) {
                tmem_ld32(s_addr + c0, x);
                tmem_ld_wait();
              };
              read(v);
              const bool whole = (k0 + 31 <= pr_min && k0 >= wr_max) || k0 + 32 <= prefix;
              modify<MODE>(v, p, f, Visible{wr - k0, pr + 1 - k0, prefix - k0}, whole, false, range, 0.f, 0, bias, step, read);
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const float e0 = tc_ex2(v[c]), e1 = tc_ex2(v[c + 1]), e2 = tc_ex2(v[c + 2]), e3 = tc_ex2(v[c + 3]);
                tc_add2(s0, s1, e0, e1);
                tc_add2(s2, s3, e2, e3);
                pk[c / 2] = Mma<T>::pack(e0, e1);
                pk[c / 2 + 1] = Mma<T>::pack(e2, e3);
              }
              l += (s0 + s1) + (s2 + s3);
            }
            if (kSepP && c0 == 0 && j > 0) {
              wait(kPVDone + g, (n - 1) & 1);
              tc_fence_after();
            }
            tmem_st16(p_addr + c0 / 2, pk);
          }
          if (kSepP) {
            tc_fence_before();
            arrive(kSRead + g);
          }
        } else {
          float v[kCols];
          auto read = [&](float (&x)[kCols]) {
            tmem_ld32(s_addr, x);
            tmem_ld32(s_addr + 32, x + 32);
            tmem_ld_wait();
          };
          read(v);
          float bias, step;
          const bool before = kbase + kCols - 1 <= pr_min;
          const bool whole = (before && kbase >= wr_max) || kbase + kCols <= prefix;
          const bool linear = (MODE & kBias) && before && kbase >= near;
          modify<MODE>(v, p, f, Visible{wr - kbase, pr + 1 - kbase, prefix - kbase}, whole, linear, range,
                       nslope, kbase - pr, bias, step, read);
          // head_dim 64: the next S may overwrite these columns once nobody reads them again
          if (kSepP) {
            tc_fence_before();
            arrive(kSRead + g);
          }
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kCols; c += 8) {
            if ((MODE & kBias) && c > 0) top -= step;          // relative to the bias of these eight columns
            top = tc_max3(tc_max3(top, v[c], v[c + 1]), tc_max3(v[c + 2], v[c + 3], v[c + 4]),
                          tc_max3(v[c + 5], v[c + 6], v[c + 7]));
          }
          if (MODE & kBias) top += bias + (kCols / 8 - 1) * step;
          // the two halves of a row agree on a reference, the larger maximum to
          // all its bits: rounded up to 16 of them it would lie 2^-8 of a score
          // above it, which at thousands is more than the weights' exponents have
          float* x = xch + (kSepP ? (n & 1) * 512 : 0);
          x[half * 32 + lane] = top;
          exchange();
          if (!ok) break;
          const float mt = fmaxf(top, x[(half ^ 1) * 32 + lane]);
          // f16 weights are normal down to 2^-14: with the reference 7 below the
          // largest score they have seven bits more before they lose any (2^15 at
          // most, as the reference lets scores grow by 2^8), and many small ones
          // beside a large one add up to what they are
          constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;
          // (the difference is exact where it counts; the sum m_ref + 15 is not from 2^24 on)
          const bool rebase = mt - m_ref > kLift + kRebase;
          const bool scale_o = rebase && m_ref != -INFINITY;
          const float alpha = scale_o ? tc_ex2(m_ref - (mt - kLift)) : 1.f;
          if (rebase) m_ref = mt - kLift;
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          uint32_t pk[kCols / 2];
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f, shift0 = bias - mu, shift1 = shift0;
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            if ((MODE & kBias) && c > 0 && c % 8 == 0) tc_add2(shift0, shift1, step, step);
            tc_add2(v[c], v[c + 1], shift0, shift1);
            tc_add2(v[c + 2], v[c + 3], shift0, shift1);
            const float e0 = tc_ex2(v[c]), e1 = tc_ex2(v[c + 1]), e2 = tc_ex2(v[c + 2]), e3 = tc_ex2(v[c + 3]);
            tc_add2(s0, s1, e0, e1);
            tc_add2(s2, s3, e2, e3);
            pk[c / 2] = Mma<T>::pack(e0, e1);
            pk[c / 2 + 1] = Mma<T>::pack(e2, e3);
          }
          l = l * alpha + ((s0 + s1) + (s2 + s3));
          if (kSepP && j > 0) {                    // the weights' columns are free once PV(n - 1) is done
            wait(kPVDone + g, (n - 1) & 1);
            tc_fence_after();
          }
          if (__any_sync(FULL_MASK, scale_o)) {    // O too (head_dim 128: PV(n - 1) was done before S(n))
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
          tmem_st32(p_addr, reinterpret_cast<const float*>(pk));
        }
        tmem_st_wait();
        tc_fence_before();
        arrive(kPFull + sub);
      }
      if (!ok) break;
      wait(kPVDone + g + (kSplit ? 2 : 0), (n - 1) & 1);   // the last; and so every warp of the tile is past its last exchange
      if (!ok) break;
      tc_fence_after();
      // the row's sum: half 1's part to half 0, the whole back
      if (half == 1) xsum[lane] = l;
      exchange();
      if (!ok) break;
      if (half == 0) {
        l += xsum[lane];
        xsum[lane] = l;
      }
      exchange();
      if (!ok) break;
      if (half == 1) l = xsum[lane];
      const float inv = l > 0.f ? 1.f / l : 0.f;
      T* dst = static_cast<T*>(p.out) + ((int64_t)(it.q0 + tb + tt) * p.hq + (int64_t)it.hk * p.group + gi) * D +
               half * (D / 2);
#pragma unroll
      for (int c4 = 0; c4 < D / 64; ++c4) {
        float o[32];
        tmem_ld32(o_addr + c4 * 32, o);
        tmem_ld_wait();
        if (c4 == D / 64 - 1) {
          tc_fence_before();
          arrive(kOFree + g);
        }
        if (live) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            mul2(o[2 * e], o[2 * e + 1], o[2 * e], o[2 * e + 1], inv, inv);
            w[e] = Mma<T>::pack(o[2 * e], o[2 * e + 1]);
          }
          T* d = dst + c4 * 32;
          if (p.wide_out) {                      // whole 32-byte sectors a store
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d + 2 * e), "r"(w[e]),
                           "r"(w[e + 1]), "r"(w[e + 2]), "r"(w[e + 3]), "r"(w[e + 4]), "r"(w[e + 5]), "r"(w[e + 6]),
                           "r"(w[e + 7])
                           : "memory");
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(d + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
          }
        }
      }
      arrive(kItemFree + r % kItemRing);
      exchange();                                // xsum is read before the next item's first maximum
    }
    if (!told) {
      if (!ok) *gave_up = 1;
      exchange();
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
cudaError_t launch_mode(const ModParams& prm, cudaStream_t stream) {
  constexpr int smem = Layout<D>::kBytes;
  cudaError_t e =
      cudaFuncSetAttribute(prefill_mod_kernel<T, D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_mod_kernel<T, D, MODE>, dim3((unsigned)prm.items), dim3(kThreads), smem, stream, prm);
}

template <typename T, int D>
cudaError_t launch_typed(const ModParams& prm, cudaStream_t stream) {
  const bool cap = prm.mod.cap_in != 0.f, bias = prm.mod.slopes != nullptr;
  if (cap && bias) return launch_mode<T, D, kCap | kBias>(prm, stream);
  if (bias) return launch_mode<T, D, kBias>(prm, stream);
  if (!cap) return launch_mode<T, D, 0>(prm, stream);
  // bf16 weights of 2^64 times a sum of 2^23 keys and a value of 2^16 stay within fp32
  if (std::is_same<T, __nv_bfloat16>::value && prm.mod.cap_out_log2 <= 64.f)
    return launch_mode<T, D, std::is_same<T, __nv_bfloat16>::value ? kCap | kBounded : kCap>(prm, stream);
  return launch_mode<T, D, kCap>(prm, stream);
}

}  // namespace

// Calls that prefill_tc_supported takes.
cudaError_t launch_prefill_mod(const PrefillArgs& a, cudaStream_t stream) {
  const pkvd_cache& c = a.cache;
  const int G = a.num_q_heads / c.num_kv_heads;
  const int seg_rows = c.block_size < kTcKeys ? c.block_size : kTcKeys;
  ModParams prm;
  prm.tile_tokens = kTcRows / G;
  if (!encode_cache_map(&prm.tmap_k, c.k_base, c, seg_rows) || !encode_cache_map(&prm.tmap_v, c.v_base, c, seg_rows) ||
      !encode_q_map(&prm.tmap_q, a.q, c.dtype, c.head_dim, a.num_q_heads, a.total_q, G, prm.tile_tokens))
    return cudaErrorInvalidValue;
  prm.out = a.out;
  prm.tables = a.block_tables;
  prm.max_blocks = a.max_blocks_per_seq;
  prm.block_limit = (uint32_t)(c.num_blocks < 0x80000000ll ? c.num_blocks : 0x80000000ll);
  prm.block_size = c.block_size;
  prm.block_shift = 0;
  while ((1 << prm.block_shift) < c.block_size) ++prm.block_shift;
  prm.seg_rows = seg_rows;
  prm.cu_q = a.cu_seqlens_q;
  prm.cu_k = a.cu_seqlens_k;
  prm.total_q = a.total_q;
  prm.hq = a.num_q_heads;
  prm.hkv = c.num_kv_heads;
  prm.group = G;
  prm.q_box = 128u * (uint32_t)(G * prm.tile_tokens);
  const int tiles = (a.max_seqlen_q + prm.tile_tokens - 1) / prm.tile_tokens;
  // With an SM for every Q tile, each has one: a chain of K tiles is shorter
  // with half the softmax warps on it (one prompt of 734 tokens, 12 + 2 heads of
  // 128: 21 instead of 27 us; four chunks of 14 to 116 tokens after 1467, 8 + 4
  // heads of 64: 27 instead of 35).  Otherwise two share a CTA, so that one's
  // products run beside the other's softmax.
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  prm.pair = (int64_t)tiles * c.num_kv_heads * a.num_seqs <= sms ? 1 : 2;
  prm.pairs = (tiles + prm.pair - 1) / prm.pair;
  prm.num_seqs = a.num_seqs;
  const int64_t items = (int64_t)prm.pairs * c.num_kv_heads * a.num_seqs;
  if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
  prm.items = (int)items;
  prm.waves = items > sms;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  prm.window = a.window;
  prm.mod = a.mod;
  prm.poly_range = cap_poly(a.mod, prm.poly);
  prm.wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  prm.err = a.err;
  if (c.dtype == PKVD_BF16)
    return c.head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(prm, stream)
                            : launch_typed<__nv_bfloat16, 128>(prm, stream);
  return c.head_dim == 64 ? launch_typed<__half, 64>(prm, stream) : launch_typed<__half, 128>(prm, stream);
}

}  // namespace pkvd
