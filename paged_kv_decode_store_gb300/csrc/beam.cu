// One step of beam search: of all continuations (beam b, id j) of a request,
// the `keep` with the largest
//   scores[b] + x_bj - logsumexp_j(x_bj),
// the lowest b * vocab + j first among equal values.
//
// Two kernels.  The scan reads every logit once and selects nothing: a warp
// takes a span of 1 KB chunks (two 16-byte loads a lane each, the next two
// chunks in flight while two are summed) and leaves the span's maximum and sum
// of exponentials and each chunk's maximum -- no barrier, no shared memory.
// The merge, one CTA per request, joins the sums into each beam's normaliser
// and finds the winners from the maxima: the maxima of `keep` chunks are
// `keep` elements, so the keep-th largest chunk maximum bounds the keep-th
// best value from below, and only the few chunks that reach it are read again
// (from L2 or DRAM, a few KB).  The same argument on the vectors of those
// chunks tightens the bound; what is left (some more than `keep` elements) is
// listed and ranked against one another.  Selecting in every 32 KB slice
// instead, as a first version did, cost 148 us for 64 x 8 rows of 151,936 f16
// ids, most of it in barriers; this one takes 40 us (floor 23 us), 31 of them
// in the scan.
//
// Rounding: the order within a beam is that of the logits; values of listed
// continuations are pairs of fp32 (about 2^-48 relative), the bounds fp32 with
// a margin for their own rounding.  The normaliser's sum is fp32 for 32 terms
// at a time and pairs of fp32 from there on, its logarithm a pair.  (FP64 has
// a sixtieth of the fp32 rate here: with a double per beam and continuation,
// and the library's log, the normalisers alone took half the merge.)
//
// Bound: for large batches the scan's loads in flight (half of them wait while
// the other half is summed: DRAM 61 % busy, issue slots 56 %), then the merge
// on as many SMs as there are requests; for small ones the two kernels'
// latency.  Where more than 2048 continuations reach the bound (uniform rows),
// every one kept costs a pass over the request's logits: 11 ms instead of 38
// us for 64 x 8 uniform rows of 151,936 and 16 kept.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kScanThreads = 256;                     // eight warps, each on its own
constexpr int kScanCtas = 4;                          // resident on an SM
constexpr int kChunkVecs = 64;                        // 16-byte vectors of a chunk
constexpr int kMergeThreads = 512;
constexpr int kGroups = 64;                           // groups of 8 lanes of the merge
constexpr int kBeamList = 2048;                       // listed elements and chunks
static_assert(kGroups >= kBeamMaxKeep && kMergeThreads == kGroups * 8, "a bound needs keep groups");

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Float bits in an order-preserving unsigned form; 0 is below every number.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// Sums in two parts, the second holding the rounding of the first (Knuth's
// two-sum, Dekker's pairs).
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float h = a + b, back = h - a;
  return make_float2(h, (a - (h - back)) + (b - back));
}
__device__ __forceinline__ float2 add_parts(float2 a, float2 b) {
  const float2 h = two_sum(a.x, b.x);
  return two_sum(h.x, h.y + (a.y + b.y));
}
// A finite pair as a key that orders by value; 0 is below every key.
__device__ __forceinline__ uint64_t pair_key(float2 v) {
  return ((uint64_t)ordered(v.x + 0.f) << 32) | ordered(v.y + 0.f);
}

// -inf in every element of a 32-bit word, the larger elements of two words,
// and the largest element of a word.
template <typename T> struct Word;
template <> struct Word<float> {
  static constexpr uint32_t kLow = 0xff800000u;
  __device__ static uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ static float most(uint32_t a) { return __uint_as_float(a); }
};
template <> struct Word<__half> {
  static constexpr uint32_t kLow = 0xfc00fc00u;
  __device__ static uint32_t max(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  __device__ static float most(uint32_t a) {
    const float2 t = __half22float2(*reinterpret_cast<__half2*>(&a));
    return fmaxf(t.x, t.y);
  }
};
template <> struct Word<__nv_bfloat16> {
  static constexpr uint32_t kLow = 0xff80ff80u;
  __device__ static uint32_t max(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  __device__ static float most(uint32_t a) {
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
};
template <typename T>
__device__ __forceinline__ uint32_t vec_max(const uint4& a) {
  return Word<T>::max(Word<T>::max(a.x, a.y), Word<T>::max(a.z, a.w));
}

// A row's elements by index, whatever its alignment: rows that hold the same
// logits are summed in the same order, so equal continuations of different
// beams are exactly equal.
template <typename T>
struct RowView {
  static constexpr int N = Vec16<T>::N;
  const T* x;
  int vocab;
  uint32_t lead;      // elements from the 16-byte boundary at or before the row to its first
  __device__ RowView(const BeamArgs& p, int row) {
    x = static_cast<const T*>(p.logits) + (int64_t)row * p.row_stride;
    vocab = p.vocab;
    lead = (uint32_t)(reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T);
  }
  // A vector that lies inside the row with the aligned vectors around it.
  __device__ bool inside(int e0) const { return e0 >= N && e0 + 2 * N <= vocab; }
  __device__ uint4 load_inside(int e0) const {
    const uint4* v = reinterpret_cast<const uint4*>(x + e0 - (int)lead);
    const uint4 a = __ldg(v);
    if (lead == 0) return a;
    // the row's vector straddles two aligned ones: the words from lead on
    const uint4 b = __ldg(v + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const uint32_t skip = lead * sizeof(T) / 4, bits = lead * sizeof(T) % 4 * 8;
    uint32_t o[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      o[k] = w[k];
      if (skip == 1 && k + 1 < 8) o[k] = w[k + 1];
      if (skip == 2 && k + 2 < 8) o[k] = w[k + 2];
      if (skip == 3 && k + 3 < 8) o[k] = w[k + 3];
    }
    return make_uint4(__funnelshift_r(o[0], o[1], bits), __funnelshift_r(o[1], o[2], bits),
                      __funnelshift_r(o[2], o[3], bits), __funnelshift_r(o[3], o[4], bits));
  }
  // Elements [e0, e0 + N), -inf past the row's end (which is not read).  e0 is
  // below the vocabulary rounded up to a chunk, so below 2^24.
  __device__ uint4 load(int e0) const {
    if (lead == 0 ? e0 + N <= vocab : inside(e0)) return load_inside(e0);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        w[k] = e0 + k < vocab ? reinterpret_cast<const uint32_t*>(x)[e0 + k] : Word<T>::kLow;
      } else {
        const unsigned short* b = reinterpret_cast<const unsigned short*>(x);
        const int e = e0 + 2 * k;
        const uint32_t lo = e < vocab ? b[e] : Word<T>::kLow & 0xffffu;
        const uint32_t hi = e + 1 < vocab ? b[e + 1] : Word<T>::kLow >> 16;
        w[k] = lo | (hi << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A vector that nobody reads again soon: not kept in L1, and asked of DRAM in
// 256 bytes (50 -> 44 us for the 64 x 8 rows from DRAM, 41 -> 40 from L2 in part).
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Two fp32 lanes in one register pair.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads, kScanCtas) beam_scan_kernel(const BeamArgs p) {
  constexpr int N = Vec16<T>::N;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  const int64_t row64 = w / p.spans;
  if (row64 >= (int64_t)p.requests * p.beams) return;
  const int row = (int)row64, span = (int)(w - row64 * p.spans);
  if (p.finished && p.finished[row]) return;           // an ended beam: its logits do not count
  const RowView<T> view(p, row);
  const int c0 = span * p.span_chunks, c1 = min(c0 + p.span_chunks, p.chunks);
  if (c0 >= c1) return;
  const int vocab = p.vocab;
  const uint4 low = make_uint4(Word<T>::kLow, Word<T>::kLow, Word<T>::kLow, Word<T>::kLow);
  // a lane's four vectors of the pair of chunks c, c + 1; chunks [in0, in1) lie
  // inside the row with the aligned vectors around them
  const int in0 = view.lead ? 1 : 0, in1 = min(c1, (view.lead ? max(vocab - N, 0) : vocab) / (kChunkVecs * N));
  const uint4* aligned = reinterpret_cast<const uint4*>(view.x) + lane;
  auto fetch = [&](int c, uint4* raw) {
    if (c >= in0 && c + 2 <= in1) {
      if (view.lead == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = load_once(aligned + c * kChunkVecs + i * 32);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = view.load_inside((c * kChunkVecs + i * 32 + lane) * N);
      }
    } else {                                            // the row's edges and the span's last chunk
#pragma unroll
      for (int i = 0; i < 4; ++i)
        raw[i] = c + (i >> 1) < c1 ? view.load((c * kChunkVecs + i * 32 + lane) * N) : low;
    }
  };
  constexpr float kLog2e = 1.4426950408889634f;
  const uint64_t scale2 = pair2(kLog2e, kLog2e);
  uint4 raw[4], next[4];
  fetch(c0, raw);
  float m = -INFINITY;
  float2 sum = make_float2(0.f, 0.f);
  for (int c = c0; c < c1; c += 2) {
    fetch(c + 2, next);
    const float most0 = warp_max(Word<T>::most(Word<T>::max(vec_max<T>(raw[0]), vec_max<T>(raw[1]))));
    const float most1 = warp_max(Word<T>::most(Word<T>::max(vec_max<T>(raw[2]), vec_max<T>(raw[3]))));
    if (lane < 2 && c + lane < c1) p.maxima[(int64_t)row * p.chunks + c + lane] = lane ? most1 : most0;
    const float up = fmaxf(most0, most1);
    if (up > m) {                                       // the same in every lane
      const float down = ex2f((m - up) * kLog2e);   // 0 the first time
      sum.x *= down;
      sum.y *= down;
      m = up;
    }
    // x - max first, which is exact for 16-bit logits and zero for the largest:
    // a rounding of max * log2(e) would shift every term of the span alike.  A
    // NaN or +inf logit makes the sum NaN: the merge then drops the beam.
    const float ref = m == -INFINITY ? 0.f : m;
    const uint64_t minus_ref = pair2(-ref, -ref);
    uint64_t part = pair2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[N];
      Vec16<T>::unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float a, b;
        unpair2(mul2(add2(pair2(v[j], v[j + 1]), minus_ref), scale2), a, b);
        part = add2(part, pair2(ex2f(a), ex2f(b)));
      }
    }
    float p0, p1;
    unpair2(part, p0, p1);
    const float2 t = two_sum(sum.x, p0 + p1);
    sum = make_float2(t.x, sum.y + t.y);
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = next[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    sum = add_parts(sum, make_float2(__shfl_xor_sync(FULL_MASK, sum.x, o), __shfl_xor_sync(FULL_MASK, sum.y, o)));
  if (lane == 0) p.sums[(int64_t)row * p.spans + span] = make_float4(m, sum.x, sum.y, 0.f);
}

// log of a positive pair, as a pair off by about 2 * 10^-9: log(2^e f) = e log 2 +
// 2 artanh(s) with s = (f - 1) / (f + 1), f in [0.7, 1.42], so |s| < 0.18 and the
// series' s^13 term is the first that is left out.  f - 1 is exact; the
// quotient's remainder, the low part of e log 2 and the series go into the
// second part.
__device__ __forceinline__ float2 log_pair(float2 t) {
  int e = (int)(__float_as_uint(t.x) >> 23) - 127;
  float f = __uint_as_float((__float_as_uint(t.x) & 0x007fffffu) | 0x3f800000u);
  if (f > 1.41421356f) {
    f *= 0.5f;
    ++e;
  }
  const float tail = t.y * __uint_as_float((uint32_t)(127 - e) << 23);
  const float num = f - 1.f;
  const float2 den = two_sum(f, 1.f);
  const float inv = __frcp_rn(den.x);
  const float s = num * inv;
  const float low = fmaf(-s, den.y + tail, fmaf(-s, den.x, num) + tail) * inv;
  const float z = s * s;
  float r = fmaf(z, 1.f / 11, 1.f / 9);
  r = fmaf(z, r, 1.f / 7);
  r = fmaf(z, r, 1.f / 5);
  r = fmaf(z, r, 1.f / 3);
  const float2 main = two_sum((float)e * 0.693145751953125f, 2.f * s);          // log 2 to 16 bits: the product is exact
  return add_parts(main, make_float2(fmaf((float)e, 1.428606765330187e-06f, 2.f * fmaf(s * z, r, low)), 0.f));
}

struct MergeSmem {
  float2 base[kBeamMaxBeams];            // score minus the log of the sum: a logit counts from its row's largest
  float2 basef[kBeamMaxBeams];           // the same in fp32 (-inf: no logits to look at) and the row's largest logit
  float2 total[kBeamMaxBeams];           // sum of exponentials
  float group[kGroups];
  float bound;
  int chunks, count;
  unsigned long long best;
  uint32_t best_at;
  int2 chunk[kBeamList];                 // beam, chunk
  float logit[kBeamList];
  uint64_t value[kBeamList];
  uint32_t at[kBeamList];                // beam * vocab + id
};

// The keep-th largest of the kGroups group maxima (a lower bound of the
// keep-th largest value, -inf if fewer groups have one), less a margin for
// the fp32 values' rounding: a beam's base, a logit's distance from its row's
// largest and their sum are each off by 2^-24 relative (the distance is at most
// value and base together), for the element that bounds and the one it is held
// against: 2^-22 of value and base, twice that to be sure.
__device__ __forceinline__ void set_bound(MergeSmem& s, float most, int keep, float base_size) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, o));
  if ((tid & 7) == 0) s.group[tid >> 3] = most;
  __syncthreads();
  // eight threads a group: how many groups come before it
  const int g = tid >> 3;
  int before = 0;
#pragma unroll
  for (int i = 0; i < kGroups / 8; ++i) {
    const int j = i * 8 + (tid & 7);
    const float o = s.group[j];
    before += o > most || (o == most && j < g);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) before += __shfl_xor_sync(FULL_MASK, before, o);
  if (before == keep - 1) s.bound = most - (fabsf(most) + base_size) * 0x1p-21f;
  __syncthreads();
}

// One CTA per request.
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamArgs p) {
  constexpr int N = Vec16<T>::N;
  constexpr int kHeld = 8;               // chunk maxima a thread keeps in registers
  extern __shared__ __align__(16) uint8_t smem_raw[];
  MergeSmem& s = *reinterpret_cast<MergeSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x, B = p.beams, K = p.keep;
  const int nc = B * p.chunks;           // fits: the host checks all rows' chunks
  if (tid == 0) s.chunks = s.count = 0;
  pdl_wait();
  pdl_trigger();
  const float* maxima = p.maxima + (int64_t)r * nc;
  float held[kHeld];                     // on their way while the normalisers are joined
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = tid + i * kMergeThreads < nc ? maxima[tid + i * kMergeThreads] : 0.f;
  const float score = tid < B ? p.scores[r * B + tid] : 0.f;
  const bool done = tid < B && p.finished && p.finished[r * B + tid];
  // ---- each beam's normaliser: a warp per beam over its spans, then a lane per beam
  for (int b = warp; b < B; b += kMergeThreads / 32) {
    const float4* part = p.sums + (int64_t)(r * B + b) * p.spans;   // not written for ended beams, and not used
    const float4 none = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    const float4 first = lane < p.spans ? part[lane] : none;
    float m = first.x;
    bool bad = !(first.y < INFINITY);
    for (int i = lane + 32; i < p.spans; i += 32) {
      const float4 t = part[i];
      m = fmaxf(m, t.x);
      bad |= !(t.y < INFINITY);
    }
    m = warp_max(m);
    float2 total = make_float2(0.f, 0.f);
    auto join = [&](const float4& t) {
      if (t.x == -INFINITY) return;
      const float w = ex2f((t.x - m) * 1.4426950408889634f);
      total = add_parts(total, make_float2(__fmul_rn(t.y, w), t.z * w));   // no FMA inside a two-sum
    };
    join(first);
    for (int i = lane + 32; i < p.spans; i += 32) join(part[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      total = add_parts(total, make_float2(__shfl_xor_sync(FULL_MASK, total.x, o),
                                           __shfl_xor_sync(FULL_MASK, total.y, o)));
    if (__any_sync(FULL_MASK, bad)) m = -INFINITY;
    if (lane == 0) {
      s.basef[b].y = m;                  // -inf: none, or one that is not finite
      s.total[b] = total;
    }
  }
  __syncthreads();
  if (tid < B) {
    const float top = s.basef[tid].y;
    const bool usable = !done && top > -INFINITY && top < INFINITY;
    float2 base = make_float2(score, 0.f);
    if (usable) {
      const float2 norm = log_pair(s.total[tid]);
      base = add_parts(base, make_float2(-norm.x, -norm.y));
    }
    const bool finite = fabsf(score) < INFINITY && (done || usable);
    s.base[tid] = base;
    s.basef[tid].x = finite && !done ? base.x : -INFINITY;
    if (finite && done) {                                                // its one continuation
      const int i = atomicAdd(&s.count, 1);
      s.value[i] = pair_key(base);
      s.at[i] = (uint32_t)tid * p.vocab + p.eos_id;
    }
  }
  __syncthreads();
  const int ended = s.count;
  float base_size = 0.f;
  for (int b = lane; b < B; b += 32) base_size = fmaxf(base_size, s.basef[b].x > -INFINITY ? fabsf(s.basef[b].x) : 0.f);
  base_size = warp_max(base_size);
  // ---- the chunks that may hold a winner
  // c / chunks by a product (Granlund and Montgomery, 1994); c < 2^31
  auto beam_of = [&](int c) { return (int)((__umulhi((uint32_t)c, p.chunk_mul) + (uint32_t)c) >> p.chunk_shift); };
  auto value_f = [&](int b, float logit) {
    const float2 base = s.basef[b];
    return base.x > -INFINITY ? base.x + (logit - base.y) : -INFINITY;
  };
  auto chunk_value = [&](int c, float top) { return value_f(beam_of(c), top); };
  float most = -INFINITY;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = tid + i * kMergeThreads;
    held[i] = c < nc ? chunk_value(c, held[i]) : -INFINITY;
    most = fmaxf(most, held[i]);
  }
  for (int c = tid + kHeld * kMergeThreads; c < nc; c += kMergeThreads) most = fmaxf(most, chunk_value(c, maxima[c]));
  set_bound(s, most, K, base_size);
  float bound = s.bound;
  auto list_chunk = [&](int c, float v) {
    if (v > -INFINITY && v >= bound) {
      const int i = atomicAdd(&s.chunks, 1), b = beam_of(c);
      if (i < kBeamList) s.chunk[i] = make_int2(b, c - b * p.chunks);
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) list_chunk(tid + i * kMergeThreads, held[i]);
  for (int c = tid + kHeld * kMergeThreads; c < nc; c += kMergeThreads) list_chunk(c, chunk_value(c, maxima[c]));
  __syncthreads();
  // calls f(beam, id of the first element, raw vector) for a thread's share of
  // the vectors of those chunks (of all chunks when they are too many to list)
  const bool listed = s.chunks <= kBeamList;
  const int64_t vecs = (int64_t)(listed ? s.chunks : nc) * kChunkVecs;
  auto each = [&](int64_t from, auto f) {
    for (int64_t i = from; i < vecs; i += kMergeThreads) {
      const int ci = (int)(i / kChunkVecs);
      int2 c;
      if (listed) {
        c = s.chunk[ci];
      } else {
        c.x = beam_of(ci);
        c.y = ci - c.x * p.chunks;
        if (s.basef[c.x].x == -INFINITY) continue;
      }
      const RowView<T> view(p, r * B + c.x);
      const int e0 = (c.y * kChunkVecs + (int)(i % kChunkVecs)) * N;
      f(c.x, e0, view.load(e0));
    }
  };
  // ---- the bound once more, on their vectors; a thread's first kKept stay in registers
  constexpr int kKept = 4;
  uint4 kept[kKept];
  int kept_beam[kKept], kept_id[kKept];
  most = -INFINITY;
#pragma unroll
  for (int k = 0; k < kKept; ++k) {
    const int64_t i = tid + (int64_t)k * kMergeThreads;
    kept_beam[k] = -1;
    if (listed && i < vecs) {
      const int2 c = s.chunk[i / kChunkVecs];
      const RowView<T> view(p, r * B + c.x);
      const int e0 = (c.y * kChunkVecs + (int)(i % kChunkVecs)) * N;
      kept_beam[k] = c.x;
      kept_id[k] = e0;
      kept[k] = view.load(e0);
    }
  }
#pragma unroll
  for (int k = 0; k < kKept; ++k)
    if (kept_beam[k] >= 0) most = fmaxf(most, value_f(kept_beam[k], Word<T>::most(vec_max<T>(kept[k]))));
  const int64_t rest = tid + (listed ? (int64_t)kKept * kMergeThreads : 0);
  each(rest, [&](int b, int, const uint4& v) { most = fmaxf(most, value_f(b, Word<T>::most(vec_max<T>(v)))); });
  set_bound(s, most, K, base_size);
  bound = fmaxf(bound, s.bound);
  auto list_vec = [&](int b, int id0, const uint4& raw) {
    if (!(value_f(b, Word<T>::most(vec_max<T>(raw))) >= bound)) return;
    float v[N];
    Vec16<T>::unpack(raw, v);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float x = value_f(b, v[j]);
      if (x > -INFINITY && x >= bound) {
        const int i = atomicAdd(&s.count, 1);
        if (i < kBeamList) {
          s.logit[i] = v[j];
          s.at[i] = (uint32_t)b * p.vocab + (id0 + j);
        }
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kKept; ++k)
    if (kept_beam[k] >= 0) list_vec(kept_beam[k], kept_id[k], kept[k]);
  each(rest, list_vec);
  __syncthreads();
  auto value_of = [&](int b, float logit) {
    return pair_key(add_parts(s.base[b], two_sum(logit, -s.basef[b].y)));     // the difference is exact
  };
  auto emit = [&](int k, uint64_t value, uint32_t at) {
    const int64_t o = (int64_t)r * K + k;
    p.out_scores[o] = value ? unordered((uint32_t)(value >> 32)) : -INFINITY;
    p.out_parents[o] = value ? (int)(at / (uint32_t)p.vocab) : -1;
    p.out_tokens[o] = value ? (int)(at % (uint32_t)p.vocab) : -1;
  };
  const int n = s.count;
  if (n <= kBeamList) {
    for (int i = ended + tid; i < n; i += kMergeThreads)
      s.value[i] = value_of((int)(s.at[i] / (uint32_t)p.vocab), s.logit[i]);
    __syncthreads();
    // eight threads an element: how many come before it
    for (int i0 = 0; i0 < n; i0 += kMergeThreads / 8) {
      const int i = i0 + (tid >> 3);
      const uint64_t value = i < n ? s.value[i] : 0;
      const uint32_t at = i < n ? s.at[i] : 0;
      int before = 0;
      for (int j = tid & 7; j < n; j += 8) {
        const uint64_t o = s.value[j];
        before += o > value || (o == value && s.at[j] < at);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) before += __shfl_xor_sync(FULL_MASK, before, o);
      if (i < n && (tid & 7) == 0 && before < K) emit(before, value, at);
    }
    for (int i = n + tid; i < K; i += kMergeThreads) emit(i, 0, 0);
    return;
  }
  // so many next to the bound: the best one after the last, keep times
  uint64_t last = ~0ull;
  uint32_t last_at = 0;
  for (int k = 0; k < K; ++k) {
    if (tid == 0) {
      s.best = 0;
      s.best_at = 0xffffffffu;
    }
    __syncthreads();
    uint64_t mine = 0;
    uint32_t mine_at = 0xffffffffu;
    auto offer = [&](uint64_t value, uint32_t at) {
      const bool after = value < last || (value == last && at > last_at);
      if (after && (value > mine || (value == mine && at < mine_at))) mine = value, mine_at = at;
    };
    if (tid < ended) offer(s.value[tid], s.at[tid]);
    each(tid, [&](int b, int id0, const uint4& raw) {
      float v[N];
      Vec16<T>::unpack(raw, v);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float x = value_f(b, v[j]);
        if (x > -INFINITY && x >= bound)
          offer(value_of(b, v[j]), (uint32_t)b * p.vocab + (id0 + j));
      }
    });
    atomicMax(&s.best, (unsigned long long)mine);
    __syncthreads();
    if (mine && mine == s.best) atomicMin(&s.best_at, mine_at);
    __syncthreads();
    last = s.best;
    last_at = s.best_at;
    if (tid == 0) emit(k, last, last_at);
    __syncthreads();
    if (last == 0) {                                     // nothing left: the rest is empty
      for (int i = k + 1 + tid; i < K; i += kMergeThreads) emit(i, 0, 0);
      break;
    }
  }
}

template <typename T>
cudaError_t launch_typed(const BeamArgs& a, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.requests * a.beams * a.spans;
  const int64_t ctas = (warps + kScanThreads / 32 - 1) / (kScanThreads / 32);
  cudaError_t e = launch_pdl(beam_scan_kernel<T>, dim3((unsigned)ctas), dim3(kScanThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  constexpr int smem = sizeof(MergeSmem);
  e = cudaFuncSetAttribute(beam_merge_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_merge_kernel<T>, dim3((unsigned)a.requests), dim3(kMergeThreads), smem, stream, a);
}

}  // namespace

// 1 KB chunks of a row.
int beam_chunks(int dtype, int vocab) {
  const int n = (dtype == PKVD_F32 ? 4 : 8) * kChunkVecs;
  return (vocab + n - 1) / n;
}

// A span's sums and a chunk's maximum; at most one span a chunk.
size_t beam_workspace_bytes(int64_t rows, int chunks) {
  return (size_t)rows * chunks * (sizeof(float4) + sizeof(float));
}

cudaError_t launch_beam(const BeamArgs& call, cudaStream_t stream) {
  BeamArgs a = call;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // as many spans as the GPU holds warps at once, so that one wave of equal
  // warps reads everything (1.05 waves took 39 us where 0.95 take 26)
  const int64_t rows = (int64_t)a.requests * a.beams, slots = (int64_t)sms * kScanCtas * (kScanThreads / 32);
  const int64_t spans = slots / rows < 1 ? 1 : slots / rows;
  a.span_chunks = (int)((a.chunks + spans - 1) / spans);
  a.spans = (a.chunks + a.span_chunks - 1) / a.span_chunks;
  int shift = 0;
  while ((1ll << shift) < a.chunks) ++shift;
  a.chunk_shift = shift;
  a.chunk_mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - (uint64_t)a.chunks)) / (uint64_t)a.chunks + 1);
  if (a.dtype == PKVD_F32) return launch_typed<float>(a, stream);
  if (a.dtype == PKVD_F16) return launch_typed<__half>(a, stream);
  return launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace pkvd
