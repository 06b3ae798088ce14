// Eviction by accumulated attention weight: which positions of a sequence stay.
//
// Row (sequence i, head h) of `weights` holds what each cached position was
// given so far.  With c = context_lens[i] > keep the first `sink` and the last
// `recent` positions stay, and of the others the heaviest, keep in all; the
// lowest position first among equal weights.  Positions come out in ascending
// order, the weights that stay close up beside them, zeros behind.
//
// A CTA a row.  Its weights are read once (rows up to 32,768: half in
// registers, half in shared memory; a longer one again for each pass, 32,768
// at a time) and looked at four times: the keep-th weight by radix selection
// over order-preserving whole numbers (11, 11 and 10 bits, a histogram in
// shared memory each, four copies of it so that lanes with equal digits do not
// all wait for one another), then what stays is written in order.  Every warp
// has a contiguous part of the row, so the order needs two prefix sums over
// warps and ballots within one, no barrier an element.  Exact: whole-number
// arithmetic on the weights' bits.
//
// Bound by bytes and, beside them, by the passes' instructions: with 1024
// threads a row, weights read again for every pass and one histogram, 64 rows
// of 8 heads of 4,096 to 32,768 weights took 135 us.
#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kInRegs = 32, kInSmem = 32;                  // weights of a thread
constexpr int kSpan = (kInRegs + kInSmem) * kThreads;      // positions of a round
constexpr int kBins = 2048, kCopies = 4;
constexpr int kSmemBytes = kInSmem * kThreads * 4 + kBins * kCopies * 4;

// Keys in the order of the numbers: -0 as 0, NaN above all.  `special`: the row
// has a -0 or a NaN.
__device__ __forceinline__ uint32_t key_of(uint32_t u, bool special) {
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  if (special) {
    if (u == 0x80000000u) return 0x80000000u;
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  }
  return k;
}

__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t* held = sm;                                     // [kInSmem][kThreads]
  uint32_t* hist = sm + kInSmem * kThreads;                // [kBins][kCopies]
  __shared__ int warp_sum[2][kWarps];
  __shared__ uint32_t found_digit;
  __shared__ int found_left;
  pdl_wait();          // (and no early trigger: counts are the next call's lengths, which it reads before it waits)
  const int h = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int c = a.context_lens[seq];
  if (c < 0 || c > a.length) {
    if (tid == 0 && h == 0) flag_error(a.err, PKVD_ERR_CONTEXT);
    c = min(max(c, 0), a.length);
  }
  const float* w = a.weights + (int64_t)seq * a.seq_stride + (int64_t)h * a.head_stride;
  float* wo = a.weights_out ? a.weights_out + (int64_t)seq * a.seq_stride + (int64_t)h * a.head_stride : nullptr;
  int32_t* out = a.positions + ((int64_t)seq * gridDim.x + h) * a.keep;
  const int count = min(c, a.keep);
  if (h == 0 && tid == 0) {
    a.counts[seq] = count;
    __threadfence();
  }
  // what competes: positions [lo, hi) for `left` places
  const bool all = c <= a.keep;
  const int lo = all ? 0 : a.sink, hi = all ? 0 : c - a.recent;
  int left = all ? 0 : a.keep - a.sink - a.recent;

  // A round: positions [base, base + span), every warp `seg` of them, 32 at a time.
  const int rounds = (c + kSpan - 1) / kSpan;
  uint32_t reg[kInRegs];
  int first = 0, n = 0, steps = 0;                         // this warp's part: position of lane 0's first, end, steps
  auto place = [&](int r) {
    const int base = r * kSpan, span = min(c - base, kSpan);
    const int seg = ((span + kWarps - 1) / kWarps + 31) / 32 * 32;
    first = base + min(warp * seg, span);
    n = base + min(warp * seg + seg, span);
    steps = (n - first + 31) / 32;
  };
  auto fetch = [&](int r) {
    place(r);
    bool odd = false;
    const float* src = w + first + lane;
    const int mine = n - first - lane;                     // positions from this lane's first to the end
#pragma unroll
    for (int i = 0; i < kInRegs; ++i) {
      reg[i] = i * 32 < mine ? __float_as_uint(src[i * 32]) : 0u;
    }
    for (int i = kInRegs; i < steps; i += 8) {
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (i + e) * 32 < mine ? __float_as_uint(src[(i + e) * 32]) : 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (i + e < steps) held[(i + e - kInRegs) * kThreads + tid] = x[e];
        odd |= x[e] == 0x80000000u || (x[e] & 0x7fffffffu) > 0x7f800000u;
      }
    }
#pragma unroll
    for (int i = 0; i < kInRegs; ++i) odd |= reg[i] == 0x80000000u || (reg[i] & 0x7fffffffu) > 0x7f800000u;
    return odd;
  };
  // f(position, bits, there) for this thread's places in order; every lane of the warp comes along
  auto each = [&](auto f) {
    if (steps >= kInRegs) {
#pragma unroll
      for (int i = 0; i < kInRegs; ++i) f(first + i * 32 + lane, reg[i], first + i * 32 + lane < n);
      for (int i = kInRegs; i < steps; ++i)
        f(first + i * 32 + lane, held[(i - kInRegs) * kThreads + tid], first + i * 32 + lane < n);
    } else {
#pragma unroll
      for (int i = 0; i < kInRegs; ++i) {
        if (i >= steps) break;
        f(first + i * 32 + lane, reg[i], first + i * 32 + lane < n);
      }
    }
  };

  bool special = false;
  uint32_t kth = 0xffffffffu;          // the key of the last one that stays, `left` of those equal to it do
  for (int r = 0; r < rounds; ++r) special |= fetch(r);    // (one round: kept from here on)
  special = __syncthreads_or(special);
  if (left > 0) {
    uint32_t prefix = 0, mask = 0;
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      const uint32_t digits = shift == 0 ? 1023u : 2047u;
      for (int i = tid; i < kBins * kCopies / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) fetch(r);
        each([&](int j, uint32_t u, bool there) {
          const uint32_t k = key_of(u, special);
          if (there && j >= lo && j < hi && (k & mask) == prefix)
            atomicAdd(&hist[((k >> shift) & digits) * kCopies + (lane & (kCopies - 1))], 1u);
        });
      }
      __syncthreads();
      // from the largest digit down: thread t has the kPer bins below kBins - kPer t
      constexpr int kPer = kBins / kThreads;
      int bin[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(hist)[kBins - 1 - (tid * kPer + i)];
        bin[i] = (int)(x.x + x.y + x.z + x.w);
        mine += bin[i];
      }
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(FULL_MASK, upto, o);
        if (lane >= o) upto += t;
      }
      if (lane == 31) warp_sum[0][warp] = upto;
      __syncthreads();
      int before = upto - mine;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) before += v < warp ? warp_sum[0][v] : 0;
      if (before < left && left <= before + mine) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (before < left && left <= before + bin[i]) {
            found_digit = kBins - 1 - (tid * kPer + i);
            found_left = left - before;
          }
          before += bin[i];
        }
      }
      __syncthreads();
      prefix |= found_digit << shift;
      mask |= digits << shift;
      left = found_left;
    }
    kth = prefix;
  }
  // in order: what stays, and of those equal to the last one the first `left`
  int kept = 0, ties = 0;              // of the rounds before
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) fetch(r);
    int more = 0, tie = 0;             // of this thread, then of the warps before
    auto stays = [&](int j, uint32_t u, bool there, bool& m, bool& t) {
      const bool inside = j >= lo && j < hi;
      const uint32_t k = key_of(u, special);
      m = there && (!inside || (left > 0 && k > kth));
      t = there && inside && left > 0 && k == kth;
    };
    each([&](int j, uint32_t u, bool there) {
      bool m, t;
      stays(j, u, there, m, t);
      more += m;
      tie += t;
    });
    more = __reduce_add_sync(FULL_MASK, more);
    tie = __reduce_add_sync(FULL_MASK, tie);
    if (lane == 0) warp_sum[0][warp] = more, warp_sum[1][warp] = tie;
    __syncthreads();                   // (and every weight of the round is read: in place it may be overwritten)
    int m_before = 0, t_before = ties, m_all = 0, t_all = ties;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      const int m = warp_sum[0][v], t = warp_sum[1][v];
      if (v < warp) m_before += m, t_before += t;
      m_all += m;
      t_all += t;
    }
    // the place of this warp's next one: those before it, ties as far as there are places for them
    int at = kept + m_before + min(t_before, left) - min(ties, left);
    int rank = t_before;
    if (more > 0 || (tie > 0 && rank < left)) {
      const uint32_t below = (1u << lane) - 1u;
      each([&](int j, uint32_t u, bool there) {
        bool m, t;
        stays(j, u, there, m, t);
        const uint32_t tb = __ballot_sync(FULL_MASK, t);
        const bool stay = m || (t && rank + __popc(tb & below) < left);
        const uint32_t sb = __ballot_sync(FULL_MASK, stay);
        if (stay) {
          const int to = at + __popc(sb & below);
          out[to] = j;
          if (wo) wo[to] = __uint_as_float(u);             // to <= j: not of a later round
        }
        at += __popc(sb);
        rank += __popc(tb);
      });
    }
    kept += m_all + min(t_all, left) - min(ties, left);
    ties = t_all;
    __syncthreads();
  }
  for (int r = count + tid; r < a.keep; r += kThreads) out[r] = -1;
  if (wo)
    for (int r = count + tid; r < a.length; r += kThreads) wo[r] = 0.f;
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, int num_seqs, int heads, cudaStream_t stream) {
  if (num_seqs == 0 || heads == 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(evict_select_kernel, dim3(heads, num_seqs), dim3(kThreads), kSmemBytes, stream, a);
}

}  // namespace pkvd
