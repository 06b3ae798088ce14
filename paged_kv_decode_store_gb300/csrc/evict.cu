// Eviction by accumulated attention weight: which positions of a sequence stay.
//
// Row (sequence i, head h) of `weights` holds what each cached position was
// given so far.  With c = context_lens[i] > keep the first `sink` and the last
// `recent` positions stay, and of the others the heaviest, keep in all; the
// lowest position first among equal weights.  Positions come out in ascending
// order, the weights that stay close up beside them, zeros behind.
//
// A CTA a row: the keep-th weight by a radix selection over order-preserving
// integer keys (a histogram in shared memory a digit), then one pass that writes what stays in
// order (block scan).  Exact: whole-number arithmetic on the weights' bits.
#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kDigitBits = 8, kBins = 1 << kDigitBits;

// Keys in the order of the numbers: -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ int warp_sum[2][32];
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
  const int lo = c > a.keep ? a.sink : 0, hi = c > a.keep ? c - a.recent : 0;
  int left = c > a.keep ? a.keep - a.sink - a.recent : 0;
  uint32_t kth = 0xffffffffu;          // the key of the last one that stays, `left` of those equal to it do
  if (c > a.keep && left > 0) {
    uint32_t prefix = 0, mask = 0;
    for (int shift = 32 - kDigitBits; shift >= 0; shift -= kDigitBits) {
      for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSelectThreads) {
        const uint32_t k = weight_key(w[j]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (kBins - 1)], 1u);
      }
      __syncthreads();
      if (warp == 0) {                 // from the largest digit down: lane l has bins [kBins - 8 (l + 1), ..)
        constexpr int kPer = kBins / 32;
        int mine = 0;
        for (int i = 0; i < kPer; ++i) mine += hist[kBins - 1 - (lane * kPer + i)];
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(FULL_MASK, upto, o);
          if (lane >= o) upto += t;
        }
        int before = upto - mine;
        if (before < left && left <= upto) {
          for (int i = 0; i < kPer; ++i) {
            const int bin = kBins - 1 - (lane * kPer + i), n = hist[bin];
            if (before + n >= left) {
              found_digit = bin;
              found_left = left - before;
              break;
            }
            before += n;
          }
        }
      }
      __syncthreads();
      prefix |= found_digit << shift;
      mask |= (uint32_t)(kBins - 1) << shift;
      left = found_left;
    }
    kth = prefix;
  }
  // in order: what stays, and of those equal to the last one the first `left`
  int kept = 0, ties = 0;
  for (int base = 0; base < c; base += kSelectThreads) {
    const int j = base + tid;
    float x = 0.f;
    bool more = false, tie = false;
    if (j < c) {
      x = w[j];
      if (c <= a.keep || j < lo || j >= hi) {
        more = true;
      } else if (left > 0) {
        const uint32_t k = weight_key(x);
        more = k > kth;
        tie = k == kth;
      }
    }
    const uint32_t mt = __ballot_sync(FULL_MASK, tie), mm = __ballot_sync(FULL_MASK, more);
    if (lane == 0) {
      warp_sum[0][warp] = __popc(mt);
      warp_sum[1][warp] = __popc(mm);
    }
    __syncthreads();
    int t_before = ties, m_before = 0, t_all = 0, m_all = 0;
#pragma unroll 8
    for (int i = 0; i < kSelectThreads / 32; ++i) {
      if (i < warp) t_before += warp_sum[0][i], m_before += warp_sum[1][i];
      t_all += warp_sum[0][i];
      m_all += warp_sum[1][i];
    }
    const uint32_t below = (1u << lane) - 1u;
    const int my_tie = t_before + __popc(mt & below);            // ties before this one
    // ties that stay before this position, in this round and in all
    const int stay_before = min(my_tie, left) - min(ties, left);
    const bool stays = more || (tie && my_tie < left);
    if (stays) {
      const int at = kept + m_before + __popc(mm & below) + stay_before;
      out[at] = j;
      if (wo) wo[at] = x;              // at <= j: in place, every weight of this round was read
    }
    kept += m_all + min(ties + t_all, left) - min(ties, left);
    ties += t_all;
    __syncthreads();
  }
  for (int r = count + tid; r < a.keep; r += kSelectThreads) out[r] = -1;
  if (wo)
    for (int r = count + tid; r < a.length; r += kSelectThreads) wo[r] = 0.f;
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, int num_seqs, int heads, cudaStream_t stream) {
  if (num_seqs == 0 || heads == 0) return cudaSuccess;
  return launch_pdl(evict_select_kernel, dim3(heads, num_seqs), dim3(kSelectThreads), 0, stream, a);
}

}  // namespace pkvd
