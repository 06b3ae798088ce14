// Eviction by accumulated attention weight: which positions of a sequence stay.
//
// Row (sequence i, head h) of `weights` holds what each cached position was
// given so far.  With c = context_lens[i] > keep the first `sink` and the last
// `recent` positions stay, and of those between the heaviest, keep in all; the
// lowest position first among equal weights.  Positions come out in ascending
// order, the weights that stay close up beside them, zeros behind.
//
// A CTA a row, two on an SM.  The weights between are read once into shared
// memory (22,528 of them; what is beyond is read again for each pass) as whole
// numbers in the order of the numbers, and looked at three times: for a histogram
// of their first 11 bits (two copies of it, so that lanes with equal digits wait
// less for one another), which says what digit the last one that stays has; for
// a list of the keys with that digit, in which the other 11 and 10 bits are found
// the same way (rows whose list would be longer than its place look at all of
// them again); and for the writing, in order.  Every warp has a contiguous part of
// the row, so the order needs prefix sums over warps once and ballots within one,
// no barrier an element.  Exact: whole-number arithmetic on the weights' bits.
//
// Bound by instructions (59 % of the issue slots) and the barriers between the
// passes: 64 x 8 rows of 4,096 to 32,768 take 50 us, of which their bytes are 15;
// 62 with every pass over the whole row and rows in order (512 equal rows of
// 16,384: 39; 43 with a weight a load instead of four).  The loops are short
// code on purpose: a form with half of the weights in registers, its passes
// written out, took 14 us for a row of 50 instead of 8: it waited for instructions.
#include <climits>

#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kPer = 44;                                   // weights of a thread in shared memory
constexpr int kBins = 2048, kCopies = 2;
constexpr int kList = 256;                                 // a warp's keys with the first digit (behind one copy)
constexpr int kStack = kBins * kCopies / kWarps / 2;       // positions and weights that a warp gathers
constexpr int kHist = kBins + kWarps * kList;              // words of all of these, one use after the other
static_assert(kHist >= kBins * kCopies, "two copies of the histogram");
constexpr int kRanked = 256;
constexpr int kSmemBytes = (kPer * kThreads + kHist) * 4;

// A weight's bits in the order of the numbers, and back.  Any NaN becomes the quiet
// one, above all numbers; 0 is left for no weight.
__device__ __forceinline__ uint32_t ordered_bits(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) u = 0x7fc00000u;
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t number_bits(uint32_t k) { return k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u); }
// What is compared: -0 and 0, next to each other, as one.
__device__ __forceinline__ uint32_t key_of(uint32_t k) { return k - (k >> 31); }

struct Row {
  const float* w;
  float* wo;
  int32_t* out;
  int lo, hi, left;                    // [lo, hi) compete for `left` places behind the first lo
};

// This warp's part: words [from, n), of which word w is position first + w (the
// first warp's may begin up to three before, on a boundary of 16 bytes); the first
// kPer * 32 are held, what is behind is read where it lies.
struct Part {
  const float* src;                    // word 0
  uint32_t* held;
  int first, from, n, steps;           // steps of 32 words: a multiple of four
  bool beyond;                         // are there parts with more than what is held?
  __device__ Part(const Row& row, uint32_t* held, int warp) : held(held) {
    const int ahead = (int)(reinterpret_cast<uintptr_t>(row.w + row.lo) / 4 % 4);
    const int span = row.hi - row.lo + ahead, seg = ((span + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int begin = (int)min((int64_t)warp * seg, (int64_t)span);
    first = row.lo - ahead + begin;
    from = warp == 0 ? ahead : 0;
    n = (int)min((int64_t)begin + seg, (int64_t)span) - begin;
    src = row.w + first;
    steps = ((n + 31) / 32 + 3) / 4 * 4;
    beyond = seg > kPer * 32;
  }
  // 0 where there is none
  __device__ uint32_t read(int w) const { return w < n ? ordered_bits(__float_as_uint(src[w])) : 0u; }
  __device__ void ask(int lane) const {
#pragma unroll 1
    for (int w = lane * 4; w < min(steps, kPer) * 32; w += 128) {
      if (w >= from && w + 4 <= n) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(held + w)), "l"(src + w) : "memory");
      } else {
        for (int e = w; e < w + 4; ++e)
          if (e >= from && e < n)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(held + e)), "l"(src + e) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // What was asked for has come (each lane's own): f(bits in order) of every one, in
  // no order.
  template <typename F>
  __device__ void take_in(int lane, F f) const {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 2
    for (int w = lane * 4; w < min(steps, kPer) * 32; w += 128) {
      uint4 x = *reinterpret_cast<const uint4*>(held + w);
      uint32_t* const v = &x.x;
      const bool whole = w >= from && w + 4 <= n;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = whole || (w + e >= from && w + e < n) ? ordered_bits(v[e]) : 0u;
        f(v[e]);
      }
      *reinterpret_cast<uint4*>(held + w) = x;
    }
#pragma unroll 4
    for (int i = kPer; i < steps; ++i) f(read(i * 32 + lane));
  }
  // The same again.
  template <typename F>
  __device__ void each(int lane, F f) const {
#pragma unroll 2
    for (int w = lane * 4; w < min(steps, kPer) * 32; w += 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(held + w);
      f(x.x);
      f(x.y);
      f(x.z);
      f(x.w);
    }
#pragma unroll 4
    for (int i = kPer; i < steps; ++i) f(read(i * 32 + lane));
  }
};

// The sequence with the y-th longest context (of equal ones the first).
// len: kRanked + 1 words, in memory used later (more of it would leave one CTA on an SM).
__device__ __forceinline__ int by_length(const int32_t* __restrict__ lens, int n, int y, int* len) {
  const int tid = threadIdx.x;
  if (tid < kRanked) len[tid] = tid < n ? lens[tid] : INT_MIN;
  __syncthreads();
  if (tid < n) {
    const int mine = len[tid];
    int rank = 0;
    for (int j = 0; j < n; j += 4) {
      const int4 x = *reinterpret_cast<const int4*>(len + j);
      rank += (x.x > mine || (x.x == mine && j < tid)) + (x.y > mine || (x.y == mine && j + 1 < tid)) +
              (x.z > mine || (x.z == mine && j + 2 < tid)) + (x.w > mine || (x.w == mine && j + 3 < tid));
    }
    if (rank == y) len[kRanked] = tid;
  }
  __syncthreads();
  const int at = len[kRanked];
  __syncthreads();
  return at;
}

__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const EvictArgs a, int ranked) {
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ int warp_sum[2][kWarps], listed_by[kWarps];
  __shared__ uint32_t found_digit;
  __shared__ int found_left;
  uint32_t* const hist = sm;                               // [kBins][copies]
  const int seq = ranked ? by_length(a.context_lens, (int)gridDim.y, (int)blockIdx.y, reinterpret_cast<int*>(sm)) : (int)blockIdx.y;
  pdl_wait();          // (and no early trigger: counts are the next call's lengths, which it reads before it waits)
  const int h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* const held = sm + kHist + warp * (kPer * 32);
  uint32_t* const list = sm + kBins + warp * kList;
  int c = a.context_lens[seq];
  if (c < 0 || c > a.length) {
    if (tid == 0 && h == 0) flag_error(a.err, PKVD_ERR_CONTEXT);
    c = min(max(c, 0), a.length);
  }
  Row row;
  row.w = a.weights + (int64_t)seq * a.seq_stride + (int64_t)h * a.head_stride;
  row.wo = a.weights_out ? a.weights_out + (int64_t)seq * a.seq_stride + (int64_t)h * a.head_stride : nullptr;
  row.out = a.positions + ((int64_t)seq * gridDim.x + h) * a.keep;
  const int count = min(c, a.keep);
  if (h == 0 && tid == 0) {
    a.counts[seq] = count;
    __threadfence();
  }
  // behind what stays; in place only when everything has been read
  auto behind = [&] {
    if (!row.wo) return;
    int r = count;
    if ((reinterpret_cast<uintptr_t>(row.wo) & 15u) == 0) {      // whole 16 bytes from the next boundary on
      const int from = min((count + 3) / 4 * 4, a.length), to = a.length / 4 * 4;
      if (count + tid < from) row.wo[count + tid] = 0.f;
#pragma unroll 1
      for (int i = from + 4 * tid; i < to; i += 4 * kThreads) *reinterpret_cast<float4*>(row.wo + i) = make_float4(0.f, 0.f, 0.f, 0.f);
      r = max(from, to);
    }
#pragma unroll 1
    for (int i = r + tid; i < a.length; i += kThreads) row.wo[i] = 0.f;
  };
  // the first ones stay where they are (all of a row that is short enough)
  const int sink = c > a.keep ? a.sink : c, recent = c > a.keep ? a.recent : 0;
  row.lo = sink;
  row.hi = c - recent;
  row.left = count - sink - recent;
  const bool selects = row.left > 0;
  Part part(row, held, warp);
  if (selects) {
    part.ask(lane);
    if (tid < kWarps) listed_by[tid] = 0;
    for (int i = tid; i < kBins * kCopies / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  }
  // rows that are read again while they are written in place: the weights follow
  // when every position is known
  const bool later = row.wo == row.w && selects && part.beyond;
  if (row.wo != row.w) behind();
#pragma unroll 1
  for (int j = count + tid; j < a.keep; j += kThreads) row.out[j] = -1;
#pragma unroll 1
  for (int j = tid; j < sink; j += kThreads) {
    row.out[j] = j;
    if (row.wo && row.wo != row.w) row.wo[j] = row.w[j];
  }
  if (selects) {
    int left = row.left;
    uint32_t kth = 0;                  // the last key that stays, so far its upper bits
    int more = 0, tie = 0;             // of this thread, then of the warp: larger keys, equal ones
    int fill = 0;                      // of this warp's list
    bool listed = false;               // the keys with the first digit are there
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 31 : pass == 1 ? 21 : 10;
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      uint32_t* const bins = hist + (lane & (kCopies - 1));
      // (no weight: key 0, the lowest digit, below every one that is looked for; it
      // counts nowhere, so that rows of few do not pile up there)
      if (pass == 0) {
        __syncthreads();               // (emptied above)
        part.take_in(lane, [&](uint32_t x) {
          const uint32_t k = key_of(x);
          if (k != 0u) atomicAdd(bins + (k >> 21) * kCopies, 1u);
        });
      } else {
        for (int i = tid; i < (listed ? kBins / 4 : kBins * kCopies / 4); i += kThreads)
          reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        if (listed) {
          for (int i = lane; i < fill; i += 32) {
            const uint32_t k = list[i];
            if (k >> above == kth >> above) atomicAdd(hist + ((k >> shift) & digits), 1u);
          }
        } else {
          part.each(lane, [&](uint32_t x) {
            const uint32_t k = key_of(x);
            if (k != 0u && k >> above == kth >> above) atomicAdd(bins + ((k >> shift) & digits) * kCopies, 1u);
          });
        }
      }
      __syncthreads();
      // from the largest digit down: thread t has the kEach bins below kBins - kEach t
      constexpr int kEach = kBins / kThreads;
      static_assert(kEach == 4 && kCopies == 2, "two loads of two bins, or one of four");
      int bin[kEach], sum = 0;
      const int top = kBins / kEach - 1 - tid;
      if (listed) {
        const uint4 x = reinterpret_cast<const uint4*>(hist)[top];
        bin[0] = (int)x.w, bin[1] = (int)x.z, bin[2] = (int)x.y, bin[3] = (int)x.x;
      } else {
        const uint4 x = reinterpret_cast<const uint4*>(hist)[2 * top + 1], y = reinterpret_cast<const uint4*>(hist)[2 * top];
        bin[0] = (int)(x.z + x.w), bin[1] = (int)(x.x + x.y), bin[2] = (int)(y.z + y.w), bin[3] = (int)(y.x + y.y);
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum += bin[i];
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(FULL_MASK, upto, o);
        if (lane >= o) upto += t;
      }
      if (lane == 31) warp_sum[0][warp] = upto;
      __syncthreads();
      // the warps before: a lane each
      int before = lane < warp ? warp_sum[0][lane % kWarps] : 0;
      before = __reduce_add_sync(FULL_MASK, before) + upto - sum;
      if (before < left && left <= before + sum) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          if (before < left && left <= before + bin[i]) {
            found_digit = kBins - 1 - (tid * kEach + i);
            found_left = left - before;
          }
          before += bin[i];
        }
      }
      __syncthreads();
      kth |= found_digit << shift;
      left = found_left;
      if (pass > 0) continue;
      // The keys with that digit, usually a few in a hundred, on a list: the other
      // two digits are looked for there.  (Digit 0 has what is no weight.)
      const uint32_t first = found_digit;
      if (first != 0u)
        part.each(lane, [&](uint32_t x) {
          const uint32_t k = key_of(x), d = k >> 21;
          more += d > first;
          if (d == first) {            // (in whatever order: they are counted)
            const int to = atomicAdd(&listed_by[warp], 1);
            if (to < kList) list[to] = k;
          }
        });
      __syncwarp();
      fill = listed_by[warp];
      listed = !__syncthreads_or(first == 0u || fill > kList);
    }
    // in order: what is larger, and of those equal to the last one the first `left`
    if (listed) {
      for (int i = lane; i < fill; i += 32) more += list[i] > kth, tie += list[i] == kth;
    } else {
      more = 0;
      part.each(lane, [&](uint32_t x) {
        const uint32_t k = key_of(x);
        more += k > kth;
        tie += k == kth;
      });
    }
    more = __reduce_add_sync(FULL_MASK, more);
    tie = __reduce_add_sync(FULL_MASK, tie);
    if (lane == 0) warp_sum[0][warp] = more, warp_sum[1][warp] = tie;
    __syncthreads();                   // (and every weight was read: in place it may be overwritten, or follows later)
    const int m = lane < warp ? warp_sum[0][lane % kWarps] : 0, t = lane < warp ? warp_sum[1][lane % kWarps] : 0;
    const int m_before = __reduce_add_sync(FULL_MASK, m), t_before = __reduce_add_sync(FULL_MASK, t);
    // the place of this warp's next one: those before it, ties as far as there are places for them
    int at = row.lo + m_before + min(t_before, left), rank = t_before;
    const uint32_t below = (1u << lane) - 1u;
    // what stays is gathered in the warp's part of the histogram's memory, so that
    // it leaves 32 side by side
    uint32_t* const stack = hist + warp * (2 * kStack);
    fill = 0;
    auto flush = [&] {
      __syncwarp();
#pragma unroll 1
      for (int e = lane; e < fill; e += 32) {
        row.out[at + e] = (int)stack[e];
        if (row.wo && !later) row.wo[at + e] = __uint_as_float(stack[kStack + e]);
      }
      __syncwarp();
      at += fill;
      fill = 0;
    };
    auto take = [&](int i, uint32_t x) {
      const uint32_t k = key_of(x);
      bool stay = k >= kth;
      uint32_t sb = __ballot_sync(FULL_MASK, stay);
      if (sb == 0u) return;
      const uint32_t tb = __ballot_sync(FULL_MASK, k == kth);
      if (tb) {
        stay = k > kth || (k == kth && rank + __popc(tb & below) < left);
        sb = __ballot_sync(FULL_MASK, stay);
        rank += __popc(tb);
      }
      if (stay) {
        const int to = fill + __popc(sb & below);
        stack[to] = (uint32_t)(part.first + i * 32 + lane);
        stack[kStack + to] = number_bits(x);
      }
      fill += __popc(sb);
      if (fill > kStack - 32) flush();
    };
    if (more > 0 || (tie > 0 && rank < left)) {
      const int n = min(part.steps, kPer);
      uint32_t next = held[lane];      // (a step is 32 of this warp's: n > 0)
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const uint32_t x = next;
        next = held[min(i + 1, kPer - 1) * 32 + lane];
        take(i, x);
      }
#pragma unroll 1
      for (int i = kPer; i < part.steps; ++i) take(i, part.read(i * 32 + lane));
      flush();
    }
    if (later) {                       // position r comes from r or behind it: a stretch read before it is written
      const int to = row.lo + row.left;
#pragma unroll 1
      for (int base = row.lo; base < to; base += kThreads) {
        const int r = base + tid;
        __syncthreads();
        const float x = r < to ? row.w[row.out[r]] : 0.f;
        __syncthreads();
        if (r < to) row.wo[r] = x;
      }
    }
    __syncthreads();
  }
  // the last ones: to <= from, a stretch read before it is written
  const int to = count - recent;
#pragma unroll 1
  for (int base = 0; base < recent; base += kThreads) {
    const int i = base + tid;
    const float x = i < recent && row.wo ? row.w[row.hi + i] : 0.f;
    __syncthreads();
    if (i < recent) {
      row.out[to + i] = row.hi + i;
      if (row.wo) row.wo[to + i] = x;
    }
  }
  if (row.wo == row.w) {
    __syncthreads();
    behind();
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, int num_seqs, int heads, cudaStream_t stream) {
  if (num_seqs == 0 || heads == 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  // More rows than fit on the card at once start with the longest ones, so that
  // none of those is left for the end (64 x 8 rows of 4,096 to 32,768: 58 us in
  // order, 51 so); the ranks cost a comparison with every sequence.
  const int ranked = (int64_t)heads * num_seqs > 2 * device_sm_count() && num_seqs > 1 && num_seqs <= kRanked;
  return launch_pdl(evict_select_kernel, dim3(heads, num_seqs), dim3(kThreads), kSmemBytes, stream, a, ranked);
}

}  // namespace pkvd
