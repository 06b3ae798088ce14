// What each cached key was given: the softmax weights of a decode step, summed
// over the query heads of a KV head (or all of them) and added to what earlier
// steps gave.
//   weights_out[i][h][j] = weights[i][h][j] + sum_g 2^(s_gj - M_g) / L_g
//
// A weight needs its row's maximum and sum, which are known when the last key
// has been read.  Reading the keys again would cost half of the attention's
// bytes once more; so the partition kernel leaves the scores it computes anyway
// (4 bytes a query head and key: 1 / 16 of the K/V bytes for 8 query heads a KV
// head of 128 in 16 bits), the merge kernel the rows' statistics, and this kernel,
// bound by bytes, turns scores into weights.  Each element has one thread, so
// no atomics: the sums are the same in every run.  64 rows of up to 32,768 keys, 64
// + 8 heads of 128 in bf16, take 408 us where the plain call takes 358 (floor 322): the
// partition kernel 361, this one 40 for 137 MB of scores, which do not stay in L2.
#include "attention_kernels.cuh"

namespace pkvd {

namespace {

constexpr int kThreads = 128, kPer = 4;     // positions of a thread, side by side

// (scores and stats are written by kernels that this one may be scheduled
// beside: plain loads, behind the wait)
__global__ void __launch_bounds__(kThreads) add_weights_kernel(const float* scores, int64_t score_ld,
                                                               const float2* stats, float lift,
                                                               const float* win, float* wout, int64_t seq_stride,
                                                               int64_t head_stride, const int32_t* __restrict__ ctx,
                                                               int ctx_cap, int window, int hq, int group, int wide) {
  const int h = blockIdx.y, i = blockIdx.z;
  const int c = min(max(ctx[i], 0), ctx_cap);
  pdl_wait();
  pdl_trigger();
  const int first = window_start(c, window);
  for (int j = ((int)blockIdx.x * kThreads + (int)threadIdx.x) * kPer; j < c; j += (int)gridDim.x * kThreads * kPer) {
    const float* w = win + (int64_t)i * seq_stride + (int64_t)h * head_stride + j;
    float* o = wout + (int64_t)i * seq_stride + (int64_t)h * head_stride + j;
    const bool whole = j + kPer <= c;
    float sum[kPer] = {}, before[kPer] = {};
    if (wide && whole) {
      const float4 x = *reinterpret_cast<const float4*>(w);
      before[0] = x.x, before[1] = x.y, before[2] = x.z, before[3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (j + k < c) before[k] = w[k];
    }
    if (j + kPer > first) {
      const int64_t row0 = (int64_t)i * hq + (int64_t)h * group;
      // rows of whole groups of eight: a group of four behind the context or before
      // the window may hold anything, and is left out below
      const float* s = scores + row0 * score_ld + j;
#pragma unroll 8
      for (int g = 0; g < group; ++g) {
        const float2 st = stats[row0 + g];
        const float4 x = *reinterpret_cast<const float4*>(s + g * score_ld);
        const float m = st.x - lift;
        const float y[kPer] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < kPer; ++k) sum[k] = fmaf(exp2f(y[k] - m), st.y, sum[k]);
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (j + k < first) sum[k] = 0.f;
    }
    if (wide && whole) {
      *reinterpret_cast<float4*>(o) =
          make_float4(before[0] + sum[0], before[1] + sum[1], before[2] + sum[2], before[3] + sum[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (j + k < c) o[k] = before[k] + sum[k];
    }
  }
}

}  // namespace

int64_t score_row(int max_context_len) { return ((int64_t)max_context_len + 7) / 8 * 8; }

cudaError_t launch_attention_weights(const AttnArgs& a, const WeightArgs& w, cudaStream_t stream) {
  cudaError_t e = launch_attention(a, stream);
  if (e != cudaSuccess || a.grid == 0) return e;
  const long long cap = (long long)a.max_blocks_per_seq * a.block_size;
  const int ctx_cap = (int)(cap < a.max_context_len ? cap : a.max_context_len);
  // f16 weights are lifted in the partition kernel's sums on the tensor cores
  const float lift = a.path == PKVD_PATH_MMA && a.dtype == PKVD_F16 ? kWeightLift<__half> : 0.f;
  auto whole16 = [](int64_t x) { return x % 16 == 0; };
  const int wide = whole16((int64_t)reinterpret_cast<uintptr_t>(w.in)) && whole16((int64_t)reinterpret_cast<uintptr_t>(w.out)) &&
                   whole16(w.seq_stride * 4) && whole16(w.head_stride * 4);
  const int span = kThreads * kPer;
  // rows are of all lengths: few CTAs each that walk it, rather than many of which most find nothing
  const int64_t rows = (int64_t)w.heads * a.num_seqs, most = (ctx_cap + span - 1) / span;
  const int64_t each = 48 * (int64_t)device_sm_count() / rows + 1;
  const dim3 grid((unsigned)(each < most ? each : most), (unsigned)w.heads, (unsigned)a.num_seqs);
  return launch_pdl(add_weights_kernel, grid, dim3(kThreads), 0, stream, (const float*)a.scores, a.score_ld,
                    (const float2*)a.stats, lift, w.in, w.out, w.seq_stride, w.head_stride, a.context_lens, ctx_cap,
                    a.window, a.num_q_heads, a.num_q_heads / w.heads, wide);
}

}  // namespace pkvd
