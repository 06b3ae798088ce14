// Rotary positions: query and key rows rotated by their position, on their
// own (rope) or together with the paged store of a decode step or of a varlen
// prefill batch, where the rotated key and the value go straight to their
// cache slot.
//
// Pair i of a head at position p turns by the angle a = p * inv_freq[i]:
//   y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a),
// (x1, x2) the elements (i, i + R/2) (half layout) or (2i, 2i + 1)
// (interleaved) of the head's first R dims; dims from R on are copied.
//
// Angles: far positions times a frequency need more than 32 bits (at p = 10^6
// an fp32 product is off by 0.06 rad).  inv_freq / 2 pi is taken as a 64-bit
// fixed-point fraction of a turn (off by at most 2^-65 turns); p times it
// wraps modulo one turn exactly in integer arithmetic, so the angle stays
// within fp32 accuracy up to positions of 2^40.  The phase is then split into a quadrant
// and a remainder of at most an eighth of a turn, which fp32 holds to 2^-24
// relative, and sincospif evaluates that.  One evaluation per (token, pair),
// shared by all heads through shared memory.
//
// Bound: bytes (every row read once and written once); the arithmetic is
// R/2 sincos per token and 4 FMAs per pair.
#include "common.cuh"
#include "launch.h"
#include "paging.cuh"

namespace pkvd {

namespace {

constexpr int kRopeThreads = 256;

enum : int { kRopeRows = 0, kRopeDecode = 1, kRopePrefill = 2 };

// cos and sin of a position's angle, times mscale; `step` is the turn per
// position in units of 2^-64 turns.
__device__ __forceinline__ float2 turn(int64_t pos, uint64_t step, float mscale) {
  const uint64_t phase = (uint64_t)pos * step;
  const uint64_t quarter = (phase + (1ull << 61)) >> 62;           // nearest quarter turn, modulo 4
  const int32_t rem = (int32_t)((int64_t)(phase - (quarter << 62)) >> 32);   // within +-2^29: an eighth of a turn
  float s, c;
  sincospif((float)rem * 0x1p-31f, &s, &c);                        // 2^-32 turns = 2^-31 half turns
  const bool swap = quarter & 1;
  float cc = swap ? s : c, ss = swap ? c : s;
  if ((quarter + 1) & 2) cc = -cc;                                 // quarters 1 and 2
  if (quarter & 2) ss = -ss;                                       // quarters 2 and 3
  return make_float2(cc * mscale, ss * mscale);
}

// inv_freq / 2 pi modulo one turn, in units of 2^-64 turns, rounded once: the
// product with 1 / 2 pi is kept in two doubles (its rounding error by FMA, and
// the part of 1 / 2 pi below a double).
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;   // 1 / 2 pi
  const double t = inv_freq * kHi;
  const double below = fma(inv_freq, kHi, -t) + inv_freq * kLo;
  const double a = (t - rint(t)) * 0x1p64, whole = rint(a);       // exact
  return (uint64_t)__double2ll_rn(whole) + (uint64_t)__double2ll_rn((a - whole) + below * 0x1p64);
}

template <typename T> struct Pack16;
template <> struct Pack16<float> {
  __device__ static uint4 run(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Pack16<__half> {
  __device__ static uint4 run(const float* f) {
    return make_uint4(Mma<__half>::pack(f[0], f[1]), Mma<__half>::pack(f[2], f[3]), Mma<__half>::pack(f[4], f[5]),
                      Mma<__half>::pack(f[6], f[7]));
  }
};
template <> struct Pack16<__nv_bfloat16> {
  __device__ static uint4 run(const float* f) {
    return make_uint4(Mma<__nv_bfloat16>::pack(f[0], f[1]), Mma<__nv_bfloat16>::pack(f[2], f[3]),
                      Mma<__nv_bfloat16>::pack(f[4], f[5]), Mma<__nv_bfloat16>::pack(f[6], f[7]));
  }
};

// One token per CTA.  A thread keeps one unit (a 16-byte vector, or the two
// vectors of a pair) of the head for all the heads it visits, so its cosines
// and sines are read from shared memory once.  VECTOR = false (half layout
// whose R / 2 is no whole number of vectors): elements instead of vectors.
template <typename T, int MODE, bool INTER, bool VECTOR>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs p) {
  constexpr int VEC = Vec16<T>::N;
  __shared__ float2 s_cs[kRopeMaxDim / 2];
  const int D = p.head_dim, R = p.rotary_dim;
  const int tok = blockIdx.x, tid = threadIdx.x;
  // the frequencies are a model's constants: no kernel of this library writes them
  uint64_t step = 0;
  if (tid < R / 2) step = turn_step(p.inv_freq[tid]);
  pdl_wait();
  pdl_trigger();
  int64_t pos, slot = -1;
  if (MODE == kRopeRows) {
    pos = p.positions[tok];
  } else {
    int32_t* err = tid == 0 ? p.err : nullptr;
    const TokenPlace at =
        MODE == kRopeDecode
            ? decode_place(p.tables, p.max_blocks, p.ctx, tok, p.block_size, p.num_blocks, err)
            : prefill_place(p.tables, p.max_blocks, p.cu_q, p.cu_k, p.num_seqs, tok, p.block_size, p.num_blocks, err);
    pos = at.pos;
    slot = at.slot;
    if (p.slots_out && tid == 0) p.slots_out[tok] = slot;
    if (pos < 0) {
      if (MODE == kRopeDecode) {       // an inactive row: its query is zero
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + (int64_t)tok * p.q_out_stride);
        for (int i = tid; i < p.num_q_heads * D / VEC; i += blockDim.x) o[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      return;
    }
  }
  if (tid < R / 2) s_cs[tid] = turn(pos, step, p.mscale);
  for (int i = tid + blockDim.x; i < R / 2; i += blockDim.x) s_cs[i] = turn(pos, turn_step(p.inv_freq[i]), p.mscale);
  __syncthreads();

  const T* q = static_cast<const T*>(p.q) + (int64_t)tok * p.q_stride;
  T* q_out = static_cast<T*>(p.q_out) + (int64_t)tok * p.q_out_stride;
  const T* k = static_cast<const T*>(p.k) + (int64_t)tok * p.k_stride;
  T* k_out;
  int64_t k_head = D;                  // elements between heads of the key's destination
  int heads = p.num_q_heads;
  int64_t base = 0;
  if (MODE == kRopeRows) {
    k_out = static_cast<T*>(p.k_out) + (int64_t)tok * p.k_out_stride;
    heads += p.num_kv_heads;
  } else {
    base = slot < 0 ? 0 : (slot / p.block_size) * p.block_stride + (slot % p.block_size) * p.token_stride;
    k_out = static_cast<T*>(p.k_out) + base;
    k_head = p.head_stride;
    if (slot >= 0) heads += p.num_kv_heads;
  }
  auto source = [&](int h) { return h < p.num_q_heads ? q + (int64_t)h * D : k + (int64_t)(h - p.num_q_heads) * D; };
  auto target = [&](int h) {
    return h < p.num_q_heads ? q_out + (int64_t)h * D : k_out + (int64_t)(h - p.num_q_heads) * k_head;
  };

  if constexpr (VECTOR) {
    const int turned = INTER ? (R + VEC - 1) / VEC : R / (2 * VEC);     // units with a rotated element
    const int units = INTER ? D / VEC : turned + (D - R) / VEC;
    const int per_pass = blockDim.x / units;
    const int u = tid % units;
    constexpr int P = INTER ? VEC / 2 : VEC;                            // pairs of a unit
    float cs[P], sn[P];
    if (u < turned) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int i = u * P + j;
        const float2 t = i < R / 2 ? s_cs[i] : make_float2(1.f, 0.f);
        cs[j] = t.x;
        sn[j] = t.y;
      }
    }
    if (tid < per_pass * units) {
#pragma unroll 2
      for (int h = tid / units; h < heads; h += per_pass) {
        const T* src = source(h);
        T* dst = target(h);
        if (u >= turned) {
          const int off = INTER ? u * VEC : R + (u - turned) * VEC;
          *reinterpret_cast<uint4*>(dst + off) = *reinterpret_cast<const uint4*>(src + off);
        } else if constexpr (INTER) {
          const int off = u * VEC;
          float x[VEC];
          const uint4 raw = *reinterpret_cast<const uint4*>(src + off);
          Vec16<T>::unpack(raw, x);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = a * cs[j] - b * sn[j];
            x[2 * j + 1] = b * cs[j] + a * sn[j];
          }
          const uint4 y = Pack16<T>::run(x);
          // a vector that R cuts through keeps the bits of the pairs past it
          // (W words a pair)
          constexpr int W = 4 / P;
          auto word = [&](int w, uint32_t rotated, uint32_t as_is) { return off + 2 * (w / W) < R ? rotated : as_is; };
          *reinterpret_cast<uint4*>(dst + off) =
              make_uint4(word(0, y.x, raw.x), word(1, y.y, raw.y), word(2, y.z, raw.z), word(3, y.w, raw.w));
        } else {
          const int off = u * VEC;
          float a[VEC], b[VEC];
          const uint4 ra = *reinterpret_cast<const uint4*>(src + off);
          const uint4 rb = *reinterpret_cast<const uint4*>(src + R / 2 + off);
          Vec16<T>::unpack(ra, a);
          Vec16<T>::unpack(rb, b);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float x1 = a[j], x2 = b[j];
            a[j] = x1 * cs[j] - x2 * sn[j];
            b[j] = x2 * cs[j] + x1 * sn[j];
          }
          *reinterpret_cast<uint4*>(dst + off) = Pack16<T>::run(a);
          *reinterpret_cast<uint4*>(dst + R / 2 + off) = Pack16<T>::run(b);
        }
      }
    }
  } else {
    const int units = R / 2 + (D - R);
    for (int idx = tid; idx < heads * units; idx += blockDim.x) {
      const int h = idx / units, u = idx - h * units;
      const T* src = source(h);
      T* dst = target(h);
      if (u < R / 2) {
        const float x1 = DT<T>::to_f(src[u]), x2 = DT<T>::to_f(src[u + R / 2]);
        const float2 t = s_cs[u];
        dst[u] = DT<T>::from_f(x1 * t.x - x2 * t.y);
        dst[u + R / 2] = DT<T>::from_f(x2 * t.x + x1 * t.y);
      } else {
        dst[u + R / 2] = src[u + R / 2];
      }
    }
  }
  if (MODE != kRopeRows && slot >= 0) {                                  // the value row as it is
    const T* v = static_cast<const T*>(p.v) + (int64_t)tok * p.v_stride;
    T* v_out = static_cast<T*>(p.v_out) + base;
    const int per_head = D / VEC;
    for (int i = tid; i < p.num_kv_heads * per_head; i += blockDim.x) {
      const int h = i / per_head, c = i - h * per_head;
      *reinterpret_cast<uint4*>(v_out + (int64_t)h * p.head_stride + c * VEC) =
          *reinterpret_cast<const uint4*>(v + (int64_t)h * D + c * VEC);
    }
  }
}

template <typename T, int MODE>
cudaError_t launch_typed(const RopeArgs& a, int tokens, cudaStream_t stream) {
  constexpr int VEC = Vec16<T>::N;
  const int work = (a.num_q_heads + a.num_kv_heads) * (a.head_dim / VEC);
  const int threads = work >= kRopeThreads ? kRopeThreads : work <= 128 ? 128 : (work + 31) / 32 * 32;
  const dim3 grid((unsigned)tokens), block(threads);
  if (a.interleaved) return launch_pdl(rope_kernel<T, MODE, true, true>, grid, block, 0, stream, a);
  if ((a.rotary_dim / 2) % VEC == 0) return launch_pdl(rope_kernel<T, MODE, false, true>, grid, block, 0, stream, a);
  return launch_pdl(rope_kernel<T, MODE, false, false>, grid, block, 0, stream, a);
}

template <int MODE>
cudaError_t launch_mode(const RopeArgs& a, int tokens, cudaStream_t stream) {
  if (tokens == 0) return cudaSuccess;
  if (a.dtype == PKVD_F32) return launch_typed<float, MODE>(a, tokens, stream);
  if (a.dtype == PKVD_F16) return launch_typed<__half, MODE>(a, tokens, stream);
  return launch_typed<__nv_bfloat16, MODE>(a, tokens, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int tokens, cudaStream_t stream) {
  if (a.positions) return launch_mode<kRopeRows>(a, tokens, stream);
  if (a.ctx) return launch_mode<kRopeDecode>(a, tokens, stream);
  return launch_mode<kRopePrefill>(a, tokens, stream);
}

}  // namespace pkvd
