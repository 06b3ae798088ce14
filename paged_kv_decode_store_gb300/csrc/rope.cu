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
// fixed-point fraction of a turn (off by at most 2^-65 turns), found in
// integer arithmetic from the double's bits; p times it wraps modulo one turn
// exactly, so the angle stays within fp32 accuracy up to positions of 2^40.
// The phase is then split into a quadrant and a remainder of at most an
// eighth of a turn, which fp32 holds to 2^-24 relative, and sincospif
// evaluates that.
//
// Layout of the work: an item is some heads of one token, one warp each, with
// no barrier between warps.  The lanes evaluate the token's R/2 angles once
// into the warp's shared memory, then share out units of two 16-byte vectors
// (the two halves of eight or four pairs, or two neighbouring vectors), two
// units a lane loaded ahead (four take more registers than the loads in
// flight are worth: 8192 prefill rows of 48 + 8 + 8 heads 60 us against 48;
// one 48 there, but 27 us for the half-rotated rows below).  Bound: bytes, every row read once and written once.  Those 8192
// rows take 48 us (5.5 TB/s of rows), 18433 rows of 16 + 16 heads of 64 half
// rotated 26 us (5.7 TB/s); one CTA a token with a barrier between angles and
// rows took 70 and 55 us.
#include "common.cuh"
#include "launch.h"
#include "paging.cuh"

namespace pkvd {

namespace {

constexpr int kRopeThreads = 128;     // four warps, each on its own
constexpr int kRopeCtas = 8;          // resident on an SM

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

// inv_freq / 2 pi modulo one turn, in units of 2^-64 turns, rounded to nearest:
// the double is M 2^E with an integer M, 1 / 2 pi is C 2^-128, and the bits of
// M C from 64 - E up are the result (those of FP64 arithmetic would take its
// pipe, which has a sixtieth of the rate).  Frequencies of 2^64 and more count
// as 0: their products would need more bits than C has.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
  constexpr uint64_t kC1 = 0x28be60db9391054aull, kC0 = 0x7f09d5f47d4d3770ull;
  const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq);
  const int ex = (int)((bits >> 52) & 0x7ff);
  const uint64_t m = (bits & 0x000fffffffffffffull) | (ex ? 1ull << 52 : 0ull);
  const int s = 64 - ((ex ? ex : 1) - 1075);                 // first bit of the result
  // M C in three words
  const uint64_t p0 = m * kC0, lo1 = m * kC1;
  const uint64_t p1 = __umul64hi(m, kC0) + lo1;
  const uint64_t p2 = __umul64hi(m, kC1) + (p1 < lo1);
  auto from = [&](int at) -> uint64_t {                      // 64 bits from bit `at` on
    const int w = at >> 6, r = at & 63;
    const uint64_t lo = w == 0 ? p0 : w == 1 ? p1 : w == 2 ? p2 : 0, hi = w == 0 ? p1 : w == 1 ? p2 : 0;
    return r ? (lo >> r) | (hi << (64 - r)) : lo;
  };
  uint64_t t = ex < 1023 + 64 && s < 192 ? from(s) + (from(s - 1) & 1u) : 0;
  return (bits >> 63) ? 0 - t : t;
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

// Where a prefill row goes, found by a whole warp: the sequence by a 32-way
// search of cu_q (two loads for up to 1024 sequences), then as prefill_place.
__device__ __forceinline__ TokenPlace prefill_place_warp(const RopeArgs& p, int t, int32_t* err) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.num_seqs + 1;                            // cu_q[lo] <= t, the last such is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    const unsigned le = __ballot_sync(FULL_MASK, i < n && p.cu_q[lo + i] <= t);
    const int k = le ? 31 - __clz(le) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  if (lo >= p.num_seqs) return {-1, -1};                     // behind the batch
  const int q0 = p.cu_q[lo], q1 = p.cu_q[lo + 1];
  const int qlen = q1 - q0, klen = p.cu_k[lo + 1] - p.cu_k[lo];
  if (t < q0 || t >= q1 || klen < qlen) {
    flag_error(err, PKVD_ERR_CONTEXT);
    return {-1, -1};
  }
  const int pos = klen - qlen + (t - q0);
  return {pos, slot_of(p.tables + (int64_t)lo * p.max_blocks, p.max_blocks, pos, p.block_size, p.num_blocks, err)};
}

// VECTOR = false (half layout whose R / 2 is no whole number of vectors):
// elements instead of vectors.
template <typename T, int MODE, bool INTER, bool VECTOR>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeArgs p) {
  constexpr int VEC = Vec16<T>::N;
  constexpr int kBatch = 2;                                  // units a lane loads ahead
  extern __shared__ float2 s_all[];
  const int D = p.head_dim, R = p.rotary_dim, half = R / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* s_cs = s_all + warp * half;
  const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / 32) + warp;
  const int tok = (int)(item / p.parts), part = (int)(item - (int64_t)tok * p.parts);
  // the frequencies are a model's constants: no kernel of this library writes them
  uint64_t step0 = 0, step1 = 0;
  if (lane < half) step0 = turn_step(p.inv_freq[lane]);
  if (lane + 32 < half) step1 = turn_step(p.inv_freq[lane + 32]);
  pdl_wait();
  pdl_trigger();
  if (tok >= p.num_tokens) return;
  // this item's heads: of the query, then the key, then the value
  const int hq = p.num_q_heads, hk = hq + p.num_kv_heads;
  const int h0 = part * p.part_heads;
  const int h1 = min(h0 + p.part_heads, MODE == kRopeRows ? hk : hk + p.num_kv_heads);
  const T* q = static_cast<const T*>(p.q) + (int64_t)tok * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + (int64_t)tok * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + (int64_t)tok * p.v_stride;
  auto source = [&](int h) {
    return h < hq ? q + (int64_t)h * D : h < hk ? k + (int64_t)(h - hq) * D : v + (int64_t)(h - hk) * D;
  };
  // a unit's two vectors: units below `turned` hold rotated elements
  const int turned = INTER ? (R + 2 * VEC - 1) / (2 * VEC) : half / VEC;
  auto first_of = [&](int u) { return INTER ? 2 * u * VEC : u < turned ? u * VEC : R + 2 * (u - turned) * VEC; };
  auto second_of = [&](int u) { return first_of(u) + (!INTER && u < turned ? half : VEC); };
  const int units = (D / VEC + 1) / 2;
  const int dh = 32 / units, du = 32 - dh * units;              // a lane's next unit: dh heads and du units on
  int h = h0 + lane / units, u = lane % units;
  uint4 xa[kBatch], xb[kBatch];
  int bh[kBatch], bu[kBatch];
  auto load = [&] {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      bh[i] = h;
      bu[i] = u;
      if (h < h1) {
        const T* src = source(h);
        xa[i] = *reinterpret_cast<const uint4*>(src + first_of(u));
        if (second_of(u) < D) xb[i] = *reinterpret_cast<const uint4*>(src + second_of(u));
      }
      h += dh;
      u += du;
      if (u >= units) u -= units, ++h;
    }
  };
  if (VECTOR) load();                                            // on its way while the row's place is looked up

  int64_t pos, slot = -1;
  if (MODE == kRopeRows) {
    pos = p.positions[tok];
  } else {
    int32_t* err = part == 0 && lane == 0 ? p.err : nullptr;
    const TokenPlace at = MODE == kRopeDecode ? decode_place(p.tables, p.max_blocks, p.ctx, tok, p.block_size,
                                                             p.num_blocks, err)
                                              : prefill_place_warp(p, tok, err);
    pos = at.pos;
    slot = at.slot;
    if (p.slots_out && part == 0 && lane == 0) p.slots_out[tok] = slot;
  }
  const int64_t base =
      slot < 0 ? 0 : (slot / p.block_size) * p.block_stride + (slot % p.block_size) * p.token_stride;
  T* q_out = static_cast<T*>(p.q_out) + (int64_t)tok * p.q_out_stride;
  T* k_out = static_cast<T*>(p.k_out) + (MODE == kRopeRows ? (int64_t)tok * p.k_out_stride : base);
  const int64_t k_head = MODE == kRopeRows ? D : p.head_stride;   // elements between heads of the key's target
  T* v_out = static_cast<T*>(p.v_out) + base;
  const int h_end = MODE != kRopeRows && slot < 0 ? min(h1, hq) : h1;   // without a slot only the query is written
  if (MODE != kRopeRows && pos < 0) {
    if (MODE == kRopeDecode) {                                    // an inactive row: its query is zero
      for (int g = h0; g < h_end; ++g)
        for (int i = lane; i < D / VEC; i += 32)
          reinterpret_cast<uint4*>(q_out + (int64_t)g * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  auto target = [&](int h) {
    return h < hq   ? q_out + (int64_t)h * D
           : h < hk ? k_out + (int64_t)(h - hq) * k_head
                    : v_out + (int64_t)(h - hk) * p.head_stride;
  };
  for (int i = lane; i < half; i += 32)
    s_cs[i] = turn(pos, i < 32 ? step0 : i < 64 ? step1 : turn_step(p.inv_freq[i]), p.mscale);
  __syncwarp();

  if constexpr (VECTOR) {
    // cos and sin of a unit's VEC pairs; a lane whose units are the same one of
    // every head keeps them (reading them a unit at a time from shared memory,
    // four lanes to a bank, takes 55 us instead of 48 for 8192 prefill rows)
    float2 t[VEC];
    auto pairs_of = [&](int u) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) t[j] = !INTER || u * VEC + j < half ? s_cs[u * VEC + j] : make_float2(1.f, 0.f);
    };
    const bool same = du == 0;
    if (same && u < turned) pairs_of(u);
    for (;;) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (bh[i] >= h_end) continue;
        const int uu = bu[i], oa = first_of(uu), ob = second_of(uu);
        T* dst = target(bh[i]);
        if (uu < turned && bh[i] < hk) {
          float a[VEC], b[VEC];
          Vec16<T>::unpack(xa[i], a);
          Vec16<T>::unpack(xb[i], b);
          if (!same) pairs_of(uu);
          if constexpr (INTER) {
            auto rotate = [&](float* x, int off, const float2* t, uint4& raw) {
#pragma unroll
              for (int j = 0; j < VEC / 2; ++j) {
                const float x1 = x[2 * j], x2 = x[2 * j + 1];
                x[2 * j] = x1 * t[j].x - x2 * t[j].y;
                x[2 * j + 1] = x2 * t[j].x + x1 * t[j].y;
              }
              const uint4 y = Pack16<T>::run(x);
              // a vector that R cuts through keeps the bits of the pairs past
              // it (W words a pair)
              constexpr int W = 4 / (VEC / 2);
              auto word = [&](int w, uint32_t rotated, uint32_t as_is) { return off + 2 * (w / W) < R ? rotated : as_is; };
              raw = make_uint4(word(0, y.x, raw.x), word(1, y.y, raw.y), word(2, y.z, raw.z), word(3, y.w, raw.w));
            };
            rotate(a, oa, t, xa[i]);
            rotate(b, ob, t + VEC / 2, xb[i]);
          } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              const float x1 = a[j], x2 = b[j];
              a[j] = x1 * t[j].x - x2 * t[j].y;
              b[j] = x2 * t[j].x + x1 * t[j].y;
            }
            xa[i] = Pack16<T>::run(a);
            xb[i] = Pack16<T>::run(b);
          }
        }
        *reinterpret_cast<uint4*>(dst + oa) = xa[i];
        if (ob < D) *reinterpret_cast<uint4*>(dst + ob) = xb[i];
      }
      if (!__any_sync(FULL_MASK, h < h_end)) break;
      load();
    }
  } else {
    const int elems = half + (D - R);
    for (int idx = lane; idx < (h_end - h0) * elems; idx += 32) {
      const int h = h0 + idx / elems, u = idx % elems;
      const T* src = source(h);
      T* dst = target(h);
      if (u < half) {
        const T r1 = src[u], r2 = src[u + half];
        const float x1 = DT<T>::to_f(r1), x2 = DT<T>::to_f(r2);
        const float2 t = s_cs[u];
        dst[u] = h < hk ? DT<T>::from_f(x1 * t.x - x2 * t.y) : r1;
        dst[u + half] = h < hk ? DT<T>::from_f(x2 * t.x + x1 * t.y) : r2;
      } else {
        dst[u + half] = src[u + half];
      }
    }
  }
}

template <typename T, int MODE>
cudaError_t launch_typed(RopeArgs a, int tokens, cudaStream_t stream) {
  constexpr int VEC = Vec16<T>::N;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // A warp's share of a token's heads: as many as make 32 warps an SM when
  // there are few tokens, at least one pass of the warp over its units and at
  // most sixteen.
  const int heads = a.num_q_heads + a.num_kv_heads * (MODE == kRopeRows ? 1 : 2);
  const int units = (a.head_dim / VEC + 1) / 2;
  const int pass = units >= 32 ? 1 : 32 / units;                  // heads of a pass
  const int passes = (heads + pass - 1) / pass;
  int64_t parts = ((int64_t)sms * 32 + tokens - 1) / tokens;
  parts = parts < (passes + 15) / 16 ? (passes + 15) / 16 : parts > passes ? passes : parts;
  a.part_heads = (passes + (int)parts - 1) / (int)parts * pass;
  a.parts = (heads + a.part_heads - 1) / a.part_heads;
  a.num_tokens = tokens;
  const int64_t ctas = ((int64_t)tokens * a.parts + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)ctas), block(kRopeThreads);
  const size_t smem = (size_t)(kRopeThreads / 32) * (a.rotary_dim / 2) * sizeof(float2);
  if (a.interleaved) return launch_pdl(rope_kernel<T, MODE, true, true>, grid, block, smem, stream, a);
  if ((a.rotary_dim / 2) % VEC == 0) return launch_pdl(rope_kernel<T, MODE, false, true>, grid, block, smem, stream, a);
  return launch_pdl(rope_kernel<T, MODE, false, false>, grid, block, smem, stream, a);
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
