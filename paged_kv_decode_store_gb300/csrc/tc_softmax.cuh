// What the tcgen05 kernels with a long softmax share (prefill_mod.cu, tree_tc.cu):
// issuing products from a whole warp, waits that look at the timer late, packed
// arithmetic with kept factors, and a cap's tanh as a polynomial.
#pragma once

#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "score_mod.cuh"
#include "tcgen05.cuh"

namespace pkvd {

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// The issuing thread's own forms: descriptors as a varying low word and a
// constant high one, so that an MMA costs it two or three instructions (it
// issues everything, and a batch's first product starts when it gets there).
constexpr uint32_t desc_hi(uint32_t sbo) { return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// mbar_wait_bounded that looks at the timer only once the wait is a long one:
// a reading takes about a microsecond, which every wait would pay.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_bounded(bar, parity);
}
// The same for the two waits that last as long as an item does: twenty times
// the limit (ten seconds), some 10^9 keys.
__device__ __forceinline__ bool wait_item(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 20; ++i)
    if (wait_bounded(bar, parity)) return true;
  return false;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Packed products: d = a * b, r = r * z + c.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  unsigned long long a, b, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(d));
}
// A factor for both of a pair.  Volatile, so that it is made once: left to
// itself the compiler makes it anew for every product.
__device__ __forceinline__ uint64_t both(float c) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(c));
  return r;
}
__device__ __forceinline__ void scale2(float& d0, float& d1, uint64_t b) {
  uint64_t a;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(d0), "f"(d1));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(a));
}
__device__ __forceinline__ void scale_add2(float& d0, float& d1, uint64_t b, float c0, float c1) {
  uint64_t a, c;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(d0), "f"(d1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(c0), "f"(c1));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a) : "l"(b), "l"(c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(a));
}

__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  unsigned long long a, b, c, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(c0), "f"(c1));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(d));
}

constexpr int kCols = kTcKeys / 2;     // keys of a softmax thread

// Bits [a, z) of a 32-bit word (clamped).
__device__ __forceinline__ uint32_t span_bits(int a, int z) {
  a = min(max(a, 0), 32);
  z = min(max(z, 0), 32);
  const uint32_t below_z = z == 32 ? 0xffffffffu : (1u << z) - 1u, below_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
  return below_z & ~below_a;
}

// The factors of a thread's products: the softmax scale, the cap's polynomial.
struct Factors {
  uint64_t scale, poly[4];
};

// s r(s^2) + add on two keys, r the polynomial; `most` keeps the largest s^2.
template <bool ADD>
__device__ __forceinline__ void odd_poly2(float& v0, float& v1, const uint64_t (&coef)[4], float add0, float add1,
                                          float& most) {
  float z0, z1, r0, r1;
  mul2(z0, z1, v0, v1, v0, v1);
  most = tc_max3(most, z0, z1);
  uint64_t z, r = coef[3];
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(z0), "f"(z1));
#pragma unroll
  for (int k = 2; k >= 0; --k) asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(r), "l"(z), "l"(coef[k]));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r0), "=f"(r1) : "l"(r));
  if (ADD) fma2(v0, v1, v0, v1, r0, r1, add0, add1);
  else mul2(v0, v1, v0, v1, r0, r1);
}

// cap tanh(s / cap) log2 e as a polynomial in the raw product s, whose scale
// goes into the coefficients (not where their powers leave fp32): the largest
// square of s it is for, -1 where there is none.
inline float cap_poly(const ScoreMod& mod, float (&poly)[4]) {
  constexpr float kRatio[4] = PKVD_TANH_RATIO4;
  const double in = mod.cap_in, size = std::fabs(in);
  const double least = std::fabs(kRatio[3]) * std::pow(size, 7) * mod.cap_out_log2;
  const bool use = size > 1e-5 && size < 1e4 && least > 1e-37 && least < 1e37;
  for (int k = 0; k < 4; ++k) poly[k] = use ? (float)(kRatio[k] * std::pow(in, 2 * k + 1) * mod.cap_out_log2) : 0.f;
  return use ? (float)(kTanhNear * kTanhNear / (size * size)) : -1.f;
}

// Tensor map over q [total_q, Hq, D]: box = 64 columns x G heads x tile_tokens tokens.
inline bool encode_q_map(CUtensorMap* map, const void* q, int dtype, int head_dim, int num_q_heads, int total_q, int group,
                         int tile_tokens) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t D = head_dim;
  const cuuint64_t dims[3] = {D, (cuuint64_t)num_q_heads, (cuuint64_t)total_q};
  const cuuint64_t strides[2] = {D * 2, D * 2 * num_q_heads};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tile_tokens};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = dtype == PKVD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(map, dt, 3, const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace pkvd
