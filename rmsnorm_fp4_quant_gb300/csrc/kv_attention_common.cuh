// kv_attention_common.cuh - device pieces of the attention kernels over the
// paged NVFP4 cache: how rows, sequences and 4-bit values are read.
//
// Arithmetic.  E2M1 codes times an E4M3 scale have at most 6 significant bits
// and lie in [2^-10, 2688]: exact in fp16, so keys and values go to the tensor
// cores as fp16 without loss.  A query row of either type is multiplied by the
// power of two that brings its largest element into [2^14, 2^15) and rounded to
// fp16: an element is off by at most 2^-25 then, half a step of fp16's smallest,
// which is 2^-39 of the row's largest, and by nothing if its last bit is 2^-24 or
// more (all bf16 elements down to 2^-31 of the largest, all fp16 ones to 2^-28).
// The power of two is taken back in the fp32 factor that turns a product into an
// exponent of 2.  Products and sums are fp32; the weights p are rounded to fp16
// (11 bits, half a step 2^-11 of p) for the second product, while their sum takes
// them in fp32.  Tensor cores take 16-bit operands at twice the rate of 32-bit ones,
// and the 4-bit values fit 16 bits: what the rounding costs is a third more error of
// fp16 outputs against 64 bits (2.8e-4 relative, 2.1e-4 with fp32 weights) and
// nothing that shows with bf16 outputs (1.7e-3 both).
#pragma once

#include "async_copy.cuh"
#include "fused_common.cuh"
#include "kv_launch.h"

namespace fp4q {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Exponents of 2 are taken against a reference r kept 6 below the largest logit
// seen when it was set, and it is set again once a logit passes r + 14: weights
// stay below 2^14 in fp16, and one that is 2^30 times smaller than the largest
// still has a bit.  A finite start keeps "nothing seen yet" free of inf - inf, and
// no logit lies below it.
constexpr float kRefStart = -3.402823466e38f;
constexpr float kRefBelow = 6.0f;
constexpr float kRefSlack = 14.0f;
// The usual exponent is one fused s * fac - r, whose product is not rounded.  r is, and
// where its steps pass kRefBelow (from 2^27) no r lies within reach of the largest
// product: the exponent of the very key that set r would be anything up to half a step
// of r.  From kRefCoarse on the product is rounded first, as the one r was made from,
// so that the largest exponent is between 0 and 8.
constexpr float kRefCoarse = 4194304.0f;
__device__ __forceinline__ bool is_coarse(float ref) { return fabsf(ref) >= kRefCoarse && ref > kRefStart; }
// The reference that a largest logit calls for.
__device__ __forceinline__ float ref_for(float ref, float product, float fac) {
  return fmaxf(ref, __fsub_rn(__fmul_rn(product, fac), kRefBelow));
}
__device__ __forceinline__ float coarse_exponent(float product, float fac, float ref) {
  return __fsub_rn(__fmul_rn(product, fac), ref);
}

// Entries of the call's small arrays (0 for one outside: the debug build's checks).
__device__ __forceinline__ int kv_len(const KvAttentionParams& p, int b) {
  return FP4Q_IN_RANGE(p, p.seq_lens + b, 4, p.seq_lens, 4LL * p.B) ? p.seq_lens[b] : 0;
}
__device__ __forceinline__ int kv_cu(const KvAttentionParams& p, int b) {
  return FP4Q_IN_RANGE(p, p.cu + b, 4, p.cu, 4LL * (p.B + 1)) ? p.cu[b] : 0;
}

// The sequence's place: rows [q0, q0 + n_q) of q, `len` keys.
struct KvSeq {
  int q0;
  int n_q;
  int len;
};
__device__ __forceinline__ KvSeq kv_sequence(const KvAttentionParams& p, int b) {
  KvSeq s;
  const int limit = static_cast<int>(p.max_pages) * p.c.page_size;
  s.len = min(max(kv_len(p, b), 0), limit);
  if (p.cu) {
    const int T = static_cast<int>(p.T);
    s.q0 = min(max(kv_cu(p, b), 0), T);
    s.n_q = max(min(kv_cu(p, b + 1), T) - s.q0, 0);
  } else {
    s.q0 = b;
    s.n_q = 1;
  }
  return s;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four bytes of two codes each -> four fp16 pairs, low nibble in the low half.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
// Two E4M3 bytes (low 16 bits of w) -> an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Bytes of two keys' codes: the low nibbles of lo, the high nibbles of hi.
__device__ __forceinline__ uint32_t low_nibbles_of(uint32_t lo, uint32_t hi) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, 0x0f0f0f0f, 0xe4;" : "=r"(d) : "r"(lo), "r"(hi));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// k with 2^k * m in [2^14, 2^15) for m > 0 (held to where 2^k and 2^-k are
// normal numbers); 0 for zero, infinity and NaN.
__device__ __forceinline__ int q_exponent(float m) {
  const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
  if (!(m > 0.0f) || e > 127) return 0;
  return min(14 - e, 100);
}
__device__ __forceinline__ float pow2(int k) {          // k in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

}  // namespace fp4q
