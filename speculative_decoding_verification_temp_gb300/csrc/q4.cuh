// Rows of a 4-bit cache.  A row of D values (one head of one token) is D / 8
// words of 32 bits, then four pairs (scale, minimum) of float16, one per group of
// D / 4 values: D / 2 + 16 bytes.  Bits 4i of word w hold the code of value 8w + 2i,
// bits 16 + 4i that of value 8w + 2i + 1, so that one mask takes two neighbouring
// values into the halves of a register, and the halves of two tokens' words can be
// swapped into pairs of tokens.  A code n stands for minimum + scale n.
//
// Four groups whatever D is: the pairs are one 16-byte piece, and rows keep the 16-byte
// alignment that copies want.  Scale and minimum are float16: eleven bits place the
// minimum to within 1/30 of a step in groups whose values lie within their spread of
// zero (bfloat16 would be off by up to 1/4 there); values beyond 61440 = 15 * 4096 are
// taken as that, so that no scale and no value that a row stands for leaves float16.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sv {

constexpr int kQ4Groups = 4;
constexpr float kQ4Limit = 61440.f;
__host__ __device__ constexpr int q4_row_bytes(int D) { return D / 2 + 16; }

// Eight codes of a word as float32, in the order of their values.
__device__ __forceinline__ void q4_codes(uint32_t w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = static_cast<float>((w >> (4 * i)) & 15u);
    x[2 * i + 1] = static_cast<float>((w >> (16 + 4 * i)) & 15u);
  }
}

__device__ __forceinline__ float2 q4_pair(uint32_t scale_min) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&scale_min));
}

// Whether a group with this (scale, minimum) pair stands for numbers: both are finite, and
// then m + s n is for every code (below 2^20, whose sixteenth is still one of float16's).
// Otherwise none of its values is: an infinite or unknown scale times any code, 0 too, is
// not finite.
__device__ __forceinline__ bool q4_finite(uint32_t scale_min) {
  return (((scale_min & 0x7C007C00u) + 0x04000400u) & 0x80008000u) == 0;
}

// Values that are the same float32 operations in a group's every thread: the codes
// are those of round((x - minimum) (1 / scale)) wherever they are computed.
struct Q4Scale {
  float low, inverse;
  uint32_t bits;
};
// lo, hi: smallest and largest value of the group; bad: one is an infinity or NaN.
__device__ __forceinline__ Q4Scale q4_scale(float lo, float hi, bool bad) {
  const __half m = __float2half_rn(lo);
  const float low = __half2float(m);
  const __half s = __float2half_rn(__fmul_rn(__fsub_rn(hi, low), 1.f / 15.f));
  Q4Scale q;
  q.low = low;
  const float scale = __half2float(s);
  q.inverse = scale == 0.f || bad ? 0.f : __fdiv_rn(1.f, scale);
  q.bits = bad ? 0x7E007E00u
               : (static_cast<uint32_t>(__half_as_ushort(m)) << 16) | __half_as_ushort(s);
  return q;
}
__device__ __forceinline__ uint32_t q4_word(const Q4Scale &q, const float (&x)[8]) {
  uint32_t w = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float n = rintf(__fmul_rn(__fsub_rn(x[e], q.low), q.inverse));
    const uint32_t code = static_cast<uint32_t>(fminf(fmaxf(n, 0.f), 15.f));
    w |= code << ((e & 1) * 16 + (e >> 1) * 4);
  }
  return w;
}

}  // namespace sv
