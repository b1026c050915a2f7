// mxg_codes.h - fp32 values -> 8-bit codes, as the quantizers and the norm write them.
#pragma once

#include "mxg_rows.h"

namespace mxg {

// ---- int8 -------------------------------------------------------------------

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23

// t = x / s + kMagic with the last bit corrected
__device__ __forceinline__ float corrected(float t, float x, float s, float half) {
  const float r = t - kMagic;
  const float d = fmaf(-r, s, x);
  const bool odd = (__float_as_int(t) & 1) != 0;
  if (d > half || (d == half && odd)) t += 1.0f;
  if (d < -half || (d == -half && odd)) t -= 1.0f;
  return t;
}

// The codes x / s of N values, rounded to the nearest integer of the real
// quotient (ties to even), in N / 4 words.
template <int N>
__device__ __forceinline__ void int8_codes(const float (&f)[N], float s, float inv, float half, uint32_t (&c)[N / 4]) {
  float t[N], far = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++) {
    t[i] = fmaf(f[i], inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(kMagic - t[i], s, f[i])));
  }
  if (__any(far >= half)) {
#pragma unroll
    for (int i = 0; i < N; i++) t[i] = corrected(t[i], f[i], s, half);
  }
#pragma unroll
  for (int i = 0; i < N / 4; i++) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 1]), __float_as_uint(t[4 * i]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 3]), __float_as_uint(t[4 * i + 2]), 0x04000c0cu);
    c[i] = lo | hi;
  }
}

// ---- E4M3 with a scale per block of 128 ---------------------------------------

constexpr int kBlock = 128;

// Scale of a block from the bits of its largest magnitude (infinities and NaNs
// are larger than all finite values): amax / 448 in fp32, at least 2^-126
// (so that 1 / s is finite); with pow2 the next power of two that is not
// smaller.  0 for a block of zeros, NaN for one that holds a NaN or an infinity.
__device__ __forceinline__ float block_scale(uint32_t amax, bool pow2) {
  if (amax >= 0x7f800000u) return __builtin_nanf("");
  if (amax == 0u) return 0.0f;
  const float s = fmaxf(__uint_as_float(amax) / 448.0f, 0x1p-126f);
  return pow2 ? __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u) : s;
}
// 1 / s in fp32, and 0 where s is 0 or NaN.
__device__ __forceinline__ float block_inverse(float s) { return s > 0.0f ? 1.0f / s : 0.0f; }

// x / s rounded to fp32, from inv = fl32(1 / s): the quotient x inv corrected by its
// remainder, which an fma gives exactly, is the nearest one (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, 1990).
// For s of at least 2^-60, where only quotients far below the smallest code have a
// remainder below fp32's range.  A zero keeps its sign.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float t = x * inv;
  return fmaf(-fmaf(s, t, -x), inv, t);
}

// E4M3 codes of 4 values: nearest, ties to even, saturated to +-448.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
  b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
  c = __builtin_amdgcn_fmed3f(c, -448.0f, 448.0f);
  d = __builtin_amdgcn_fmed3f(d, -448.0f, 448.0f);
  const int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
// The codes of N values in N / 4 words; `live` false: zeros (a block that holds NaNs
// or infinities).
template <int N>
__device__ __forceinline__ void e4m3_codes(const float (&f)[N], bool live, uint32_t (&c)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 4; i++) {
    const uint32_t v = e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    c[i] = live ? v : 0u;
  }
}
// Those of f / s, s and inv the block's scale and its inverse.
template <int N>
__device__ __forceinline__ void e4m3_block_codes(const float (&f)[N], float s, float inv, uint32_t (&c)[N / 4]) {
  float t[N];
  if (inv > 0x1p60f) {
#pragma unroll
    for (int i = 0; i < N; i++) t[i] = f[i] / s;
  } else {
#pragma unroll
    for (int i = 0; i < N; i++) t[i] = quotient(f[i], s, inv);
  }
  e4m3_codes<N>(t, s == s, c);
}

// Largest of a value over groups of L consecutive lanes (L = 4 .. 64), by register
// moves up to 16 lanes.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));   // neighbours
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));   // pairs
  if constexpr (L > 4) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false));  // quads
  if constexpr (L > 8) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, false));  // eights
  if constexpr (L > 16) x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  if constexpr (L > 32) x = max(x, (uint32_t)__shfl_xor((int)x, 32));
  return x;
}

template <int N>
__device__ __forceinline__ uint32_t magnitude_bits(const float (&f)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; i++) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

// Codes of N = 4 or 8 values to memory.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* q, const uint32_t (&c)[N / 4]) {
  if constexpr (N == 8)
    *reinterpret_cast<v2i*>(q) = v2i{(int)c[0], (int)c[1]};
  else
    *reinterpret_cast<uint32_t*>(q) = c[0];
}

}  // namespace mxg
