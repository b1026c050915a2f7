// mxg_rows.h - rows of fp32, bf16 or fp16 elements as the int8 quantizer and
// the expert kernels read and write them, and scans over a wave.
#pragma once

#include "mxg_epilogue.h"

namespace mxg {

// An element type by its kOut* id: VEC elements make 16 bytes.
template <int TYPE>
struct RowElem;
template <>
struct RowElem<kOutF32> {
  using type = float;
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct RowElem<kOutBF16> {
  using type = uint16_t;
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
  static __device__ __forceinline__ uint16_t put(float x) { return (uint16_t)bf16_bits(x); }
};
template <>
struct RowElem<kOutF16> {
  using type = uint16_t;
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }
  static __device__ __forceinline__ uint16_t put(float x) { return (uint16_t)f16_bits(x); }
};

// The VEC elements of 16 bytes as fp32, and back.
template <int TYPE>
__device__ __forceinline__ void unpack16(const v4i& w, float (&f)[RowElem<TYPE>::VEC]) {
  if constexpr (TYPE == kOutF32) {
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = __int_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = RowElem<TYPE>::get((uint16_t)((uint32_t)w[i] & 0xffffu));
      f[2 * i + 1] = RowElem<TYPE>::get((uint16_t)((uint32_t)w[i] >> 16));
    }
  }
}
template <int TYPE>
__device__ __forceinline__ v4i pack16(const float (&f)[RowElem<TYPE>::VEC]) {
  v4i w;
  if constexpr (TYPE == kOutF32) {
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = __float_as_int(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      w[i] = (int)((uint32_t)RowElem<TYPE>::put(f[2 * i]) | ((uint32_t)RowElem<TYPE>::put(f[2 * i + 1]) << 16));
  }
  return w;
}

// LDS written by some lanes of a wave is read by others behind this (the wave's
// LDS instructions run in order; the fences keep the compiler to it).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Inclusive scans over the lanes of a wave by DPP (shifts within rows of 16,
// then the rows' last values passed on): a few cycles a step, where a shuffle
// goes through LDS.
template <bool MAX>
__device__ __forceinline__ int scan_op(int x, int y) {
  return MAX ? max(x, y) : x + y;
}
template <bool MAX>
__device__ __forceinline__ int wave_scan(int x) {  // MAX: values of at least 0
  x = scan_op<MAX>(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
  x = scan_op<MAX>(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
  x = scan_op<MAX>(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
  x = scan_op<MAX>(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
  x = scan_op<MAX>(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
  x = scan_op<MAX>(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
  return x;
}

}  // namespace mxg
