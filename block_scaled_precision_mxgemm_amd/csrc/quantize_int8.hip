// quantize_int8.hip - fp32, bf16 or fp16 rows -> int8 codes with one fp32
// scale per row (a token's activations, or an output channel's weights).
//
// Rule: s = fl32(max_k |x_k| / 127), at least 2^-126 unless the row is zero
// (then s = 0); q_k = x_k / s rounded to the nearest integer, ties to even.
// A row that holds a NaN or an infinity gets s = NaN and zero codes, as a
// block of the MX quantizer does.
//
// The quotient is not formed: r = rne(x * fl32(1/s)) is within one of the
// code (|x / s| <= 127.5, so the product is off by less than 2^-16), and
// d = x - r s decides: x / s rounds up when d > s/2, down when d < -s/2, and
// at |d| = s/2 to the even one.  d is exact in fp32: it is a multiple of
// ulp(s) / 2 (or of x's own ulp where r = 0) and below 2 s.  So the codes are
// those of the real quotient, at one fma and two compares more than a
// product.
#include "mxg_internal.h"
#include "mxg_rows.h"

namespace mxg {
namespace {

constexpr int kQThreads = 256;

__device__ __forceinline__ int int8_code(float x, float s, float inv, float half) {
  float r = rintf(x * inv);
  const float d = fmaf(-r, s, x);
  const bool odd = ((int)r & 1) != 0;
  if (d > half || (d == half && odd)) r += 1.0f;
  if (d < -half || (d == -half && odd)) r -= 1.0f;
  return (int)r;
}

template <int IN>
__global__ __launch_bounds__(kQThreads) void quantize_int8_kernel(const typename RowElem<IN>::type* __restrict__ X,
                                                                  int64_t K, int8_t* __restrict__ Q,
                                                                  float* __restrict__ S) {
  constexpr int VEC = RowElem<IN>::VEC;
  __shared__ float part[kQThreads / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const v4i* x = reinterpret_cast<const v4i*>(X + row * K);
  const int nv = (int)(K / VEC);
  float amax = 0.0f;
  bool bad = false;
  for (int i = tid; i < nv; i += kQThreads) {
    float f[VEC];
    unpack16<IN>(x[i], f);
#pragma unroll
    for (int t = 0; t < VEC; t++) {
      amax = fmaxf(amax, fabsf(f[t]));
      bad |= !(fabsf(f[t]) < __builtin_inff());
    }
  }
  amax = wave_max(amax);
  if (__any(bad)) amax = __builtin_inff();
  if ((tid & 63) == 0) part[tid >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQThreads / 64; w++) amax = fmaxf(amax, part[w]);
  const bool finite = amax < __builtin_inff();
  float s = amax / 127.0f;
  if (amax > 0.0f) s = fmaxf(s, 0x1p-126f);
  if (tid == 0) S[row] = finite ? s : __builtin_nanf("");
  const bool live = finite && amax > 0.0f;
  const float inv = live ? 1.0f / s : 0.0f, half = 0.5f * s;
  for (int i = tid; i < nv; i += kQThreads) {
    float f[VEC];
    unpack16<IN>(x[i], f);
    uint32_t w[VEC / 4];
#pragma unroll
    for (int t = 0; t < VEC; t++) {
      const uint32_t c = live ? (uint32_t)(int8_code(f[t], s, inv, half) & 0xff) : 0u;
      w[t >> 2] = (t & 3) ? w[t >> 2] | (c << (8 * (t & 3))) : c;
    }
    uint32_t* q = reinterpret_cast<uint32_t*>(Q + row * K + (int64_t)i * VEC);
    q[0] = w[0];
    if constexpr (VEC == 8) q[1] = w[1];
  }
}

}  // namespace

hipError_t launch_quantize_int8(const void* X, int in_type, int64_t rows, int64_t K, int8_t* Q, float* S,
                                hipStream_t stream) {
  const dim3 grid((unsigned)rows), block(kQThreads);
  switch (in_type) {
    case kOutF32:
      hipLaunchKernelGGL(quantize_int8_kernel<kOutF32>, grid, block, 0, stream, (const float*)X, K, Q, S);
      break;
    case kOutBF16:
      hipLaunchKernelGGL(quantize_int8_kernel<kOutBF16>, grid, block, 0, stream, (const uint16_t*)X, K, Q, S);
      break;
    default:
      hipLaunchKernelGGL(quantize_int8_kernel<kOutF16>, grid, block, 0, stream, (const uint16_t*)X, K, Q, S);
  }
  return hipGetLastError();
}

}  // namespace mxg
