// quantize_fp8.hip - fp32, bf16 or fp16 rows -> E4M3 codes with one fp32 scale
// per row and 128 columns (activations) or per 128 x 128 block (weights).
//
// Rule: s from the block's largest magnitude (block_scale in mxg_codes.h);
// code = fl32(x / s) rounded to the nearest E4M3 value, ties to even, saturated to
// +-448.  A block that holds a NaN or an infinity gets s = NaN and
// zero codes, as a block of the MX quantizer does.
//
// Both kernels hold a block in registers between its maximum and its codes, so
// that X is read once; they are bound by memory: 14336 x 4096 of fp32 by blocks takes
// 48.8 us (294 MB, 6.0 TB/s, where a large copy reaches 5.0 and a read 5.9), 16 x 8192 of
// bf16 by rows 3.6, of a call's 9.5 through Python.
#include "mxg_codes.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

// ---- a scale per row and 128 columns -----------------------------------------
//
// A block is 16 (fp32: 32) lanes of 16 bytes; a workgroup takes kUnroll runs of
// 256 lanes.  WHOLE: K is a multiple of 128, so that the blocks follow one
// another in memory; else the row of a block is found by a division (by
// multiplication: d below 2^31).
constexpr int kUnroll = 4;

struct RowDiv {
  uint32_t mul;
  int shift;
};

template <int IN, bool WHOLE>
__global__ __launch_bounds__(256) void quantize_fp8_rows_kernel(const typename RowElem<IN>::type* __restrict__ X,
                                                                int total, int KB, int K, RowDiv div, bool pow2,
                                                                uint8_t* __restrict__ Q, float* __restrict__ S) {
  constexpr int VEC = RowElem<IN>::VEC, L = kBlock / VEC, PER = 256 / L;
  const int sub = threadIdx.x % L;
  const int64_t b0 = (int64_t)blockIdx.x * (PER * kUnroll) + threadIdx.x / L;
  v4i w[kUnroll];
  int64_t at[kUnroll];  // element; -1: none
#pragma unroll
  for (int u = 0; u < kUnroll; u++) {
    const int64_t b = b0 + u * PER;
    at[u] = -1;
    if (b < total) {
      if (WHOLE) {
        at[u] = b * kBlock + sub * VEC;
      } else {
        const uint32_t row = (uint32_t)(((uint64_t)(uint32_t)b * div.mul) >> div.shift);
        const int k = ((int)b - (int)row * KB) * kBlock + sub * VEC;
        if (k < K) at[u] = (int64_t)row * K + k;
      }
    }
    w[u] = at[u] >= 0 ? __builtin_nontemporal_load(reinterpret_cast<const v4i*>(X + at[u])) : v4i{0, 0, 0, 0};
  }
#pragma unroll
  for (int u = 0; u < kUnroll; u++) {
    const int64_t b = b0 + u * PER;
    float f[VEC];
    uint32_t c[VEC / 4];
    unpack16<IN>(w[u], f);
    const uint32_t amax = lanes_max<L>(magnitude_bits<VEC>(f));
    const float s = block_scale(amax, pow2), inv = block_inverse(s);
    e4m3_block_codes<VEC>(f, s, inv, c);
    if (at[u] >= 0) store_codes<VEC>(Q + at[u], c);
    if (b < total && sub == 0) S[b] = s;
  }
}

// ---- a scale per 128 x 128 block ----------------------------------------------
//
// A workgroup of 512 takes a block: 4 (fp32: 8) pieces of 16 bytes a lane.
template <int IN>
__global__ __launch_bounds__(512) void quantize_fp8_blocks_kernel(const typename RowElem<IN>::type* __restrict__ X,
                                                                  int rows, int K, bool pow2, uint8_t* __restrict__ Q,
                                                                  float* __restrict__ S) {
  constexpr int VEC = RowElem<IN>::VEC, L = kBlock / VEC, STEP = 512 / L, U = kBlock / STEP;
  __shared__ uint32_t part[8];
  const int64_t base = (int64_t)blockIdx.z * rows * K;
  const int k = blockIdx.x * kBlock + threadIdx.x % L * VEC;
  const int row0 = blockIdx.y * kBlock + threadIdx.x / L;
  v4i w[U];
  uint32_t most = 0;
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int row = row0 + u * STEP;
    w[u] = row < rows && k < K
               ? __builtin_nontemporal_load(reinterpret_cast<const v4i*>(X + base + (int64_t)row * K + k))
               : v4i{0, 0, 0, 0};
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    float f[VEC];
    unpack16<IN>(w[u], f);
    most = max(most, magnitude_bits<VEC>(f));
  }
  most = lanes_max<64>(most);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; i++) most = max(most, part[i]);
  const float s = block_scale(most, pow2), inv = block_inverse(s);
  if (threadIdx.x == 0) S[((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = s;
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int row = row0 + u * STEP;
    if (row < rows && k < K) {
      float f[VEC];
      uint32_t c[VEC / 4];
      unpack16<IN>(w[u], f);
      e4m3_block_codes<VEC>(f, s, inv, c);
      store_codes<VEC>(Q + base + (int64_t)row * K + k, c);
    }
  }
}

template <int IN>
hipError_t quantize_in(const void* X, int64_t E, int64_t rows, int64_t K, int block_rows, bool pow2, uint8_t* Q, float* S,
                       hipStream_t stream) {
  using T = typename RowElem<IN>::type;
  const int KB = (int)((K + kBlock - 1) / kBlock);
  if (block_rows == kBlock) {
    const dim3 grid((unsigned)KB, (unsigned)((rows + kBlock - 1) / kBlock), (unsigned)E);
    hipLaunchKernelGGL((quantize_fp8_blocks_kernel<IN>), grid, dim3(512), 0, stream, (const T*)X, (int)rows, (int)K, pow2,
                       Q, S);
    return hipGetLastError();
  }
  RowDiv div;
  int s = 0;
  while (((int64_t)1 << s) < KB) s++;
  div.mul = (uint32_t)(((uint64_t)1 << (31 + s)) / (uint32_t)KB + 1);
  div.shift = 31 + s;
  // at most 2^26 blocks in a launch: their numbers are 32-bit, its threads fewer than 2^32
  constexpr int per = 256 / (kBlock / RowElem<IN>::VEC) * kUnroll;
  const int64_t all = E * rows, most = ((int64_t)1 << 26) / KB;
  for (int64_t r = 0; r < all; r += most) {
    const int64_t n = all - r < most ? all - r : most;
    const dim3 grid((unsigned)((n * KB + per - 1) / per));
    if (K % kBlock == 0)
      hipLaunchKernelGGL((quantize_fp8_rows_kernel<IN, true>), grid, dim3(256), 0, stream, (const T*)X + r * K,
                         (int)(n * KB), KB, (int)K, div, pow2, Q + r * K, S + r * KB);
    else
      hipLaunchKernelGGL((quantize_fp8_rows_kernel<IN, false>), grid, dim3(256), 0, stream, (const T*)X + r * K,
                         (int)(n * KB), KB, (int)K, div, pow2, Q + r * K, S + r * KB);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize_fp8(const void* X, int in_type, int64_t E, int64_t rows, int64_t K, int block_rows, bool pow2,
                               uint8_t* Q, float* S, hipStream_t stream) {
  switch (in_type) {
    case kOutF32:
      return quantize_in<kOutF32>(X, E, rows, K, block_rows, pow2, Q, S, stream);
    case kOutBF16:
      return quantize_in<kOutBF16>(X, E, rows, K, block_rows, pow2, Q, S, stream);
    default:
      return quantize_in<kOutF16>(X, E, rows, K, block_rows, pow2, Q, S, stream);
  }
}

}  // namespace mxg
