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
// those of the real quotient.  |d| >= s/2 is rare (about one value in 10^5):
// a lane looks at the largest |d| of the values that it holds, and a wave takes
// the corrections only if one of its lanes needs them.
//
// The sum x / s + 1.5 2^23 rounds to an integer by itself and has the code in
// its last byte, so that a value takes about 7 instructions; with 20 (a
// rounding instruction, tests on each value) the arithmetic, not the memory,
// bound the kernel: 8192 x 14336 bf16 took 80 us.
#include "mxg_codes.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

// The codes of 16 bytes of a row.
template <int IN>
__device__ __forceinline__ void put_codes(int8_t* q, const v4i& w, float s, float inv, float half) {
  constexpr int VEC = RowElem<IN>::VEC;
  float f[VEC];
  uint32_t c[VEC / 4];
  unpack16<IN>(w, f);
  int8_codes<VEC>(f, s, inv, half, c);
  store_codes<VEC>((uint8_t*)q, c);
}

// Largest magnitude bits of the elements of 16 bytes, in the element type;
// infinities and NaNs are larger than all finite values.  Two 16-bit elements
// go through one packed maximum.
typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));
template <int IN>
__device__ __forceinline__ uint32_t larger_bits(uint32_t m, const v4i& w) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (IN == kOutF32) {
      m = max(m, (uint32_t)w[i] & 0x7fffffffu);
    } else {
      const uint32_t x = (uint32_t)w[i] & 0x7fff7fffu;
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u16, m), __builtin_bit_cast(v2u16, x)));
    }
  }
  return m;
}
template <int IN>
__device__ __forceinline__ float magnitude(uint32_t m) {
  if constexpr (IN == kOutF32)
    return __uint_as_float(m);
  else
    return RowElem<IN>::get((uint16_t)max(m & 0xffffu, m >> 16));
}

// L lanes per row, in workgroups of 256 or (L = 1024) 1024.  HELD > 0: the
// row's 16-byte pieces, at most HELD of them a lane, stay in registers between
// the maximum and the codes, so that the row is read once; HELD = 0: longer
// rows are read twice, the second time from the caches.
constexpr int rows_threads(int L) { return L > 256 ? L : 256; }
template <int IN, int HELD, int L>
__global__ __launch_bounds__(rows_threads(L)) void quantize_int8_kernel(
    const typename RowElem<IN>::type* __restrict__ X, int64_t rows, int64_t K, int8_t* __restrict__ Q,
    float* __restrict__ S) {
  constexpr int VEC = RowElem<IN>::VEC;
  __shared__ float part[rows_threads(L) / 64];
  const int64_t group = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = group * (rows_threads(L) / L) + threadIdx.x / L;
  if (row >= rows) return;
  const int tid = threadIdx.x % L;
  const v4i* x = reinterpret_cast<const v4i*>(X + row * K);
  const int nv = (int)(K / VEC);
  uint32_t most = 0;
  v4i held[HELD > 0 ? HELD : 1];
  if constexpr (HELD > 0) {
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      const int i = tid + u * L;
      held[u] = i < nv ? __builtin_nontemporal_load(x + i) : v4i{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < HELD; u++) most = larger_bits<IN>(most, held[u]);
  } else {
    for (int i = tid; i < nv; i += L) most = larger_bits<IN>(most, x[i]);
  }
  float amax = magnitude<IN>(most);
  if (!(amax < __builtin_inff())) amax = __builtin_inff();  // a NaN too
#pragma unroll
  for (int d = (L < 64 ? L : 64) / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
  if constexpr (L > 64) {
    if ((tid & 63) == 0) part[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < L / 64; w++) amax = fmaxf(amax, part[w]);
  }
  const bool finite = amax < __builtin_inff();
  float s = amax / 127.0f;
  if (amax > 0.0f) s = fmaxf(s, 0x1p-126f);
  if (tid == 0) S[row] = finite ? s : __builtin_nanf("");
  const bool live = finite && amax > 0.0f;
  const float inv = live ? 1.0f / s : 0.0f, half = 0.5f * s;
  int8_t* q = Q + row * K;
  if (!live) {
    for (int i = tid; i < (int)(K / 16); i += L) reinterpret_cast<v4i*>(q)[i] = v4i{0, 0, 0, 0};
  } else if constexpr (HELD > 0) {
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      const int i = tid + u * L;
      if (i < nv) put_codes<IN>(q + (int64_t)i * VEC, held[u], s, inv, half);
    }
  } else {
    for (int i = tid; i < nv; i += L) put_codes<IN>(q + (int64_t)i * VEC, x[i], s, inv, half);
  }
}

template <int IN, int HELD, int L>
void quantize_rows(const void* X, int64_t rows, int64_t K, int8_t* Q, float* S, hipStream_t stream) {
  constexpr int threads = rows_threads(L), per = threads / L;
  // in two dimensions: a launch has less than 2^32 threads in one
  const int64_t groups = (rows + per - 1) / per, most = 1 << 20;
  const dim3 grid((unsigned)(groups < most ? groups : most), (unsigned)((groups + most - 1) / most));
  hipLaunchKernelGGL((quantize_int8_kernel<IN, HELD, L>), grid, dim3(threads), 0, stream,
                     (const typename RowElem<IN>::type*)X, rows, K, Q, S);
}

// Short rows share a wave (100000 x 128 bf16: 13 us, 34 with a wave each).  A
// wave for each row where there are enough of them to fill the chip (no barrier,
// no idle threads: 100000 x 512 in 43 us, 82 with a workgroup each).  Few rows,
// and long ones, have 16 waves each (16 x 14336: 3.7 us, 5.1 with 4 waves; 4096
// x 28672: 58 and 62; but 2047 x 8192: 15.7 and 12.6).
template <int IN>
void quantize_in(const void* X, int64_t rows, int64_t K, int8_t* Q, float* S, hipStream_t stream) {
  const int64_t pieces = K / RowElem<IN>::VEC;
  if (pieces <= 16)
    quantize_rows<IN, 1, 16>(X, rows, K, Q, S, stream);
  else if (pieces <= 2 * 16)
    quantize_rows<IN, 2, 16>(X, rows, K, Q, S, stream);
  else if (rows >= 2048 && pieces <= 64)
    quantize_rows<IN, 1, 64>(X, rows, K, Q, S, stream);
  else if (rows >= 2048 && pieces <= 2 * 64)
    quantize_rows<IN, 2, 64>(X, rows, K, Q, S, stream);
  else if (rows >= 2048 && pieces <= 4 * 64)
    quantize_rows<IN, 4, 64>(X, rows, K, Q, S, stream);
  else if (rows >= 2048 && pieces <= 8 * 64)
    quantize_rows<IN, 8, 64>(X, rows, K, Q, S, stream);
  else if (pieces <= 2 * 256)
    quantize_rows<IN, 2, 256>(X, rows, K, Q, S, stream);
  else if (rows > 512 && pieces <= 4 * 256)
    quantize_rows<IN, 4, 256>(X, rows, K, Q, S, stream);
  else if (rows > 512 && pieces <= 8 * 256)
    quantize_rows<IN, 8, 256>(X, rows, K, Q, S, stream);
  else if (pieces <= 2 * 1024)
    quantize_rows<IN, 2, 1024>(X, rows, K, Q, S, stream);
  else if (pieces <= 4 * 1024)
    quantize_rows<IN, 4, 1024>(X, rows, K, Q, S, stream);
  else if (pieces <= 8 * 1024)
    quantize_rows<IN, 8, 1024>(X, rows, K, Q, S, stream);
  else if (pieces <= 16 * 1024)
    quantize_rows<IN, 16, 1024>(X, rows, K, Q, S, stream);
  else
    quantize_rows<IN, 0, 1024>(X, rows, K, Q, S, stream);
}

}  // namespace

hipError_t launch_quantize_int8(const void* X, int in_type, int64_t rows, int64_t K, int8_t* Q, float* S,
                                hipStream_t stream) {
  switch (in_type) {
    case kOutF32:
      quantize_in<kOutF32>(X, rows, K, Q, S, stream);
      break;
    case kOutBF16:
      quantize_in<kOutBF16>(X, rows, K, Q, S, stream);
      break;
    default:
      quantize_in<kOutF16>(X, rows, K, Q, S, stream);
  }
  return hipGetLastError();
}

}  // namespace mxg
