// fp8_weight_grad.hip - the weights' gradient of a product whose activations
// were kept as E4M3 codes with a scale per row and 128 columns:
//   dW[n][k] = sum_m dY[m][n] x[m][k],   x[m][k] = s[m][k / 128] q[m][k],
// dense and by expert (rows offsets[e] .. offsets[e+1] of dY, against rows
// index[p] / index_div of the codes, give dW of expert e).
//
// Products of bf16 values on the bf16 MFMA, summed in fp32.  x is rounded to
// bf16: exact where s is a power of two (a code has 4 significant bits).  dY in
// fp16 or fp32 is taken as the sum of two bf16 values (TERMS = 2), its nearest
// one and that of the rest: exact for fp16, within 2^-17 of the value for fp32.
//
// Both operands are contracted over their rows, so that a lane's 8 elements of
// an MFMA operand are a column of LDS: ds_read_b64_tr_b16 reads 4 rows of 16
// columns and hands each lane a column.  Which of the 32 rows of a step an
// element is cancels out, as both operands use the same: rows 4 g .. 4 g + 3
// and 16 + 4 g .. 16 + 4 g + 3 for lanes 16 g .. 16 g + 15, so that the 8 rows that
// 32 lanes read at once lie in different banks (rows are 288 bytes apart).
#include "mxg_experts.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kT = 128;            // tile: 128 x 128 of dW
constexpr int kBMs = 64;           // rows of a slice
constexpr int kPitch = 288;        // bytes of a row in LDS
constexpr int kTile = kBMs * kPitch;

__device__ __forceinline__ v4s read_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p));
}
// Operand of 16 columns at p (LDS; already at the lane's place) for one step of 32 rows.
__device__ __forceinline__ v8b read_operand(const uint8_t* p) {
  const v4s lo = read_tr(p), hi = read_tr(p + 16 * kPitch);
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v8s v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(v8b, v);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) { return bf16_bits(a) | (bf16_bits(b) << 16); }

// bf16 bits of f, and what they leave of it.  A finite value beyond bf16's range is
// cut off instead of rounded; infinities and NaNs leave nothing.
__device__ __forceinline__ uint32_t split_bf16(float& f) {
  uint32_t h = bf16_bits(f);
  if ((h & 0x7fffu) == 0x7f80u) h = __float_as_uint(f) >> 16;
  const float rest = f - __uint_as_float(h << 16);
  f = rest == rest ? rest : 0.0f;
  return h;
}

// 8 elements n .. n + 7 of a row of dY in fp32; past its end zeros.
template <int IN>
__device__ __forceinline__ void load8(const void* p, int64_t at, int n, int N, float (&f)[8]) {
  using T = typename RowElem<IN>::type;
  const T* q = (const T*)p + at + n;
  if (n + 8 <= N) {
    if constexpr (IN == kOutF32) {
      const v4f_any a = *reinterpret_cast<const v4f_any*>(q), b = *reinterpret_cast<const v4f_any*>(q + 4);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        f[i] = a[i];
        f[4 + i] = b[i];
      }
    } else {
      const v4i w = *reinterpret_cast<const v4i_any*>(q);
      unpack16<IN>(w, f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = n + i < N ? RowElem<IN>::get(q[i]) : 0.0f;
  }
}

template <int IN>
__global__ __launch_bounds__(256) void fp8_weight_grad_kernel(F8GradArgs a) {
  constexpr int TERMS = IN == kOutBF16 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds[(1 + TERMS) * kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int k0 = blockIdx.x * kT, n0 = blockIdx.y * kT, e = blockIdx.z;
  int m0 = 0, m1 = (int)a.M;
  if (a.offsets != nullptr) {
    // as the products read them: inside 0 .. M and never falling
    int top = max(0, min(a.offsets[0], m1));
    for (int i = 1; i <= e; i++) top = max(top, min(a.offsets[i], m1));
    m0 = top;
    m1 = max(top, min(a.offsets[e + 1], m1));
  }
  const int wk = (wave >> 1) * 64, wn = (wave & 1) * 64;
  uint8_t* lx = lds;
  uint8_t* ly = lds + kTile;
  const int g = lane >> 4, i16 = lane & 15;
  const int place = (4 * g + (i16 >> 2)) * kPitch + (i16 & 3) * 8;
  v4f acc[4][4] = {};
  for (int m = m0; m < m1; m += kBMs) {
    // codes: 64 rows x 128 columns, 16 at a time
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const int c = tid + u * 256, row = c >> 3, k = k0 + (c & 7) * 16;
      v4i w = {0, 0, 0, 0};
      float s = 0.0f;
      if (m + row < m1 && k < a.K) {
        const int64_t ar = a_row(a, m + row);
        s = __builtin_nanf("");  // rows outside A are NaN
        if (ar >= 0) {
          w = *reinterpret_cast<const v4i*>(a.A + ar * a.K + k);
          s = a.SA[ar * a.KB + blockIdx.x];
        }
      }
      v4i out[2];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[j], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[j], true);
        out[j >> 1][2 * (j & 1)] = (int)pack_bf16(lo[0] * s, lo[1] * s);
        out[j >> 1][2 * (j & 1) + 1] = (int)pack_bf16(hi[0] * s, hi[1] * s);
      }
      v4i* to = reinterpret_cast<v4i*>(lx + row * kPitch + (c & 7) * 32);
      to[0] = out[0];
      to[1] = out[1];
    }
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int c = tid + u * 256, row = c >> 4, n = n0 + (c & 15) * 8;
      float f[8];
      if (m + row < m1) {
        load8<IN>(a.dY, (int64_t)(m + row) * a.N, n, a.N, f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = 0.0f;
      }
#pragma unroll
      for (int t = 0; t < TERMS; t++) {
        v4i w;
#pragma unroll
        for (int i = 0; i < 4; i++)
          w[i] = t + 1 < TERMS ? (int)(split_bf16(f[2 * i]) | (split_bf16(f[2 * i + 1]) << 16))
                               : (int)pack_bf16(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<v4i*>(ly + t * kTile + row * kPitch + (c & 15) * 16) = w;
      }
    }
    __syncthreads();
#pragma unroll
    for (int step = 0; step < kBMs / 32; step++) {
      v8b fx[4];
#pragma unroll
      for (int i = 0; i < 4; i++) fx[i] = read_operand(lx + step * 32 * kPitch + place + (wk + 16 * i) * 2);
#pragma unroll
      for (int t = 0; t < TERMS; t++) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const v8b fy = read_operand(ly + t * kTile + step * 32 * kPitch + place + (wn + 16 * j) * 2);
#pragma unroll
          for (int i = 0; i < 4; i++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[i], fy, acc[i][j], 0, 0, 0);
        }
      }
    }
    __syncthreads();
  }
  // a lane holds columns 4 g .. 4 g + 3 of row n = lane % 16 of each fragment
  const Epi out{a.dW, nullptr, a.out_type, kActNone};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int n = n0 + wn + 16 * j + i16;
    if (n >= a.N) continue;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int k = k0 + wk + 16 * i + 4 * g;
      if (k < a.K) store_columns<true>(out, a.K, (int64_t)e * a.N + n, k, acc[i][j]);
    }
  }
}

}  // namespace

int64_t fp8_weight_grad_bytes(int64_t M, int64_t N, int64_t K, int64_t E) { return 0; }

hipError_t launch_fp8_weight_grad(const F8GradArgs& args, int y_type, hipStream_t stream) {
  F8GradArgs a = args;
  set_division(a);
  const dim3 grid((unsigned)a.KB, (unsigned)((a.N + kT - 1) / kT), (unsigned)a.E);
  if (y_type == kOutF32)
    hipLaunchKernelGGL(fp8_weight_grad_kernel<kOutF32>, grid, dim3(256), 0, stream, a);
  else if (y_type == kOutBF16)
    hipLaunchKernelGGL(fp8_weight_grad_kernel<kOutBF16>, grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(fp8_weight_grad_kernel<kOutF16>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace mxg
