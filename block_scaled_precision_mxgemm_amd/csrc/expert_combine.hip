// expert_combine.hip - the experts' outputs weighted and summed per token,
//   out_t = sum_j w_tj y[position_tj],
// and its gradient, dy[position_tj] = w_tj dout_t, dw_tj = <dout_t, y[position_tj]>.
// Sums are in fp32, j ascending.  A position outside 0 .. rows-1 (a slot
// without an expert) adds nothing, and its weight's gradient is zero.
//
// Rows whose bytes are a multiple of 16 move in 16-byte pieces, others by
// element.
#include "mxg_internal.h"
#include "mxg_rows.h"

namespace mxg {
namespace {

constexpr int kCThreads = 256;

// 8 columns n .. n+7 of a row, fp32; `vec`: whole 16-byte pieces
template <int TYPE>
__device__ __forceinline__ void load8(const void* base, int64_t row, int64_t N, int64_t n, bool vec, float (&f)[8]) {
  using E = RowElem<TYPE>;
  const auto* p = reinterpret_cast<const typename E::type*>(base) + row * N + n;
  if (vec) {
#pragma unroll
    for (int h = 0; h < 8 / E::VEC; h++) {
      float x[E::VEC];
      unpack16<TYPE>(*reinterpret_cast<const v4i*>(p + h * E::VEC), x);
#pragma unroll
      for (int i = 0; i < E::VEC; i++) f[h * E::VEC + i] = x[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = n + i < N ? E::get(p[i]) : 0.0f;
  }
}
template <int TYPE>
__device__ __forceinline__ void save8(void* base, int64_t row, int64_t N, int64_t n, bool vec, const float (&f)[8]) {
  using E = RowElem<TYPE>;
  auto* p = reinterpret_cast<typename E::type*>(base) + row * N + n;
  if (vec) {
#pragma unroll
    for (int h = 0; h < 8 / E::VEC; h++) {
      float x[E::VEC];
#pragma unroll
      for (int i = 0; i < E::VEC; i++) x[i] = f[h * E::VEC + i];
      *reinterpret_cast<v4i*>(p + h * E::VEC) = pack16<TYPE>(x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (n + i < N) p[i] = E::put(f[i]);
  }
}

template <int Y, int O>
__global__ __launch_bounds__(kCThreads) void combine_kernel(CombineArgs a) {
  const bool vec = (a.N & 7) == 0;
  const int64_t nq = (a.N + 7) >> 3;
  const int64_t total = a.T * nq;
  for (int64_t u = (int64_t)blockIdx.x * kCThreads + threadIdx.x; u < total; u += (int64_t)gridDim.x * kCThreads) {
    const int64_t t = u / nq, n = (u - t * nq) << 3;
    float s[8] = {};
    for (int j = 0; j < a.k; j++) {
      const int p = a.position[t * a.k + j];
      if (p < 0 || p >= a.rows) continue;
      const float w = a.weights[t * a.k + j];
      float y[8];
      load8<Y>(a.Y, p, a.N, n, vec, y);
#pragma unroll
      for (int i = 0; i < 8; i++) s[i] = fmaf(w, y[i], s[i]);
    }
    save8<O>(a.out, t, a.N, n, vec, s);
  }
}

// one wave per slot
template <int Y, int O>
__global__ __launch_bounds__(kCThreads) void combine_backward_kernel(CombineArgs a, void* __restrict__ dY,
                                                                     float* __restrict__ dW) {
  const int lane = threadIdx.x & 63;
  const int64_t slot = (int64_t)blockIdx.x * (kCThreads / 64) + (threadIdx.x >> 6);
  if (slot >= a.T * a.k) return;
  const int64_t t = slot / a.k;
  const int p = a.position[slot];
  const bool live = p >= 0 && p < a.rows;
  const float w = live ? a.weights[slot] : 0.0f;
  const bool vec = (a.N & 7) == 0;
  float dot = 0.0f;
  if (live)
    for (int64_t n = lane * 8; n < a.N; n += 512) {
      float d[8], y[8];
      load8<O>(a.out, t, a.N, n, vec, d);
      load8<Y>(a.Y, p, a.N, n, vec, y);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        dot = fmaf(d[i], y[i], dot);
        d[i] *= w;
      }
      save8<Y>(dY, p, a.N, n, vec, d);
    }
  dot = wave_sum(dot);
  if (lane == 0) dW[slot] = dot;
}

template <int Y, int O>
hipError_t combine_launch(const CombineArgs& a, void* dY, float* dW, hipStream_t stream) {
  if (dW != nullptr) {
    const int64_t grid = (a.T * a.k + kCThreads / 64 - 1) / (kCThreads / 64);
    hipLaunchKernelGGL((combine_backward_kernel<Y, O>), dim3((unsigned)grid), dim3(kCThreads), 0, stream, a, dY, dW);
  } else {
    int64_t grid = (a.T * ((a.N + 7) >> 3) + kCThreads - 1) / kCThreads;
    if (grid > 256 * 64) grid = 256 * 64;
    hipLaunchKernelGGL((combine_kernel<Y, O>), dim3((unsigned)grid), dim3(kCThreads), 0, stream, a);
  }
  return hipGetLastError();
}

template <int Y>
hipError_t combine_out(const CombineArgs& a, int out_type, void* dY, float* dW, hipStream_t stream) {
  switch (out_type) {
    case kOutF32:
      return combine_launch<Y, kOutF32>(a, dY, dW, stream);
    case kOutBF16:
      return combine_launch<Y, kOutBF16>(a, dY, dW, stream);
    default:
      return combine_launch<Y, kOutF16>(a, dY, dW, stream);
  }
}

hipError_t combine_type(const CombineArgs& a, int y_type, int out_type, void* dY, float* dW, hipStream_t stream) {
  switch (y_type) {
    case kOutF32:
      return combine_out<kOutF32>(a, out_type, dY, dW, stream);
    case kOutBF16:
      return combine_out<kOutBF16>(a, out_type, dY, dW, stream);
    default:
      return combine_out<kOutF16>(a, out_type, dY, dW, stream);
  }
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, int y_type, int out_type, hipStream_t stream) {
  return combine_type(a, y_type, out_type, nullptr, nullptr, stream);
}

hipError_t launch_combine_backward(const CombineArgs& a, int y_type, int out_type, void* dY, float* dW,
                                   hipStream_t stream) {
  return combine_type(a, y_type, out_type, dY, dW, stream);
}

}  // namespace mxg
