// expert_combine.hip - the experts' outputs weighted and summed per token,
//   out_t = sum_j w_tj y[position_tj],
// and its gradient, dy[position_tj] = w_tj dout_t, dw_tj = <dout_t, y[position_tj]>.
// Sums are in fp32, j ascending.  A position outside 0 .. rows-1 (a slot
// without an expert) adds nothing, and its weight's gradient is zero.
//
// Both are bound by the rows' bytes.  A lane takes 8 columns; rows of any length
// start at any element's address (global memory takes such vectors in one
// instruction), and only a row's last columns go by element.
#include "mxg_internal.h"
#include "mxg_rows.h"

namespace mxg {
namespace {

constexpr int kCThreads = 256;
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));

// 8 columns n .. n+7 of a row, fp32; zeros past its end.  NT: rows that are not
// read again leave no trace in the caches.
template <int TYPE, bool NT>
__device__ __forceinline__ void load8(const void* base, int64_t row, int64_t N, int64_t n, float (&f)[8]) {
  using E = RowElem<TYPE>;
  const auto* p = reinterpret_cast<const typename E::type*>(base) + row * N + n;
  if (n + 7 < N) {
#pragma unroll
    for (int h = 0; h < 8 / E::VEC; h++) {
      float x[E::VEC];
      const v4i w = NT ? __builtin_nontemporal_load(reinterpret_cast<const v4i_any*>(p + h * E::VEC))
                       : *reinterpret_cast<const v4i_any*>(p + h * E::VEC);
      unpack16<TYPE>(w, x);
#pragma unroll
      for (int i = 0; i < E::VEC; i++) f[h * E::VEC + i] = x[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = n + i < N ? E::get(p[i]) : 0.0f;
  }
}
template <int TYPE, bool NT>
__device__ __forceinline__ void save8(void* base, int64_t row, int64_t N, int64_t n, const float (&f)[8]) {
  using E = RowElem<TYPE>;
  auto* p = reinterpret_cast<typename E::type*>(base) + row * N + n;
  if (n + 7 < N) {
#pragma unroll
    for (int h = 0; h < 8 / E::VEC; h++) {
      float x[E::VEC];
#pragma unroll
      for (int i = 0; i < E::VEC; i++) x[i] = f[h * E::VEC + i];
      if (NT)
        __builtin_nontemporal_store((v4i_any)pack16<TYPE>(x), reinterpret_cast<v4i_any*>(p + h * E::VEC));
      else
        *reinterpret_cast<v4i_any*>(p + h * E::VEC) = pack16<TYPE>(x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (n + i < N) p[i] = E::put(f[i]);
  }
}

// A workgroup per token and 2048 columns: the positions and weights are the
// same for all its lanes, and the rows of 4 choices are loaded at a time.  8192
// tokens of 4 choices and 4096 columns (bf16): 58 us, 5.8 TB/s; 66 with rows
// that stay in the caches, 69 with a choice at a time.
// L = 16: for rows of at most 128 columns, 16 tokens in a workgroup.
template <int Y, int O, int L>
__global__ __launch_bounds__(kCThreads) void combine_kernel(CombineArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (kCThreads / L) + (L < kCThreads ? threadIdx.x / L : 0);
  const int64_t n = ((int64_t)blockIdx.y * L + threadIdx.x % L) * 8;
  if (t >= a.T || n >= a.N) return;
  const int32_t* pos = a.position + t * a.k;
  const float* wt = a.weights + t * a.k;
  float s[8] = {};
  for (int j = 0; j < a.k; j += 4) {
    float y[4][8];
    bool there[4];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int p = j + u < a.k ? pos[j + u] : -1;
      there[u] = p >= 0 && p < a.rows;
      if (there[u]) load8<Y, true>(a.Y, p, a.N, n, y[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; u++)
      if (there[u]) {
        const float w = wt[j + u];
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] = fmaf(w, y[u][i], s[i]);
      }
  }
  save8<O, true>(a.out, t, a.N, n, s);
}

// L lanes per slot, two pieces of a row at a time.  2047 tokens of 8 choices
// and 4096 columns (bf16), a wave for each slot: 64 us from memory, 4.5 TB/s of
// reads and writes in equal parts, of which a large copy reaches 5.0.  A
// workgroup per token, which reads the token's gradient once for all its
// choices, takes 69 us there and twice as long for few tokens; the gradient
// comes from the L2 for the second choice on anyway.
// dY may be Y: a lane reads its columns of a row before it writes them, and no
// other slot reads that row (dY is not __restrict__, which would let a store go
// ahead of the load).
template <int Y, int O, int L, bool NT>
__global__ __launch_bounds__(kCThreads) void combine_backward_kernel(CombineArgs a, void* dY,
                                                                     float* __restrict__ dW) {
  __shared__ float part[kCThreads / 64];
  const int lane = threadIdx.x % L;
  const int64_t group = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t slot = group * (kCThreads / L) + threadIdx.x / L;
  if (slot >= a.T * a.k) return;
  const int64_t t = slot / a.k;
  const int p = a.position[slot];
  const bool live = p >= 0 && p < a.rows;
  const float w = live ? a.weights[slot] : 0.0f;
  constexpr int STEP = 8 * L;
  float dot = 0.0f;
  if (live)
    for (int64_t n = lane * 8; n < a.N; n += 2 * STEP) {
      float d[2][8], y[2][8];
#pragma unroll
      for (int u = 0; u < 2; u++)
        if (n + STEP * u < a.N) {
          load8<Y, true>(a.Y, p, a.N, n + STEP * u, y[u]);
          load8<O, false>(a.out, t, a.N, n + STEP * u, d[u]);
        }
#pragma unroll
      for (int u = 0; u < 2; u++)
        if (n + STEP * u < a.N) {
#pragma unroll
          for (int i = 0; i < 8; i++) {
            dot = fmaf(d[u][i], y[u][i], dot);
            d[u][i] *= w;
          }
          save8<Y, NT>(dY, p, a.N, n + STEP * u, d[u]);
        }
    }
#pragma unroll
  for (int d = (L < 64 ? L : 64) / 2; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
  if constexpr (L > 64) {
    if ((lane & 63) == 0) part[lane >> 6] = dot;
    __syncthreads();
    dot = (part[0] + part[1]) + (part[2] + part[3]);
  }
  if (lane == 0) dW[slot] = dot;
}

template <int Y, int O, int L, bool NT>
void backward_launch(const CombineArgs& a, void* dY, float* dW, hipStream_t stream) {
  // in two dimensions: a launch has less than 2^32 threads in one
  const int64_t groups = (a.T * a.k + kCThreads / L - 1) / (kCThreads / L), most = 1 << 20;
  const dim3 grid((unsigned)(groups < most ? groups : most), (unsigned)((groups + most - 1) / most));
  hipLaunchKernelGGL((combine_backward_kernel<Y, O, L, NT>), grid, dim3(kCThreads), 0, stream, a, dY, dW);
}

template <int Y, int O, int L>
void combine_tokens(const CombineArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kCThreads / L - 1) / (kCThreads / L)), (unsigned)((a.N + L * 8 - 1) / (L * 8)));
  hipLaunchKernelGGL((combine_kernel<Y, O, L>), grid, dim3(kCThreads), 0, stream, a);
}

template <int Y, int O>
hipError_t combine_launch(const CombineArgs& a, void* dY, float* dW, hipStream_t stream) {
  if (dW != nullptr) {
    // Short rows: 16 lanes for each (20000 tokens of 2 and 100 columns: 11.8 us
    // instead of 25.9).  Few slots of long rows: four waves for each (64 tokens
    // of 8 and 7168 columns: 8.0 us instead of 13.8, 256 of 8: 16.8 and 20.7, but
    // 512 of 8: 29.6 and 27.9).  More than the last cache holds: rows that pass
    // it by (4096 tokens of 8 and 7168 columns: 191 us instead of 206, 8192 of 4
    // and 4096: 126 and 129; but 512 of 8 and 4096: 18.5 and 17.7, and what reads
    // the gradient next would miss it).
    const int64_t slots = a.T * a.k;
    if (a.N <= 16 * 8)
      backward_launch<Y, O, 16, false>(a, dY, dW, stream);
    else if (slots <= 2048 && a.N > 64 * 8)
      backward_launch<Y, O, 256, false>(a, dY, dW, stream);
    else if (slots * a.N * (int64_t)sizeof(typename RowElem<Y>::type) >= ((int64_t)256 << 20))
      backward_launch<Y, O, 64, true>(a, dY, dW, stream);
    else
      backward_launch<Y, O, 64, false>(a, dY, dW, stream);
  } else {
    // Short rows share a workgroup (20000 tokens of 2 and 100 columns: 7.6 us,
    // 22.5 with a workgroup each; with 64 lanes for up to 512 columns nothing
    // was gained).
    if (a.N <= 16 * 8)
      combine_tokens<Y, O, 16>(a, stream);
    else
      combine_tokens<Y, O, 256>(a, stream);
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
