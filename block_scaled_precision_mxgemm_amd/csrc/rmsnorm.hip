// rmsnorm.hip - root-mean-square norm of rows, with the addition of a residual
// before it and an output in 8-bit codes with scales, and its gradients.
//
//   h = x + r, rounded to the rows' type (what the backward pass is given is
//       what was normed);
//   rstd = 1 / sqrt(sum_k h_k^2 / K + eps);   y_k = h_k rstd w_k, rounded to fp32;
//   codes of y: int8 with a scale per row, E4M3 with one per 128 columns, or
//   E4M3 with a UE8M0 scale per 32 (the rules of the three quantizers, applied
//   to the fp32 values: y is not rounded to 16 bits in between).
//
// One pass over memory, which is what bounds it: a row is held in registers between
// its sum and its codes (8192 x 8192 of bf16 with a residual to MXFP8 codes: 470 MB,
// 92.5 us, 5.1 TB/s).  The squares are summed in 64 bits (those of 16-bit values exactly, and
// whatever the lanes' share, the same rstd), the gradients' sums in fp32: a lane's
// own, then over the lanes, then over the waves of a row.
#include "mxg_codes.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

template <class F>
__device__ __forceinline__ F wave_sum(F x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// Sum / largest over the L lanes of a row (all lanes of the workgroup that
// belong to it call these); `part` is 16 elements of LDS.
template <int L, class F>
__device__ __forceinline__ F row_sum(F x, F* part) {
  x = wave_sum(x);
  if constexpr (L > 64) {
    __syncthreads();  // what `part` held has been read
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < L / 64; w++) x += part[w];
  }
  return x;
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t x, double* sums) {
  uint32_t* const part = reinterpret_cast<uint32_t*>(sums);
  x = lanes_max<64>(x);
  if constexpr (L > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < L / 64; w++) x = max(x, part[w]);
  }
  return x;
}

// Weights k .. k + N - 1 in fp32.
template <int N>
__device__ __forceinline__ void load_weights(const void* W, int type, int k, float (&w)[N]) {
  if (type == kOutF32) {
#pragma unroll
    for (int i = 0; i < N / 4; i++) {
      const v4f v = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(W) + k + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; j++) w[4 * i + j] = v[j];
    }
    return;
  }
  const uint16_t* p = reinterpret_cast<const uint16_t*>(W) + k;
  uint32_t v[N / 2];
  if constexpr (N == 8) {
    const v4i u = *reinterpret_cast<const v4i*>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = (uint32_t)u[i];
  } else {
    const v2i u = *reinterpret_cast<const v2i*>(p);
    v[0] = (uint32_t)u[0];
    v[1] = (uint32_t)u[1];
  }
#pragma unroll
  for (int i = 0; i < N / 2; i++) {
    const uint16_t lo = (uint16_t)(v[i] & 0xffffu), hi = (uint16_t)(v[i] >> 16);
    w[2 * i] = type == kOutBF16 ? RowElem<kOutBF16>::get(lo) : RowElem<kOutF16>::get(lo);
    w[2 * i + 1] = type == kOutBF16 ? RowElem<kOutBF16>::get(hi) : RowElem<kOutF16>::get(hi);
  }
}

constexpr int norm_threads(int L) { return L > 256 ? L : 256; }

// Row of this thread; -1: none.
template <int L>
__device__ __forceinline__ int64_t norm_row(int64_t rows) {
  const int64_t group = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = group * (norm_threads(L) / L) + threadIdx.x / L;
  return row < rows ? row : -1;
}

// L lanes per row.  HELD > 0: its 16-byte pieces, at most HELD of them a lane,
// stay in registers; HELD = 0: longer rows are read twice (three times for
// int8), after the first time from the caches.
template <int IN, int HELD, int L>
__global__ __launch_bounds__(norm_threads(L)) void rmsnorm_kernel(NormArgs a) {
  constexpr int VEC = RowElem<IN>::VEC;
  using T = typename RowElem<IN>::type;
  __shared__ double part[16];
  const int64_t row = norm_row<L>(a.rows);
  if (row < 0) return;
  const int tid = threadIdx.x % L;
  const int nv = a.K / VEC;
  const int64_t base = row * a.K;
  const v4i* x = reinterpret_cast<const v4i*>((const T*)a.X + base);
  const v4i* res = reinterpret_cast<const v4i*>((const T*)a.R + base);
  v4i* h = reinterpret_cast<v4i*>((T*)a.H + base);
  const v4i zero = {0, 0, 0, 0};
  const int steps = HELD > 0 ? HELD : (nv + L - 1) / L;

  // the rounded sum's piece i, with the sum of its squares
  double sum = 0.0;
  auto add = [&](int i, v4i w) {
    float f[VEC];
    unpack16<IN>(w, f);
    if (a.R != nullptr) {
      float g[VEC];
      unpack16<IN>(res[i], g);
#pragma unroll
      for (int j = 0; j < VEC; j++) f[j] += g[j];
      w = pack16<IN>(f);
      h[i] = w;
      unpack16<IN>(w, f);
    }
#pragma unroll
    for (int j = 0; j < VEC; j++) sum = fma((double)f[j], (double)f[j], sum);
    return w;
  };
  v4i held[HELD > 0 ? HELD : 1];
  if constexpr (HELD > 0) {
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      const int i = tid + u * L;
      held[u] = i < nv ? x[i] : zero;
    }
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      const int i = tid + u * L;
      if (i < nv) held[u] = add(i, held[u]);
    }
  } else {
    for (int i = tid; i < nv; i += L) add(i, x[i]);
  }
  // An error of rstd is the whole row's: in 64 bits, and y takes it and the rest of it, so
  // that all of h rstd w is rounded once.  At 8192 x 8192 in MXFP8 codes 19 of 67 million
  // are not those of the real y, which is what fp32 values leave; with sums in fp32 and
  // y = (h rstd) w 46.  8192 x 4096 takes 41.6 us instead of 39.1, 8192 x 8192 92.5
  // instead of 91.9.
  const double exact = 1.0 / sqrt(row_sum<L>(sum, part) / a.K + (double)a.eps);
  if (a.rstd != nullptr && tid == 0) a.rstd[row] = (float)exact;
  // Where that is no fp32 value or one of few bits (eps = 0 and rows below 2^-127, rows above
  // 2^126), h is multiplied by its power of two first, exactly.
  const int shift = __builtin_amdgcn_readfirstlane(exact >= 0x1p-100 && exact <= 0x1p100 ? 0 : __builtin_amdgcn_frexp_exp(exact));
  const double scaled = ldexp(exact, -shift);
  const float rstd = (float)scaled, rest = (float)(scaled - (double)rstd);

  // y of step u (zeros past the row's end)
  const v4i* from = a.R != nullptr ? h : x;
  auto value = [&](int u, float (&y)[VEC]) {
    const int i = tid + u * L;
    if (i < nv) {
      float w[VEC];
      if constexpr (HELD > 0)
        unpack16<IN>(held[u], y);
      else
        unpack16<IN>(from[i], y);
      load_weights<VEC>(a.W, a.w_type, i * VEC, w);
      if (shift != 0) {
#pragma unroll
        for (int j = 0; j < VEC; j++) y[j] = ldexpf(y[j], shift);
      }
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float p = y[j] * rstd;
        const float low = fmaf(y[j], rest, fmaf(y[j], rstd, -p));  // h rstd - p
        y[j] = fmaf(p, w[j], low * w[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j++) y[j] = 0.0f;
    }
    return i;
  };
  float s = 0.0f, inv = 0.0f;
  if (a.quant == kQuantInt8) {
    uint32_t most = 0;
#pragma unroll
    for (int u = 0; u < steps; u++) {
      float y[VEC];
      value(u, y);
      most = max(most, magnitude_bits<VEC>(y));
    }
    most = row_max<L>(most, part);
    if (most >= 0x7f800000u) {
      s = __builtin_nanf("");
    } else if (most > 0u) {
      s = fmaxf(__uint_as_float(most) / 127.0f, 0x1p-126f);
      inv = 1.0f / s;
    }
    if (tid == 0) reinterpret_cast<float*>(a.S)[row] = s;
  }
  const int KB = (a.K + kBlock - 1) / kBlock;
  uint8_t* q = a.Q + base;
#pragma unroll
  for (int u = 0; u < steps; u++) {
    float y[VEC];
    const int i = value(u, y);
    const bool valid = i < nv;
    if (a.Y != nullptr && valid) reinterpret_cast<v4i*>((T*)a.Y + base)[i] = pack16<IN>(y);
    uint32_t c[VEC / 4];
    if (a.quant == kQuantInt8) {
      if (inv > 0.0f) {
        int8_codes<VEC>(y, s, inv, 0.5f * s, c);
      } else {
#pragma unroll
        for (int j = 0; j < VEC / 4; j++) c[j] = 0;
      }
    } else if (a.quant == kQuantMx) {
      constexpr int LB = 32 / VEC;
      const uint32_t amax = lanes_max<LB>(magnitude_bits<VEC>(y));
      const bool bad = amax >= 0x7f800000u;
      const int exponent = amax == 0u ? -127 : min(max(__builtin_amdgcn_frexp_expf(__uint_as_float(amax)) - 9, -127), 127);
#pragma unroll
      for (int j = 0; j < VEC; j++) y[j] = ldexpf(y[j], -exponent);
      e4m3_codes<VEC>(y, !bad, c);
      if (valid && i % LB == 0)
        reinterpret_cast<uint8_t*>(a.S)[row * (a.K / 32) + i / LB] = bad ? (uint8_t)255 : (uint8_t)(exponent + 127);
    } else if (a.quant != kQuantNone) {
      constexpr int LB = kBlock / VEC;
      const float sb = block_scale(lanes_max<LB>(magnitude_bits<VEC>(y)), a.quant == kQuantFp8Pow2);
      e4m3_block_codes<VEC>(y, sb, block_inverse(sb), c);
      if (valid && i % LB == 0) reinterpret_cast<float*>(a.S)[row * KB + i / LB] = sb;
    }
    if (a.quant != kQuantNone && valid) store_codes<VEC>(q + (int64_t)i * VEC, c);
  }
}

template <int IN, int HELD, int L>
void norm_rows(const NormArgs& a, hipStream_t stream) {
  constexpr int threads = norm_threads(L), per = threads / L;
  // in two dimensions: a launch has less than 2^32 threads in one
  const int64_t groups = (a.rows + per - 1) / per, most = 1 << 20;
  const dim3 grid((unsigned)(groups < most ? groups : most), (unsigned)((groups + most - 1) / most));
  hipLaunchKernelGGL((rmsnorm_kernel<IN, HELD, L>), grid, dim3(threads), 0, stream, a);
}

template <int IN>
void norm_in(const NormArgs& a, hipStream_t stream) {
  const int64_t pieces = a.K / RowElem<IN>::VEC;
  if (pieces <= 64)
    norm_rows<IN, 1, 64>(a, stream);
  else if (pieces <= 2 * 64)
    norm_rows<IN, 2, 64>(a, stream);
  else if (pieces <= 2 * 256)
    norm_rows<IN, 2, 256>(a, stream);
  else if (pieces <= 4 * 256)
    norm_rows<IN, 4, 256>(a, stream);
  else if (pieces <= 4 * 512)  // 8192 x 14336 of bf16 171 us; 1024 lanes 230, 2 pieces each 180
    norm_rows<IN, 4, 512>(a, stream);
  else if (pieces <= 4 * 1024)
    norm_rows<IN, 4, 1024>(a, stream);
  else
    norm_rows<IN, 0, 1024>(a, stream);
}

// ---- gradients ----------------------------------------------------------------
//
//   hat = h rstd, g = dy w:   dx = rstd (g - hat sum_k(g hat) / K) + dh,
//   dw = sum over rows of dy hat.
template <int IN, int HELD, int L>
__global__ __launch_bounds__(norm_threads(L)) void rmsnorm_backward_kernel(NormGradArgs a) {
  constexpr int VEC = RowElem<IN>::VEC;
  using T = typename RowElem<IN>::type;
  __shared__ float part[16];
  const int64_t row = norm_row<L>(a.rows);
  if (row < 0) return;
  const int tid = threadIdx.x % L;
  const int nv = a.K / VEC;
  const int64_t base = row * a.K;
  const v4i* dy = reinterpret_cast<const v4i*>((const T*)a.dY + base);
  const v4i* h = reinterpret_cast<const v4i*>((const T*)a.H + base);
  const v4i* dh = reinterpret_cast<const v4i*>((const T*)a.dH + base);
  v4i* dx = reinterpret_cast<v4i*>((T*)a.dX + base);
  const v4i zero = {0, 0, 0, 0};
  const float rstd = a.rstd[row];
  v4i hy[HELD > 0 ? HELD : 1], hh[HELD > 0 ? HELD : 1];
  float sum = 0.0f;
  auto dot = [&](int i, const v4i& y, const v4i& x) {
    float f[VEC], g[VEC], w[VEC];
    unpack16<IN>(y, g);
    unpack16<IN>(x, f);
    load_weights<VEC>(a.W, a.w_type, i * VEC, w);
#pragma unroll
    for (int j = 0; j < VEC; j++) sum = fmaf(g[j] * w[j], f[j] * rstd, sum);
  };
  if constexpr (HELD > 0) {
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      const int i = tid + u * L;
      hy[u] = i < nv ? dy[i] : zero;
      hh[u] = i < nv ? h[i] : zero;
    }
#pragma unroll
    for (int u = 0; u < HELD; u++)
      if (tid + u * L < nv) dot(tid + u * L, hy[u], hh[u]);
  } else {
    for (int i = tid; i < nv; i += L) dot(i, dy[i], h[i]);
  }
  const float c = row_sum<L>(sum, part) / (float)a.K;
  auto put = [&](int i, const v4i& y, const v4i& x) {
    float f[VEC], g[VEC], w[VEC];
    unpack16<IN>(y, g);
    unpack16<IN>(x, f);
    load_weights<VEC>(a.W, a.w_type, i * VEC, w);
#pragma unroll
    for (int j = 0; j < VEC; j++) f[j] = rstd * (g[j] * w[j] - f[j] * rstd * c);
    if (a.dH != nullptr) {
      unpack16<IN>(dh[i], g);
#pragma unroll
      for (int j = 0; j < VEC; j++) f[j] += g[j];
    }
    dx[i] = pack16<IN>(f);
  };
  if constexpr (HELD > 0) {
#pragma unroll
    for (int u = 0; u < HELD; u++)
      if (tid + u * L < nv) put(tid + u * L, hy[u], hh[u]);
  } else {
    for (int i = tid; i < nv; i += L) put(i, dy[i], h[i]);
  }
}

// Sums of dy hat over strips of rows, then over the strips: no atomics, so that
// every run gives the same bits.
template <int IN>
__global__ __launch_bounds__(256) void rmsnorm_dweight_kernel(NormGradArgs a, int64_t strip, float* part) {
  constexpr int VEC = RowElem<IN>::VEC;
  using T = typename RowElem<IN>::type;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.K / VEC) return;
  const int64_t r0 = blockIdx.y * strip, r1 = min(r0 + strip, a.rows);
  float acc[VEC] = {};
  for (int64_t r = r0; r < r1; r++) {
    float f[VEC], g[VEC];
    unpack16<IN>(reinterpret_cast<const v4i*>((const T*)a.dY + r * a.K)[i], g);
    unpack16<IN>(reinterpret_cast<const v4i*>((const T*)a.H + r * a.K)[i], f);
    const float rstd = a.rstd[r];
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] = fmaf(g[j], f[j] * rstd, acc[j]);
  }
  float* p = part + (int64_t)blockIdx.y * a.K + i * VEC;
#pragma unroll
  for (int j = 0; j < VEC / 4; j++)
    *reinterpret_cast<v4f*>(p + 4 * j) = v4f{acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]};
}

// 32 columns a workgroup: 8 lanes of 4 columns, 8 WAVES of them at a time over the
// strips; 16 waves above 64 strips, else 2 (the whole backward pass of
// 8191 x 4096 53.3 us, 59.4 with 4 waves on 64 columns; of 1 x 131072 26.9 with 2 waves,
// 37.1 with 16).
template <int WAVES>
__global__ __launch_bounds__(WAVES * 64) void rmsnorm_dweight_sum_kernel(const float* part, int strips, int K, float* dW) {
  __shared__ __attribute__((aligned(16))) v4f sums[WAVES][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = blockIdx.x * 32 + (lane & 7) * 4;
  v4f s = {0, 0, 0, 0};
  if (k < K) {
#pragma unroll 4
    for (int i = threadIdx.x >> 3; i < strips; i += WAVES * 8) s += *reinterpret_cast<const v4f*>(part + (int64_t)i * K + k);
  }
#pragma unroll
  for (int d = 8; d < 64; d <<= 1) {
#pragma unroll
    for (int x = 0; x < 4; x++) s[x] += __shfl_xor(s[x], d);
  }
  if (lane < 8) sums[wave][lane] = s;
  __syncthreads();
  if (threadIdx.x < 8 && k < K) {
    s = sums[0][lane];
#pragma unroll
    for (int i = 1; i < WAVES; i++) s += sums[i][lane];
    *reinterpret_cast<v4f*>(dW + k) = s;
  }
}

// Both gradients in one pass over dY and H (8191 x 4096 of bf16 with dH: 268 MB, 53 us,
// of which this kernel takes 46, 5.8 TB/s; a pass each took 136): a workgroup takes every G-th row (or
// group of rows, where L lanes are less than a workgroup), holds a row's pieces and
// the sums of its columns in registers, and has the next row on its way meanwhile.
// The sums go to `part`, one row of them for each workgroup.
template <int IN, int HELD, int L>
__global__ __launch_bounds__(norm_threads(L)) void rmsnorm_backward_fused_kernel(NormGradArgs a, float* sums) {
  constexpr int VEC = RowElem<IN>::VEC, PER = norm_threads(L) / L;
  using T = typename RowElem<IN>::type;
  __shared__ float part[16];
  __shared__ __attribute__((aligned(16))) float join[PER > 1 ? (PER - 1) * HELD * L * VEC : 1];
  const int tid = threadIdx.x % L, sub = threadIdx.x / L;
  const int nv = a.K / VEC;
  const v4i zero = {0, 0, 0, 0};
  float acc[HELD][VEC] = {}, w[HELD][VEC];
#pragma unroll
  for (int u = 0; u < HELD; u++) {
    const int i = tid + u * L;
#pragma unroll
    for (int j = 0; j < VEC; j++) w[u][j] = 0.0f;
    if (i < nv) load_weights<VEC>(a.W, a.w_type, i * VEC, w[u]);
  }
  v4i y[HELD], h[HELD];
  float rstd = 0.0f;
  auto load = [&](int64_t row) {
    const bool live = row < a.rows;
    rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      const int i = tid + u * L;
      const bool some = live && i < nv;
      y[u] = some ? __builtin_nontemporal_load(reinterpret_cast<const v4i*>((const T*)a.dY + row * a.K) + i) : zero;
      h[u] = some ? __builtin_nontemporal_load(reinterpret_cast<const v4i*>((const T*)a.H + row * a.K) + i) : zero;
    }
  };
  // rows of all of a workgroup's parts together, so that its barriers are passed by all
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t row = (int64_t)blockIdx.x * PER + sub;
  load(row);
  for (int64_t base = (int64_t)blockIdx.x * PER; base < a.rows; base += step, row += step) {
    v4i ny[HELD], nh[HELD], dh[HELD];
    const float r = rstd;
    const bool live = row < a.rows;
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      ny[u] = y[u];
      nh[u] = h[u];
      const int i = tid + u * L;
      dh[u] = zero;
      if (a.dH != nullptr && live && i < nv)
        dh[u] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>((const T*)a.dH + row * a.K) + i);
    }
    load(row + step);
    float dot = 0.0f;
#pragma unroll
    for (int u = 0; u < HELD; u++) {
      float f[VEC], g[VEC];
      unpack16<IN>(ny[u], g);
      unpack16<IN>(nh[u], f);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float hat = f[j] * r;
        acc[u][j] = fmaf(g[j], hat, acc[u][j]);
        dot = fmaf(g[j] * w[u][j], hat, dot);
      }
    }
    const float c = row_sum<L>(dot, part) / (float)a.K;
    if (live) {
      v4i* dx = reinterpret_cast<v4i*>((T*)a.dX + row * a.K);
#pragma unroll
      for (int u = 0; u < HELD; u++) {
        const int i = tid + u * L;
        if (i >= nv) continue;
        float f[VEC], g[VEC], o[VEC];
        unpack16<IN>(ny[u], g);
        unpack16<IN>(nh[u], f);
        unpack16<IN>(dh[u], o);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          f[j] = r * (g[j] * w[u][j] - f[j] * r * c);
          if (a.dH != nullptr) f[j] += o[j];
        }
        __builtin_nontemporal_store(pack16<IN>(f), dx + i);
      }
    }
  }
  if constexpr (PER > 1) {
    // the workgroup's parts, in their order
    if (sub > 0) {
#pragma unroll
      for (int u = 0; u < HELD; u++)
#pragma unroll
        for (int j = 0; j < VEC; j++) join[((sub - 1) * HELD + u) * L * VEC + j * L + tid] = acc[u][j];
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int p = 0; p < PER - 1; p++)
#pragma unroll
      for (int u = 0; u < HELD; u++)
#pragma unroll
        for (int j = 0; j < VEC; j++) acc[u][j] += join[(p * HELD + u) * L * VEC + j * L + tid];
  }
  float* out = sums + (int64_t)blockIdx.x * a.K;
#pragma unroll
  for (int u = 0; u < HELD; u++) {
    const int i = tid + u * L;
    if (i >= nv) continue;
#pragma unroll
    for (int j = 0; j < VEC / 4; j++)
      *reinterpret_cast<v4f*>(out + i * VEC + 4 * j) = v4f{acc[u][4 * j], acc[u][4 * j + 1], acc[u][4 * j + 2], acc[u][4 * j + 3]};
  }
}

// Few and short rows, where a second launch takes longer than the work: each
// workgroup of 16 waves forms the sums of all rows for itself (they come from the
// caches) and then the gradients of 64 pieces of their columns, a wave a row.
// fp32, one launch against two, in us: replayed in a graph 2 x 4096 3.6 and 5.2, 8 x
// 4096 5.6 and 5.4, 17 x 2048 5.8 and 4.8, 64 x 2048 15.7 and 4.7; called one by one,
// where a launch costs the host 4, 17 x 2064 10.6 and 14.9.
constexpr int kFewRows = 64;
constexpr int64_t kFewElements = 48 * 1024;
template <int IN>
__global__ __launch_bounds__(1024) void rmsnorm_backward_few_kernel(NormGradArgs a) {
  constexpr int VEC = RowElem<IN>::VEC;
  using T = typename RowElem<IN>::type;
  __shared__ float c[kFewRows];  // of each row, or (fewer than 9) of each of its parts
  __shared__ float sums[16][VEC][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nv = a.K / VEC, rows = (int)a.rows;
  const int parts = rows > 8 ? 1 : rows > 4 ? 2 : rows > 2 ? 4 : rows > 1 ? 8 : 16;
  for (int item = wave; item < rows * parts; item += 16) {
    const int row = item / parts;
    const v4i* dy = reinterpret_cast<const v4i*>((const T*)a.dY + (int64_t)row * a.K);
    const v4i* h = reinterpret_cast<const v4i*>((const T*)a.H + (int64_t)row * a.K);
    const float r = a.rstd[row];
    float dot = 0.0f;
#pragma unroll 4
    for (int i = item % parts * 64 + lane; i < nv; i += 64 * parts) {
      float f[VEC], g[VEC], w[VEC];
      unpack16<IN>(dy[i], g);
      unpack16<IN>(h[i], f);
      load_weights<VEC>(a.W, a.w_type, i * VEC, w);
#pragma unroll
      for (int j = 0; j < VEC; j++) dot = fmaf(g[j] * w[j], f[j] * r, dot);
    }
    dot = wave_sum(dot);
    if (lane == 0) c[item] = dot;
  }
  __syncthreads();
  const int i = blockIdx.x * 64 + lane;
  float acc[VEC] = {};
  if (i < nv) {
    float w[VEC];
    load_weights<VEC>(a.W, a.w_type, i * VEC, w);
    for (int row = wave; row < rows; row += 16) {
      const int64_t base = (int64_t)row * a.K;
      float f[VEC], g[VEC], o[VEC];
      unpack16<IN>(reinterpret_cast<const v4i*>((const T*)a.dY + base)[i], g);
      unpack16<IN>(reinterpret_cast<const v4i*>((const T*)a.H + base)[i], f);
      if (a.dH != nullptr) unpack16<IN>(reinterpret_cast<const v4i*>((const T*)a.dH + base)[i], o);
      const float r = a.rstd[row];
      float mean = 0.0f;
      for (int p = 0; p < parts; p++) mean += c[row * parts + p];
      mean /= (float)a.K;
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        acc[j] = fmaf(g[j], f[j] * r, acc[j]);
        f[j] = r * (g[j] * w[j] - f[j] * r * mean);
        if (a.dH != nullptr) f[j] += o[j];
      }
      reinterpret_cast<v4i*>((T*)a.dX + base)[i] = pack16<IN>(f);
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; j++) sums[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave >= VEC || i >= nv) return;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++) s += sums[k][wave][lane];
  a.dW[i * VEC + wave] = s;
}

void sum_strips(const float* part, int strips, const NormGradArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.K + 31) / 32));
  if (strips > 64)
    hipLaunchKernelGGL(rmsnorm_dweight_sum_kernel<16>, grid, dim3(1024), 0, stream, part, strips, a.K, a.dW);
  else
    hipLaunchKernelGGL(rmsnorm_dweight_sum_kernel<2>, grid, dim3(128), 0, stream, part, strips, a.K, a.dW);
}

bool few_rows(int64_t rows, int64_t K) { return rows <= kFewRows && rows * K <= kFewElements; }

// Rows of partial sums: as many as workgroups that have two a CU (their traffic
// is 1 / 16 of the rest at 8192 rows), or strips of the long rows' kernel.
constexpr int kStrips = 512;
int strips_of(int64_t rows) { return (int)(rows < kStrips ? rows : kStrips); }

template <int IN, int HELD, int L>
void backward_fused(const NormGradArgs& a, hipStream_t stream) {
  constexpr int per = norm_threads(L) / L;
  const int64_t groups = (a.rows + per - 1) / per;
  const int grid = strips_of(groups);
  float* part = reinterpret_cast<float*>(a.workspace);
  // one workgroup's sums are the result
  hipLaunchKernelGGL((rmsnorm_backward_fused_kernel<IN, HELD, L>), dim3((unsigned)grid), dim3(norm_threads(L)), 0, stream, a,
                     grid == 1 ? a.dW : part);
  if (grid > 1) sum_strips(part, grid, a, stream);
}

template <int IN>
void backward_in(const NormGradArgs& a, hipStream_t stream) {
  const int64_t pieces = a.K / RowElem<IN>::VEC;
  if (few_rows(a.rows, a.K)) {
    hipLaunchKernelGGL((rmsnorm_backward_few_kernel<IN>), dim3((unsigned)((pieces + 63) / 64)), dim3(1024), 0, stream, a);
    return;
  }
  if (pieces <= 64) return backward_fused<IN, 1, 64>(a, stream);
  if (pieces <= 2 * 64) return backward_fused<IN, 2, 64>(a, stream);
  if (pieces <= 256) return backward_fused<IN, 1, 256>(a, stream);
  if (pieces <= 2 * 256) return backward_fused<IN, 2, 256>(a, stream);
  if (pieces <= 4 * 256) return backward_fused<IN, 4, 256>(a, stream);
  if (pieces <= 2 * 1024) return backward_fused<IN, 2, 1024>(a, stream);
  // longer rows: the sums of the columns in a pass of their own
  const int strips = strips_of(a.rows);
  float* part = reinterpret_cast<float*>(a.workspace);
  const int64_t strip = (a.rows + strips - 1) / strips;
  const int used = (int)((a.rows + strip - 1) / strip);
  hipLaunchKernelGGL((rmsnorm_dweight_kernel<IN>), dim3((unsigned)((pieces + 255) / 256), (unsigned)used), dim3(256), 0,
                     stream, a, strip, part);
  sum_strips(part, used, a, stream);
  const int64_t most = 1 << 20;
  const dim3 grid((unsigned)(a.rows < most ? a.rows : most), (unsigned)((a.rows + most - 1) / most));
  if (pieces <= 4 * 1024)
    hipLaunchKernelGGL((rmsnorm_backward_kernel<IN, 4, 1024>), grid, dim3(1024), 0, stream, a);
  else
    hipLaunchKernelGGL((rmsnorm_backward_kernel<IN, 0, 1024>), grid, dim3(1024), 0, stream, a);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, int type, hipStream_t stream) {
  switch (type) {
    case kOutF32:
      norm_in<kOutF32>(a, stream);
      break;
    case kOutBF16:
      norm_in<kOutBF16>(a, stream);
      break;
    default:
      norm_in<kOutF16>(a, stream);
  }
  return hipGetLastError();
}

int64_t rmsnorm_backward_bytes(int64_t rows, int64_t K) {
  return few_rows(rows, K) ? 0 : (int64_t)strips_of(rows) * K * 4;
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& a, int type, hipStream_t stream) {
  switch (type) {
    case kOutF32:
      backward_in<kOutF32>(a, stream);
      break;
    case kOutBF16:
      backward_in<kOutBF16>(a, stream);
      break;
    default:
      backward_in<kOutF16>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace mxg
