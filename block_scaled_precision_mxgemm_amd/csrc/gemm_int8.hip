// gemm_int8.hip - int8 x int8 products with one scale per token (row of A)
// and per output channel (row of B), dense and by expert:
//   C[i][j] = out(act(sa_i sb_j sum_k a_ik b_jk + bias_j)).
// The sum is exact: it stays in int32 (K < 2^17, so |sum| < 2^31 for any
// codes), and is rounded once, to fp32, before the scales.
//
// By expert, rows offsets[e] .. offsets[e+1] of C take B, its scales and its
// bias of expert e, and row p of C takes row index[p] / index_div of A (row p
// without an index).  The workgroups find their tile from the offsets on the
// device: no host copy of the row counts, and no work but a scan of them.
#include "mxg_int8.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

// 64 x 64 tiles, 4 waves of 32 x 32, slices of 128 k.
constexpr int kBM = 64, kBN = 64, kBK = 128;

__global__ __launch_bounds__(256) void int8_tile_kernel(I8Args a, int tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t sa[kBM * kBK], sb[kBN * kBK];
  __shared__ I8Tile tile;
  __shared__ int64_t arow[kBM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
  if (wave == 0) find_tile(a, kBM, tm, lane, &tile);
  __syncthreads();
  const I8Tile t = tile;
  if (t.rows <= 0) return;
  if (tid < kBM) arow[tid] = tid < t.rows ? a_row(a, t.row0 + tid) : -1;
  __syncthreads();
  const int8_t* B = a.B + (int64_t)t.expert * a.N * a.K;
  const int n0 = tn * kBN;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  v4i acc[2][2] = {};
  for (int k0 = 0; k0 < a.K; k0 += kBK) {
    for (int c = tid; c < kBM * 8; c += 256) {
      const int row = c >> 3, ch = c & 7, k = k0 + ch * 16;
      const int64_t ar = arow[row];
      v4i va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
      if (ar >= 0 && k < a.K) va = *reinterpret_cast<const v4i*>(a.A + ar * a.K + k);
      if (n0 + row < a.N && k < a.K) vb = *reinterpret_cast<const v4i*>(B + (int64_t)(n0 + row) * a.K + k);
      const int o = row * kBK + ((ch ^ swz8(row)) << 4);
      *reinterpret_cast<v4i*>(sa + o) = va;
      *reinterpret_cast<v4i*>(sb + o) = vb;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; h++) {
      v4i fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int ra = wm + 16 * i + r, rb = wn + 16 * i + r;
        fa[i] = *reinterpret_cast<const v4i*>(sa + ra * kBK + (((4 * h + g) ^ swz8(ra)) << 4));
        fb[i] = *reinterpret_cast<const v4i*>(sb + rb * kBK + (((4 * h + g) ^ swz8(rb)) << 4));
      }
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) acc[i][j] = mfma_i8(fb[j], fa[i], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int row = wm + 16 * i + r;
    if (row >= t.rows) continue;
    const float s = a_scale(a, arow[row]);
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int n = n0 + wn + 16 * j + 4 * g;
      if (n < a.N) store4(a, t.expert, t.row0 + row, n, acc[i][j], s);
    }
  }
}

}  // namespace

hipError_t launch_int8(const I8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + kBN - 1) / kBN;
  const int64_t tiles = tiles_n * i8_tiles_m(a, kBM);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(int8_tile_kernel, dim3((unsigned)tiles), dim3(256), 0, stream, a, (int)tiles_n);
  return hipGetLastError();
}

}  // namespace mxg
