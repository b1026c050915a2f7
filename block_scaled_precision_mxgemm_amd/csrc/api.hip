// api.hip - the exported C ABI (declared in include/mxgemm.h): argument
// validation, device check and kernel choice.  No entry point allocates,
// frees or synchronizes; all work is enqueued on the caller's stream.
#include <string.h>

#include "../../include/mxgemm.h"
#include "mxg_fp8.h"
#include "mxg_int8.h"
#include "mxg_internal.h"

namespace {

// gfx950 check, cached per device (the library runs on one kind of GPU).
constexpr int kMaxDevices = 64;
int g_arch_ok[kMaxDevices];  // 0 = unknown, 1 = gfx950, -1 = other

int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MXG_EHIP;
  if (dev < 0 || dev >= kMaxDevices) return MXG_EUNSUPPORTED;
  int v = __atomic_load_n(&g_arch_ok[dev], __ATOMIC_RELAXED);
  if (v == 0) {
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, dev) != hipSuccess) return MXG_EHIP;
    v = (strncmp(p.gcnArchName, "gfx950", 6) == 0) ? 1 : -1;
    __atomic_store_n(&g_arch_ok[dev], v, __ATOMIC_RELAXED);
  }
  return v == 1 ? MXG_OK : MXG_EUNSUPPORTED;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool dim_ok(int64_t d) { return d >= 1 && d <= MXG_MAX_DIM; }

int to_status(hipError_t e) { return e == hipSuccess ? MXG_OK : MXG_EHIP; }

int validate_mx(const void* A, const uint8_t* SA, const void* B, const uint8_t* SB, const void* C, int64_t M,
                int64_t N, int64_t K, int fmt) {
  if (!A || !SA || !B || !SB || !C) return MXG_EINVAL;
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || (K % 32) != 0) return MXG_EINVAL;
  if (fmt < MXG_FMT_FP8_FP8 || fmt > MXG_FMT_FP8_BF6) return MXG_EINVAL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(C)) return MXG_EALIGN;
  return MXG_OK;
}

int validate_epi(const float* bias, int act, int out_type) {
  if (act != MXG_ACT_NONE && act != MXG_ACT_GELU) return MXG_EINVAL;
  if (out_type != MXG_OUT_F32 && out_type != MXG_OUT_BF16 && out_type != MXG_OUT_F16) return MXG_EINVAL;
  if (bias != nullptr && !aligned16(bias)) return MXG_EALIGN;
  return MXG_OK;
}

// integer weights (remapped in registers to MFMA operand codes) and FP6
// weights (MFMA operands as stored): the split-K kernel takes them for every
// M the decode and tiled kernels do not
bool remapped_weights(int fmt) {
  return fmt == MXG_FMT_FP8_INT4 || fmt == MXG_FMT_FP8_INT2 || fmt == MXG_FMT_FP8_FP6 || fmt == MXG_FMT_FP8_BF6;
}

// Kernel choice for an MX product (arguments validated): the weight-streaming
// decode kernel (E4M3 activations against E4M3, E2M1, E2M3, E3M2, INT4 or
// INT2 weights), the split-K skinny kernel (the same), or the tiled /
// ping-pong kernels (every 8- and 4-bit float format pair; integer weights,
// and FP6 weights when K is a multiple of 128, on the tiled kernel).  FP6
// weights with other K and more than 64 rows of activations run the split-K
// kernel once per 64 rows (B is read once per 64 rows: a correct path for
// such shapes, not a tuned one).
int run_mx(const void* A, const uint8_t* SA, const void* B, const uint8_t* SB, const mxg::Epi& e, int64_t M,
           int64_t N, int64_t K, int fmt, hipStream_t st) {
  if (mxg::decode_ok(M, K, fmt, SA, SB, e)) return to_status(mxg::launch_mx_decode(A, SA, B, SB, e, M, N, K, fmt, st));
  // FP6 weights with more rows, K in whole 128-k slices: the tiled kernel
  // (the byte offsets of 128 weight rows stay below 2^31)
  if ((fmt == MXG_FMT_FP8_FP6 || fmt == MXG_FMT_FP8_BF6) && M > mxg::kSkinnyMaxM && K % 128 == 0 && K < (1 << 24))
    return to_status(mxg::launch_mx_tiled(A, SA, B, SB, e, M, N, K, fmt, st));
  // integer weights with more rows: the tiled kernel (any K; in a partial
  // last slice the codes past K are finite and meet zeroed activations)
  if ((fmt == MXG_FMT_FP8_INT4 || fmt == MXG_FMT_FP8_INT2) && M > mxg::kSkinnyMaxM)
    return to_status(mxg::launch_mx_tiled(A, SA, B, SB, e, M, N, K, fmt, st));
  if (remapped_weights(fmt) && M > mxg::kSkinnyMaxM) {
    const int64_t eb = mxg::epi_elem_bytes(e.out);
    for (int64_t m0 = 0; m0 < M; m0 += mxg::kSkinnyMaxM) {
      mxg::Epi ec = e;
      ec.C = (uint8_t*)e.C + m0 * N * eb;
      const int64_t mc = M - m0 < mxg::kSkinnyMaxM ? M - m0 : mxg::kSkinnyMaxM;
      const hipError_t err = mxg::launch_mx_skinny((const uint8_t*)A + m0 * K, SA + m0 * (K / 32), B, SB, ec, mc,
                                                   N, K, fmt, st);
      if (err != hipSuccess) return to_status(err);
    }
    return MXG_OK;
  }
  if (M <= mxg::kSkinnyMaxM &&
      (fmt == MXG_FMT_FP8_FP8 || fmt == MXG_FMT_FP8_FP4 || remapped_weights(fmt))) {
    // K not a multiple of 1024, up to 16 rows, fp32 C: the decode kernel
    // takes the largest multiple of 1024 below K, the split-K kernel adds the
    // rest (with more rows the split-K kernel alone measured faster at
    // N = 4096)
    const int64_t k1 = K - K % 1024;
    const mxg::Epi plain{e.C, nullptr, mxg::kOutF32, mxg::kActNone};
    if (M <= 16 && e.out == mxg::kOutF32 && mxg::decode_ok(M, k1, fmt, SA, SB, plain)) {
      const hipError_t err = mxg::launch_mx_decode(A, SA, B, SB, plain, M, N, K, fmt, st, k1);
      if (err != hipSuccess) return to_status(err);
      return to_status(mxg::launch_mx_skinny(A, SA, B, SB, e, M, N, K, fmt, st, k1));
    }
    return to_status(mxg::launch_mx_skinny(A, SA, B, SB, e, M, N, K, fmt, st));
  }
  return to_status(mxg::launch_mx_tiled(A, SA, B, SB, e, M, N, K, fmt, st));
}

bool type_ok(int t) { return t == MXG_OUT_F32 || t == MXG_OUT_BF16 || t == MXG_OUT_F16; }

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
// start of a row of elements that the kernels may also read one by one
bool aligned_elem(const void* p, int type) { return ((uintptr_t)p & (type == MXG_OUT_F32 ? 3u : 1u)) == 0; }

// int8 products: validated arguments of the dense and the expert form
int run_int8(const mxg::I8Args& a, const float* bias, int act, int out_type, hipStream_t st) {
  if (!a.A || !a.SA || !a.B || !a.SB || !a.e.C) return MXG_EINVAL;
  if (a.N < 1 || a.K < 16 || (a.K % 16) != 0 || a.K > MXG_INT8_MAX_K) return MXG_EINVAL;
  if (!aligned16(a.A) || !aligned16(a.B) || !aligned16(a.e.C) || !aligned16(a.SB)) return MXG_EALIGN;
  if (!aligned4(a.SA) || !aligned4(a.offsets) || !aligned4(a.index)) return MXG_EALIGN;
  int s = validate_epi(bias, act, out_type);
  if (s != MXG_OK) return s;
  s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_int8(a, st));
}

int validate_route(const void* logits, int in_type, int64_t T, int64_t E, int k, int score) {
  if (!logits || !type_ok(in_type) || !dim_ok(T)) return MXG_EINVAL;
  if (E < 1 || E > MXG_MAX_EXPERTS || k < 1 || k > MXG_MAX_CHOICES || k > E) return MXG_EINVAL;
  if (score != MXG_SCORE_SOFTMAX && score != MXG_SCORE_SIGMOID) return MXG_EINVAL;
  return aligned_elem(logits, in_type) ? MXG_OK : MXG_EALIGN;
}

int validate_combine(const mxg::CombineArgs& a, int y_type, int out_type) {
  if (!a.Y || !a.position || !a.weights || !a.out || !type_ok(y_type) || !type_ok(out_type)) return MXG_EINVAL;
  if (!dim_ok(a.N) || !dim_ok(a.T) || a.k < 1 || a.k > MXG_MAX_CHOICES) return MXG_EINVAL;
  if (a.rows < 1 || a.rows > MXG_MAX_SLOTS) return MXG_EINVAL;
  if (!aligned16(a.Y) || !aligned16(a.out) || !aligned4(a.position) || !aligned4(a.weights)) return MXG_EALIGN;
  return MXG_OK;
}

int blocks_of(int64_t d) { return (int)((d + 127) / 128); }

// sizes and operands of the E4M3 products and of their weights' gradients
bool fp8_dims_ok(int64_t N, int64_t K) { return dim_ok(N) && dim_ok(K) && K % 16 == 0; }
bool experts_ok(const int32_t* offsets, const int32_t* index, int index_div, int64_t rows, int64_t rowsA, int64_t E) {
  if (!offsets || rows < 1 || rows > MXG_MAX_SLOTS || rowsA < 1 || rowsA > MXG_MAX_SLOTS) return false;
  return E >= 1 && E <= MXG_MAX_EXPERTS && index_div >= 1 && (index != nullptr || rowsA >= rows);
}

int run_fp8(const mxg::F8Args& a, const float* bias, int act, int out_type, hipStream_t st) {
  if (!a.A || !a.SA || !a.B || !a.SB || !a.e.C) return MXG_EINVAL;
  if (!aligned16(a.A) || !aligned16(a.B) || !aligned16(a.e.C)) return MXG_EALIGN;
  if (!aligned4(a.SA) || !aligned4(a.SB) || !aligned4(a.offsets) || !aligned4(a.index)) return MXG_EALIGN;
  int s = validate_epi(bias, act, out_type);
  if (s != MXG_OK) return s;
  s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_fp8(a, st));
}

int run_fp8_grad(const mxg::F8GradArgs& a, int c_type, hipStream_t st) {
  const bool any_scale = c_type >= 0 && (c_type & MXG_GRAD_ANY_SCALE) != 0;
  if (any_scale) c_type -= MXG_GRAD_ANY_SCALE;
  if (!a.dY || !a.A || !a.SA || !a.dW || !type_ok(c_type) || !type_ok(a.out_type)) return MXG_EINVAL;
  if (mxg::fp8_weight_grad_bytes(a.M, a.N, a.K, a.E) > 0 && !a.workspace) return MXG_EINVAL;
  if (!aligned16(a.dY) || !aligned16(a.A) || !aligned16(a.dW) || !aligned16(a.workspace)) return MXG_EALIGN;
  if (!aligned4(a.SA) || !aligned4(a.offsets) || !aligned4(a.index)) return MXG_EALIGN;
  const int s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_fp8_weight_grad(a, c_type, any_scale, st));
}

bool norm_dims_ok(int64_t rows, int64_t K) {
  return rows >= 1 && rows <= MXG_MAX_SLOTS && dim_ok(K) && K % 16 == 0;
}

static_assert(MXG_QUANT_NONE == mxg::kQuantNone && MXG_QUANT_INT8 == mxg::kQuantInt8 &&
                  MXG_QUANT_FP8 == mxg::kQuantFp8 && MXG_QUANT_FP8_POW2 == mxg::kQuantFp8Pow2 &&
                  MXG_QUANT_MXFP8 == mxg::kQuantMx,
              "code ids of the norm");
static_assert(MXG_OUT_F32 == mxg::kOutF32 && MXG_OUT_BF16 == mxg::kOutBF16 && MXG_OUT_F16 == mxg::kOutF16,
              "output type ids");
static_assert(MXG_SCORE_SOFTMAX == mxg::kScoreSoftmax && MXG_SCORE_SIGMOID == mxg::kScoreSigmoid, "score ids");
static_assert(MXG_ACT_NONE == mxg::kActNone && MXG_ACT_GELU == mxg::kActGelu, "activation ids");
static_assert(MXG_ELEM_E4M3 == mxg::kFmtFp8 && MXG_ELEM_E5M2 == mxg::kFmtBf8 && MXG_ELEM_E2M1 == mxg::kFmtFp4,
              "element ids are the MFMA format ids");
static_assert(MXG_ELEM_INT4 == mxg::kElemInt4 && MXG_ELEM_INT2 == mxg::kElemInt2, "integer element ids");
static_assert(MXG_ELEM_E2M3 == mxg::kFmtFp6 && MXG_ELEM_E3M2 == mxg::kFmtBf6, "FP6 element ids");
static_assert(MXG_FMT_FP8_FP6 == 8 && MXG_FMT_FP8_BF6 == 9, "FP6 pair ids the split-K launch switches on");

}  // namespace

extern "C" {

const char* mxgemm_status_string(int status) {
  switch (status) {
    case MXG_OK:
      return "ok";
    case MXG_EINVAL:
      return "invalid argument (null pointer, dimension out of range, K not a multiple of 32 (int8, fp8 and norm: 16), or unknown format)";
    case MXG_EALIGN:
      return "pointer not aligned (data: 16 bytes; the int8, fp8, norm and expert calls' other arrays: their element)";
    case MXG_EUNSUPPORTED:
      return "device is not gfx950 (MI355X)";
    case MXG_EHIP:
      return "HIP runtime error at launch";
    default:
      return "unknown status";
  }
}

int mxgemm_device_supported(void) {
  const int s = check_device();
  if (s == MXG_OK) return 1;
  if (s == MXG_EUNSUPPORTED) return 0;
  return -s;
}

int mxgemm_quantize(const float* X, int64_t rows, int64_t K, int elem, void* Q, uint8_t* S, void* stream) {
  if (!X || !Q || !S) return MXG_EINVAL;
  if (!dim_ok(rows) || !dim_ok(K) || (K % 32) != 0) return MXG_EINVAL;
  if (elem != MXG_ELEM_E4M3 && elem != MXG_ELEM_E5M2 && elem != MXG_ELEM_E2M1 && elem != MXG_ELEM_INT4 &&
      elem != MXG_ELEM_INT2 && elem != MXG_ELEM_E2M3 && elem != MXG_ELEM_E3M2)
    return MXG_EINVAL;
  if (!aligned16(X) || !aligned16(Q)) return MXG_EALIGN;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(mxg::launch_quantize(X, rows, K, elem, Q, S, (hipStream_t)stream));
}

int mxgemm_run(const void* A, const uint8_t* scaleA, const void* B, const uint8_t* scaleB, float* C, int64_t M,
               int64_t N, int64_t K, int fmt, void* stream) {
  int s = validate_mx(A, scaleA, B, scaleB, C, M, N, K, fmt);
  if (s != MXG_OK) return s;
  s = check_device();
  if (s != MXG_OK) return s;
  return run_mx(A, scaleA, B, scaleB, mxg::Epi{C, nullptr, mxg::kOutF32, mxg::kActNone}, M, N, K, fmt,
                (hipStream_t)stream);
}

int mxgemm_run_fused(const void* A, const uint8_t* scaleA, const void* B, const uint8_t* scaleB, void* C,
                     int64_t M, int64_t N, int64_t K, int fmt, const float* bias, int act, int out_type,
                     void* stream) {
  int s = validate_mx(A, scaleA, B, scaleB, C, M, N, K, fmt);
  if (s != MXG_OK) return s;
  s = validate_epi(bias, act, out_type);
  if (s != MXG_OK) return s;
  s = check_device();
  if (s != MXG_OK) return s;
  return run_mx(A, scaleA, B, scaleB, mxg::Epi{C, bias, out_type, act}, M, N, K, fmt, (hipStream_t)stream);
}

int mxgemm_epilogue(const float* X, int64_t M, int64_t N, const float* bias, int act, int out_type, void* Y,
                    void* stream) {
  if (!X || !Y) return MXG_EINVAL;
  if (!dim_ok(M) || !dim_ok(N)) return MXG_EINVAL;
  if (!aligned16(X) || !aligned16(Y)) return MXG_EALIGN;
  int s = validate_epi(bias, act, out_type);
  if (s != MXG_OK) return s;
  s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_epilogue(X, M, N, mxg::Epi{Y, bias, out_type, act}, (hipStream_t)stream));
}

int fp16gemm_run(const uint16_t* A, const uint16_t* B, float* C, int64_t M, int64_t N, int64_t K, int b_is_nk,
                 void* stream) {
  if (!A || !B || !C) return MXG_EINVAL;
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || (K % 8) != 0) return MXG_EINVAL;
  if (b_is_nk != 0 && b_is_nk != 1) return MXG_EINVAL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(C)) return MXG_EALIGN;
  const int s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_f16_tiled(A, B, C, M, N, K, b_is_nk, (hipStream_t)stream));
}

int mxgemm_run_dequant_fp16(const void* A, const uint8_t* scaleA, const void* B, const uint8_t* scaleB, float* C,
                            int64_t M, int64_t N, int64_t K, int fmt, void* stream) {
  int s = validate_mx(A, scaleA, B, scaleB, C, M, N, K, fmt);
  if (s != MXG_OK) return s;
  if (fmt != MXG_FMT_FP8_FP8) return MXG_EINVAL;
  s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_deq_tiled(A, scaleA, B, scaleB, C, M, N, K, (hipStream_t)stream));
}

int int8gemm_quantize(const void* X, int in_type, int64_t rows, int64_t K, int8_t* Q, float* S, void* stream) {
  if (!X || !Q || !S || !type_ok(in_type)) return MXG_EINVAL;
  if (rows < 1 || rows > MXG_MAX_SLOTS || !dim_ok(K) || (K % 16) != 0) return MXG_EINVAL;
  if (!aligned16(X) || !aligned16(Q) || !aligned4(S)) return MXG_EALIGN;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(mxg::launch_quantize_int8(X, in_type, rows, K, Q, S, (hipStream_t)stream));
}

int int8gemm_run(const int8_t* A, const float* scaleA, const int8_t* B, const float* scaleB, void* C, int64_t M,
                 int64_t N, int64_t K, const float* bias, int act, int out_type, void* stream) {
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return MXG_EINVAL;
  return run_int8(mxg::I8Args{A, scaleA, M, B, scaleB, mxg::Epi{C, bias, out_type, act}, M, (int)N, (int)K, 1, nullptr,
                              nullptr, 1, 0, 0},
                  bias, act, out_type, (hipStream_t)stream);
}

int int8gemm_run_grouped(const int8_t* A, const float* scaleA, int64_t rowsA, const int8_t* B, const float* scaleB,
                         void* C, int64_t rows, int64_t N, int64_t K, int64_t E, const int32_t* offsets,
                         const int32_t* index, int index_div, const float* bias, int act, int out_type,
                         void* stream) {
  if (!offsets || rows < 1 || rows > MXG_MAX_SLOTS || rowsA < 1 || rowsA > MXG_MAX_SLOTS) return MXG_EINVAL;
  if (!dim_ok(N) || !dim_ok(K) || E < 1 || E > MXG_MAX_EXPERTS || index_div < 1) return MXG_EINVAL;
  if (index == nullptr && rowsA < rows) return MXG_EINVAL;
  return run_int8(mxg::I8Args{A, scaleA, rowsA, B, scaleB, mxg::Epi{C, bias, out_type, act}, rows, (int)N, (int)K,
                              (int)E, offsets, index, index_div, 0, 0},
                  bias, act, out_type, (hipStream_t)stream);
}

int expert_route(const void* logits, int in_type, int64_t T, int64_t E, int k, int score, const float* bias, int groups,
                 int top_groups, int group_top, int renormalize, float scale, int32_t* ids, float* weights,
                 void* stream) {
  int s = validate_route(logits, in_type, T, E, k, score);
  if (s != MXG_OK) return s;
  if (!ids || !weights || (renormalize != 0 && renormalize != 1)) return MXG_EINVAL;
  if (groups < 1 || groups > MXG_MAX_GROUPS || E % groups != 0 || top_groups < 1 || top_groups > groups)
    return MXG_EINVAL;
  if (group_top != 1 && group_top != 2) return MXG_EINVAL;
  if (E / groups * top_groups < k) return MXG_EINVAL;
  if (!aligned4(bias) || !aligned4(ids) || !aligned4(weights)) return MXG_EALIGN;
  s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_route(mxg::RouteArgs{logits, bias, T, (int)E, k, score, groups, top_groups, group_top,
                                                    renormalize, scale, ids, weights},
                                     in_type, (hipStream_t)stream));
}

int expert_route_backward(const void* logits, int in_type, int64_t T, int64_t E, const int32_t* ids,
                          const float* d_weights, int k, int score, int renormalize, float scale, void* d_logits,
                          void* stream) {
  int s = validate_route(logits, in_type, T, E, k, score);
  if (s != MXG_OK) return s;
  if (!ids || !d_weights || !d_logits || (renormalize != 0 && renormalize != 1)) return MXG_EINVAL;
  if (!aligned4(ids) || !aligned4(d_weights) || !aligned_elem(d_logits, in_type)) return MXG_EALIGN;
  s = check_device();
  if (s != MXG_OK) return s;
  return to_status(mxg::launch_route_backward(mxg::RouteArgs{logits, nullptr, T, (int)E, k, score, 1, 1, 1,
                                                             renormalize, scale, const_cast<int32_t*>(ids), nullptr},
                                              in_type, d_weights, d_logits, (hipStream_t)stream));
}

int64_t expert_plan_workspace(int64_t T, int k, int64_t E) {
  if (!dim_ok(T) || k < 1 || k > MXG_MAX_CHOICES || E < 1 || E > MXG_MAX_EXPERTS) return -1;
  return mxg::plan_workspace(T * k, (int)E);
}

int expert_plan(const int32_t* ids, int64_t T, int k, int64_t E, int32_t* offsets, int32_t* order, int32_t* position,
                void* workspace, void* stream) {
  if (!ids || !offsets || !order || !position) return MXG_EINVAL;
  const int64_t need = expert_plan_workspace(T, k, E);
  if (need < 0 || (need > 0 && !workspace)) return MXG_EINVAL;
  if (!aligned4(ids) || !aligned4(offsets) || !aligned4(order) || !aligned4(position) || !aligned4(workspace))
    return MXG_EALIGN;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(
      mxg::launch_plan(ids, T * k, (int)E, offsets, order, position, workspace, (hipStream_t)stream));
}

int expert_combine(const void* Y, int y_type, int64_t rows, int64_t N, const int32_t* position, const float* weights,
                   int64_t T, int k, void* out, int out_type, void* stream) {
  const mxg::CombineArgs a{Y, rows, N, position, weights, T, k, out};
  const int s = validate_combine(a, y_type, out_type);
  if (s != MXG_OK) return s;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(mxg::launch_combine(a, y_type, out_type, (hipStream_t)stream));
}

int expert_combine_backward(const void* dOut, int out_type, const void* Y, int y_type, int64_t rows, int64_t N,
                            const int32_t* position, const float* weights, int64_t T, int k, void* dY, float* dW,
                            void* stream) {
  const mxg::CombineArgs a{Y, rows, N, position, weights, T, k, const_cast<void*>(dOut)};
  const int s = validate_combine(a, y_type, out_type);
  if (s != MXG_OK) return s;
  if (!dY || !dW) return MXG_EINVAL;
  if (!aligned16(dY) || !aligned4(dW)) return MXG_EALIGN;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(mxg::launch_combine_backward(a, y_type, out_type, dY, dW, (hipStream_t)stream));
}

int fp8gemm_quantize(const void* X, int in_type, int64_t E, int64_t rows, int64_t K, int block_rows, int pow2, uint8_t* Q,
                     float* S, void* stream) {
  if (!X || !Q || !S || !type_ok(in_type) || (pow2 != 0 && pow2 != 1)) return MXG_EINVAL;
  if (E < 1 || E > MXG_MAX_EXPERTS || !dim_ok(K) || (K % 16) != 0) return MXG_EINVAL;
  if (block_rows == 1) {
    if (rows < 1 || rows > MXG_MAX_SLOTS || E * rows > MXG_MAX_SLOTS) return MXG_EINVAL;
  } else if (block_rows != 128 || !dim_ok(rows)) {
    return MXG_EINVAL;
  }
  if (!aligned16(X) || !aligned16(Q) || !aligned4(S)) return MXG_EALIGN;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(
      mxg::launch_quantize_fp8(X, in_type, E, rows, K, block_rows, pow2 != 0, Q, S, (hipStream_t)stream));
}

int fp8gemm_run(const uint8_t* A, const float* scaleA, const uint8_t* B, const float* scaleB, void* C, int64_t M, int64_t N,
                int64_t K, const float* bias, int act, int out_type, void* stream) {
  if (!dim_ok(M) || !fp8_dims_ok(N, K)) return MXG_EINVAL;
  return run_fp8(mxg::F8Args{A, scaleA, M, B, scaleB, mxg::Epi{C, bias, out_type, act}, M, (int)N, (int)K, 1, nullptr,
                             nullptr, 1, 0, 0, blocks_of(K), blocks_of(N)},
                 bias, act, out_type, (hipStream_t)stream);
}

int fp8gemm_run_grouped(const uint8_t* A, const float* scaleA, int64_t rowsA, const uint8_t* B, const float* scaleB,
                        void* C, int64_t rows, int64_t N, int64_t K, int64_t E, const int32_t* offsets,
                        const int32_t* index, int index_div, const float* bias, int act, int out_type, void* stream) {
  if (!fp8_dims_ok(N, K) || !experts_ok(offsets, index, index_div, rows, rowsA, E)) return MXG_EINVAL;
  return run_fp8(mxg::F8Args{A, scaleA, rowsA, B, scaleB, mxg::Epi{C, bias, out_type, act}, rows, (int)N, (int)K, (int)E,
                             offsets, index, index_div, 0, 0, blocks_of(K), blocks_of(N)},
                 bias, act, out_type, (hipStream_t)stream);
}

int64_t fp8gemm_weight_grad_workspace(int64_t M, int64_t N, int64_t K, int64_t E) {
  if (M < 1 || M > MXG_MAX_SLOTS || !fp8_dims_ok(N, K) || E < 1 || E > MXG_MAX_EXPERTS) return -1;
  return mxg::fp8_weight_grad_bytes(M, N, K, E);
}

int fp8gemm_weight_grad(const void* dC, int c_type, int64_t M, int64_t N, const uint8_t* A, const float* scaleA, int64_t K,
                        void* dW, int out_type, void* workspace, void* stream) {
  if (M < 1 || M > MXG_MAX_SLOTS || !fp8_dims_ok(N, K)) return MXG_EINVAL;
  return run_fp8_grad(mxg::F8GradArgs{dC, M, A, scaleA, M, (int)N, (int)K, blocks_of(K), 1, nullptr, nullptr, 1, 0, 0, dW,
                                      out_type, workspace},
                      c_type, (hipStream_t)stream);
}

int fp8gemm_weight_grad_grouped(const void* dC, int c_type, int64_t rows, int64_t N, const uint8_t* A,
                                const float* scaleA, int64_t rowsA, int64_t K, int64_t E, const int32_t* offsets,
                                const int32_t* index, int index_div, void* dW, int out_type, void* workspace,
                                void* stream) {
  if (!fp8_dims_ok(N, K) || !experts_ok(offsets, index, index_div, rows, rowsA, E)) return MXG_EINVAL;
  return run_fp8_grad(mxg::F8GradArgs{dC, rows, A, scaleA, rowsA, (int)N, (int)K, blocks_of(K), (int)E, offsets, index,
                                      index_div, 0, 0, dW, out_type, workspace},
                      c_type, (hipStream_t)stream);
}

int rmsnorm_quantize(const void* X, const void* R, int type, const void* W, int w_type, int64_t rows, int64_t K, float eps,
                     void* H, void* Y, int quant, uint8_t* Q, void* S, float* rstd, void* stream) {
  if (!X || !W || !type_ok(type) || !type_ok(w_type) || !norm_dims_ok(rows, K)) return MXG_EINVAL;
  if (!(eps >= 0.0f) || eps > 3.0e38f || (R == nullptr) != (H == nullptr)) return MXG_EINVAL;
  if (quant < MXG_QUANT_NONE || quant > MXG_QUANT_MXFP8 || (quant == MXG_QUANT_MXFP8 && K % 32 != 0)) return MXG_EINVAL;
  if (quant == MXG_QUANT_NONE ? (!Y || Q || S) : (!Q || !S)) return MXG_EINVAL;
  if (!aligned16(X) || !aligned16(R) || !aligned16(W) || !aligned16(H) || !aligned16(Y) || !aligned16(Q)) return MXG_EALIGN;
  if (!aligned4(rstd) || (quant != MXG_QUANT_MXFP8 && !aligned4(S))) return MXG_EALIGN;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(mxg::launch_rmsnorm(mxg::NormArgs{X, R, W, w_type, rows, (int)K, eps, H, Y, quant, Q, S, rstd}, type,
                                       (hipStream_t)stream));
}

int64_t rmsnorm_backward_workspace(int64_t rows, int64_t K) {
  return norm_dims_ok(rows, K) ? mxg::rmsnorm_backward_bytes(rows, K) : -1;
}

int rmsnorm_backward(const void* dY, const void* H, const void* dH, int type, const void* W, int w_type, const float* rstd,
                     int64_t rows, int64_t K, void* dX, float* dW, void* workspace, void* stream) {
  if (!dY || !H || !W || !rstd || !dX || !dW) return MXG_EINVAL;
  if (!type_ok(type) || !type_ok(w_type) || !norm_dims_ok(rows, K)) return MXG_EINVAL;
  if (!workspace && mxg::rmsnorm_backward_bytes(rows, K) > 0) return MXG_EINVAL;
  if (!aligned16(dY) || !aligned16(H) || !aligned16(dH) || !aligned16(W) || !aligned16(dX) || !aligned16(dW) ||
      !aligned16(workspace) || !aligned4(rstd))
    return MXG_EALIGN;
  const int d = check_device();
  if (d != MXG_OK) return d;
  return to_status(mxg::launch_rmsnorm_backward(
      mxg::NormGradArgs{dY, H, dH, W, w_type, rstd, rows, (int)K, dX, dW, workspace}, type, (hipStream_t)stream));
}

}  // extern "C"
