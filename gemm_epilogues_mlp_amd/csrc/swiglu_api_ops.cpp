// swiglu_api_ops.cpp -- the extern "C" entry points of the mixture-of-experts,
// MXFP4 and 8-bit integer operators.  Checks first (swiglu_checks.hpp), then the device of the
// handle, then the launch; on any error nothing is enqueued.
#include "swiglu.h"

#include <hip/hip_runtime.h>

#include "swiglu_checks.hpp"
#include "swiglu_internal.h"

namespace {

using namespace swiglu;

swiglu_status_t check_device(swiglu_handle_t h) {
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess) return SWIGLU_ERR_DEVICE;
  return cur == handle_device(h) ? SWIGLU_OK : SWIGLU_ERR_DEVICE;
}

swiglu_status_t launched(hipError_t e) { return e == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH; }

swiglu_status_t run_grouped(swiglu_handle_t h, bool up, const void* A, const int32_t* rows,
                            const int32_t* offsets, const void* W, void* Y, int64_t TA, int64_t R,
                            int64_t N, int64_t K, int64_t E, int64_t k, int32_t variant,
                            hipStream_t stream) {
  if (!h || variant >= kGroupedVariants) return SWIGLU_ERR_INVALID_ARG;
  bool noop;
  const int c = checks::grouped(up, A, rows, offsets, W, Y, TA, R, N, K, E, k, variant, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_grouped(up, (const uint16_t*)A, rows, offsets, (const uint16_t*)W,
                                 (uint16_t*)Y, (int)TA, (int)R, (int)N, (int)K, (int)E, (int)k,
                                 variant, stream));
}

swiglu_status_t run_int8(swiglu_handle_t h, bool gated, bool grouped, const void* A,
                         const float* SA, const int32_t* rows, const int32_t* offsets,
                         const void* W, const float* SW, void* Y, int64_t TA, int64_t R, int64_t N,
                         int64_t K, int64_t E, int64_t k, int32_t variant, hipStream_t stream) {
  if (!h || variant >= kInt8Variants) return SWIGLU_ERR_INVALID_ARG;
  const Int8Call call{gated,       grouped, (const uint8_t*)A, SA, rows, offsets, (const uint8_t*)W,
                      SW,          (uint16_t*)Y, TA, R, N, K, E, k, handle_cu_count(h)};
  bool noop;
  const int c = checks::int8_product(call, variant, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_int8(call, variant, stream));
}

}  // namespace

extern "C" {

int64_t swiglu_route_workspace_bytes(int64_t T, int64_t E, int64_t k) {
  if (T < 0 || E < 1 || k < 1 || k > E || E > kMaxExperts || k > kMaxChoices ||
      T > checks::kMaxSlots || T * k > checks::kMaxSlots)
    return 0;
  return route_workspace_bytes(T, E, k);
}

swiglu_status_t swiglu_route(swiglu_handle_t h, const void* logits, float* weights,
                             int32_t* experts, int32_t* offsets, int32_t* rows, void* workspace,
                             int64_t workspace_bytes, int64_t T, int64_t E, int64_t k,
                             int32_t renormalize, swiglu_dtype_t dtype, hipStream_t stream) {
  if (!h) return SWIGLU_ERR_INVALID_ARG;
  const int c = checks::route(logits, weights, experts, offsets, rows, workspace, workspace_bytes,
                              T, E, k, (int)dtype);
  if (c != checks::kOk) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_route(logits, dtype == SWIGLU_DTYPE_F32, weights, experts, offsets, rows,
                               workspace, (int)T, (int)E, (int)k, renormalize != 0, stream));
}

swiglu_status_t swiglu_route_scored(swiglu_handle_t h, const void* logits, const float* bias,
                                    float* weights, int32_t* experts, int32_t* offsets,
                                    int32_t* rows, void* workspace, int64_t workspace_bytes,
                                    int64_t T, int64_t E, int64_t k, swiglu_score_t score,
                                    int32_t renormalize, float scale, int32_t groups,
                                    int32_t top_groups, int32_t group_best, swiglu_dtype_t dtype,
                                    hipStream_t stream) {
  if (!h) return SWIGLU_ERR_INVALID_ARG;
  int c = checks::route(logits, weights, experts, offsets, rows, workspace, workspace_bytes, T, E,
                        k, (int)dtype);
  if (c != checks::kOk) return (swiglu_status_t)c;
  const RouteScore s{bias,   score == SWIGLU_SCORE_SIGMOID, scale, groups, top_groups, group_best};
  c = checks::route_score(s, weights, experts, offsets, rows, workspace, T, E, k, (int)score);
  if (c != checks::kOk) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_route_scored(logits, dtype == SWIGLU_DTYPE_F32, weights, experts, offsets,
                                      rows, workspace, (int)T, (int)E, (int)k, renormalize != 0, s,
                                      stream));
}

swiglu_status_t swiglu_grouped_forward(swiglu_handle_t h, const void* A, const int32_t* rows,
                                       const int32_t* offsets, const void* W, void* Y, int64_t T,
                                       int64_t R, int64_t N, int64_t K, int64_t E, int64_t k,
                                       int32_t variant, hipStream_t stream) {
  return run_grouped(h, true, A, rows, offsets, W, Y, T, R, N, K, E, k, variant, stream);
}

swiglu_status_t swiglu_grouped_matmul(swiglu_handle_t h, const void* A, const int32_t* rows,
                                      const int32_t* offsets, const void* W, void* Y, int64_t R,
                                      int64_t N, int64_t K, int64_t E, int32_t variant,
                                      hipStream_t stream) {
  return run_grouped(h, false, A, rows, offsets, W, Y, R, R, N, K, E, 1, variant, stream);
}

swiglu_status_t swiglu_combine_norm(swiglu_handle_t h, const void* B, const float* weights,
                                    const int32_t* experts, const void* S, const void* X,
                                    const void* post, const void* gate, const void* pre,
                                    void* X_out, void* H, int64_t T, int64_t D, int64_t k,
                                    float scale, float eps, int64_t gate_ld, swiglu_dtype_t dtype,
                                    hipStream_t stream) {
  if (!h) return SWIGLU_ERR_INVALID_ARG;
  const NormCall call{B, weights, experts, S, X,   post,  gate, pre, X_out,
                      H, T,       D,       k, scale, eps, gate_ld, dtype == SWIGLU_DTYPE_F32};
  bool noop;
  const int c = checks::combine_norm(call, (int)dtype, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_combine_norm(call, stream));
}

int64_t swiglu_mxfp4_bytes(int64_t rows, int64_t K) {
  if (rows <= 0 || K <= 0 || rows > 0x7fffffffLL || K > 0x7fffffffLL) return 0;
  return fp4_code_bytes(rows, K);
}

int64_t swiglu_mxfp4_scale_bytes(int64_t rows, int64_t K) {
  if (rows <= 0 || K <= 0 || rows > 0x7fffffffLL || K > 0x7fffffffLL) return 0;
  return fp4_scale_bytes(rows, K);
}

swiglu_status_t swiglu_quantize_mxfp4(swiglu_handle_t h, const void* X, void* Q, void* S,
                                      int64_t rows, int64_t K, hipStream_t stream) {
  if (!h) return SWIGLU_ERR_INVALID_ARG;
  bool noop;
  const int c = checks::convert_mxfp4(X, Q, S, rows, K, false, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_quantize_mxfp4((const uint16_t*)X, (uint8_t*)Q, (uint8_t*)S, (int)rows,
                                        (int)K, stream));
}

swiglu_status_t swiglu_dequantize_mxfp4(swiglu_handle_t h, const void* Q, const void* S, void* X,
                                        int64_t rows, int64_t K, hipStream_t stream) {
  if (!h) return SWIGLU_ERR_INVALID_ARG;
  bool noop;
  const int c = checks::convert_mxfp4(X, Q, S, rows, K, true, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_dequantize_mxfp4((const uint8_t*)Q, (const uint8_t*)S, (uint16_t*)X,
                                          (int)rows, (int)K, stream));
}

swiglu_status_t swiglu_forward_mxfp4(swiglu_handle_t h, const void* Q, const void* SQ,
                                     const void* W, const void* SW, void* Y, int64_t M, int64_t N,
                                     int64_t K, int32_t variant, hipStream_t stream) {
  if (!h || variant >= kFp4Variants) return SWIGLU_ERR_INVALID_ARG;
  const Fp4Call call{(const uint8_t*)Q, (const uint8_t*)SQ, (const uint8_t*)W, (const uint8_t*)SW,
                     (uint16_t*)Y,      M,                  N,                 K,
                     handle_cu_count(h)};
  bool noop;
  const int c = checks::forward_mxfp4(call, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  if ((variant == 0 || variant == 1) && (M + 31) / 32 > 65535) return SWIGLU_ERR_UNSUPPORTED;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_forward_mxfp4(call, variant, stream));
}

int64_t swiglu_int8_packed_bytes(int64_t rows, int64_t K) {
  if (rows <= 0 || K <= 0 || rows > 0x7fffffffLL || K > 0x7fffffffLL) return 0;
  return int8_packed_bytes(rows, K);
}

swiglu_status_t swiglu_pack_int8_fragments(swiglu_handle_t h, const void* W8, void* P, int64_t E,
                                           int64_t rows, int64_t K, hipStream_t stream) {
  if (!h) return SWIGLU_ERR_INVALID_ARG;
  bool noop;
  const int c = checks::pack_int8(W8, P, E, rows, K, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_pack_int8((const uint8_t*)W8, (uint8_t*)P, E, (int)rows, (int)K, stream));
}

swiglu_status_t swiglu_quantize_int8(swiglu_handle_t h, const void* X, void* Q, float* S,
                                     int64_t rows, int64_t K, hipStream_t stream) {
  if (!h) return SWIGLU_ERR_INVALID_ARG;
  bool noop;
  const int c = checks::quantize_int8(X, Q, S, rows, K, &noop);
  if (c != checks::kOk || noop) return (swiglu_status_t)c;
  const swiglu_status_t st = check_device(h);
  if (st != SWIGLU_OK) return st;
  return launched(launch_quantize_int8((const uint16_t*)X, (uint8_t*)Q, S, (int)rows, (int)K, stream));
}

swiglu_status_t swiglu_forward_int8(swiglu_handle_t h, const void* Q, const float* SQ,
                                    const void* P, const float* SW, void* Y, int64_t M, int64_t N,
                                    int64_t K, int32_t variant, hipStream_t stream) {
  return run_int8(h, true, false, Q, SQ, nullptr, nullptr, P, SW, Y, M, M, N, K, 1, 1, variant, stream);
}

swiglu_status_t swiglu_matmul_int8(swiglu_handle_t h, const void* Q, const float* SQ,
                                   const void* P, const float* SW, void* Y, int64_t M, int64_t N,
                                   int64_t K, int32_t variant, hipStream_t stream) {
  return run_int8(h, false, false, Q, SQ, nullptr, nullptr, P, SW, Y, M, M, N, K, 1, 1, variant, stream);
}

swiglu_status_t swiglu_grouped_forward_int8(swiglu_handle_t h, const void* Q, const float* SQ,
                                            const int32_t* rows, const int32_t* offsets,
                                            const void* P, const float* SW, void* Y, int64_t T,
                                            int64_t R, int64_t N, int64_t K, int64_t E, int64_t k,
                                            int32_t variant, hipStream_t stream) {
  return run_int8(h, true, true, Q, SQ, rows, offsets, P, SW, Y, T, R, N, K, E, k, variant, stream);
}

swiglu_status_t swiglu_grouped_matmul_int8(swiglu_handle_t h, const void* Q, const float* SQ,
                                           const int32_t* rows, const int32_t* offsets,
                                           const void* P, const float* SW, void* Y, int64_t R,
                                           int64_t N, int64_t K, int64_t E, int32_t variant,
                                           hipStream_t stream) {
  return run_int8(h, false, true, Q, SQ, rows, offsets, P, SW, Y, R, R, N, K, E, 1, variant, stream);
}

}  // extern "C"
