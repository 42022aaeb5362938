// api.cu -- the C ABI of libnvfp4.so: argument checks, workspace sizing and
// dispatch.  Host-detectable errors return before anything is launched.
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "grouped.cuh"
#include "nvfp4.h"
#include "nvfp4_internal.h"

namespace {

constexpr uint32_t kQuantFlags = NVFP4_ROWWISE | NVFP4_COLWISE | NVFP4_BLOCK2D | NVFP4_SINGLE_PASS | NVFP4_HEADROOM |
                                 NVFP4_ALPHA_PROVIDED | NVFP4_GEMM_SCALE_LAYOUT | NVFP4_RHT | NVFP4_VECTOR_SCALES |
                                 NVFP4_AMAX_PROVIDED;
constexpr uint32_t kDequantFlags = NVFP4_BLOCK2D | NVFP4_GEMM_SCALE_LAYOUT | NVFP4_INVERSE_RHT | NVFP4_OUT_BF16;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

nvfp4_status_t launch_status(cudaError_t e) {
  if (e == cudaSuccess) return NVFP4_OK;
  return (e == cudaErrorInvalidConfiguration || e == cudaErrorLaunchOutOfResources ||
          e == cudaErrorInvalidDeviceFunction || e == cudaErrorNoKernelImageForDevice ||
          e == cudaErrorCooperativeLaunchTooLarge)
             ? NVFP4_ERR_LAUNCH
             : NVFP4_ERR_CUDA;
}

std::atomic<uint64_t> g_launches{0};

// Checks shared by the grouped calls: group count, row count, offsets.
nvfp4_status_t check_groups(const int32_t* offsets, int64_t E, int64_t T) {
  if (E < 1 || E > nvfp4::kMaxGroups || T < 0 || T >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (!offsets) return NVFP4_ERR_ARG;
  return aligned(offsets, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// Checks shared by the adapter calls: sizes, the adapters, the token list.
nvfp4_status_t check_lora(const void* A, const void* B, const float* scaling, const int32_t* ids, int64_t T, int64_t K,
                          int64_t N, int64_t r, int64_t n) {
  constexpr int64_t most = int64_t(1) << 22;
  if (T < 0 || T >= (int64_t(1) << 31) || K < 8 || N < 8 || K > most || N > most || K % 8 || N % 8 || r < 8 || r > 128 ||
      r % 8 || n < 1 || n > 65535)
    return NVFP4_ERR_SHAPE;
  if (!A || !B || !scaling || (T && !ids)) return NVFP4_ERR_ARG;
  return aligned(A, 16) && aligned(B, 16) && aligned(scaling, 4) && aligned(ids, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// A bf16 matrix of T rows: present, 16-byte aligned, rows of at least `cols`.
nvfp4_status_t check_rows(const void* p, int64_t ld, int64_t cols) {
  if (!p) return NVFP4_ERR_ARG;
  if (ld < cols) return NVFP4_ERR_SHAPE;
  return aligned(p, 16) && ld % 8 == 0 ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

constexpr int64_t kMost = int64_t(1) << 31;

// Tokens and their choices: T k pairs are counted in 32 bits.
bool bad_pairs(int64_t T, int64_t k) { return T < 0 || T >= kMost || k < 1 || k > 32 || T * k >= kMost; }

// Checks shared by the routing calls.
nvfp4_status_t check_route(const void* logits, int64_t ldl, int dtype, int64_t T, int64_t E, int64_t k, int score,
                           uint32_t flags) {
  if (dtype != NVFP4_OUT_DTYPE_BF16 && dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  if (score != NVFP4_ROUTE_SOFTMAX && score != NVFP4_ROUTE_SIGMOID) return NVFP4_ERR_ARG;
  if (flags & ~(NVFP4_ROUTE_RENORM | NVFP4_ROUTE_GROUP_PAIR)) return NVFP4_ERR_ARG;
  if (bad_pairs(T, k) || E < 1 || E > nvfp4::kMaxGroups || k > E || ldl < E) return NVFP4_ERR_SHAPE;
  if (T && !logits) return NVFP4_ERR_ARG;
  return aligned(logits, dtype == NVFP4_OUT_DTYPE_BF16 ? 2 : 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// Checks shared by the calls that move rows between tokens and pairs.
nvfp4_status_t check_pairs(const int32_t* rows, const float* weights, int64_t T, int64_t k, int64_t C, int64_t R,
                           const int32_t* status) {
  if (bad_pairs(T, k) || R < 0 || R >= kMost || C < 8 || C % 8 || C >= kMost) return NVFP4_ERR_SHAPE;
  if (!rows && T * k > R) return NVFP4_ERR_SHAPE;   // pair p has row p
  return aligned(rows, 4) && aligned(weights, 4) && aligned(status, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

}  // namespace

namespace nvfp4 {
void note_launch(int n) { g_launches.fetch_add(static_cast<uint64_t>(n), std::memory_order_relaxed); }

nvfp4_status_t check_quantize_args(const void* x, int64_t R, int64_t C, int64_t ld, nvfp4_mode_t mode,
                                   uint32_t flags, uint32_t stream_id, const float* alpha_in,
                                   const nvfp4_qtensor_t* out, bool* empty) {
  *empty = false;
  if (!out) return NVFP4_ERR_ARG;
  if (static_cast<int>(mode) < NVFP4_RTN || static_cast<int>(mode) > NVFP4_RHT_SR_HW) return NVFP4_ERR_ARG;
  if (flags & ~kQuantFlags) return NVFP4_ERR_ARG;
  const bool row = flags & NVFP4_ROWWISE, col = flags & NVFP4_COLWISE, two_d = flags & NVFP4_BLOCK2D;
  const bool gemm = flags & NVFP4_GEMM_SCALE_LAYOUT;
  if (!row && !col) return NVFP4_ERR_ARG;
  if (two_d && (mode == NVFP4_RHT_SR || mode == NVFP4_MS_EDEN || mode == NVFP4_RHT_SR_HW || (flags & NVFP4_RHT)))
    return NVFP4_ERR_ARG;
  if (stream_id >= 0x80000000u) return NVFP4_ERR_ARG;
  if ((flags & NVFP4_VECTOR_SCALES) && (flags & (NVFP4_BLOCK2D | NVFP4_SINGLE_PASS | NVFP4_ALPHA_PROVIDED)))
    return NVFP4_ERR_ARG;
  if ((flags & NVFP4_AMAX_PROVIDED) &&
      (flags & (NVFP4_ALPHA_PROVIDED | NVFP4_SINGLE_PASS | NVFP4_VECTOR_SCALES)))
    return NVFP4_ERR_ARG;
  if (R < 0 || C < 0 || ld < C) return NVFP4_ERR_SHAPE;
  if (C % 16) return NVFP4_ERR_SHAPE;
  if ((col || two_d) && R % 16) return NVFP4_ERR_SHAPE;
  if (R * (C / 16) >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (gemm) {
    if (row && (R % 128 || C % 64)) return NVFP4_ERR_SHAPE;
    if (col && (C % 128 || R % 64)) return NVFP4_ERR_SHAPE;
  }
  if (R == 0 || C == 0) {  // empty tensor: nothing to write
    *empty = true;
    return NVFP4_OK;
  }
  if ((flags & (NVFP4_ALPHA_PROVIDED | NVFP4_AMAX_PROVIDED)) && !alpha_in) return NVFP4_ERR_ARG;
  if ((flags & NVFP4_AMAX_PROVIDED) && !aligned(alpha_in, 4)) return NVFP4_ERR_ALIGN;
  if (row && (!out->codes_row || !out->scales_row || !out->alpha_row)) return NVFP4_ERR_ARG;
  if (col && (!out->codes_col || !out->scales_col || !out->alpha_col)) return NVFP4_ERR_ARG;
  if (!x) return NVFP4_ERR_ARG;
  if (!aligned(x, 16) || ld % 8) return NVFP4_ERR_ALIGN;
  if (row && !aligned(out->codes_row, 16)) return NVFP4_ERR_ALIGN;
  if (col && !aligned(out->codes_col, 16)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}
}  // namespace nvfp4

extern "C" {

uint64_t nvfp4_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

nvfp4_status_t nvfp4_amax(const void* x, int64_t R, int64_t C, int64_t ld, uint32_t flags, uint64_t seed,
                          float* amax_out, int32_t* status, void* stream) {
  if (flags & ~(NVFP4_ROWWISE | NVFP4_COLWISE | NVFP4_RHT)) return NVFP4_ERR_ARG;
  if (!amax_out) return NVFP4_ERR_ARG;
  if (R < 0 || C < 0 || ld < C || C % 16) return NVFP4_ERR_SHAPE;
  if ((flags & NVFP4_RHT) && (flags & NVFP4_COLWISE) && R % 16) return NVFP4_ERR_SHAPE;
  if (R * (C / 8) >= (int64_t(1) << 32)) return NVFP4_ERR_SHAPE;
  if (!aligned(amax_out, 4) || (status && !aligned(status, 4))) return NVFP4_ERR_ALIGN;
  if (R > 0 && C > 0) {
    if (!x) return NVFP4_ERR_ARG;
    if (!aligned(x, 16) || ld % 8) return NVFP4_ERR_ALIGN;
  }
  return launch_status(nvfp4::amax_launch(x, R, C, ld, flags, seed, amax_out, status,
                                          static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t mxfp4_quantize(const void* x, int64_t R, int64_t C, int64_t ld, uint32_t flags, uint64_t seed,
                              uint8_t* codes_row, uint8_t* scales_row, uint8_t* codes_col, uint8_t* scales_col,
                              int32_t* status, void* stream) {
  if (flags & ~(NVFP4_ROWWISE | NVFP4_COLWISE | NVFP4_RHT | NVFP4_GEMM_SCALE_LAYOUT)) return NVFP4_ERR_ARG;
  const bool row = flags & NVFP4_ROWWISE, col = flags & NVFP4_COLWISE;
  if (!row && !col) return NVFP4_ERR_ARG;
  if (R < 0 || C < 0 || ld < C) return NVFP4_ERR_SHAPE;
  if (C % 16 || (row && C % 32) || (col && R % 32)) return NVFP4_ERR_SHAPE;
  if ((flags & NVFP4_GEMM_SCALE_LAYOUT) && (R % 128 || C % 128)) return NVFP4_ERR_SHAPE;
  if (R * (C / 16) >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (R == 0 || C == 0) return NVFP4_OK;
  if (!x || (row && (!codes_row || !scales_row)) || (col && (!codes_col || !scales_col))) return NVFP4_ERR_ARG;
  if (!aligned(x, 16) || ld % 8) return NVFP4_ERR_ALIGN;
  if ((row && !aligned(codes_row, 16)) || (col && !aligned(codes_col, 16))) return NVFP4_ERR_ALIGN;
  return launch_status(nvfp4::mx_quantize_launch(x, R, C, ld, flags, seed, row ? codes_row : nullptr,
                                                 row ? scales_row : nullptr, col ? codes_col : nullptr,
                                                 col ? scales_col : nullptr, status,
                                                 static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t mxfp4_gemm(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB, int64_t M,
                          int64_t N, int64_t K, void* D, int out_dtype, int64_t ldd, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (out_dtype != NVFP4_OUT_DTYPE_BF16 && out_dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  if (M <= 0 || N <= 0 || K <= 0) return NVFP4_ERR_SHAPE;
  if (M % 256 || N % 256 || K % 128 || ldd < N) return NVFP4_ERR_SHAPE;
  if (M > (int64_t(1) << 31) || N > (int64_t(1) << 31) || K > (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (!A || !sA || !B || !sB || !D) return NVFP4_ERR_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 16) || !aligned(sB, 16) || !aligned(D, 16))
    return NVFP4_ERR_ALIGN;
  if ((ldd * (out_dtype == NVFP4_OUT_DTYPE_BF16 ? 2 : 4)) % 16) return NVFP4_ERR_ALIGN;
  int32_t* status = (workspace && workspace_bytes >= sizeof(int32_t) && aligned(workspace, 4))
                        ? static_cast<int32_t*>(workspace)
                        : nullptr;
  return launch_status(nvfp4::mx_gemm_launch(A, sA, B, sB, M, N, K, D, out_dtype, ldd, status,
                                             static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t C, uint32_t flags,
                                uint64_t seed, void* y, void* stream) {
  if (flags & ~(NVFP4_INVERSE_RHT | NVFP4_OUT_BF16)) return NVFP4_ERR_ARG;
  if (R < 0 || C < 0 || C % 32) return NVFP4_ERR_SHAPE;
  if (R * (C / 16) >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (R == 0 || C == 0) return NVFP4_OK;
  if (!codes || !scales || !y) return NVFP4_ERR_ARG;
  if (!aligned(codes, 8) || !aligned(y, 16)) return NVFP4_ERR_ALIGN;
  return launch_status(nvfp4::mx_dequantize_launch(codes, scales, R, C, flags, seed, y,
                                                   static_cast<cudaStream_t>(stream)));
}

int nvfp4_version(void) { return 10000; }

const char* nvfp4_status_string(nvfp4_status_t s) {
  switch (s) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_ARG: return "invalid argument (mode, flags or null pointer)";
    case NVFP4_ERR_SHAPE: return "shape breaks the block or tile rules";
    case NVFP4_ERR_ALIGN: return "pointer or stride not 16-byte aligned";
    case NVFP4_ERR_NONFINITE: return "input holds a NaN or an infinity";
    case NVFP4_ERR_LAUNCH: return "kernel launch failed";
    case NVFP4_ERR_TIMEOUT: return "a bounded device wait gave up";
    case NVFP4_ERR_CUDA: return "CUDA runtime error";
    case NVFP4_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

size_t nvfp4_workspace_size(int64_t R, int64_t C, uint32_t flags) {
  return nvfp4::quant_workspace_bytes(R, C, flags);
}

nvfp4_status_t nvfp4_quantize(const void* x, int64_t R, int64_t C, int64_t ld, nvfp4_mode_t mode,
                              uint32_t flags, uint64_t seed, uint32_t stream_id,
                              const float* alpha_in, const nvfp4_qtensor_t* out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  bool empty = false;
  const nvfp4_status_t chk = nvfp4::check_quantize_args(x, R, C, ld, mode, flags, stream_id, alpha_in, out, &empty);
  if (chk != NVFP4_OK || empty) return chk;
  const bool row = flags & NVFP4_ROWWISE, col = flags & NVFP4_COLWISE;
  const size_t need = nvfp4::quant_workspace_bytes(R, C, flags);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return NVFP4_ERR_WORKSPACE;
  nvfp4::QuantOutputs o{out->codes_row, out->scales_row, out->alpha_row, out->codes_col,
                        out->scales_col, out->alpha_col, out->amax_out, out->status};
  if (!row) o.codes_row = nullptr, o.scales_row = nullptr, o.alpha_row = nullptr;
  if (!col) o.codes_col = nullptr, o.scales_col = nullptr, o.alpha_col = nullptr;
  return launch_status(nvfp4::quantize_launch(x, R, C, ld, static_cast<int>(mode), flags, seed, stream_id,
                                              alpha_in, o, workspace, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* alpha,
                                int64_t R, int64_t C, uint32_t flags, uint64_t seed, void* y,
                                void* stream) {
  if (flags & ~kDequantFlags) return NVFP4_ERR_ARG;
  const bool two_d = flags & NVFP4_BLOCK2D, gemm = flags & NVFP4_GEMM_SCALE_LAYOUT;
  if (two_d && (flags & NVFP4_INVERSE_RHT)) return NVFP4_ERR_ARG;
  if (two_d && gemm) return NVFP4_ERR_ARG;
  if (R < 0 || C < 0 || C % 16) return NVFP4_ERR_SHAPE;
  if (two_d && R % 16) return NVFP4_ERR_SHAPE;
  if (gemm && (R % 128 || C % 64)) return NVFP4_ERR_SHAPE;
  if (R * (C / 16) >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (R == 0 || C == 0) return NVFP4_OK;
  if (!codes || !scales || !alpha || !y) return NVFP4_ERR_ARG;
  if (!aligned(codes, 8) || !aligned(y, 16)) return NVFP4_ERR_ALIGN;
  return launch_status(nvfp4::dequantize_launch(codes, scales, alpha, R, C, flags, seed, y,
                                                static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_gemm(const uint8_t* A, const uint8_t* sA, const float* alphaA, const uint8_t* B,
                          const uint8_t* sB, const float* alphaB, int64_t M, int64_t N, int64_t K,
                          void* D, int out_dtype, int64_t ldd, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (out_dtype != NVFP4_OUT_DTYPE_BF16 && out_dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  if (M <= 0 || N <= 0 || K <= 0) return NVFP4_ERR_SHAPE;
  if (M % 128 || N % 128 || K % 128 || ldd < N) return NVFP4_ERR_SHAPE;
  if (M > (int64_t(1) << 31) || N > (int64_t(1) << 31) || K > (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (!A || !sA || !alphaA || !B || !sB || !alphaB || !D) return NVFP4_ERR_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 16) || !aligned(sB, 16) || !aligned(D, 16))
    return NVFP4_ERR_ALIGN;
  if ((ldd * (out_dtype == NVFP4_OUT_DTYPE_BF16 ? 2 : 4)) % 16) return NVFP4_ERR_ALIGN;
  int32_t* status = (workspace && workspace_bytes >= sizeof(int32_t) && aligned(workspace, 4))
                        ? static_cast<int32_t*>(workspace)
                        : nullptr;
  return launch_status(nvfp4::gemm_launch(A, sA, alphaA, B, sB, alphaB, M, N, K, D, out_dtype, ldd, status,
                                          static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_gemm_vector_scales(const uint8_t* A, const uint8_t* sA, const float* alphaA, const uint8_t* B,
                                        const uint8_t* sB, const float* alphaB, int64_t M, int64_t N, int64_t K,
                                        void* D, int out_dtype, int64_t ldd, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  if (out_dtype != NVFP4_OUT_DTYPE_BF16 && out_dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  if (M <= 0 || N <= 0 || K <= 0) return NVFP4_ERR_SHAPE;
  if (M % 256 || N % 256 || K % 128 || ldd < N) return NVFP4_ERR_SHAPE;
  if (M > (int64_t(1) << 31) || N > (int64_t(1) << 31) || K > (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (!A || !sA || !alphaA || !B || !sB || !alphaB || !D) return NVFP4_ERR_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 16) || !aligned(sB, 16) || !aligned(D, 16))
    return NVFP4_ERR_ALIGN;
  if (!aligned(alphaA, 4) || !aligned(alphaB, 4)) return NVFP4_ERR_ALIGN;
  if ((ldd * (out_dtype == NVFP4_OUT_DTYPE_BF16 ? 2 : 4)) % 16) return NVFP4_ERR_ALIGN;
  int32_t* status = (workspace && workspace_bytes >= sizeof(int32_t) && aligned(workspace, 4))
                        ? static_cast<int32_t*>(workspace)
                        : nullptr;
  return launch_status(nvfp4::gemm_vs_launch(A, sA, alphaA, B, sB, alphaB, M, N, K, D, out_dtype, ldd, status,
                                             static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_gemm_quantize(const uint8_t* A, const uint8_t* sA, const float* alphaA, const uint8_t* B,
                                   const uint8_t* sB, const float* alphaB, int64_t M, int64_t N, int64_t K, void* D,
                                   int64_t ldd, nvfp4_mode_t mode, uint32_t flags, const float* alpha_out,
                                   uint8_t* codes, uint8_t* scales, float* amax_out, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (mode != NVFP4_RTN && mode != NVFP4_FOUR_SIX) return NVFP4_ERR_ARG;
  if (flags & ~NVFP4_GEMM_SCALE_LAYOUT) return NVFP4_ERR_ARG;
  if (M <= 0 || N <= 0 || K <= 0) return NVFP4_ERR_SHAPE;
  if (M % 256 || N % 256 || K % 128) return NVFP4_ERR_SHAPE;
  if (M > (int64_t(1) << 31) || N > (int64_t(1) << 31) || K > (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (M * (N / 16) >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (D && ldd < N) return NVFP4_ERR_SHAPE;
  if (!A || !sA || !alphaA || !B || !sB || !alphaB || !alpha_out || !codes || !scales) return NVFP4_ERR_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 16) || !aligned(sB, 16) || !aligned(codes, 16))
    return NVFP4_ERR_ALIGN;
  if (D && (!aligned(D, 16) || (ldd * 2) % 16)) return NVFP4_ERR_ALIGN;
  if (amax_out && !aligned(amax_out, 4)) return NVFP4_ERR_ALIGN;
  int32_t* status = (workspace && workspace_bytes >= sizeof(int32_t) && aligned(workspace, 4))
                        ? static_cast<int32_t*>(workspace)
                        : nullptr;
  return launch_status(nvfp4::gemm_quantize_launch(A, sA, alphaA, B, sB, alphaB, M, N, K, D, ldd,
                                                   static_cast<int>(mode), (flags & NVFP4_GEMM_SCALE_LAYOUT) != 0,
                                                   alpha_out, codes, scales, amax_out, status,
                                                   static_cast<cudaStream_t>(stream)));
}

int64_t nvfp4_grouped_capacity(int64_t T, int64_t E, int64_t step) {
  return (T < 0 || E < 0 || step < 1) ? 0 : nvfp4::grouped_capacity(T, E, step);
}

size_t nvfp4_grouped_workspace_size(int64_t E) { return E < 0 ? 0 : nvfp4::grouped_workspace_bytes(E); }

nvfp4_status_t nvfp4_quantize_grouped(const void* x, int64_t T, int64_t C, int64_t ld, const int32_t* offsets, int64_t E,
                                      nvfp4_mode_t mode, uint32_t flags, uint64_t seed, uint32_t stream_id,
                                      const nvfp4_qtensor_t* out, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  constexpr uint32_t allowed =
      NVFP4_ROWWISE | NVFP4_COLWISE | NVFP4_RHT | NVFP4_HEADROOM | NVFP4_GEMM_SCALE_LAYOUT;
  const bool row = flags & NVFP4_ROWWISE, col = flags & NVFP4_COLWISE;
  if (!out || (flags & ~allowed) || (!row && !col)) return NVFP4_ERR_ARG;
  if (static_cast<int>(mode) < NVFP4_RTN || static_cast<int>(mode) > NVFP4_RHT_SR_HW) return NVFP4_ERR_ARG;
  const nvfp4_status_t chk = check_groups(offsets, E, T);
  if (chk != NVFP4_OK) return chk;
  if (stream_id >= 0x80000000u - static_cast<uint32_t>(E) + 1u) return NVFP4_ERR_ARG;
  if (C <= 0 || ld < C || C % (col ? 128 : 64)) return NVFP4_ERR_SHAPE;
  if (nvfp4::grouped_capacity(T, E, 128) * (C / 16) >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (row && (!out->alpha_row || (T && (!out->codes_row || !out->scales_row)))) return NVFP4_ERR_ARG;
  if (col && (!out->alpha_col || (T && (!out->codes_col || !out->scales_col)))) return NVFP4_ERR_ARG;
  if (T && !x) return NVFP4_ERR_ARG;
  if (!aligned(x, 16) || ld % 8) return NVFP4_ERR_ALIGN;
  if (row && (!aligned(out->codes_row, 16) || !aligned(out->scales_row, 16))) return NVFP4_ERR_ALIGN;
  if (col && (!aligned(out->codes_col, 16) || !aligned(out->scales_col, 16))) return NVFP4_ERR_ALIGN;
  if ((row && !aligned(out->alpha_row, 4)) || (col && !aligned(out->alpha_col, 4)) || !aligned(out->amax_out, 4) ||
      !aligned(out->status, 4))
    return NVFP4_ERR_ALIGN;
  if (!workspace || workspace_bytes < nvfp4::grouped_workspace_bytes(E) || !aligned(workspace, 16))
    return NVFP4_ERR_WORKSPACE;
  const nvfp4::QuantOutputs o{out->codes_row, out->scales_row, out->alpha_row, out->codes_col,
                              out->scales_col, out->alpha_col, out->amax_out, out->status};
  return launch_status(nvfp4::grouped_quantize_launch(x, T, C, ld, offsets, E, static_cast<int>(mode), flags, seed,
                                                      stream_id, o, workspace, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_dequantize_grouped(const uint8_t* codes, const uint8_t* scales, const float* alpha, int64_t T,
                                        int64_t C, const int32_t* offsets, int64_t E, uint32_t flags, uint64_t seed,
                                        void* y, int32_t* status, void* stream) {
  if (flags & ~(NVFP4_ROWWISE | NVFP4_COLWISE | NVFP4_INVERSE_RHT | NVFP4_OUT_BF16 | NVFP4_GEMM_SCALE_LAYOUT))
    return NVFP4_ERR_ARG;
  const bool row = flags & NVFP4_ROWWISE, col = flags & NVFP4_COLWISE;
  if (row == col) return NVFP4_ERR_ARG;
  const nvfp4_status_t chk = check_groups(offsets, E, T);
  if (chk != NVFP4_OK) return chk;
  if (C <= 0 || C % (col ? 128 : 64)) return NVFP4_ERR_SHAPE;
  if (nvfp4::grouped_capacity(T, E, 128) * (C / 16) >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!codes || !scales || !alpha || !y) return NVFP4_ERR_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(y, 16) || !aligned(alpha, 4) || !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  return launch_status(nvfp4::grouped_dequantize_launch(codes, scales, alpha, T, C, offsets, E, flags, seed, y, status,
                                                        static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_gemm_grouped(const uint8_t* A, const uint8_t* sA, const float* alphaA, const uint8_t* B,
                                  const uint8_t* sB, const float* alphaB, const int32_t* offsets, int64_t E, int64_t T,
                                  int64_t N, int64_t K, void* D, int out_dtype, int64_t ldd, int32_t* status,
                                  void* stream) {
  if (out_dtype != NVFP4_OUT_DTYPE_BF16 && out_dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  const nvfp4_status_t chk = check_groups(offsets, E, T);
  if (chk != NVFP4_OK) return chk;
  if (N <= 0 || K <= 0 || N % 128 || K % 64 || ldd < N) return NVFP4_ERR_SHAPE;
  if (N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  // operand rows, scale atoms and tiles are counted in 32 bits
  if (E * N >= (int64_t(1) << 31) || E * (N / 128) * (K / 64) >= (int64_t(1) << 29) ||
      nvfp4::grouped_capacity(T, E, 128) / 128 * (K / 64) >= (int64_t(1) << 29) ||
      nvfp4::grouped_capacity(T, E, 128) / 128 * (N / 128) >= (int64_t(1) << 29))
    return NVFP4_ERR_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!A || !sA || !alphaA || !B || !sB || !alphaB || !D) return NVFP4_ERR_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 16) || !aligned(sB, 16) || !aligned(D, 16) ||
      !aligned(alphaA, 4) || !aligned(alphaB, 4) || !aligned(status, 4) || (ldd * (out_dtype == NVFP4_OUT_DTYPE_BF16 ? 2 : 4)) % 16)
    return NVFP4_ERR_ALIGN;
  return launch_status(nvfp4::grouped_gemm_launch(A, sA, alphaA, B, sB, alphaB, offsets, E, T, N, K, D, out_dtype, ldd,
                                                  status, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_gemm_grouped_wgrad(const uint8_t* A, const uint8_t* sA, const float* alphaA, const uint8_t* B,
                                        const uint8_t* sB, const float* alphaB, const int32_t* offsets, int64_t E,
                                        int64_t T, int64_t M, int64_t N, void* D, int out_dtype, int32_t* status,
                                        void* stream) {
  if (out_dtype != NVFP4_OUT_DTYPE_BF16 && out_dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  const nvfp4_status_t chk = check_groups(offsets, E, T);
  if (chk != NVFP4_OK) return chk;
  if (M <= 0 || N <= 0 || M % 128 || N % 128) return NVFP4_ERR_SHAPE;
  if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  const int64_t kblocks = nvfp4::grouped_capacity(T, E, 64) / 64;
  if (E * M >= (int64_t(1) << 31) || E * (M / 128) * (N / 128) >= (int64_t(1) << 31) ||
      (M / 128) * kblocks >= (int64_t(1) << 29) || (N / 128) * kblocks >= (int64_t(1) << 29))
    return NVFP4_ERR_SHAPE;
  if (!D || (T && (!A || !sA || !alphaA || !B || !sB || !alphaB))) return NVFP4_ERR_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 16) || !aligned(sB, 16) || !aligned(D, 16) ||
      !aligned(alphaA, 4) || !aligned(alphaB, 4) || !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  return launch_status(nvfp4::grouped_wgrad_launch(A, sA, alphaA, B, sB, alphaB, offsets, E, T, M, N, D, out_dtype,
                                                   status, static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_lora_workspace_size(int64_t T, int64_t K, int64_t N, int64_t r, int64_t n, int backward) {
  return (T < 0 || K < 1 || N < 1 || r < 1 || n < 1) ? 0 : nvfp4::lora_workspace_bytes(T, K, N, r, n, backward != 0);
}

nvfp4_status_t nvfp4_lora_apply(const void* x, int64_t ldx, const void* A, const void* B, const float* scaling,
                                const int32_t* ids, int64_t T, int64_t K, int64_t N, int64_t r, int64_t n,
                                const void* y, int64_t ldy, void* out, int64_t ldo, float* h, void* workspace,
                                size_t workspace_bytes, int32_t* status, void* stream) {
  nvfp4_status_t chk = check_lora(A, B, scaling, ids, T, K, N, r, n);
  if (chk != NVFP4_OK) return chk;
  if (T == 0) return NVFP4_OK;
  if ((chk = check_rows(x, ldx, K)) != NVFP4_OK || (chk = check_rows(out, ldo, N)) != NVFP4_OK) return chk;
  if (y && (chk = check_rows(y, ldy, N)) != NVFP4_OK) return chk;
  if (!aligned(h, 16) || !aligned(status, 4)) return NVFP4_ERR_ALIGN;
  if (!workspace || workspace_bytes < nvfp4::lora_workspace_bytes(T, K, N, r, n, false) || !aligned(workspace, 16))
    return NVFP4_ERR_WORKSPACE;
  nvfp4::LoraArgs l{};
  l.x = static_cast<const __nv_bfloat16*>(x);
  l.ldx = ldx;
  l.A = static_cast<const __nv_bfloat16*>(A);
  l.B = static_cast<const __nv_bfloat16*>(B);
  l.scaling = scaling;
  l.ids = ids;
  l.T = T;
  l.K = K;
  l.N = N;
  l.r = r;
  l.n = n;
  l.in = static_cast<const __nv_bfloat16*>(y);
  l.ldi = ldy;
  l.out = static_cast<__nv_bfloat16*>(out);
  l.ldo = ldo;
  l.h = h;
  l.status = status;
  return launch_status(nvfp4::lora_forward_launch(l, workspace, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_lora_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* h,
                                   const void* A, const void* B, const float* scaling, const int32_t* ids, int64_t T,
                                   int64_t K, int64_t N, int64_t r, int64_t n, const void* dx_in, int64_t ld_in, void* dx,
                                   int64_t lddx, void* dA, void* dB, int out_dtype, void* workspace,
                                   size_t workspace_bytes, int32_t* status, void* stream) {
  if (out_dtype != NVFP4_OUT_DTYPE_BF16 && out_dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  nvfp4_status_t chk = check_lora(A, B, scaling, ids, T, K, N, r, n);
  if (chk != NVFP4_OK) return chk;
  if (!dx && !dA && !dB) return NVFP4_ERR_ARG;
  if (T) {
    if ((chk = check_rows(dy, lddy, N)) != NVFP4_OK) return chk;
    if (dx && (chk = check_rows(dx, lddx, K)) != NVFP4_OK) return chk;
    if (dx && dx_in && (chk = check_rows(dx_in, ld_in, K)) != NVFP4_OK) return chk;
    if (dA && (chk = check_rows(x, ldx, K)) != NVFP4_OK) return chk;
    if (dB && !h) return NVFP4_ERR_ARG;
  }
  if (!aligned(h, 16) || !aligned(dA, 16) || !aligned(dB, 16) || !aligned(status, 4)) return NVFP4_ERR_ALIGN;
  if (T && (!workspace || workspace_bytes < nvfp4::lora_workspace_bytes(T, K, N, r, n, true) || !aligned(workspace, 16)))
    return NVFP4_ERR_WORKSPACE;
  if (T && dx && (dA || dB) && (dx == x || dx == dy)) return NVFP4_ERR_ARG;   // written before dA and dB read them
  nvfp4::LoraArgs l{};
  l.dy = static_cast<const __nv_bfloat16*>(dy);
  l.lddy = lddy;
  l.x = static_cast<const __nv_bfloat16*>(x);
  l.ldx = ldx;
  l.h = const_cast<float*>(h);
  l.A = static_cast<const __nv_bfloat16*>(A);
  l.B = static_cast<const __nv_bfloat16*>(B);
  l.scaling = scaling;
  l.ids = ids;
  l.T = T;
  l.K = K;
  l.N = N;
  l.r = r;
  l.n = n;
  l.in = dx ? static_cast<const __nv_bfloat16*>(dx_in) : nullptr;
  l.ldi = ld_in;
  l.out = static_cast<__nv_bfloat16*>(dx);
  l.ldo = lddx;
  l.dA = dA;
  l.dB = dB;
  l.fp32 = out_dtype == NVFP4_OUT_DTYPE_FP32;
  l.status = status;
  return launch_status(nvfp4::lora_backward_launch(l, workspace, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_route(const void* logits, int64_t ldl, int dtype, const float* bias, int64_t T, int64_t E, int64_t k,
                           int64_t groups, int64_t groups_kept, int score, uint32_t flags, float scale, int32_t* ids,
                           float* weights, int32_t* status, void* stream) {
  const nvfp4_status_t chk = check_route(logits, ldl, dtype, T, E, k, score, flags);
  if (chk != NVFP4_OK) return chk;
  if (groups < 1 || groups > 32 || E % groups || groups_kept < 1 || groups_kept > groups || k > groups_kept * (E / groups))
    return NVFP4_ERR_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!ids || !weights) return NVFP4_ERR_ARG;
  if (!aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(status, 4)) return NVFP4_ERR_ALIGN;
  const nvfp4::RouteArgs a{logits, ldl, bias, T, E, k, groups, groups_kept, score, flags, scale,
                           dtype == NVFP4_OUT_DTYPE_FP32, ids, weights, status};
  return launch_status(nvfp4::route_launch(a, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_route_backward(const float* dweights, const int32_t* ids, const void* logits, int64_t ldl, int dtype,
                                    int64_t T, int64_t E, int64_t k, int score, uint32_t flags, float scale, void* dlogits,
                                    int64_t ldd, int32_t* status, void* stream) {
  const nvfp4_status_t chk = check_route(logits, ldl, dtype, T, E, k, score, flags);
  if (chk != NVFP4_OK) return chk;
  if (ldd < E) return NVFP4_ERR_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!dweights || !ids || !dlogits) return NVFP4_ERR_ARG;
  if (dlogits == logits && ldd != ldl) return NVFP4_ERR_ARG;   // in place only row by row
  if (!aligned(dweights, 4) || !aligned(ids, 4) || !aligned(dlogits, dtype == NVFP4_OUT_DTYPE_BF16 ? 2 : 4) ||
      !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4::RouteArgs a{logits, ldl, nullptr, T, E, k, 1, 1, score, flags, scale,
                           dtype == NVFP4_OUT_DTYPE_FP32, const_cast<int32_t*>(ids), nullptr, status};
  return launch_status(nvfp4::route_backward_launch(a, dweights, dlogits, ldd, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_dispatch(const void* x, int64_t ldx, const int32_t* ids, int64_t T, int64_t k, int64_t E, int64_t C,
                              void* xs, int64_t ldxs, int32_t* offsets, int32_t* rows, int32_t* status, void* stream) {
  if (E < 1 || E > nvfp4::kMaxGroups) return NVFP4_ERR_SHAPE;
  nvfp4_status_t chk = check_pairs(rows, nullptr, T, k, x || xs ? C : 8, T * k, status);
  if (chk != NVFP4_OK) return chk;
  if (!offsets || (T && (!ids || !rows || !x != !xs))) return NVFP4_ERR_ARG;
  if (!aligned(offsets, 4) || !aligned(ids, 4)) return NVFP4_ERR_ALIGN;
  if (T && x && ((chk = check_rows(x, ldx, C)) != NVFP4_OK || (chk = check_rows(xs, ldxs, C)) != NVFP4_OK)) return chk;
  if (x && x == xs) return NVFP4_ERR_ARG;
  nvfp4::RowArgs a{};
  a.in = T ? static_cast<const __nv_bfloat16*>(x) : nullptr;
  a.ldi = ldx;
  a.rows = rows;
  a.T = T;
  a.k = k;
  a.C = C;
  a.R = T * k;
  a.out = static_cast<__nv_bfloat16*>(xs);
  a.ldo = ldxs;
  a.status = status;
  return launch_status(nvfp4::dispatch_launch(a, ids, E, offsets, rows, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_combine(const void* y, int64_t ldy, int64_t R, const int32_t* rows, const float* weights, int64_t T,
                             int64_t k, int64_t C, const void* residual, int64_t ldr, void* out, int64_t ldo,
                             int32_t* status, void* stream) {
  nvfp4_status_t chk = check_pairs(rows, weights, T, k, C, R, status);
  if (chk != NVFP4_OK) return chk;
  if (T == 0) return NVFP4_OK;
  if (R && (chk = check_rows(y, ldy, C)) != NVFP4_OK) return chk;
  if ((chk = check_rows(out, ldo, C)) != NVFP4_OK) return chk;
  if (residual && (chk = check_rows(residual, ldr, C)) != NVFP4_OK) return chk;
  if (out == y || (out == residual && ldr != ldo)) return NVFP4_ERR_ARG;
  nvfp4::RowArgs a{};
  a.in = static_cast<const __nv_bfloat16*>(residual);
  a.ldi = ldr;
  a.y = static_cast<const __nv_bfloat16*>(y);
  a.ldy = ldy;
  a.rows = rows;
  a.weights = weights;
  a.T = T;
  a.k = k;
  a.C = C;
  a.R = R;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.ldo = ldo;
  a.status = status;
  return launch_status(nvfp4::combine_launch(a, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_combine_backward(const void* dout, int64_t lddo, const void* y, int64_t ldy, int64_t R,
                                      const int32_t* rows, const float* weights, int64_t T, int64_t k, int64_t C, void* dy,
                                      int64_t lddy, float* dweights, int32_t* status, void* stream) {
  nvfp4_status_t chk = check_pairs(rows, weights, T, k, C, R, status);
  if (chk != NVFP4_OK) return chk;
  if (!dy && !dweights) return NVFP4_ERR_ARG;
  if (T == 0) return NVFP4_OK;
  if ((chk = check_rows(dout, lddo, C)) != NVFP4_OK) return chk;
  if (R && dweights && (chk = check_rows(y, ldy, C)) != NVFP4_OK) return chk;
  if (R && dy && (chk = check_rows(dy, lddy, C)) != NVFP4_OK) return chk;
  if (!aligned(dweights, 4)) return NVFP4_ERR_ALIGN;
  if (dy && (dy == dout || (dweights && dy == y))) return NVFP4_ERR_ARG;
  nvfp4::RowArgs a{};
  a.in = static_cast<const __nv_bfloat16*>(dout);
  a.ldi = lddo;
  a.y = static_cast<const __nv_bfloat16*>(y);
  a.ldy = ldy;
  a.rows = rows;
  a.weights = weights;
  a.T = T;
  a.k = k;
  a.C = C;
  a.R = R;
  a.out = static_cast<__nv_bfloat16*>(dy);
  a.ldo = lddy;
  a.dweights = dweights;
  a.status = status;
  return launch_status(nvfp4::combine_backward_launch(a, static_cast<cudaStream_t>(stream)));
}

nvfp4_status_t nvfp4_gemv(const void* x, int64_t ldx, const int32_t* ids, int64_t P, int64_t rep, const uint8_t* W,
                          const uint8_t* sW, const float* alphaW, int64_t E, int64_t N, int64_t K, void* out, int out_dtype,
                          int64_t ldo, int32_t* status, void* stream) {
  if (out_dtype != NVFP4_OUT_DTYPE_BF16 && out_dtype != NVFP4_OUT_DTYPE_FP32) return NVFP4_ERR_ARG;
  if (P < 0 || P > 1024 || rep < 1 || rep > 1024 || E < 1 || E > nvfp4::kMaxGroups || (!ids && E != 1)) return NVFP4_ERR_SHAPE;
  if (N <= 0 || K <= 0 || N % 128 || K % 64 || ldo < N || N > (int64_t(1) << 25) || K >= kMost) return NVFP4_ERR_SHAPE;
  if (P == 0) return NVFP4_OK;
  if (!W || !sW || !alphaW || !out) return NVFP4_ERR_ARG;
  const nvfp4_status_t chk = check_rows(x, ldx, K);
  if (chk != NVFP4_OK) return chk;
  if (!aligned(W, 16) || !aligned(sW, 16) || !aligned(alphaW, 4) || !aligned(ids, 4) || !aligned(status, 4) ||
      !aligned(out, out_dtype == NVFP4_OUT_DTYPE_BF16 ? 2 : 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4::GemvArgs a{static_cast<const __nv_bfloat16*>(x), ldx, ids, P, rep, W, sW, alphaW, E, N, K, out, ldo,
                          out_dtype == NVFP4_OUT_DTYPE_FP32, status};
  return launch_status(nvfp4::gemv_launch(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
