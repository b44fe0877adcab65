// Entry points of the int8 products (include/colibri.h): quantise rows, dense product, products of
// rows grouped by expert.  No context and no allocation; arguments are checked here, before
// anything is launched.
#include <cstdarg>
#include <cstdio>

#include "common.cuh"

namespace colibri {
colibri_status report(colibri_ctx* ctx, colibri_status st, const char* msg);
}

using namespace colibri;

namespace {

colibri_status refuse(colibri_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report(nullptr, st, buf);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Buf {
  const char* name;
  const void* p;
};

// Every buffer non-NULL, 16-byte aligned and device memory of the current device.
template <int N>
colibri_status check_buffers(const Buf (&bufs)[N]) {
  for (const Buf& b : bufs)
    if (!b.p) return refuse(COLIBRI_ERR_INVALID_ARG, "%s is NULL", b.name);
  for (const Buf& b : bufs)
    if (!aligned16(b.p)) return refuse(COLIBRI_ERR_ALIGNMENT, "%s is not 16-byte aligned", b.name);
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return refuse(COLIBRI_ERR_CUDA, "cudaGetDevice failed");
  }
  for (const Buf& b : bufs) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, b.p) != cudaSuccess) {
      cudaGetLastError();
      return refuse(COLIBRI_ERR_INVALID_ARG, "%s is not device memory", b.name);
    }
    if (!((at.type == cudaMemoryTypeDevice && at.device == dev) || at.type == cudaMemoryTypeManaged))
      return refuse(COLIBRI_ERR_INVALID_ARG, "%s is not device memory of the current device", b.name);
  }
  return COLIBRI_OK;
}

colibri_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return COLIBRI_OK;
  cudaGetLastError();
  return refuse(COLIBRI_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// A leading dimension: at least `cols` elements, rows 16-byte aligned when `aligned`.
colibri_status check_ld(const char* name, int64_t ld, int64_t cols, int esize, bool aligned) {
  if (ld < cols || ld > kIntMaxLd)
    return refuse(COLIBRI_ERR_INVALID_ARG, "%s=%lld must be in [%lld, 2^31)", name, (long long)ld, (long long)cols);
  if (aligned && (ld * esize) % 16 != 0)
    return refuse(COLIBRI_ERR_ALIGNMENT, "%s=%lld: rows must start on 16-byte boundaries", name, (long long)ld);
  return COLIBRI_OK;
}

#define COLIBRI_CHECK(expr)                 \
  do {                                      \
    const colibri_status st_ = (expr);      \
    if (st_ != COLIBRI_OK) return st_;      \
  } while (0)

colibri_status check_sizes(int32_t rows, int32_t N, int32_t K, int32_t out_dtype) {
  if (out_dtype != COLIBRI_F32 && out_dtype != COLIBRI_BF16)
    return refuse(COLIBRI_ERR_UNSUPPORTED, "out_dtype must be COLIBRI_F32 or COLIBRI_BF16");
  if (rows < 0 || rows > kIntMaxRows) return refuse(COLIBRI_ERR_INVALID_ARG, "rows=%d outside [0, %d]", rows, kIntMaxRows);
  if (N < 1 || N > kIntMaxN) return refuse(COLIBRI_ERR_INVALID_ARG, "N=%d outside [1, %d]", N, kIntMaxN);
  if (K < 16 || K > kIntMaxK || K % 16 != 0)
    return refuse(COLIBRI_ERR_INVALID_ARG, "K=%d must be a multiple of 16 in [16, %d]", K, kIntMaxK);
  return COLIBRI_OK;
}

colibri_status experts(bool swiglu, const int8_t* A, int64_t lda, const float* a_scale, int32_t rows,
                       const int32_t* offsets, int32_t E, const int8_t* W, int64_t w_stride, const float* w_scale,
                       int64_t s_stride, int32_t N, int32_t K, void* y, int64_t ldy, int32_t out_dtype, void* stream) {
  COLIBRI_CHECK(check_sizes(rows, N, K, out_dtype));
  if (E < 1 || E > kMaxExperts) return refuse(COLIBRI_ERR_INVALID_ARG, "num_experts=%d outside [1, %d]", E, kMaxExperts);
  const int64_t cols = swiglu ? 2 * (int64_t)N : N;
  COLIBRI_CHECK(check_ld("lda", lda, K, 1, true));
  COLIBRI_CHECK(check_ld("ldy", ldy, N, out_dtype == COLIBRI_F32 ? 4 : 2, false));
  if (w_stride < cols * K || w_stride > kIntMaxStride)
    return refuse(COLIBRI_ERR_INVALID_ARG, "w_stride=%lld must be in [%lld, 2^38]", (long long)w_stride, (long long)(cols * K));
  if (w_stride % 16 != 0) return refuse(COLIBRI_ERR_ALIGNMENT, "w_stride must be a multiple of 16");
  if (s_stride < cols || s_stride > kIntMaxStride)
    return refuse(COLIBRI_ERR_INVALID_ARG, "s_stride=%lld must be in [%lld, 2^38]", (long long)s_stride, (long long)cols);
  if (rows == 0) return COLIBRI_OK;
  COLIBRI_CHECK(check_buffers({Buf{"A", A}, Buf{"a_scale", a_scale}, Buf{"offsets", offsets}, Buf{"W", W},
                               Buf{"w_scale", w_scale}, Buf{"y", y}}));
  IntGemmArgs a{A, lda, a_scale, rows, offsets, E, W, w_stride, K, w_scale, s_stride, N, K, y, ldy, out_dtype, nullptr};
  return launched(launch_int_gemm(a, swiglu, reinterpret_cast<cudaStream_t>(stream)), "int8 expert product");
}

}  // namespace

extern "C" {

colibri_status colibri_quantize_rows(const void* x, int32_t act_dtype, int32_t rows, int32_t cols, int64_t ldx,
                                     int8_t* q, int64_t ldq, float* scale, void* stream) {
  if (act_dtype != COLIBRI_F32 && act_dtype != COLIBRI_BF16)
    return refuse(COLIBRI_ERR_UNSUPPORTED, "act_dtype must be COLIBRI_F32 or COLIBRI_BF16");
  COLIBRI_CHECK(check_sizes(rows, 1, cols, COLIBRI_F32));
  COLIBRI_CHECK(check_ld("ldx", ldx, cols, act_dtype == COLIBRI_F32 ? 4 : 2, true));
  COLIBRI_CHECK(check_ld("ldq", ldq, cols, 1, true));
  if (rows == 0) return COLIBRI_OK;
  COLIBRI_CHECK(check_buffers({Buf{"x", x}, Buf{"q", q}, Buf{"scale", scale}}));
  return launched(launch_quantize_rows(x, act_dtype, rows, cols, ldx, q, ldq, scale, reinterpret_cast<cudaStream_t>(stream)),
                  "quantize_rows");
}

colibri_status colibri_int_gemm(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* W, int64_t ldw,
                                const float* w_scale, int32_t M, int32_t N, int32_t K, void* y, int64_t ldy,
                                int32_t out_dtype, void* stream) {
  COLIBRI_CHECK(check_sizes(M, N, K, out_dtype));
  COLIBRI_CHECK(check_ld("lda", lda, K, 1, true));
  COLIBRI_CHECK(check_ld("ldw", ldw, K, 1, true));
  COLIBRI_CHECK(check_ld("ldy", ldy, N, out_dtype == COLIBRI_F32 ? 4 : 2, false));
  if (M == 0) return COLIBRI_OK;
  COLIBRI_CHECK(check_buffers({Buf{"A", A}, Buf{"a_scale", a_scale}, Buf{"W", W}, Buf{"w_scale", w_scale}, Buf{"y", y}}));
  IntGemmArgs a{A, lda, a_scale, M, nullptr, 1, W, 0, ldw, w_scale, 0, N, K, y, ldy, out_dtype, nullptr};
  return launched(launch_int_gemm(a, false, reinterpret_cast<cudaStream_t>(stream)), "int8 product");
}

colibri_status colibri_int_gemm_experts(const int8_t* A, int64_t lda, const float* a_scale, int32_t rows,
                                        const int32_t* offsets, int32_t num_experts, const int8_t* W, int64_t w_stride,
                                        const float* w_scale, int64_t s_stride, int32_t N, int32_t K, void* y,
                                        int64_t ldy, int32_t out_dtype, void* stream) {
  return experts(false, A, lda, a_scale, rows, offsets, num_experts, W, w_stride, w_scale, s_stride, N, K, y, ldy,
                 out_dtype, stream);
}

colibri_status colibri_int_swiglu_experts(const int8_t* A, int64_t lda, const float* a_scale, int32_t rows,
                                          const int32_t* offsets, int32_t num_experts, const int8_t* W,
                                          int64_t w_stride, const float* w_scale, int64_t s_stride, int32_t N,
                                          int32_t K, void* h, int64_t ldh, int32_t out_dtype, void* stream) {
  return experts(true, A, lda, a_scale, rows, offsets, num_experts, W, w_stride, w_scale, s_stride, N, K, h, ldh,
                 out_dtype, stream);
}

colibri_status colibri_int_check(void* stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return refuse(COLIBRI_ERR_CUDA, "stream synchronize failed");
  }
  uint32_t word = 0;
  const cudaError_t e = int_gemm_take_error(&word, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return launched(e, "reading the error word");
  if (word) return refuse(COLIBRI_ERR_TIMEOUT, "a bounded device wait of an int8 product gave up");
  return COLIBRI_OK;
}

}  // extern "C"
