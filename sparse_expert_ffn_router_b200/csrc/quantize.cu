// Rows of activations as int8 with one fp32 scale per row, the left operand of the int8 products
// (gemm_i8.cu):
//
//   top = max_k |x[k]|,  s = fl32(top / 127),  q[k] = the integer nearest to x[k] / s, halves to even
//
// q is the rounding of the exact quotient, not of a rounded one: h = the integer nearest to
// x * fl(1 / s) (one multiply-add with 1.5 * 2^23, whose rounding is to integers) is within one of it
// (|x / s| <= 127, so the product is off by less than 127 * 2^-22), and the remainder r = x - h s has
// no rounding error in fp32 (it is a multiple of the smaller of the two ulps and at most about s / 2):
// where |r| < s / 2 h is the answer; otherwise comparing 2 |r| with s settles it, ties included.  The
// second case is rare, so a thread looks at the largest |r| of its 16 values first.  The result does not
// depend on how a division is carried out.
//
// A row whose s would be below 2^-126 (all zeros, or nothing above 127 * 2^-126) gets s = 1 and
// zeros.  A row that holds a NaN or an infinity gets s = NaN and zeros: every product with it is
// then NaN.
//
// Bound by memory: a row is read once, kept in registers while its maximum is formed, and written
// once (3 bytes per bf16 element); the next row is on its way meanwhile.  Each thread owns units of 16 elements (two or four 16-byte
// loads, one 16-byte store).  Measured (B200): 16384 x 16384 bf16 142 us = 5.7 TB/s, fp32 206 us = 6.5 TB/s;
// 4096 x 4096 bf16 14.5 us = 3.5 TB/s, launch and latency among it (21 us with the comparison made for every
// value).
#include <algorithm>

#include "common.cuh"

namespace colibri {
namespace {

constexpr int kQThreads = 256;

template <typename T>
struct Unit16 {  // 16 consecutive elements of a row
  uint4 v[sizeof(T)];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ float get(int i) const;
};
template <>
__device__ __forceinline__ float Unit16<__nv_bfloat16>::get(int i) const {
  const uint4& q = v[i >> 3];
  const int j = (i >> 1) & 3;
  const uint32_t w = j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}
template <>
__device__ __forceinline__ float Unit16<float>::get(int i) const {
  const uint4& q = v[i >> 2];
  const int j = i & 3;
  return __uint_as_float(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w);
}

// Largest magnitude as the bits of a non-negative float: their order as integers is the order of
// the values, and infinities and NaNs come out above every finite value.
__device__ __forceinline__ uint32_t unit_top(const Unit16<__nv_bfloat16>& u) {
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u.v[0].x));
  const uint32_t w[7] = {u.v[0].y, u.v[0].z, u.v[0].w, u.v[1].x, u.v[1].y, u.v[1].z, u.v[1].w};
#pragma unroll
  for (int i = 0; i < 7; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
  return max((b & 0x7fffu) << 16, b & 0x7fff0000u);
}
__device__ __forceinline__ uint32_t unit_top(const Unit16<float>& u) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(u.get(i)) & 0x7fffffffu);
  return m;
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum with it is rounded to an integer, in its low bits

// The 16 integers as bytes.
template <typename T>
__device__ __forceinline__ uint4 unit_quantize(const Unit16<T>& u, float s, float inv) {
  uint32_t b[16];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float h = fmaf(u.get(i), inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(kMagic - h, s, u.get(i))));
    b[i] = __float_as_uint(h);
  }
  if (2.f * far >= s) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float h = __uint_as_float(b[i]) - kMagic, r = fmaf(-h, s, u.get(i)), r2 = 2.f * fabsf(r);
      if (r2 > s || (r2 == s && ((int)h & 1))) b[i] = __float_as_uint(h + copysignf(1.f, r) + kMagic);
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040), __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// TPR threads per row, each with up to kQUnits units in registers (a longer row is read twice)
template <typename T, int TPR, int kQUnits>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 ? 3 : 2) quantize_rows_kernel(const T* __restrict__ x, int rows, int units,
                                                                  int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
                                                                  float* __restrict__ scale,
                                                                  const int32_t* __restrict__ dst, int k) {
  pdl_trigger();
  pdl_wait();
  constexpr int kRows = kQThreads / TPR;
  __shared__ uint32_t part[kQThreads / 32];
  const int t = threadIdx.x % TPR;
  constexpr bool kAhead = kQUnits <= 2;  // the next row is loaded while this one is rounded
  const int64_t step = (int64_t)gridDim.x * kRows;
  Unit16<T> next[kAhead ? kQUnits : 1];
  auto fetch = [&](Unit16<T>* v, int64_t r) {
    const T* src = x + (r < rows ? r : 0) * ldx;
#pragma unroll
    for (int i = 0; i < kQUnits; ++i)
      if (r < rows && t + i * TPR < units) v[i].load(src + (size_t)(t + i * TPR) * 16);
  };
  if (kAhead) fetch(next, (int64_t)blockIdx.x * kRows + threadIdx.x / TPR);
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += step) {
    const int64_t r = r0 + threadIdx.x / TPR;
    const bool live = r < rows;
    const T* src = x + (live ? r : 0) * ldx;
    Unit16<T> u[kQUnits];
    uint32_t top = 0;
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < kQUnits; ++i) u[i] = next[kAhead ? i : 0];
      fetch(next, r + step);
    } else {
      fetch(u, r);
    }
#pragma unroll
    for (int i = 0; i < kQUnits; ++i)
      if (live && t + i * TPR < units) top = max(top, unit_top(u[i]));
    for (int c = t + kQUnits * TPR; live && c < units; c += TPR) {  // a row longer than the registers hold
      Unit16<T> more;
      more.load(src + (size_t)c * 16);
      top = max(top, unit_top(more));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (TPR > 32) {
      __syncthreads();  // the previous row's readers are done
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TPR / 32; ++i) top = max(top, part[threadIdx.x / TPR * (TPR / 32) + i]);
    }
    const bool finite = top < 0x7f800000u;
    float s = __fdiv_rn(__uint_as_float(top), 127.f);
    bool zero = !finite;
    if (finite && s < 1.17549435e-38f) {  // 2^-126
      s = 1.f;
      zero = true;
    }
    if (!finite) s = __uint_as_float(0x7fc00000u);
    if (!live) continue;
    const float inv = 1.f / s;
    // to row r itself, or to the k rows it is grouped into
    auto put = [&](int c, const Unit16<T>& v) {
      const uint4 w = zero ? make_uint4(0, 0, 0, 0) : unit_quantize(v, s, inv);
      if (!dst) {
        reinterpret_cast<uint4*>(q + r * ldq)[c] = w;
        if (c == 0) scale[r] = s;
        return;
      }
#pragma unroll 1
      for (int j = 0; j < k; ++j) {
        const int64_t to = dst[r * k + j];
        reinterpret_cast<uint4*>(q + to * ldq)[c] = w;
        if (c == 0) scale[to] = s;
      }
    };
#pragma unroll
    for (int i = 0; i < kQUnits; ++i)
      if (t + i * TPR < units) put(t + i * TPR, u[i]);
    for (int c = t + kQUnits * TPR; c < units; c += TPR) {
      Unit16<T> more;
      more.load(src + (size_t)c * 16);
      put(c, more);
    }
  }
}

template <typename T, int TPR, int kQUnits>
cudaError_t launch_q(const T* x, int rows, int units, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                     const int32_t* dst, int k, int sms, cudaStream_t s) {
  constexpr int kRows = kQThreads / TPR;
  // rows loaded ahead: the CTAs that fit on the GPU at once go round (else a CTA takes few rows)
  const int most = kQUnits <= 2 ? sms * (sizeof(T) == 2 ? 3 : 2) : sms * 64;
  const int grid = std::min((rows + kRows - 1) / kRows, most);
  return launch_kernel(quantize_rows_kernel<T, TPR, kQUnits>, dim3(grid), dim3(kQThreads), 0, s, 1, x, rows, units, ldx,
                       q, ldq, scale, dst, k);
}

// The fewest threads per row that hold it in two units each, so that the next row's two fit beside them
// (4096 x 4096 bf16: 16.3 us with four units and no row ahead, 19.3 with four and a row ahead, which
// spills); longer rows four units on 256 threads.
template <typename T>
cudaError_t launch_rows(const T* x, int rows, int cols, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                        const int32_t* dst, int k, int sms, cudaStream_t s) {
  const int units = cols / 16;
  if (units <= 32) return launch_q<T, 32, 1>(x, rows, units, ldx, q, ldq, scale, dst, k, sms, s);
  if (units <= 64) return launch_q<T, 32, 2>(x, rows, units, ldx, q, ldq, scale, dst, k, sms, s);
  if (units <= 128) return launch_q<T, 64, 2>(x, rows, units, ldx, q, ldq, scale, dst, k, sms, s);
  if (units <= 256) return launch_q<T, 128, 2>(x, rows, units, ldx, q, ldq, scale, dst, k, sms, s);
  if (units <= 512) return launch_q<T, 256, 2>(x, rows, units, ldx, q, ldq, scale, dst, k, sms, s);
  return launch_q<T, 256, 4>(x, rows, units, ldx, q, ldq, scale, dst, k, sms, s);
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, int act, int rows, int cols, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* scale, cudaStream_t s, const int32_t* dst, int k) {
  if (rows <= 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (act == COLIBRI_BF16) return launch_rows((const __nv_bfloat16*)x, rows, cols, ldx, q, ldq, scale, dst, k, sms, s);
  return launch_rows((const float*)x, rows, cols, ldx, q, ldq, scale, dst, k, sms, s);
}

}  // namespace colibri
