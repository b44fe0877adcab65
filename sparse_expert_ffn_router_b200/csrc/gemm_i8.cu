// Products of int8 rows with int8 weights, one fp32 scale per row and one per output channel:
//
//   plain:   y[r][n] = s_r t_n sum_k q[r][k] w[n][k]
//   SwiGLU:  g, u = the plain products with W1 and W3;  h[r][n] = silu(g) * u
//
// The rows may be grouped: rows [offsets[e], offsets[e+1]) meet the weights of expert e.  The sums
// over k are exact int32 (K <= 131056, so that K * 128 * 128 stays below 2^31); the conversion to
// fp32 and the two scales round once each, and the result once to its type.
#include <algorithm>

#include "common.cuh"

namespace colibri {
namespace {

constexpr int kTile = 64;       // rows and output columns of a tile
constexpr int kChunk = 64;      // bytes of k per step
constexpr int kPitch = kChunk + 4;

template <bool kSwiglu, typename Out>
__global__ void __launch_bounds__(256) int_gemm_kernel(const IntGemmArgs a, Out* __restrict__ y) {
  __shared__ int s_row0, s_end, s_e;
  __shared__ __align__(16) int8_t sa[kTile * kPitch], sb[2][kTile * kPitch];
  if (threadIdx.x == 0) {
    int e = 0, tile = blockIdx.x, beg = 0, end = a.rows;
    if (a.offsets) {
      int prev = 0;
      e = -1;
      for (int g = 0; g < a.E; ++g) {
        const int b = min(max(a.offsets[g], prev), a.rows), n = min(max(a.offsets[g + 1], b), a.rows);
        prev = n;
        const int mt = (n - b + kTile - 1) / kTile;
        if (tile < mt) {
          e = g;
          beg = b;
          end = n;
          break;
        }
        tile -= mt;
      }
    }
    s_e = e;
    s_row0 = beg + tile * kTile;
    s_end = end;
  }
  __syncthreads();
  if (s_e < 0 || s_row0 >= s_end) return;
  const int row0 = s_row0, row_end = s_end, e = s_e, n0 = blockIdx.y * kTile;
  const int8_t* W = a.W + (size_t)e * a.w_stride;
  const float* ws = a.w_scale + (size_t)e * a.s_stride;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[2][4][4] = {};
  const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 16;
  for (int k0 = 0; k0 < a.K; k0 += kChunk) {
    const bool kin = k0 + lc < a.K;
    uint4 va = make_uint4(0, 0, 0, 0), vb[2] = {va, va};
    if (kin && row0 + lr < row_end) va = *reinterpret_cast<const uint4*>(a.A + (size_t)(row0 + lr) * a.lda + k0 + lc);
    if (kin && n0 + lr < a.N) {
      vb[0] = *reinterpret_cast<const uint4*>(W + (size_t)(n0 + lr) * a.ldw + k0 + lc);
      if (kSwiglu) vb[1] = *reinterpret_cast<const uint4*>(W + (size_t)(a.N + n0 + lr) * a.ldw + k0 + lc);
    }
    __syncthreads();
    auto put = [&](int8_t* dst, const uint4& v) {
      uint32_t* p = reinterpret_cast<uint32_t*>(dst + lr * kPitch + lc);
      p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    };
    put(sa, va);
    put(sb[0], vb[0]);
    if (kSwiglu) put(sb[1], vb[1]);
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kChunk; k += 4) {
      int av[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) av[i] = *reinterpret_cast<const int*>(sa + (ty + 16 * i) * kPitch + k);
#pragma unroll
      for (int m = 0; m < (kSwiglu ? 2 : 1); ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int bv = *reinterpret_cast<const int*>(sb[m] + (tx + 16 * j) * kPitch + k);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][i][j] = __dp4a(av[i], bv, acc[m][i][j]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + ty + 16 * i;
    if (r >= row_end) continue;
    const float sr = a.a_scale[r];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= a.N) continue;
      float v = (float)acc[0][i][j] * (sr * ws[n]);
      if (kSwiglu) v = silu_mul(v, (float)acc[1][i][j] * (sr * ws[a.N + n]));
      y[(size_t)r * a.ldy + n] = from_f32<Out>(v);
    }
  }
}

}  // namespace

cudaError_t launch_int_gemm(const IntGemmArgs& a, bool swiglu, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  const dim3 grid(a.rows / kTile + (a.offsets ? a.E : 1), (a.N + kTile - 1) / kTile), block(256);
  if (a.out_dtype == COLIBRI_BF16) {
    __nv_bfloat16* y = (__nv_bfloat16*)a.y;
    return swiglu ? launch_kernel(int_gemm_kernel<true, __nv_bfloat16>, grid, block, 0, s, 1, a, y)
                  : launch_kernel(int_gemm_kernel<false, __nv_bfloat16>, grid, block, 0, s, 1, a, y);
  }
  float* y = (float*)a.y;
  return swiglu ? launch_kernel(int_gemm_kernel<true, float>, grid, block, 0, s, 1, a, y)
                : launch_kernel(int_gemm_kernel<false, float>, grid, block, 0, s, 1, a, y);
}

}  // namespace colibri
