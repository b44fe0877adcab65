// The int8 product for at most 16 rows (gemm_i8.cu has the formula and the other sizes):
//
//   y[m][n] = s_m t_n sum_k q[m][k] w[n][k]
//
// Every weight byte is read once and meets a few rows, so the work is a stream over the weights and the
// bound is HBM (or, for a small product, the latency of one round trip).  Each CTA owns an equal share
// of the output columns, in groups of at most 32; the groups' chunks of 64 bytes of k, laid end to
// end, go to its 16 warps in equal runs.  A lane keeps 4 weight rows x 4 chunks of 16 bytes in flight in a
// ring of shared memory that the same lane fills (cp.async) and drains, so the ring needs no barrier and
// runs ahead into the next group.
// The products are mma.m16n8k32 on int8 with the weights as the 16-row operand and the rows as its 8
// columns: the order of k within an instruction is free, so 16 bytes of a weight row and of a token row
// feed two instructions as they are.  Sums are exact int32; the warps' parts meet in shared memory once
// per 8 groups (meeting after each group: 14336 x 4096 at 13 rows 15.7 us against 14.4).
// Measured (B200), weights in L2 (20 calls in a row) / from HBM (events around one call; an empty kernel
// takes 4.1 us there): 4096 x 4096 at one row 6.2 / 10.3 us (12.6 / 16.1 as tcgen05 tiles: 16 column tiles
// keep 32 SMs busy), at 16 rows 6.8 / 11.6 (12.6 / 16.3); 4096 x 14336 at one row 10.3 / 20.5, at 16
// 12.4 / 22.5 (24.6 as tiles); 1024 x 1024 4.2 / 7.4.  A bare read of 58 MB from HBM takes 18 us by the
// same events, 14 without the launch; this kernel is 2 to 4 us behind it, so that wide products leave it
// (launch_int_gemm).
#include <algorithm>

#include "common.cuh"

namespace colibri {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kDepth = 4;             // ring stages of a warp
constexpr int kStage = 4 * 512;       // bytes of a warp's stage: 4 rows of 16 bytes per lane
constexpr int kGroup = 32;            // columns (weight rows) of a group
constexpr int kPitch = kSkinnyRows + 2;
constexpr size_t kRing = (size_t)kWarps * kDepth * kStage;
constexpr int kBatch = 8;             // groups whose partial sums meet at a time
constexpr int kSlot = kGroup * kPitch;
// consecutive warps have consecutive runs, so the parts of (group i, warp w) go to slot i + w
constexpr size_t kSmem = kRing + (size_t)(kBatch + kWarps - 1) * kSlot * 4;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct SkinnyParams {
  const int8_t* A;
  int64_t lda;
  const float* a_scale;
  const int8_t* W;
  int64_t ldw;
  const float* w_scale;
  int64_t ldy;
  int M, K, chunks;
  // CTA i has each + (i < rest) columns, in groups[i < rest] groups of wide columns or, the first `wider`,
  // one more (divided on the host: the divisions cost the kernel a third of its 1.7 us before the first copy)
  int each, rest;
  int groups[2], wide[2], wider[2];
};

template <int NT, typename Out>
__global__ void __launch_bounds__(kThreads, 1) i8_skinny_kernel(const SkinnyParams p, Out* __restrict__ y) {
  extern __shared__ __align__(16) uint8_t smem[];
  int* red = reinterpret_cast<int*>(smem + kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_trigger();
  pdl_wait();

  // this CTA's columns and its groups of nearly equal width
  const int i0 = blockIdx.x;
  const bool more = i0 < p.rest;
  const int n0 = p.each * i0 + min(i0, p.rest), chunks = p.chunks;
  const int groups = more ? p.groups[1] : p.groups[0], wide = more ? p.wide[1] : p.wide[0],
            wider = more ? p.wider[1] : p.wider[0];
  auto first = [&](int i) { return n0 + wide * i + min(i, wider); };
  // the run of warp w over the chunks of the batch of groups that starts at group b: where it begins, and
  // the group of the batch that this lies in
  auto bound = [&](int b, int w) { return min(kBatch, groups - b) * chunks * w / kWarps; };
  auto group_of = [&](int b, int w) { return min(kBatch, groups - b) * w / kWarps; };

  // the stream: chunk `sc` of group `sb` + `si` is copied next; `left` chunks of its run in the batch
  const uint32_t ring = smem_u32(smem) + warp * (kDepth * kStage) + lane * 16;
  int sb = -kBatch, si = 0, sc = 0, left = 0;
  const int8_t* sp = nullptr;
  uint32_t live = 0;
  auto open = [&]() {
    while (left == 0) {
      sb += kBatch;
      if (sb >= groups) return;
      const int a = bound(sb, warp);
      left = bound(sb, warp + 1) - a;
      si = group_of(sb, warp);
      sc = a - si * chunks;
    }
    const int a = first(sb + si), b = first(sb + si + 1);
    sp = p.W + (int64_t)(a + g) * p.ldw + 16 * t;
    live = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) live |= (a + g + 8 * q < b ? 1u : 0u) << q;
  };
  auto issue = [&](uint32_t dst) {
    if (sb < groups) {
      if (sc * 64 + 16 * t < p.K) {  // the rest of a last chunk meets zeros of the rows
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (live >> q & 1u) cp_async16(dst + q * 512, sp + (int64_t)(8 * q) * p.ldw + (int64_t)sc * 64);
      }
      --left;
      if (++sc == chunks) {
        sc = 0;
        ++si;
      }
      if (left == 0 || sc == 0) open();
    }
    cp_async_commit();
  };
  open();
#pragma unroll
  for (int s = 0; s < kDepth; ++s) issue(ring + s * kStage);

  const int8_t* src[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) src[j] = g + 8 * j < p.M ? p.A + (g + 8 * j) * p.lda + 16 * t : nullptr;
  auto rows16 = [&](int j, int c) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (src[j] && c * 64 + 16 * t < p.K) v = __ldg(reinterpret_cast<const uint4*>(src[j] + (int64_t)c * 64));
    return v;
  };
  int slot = 0;
  for (int b = 0; b < groups; b += kBatch) {
    const int end = bound(b, warp + 1);
    int i = group_of(b, warp);
    for (int pos = bound(b, warp); pos < end; ++i) {
      const int ca = pos - i * chunks, cb = min(chunks, end - i * chunks);
      int acc[2][NT][4] = {};
      uint4 xn[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) xn[j] = rows16(j, ca);
      for (int c = ca; c < cb; ++c) {
        uint4 xb[NT];  // the rows' bytes of the next chunk are loaded while this one is multiplied
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          xb[j] = xn[j];
          if (c + 1 < cb) xn[j] = rows16(j, c + 1);
        }
        cp_async_wait<kDepth - 1>();
        uint4 w[4];
        const uint32_t from = ring + slot * kStage;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = lds16(from + q * 512);
        slot = slot + 1 == kDepth ? 0 : slot + 1;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_s8(acc[m][j], w[2 * m].x, w[2 * m + 1].x, w[2 * m].y, w[2 * m + 1].y, xb[j].x, xb[j].y);
            mma_s8(acc[m][j], w[2 * m].z, w[2 * m + 1].z, w[2 * m].w, w[2 * m + 1].w, xb[j].z, xb[j].w);
          }
        issue(from);  // the stage's values have been used: it may be filled again
      }
      // column 8 (2 m + h) + g of the group, rows 8 j + 2 t and the next
      int* mine = red + (i + warp) * kSlot;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<int2*>(mine + ((2 * m + h) * 8 + g) * kPitch + 8 * j + 2 * t) =
                make_int2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
      pos += cb - ca;
    }
    __syncthreads();
    const int nb = min(kBatch, groups - b);
    for (int i = 0; warp < p.M && i < nb; ++i) {  // warp = row, lane = column
      const int n = first(b + i) + lane;
      if (n >= first(b + i + 1)) continue;
      int s = 0, from = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {  // the warps whose runs have a part in the group
        const int to = bound(b, w + 1);
        if (max(from, i * chunks) < min(to, (i + 1) * chunks)) s += red[(i + w) * kSlot + lane * kPitch + warp];
        from = to;
      }
      y[warp * p.ldy + n] = from_f32<Out>(scaled(s, __ldg(p.a_scale + warp), __ldg(p.w_scale + n)));
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

}  // namespace

cudaError_t launch_int_skinny(const IntGemmArgs& a, int sms, cudaStream_t s) {
  const int ctas = std::min(sms, a.N);
  SkinnyParams p{a.A, a.lda, a.a_scale, a.W, a.ldw, a.w_scale, a.ldy, a.rows, a.K, (a.K + 63) / 64, a.N / ctas, a.N % ctas};
  for (int more = 0; more < 2; ++more) {
    const int cols = p.each + more;
    p.groups[more] = (cols + kGroup - 1) / kGroup;
    p.wide[more] = cols / p.groups[more];
    p.wider[more] = cols % p.groups[more];
  }
  const dim3 grid(ctas), block(kThreads);
  auto launch = [&](auto kern, auto* y) {
    const cudaError_t e2 = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    return e2 != cudaSuccess ? e2 : launch_kernel(kern, grid, block, kSmem, s, 1, p, y);
  };
  if (a.out_dtype == COLIBRI_BF16) {
    __nv_bfloat16* y = (__nv_bfloat16*)a.y;
    return a.rows <= 8 ? launch(i8_skinny_kernel<1, __nv_bfloat16>, y) : launch(i8_skinny_kernel<2, __nv_bfloat16>, y);
  }
  float* y = (float*)a.y;
  return a.rows <= 8 ? launch(i8_skinny_kernel<1, float>, y) : launch(i8_skinny_kernel<2, float>, y);
}

}  // namespace colibri
