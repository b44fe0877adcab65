// Products of int8 rows with int8 weights, one fp32 scale per row and one per output channel:
//
//   plain:   y[r][n] = s_r t_n sum_k q[r][k] w[n][k]
//   SwiGLU:  g, u = the plain products with W1 and W3;  h[r][n] = silu(g) * u
//
// The rows may be grouped: rows [offsets[e], offsets[e+1]) meet the weights of expert e.  The sums
// over k are exact int32 (K <= 131056, so that K * 128 * 128 stays below 2^31); the conversion to
// fp32 and the two scales round once each (with a scale outside 2^-63..2^63 once in all, from 64 bits),
// and the result once to its type.
//
// i8_pair_kernel: clusters of two CTAs (tcgen05 cta_group::2, kind::i8), persistent, one pair per two
// SMs, 352 threads per CTA:
//   warp 0      TMA producer: this CTA's 128 rows of A and 128 of the 256 weight rows of the tile
//               (SwiGLU: the leader W1, the peer W3), 128 bytes of k per stage, into a ring of 32 KB
//               stages; both CTAs' copies count on the leader's barrier.
//   warp 1      the leader issues the M = 256, N = 256, K = 32 MMAs, four per stage, into one of two
//               accumulators (128 rows x 256 int32 columns of TMEM in each CTA).
//   warps 2-9   epilogue: TMEM -> registers, scales, SwiGLU, stores; it overlaps the next tile's MMAs.
//   warp 10     planner: finds the tiles ahead of the other roles and fetches their scales (done by the
//               roles themselves this cost 1.5 us between two tiles of MMAs and 3 us per epilogue)
// A group's last m-tile of at most 128 rows runs with the operands swapped (weights the M side, its
// rows rounded up to 32 the N side), so that a group of a few rows costs the stream of its weights
// and little else; with at most 32 rows a stage holds two k blocks of weights (one: skewed experts 154 -> 163 us).  For SwiGLU a swapped
// tile's 128 weight rows per CTA are 4 x (16 of W1, the same 16 of W3), so that gate and up of a
// column meet in one warp; that needs N to be a multiple of 16, other N take the full tile.
// Tiles are numbered group-major, then n-tile, then m-tile fastest, so that the pairs running together
// share weight tiles through L2; groups of a single m-tile (streams of weights) are interleaved with
// the others in proportion.  Pair i takes tiles i, i + pairs, ...
//
// The producer's and the MMA warp's loops run converged and one elected lane issues (under a branch on the
// lane number the compiler moves every operand to the uniform registers in turn: 0.1 us per copy, 0.05 us
// per MMA, so that a stage took 0.31 us whatever it held).
//
// What bounds a full tile: the MMAs.  A stage of 64 KB per pair feeds 512 cycles of them (8192 multiply-adds
// per cycle and SM); with all pairs at work it takes 0.36 us at the 1.6 GHz that the power limit leaves, the
// tensor pipe 89 % busy (82 % of the launch: 12.1 rounds of tiles take 13).  160 KB in flight per SM are
// just enough (4 stages: 157 us where 5 take 150; 3: 179).  Measured (B200): 4096 x 14336 x 4096 145 to 155 us,
// one call and 20 in a row = 3.1 to 3.3 POP/s; 8192 rows of 8 experts times [2 x 14336, 4096] with SwiGLU 630 to
// 660 us = 2.9 to 3.05 POP/s (790 to 800 without a pause between calls, the clock lower still); 64 rows on 8
// experts (940 MB of weights) 143 us = 6.6 TB/s.
// With little k per tile the epilogue bounds it (1.9 us per 256 x 256 tile).
//
// i8_split_kernel: products of too few pair tiles to occupy the GPU.  Tiles of 128 x 128 (one CTA each,
// cta_group::1) whose k range is split over the S = 1, 2 or 4 CTAs of a cluster; the int32 partial
// sums, exact in any order, are exchanged through the cluster's shared memory (the idle ring), each
// CTA finishing 1 / S of the columns.  What bounds such a product is the feed of one SM's shared
// memory (about 100 GB/s measured, against 43 GB/s of HBM per SM), so the SMs left idle are worth more
// than the larger tile: 4096 x 4096 at 128 rows 12.5 us against 17.1 as pair tiles, 4096 x 14336 at 64 rows
// 16.7 against 33.9; 14336 x 4096 at 256 rows has 224 such tiles and stays with the pairs (18.7 us).
//
// Every wait is bounded (kWaitTimeoutNs); one that gives up sets the error word and ends all roles.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "common.cuh"

namespace colibri {
namespace {

// Set by a bounded wait that gave up, when the caller brings no word of its own.
__device__ uint32_t g_int_err;
// What a check found there on its way to the host: a word per check, in turn, since checks may run at once.
constexpr unsigned kTaken = 256;
__device__ uint32_t g_int_taken[kTaken];

// Reads and clears the error word in one step: a wait that gives up meanwhile stays for the next check.
__global__ void take_error_kernel(unsigned slot) {
  pdl_trigger();
  pdl_wait();
  g_int_taken[slot] = atomicExch(&g_int_err, 0u);
}

constexpr int kEpiWarps = 8;          // two per quarter of the TMEM lanes (one: fine-grained down 96 against 92 us)
constexpr int kEpiHalves = kEpiWarps / 4;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 96 + kEpiThreads;
constexpr int kPlans = 4;            // tiles the planner may be ahead
constexpr int kBM = 256;             // rows of a pair tile
constexpr int kBN = 256;             // weight rows of a pair tile
constexpr int kKB = 128;             // bytes of k per stage: one 128-byte swizzle atom
constexpr int kHalf = 128 * kKB;     // 16 KB: this CTA's A or B part of a stage
constexpr int kStage = 2 * kHalf;
constexpr int kStages = 5;
constexpr int kLightRows = 128;      // swapped tiles: at most 64 token rows per CTA
constexpr int kDenseRows = 32;       // swapped tiles with two k blocks per stage
constexpr int kTok = 16 * kKB;       // a 16-row box of token rows
constexpr int kTmemCols = 512;
constexpr int kOutRow = 128;         // bytes of an output row that the epilogue gathers before it stores them
constexpr int kOutPitch = kOutRow + 16;

struct alignas(64) PairParams {
  CUtensorMap mapA, mapA16, mapA32, mapA64;  // rows, in boxes of 128, 16, 32 and 64
  CUtensorMap mapB;                          // weights, 128-row boxes
  CUtensorMap mapB16;                        // SwiGLU: boxes of 4 x (16 W1 rows, the same 16 W3 rows)
  const int32_t* offsets;
  const float* a_scale;
  const float* w_scale;
  int64_t s_stride;
  void* y;
  int64_t ldy;
  uint32_t* err;
  int E, rows, N;
  int n_tiles, num_kb;
  int light_rows;  // m-tiles with at most this many rows run swapped (0: none)
  bool vec;        // rows of y are 16-byte aligned
};

struct Tile {
  int e, row0, row_end, n0, mtiles;
};

struct PairSmem {
  static constexpr bool kClasses = true;  // tiles of groups with one m-tile are interleaved with the others
  uint64_t full[kStages];   // used in the leader: both CTAs' copies
  uint64_t empty[kStages];  // per CTA: freed by the leader's multicast commit
  uint64_t tfull[2];        // per CTA: accumulator ready (multicast commit)
  uint64_t tempty[2];       // used in the leader: both CTAs' epilogue warps
  uint64_t ifull[kPlans];   // tile found
  uint64_t sfull[kPlans];   // its scales are there
  uint64_t pfree[kPlans];   // producer, MMA thread (leader) and epilogue warps are done with it
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int32_t off[kMaxExperts + 1];
  int32_t mt[kMaxExperts + 1];  // m-tile prefix over all groups,
  int32_t hv[kMaxExperts + 1];  // over groups with two or more m-tiles,
  int32_t lt[kMaxExperts + 1];  // over groups with exactly one
  Tile tile[kPlans];
  alignas(16) float col[kPlans][kBN];  // column scales of the tile (SwiGLU: gate | up)
  alignas(16) float row[kPlans][128];  // row scales: of this CTA's rows, or of a swapped tile's
  int wide[kPlans];                    // some scale is wide (the others' tiles are spared the question per value)
  alignas(16) uint8_t out[kEpiWarps][32 * kOutPitch];
};
constexpr size_t kPairTok = (size_t)kStages * 2 * kTok;
constexpr size_t kPairSmem = (size_t)kStages * kStage + kPairTok + sizeof(PairSmem);
static_assert(kPairSmem <= 232448, "shared memory of one CTA");

// Group offsets (entry i counts as the largest of entries 0..i, within [0, rows]) and the m-tile
// prefixes for tiles of kRows rows; one full warp.
template <int kRows, typename Smem>
__device__ void schedule(Smem& m, const int32_t* offsets, int E, int rows) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kMaxExperts / 32;
  const int per = (E + 31) / 32, e0 = lane * per;  // this lane's groups
  int end[kPer];                                     // entry e0 + i + 1
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    end[i] = 0;
    if (i < per && e0 + i < E) end[i] = offsets ? min(max(offsets[e0 + i + 1], 0), rows) : rows;
  }
  int first = 0;
  if (lane == 0 && offsets) first = min(max(offsets[0], 0), rows);
  int top = first;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = max(top, end[i]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, top, o);
    if (lane >= o) top = max(top, v);
  }
  int begin = __shfl_up_sync(0xffffffffu, top, 1);  // where this lane's first group begins
  if (lane == 0) begin = first;
  int all = 0, heavy = 0;
  int at = begin;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i < per && e0 + i < E) {
      const int to = max(at, end[i]), mt = (to - at + kRows - 1) / kRows;
      end[i] = to;
      all += mt;
      heavy += mt >= 2 ? mt : 0;
      at = to;
    }
  }
  int ia = all, ih = heavy;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ih, o);
    if (lane >= o) {
      ia += x;
      ih += y;
    }
  }
  all = ia - all;
  heavy = ih - heavy;
  if (lane == 0) {
    m.off[0] = first;
    m.mt[0] = 0;
    if constexpr (Smem::kClasses) m.hv[0] = m.lt[0] = 0;
  }
  at = begin;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i < per && e0 + i < E) {
      const int mt = (end[i] - at + kRows - 1) / kRows;
      all += mt;
      heavy += mt >= 2 ? mt : 0;
      m.off[e0 + i + 1] = end[i];
      m.mt[e0 + i + 1] = all;
      if constexpr (Smem::kClasses) {
        m.hv[e0 + i + 1] = heavy;
        m.lt[e0 + i + 1] = all - heavy;  // a group has one m-tile, or is heavy, or is empty
      }
      at = end[i];
    }
  }
}

// largest e in [0, E) with pre[e] * n_tiles <= L
__device__ __forceinline__ int find_group(const int32_t* pre, int E, int n_tiles, int L) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] * n_tiles <= L) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ Tile pair_tile(const PairParams& p, const PairSmem& m, int L, int ncols) {
  const int nh = m.hv[p.E] * p.n_tiles, nl = m.lt[p.E] * p.n_tiles;
  const int32_t* pre = m.mt;
  int idx = L;
  if (nh > 0 && nl > 0) {
    const long long tot = (long long)nh + nl;
    const int b = (int)((long long)L * nl / tot);
    const bool light = (int)((long long)(L + 1) * nl / tot) > b;
    pre = light ? m.lt : m.hv;
    idx = light ? b : L - b;
  }
  Tile t;
  t.e = find_group(pre, p.E, p.n_tiles, idx);
  t.mtiles = m.mt[t.e + 1] - m.mt[t.e];
  const int r = idx - pre[t.e] * p.n_tiles, n = r / t.mtiles, mm = r - n * t.mtiles;
  t.row0 = m.off[t.e] + mm * kBM;
  t.row_end = m.off[t.e + 1];
  t.n0 = n * ncols;
  return t;
}

// Bounded wait that also gives up as soon as another role has aborted (kCluster: acquire at cluster
// scope, for barriers the other CTA of the pair arrives on).
template <bool kCluster = false>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  auto try_wait = [&]() { return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (try_wait()) return true;
  const unsigned long long t0 = global_ns();
  uint32_t n = 0;
  while (true) {
    if (try_wait()) return true;
    if ((++n & 255u) == 0) {
      if (*abort_flag) return false;
      if (global_ns() - t0 > kWaitTimeoutNs) return false;
    }
  }
}

template <typename Smem>
__device__ __forceinline__ void raise_abort(Smem& m, uint32_t* err) {
  *(volatile int*)&m.abort = 1;
  atomicOr(err, kErrWaitTimeout);
}

__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Arrival that publishes no memory: it frees an accumulator whose values are in registers.  With release
// semantics it waits for the epilogue's stores to global memory (1.1 us per tile, measured).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 32 lanes x 32 bits, 16 consecutive columns per thread, as integers
__device__ __forceinline__ void tmem_ld16i(uint32_t taddr, int (&v)[16]) {
  float f[16];
  tmem_ld16(taddr, f);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __float_as_int(f[i]);
}

// Two fp32 values per instruction: the epilogue is bound by the instructions it issues.
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void halves(const Pair& p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ Pair operator*(const Pair& a, const Pair& b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// silu(g) * u = g / (1 + 2^(-g log2 e)) * u.  The exponential is good to 2^-22 and the rounding of its
// argument, the reciprocal to 2^-23; what they flush (an exponential below 2^-126, a reciprocal of one
// above 2^126) does not show beside the 1, or is below 1e-36.
__device__ __forceinline__ Pair silu_mul(const Pair& g, const Pair& u) {
  float a, b;
  halves(g * pair_of(-1.44269504f, -1.44269504f), a, b);
  halves(pair_of(exp2_approx(a), exp2_approx(b)) + pair_of(1.f, 1.f), a, b);
  return g * pair_of(rcp_approx(a), rcp_approx(b)) * u;
}
__device__ __forceinline__ float silu_mul_fast(float g, float u) {
  return g * rcp_approx(1.f + exp2_approx(g * -1.44269504f)) * u;
}

// 16 values of this lane's row into the gathered block, at byte `at` of its 128.
template <typename Out>
__device__ __forceinline__ void gather16(uint8_t* block, int lane, int at, const float (&v)[16]) {
  uint4* d = reinterpret_cast<uint4*>(block + lane * kOutPitch + at);
  if constexpr (sizeof(Out) == 2) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                        __float_as_uint(v[4 * i + 3]));
  }
}

// One warp: the gathered block of 32 rows by 128 bytes to `dst` (row 0, first column); `rows` and `cols`
// of it exist.  Whole aligned rows go 8 lanes to a row, 128 contiguous bytes; others value by value,
// the lanes on consecutive columns.  (Stores from the registers, a lane per row, touch 32 lines per
// instruction: 3.3 us per 256 x 256 bf16 tile, 32 us where the rows are not aligned.)
template <typename Out>
__device__ __forceinline__ void store_block(Out* dst, int64_t ldy, const uint8_t* block, int rows, int cols, bool vec,
                                            int lane) {
  constexpr int kCols = kOutRow / (int)sizeof(Out);
  __syncwarp();
  const int n = min(rows, 32);
  if (vec && cols >= kCols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const uint4 v = *reinterpret_cast<const uint4*>(block + r * kOutPitch + (lane & 7) * 16);
      if (r < n) reinterpret_cast<uint4*>(dst + r * ldy)[lane & 7] = v;
    }
  } else {
    for (int c = lane; c < min(cols, kCols); c += 32)
#pragma unroll 8
      for (int r = 0; r < n; ++r) dst[r * ldy + c] = reinterpret_cast<const Out*>(block + r * kOutPitch)[c];
  }
  __syncwarp();
}

// The epilogue of a tile with a wide scale, apart from the others': value by value, a lane per row, or in a swapped
// tile per column.
template <bool kSwiglu, typename Out>
__device__ __noinline__ void wide_tile(const PairParams& p, PairSmem& m, int slot, uint32_t tb, int rank, int q, int half,
                                       int lane) {
  const Tile t = m.tile[slot];
  const int trows = t.row_end - t.row0;
  const float *col = m.col[slot], *rs = m.row[slot];
  Out* const y = static_cast<Out*>(p.y);
  constexpr int kCols = kSwiglu ? kBN / 2 : kBN;
  const bool light = trows <= p.light_rows;
  // the accumulator's column c and lane are row c and column `oc` of a swapped tile, column c and row `row` of
  // a full one
  const int c0 = kSwiglu ? 64 * rank + 16 * q + (lane & 15) : 128 * rank + 32 * q + lane;
  const int oc = t.n0 + c0, row = 128 * rank + 32 * q + lane;
  const int n = light ? trows : (128 * rank + 32 * q < trows ? min(kCols, p.N - t.n0) : 0);
  const bool gate = !kSwiglu || lane < 16;
  for (int c = 16 * half; c < n; c += 16 * kEpiHalves) {
    int v[16], u[16];
    tmem_ld16i(tb + c, v);
    tmem_ld16i(tb + (kSwiglu && !light ? kBN / 2 : 0) + c, u);
    tmem_ld_wait(v, u);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x;
      if (light) {
        const float tn = col[(gate ? 0 : kBN / 2) + c0];
        x = c + i < trows ? scaled(v[i], rs[c + i], tn) : 0.f;
        if (kSwiglu) x = silu_mul_fast(x, __shfl_down_sync(0xffffffffu, x, 16));
        if (gate && c + i < trows && oc < p.N) y[(int64_t)(t.row0 + c + i) * p.ldy + oc] = from_f32<Out>(x);
      } else {
        const float sr = rs[32 * q + lane];
        x = scaled(v[i], sr, col[c + i]);
        if (kSwiglu) x = silu_mul_fast(x, scaled(u[i], sr, col[kBN / 2 + c + i]));
        if (row < trows && c + i < n) y[(int64_t)(t.row0 + row) * p.ldy + t.n0 + c + i] = from_f32<Out>(x);
      }
    }
  }
}

template <bool kSwiglu, typename Out>
__global__ void __launch_bounds__(kThreads, 1) i8_pair_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* err = p.err ? p.err : &g_int_err;
  // The 128-byte swizzle needs 1024-byte aligned stages; the dynamic shared window of a CTA starts
  // 1024-byte aligned (both CTAs of a pair take this branch together).
  if (smem_u32(smem) & 1023u) {
    pdl_wait();
    if (threadIdx.x == 0) atomicOr(err, kErrWaitTimeout);
    return;
  }
  uint8_t* tok_base = smem + (size_t)kStages * kStage;  // [kStages][2] token boxes of dense swapped tiles
  PairSmem& m = *reinterpret_cast<PairSmem*>(smem + (size_t)kStages * kStage + kPairTok);
  volatile int* abort_flag = &m.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = (int)cluster_id_x(), npairs = (int)num_clusters_x();
  constexpr int kCols = kSwiglu ? kBN / 2 : kBN;  // output columns of a tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&m.tfull[a], 1);
      mbar_init(&m.tempty[a], 2 * kEpiWarps);
    }
    for (int i = 0; i < kPlans; ++i) {
      mbar_init(&m.ifull[i], 1);
      mbar_init(&m.sfull[i], 1);
      mbar_init(&m.pfree[i], (rank == 0 ? 2 : 1) + kEpiWarps);
    }
    mbar_init(&m.drain, 1);
    m.abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&p.mapA);
    tma_prefetch_desc(&p.mapB);
  }
  pdl_wait();  // below: reads of earlier kernels' output; TMEM once the previous kernel released its own
  if (warp == 1) {
    tmem_alloc_pair(&m.tmem_base, kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  if (warp == 0) schedule<kBM>(m, p.offsets, p.E, p.rows);
  __syncthreads();
  cluster_sync_all();  // the peer's barriers are initialised before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = m.tmem_base;
  const int total = m.mt[p.E] * p.n_tiles;

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer (both CTAs)
    const bool lead = elect_one();
    int s = 0;
    uint32_t ph = 0;
    const uint64_t evict_first = l2_evict_first_policy();
    const uint32_t full0 = mapa_shared(smem_u32(&m.full[0]), 0);
    bool ok = true;
    int it = 0;
    for (int L = pair; ok && L < total; L += npairs, ++it) {
      const int slot = it % kPlans;
      if (!__all_sync(0xffffffffu, wait_or_abort(&m.ifull[slot], (uint32_t)(it / kPlans) & 1u, abort_flag))) {
        if (lead) raise_abort(m, err);
        break;
      }
      const Tile& ts = m.tile[slot];
      const int e = __shfl_sync(0xffffffffu, ts.e, 0), row0 = __shfl_sync(0xffffffffu, ts.row0, 0);
      const int trows = __shfl_sync(0xffffffffu, ts.row_end, 0) - row0, n0 = __shfl_sync(0xffffffffu, ts.n0, 0);
      const int mtiles = __shfl_sync(0xffffffffu, ts.mtiles, 0);
      if (lead) mbar_arrive(&m.pfree[slot]);
      const bool light = trows <= p.light_rows, dense = light && trows <= kDenseRows;
      const bool once = light && mtiles == 1;  // its weights are read by this tile alone: evict them first
      const int nh = (trows + 31) / 32 * 16;   // swapped: token rows (N / 2) per CTA
      const int steps = dense ? (p.num_kb + 1) / 2 : p.num_kb;
      for (int step = 0; step < steps; ++step) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&m.empty[s], ph ^ 1u, abort_flag))) {
          if (lead) raise_abort(m, err);
          ok = false;
          break;
        }
        if (lead) {
          uint8_t* sA = smem + (size_t)s * kStage;
          uint8_t* sB = sA + kHalf;
          const uint32_t bar = full0 + (uint32_t)s * 8u;
          // 128 weight rows of a swapped tile
          auto weights = [&](uint8_t* dst, int kx) {
            if (kSwiglu) {
              if (once) tma2_load_5d_hint(dst, &p.mapB16, bar, kx, 0, 0, (n0 + 64 * (int)rank) / 16, e, evict_first);
              else tma2_load_5d(dst, &p.mapB16, bar, kx, 0, 0, (n0 + 64 * (int)rank) / 16, e);
            } else {
              if (once) tma2_load_3d_hint(dst, &p.mapB, bar, kx, n0 + 128 * (int)rank, e, evict_first);
              else tma2_load_3d(dst, &p.mapB, bar, kx, n0 + 128 * (int)rank, e);
            }
          };
          if (dense) {
            const int nk = min(2, p.num_kb - 2 * step);
            if (rank == 0) mbar_arrive_expect_tx(&m.full[s], (uint32_t)(2 * nk * (kHalf + kTok)));
            for (int j = 0; j < nk; ++j) {
              const int kx = (2 * step + j) * kKB;
              weights(sA + (size_t)j * kHalf, kx);
              tma2_load_2d(tok_base + (size_t)(2 * s + j) * kTok, &p.mapA16, bar, kx, row0 + (int)rank * nh);
            }
          } else if (light) {
            const int box = nh <= 32 ? 32 : 64;
            if (rank == 0) mbar_arrive_expect_tx(&m.full[s], (uint32_t)(2 * (kHalf + box * kKB)));
            weights(sA, step * kKB);
            tma2_load_2d(sB, nh <= 32 ? &p.mapA32 : &p.mapA64, bar, step * kKB, row0 + (int)rank * nh);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&m.full[s], 2 * kStage);
            tma2_load_2d(sA, &p.mapA, bar, step * kKB, row0 + 128 * (int)rank);
            if (kSwiglu) tma2_load_4d(sB, &p.mapB, bar, step * kKB, n0, (int)rank, e);
            else tma2_load_3d(sB, &p.mapB, bar, step * kKB, n0 + 128 * (int)rank, e);
          }
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    pdl_trigger();  // every copy of this CTA is issued: let the next kernel be scheduled
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (leader only)
    if (rank == 0) {
      const bool lead = elect_one();
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int L = pair; ok && L < total; L += npairs, ++it) {
        const int slot = it % kPlans;
        if (!__all_sync(0xffffffffu, wait_or_abort(&m.ifull[slot], (uint32_t)(it / kPlans) & 1u, abort_flag))) {
          ok = false;
          break;
        }
        const int trows = __shfl_sync(0xffffffffu, m.tile[slot].row_end - m.tile[slot].row0, 0);
        if (lead) mbar_arrive(&m.pfree[slot]);
        const int a = it & 1;
        if (!__all_sync(0xffffffffu, wait_or_abort(&m.tempty[a], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(a * kBN);
        const bool light = trows <= p.light_rows, dense = light && trows <= kDenseRows;
        const uint32_t idesc = light ? idesc_s8_s32(kBM, (trows + 31) / 32 * 32) : idesc_s8_s32(kBM, kBN);
        const int steps = dense ? (p.num_kb + 1) / 2 : p.num_kb;
        for (int step = 0; step < steps; ++step) {
          if (!__all_sync(0xffffffffu, wait_or_abort(&m.full[s], ph, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sA = smem_u32(smem) + (uint32_t)s * kStage;
          if (lead) {
            if (dense) {
              const int nk = min(2, p.num_kb - 2 * step);
              for (int j = 0; j < nk; ++j) {
                const uint64_t wa = smem_desc_sw128(sA + (uint32_t)(j * kHalf));
                const uint64_t tb = smem_desc_sw128(smem_u32(tok_base) + (uint32_t)(2 * s + j) * kTok);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_i8_pair(d_tmem, wa + 2 * kk, tb + 2 * kk, idesc, (step | j | kk) != 0 ? 1u : 0u);
              }
            } else {
              const uint64_t da = smem_desc_sw128(sA), db = smem_desc_sw128(sA + kHalf);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) tc_mma_i8_pair(d_tmem, da + 2 * kk, db + 2 * kk, idesc, (step | kk) != 0 ? 1u : 0u);
            }
            tc_commit_pair_mc(&m.empty[s], 0x3);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok && lead) tc_commit_pair_mc(&m.tfull[a], 0x3);
        __syncwarp();
      }
      if (lead) {
        if (!ok) raise_abort(m, err);
        tc_commit_pair(&m.drain);
        if (!mbar_wait_bounded(&m.drain, 0)) raise_abort(m, err);
      }
    }
    __syncwarp();
  } else if (warp == 2 + kEpiWarps) {
    // ------------------------------------------------------------- planner (both CTAs)
    int it = 0;
    for (int L = pair; L < total; L += npairs, ++it) {
      const int slot = it % kPlans;
      const bool got = wait_or_abort(&m.pfree[slot], ((uint32_t)(it / kPlans) & 1u) ^ 1u, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) raise_abort(m, err);
        break;
      }
      const Tile t = pair_tile(p, m, L, kCols);
      if (lane == 0) {
        m.tile[slot] = t;
        mbar_arrive(&m.ifull[slot]);
      }
      const int trows = t.row_end - t.row0;
      const float* ws = p.w_scale + (size_t)t.e * p.s_stride;
      float cs[kBN / 32], rs[4];
#pragma unroll
      for (int i = 0; i < kBN / 32; ++i) {
        const int c = lane + 32 * i, n = t.n0 + (kSwiglu ? c & (kBN / 2 - 1) : c);
        cs[i] = n < p.N ? __ldg(ws + (kSwiglu && c >= kBN / 2 ? p.N : 0) + n) : 0.f;
      }
      const int r0 = trows <= p.light_rows ? t.row0 : t.row0 + 128 * (int)rank;
#pragma unroll
      for (int i = 0; i < 4; ++i) rs[i] = r0 + lane + 32 * i < t.row_end ? __ldg(p.a_scale + r0 + lane + 32 * i) : 0.f;
      bool wide = false;
#pragma unroll
      for (int i = 0; i < kBN / 32; ++i) {
        m.col[slot][lane + 32 * i] = cs[i];
        wide |= scale_wide(cs[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m.row[slot][lane + 32 * i] = rs[i];
        wide |= scale_wide(rs[i]);
      }
      wide = __any_sync(0xffffffffu, wide);
      if (lane == 0) m.wide[slot] = wide;
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.sfull[slot]);
    }
  } else {
    // ------------------------------------------------------------- epilogue (warps 2..9, both CTAs)
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // the quarter's two warps take alternate blocks
    uint8_t* block = m.out[warp - 2];
    Out* const y = static_cast<Out*>(p.y);
    int it = 0;
    for (int L = pair; L < total; L += npairs, ++it) {
      const int a = it & 1, slot = it % kPlans;
      const bool got = wait_or_abort(&m.sfull[slot], (uint32_t)(it / kPlans) & 1u, abort_flag) &&
                       wait_or_abort(&m.tfull[a], (uint32_t)(it >> 1) & 1u, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) raise_abort(m, err);
        break;
      }
      tc_fence_after();
      const Tile t = m.tile[slot];
      const int trows = t.row_end - t.row0;
      const bool light = trows <= p.light_rows;
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * kBN);
      const float* col = m.col[slot];
      if (m.wide[slot]) {
        wide_tile<kSwiglu, Out>(p, m, slot, tb, (int)rank, q, half, lane);
      } else if (light) {
        // TMEM lane = weight row of this CTA, column c = the tile's row t.row0 + c
        const float* rs = m.row[slot];
        if (kSwiglu) {
          // lanes 0-15: gate of column 64 rank + 16 q + lane, lanes 16-31: up of the same columns
          const int c0 = 64 * (int)rank + 16 * q + (lane & 15), oc = t.n0 + c0;
          const float tn = col[(lane < 16 ? 0 : kBN / 2) + c0];
          for (int c = 16 * half; c < trows; c += 16 * kEpiHalves) {
            int v[16];
            tmem_ld16i(tb + c, v);
            tmem_ld_wait(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = c + i < trows ? (float)v[i] * (rs[(c + i) & (kLightRows - 1)] * tn) : 0.f;
              const float up = __shfl_down_sync(0xffffffffu, x, 16);
              if (lane < 16 && c + i < trows && oc < p.N)
                y[(int64_t)(t.row0 + c + i) * p.ldy + oc] = from_f32<Out>(silu_mul_fast(x, up));
            }
          }
        } else {
          const int c0 = 128 * (int)rank + q * 32 + lane, oc = t.n0 + c0;
          const float tn = col[c0];
          for (int c = 16 * half; c < trows; c += 16 * kEpiHalves) {
            int v[16];
            tmem_ld16i(tb + c, v);
            tmem_ld_wait(v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < trows && oc < p.N)
                y[(int64_t)(t.row0 + c + i) * p.ldy + oc] = from_f32<Out>((float)v[i] * (rs[c + i] * tn));
          }
        }
      } else {
        // 16 columns at a time; the next 16 leave TMEM while these are scaled and stored
        const int row_first = t.row0 + 128 * (int)rank + q * 32, rows = t.row_end - row_first;
        const int ncols = rows > 0 ? min(kCols, p.N - t.n0) : 0;
        const float sr = m.row[slot][q * 32 + lane];
        Out* const out = y + (int64_t)row_first * p.ldy + t.n0;
        auto load = [&](int c, int (&g)[16], int (&u)[16]) {
          tmem_ld16i(tb + c, g);
          if (kSwiglu) tmem_ld16i(tb + kBN / 2 + c, u);
        };
        auto finish = [&](int c, const int (&g)[16], const int (&u)[16]) {
          float v[16];
          const Pair s2 = pair_of(sr, sr);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const ulonglong2 tg = *reinterpret_cast<const ulonglong2*>(col + c + i);
            const ulonglong2 tu = *reinterpret_cast<const ulonglong2*>(col + (kSwiglu ? kBN / 2 : 0) + c + i);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              Pair r = pair_of((float)g[i + j], (float)g[i + j + 1]) * (s2 * Pair{j ? tg.y : tg.x});
              if (kSwiglu)
                r = silu_mul(r, pair_of((float)u[i + j], (float)u[i + j + 1]) * (s2 * Pair{j ? tu.y : tu.x}));
              halves(r, v[i + j], v[i + j + 1]);
            }
          }
          gather16<Out>(block, lane, c * (int)sizeof(Out) & (kOutRow - 1), v);
        };
        constexpr int kBlocks = kOutRow / 16 / (int)sizeof(Out);  // of 16 columns, in a gathered block
#pragma unroll 1
        for (int c0 = 16 * kBlocks * half; c0 < ncols; c0 += 16 * kBlocks * kEpiHalves) {
          int g[2][16], u[2][16];
          load(c0, g[0], u[0]);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int c = c0 + 16 * b;
            if (c < ncols) {
              if (kSwiglu) tmem_ld_wait(g[b & 1], u[b & 1]);
              else tmem_ld_wait(g[b & 1]);
              if (b + 1 < kBlocks && c + 16 < ncols) load(c + 16, g[(b + 1) & 1], u[(b + 1) & 1]);
              finish(c, g[b & 1], u[b & 1]);
            }
          }
          store_block(out + c0, p.ldy, block, rows, ncols - c0, p.vec, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&m.tempty[a]), 0));
        mbar_arrive(&m.pfree[slot]);
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && m.abort) {
    // error path: give copies still in flight time to land before the CTA leaves
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 2000000ull) {
    }
  }
  cluster_sync_all();  // the peer no longer reads this CTA's shared memory or arrives on it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ------------------------------------------------------------------------- split kernel
constexpr int kSplitTile = 128;    // rows and weight rows of a tile
constexpr int kSplitStages = 6;
constexpr int kSplitThreads = 192;  // producer, MMA, four epilogue warps
constexpr int kSplitMax = 4;
constexpr int kSplitTmem = 128;

struct alignas(64) SplitParams {
  CUtensorMap mapA;  // rows, boxes of 128
  CUtensorMap mapB;  // weights, boxes of 128 rows (SwiGLU: 64)
  const int32_t* offsets;
  const float* a_scale;
  const float* w_scale;
  int64_t s_stride;
  void* y;
  int64_t ldy;
  uint32_t* err;
  int E, rows, N;
  int n_tiles, num_kb, split;
  bool vec;
};

struct SplitSmem {
  static constexpr bool kClasses = false;
  uint64_t full[kSplitStages];
  uint64_t empty[kSplitStages];
  uint64_t tfull;
  uint32_t tmem_base;
  int abort;
  int issued, consumed;
  int wide;  // some scale of the tile is wide
  int32_t off[kMaxExperts + 1];
  int32_t mt[kMaxExperts + 1];
  alignas(16) float col[kSplitTile];
  alignas(16) float row[kSplitTile];
  alignas(16) uint8_t out[4][32 * kOutPitch];
};
constexpr size_t kSplitSmem = (size_t)kSplitStages * kStage + sizeof(SplitSmem);
static_assert(kSplitSmem <= 232448, "shared memory of one CTA");
// partial sums received: [source][16-byte unit of 4 columns][row]
static_assert((size_t)kSplitMax * kSplitTile * kSplitTile / kSplitMax * 4 <= (size_t)kSplitStages * kStage, "exchange");

__device__ __forceinline__ void st_shared_cluster_v4(uint32_t cluster_addr, int a, int b, int c, int d) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <bool kSwiglu, typename Out>
__global__ void __launch_bounds__(kSplitThreads, 1) i8_split_kernel(const __grid_constant__ SplitParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* err = p.err ? p.err : &g_int_err;
  SplitSmem& m = *reinterpret_cast<SplitSmem*>(smem + (size_t)kSplitStages * kStage);
  volatile int* abort_flag = &m.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split, rank = S > 1 ? (int)cluster_ctarank() : 0;
  constexpr int kCols = kSwiglu ? kSplitTile / 2 : kSplitTile;  // output columns of a tile
  const bool aligned = (smem_u32(smem) & 1023u) == 0;  // needed by the 128-byte swizzle; the same in every CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSplitStages; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    mbar_init(&m.tfull, 1);
    m.abort = 0;
    m.issued = m.consumed = m.wide = 0;
    mbar_fence_init();
    tma_prefetch_desc(&p.mapA);
    tma_prefetch_desc(&p.mapB);
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 1) {
    tmem_alloc(&m.tmem_base, kSplitTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  if (warp == 0) schedule<kSplitTile>(m, p.offsets, p.E, p.rows);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = m.tmem_base;

  // the tile: group-major, then n, then m
  const int L = (int)blockIdx.x / S;
  const bool work = aligned && L < m.mt[p.E] * p.n_tiles;  // the same in every CTA of the cluster
  Tile t = {0, 0, 0, 0, 1};
  if (work) {
    t.e = find_group(m.mt, p.E, p.n_tiles, L);
    t.mtiles = m.mt[t.e + 1] - m.mt[t.e];
    const int r = L - m.mt[t.e] * p.n_tiles, n = r / t.mtiles;
    t.row0 = m.off[t.e] + (r - n * t.mtiles) * kSplitTile;
    t.row_end = m.off[t.e + 1];
    t.n0 = n * kCols;
  } else if (!aligned && threadIdx.x == 0) {
    atomicOr(err, kErrWaitTimeout);
  }
  const int kb0 = p.num_kb * rank / S, kb1 = p.num_kb * (rank + 1) / S;  // this CTA's k blocks

  if (work && warp == 0) {
    const bool lead = elect_one();
    int issued = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++issued) {
      const int s = issued % kSplitStages;
      if (!__all_sync(0xffffffffu, wait_or_abort(&m.empty[s], ((uint32_t)(issued / kSplitStages) & 1u) ^ 1u, abort_flag))) {
        if (lead) raise_abort(m, err);
        break;
      }
      if (lead) {
        uint8_t* sA = smem + (size_t)s * kStage;
        uint8_t* sB = sA + kHalf;
        mbar_arrive_expect_tx(&m.full[s], kStage);
        tma_load_2d(sA, &p.mapA, &m.full[s], kb * kKB, t.row0);
        if (kSwiglu) {
          tma_load_4d(sB, &p.mapB, &m.full[s], kb * kKB, t.n0, 0, t.e);
          tma_load_4d(sB + kHalf / 2, &p.mapB, &m.full[s], kb * kKB, t.n0, 1, t.e);
        } else {
          tma_load_3d(sB, &p.mapB, &m.full[s], kb * kKB, t.n0, t.e);
        }
      }
      __syncwarp();
    }
    if (lead) m.issued = issued;
  } else if (work && warp == 1) {
    const bool lead = elect_one();
    int consumed = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++consumed) {
      const int s = consumed % kSplitStages;
      if (!__all_sync(0xffffffffu, wait_or_abort(&m.full[s], (uint32_t)(consumed / kSplitStages) & 1u, abort_flag))) {
        if (lead) raise_abort(m, err);
        break;
      }
      tc_fence_after();
      if (lead) {
        const uint64_t da = smem_desc_sw128(smem_u32(smem) + (uint32_t)s * kStage);
        const uint64_t db = smem_desc_sw128(smem_u32(smem) + (uint32_t)s * kStage + kHalf);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_i8(tmem_base, da + 2 * kk, db + 2 * kk, idesc_s8_s32(kSplitTile, kSplitTile),
                    (consumed | kk) != 0 ? 1u : 0u);
        tc_commit(&m.empty[s]);
      }
      __syncwarp();
    }
    if (lead) {
      m.consumed = consumed;
      tc_commit(&m.tfull);  // also after an error: every MMA issued has ended
      if (!mbar_wait_bounded(&m.tfull, 0)) raise_abort(m, err);  // no sums: nothing is exchanged or stored
    }
    __syncwarp();
  } else if (work && warp >= 2) {
    // the tile's scales, while the products run
    const int i = threadIdx.x - 64;
    const float* ws = p.w_scale + (size_t)t.e * p.s_stride;
    const int n = t.n0 + (kSwiglu ? i & (kCols - 1) : i);
    m.col[i] = n < p.N ? __ldg(ws + (kSwiglu && i >= kCols ? p.N : 0) + n) : 0.f;
    m.row[i] = t.row0 + i < t.row_end ? __ldg(p.a_scale + t.row0 + i) : 0.f;
    if (scale_wide(m.col[i]) || scale_wide(m.row[i])) m.wide = 1;
  }
  __syncthreads();  // this CTA's products have ended: its ring is idle
  if (threadIdx.x == 0 && m.abort)
    for (int i = m.consumed; i < m.issued; ++i)  // error path: copies that no product waited for
      if (!mbar_wait_bounded(&m.full[i % kSplitStages], (uint32_t)(i / kSplitStages) & 1u)) break;
  __syncthreads();
  const bool ok = work && !m.abort;
  tc_fence_after();

  // columns of the tile that this CTA finishes: 1 / S of them (SwiGLU: of the gate and of the up columns)
  const int own = kCols / S;
  const int q = warp & 3;
  const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16);
  constexpr int kParts = kSwiglu ? 2 : 1;
  const int units = own * kParts / 4;  // 16-byte units of 4 columns per source and row
  if (S > 1) {
    cluster_sync_all();  // the rings of all CTAs are idle
    if (ok && warp >= 2) {
      const int row = q * 32 + lane;
      for (int j = 1; j < S; ++j) {
        const int to = (rank + j) % S;
        for (int part = 0; part < kParts; ++part)
          for (int c = 0; c < own; c += 16) {
            int v[16];
            tmem_ld16i(tb + part * kCols + to * own + c, v);
            tmem_ld_wait(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int unit = rank * units + (part * own + c) / 4 + i;
              st_shared_cluster_v4(mapa_shared(smem_u32(smem) + (uint32_t)(unit * kSplitTile + row) * 16u, (uint32_t)to),
                                   v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
          }
      }
    }
    cluster_sync_all();  // the partial sums have arrived
  }
  if (ok && warp >= 2) {
    const int row_first = t.row0 + q * 32, rows = t.row_end - row_first, c_first = rank * own;
    const int ncols = rows > 0 ? min(own, p.N - t.n0 - c_first) : 0;
    const float sr = m.row[q * 32 + lane];
    Out* const out = static_cast<Out*>(p.y) + (int64_t)row_first * p.ldy + t.n0 + c_first;
    constexpr int kBlock = kOutRow / (int)sizeof(Out);  // columns of a gathered block
    auto sums = [&](int part, int c, int (&v)[16]) {
      tmem_ld16i(tb + part * kCols + c_first + c, v);
      tmem_ld_wait(v);
      for (int j = 1; j < S; ++j) {
        const int from = (rank + j) % S;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int unit = from * units + (part * own + c) / 4 + i;
          const int4 w = *reinterpret_cast<const int4*>(smem + (size_t)(unit * kSplitTile + q * 32 + lane) * 16);
          v[4 * i] += w.x;
          v[4 * i + 1] += w.y;
          v[4 * i + 2] += w.z;
          v[4 * i + 3] += w.w;
        }
      }
    };
    for (int c = 0; c < ncols; c += 16) {
      int g[16], u[16];
      sums(0, c, g);
      if (kSwiglu) sums(1, c, u);
      float v[16];
      if (m.wide) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[i] = scaled(g[i], sr, m.col[c_first + c + i]);
          if (kSwiglu) v[i] = silu_mul_fast(v[i], scaled(u[i], sr, m.col[kCols + c_first + c + i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[i] = (float)g[i] * (sr * m.col[c_first + c + i]);
          if (kSwiglu) v[i] = silu_mul_fast(v[i], (float)u[i] * (sr * m.col[kCols + c_first + c + i]));
        }
      }
      gather16<Out>(m.out[q], lane, c * (int)sizeof(Out) & (kOutRow - 1), v);
      const int at = c & ~(kBlock - 1);  // the block's first column
      if (c + 16 >= ncols || c + 16 - at == kBlock)
        store_block(out + at, p.ldy, m.out[q], rows, ncols - at, p.vec, lane);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kSplitTmem);
  }
}

bool byte_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
              const uint32_t* box) {
  return make_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rank, dims, strides, box);
}

// What both kernels are told.
template <typename Params>
void fill_params(Params& p, const IntGemmArgs& a, int tile_cols) {
  p.offsets = a.offsets;
  p.a_scale = a.a_scale;
  p.w_scale = a.w_scale;
  p.s_stride = a.s_stride;
  p.y = a.y;
  p.ldy = a.ldy;
  p.err = a.err;
  p.E = a.E;
  p.rows = a.rows;
  p.N = a.N;
  p.num_kb = (a.K + kKB - 1) / kKB;
  p.n_tiles = (a.N + tile_cols - 1) / tile_cols;
  p.vec = (a.ldy * (a.out_dtype == COLIBRI_BF16 ? 2 : 4)) % 16 == 0;
}

// Weights as [K, N, E], or for SwiGLU [K, N, W1 | W3, E], in boxes of `rows` weight rows.
bool weight_map(CUtensorMap* map, const IntGemmArgs& a, bool swiglu, uint32_t rows) {
  const uint64_t K = a.K, N = a.N, E = a.E;
  const uint64_t es = a.w_stride > 0 ? (uint64_t)a.w_stride : (uint64_t)a.ldw;  // a single group: not used
  if (swiglu) {
    uint64_t dims[4] = {K, N, 2, E}, st[3] = {K, N * K, es};
    uint32_t box[4] = {kKB, rows, 1, 1};
    return byte_map(map, a.W, 4, dims, st, box);
  }
  uint64_t dims[3] = {K, N, E}, st[2] = {(uint64_t)a.ldw, es};
  uint32_t box[3] = {kKB, rows, 1};
  return byte_map(map, a.W, 3, dims, st, box);
}

bool row_map(CUtensorMap* map, const IntGemmArgs& a, uint32_t rows) {
  uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.rows}, st[1] = {(uint64_t)a.lda};
  uint32_t box[2] = {kKB, rows};
  return byte_map(map, a.A, 2, dims, st, box);
}

template <typename Kernel, typename Params>
cudaError_t launch_configured(Kernel kern, unsigned grid, int threads, size_t smem, unsigned cluster, const Params& p,
                              cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  return e != cudaSuccess ? e : launch_kernel(kern, dim3(grid), dim3(threads), smem, s, cluster, p);
}

template <bool kSwiglu>
cudaError_t launch_pair(const IntGemmArgs& a, int sms, cudaStream_t s) {
  PairParams p;
  memset(&p, 0, sizeof(p));
  constexpr int cols = kSwiglu ? kBN / 2 : kBN;
  fill_params(p, a, cols);
  bool ok = row_map(&p.mapA, a, 128) && row_map(&p.mapA16, a, 16) && row_map(&p.mapA32, a, 32) &&
            row_map(&p.mapA64, a, 64) && weight_map(&p.mapB, a, kSwiglu, 128);
  p.light_rows = kLightRows;
  if (kSwiglu) {
    const uint64_t K = a.K, N = a.N;
    if (N % 16 == 0) {
      uint64_t dims[5] = {K, 16, 2, N / 16, (uint64_t)a.E}, st[4] = {K, N * K, 16 * K, (uint64_t)a.w_stride};
      uint32_t box[5] = {kKB, 16, 2, 4, 1};
      ok = ok && byte_map(&p.mapB16, a.W, 5, dims, st, box);
    } else {
      p.light_rows = 0;
    }
  }
  if (!ok) return cudaErrorInvalidValue;
  const long long bound = (long long)(a.rows / kBM + (a.offsets ? a.E : 1)) * p.n_tiles;
  const unsigned pairs = (unsigned)std::min<long long>(bound, sms / 2);
  auto kern = a.out_dtype == COLIBRI_BF16 ? i8_pair_kernel<kSwiglu, __nv_bfloat16> : i8_pair_kernel<kSwiglu, float>;
  return launch_configured(kern, 2 * pairs, kThreads, kPairSmem, 2, p, s);
}

// `tiles`: how many 128 x 128 tiles there may be; each on `split` CTAs.
template <bool kSwiglu>
cudaError_t launch_split(const IntGemmArgs& a, int tiles, int split, cudaStream_t s) {
  SplitParams p;
  memset(&p, 0, sizeof(p));
  fill_params(p, a, kSwiglu ? kSplitTile / 2 : kSplitTile);
  if (!row_map(&p.mapA, a, kSplitTile) || !weight_map(&p.mapB, a, kSwiglu, kSwiglu ? kSplitTile / 2 : kSplitTile))
    return cudaErrorInvalidValue;
  p.split = split;
  auto kern = a.out_dtype == COLIBRI_BF16 ? i8_split_kernel<kSwiglu, __nv_bfloat16> : i8_split_kernel<kSwiglu, float>;
  return launch_configured(kern, (unsigned)(tiles * split), kSplitThreads, kSplitSmem, (unsigned)split, p, s);
}

}  // namespace

cudaError_t launch_int_gemm(const IntGemmArgs& a, bool swiglu, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // At most 16 rows of one product: the stream of gemv_i8.cu, until the weights are so many that the pair
  // kernel's copies, with a tile for at least half its pairs, make up for its set-up.  Weights from HBM,
  // there and here: 1 row of 9728 x 4096 16.4 / 18.0 us, 14336 x 4096 22.6 / 20.4, 152000 x 1024 55 / 38;
  // 16 rows of 16384 x 2048 18.5 / 16.4, 14336 x 4096 24.5 / 20.4, 152000 x 1024 61 / 39 (with 14336 x 4096
  // in L2 10.4 / 13 at 1 row and 14.1 / 13 at 16).
  if (!swiglu && !a.offsets && a.rows <= kSkinnyRows &&
      ((a.N + kBN - 1) / kBN <= sms / 4 || (int64_t)a.N * a.K < (a.rows <= 8 ? 5 : 4) * (int64_t(1) << 23)))
    return launch_int_skinny(a, sms, s);
  // Fewer tiles of 128 x 128 than SMs: one CTA per tile, or with k split 2 or 4 CTAs, all at once;
  // more tiles keep the pair kernel's SMs busy (both sides: the header comment).  With at most 32 rows the
  // pair kernel streams two k blocks of weights per stage and is ahead too, unless four CTAs share a
  // long k (32 rows, weights from HBM: 14336 x 4096 20.7 against 24.0 us, 8192 x 4096 18.2 / 20.2, 4096 x 5120
  // 16.7 / 18.4, but 2048 x 8192 20.6 / 18.3, 4096 x 14336 28.8 / 26.6).
  const int groups = a.offsets ? a.E : 1, cols = swiglu ? kSplitTile / 2 : kSplitTile;
  const long long tiles = (a.offsets ? (long long)a.rows / kSplitTile + groups : (a.rows + kSplitTile - 1) / kSplitTile) *
                          ((a.N + cols - 1) / cols);
  if (tiles <= sms) {
    const int kbs = (a.K + kKB - 1) / kKB;
    int split = 1;
    while (split < kSplitMax && tiles * split * 2 <= sms && kbs >= 4 * split) split *= 2;
    const bool swapped = a.rows <= kDenseRows && (!swiglu || a.N % 16 == 0);
    if (!swapped || (split == kSplitMax && kbs > 40))
      return swiglu ? launch_split<true>(a, (int)tiles, split, s) : launch_split<false>(a, (int)tiles, split, s);
  }
  return swiglu ? launch_pair<true>(a, sms, s) : launch_pair<false>(a, sms, s);
}

// Allows the kernels that a context's forward may launch their shared memory, before the first launch.
cudaError_t configure_int_kernels() {
  const auto set = [](auto kern, size_t smem) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  };
  cudaError_t e = set(i8_pair_kernel<true, __nv_bfloat16>, kPairSmem);
  if (e == cudaSuccess) e = set(i8_pair_kernel<false, __nv_bfloat16>, kPairSmem);
  if (e == cudaSuccess) e = set(i8_split_kernel<true, __nv_bfloat16>, kSplitSmem);
  if (e == cudaSuccess) e = set(i8_split_kernel<false, __nv_bfloat16>, kSplitSmem);
  return e;
}

cudaError_t int_gemm_error_word(uint32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_int_err);
}

// The error word of calls without one of their own, read and cleared behind the work on `s`.
cudaError_t int_gemm_take_error(uint32_t* word, cudaStream_t s) {
  static std::atomic<unsigned> next{0};
  const unsigned slot = next.fetch_add(1u) % kTaken;
  cudaError_t e = launch_kernel(take_error_kernel, dim3(1), dim3(1), 0, s, 1, slot);
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(word, g_int_taken, sizeof(uint32_t), slot * sizeof(uint32_t), cudaMemcpyDeviceToHost, s);
  const cudaError_t done = cudaStreamSynchronize(s);
  return e != cudaSuccess ? e : done;
}

}  // namespace colibri
