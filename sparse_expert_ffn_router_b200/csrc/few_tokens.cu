// The whole MoE layer for at most 16 tokens in one cooperative launch (bf16 or fp32 weights, with
// the shared expert): router, top-k, gate/up, down, weighted sum.
//
//   logits[t][e] = x_t . Wr_e + b_e;  the k chosen experts and their weights p (few_topk)
//   h[t][e]      = silu(W1_e x_t) * (W3_e x_t)
//   y[t]         = sum_(e chosen by t) p[t][e] W2_e h[t][e]  (+ W2_s h_s[t])
//
// With a few tokens every touched expert's weights are read once and meet a few rows, so the work
// is a stream over those weights (2 or 4 bytes per 2 x tokens FLOP) and the bound is HBM.  Three
// phases, two grid barriers between them:
//   router   the logits, one task per expert and a few tokens, the tasks over the CTAs.
//   gate/up  every CTA selects the experts of all tokens from the logits (the same result in each),
//            then owns an equal share of the gate columns of all touched experts together, whatever
//            expert they fall in.
//   down     every CTA owns an equal share of the output columns, for all touched experts, so the
//            weighted sum is formed where it is needed, in ascending expert order: no third
//            barrier, no atomics, the same bits in every run.  Where that would leave a CTA fewer
//            than kFewSplitRows columns (a lane's loads would mostly have no row), 32 columns go to
//            a team of CTAs that split the sum, and a third barrier lets all CTAs add the parts up.
// The shares are split to single columns (a partly filled tile loads only its own rows), so that no
// CTA reads more than one row above the average.
//
// Inside a CTA the 16 warps split the inner dimension: all tiles' chunks of 64 bytes of a row, laid
// end to end, go to the warps in equal runs, so a warp crosses tiles and experts without meeting the
// others.  Partial sums meet in shared memory, in warp order, once per 16 tiles (gate/up) or once per
// 32 output columns (down: a warp adds its experts up, weighted, in its own part of it); meeting after
// every tile cost 2 us per tile.  Each lane keeps its weights in flight through a ring of shared memory
// that the same lane fills (cp.async) and drains: no lane reads what another lane copied, so the ring
// needs no barrier, and a warp's copies run ahead across tiles, experts and the barrier between the
// two projections.  The copies fetch 256 bytes of a row at a time into L2 (a warp walks along rows 64
// bytes per step; without that one token took 141 us instead of 124).  bf16: mma.m16n8k16, weights as
// the 16-row operand (8 gate rows and the 8 up rows of the same columns; for down 16 output columns),
// tokens as the 8 columns; the order of k inside an instruction is free, so a lane's 16 bytes of a weight
// row feed two instructions as they are, and the token operand is 16 bytes of the token's row.  fp32:
// FMA on the CUDA cores.  H is kept as fp32, or as two bf16 (its rounding and what that left, 2^-16 in
// all): one rounding to bf16 would double the variance of the output's own rounding error (0.0023
// against 0.0017 of the output's norm); the second product and its sums, kept apart, cost 5 us of 67 on 128
// small experts, 1 of 122 at one token of large ones and nothing at 16.
//
// Measured (B200, copy bandwidth 6455 GB/s; 20 calls in a row, a call by itself is 1 to 4 % slower): d = 4096,
// f = 14336, 8 experts, top-2, bf16: 1 token (704 MB) 122 us, 5.8 TB/s; 16 tokens (2.8 GB) 453 us, 6.2 TB/s.
// 128 experts of d = 2048, f = 768, top-4, with a shared expert of 1536: 8 tokens (291 MB) 67.5 us.  An fp32
// layer of 256 x 512: 16.5 us, latency alone (logits 2.5, selection 1.8, gate/up 4, down 2, the barriers 2
// each, the launch 3).  fp32 with many tokens is bound by the lanes' exchanges and FMAs: two experts of
// 1024 x 2688 (66 MB) 23 us at one token, 37 at 8, 65 at 16.
#include "common.cuh"

namespace colibri {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewDepth = 4;             // ring stages of a warp
constexpr int kFewStage = 4 * 512;       // bytes of a warp's stage: 4 rows of 16 bytes per lane
constexpr int kFewEntries = kFewMaxT * kMaxTopK + 1;  // touched experts and the shared one
constexpr int kFewPitch = kFewMaxT + 2;  // floats per weight row of the partial sums (16 token columns)
constexpr int kFewSplitRows = 9;         // fewer output columns per CTA: the down projection is split
constexpr int kFewBatch = 16;            // gate/up tiles whose partial sums meet at a time
constexpr int kFewSlot = kFewRowsW * kFewPitch;       // floats of one warp's partial sums of one tile

struct FewCtl {
  int32_t idx[kFewMaxT * kMaxTopK];
  float w[kFewMaxT * kMaxTopK];
  uint32_t mask[kMaxExperts];            // tokens that chose the expert
  int32_t off[kMaxExperts + 1];
  // the experts to compute, the shared one first
  int32_t ent_e[kFewEntries];            // expert, or -1: shared
  int32_t ent_row[kFewEntries];          // first row in H (shared: Hs)
  int32_t ent_n[kFewEntries];            // tokens
  uint8_t ent_tok[kFewEntries][kFewMaxT];
  float ent_w[kFewEntries][kFewMaxT];    // weight by token
  int32_t warp_rows[kMaxExperts / 32];   // while selecting
  int32_t warp_has[kMaxExperts / 32];
  int32_t n_ent;
  int32_t ok;
  int32_t abort;
  float part[kFewWarps][kFewMaxT];       // router partial sums
};

// the tiles of a batch are consecutive, and so are the warps' runs over them: the partial sums of
// (tile i, warp w) go to slot i + w
constexpr size_t kFewRing = (size_t)kFewWarps * kFewDepth * kFewStage;
constexpr size_t kFewRed = (size_t)(kFewBatch + kFewWarps - 1) * kFewSlot * 4;
constexpr size_t kFewSmem = kFewRing + kFewRed + sizeof(FewCtl);
static_assert(kFewSmem <= 232448, "shared memory of the few-token kernel");
static_assert((size_t)kFewMaxT * kMaxExperts * 4 <= kFewRed, "logits are staged in the partial sums' memory");

template <typename T>
struct FewParams {
  const T* x;          // [T, d]
  const T* router_w;   // [E, d]
  const float* router_b;
  const T* W;
  int64_t wstride;
  const T* Ws;         // shared expert or nullptr
  T* H;                // [T*k, f]
  T* Hs;               // [T, fs]
  T* Hlo;              // bf16: what rounding left of H and Hs, as bf16 again
  T* Hslo;
  float* part;         // [splits, T, d] partial sums of a split down projection
  T* y;                // [T, d]
  float* logits;       // [T, E]
  int32_t *topk_idx, *counts, *offsets, *src_row, *dst_row;
  float* topk_w;
  int32_t* bar;        // [3]
  uint32_t* err;
  int T_, d, f, fs, E, k, flags;
  int tg;              // router: tokens per task
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The runs of chunks of one CTA.  Gate/up: the gate columns of all entries laid end to end, cut into
// tiles of 16 (every width is a multiple of 64, so a tile lies in one entry); the CTA owns columns
// [c0, c1) and takes their tiles in batches.  Down: the CTA owns output columns [o0, o1), in groups of
// 32, each group over the chunks [d0, d1) of all entries laid end to end.
template <typename T>
struct FewShare {
  static constexpr int CE = 64 / sizeof(T);  // elements of a chunk
  int c0, c1;
  int o0, o1;
  int tiles, batches, groups;
  int cd, cf, cs;  // chunks of a row of d, f, fs elements
  int d0, d1;      // down: this CTA's run over the chunks of all entries
  int teams, splits, split;  // down, split: teams of `splits` CTAs, and this CTA's place in its team (teams 0: not)
  int fs, f;

  __device__ FewShare(const FewParams<T>& p, int n_ent) {
    fs = p.fs;
    f = p.f;
    const int routed = n_ent - (fs > 0 ? 1 : 0);
    const int G = gridDim.x, b = blockIdx.x;
    cut(fs + routed * f, G, b, c0, c1);  // at most 129 * 2^18 columns
    tiles = c1 > c0 ? (c1 + 15) / 16 - c0 / 16 : 0;
    batches = (tiles + kFewBatch - 1) / kFewBatch;
    cd = p.d / CE;
    cf = f / CE;
    cs = fs / CE;
    d0 = 0;
    d1 = cs + routed * cf;
    teams = 0;
    if (p.d < kFewSplitRows * G) {
      teams = (p.d + kFewRowsW - 1) / kFewRowsW;
      splits = G / teams;
      const int team = b % teams;
      split = b / teams;
      groups = split < splits ? 1 : 0;
      o0 = team * kFewRowsW;
      o1 = min(p.d, o0 + kFewRowsW);
      if (groups) cut(d1, splits, split, d0, d1);
    } else {
      cut(p.d, G, b, o0, o1);
      groups = (o1 - o0 + kFewRowsW - 1) / kFewRowsW;
    }
  }
  // part i of n things in G nearly equal parts
  __device__ static __forceinline__ void cut(int n, int G, int i, int& a, int& b) {
    const int each = n / G, rest = n - each * G;
    a = each * i + min(i, rest);
    b = a + each + (i < rest ? 1 : 0);
  }
  __device__ __forceinline__ int batch_tiles(int s) const { return min(kFewBatch, tiles - s * kFewBatch); }
  // chunks that warp w takes of the batch or group
  __device__ __forceinline__ int begin(int phase, int s, int w) const {
    return phase == 0 ? batch_tiles(s) * cd * w / kFewWarps : d0 + (d1 - d0) * w / kFewWarps;
  }
};

// A run's part within one tile (gate/up) or entry (down).
struct FewSeg {
  int ent, chunk, left;
  int tile;            // gate/up: its number in the batch
  int col, lo, hi;     // gate/up: the tile's first column in the entry, and the columns [lo, hi) of it that are owned
};
template <typename T>
__device__ __forceinline__ FewSeg few_segment(const FewShare<T>& h, int phase, int s, int pos, int end) {
  FewSeg g;
  const int shared = h.fs > 0 ? 1 : 0;
  if (phase == 0) {
    g.tile = pos / h.cd;
    g.chunk = pos - g.tile * h.cd;
    g.left = min(end - pos, h.cd - g.chunk);
    const int gc = (h.c0 / 16 + s * kFewBatch + g.tile) * 16;
    g.lo = max(0, h.c0 - gc);
    g.hi = min(16, h.c1 - gc);
    if (gc < h.fs) {
      g.ent = 0;
      g.col = gc;
    } else {
      const int r = gc - h.fs, i = r / h.f;
      g.ent = shared + i;
      g.col = r - i * h.f;
    }
  } else {
    g.tile = g.col = g.lo = g.hi = 0;
    if (pos < h.cs) {
      g.ent = 0;
      g.chunk = pos;
      g.left = min(end, h.cs) - pos;
    } else {
      const int r = pos - h.cs, i = r / h.cf;
      g.ent = shared + i;
      g.chunk = r - i * h.cf;
      g.left = min(end - pos, h.cf - g.chunk);
    }
  }
  return g;
}

// The weight stream of one lane: 4 rows (q = 0..3) of the current tile, 16 bytes per row and chunk.
// Gate/up: q & 1 picks W1 or W3, q >> 1 the upper 8 columns; down: 8 columns per q.
template <typename T>
struct FewStream {
  const FewParams<T>& p;
  const FewCtl& c;
  const FewShare<T>& h;
  const T* ptr;
  int64_t s1, s2;  // offsets of q & 1 and q >> 1
  uint32_t live;   // q's whose row exists
  int phase, s, pos, end, left;
  int warp, g, t;

  __device__ FewStream(const FewParams<T>& p_, const FewCtl& c_, const FewShare<T>& h_, int warp_, int lane)
      : p(p_), c(c_), h(h_), phase(0), s(-1), pos(0), end(0), warp(warp_), g(lane >> 2), t(lane & 3) {
    open();
  }
  __device__ __forceinline__ void open() {  // the segment at pos, or the next batch or group with chunks for this warp
    while (pos >= end) {
      ++s;
      if (phase == 0 && s >= h.batches) {
        phase = 1;
        s = 0;
      }
      if (phase == 1 && s >= h.groups) {
        phase = 2;
        return;
      }
      pos = h.begin(phase, s, warp);
      end = h.begin(phase, s, warp + 1);
    }
    const FewSeg sg = few_segment(h, phase, s, pos, end);
    left = sg.left;
    const int e = c.ent_e[sg.ent];
    const int64_t f = e < 0 ? p.fs : p.f, d = p.d;
    const T* base = e < 0 ? p.Ws : p.W + (int64_t)e * p.wstride;
    live = 0;
    if (phase == 0) {
      ptr = base + (int64_t)(sg.col + g) * d;
      s1 = f * d;
      s2 = 8 * d;
      live = (g >= sg.lo && g < sg.hi ? 3u : 0u) | (g + 8 >= sg.lo && g + 8 < sg.hi ? 12u : 0u);
    } else {
      const int o = h.o0 + s * kFewRowsW;
      ptr = base + 2 * f * d + (int64_t)(o + g) * f;
      s1 = 8 * f;
      s2 = 16 * f;
#pragma unroll
      for (int q = 0; q < 4; ++q) live |= (o + g + 8 * q < h.o1 ? 1u : 0u) << q;
    }
    ptr += (int64_t)sg.chunk * (64 / sizeof(T)) + t * (16 / sizeof(T));
  }
  // copies the next chunk into the stage (nothing once the share has ended) and closes the group
  __device__ __forceinline__ void issue(uint32_t dst) {
    if (phase < 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (live >> q & 1u) cp_async16(dst + q * 512, ptr + (q & 1) * s1 + (q >> 1) * s2);
      ptr += 64 / sizeof(T);
      ++pos;
      if (--left == 0) open();
    }
    cp_async_commit();
  }
};

// Sums of one lane over chunks: bf16 [P parts of the columns' values][2 blocks of 16 weight rows][NT blocks
// of 8 columns][4], in the instruction's layout; fp32 [4 rows][8 NT columns], this lane's part of each chunk.
// The sum over the second part of H stands apart, because it counts only beside a finite sum over the
// first: where that is infinite (a weight or H is), this one is infinite of either sign or NaN.
template <typename T, int NT, int P>
struct FewAcc;
template <int NT, int P>
struct FewAcc<__nv_bfloat16, NT, P> {
  float v[P][2][NT][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int h = 0; h < P; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[h][m][j][i] = 0.f;
  }
  __device__ __forceinline__ float sum(int m, int j, int i) const {
    const float hi = v[0][m][j][i];
    return P == 2 && fabsf(hi) < INFINITY ? hi + v[P - 1][m][j][i] : hi;
  }
  // row q * 8 + g of the tile, token columns 8 j + 2 t and the next
  __device__ __forceinline__ void store(float* red, int, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float2*>(red + ((2 * m + i) * 8 + g) * kFewPitch + 8 * j + 2 * t) =
              make_float2(sum(m, j, 2 * i), sum(m, j, 2 * i + 1));
  }
  // the sums of column j, times its weight, onto column tok[j] of red
  __device__ __forceinline__ void add(float* red, const uint8_t* tok, const float* w, int n, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int col = 8 * j + 2 * t + b;
        if (col < n) {
          const int to = tok[col];
          const float wt = w[to];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float* d = red + (q * 8 + g) * kFewPitch + to;
            *d = fmaf(wt, sum(q >> 1, j, 2 * (q & 1) + b), *d);
          }
        }
      }
  }
};
template <int NT, int P>
struct FewAcc<float, NT, P> {
  float v[4][8 * NT];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 8 * NT; ++j) v[q][j] = 0.f;
  }
  // The sum over the row's four lanes of column j0 + t, for lane t: each step hands half of the columns
  // over (3 exchanges per 4 columns; all columns in all lanes take 8).
  __device__ __forceinline__ float column(int q, int j0, int t) const {
    const float* a = v[q] + j0;
    const bool hi = t & 2, odd = t & 1;
    const float k0 = (hi ? a[2] : a[0]) + __shfl_xor_sync(0xffffffffu, hi ? a[0] : a[2], 2);
    const float k1 = (hi ? a[3] : a[1]) + __shfl_xor_sync(0xffffffffu, hi ? a[1] : a[3], 2);
    return (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
  }
  __device__ __forceinline__ void store(float* red, int n, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j0 = 0; j0 < 8 * NT; j0 += 4) {
      if (j0 >= n) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) red[(q * 8 + g) * kFewPitch + j0 + t] = column(q, j0, t);
    }
  }
  __device__ __forceinline__ void add(float* red, const uint8_t* tok, const float* w, int n, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j0 = 0; j0 < 8 * NT; j0 += 4) {
      if (j0 >= n) break;
      const bool own = j0 + t < n;
      const int to = own ? tok[j0 + t] : 0;
      const float wt = own ? w[to] : 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = column(q, j0, t);
        float* d = red + (q * 8 + g) * kFewPitch + to;
        if (own) *d = fmaf(wt, x, *d);
      }
    }
  }
};

// `n` chunks of the stream times the rows of `ncol` columns; column j has its row at row(j) elements
// behind `rows`; `at`: the first chunk's element.  kH: the rows were written by this launch (read them
// from L2; bf16: their second part lies `lo` elements behind the first).
template <typename T, int NT, bool kH, int P, typename Row>
__device__ __forceinline__ void few_chunks(FewStream<T>& st, uint32_t ring, int& slot, int n, const T* rows, int64_t lo,
                                           int at, int ncol, Row row, FewAcc<T, NT, P>& acc, int lane) {
  const int g = lane >> 2, t = lane & 3;
  constexpr int CE = 64 / sizeof(T);
  // volatile: the compiler would move the loads for the next chunk behind the wait for this one
  auto load = [](const T* s) {
    uint4 v;
    if (kH)
      asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(s) : "memory");
    else
      asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(s) : "memory");
    return v;
  };
  const T* src[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    src[j] = g + 8 * j < ncol ? rows + row(g + 8 * j) + at + t * (16 / (int)sizeof(T)) : nullptr;
  // a lane holds 16 bytes of the columns g and g + 8; those of the next chunk are loaded while this one is
  // multiplied; the parts of H, which come from L2, two chunks ahead (16 tokens 465 -> 457 us; for x,
  // mostly in L1, a second measured slower, and two blocks of columns have no registers for it)
  constexpr int D = kH && NT == 1 ? 2 : 1;
  uint4 xn[D][P][NT];
#pragma unroll
  for (int k = 0; k < D; ++k)
#pragma unroll
    for (int h = 0; h < P; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        xn[k][h][j] = make_uint4(0, 0, 0, 0);
        if (src[j] && k < n) xn[k][h][j] = load(src[j] + h * lo + k * CE);
      }
  for (int i = 0; i < n; ++i) {
    uint4 xb[P][NT];
#pragma unroll
    for (int h = 0; h < P; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        xb[h][j] = xn[0][h][j];
        if (D == 2) xn[0][h][j] = xn[D - 1][h][j];
        if (src[j] && i + D < n) xn[D - 1][h][j] = load(src[j] + h * lo + (i + D) * CE);
      }
    cp_async_wait<kFewDepth - 1>();
    uint4 wq[4];
    const uint32_t from = ring + slot * kFewStage;
#pragma unroll
    for (int q = 0; q < 4; ++q) wq[q] = lds16(from + q * 512);
    slot = slot + 1 == kFewDepth ? 0 : slot + 1;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int h = 0; h < P; ++h)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4& x = xb[h][j];
            mma_bf16(acc.v[h][m][j], wq[2 * m].x, wq[2 * m + 1].x, wq[2 * m].y, wq[2 * m + 1].y, x.x, x.y);
            mma_bf16(acc.v[h][m][j], wq[2 * m].z, wq[2 * m + 1].z, wq[2 * m].w, wq[2 * m + 1].w, x.z, x.w);
          }
    } else {
      // every lane needs every column's bytes: they come from the lane that loaded them, J columns at a
      // time (zeros beyond the last; with four at a time one token of 4 x 1024 x 2688 took 29 us, not 23)
      constexpr int J = NT;
#pragma unroll
      for (int j0 = 0; j0 < 8 * NT; j0 += J) {
        if (j0 >= ncol) break;
        const uint4& x = xb[0][j0 >> 3];
        float xs[J][4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int from_lane = ((j0 + j) & 7) * 4 + t;
          xs[j][0] = __shfl_sync(0xffffffffu, __uint_as_float(x.x), from_lane);
          xs[j][1] = __shfl_sync(0xffffffffu, __uint_as_float(x.y), from_lane);
          xs[j][2] = __shfl_sync(0xffffffffu, __uint_as_float(x.z), from_lane);
          xs[j][3] = __shfl_sync(0xffffffffu, __uint_as_float(x.w), from_lane);
        }
        // four products first, then one addition to the long sum: a quarter of its roundings
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float four = xs[j][0] * __uint_as_float(wq[q].x);
            four = fmaf(xs[j][1], __uint_as_float(wq[q].y), four);
            four = fmaf(xs[j][2], __uint_as_float(wq[q].z), four);
            four = fmaf(xs[j][3], __uint_as_float(wq[q].w), four);
            acc.v[q][j0 + j] += four;
          }
      }
    }
    st.issue(from);  // the stage's values have been used: it may be filled again
  }
}

// Gate/up of one segment: partial sums [32 weight rows][tokens of the entry] into red.
template <typename T, int NT>
__device__ __forceinline__ void few_gate_up(FewStream<T>& st, uint32_t ring, int& slot, const FewSeg& sg, const T* x,
                                            int d, const uint8_t* tok, int ntok, float* red, int lane) {
  FewAcc<T, NT, 1> acc;
  acc.clear();
  few_chunks<T, NT, false>(st, ring, slot, sg.left, x, 0, sg.chunk * (64 / (int)sizeof(T)), ntok,
                           [&](int j) { return (int64_t)tok[j] * d; }, acc, lane);
  acc.store(red, ntok, lane);
}

// Down of one group of 32 output columns: this warp's run over all entries, partial sums
// [32 columns][tokens] of the weighted sum into red (each value is one lane's alone).
template <typename T, int NT>
__device__ __forceinline__ void few_down_segment(FewStream<T>& st, uint32_t ring, int& slot, const FewSeg& sg, const T* H,
                                                 int64_t lo, int f, const uint8_t* tok, const float* w, int ntok,
                                                 float* red, int lane) {
  FewAcc<T, NT, sizeof(T) == 2 ? 2 : 1> acc;
  acc.clear();
  few_chunks<T, NT, true>(st, ring, slot, sg.left, H, lo, sg.chunk * (64 / (int)sizeof(T)), ntok,
                          [&](int j) { return (int64_t)j * f; }, acc, lane);
  acc.add(red, tok, w, ntok, lane);
}
template <typename T>
__device__ __forceinline__ void few_down(FewStream<T>& st, uint32_t ring, int& slot, const FewParams<T>& p,
                                         const FewCtl& c, const FewShare<T>& h, int s, int warp, float* red, int lane) {
  for (int i = lane; i < kFewSlot; i += 32) red[i] = 0.f;
  __syncwarp();
  const int end = h.begin(1, s, warp + 1);
  for (int pos = h.begin(1, s, warp); pos < end;) {
    const FewSeg sg = few_segment(h, 1, s, pos, end);
    const bool shared = c.ent_e[sg.ent] < 0;
    const int f = shared ? p.fs : p.f, ntok = c.ent_n[sg.ent];
    const T* H = (shared ? p.Hs : p.H) + (int64_t)c.ent_row[sg.ent] * f;
    const int64_t lo = sizeof(T) == 2 ? (shared ? p.Hslo - p.Hs : p.Hlo - p.H) : 0;
    const uint8_t* tok = c.ent_tok[sg.ent];
    const float* w = c.ent_w[sg.ent];
    if (ntok <= 8) few_down_segment<T, 1>(st, ring, slot, sg, H, lo, f, tok, w, ntok, red, lane);
    else few_down_segment<T, 2>(st, ring, slot, sg, H, lo, f, tok, w, ntok, red, lane);
    pos += sg.left;
  }
}

// Logits: one task per (expert, tg tokens); a CTA's threads split d, B token rows at a time.
template <typename T, int B>
__device__ __forceinline__ void few_logits(const FewParams<T>& p, FewCtl& c, const uint4* wr, int t0, int nt, int tb) {
  const int nvec = p.d / (16 / (int)sizeof(T)), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + tb) * p.d);
  float acc[B];
#pragma unroll
  for (int i = 0; i < B; ++i) acc[i] = 0.f;
  for (int v = threadIdx.x; v < nvec; v += kFewThreads) {
    const uint4 w = __ldg(wr + v);
    uint4 x[B];
#pragma unroll
    for (int i = 0; i < B; ++i) x[i] = __ldg(xr + (int64_t)(tb + i < nt ? i : 0) * nvec + v);
#pragma unroll
    for (int i = 0; i < B; ++i) acc[i] = dot16(x[i], w, acc[i], p.x);
  }
#pragma unroll
  for (int i = 0; i < B; ++i) {
#pragma unroll
    for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane == 0 && tb + i < nt) c.part[warp][tb + i] = acc[i];
  }
}
template <typename T>
__device__ __forceinline__ void few_router(const FewParams<T>& p, FewCtl& c) {
  const int ntg = (p.T_ + p.tg - 1) / p.tg;
  for (int task = blockIdx.x; task < p.E * ntg; task += gridDim.x) {
    const int e = task / ntg, t0 = (task - e * ntg) * p.tg, nt = min(p.tg, p.T_ - t0);
    const uint4* wr = reinterpret_cast<const uint4*>(p.router_w + (int64_t)e * p.d);
    if (nt <= 2) few_logits<T, 2>(p, c, wr, t0, nt, 0);
    else
      for (int tb = 0; tb < nt; tb += 8) few_logits<T, 8>(p, c, wr, t0, nt, tb);
    __syncthreads();
    if (threadIdx.x < nt) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) s += c.part[w][threadIdx.x];
      p.logits[(int64_t)(t0 + threadIdx.x) * p.E + e] = s + (p.router_b ? __ldg(p.router_b + e) : 0.f);
    }
    __syncthreads();
  }
}

// One warp selects the top-k of one token from its E logits in shared memory: the largest value first,
// lower index on ties.  The values are compared as integers in their order (adding zero makes -0 and 0
// the same value), so that a step is two warp reductions.  A NaN comes after every number and weighs
// nothing beside one (the layer's other selections never take it); it is asked for by itself, since its bits
// after an addition are the compiler's choice.  The experts chosen are distinct whatever the values are.
__device__ __forceinline__ void few_topk(const float* lg, int E, int k, int flags, int lane, int32_t* idx, float* w) {
  constexpr uint32_t kNan = 1u;  // below the key of -infinity
  uint32_t key[kMaxExperts / 32];
#pragma unroll
  for (int m = 0; m < kMaxExperts / 32; ++m) {
    const int e = lane + 32 * m;
    key[m] = 0u;  // no such expert, or chosen already
    if (e < E) {
      const uint32_t b = __float_as_uint(router_clamp(lg[e], flags) + 0.f);
      key[m] = (b & 0x7fffffffu) > 0x7f800000u ? kNan : b & 0x80000000u ? ~b : b | 0x80000000u;
    }
  }
  float den = 0.f, first = 0.f, mine = 0.f;
  int at = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
    int e_best = lane;
#pragma unroll
    for (int m = 1; m < kMaxExperts / 32; ++m)
      if (key[m] > best) {
        best = key[m];
        e_best = lane + 32 * m;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)e_best : 0xffffffffu);
#pragma unroll
    for (int m = 0; m < kMaxExperts / 32; ++m)
      if (e == lane + 32 * m) key[m] = 0u;
    const float v = top == kNan ? -INFINITY : __uint_as_float(top & 0x80000000u ? top & 0x7fffffffu : ~top);
    if (j == 0) first = v;
    const float p = (flags & kRouterRaw) ? v : expf(v - first);
    den += p;
    if (lane == j) {
      mine = p;
      at = e;
    }
  }
  if (lane < k) {
    idx[lane] = at;
    w[lane] = (flags & kRouterRaw) ? mine : mine / den;
  }
}

// Top-k of every token, the touched experts and their tokens (every CTA the same); CTA 0 also
// leaves the routing state in the workspace.
template <typename T>
__device__ __forceinline__ void few_select(const FewParams<T>& p, FewCtl& c, float* lg) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = p.k, E = p.E, T_ = p.T_;
  for (int i = threadIdx.x; i < T_ * E; i += kFewThreads) lg[i] = __ldcg(p.logits + i);
  if (threadIdx.x < kMaxExperts) c.mask[threadIdx.x] = 0;
  __syncthreads();
  if (warp < T_) {
    few_topk(lg + warp * E, E, k, p.flags, lane, c.idx + warp * k, c.w + warp * k);
    __syncwarp();
    if (lane < k) atomicOr(&c.mask[c.idx[warp * k + lane]], 1u << warp);
  }
  __syncthreads();
  // warp w: experts 32 w + lane; rows and touched experts before them by the warps' totals
  const int e = threadIdx.x, shared = p.fs > 0 ? 1 : 0;
  uint32_t m = 0, has = 0;
  int cnt = 0, incl = 0;
  if (warp < kMaxExperts / 32) {
    m = c.mask[e];
    cnt = incl = __popc(m);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += a;
    }
    has = __ballot_sync(0xffffffffu, cnt > 0);
    if (lane == 31) {
      c.warp_rows[warp] = incl;
      c.warp_has[warp] = __popc(has);
    }
  } else if (warp == kMaxExperts / 32 && shared) {
    if (lane == 0) {
      c.ent_e[0] = -1;
      c.ent_row[0] = 0;
      c.ent_n[0] = T_;
    }
    if (lane < kFewMaxT) {
      c.ent_tok[0][lane] = (uint8_t)lane;
      c.ent_w[0][lane] = 1.f;
    }
  }
  __syncthreads();
  if (warp < kMaxExperts / 32) {
    int row = 0, n = shared;
    for (int w = 0; w < warp; ++w) {
      row += c.warp_rows[w];
      n += c.warp_has[w];
    }
    if (e <= E) c.off[e] = row + incl - cnt;
    if (e == kMaxExperts - 1) c.off[kMaxExperts] = row + incl;
    if (lane == 31 && warp == kMaxExperts / 32 - 1) c.n_ent = n + __popc(has);
    if (cnt > 0) {
      const int i = n + __popc(has & ((1u << lane) - 1u));
      c.ent_e[i] = e;
      c.ent_row[i] = row + incl - cnt;
      c.ent_n[i] = cnt;
      c.mask[e] = m | (uint32_t)i << 16;  // the entry beside the tokens
      uint32_t left = m;
      for (int j = 0; left; ++j, left &= left - 1) c.ent_tok[i][j] = (uint8_t)(__ffs(left) - 1);
    }
  }
  __syncthreads();
  if (threadIdx.x < T_ * k) c.ent_w[c.mask[c.idx[threadIdx.x]] >> 16][threadIdx.x / k] = c.w[threadIdx.x];
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= E; i += kFewThreads) {
      p.offsets[i] = c.off[i];
      if (i < E) p.counts[i] = __popc(c.mask[i] & 0xffffu);
    }
    for (int i = threadIdx.x; i < T_ * k; i += kFewThreads) {
      const int t = i / k, ex = c.idx[i], r = c.off[ex] + __popc(c.mask[ex] & ((1u << t) - 1u));
      p.topk_idx[i] = ex;
      p.topk_w[i] = c.w[i];
      p.dst_row[i] = r;
      p.src_row[r] = t;
    }
  }
}

// Barrier over the CTAs of the grid; every CTA arrives exactly once per launch, also after an error.
template <typename T>
__device__ __forceinline__ bool few_barrier(const FewParams<T>& p, FewCtl& c, int i) {
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool was = c.ok != 0;
    const bool got = grid_sync<0>(p.bar + i, gridDim.x, &c.abort);
    if (!got) {
      c.abort = 1;
      atomicOr(p.err, kErrWaitTimeout);
    }
    c.ok = was && got;
  }
  __syncthreads();
  return c.ok != 0;
}

template <typename T>
__global__ void __launch_bounds__(kFewThreads, 1) few_tokens_kernel(const __grid_constant__ FewParams<T> p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem + kFewRing);
  FewCtl& c = *reinterpret_cast<FewCtl*>(smem + kFewRing + kFewRed);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    c.abort = 0;
    c.ok = 1;
  }
  few_router(p, c);
  if (!few_barrier(p, c, 0)) {
    (void)few_barrier(p, c, 1);  // arrivals only: the counters stay in step
    if (p.d < kFewSplitRows * (int)gridDim.x) (void)few_barrier(p, c, 2);
    return;
  }
  few_select(p, c, red);

  const FewShare<T> h(p, c.n_ent);
  const uint32_t ring = smem_u32(smem) + warp * (kFewDepth * kFewStage) + lane * 16;
  FewStream<T> st(p, c, h, warp, lane);
  for (int s = 0; s < kFewDepth; ++s) st.issue(ring + s * kFewStage);
  int slot = 0;

  for (int s = 0; s < h.batches; ++s) {
    const int end = h.begin(0, s, warp + 1);
    for (int pos = h.begin(0, s, warp); pos < end;) {
      const FewSeg sg = few_segment(h, 0, s, pos, end);
      const int ntok = c.ent_n[sg.ent];
      float* mine = red + (sg.tile + warp) * kFewSlot;
      if (ntok <= 8) few_gate_up<T, 1>(st, ring, slot, sg, p.x, p.d, c.ent_tok[sg.ent], ntok, mine, lane);
      else few_gate_up<T, 2>(st, ring, slot, sg, p.x, p.d, c.ent_tok[sg.ent], ntok, mine, lane);
      pos += sg.left;
    }
    __syncthreads();
    // h = silu(g) * u: a thread per column of the batch's tiles, and token
    const int nt = h.batch_tiles(s), all = nt * h.cd;
    for (int i = threadIdx.x; i < nt * 256; i += kFewThreads) {
      const int tile = i >> 8, col = i & 15, n = (i >> 4) & 15;
      const FewSeg sg = few_segment(h, 0, s, tile * h.cd, all);
      if (n >= c.ent_n[sg.ent] || col < sg.lo || col >= sg.hi) continue;
      const int r = (col >> 3) * 16 + (col & 7);
      float gt = 0.f, up = 0.f;
      for (int w = 0; w < kFewWarps; ++w) {
        const int a = all * w / kFewWarps, b = all * (w + 1) / kFewWarps;
        if (max(a, tile * h.cd) < min(b, (tile + 1) * h.cd)) {
          const float* v = red + (tile + w) * kFewSlot + r * kFewPitch + n;
          gt += v[0];
          up += v[8 * kFewPitch];
        }
      }
      const bool shared = c.ent_e[sg.ent] < 0;
      const int f = shared ? p.fs : p.f;
      const int64_t at = (int64_t)(c.ent_row[sg.ent] + n) * f + sg.col + col;
      const float v = silu_mul(gt, up);
      const T hi = from_f32<T>(v);
      (shared ? p.Hs : p.H)[at] = hi;
      if (sizeof(T) == 2)  // nothing is left of an infinity
        (shared ? p.Hslo : p.Hlo)[at] = from_f32<T>(fabsf(to_f32(hi)) < INFINITY ? v - to_f32(hi) : 0.f);
    }
    __syncthreads();
  }

  // H of every CTA is written; the copies of the first W2 chunks are already in flight
  const bool ok = few_barrier(p, c, 1);
  for (int s = 0; ok && s < h.groups; ++s) {
    few_down(st, ring, slot, p, c, h, s, warp, red + warp * kFewSlot, lane);
    __syncthreads();
    const int o = h.o0 + s * kFewRowsW + lane;
    if (warp < p.T_ && o < h.o1) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += red[w * kFewSlot + lane * kFewPitch + warp];
      if (h.teams) p.part[((int64_t)h.split * p.T_ + warp) * p.d + o] = v;
      else p.y[(int64_t)warp * p.d + o] = from_f32<T>(v);
    }
    __syncthreads();
  }
  cp_async_wait<0>();
  if (h.teams && few_barrier(p, c, 2)) {
    const int n = p.T_ * p.d;
    for (int i = blockIdx.x * kFewThreads + threadIdx.x; i < n; i += gridDim.x * kFewThreads) {
      float v = 0.f;
#pragma unroll 8
      for (int s = 0; s < h.splits; ++s) v += __ldcg(p.part + (int64_t)s * n + i);
      p.y[i] = from_f32<T>(v);
    }
  }
}

template <typename T>
cudaError_t launch_few(const FewArgs& a, cudaStream_t s) {
  FewParams<T> p;
  p.x = (const T*)a.x;
  p.router_w = (const T*)a.router_w;
  p.router_b = a.router_b;
  p.W = (const T*)a.W;
  p.wstride = a.wstride;
  p.Ws = (const T*)a.W_sh;
  p.H = (T*)a.H;
  p.Hs = (T*)a.Hs;
  p.Hlo = (T*)a.Hlo;
  p.Hslo = (T*)a.Hslo;
  p.part = a.part;
  p.y = (T*)a.y;
  p.logits = a.logits;
  p.topk_idx = a.topk_idx;
  p.topk_w = a.topk_w;
  p.counts = a.counts;
  p.offsets = a.offsets;
  p.src_row = a.src_row;
  p.dst_row = a.dst_row;
  p.bar = a.bar;
  p.err = a.err;
  p.T_ = a.T;
  p.d = a.d;
  p.f = a.f;
  p.fs = a.fs;
  p.E = a.E;
  p.k = a.k;
  p.flags = a.router_flags;
  // as few tokens per task as lets all tasks run at once
  const int groups = a.sm_count / a.E < 1 ? 1 : (a.sm_count / a.E < a.T ? a.sm_count / a.E : a.T);
  p.tg = (a.T + groups - 1) / groups;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.sm_count);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kFewSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident: the grid barriers need it
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  launch_chain_break();  // an ordinary launch: it must not overlap its neighbours
  const cudaError_t e = cudaLaunchKernelEx(&cfg, few_tokens_kernel<T>, p);
  launch_chain_break();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t configure_few_kernels() {
  cudaError_t e = cudaFuncSetAttribute(few_tokens_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(few_tokens_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmem);
  return e;
}

cudaError_t launch_few_tokens(const FewArgs& a, int act, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  if (a.T > kFewMaxT) return cudaErrorInvalidValue;
  return act == COLIBRI_BF16 ? launch_few<__nv_bfloat16>(a, s) : launch_few<float>(a, s);
}

}  // namespace colibri
