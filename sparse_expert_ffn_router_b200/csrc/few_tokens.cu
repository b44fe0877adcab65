// The whole MoE layer for at most 16 tokens in one cooperative launch (bf16 or fp32 weights, with
// the shared expert): router, top-k, gate/up, down, weighted sum.
//
//   logits[t][e] = x_t . Wr_e + b_e;  the k chosen experts and their weights p (warp_topk)
//   h[t][e]      = silu(W1_e x_t) * (W3_e x_t)
//   y[t]         = sum_(e chosen by t) p[t][e] W2_e h[t][e]  (+ W2_s h_s[t])
//
// With a few tokens every touched expert's weights are read once and meet a few rows, so the work
// is a stream over those weights (2 or 4 bytes per 2 x tokens FLOP) and the bound is HBM.  Three
// phases, two grid barriers between them:
//   router   CTA e (round-robin) forms the logits of expert e for all tokens.
//   gate/up  every CTA selects the experts of all tokens from the logits (the same result in each),
//            then owns an equal share of the gate columns of all touched experts together, whatever
//            expert they fall in.
//   down     every CTA owns an equal share of the output columns, for all touched experts, so the
//            weighted sum is formed where it is needed, in ascending expert order: no third
//            barrier, no atomics, the same bits in every run.
// The shares are split to single columns (a partly filled last tile loads only its own rows), so
// that no CTA reads more than one row above the average.
//
// Inside a CTA the 16 warps split the inner dimension and each keeps its weights in flight through
// a ring of shared memory that the same lane fills (cp.async) and drains: no lane reads what
// another lane copied, so the ring needs no barrier, and a warp's copies run ahead across tiles,
// experts and the barrier between the two projections.  bf16: mma.m16n8k16, weights as the 16-row
// operand (8 gate rows and the 8 up rows of the same columns; for down 16 output columns), tokens
// as the 8 columns; the order of k inside an instruction is free, so a lane's 16 bytes of a weight
// row feed two instructions as they are, and the token operand is 16 bytes of the token's row.
// fp32: FMA on the CUDA cores.  Partial sums of the warps meet in shared memory once per tile, in
// warp order.  H is kept in the activation type between the projections (bf16: rounded once), as
// on the library's other paths.
#include "common.cuh"

namespace colibri {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewDepth = 4;             // ring stages of a warp
constexpr int kFewRowsW = 32;            // weight rows of a tile: 4 per lane
constexpr int kFewStage = 4 * 512;       // bytes of a warp's stage: 4 rows of 16 bytes per lane
constexpr int kFewEntries = kFewMaxT * kMaxTopK + 1;  // touched experts and the shared one
constexpr int kFewPitch = kFewMaxT + 2;  // floats per weight row of the partial sums (16 token columns)

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
  int32_t n_ent;
  int32_t ok;
  int32_t abort;
  float part[kFewWarps][kFewMaxT];       // router partial sums
  float yacc[kFewMaxT][kFewRowsW];
};

constexpr size_t kFewRing = (size_t)kFewWarps * kFewDepth * kFewStage;
constexpr size_t kFewRed = (size_t)kFewWarps * kFewRowsW * kFewPitch * 4;  // one of two
constexpr size_t kFewSmem = kFewRing + 2 * kFewRed + sizeof(FewCtl);
static_assert(kFewSmem <= 232448, "shared memory of the few-token kernel");

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
  T* y;                // [T, d]
  float* logits;       // [T, E]
  int32_t *topk_idx, *counts, *offsets, *src_row, *dst_row;
  float* topk_w;
  int32_t* bar;        // [2]
  uint32_t* err;
  int T_, d, f, fs, E, k, flags;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One CTA's sequence of tiles.  Phase 0 (gate/up): columns [c0, c1) of all entries' gate columns
// laid end to end, in tiles of at most 16 columns of one entry.  Phase 1 (down): output columns
// [o0, o1) in groups of 32, every entry in turn per group.
template <typename T>
struct FewWalk {
  const FewParams<T>& p;
  const FewCtl& c;
  int phase;  // 2: no tiles left
  int ent, col, n;  // current tile: entry, first column, columns
  int64_t c1;       // phase 0: end of the CTA's share, counted from the current entry's column 0
  int o1;

  __device__ FewWalk(const FewParams<T>& p_, const FewCtl& c_) : p(p_), c(c_), phase(0), ent(0) {
    const int G = gridDim.x, b = blockIdx.x;
    const int64_t total = (int64_t)p.fs + (int64_t)(c.n_ent - (p.fs > 0 ? 1 : 0)) * p.f;
    int64_t at = total * b / G;
    c1 = total * (b + 1) / G;
    while (ent < c.n_ent && at >= width()) {
      at -= width();
      c1 -= width();
      ++ent;
    }
    col = (int)at;
    settle();
  }
  __device__ __forceinline__ int width() const { return c.ent_e[ent] < 0 ? p.fs : p.f; }
  __device__ __forceinline__ void settle() {  // phase 0: the tile at (ent, col), or on to phase 1
    if (col >= c1) {
      start_down();
      return;
    }
    n = (int)min((int64_t)min(16, width() - col), c1 - col);
  }
  __device__ __forceinline__ void start_down() {
    phase = 1;
    ent = 0;
    col = (int)((int64_t)p.d * blockIdx.x / gridDim.x);
    o1 = (int)((int64_t)p.d * (blockIdx.x + 1) / gridDim.x);
    if (col >= o1 || c.n_ent == 0) phase = 2;
    else n = min(kFewRowsW, o1 - col);
  }
  __device__ __forceinline__ void next() {
    if (phase == 0) {
      col += n;
      if (col >= width() && c1 > width()) {
        c1 -= width();
        col = 0;
        ++ent;
      }
      settle();
    } else if (phase == 1) {
      if (++ent == c.n_ent) {
        ent = 0;
        col += n;
        if (col >= o1) {
          phase = 2;
          return;
        }
        n = min(kFewRowsW, o1 - col);
      }
    }
  }
  // the tile's inner dimension and this warp's share of it, in chunks of 64 bytes of a row
  __device__ __forceinline__ int inner() const { return phase == 0 ? p.d : (c.ent_e[ent] < 0 ? p.fs : p.f); }
  __device__ __forceinline__ void span(int warp, int& a, int& b) const {
    const int chunks = inner() / (64 / (int)sizeof(T));
    a = chunks * warp / kFewWarps;
    b = chunks * (warp + 1) / kFewWarps;
  }
};

// The weight stream of one lane: 4 rows (q = 0..3) of the walk's current tile, 16 bytes per row
// and chunk.  Gate/up: q & 1 picks W1 or W3, q >> 1 the upper 8 columns; down: 8 columns per q.
template <typename T>
struct FewStream {
  FewWalk<T> walk;
  const T* ptr;
  int64_t s1, s2;  // offsets of q & 1 and q >> 1
  uint32_t live;   // q's whose row exists
  int chunk, end;
  int warp, g, t;

  __device__ FewStream(const FewParams<T>& p, const FewCtl& c, int warp_, int lane)
      : walk(p, c), warp(warp_), g(lane >> 2), t(lane & 3) {
    open();
  }
  __device__ __forceinline__ void open() {  // the first tile from here on in which this warp has chunks
    while (walk.phase < 2) {
      walk.span(warp, chunk, end);
      if (chunk < end) break;
      walk.next();
    }
    if (walk.phase == 2) return;
    const FewParams<T>& p = walk.p;
    const int e = walk.c.ent_e[walk.ent];
    const int64_t f = e < 0 ? p.fs : p.f, d = p.d;
    const T* base = e < 0 ? p.Ws : p.W + (int64_t)e * p.wstride;
    live = 0;
    if (walk.phase == 0) {
      ptr = base + (walk.col + g) * d;
      s1 = f * d;
      s2 = 8 * d;
      live = (g < walk.n ? 3u : 0u) | (g + 8 < walk.n ? 12u : 0u);
    } else {
      ptr = base + 2 * f * d + (walk.col + g) * f;
      s1 = 8 * f;
      s2 = 16 * f;
#pragma unroll
      for (int q = 0; q < 4; ++q) live |= (g + 8 * q < walk.n ? 1u : 0u) << q;
    }
    ptr += (int64_t)chunk * (64 / sizeof(T)) + t * (16 / sizeof(T));
  }
  // copies the next chunk into the stage (nothing once the walk has ended) and closes the group
  __device__ __forceinline__ void issue(uint32_t dst) {
    if (walk.phase < 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (live >> q & 1u) cp_async16(dst + q * 512, ptr + (q & 1) * s1 + (q >> 1) * s2);
      ptr += 64 / sizeof(T);
      if (++chunk == end) {
        walk.next();
        open();
      }
    }
    cp_async_commit();
  }
};

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// One tile of one warp: its partial sums [32 weight rows][ntok] into red.  rows: the token operand's
// rows (x by token in phase 0, H by row in phase 1), this lane's 16 bytes at chunk `a`.
template <typename T, int NT>
__device__ __forceinline__ void few_tile(FewStream<T>& st, uint32_t ring, int& slot, int a, int b, bool down,
                                         const T* rows, int64_t ld, const uint8_t* tok, int ntok, float* red, int lane) {
  const int g = lane >> 2, t = lane & 3;
  constexpr int CE = 64 / sizeof(T);  // elements of a chunk
  if constexpr (sizeof(T) == 2) {
    float acc[2][NT][4] = {};
    const T* src[NT];
    bool has[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      has[j] = g + 8 * j < ntok;
      const int r = has[j] ? (tok ? tok[g + 8 * j] : g + 8 * j) : 0;
      src[j] = rows + r * ld + (int64_t)a * CE + t * 8;
    }
    for (int ch = a; ch < b; ++ch) {
      uint4 xb[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        xb[j] = make_uint4(0, 0, 0, 0);
        if (has[j]) xb[j] = down ? __ldcg(reinterpret_cast<const uint4*>(src[j])) : __ldg(reinterpret_cast<const uint4*>(src[j]));
        src[j] += CE;
      }
      cp_async_wait<kFewDepth - 1>();
      uint4 wq[4];
      const uint32_t at = ring + slot * kFewStage;
#pragma unroll
      for (int q = 0; q < 4; ++q) wq[q] = lds16(at + q * 512);
      slot = slot + 1 == kFewDepth ? 0 : slot + 1;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_bf16(acc[m][j], wq[2 * m].x, wq[2 * m + 1].x, wq[2 * m].y, wq[2 * m + 1].y, xb[j].x, xb[j].y);
          mma_bf16(acc[m][j], wq[2 * m].z, wq[2 * m + 1].z, wq[2 * m].w, wq[2 * m + 1].w, xb[j].z, xb[j].w);
        }
      st.issue(at);  // the stage's values have been used: it may be filled again
    }
    // row q * 8 + g of the tile, token columns 8 j + 2 t and the next
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(red + ((2 * m + h) * 8 + g) * kFewPitch + 8 * j + 2 * t) =
              make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
  } else {
    float acc[4][8 * NT];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 8 * NT; ++j) acc[q][j] = 0.f;
    for (int ch = a; ch < b; ++ch) {
      cp_async_wait<kFewDepth - 1>();
      uint4 wq[4];
      const uint32_t at = ring + slot * kFewStage;
#pragma unroll
      for (int q = 0; q < 4; ++q) wq[q] = lds16(at + q * 512);
      slot = slot + 1 == kFewDepth ? 0 : slot + 1;
#pragma unroll
      for (int j = 0; j < 8 * NT; ++j) {
        if (j < ntok) {
          const uint4* src = reinterpret_cast<const uint4*>(rows + (tok ? tok[j] : j) * ld + (int64_t)ch * CE + t * 4);
          const uint4 xb = down ? __ldcg(src) : __ldg(src);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q][j] = dot16(xb, wq[q], acc[q][j], (const float*)nullptr);
        }
      }
      st.issue(at);  // the stage's values have been used: it may be filled again
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 8 * NT; ++j) {
        acc[q][j] += __shfl_xor_sync(0xffffffffu, acc[q][j], 1);
        acc[q][j] += __shfl_xor_sync(0xffffffffu, acc[q][j], 2);
        if ((j & 3) == t) red[(q * 8 + g) * kFewPitch + j] = acc[q][j];
      }
  }
}

template <typename T>
__device__ __forceinline__ void few_router(const FewParams<T>& p, FewCtl& c) {
  constexpr int V = 16 / sizeof(T);
  const int nvec = p.d / V, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = blockIdx.x; e < p.E; e += gridDim.x) {
    float acc[kFewMaxT];
#pragma unroll
    for (int t = 0; t < kFewMaxT; ++t) acc[t] = 0.f;
    const uint4* wr = reinterpret_cast<const uint4*>(p.router_w + (int64_t)e * p.d);
    for (int v = threadIdx.x; v < nvec; v += kFewThreads) {
      const uint4 w = __ldg(wr + v);
#pragma unroll
      for (int t = 0; t < kFewMaxT; ++t)
        if (t < p.T_) acc[t] = dot16(__ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.d) + v), w, acc[t], p.x);
    }
#pragma unroll
    for (int t = 0; t < kFewMaxT; ++t) {
      if (t >= p.T_) break;
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
      if (lane == 0) c.part[warp][t] = acc[t];
    }
    __syncthreads();
    if (threadIdx.x < p.T_) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) s += c.part[w][threadIdx.x];
      p.logits[(int64_t)threadIdx.x * p.E + e] = s + (p.router_b ? __ldg(p.router_b + e) : 0.f);
    }
    __syncthreads();
  }
}

// Top-k of every token, the touched experts and their tokens (every CTA the same); CTA 0 also
// leaves the routing state in the workspace.
template <typename T>
__device__ __forceinline__ void few_select(const FewParams<T>& p, FewCtl& c, float* lg) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = p.k, E = p.E, T_ = p.T_;
  for (int i = threadIdx.x; i < T_ * E; i += kFewThreads) lg[i] = __ldcg(p.logits + i);
  for (int e = threadIdx.x; e < E; e += kFewThreads) c.mask[e] = 0;
  __syncthreads();
  if (warp < T_) {
    warp_topk(lg + warp * E, E, k, p.flags, lane, c.idx + warp * k, c.w + warp * k);
    __syncwarp();
    if (lane < k) {
      const int e = min(max(c.idx[warp * k + lane], 0), E - 1);
      c.idx[warp * k + lane] = e;
      atomicOr(&c.mask[e], 1u << warp);
    }
  }
  __syncthreads();
  if (warp == 0) {
    int n = p.fs > 0 ? 1 : 0, row = 0;
    if (n && lane == 0) {
      c.ent_e[0] = -1;
      c.ent_row[0] = 0;
      c.ent_n[0] = T_;
    }
    if (n && lane < kFewMaxT) c.ent_tok[0][lane] = (uint8_t)lane;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const uint32_t m = e < E ? c.mask[e] : 0u;
      const int cnt = __popc(m);
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += a;
      }
      const uint32_t has = __ballot_sync(0xffffffffu, cnt > 0);
      if (e < E) c.off[e] = row + incl - cnt;
      if (cnt > 0) {
        const int i = n + __popc(has & ((1u << lane) - 1u));
        c.ent_e[i] = e;
        c.ent_row[i] = row + incl - cnt;
        c.ent_n[i] = cnt;
        uint32_t left = m;
        for (int j = 0; left; ++j, left &= left - 1) c.ent_tok[i][j] = (uint8_t)(__ffs(left) - 1);
      }
      n += __popc(has);
      row += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      c.n_ent = n;
      c.off[E] = row;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e <= E; e += kFewThreads) {
      p.offsets[e] = c.off[e];
      if (e < E) p.counts[e] = __popc(c.mask[e]);
    }
    for (int i = threadIdx.x; i < T_ * k; i += kFewThreads) {
      const int t = i / k, e = c.idx[i], r = c.off[e] + __popc(c.mask[e] & ((1u << t) - 1u));
      p.topk_idx[i] = e;
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
    const bool got = grid_sync(p.bar + i, gridDim.x, &c.abort);
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
  float* red0 = reinterpret_cast<float*>(smem + kFewRing);
  FewCtl& c = *reinterpret_cast<FewCtl*>(smem + kFewRing + 2 * kFewRed);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    c.abort = 0;
    c.ok = 1;
  }
  few_router(p, c);
  if (!few_barrier(p, c, 0)) {
    few_barrier(p, c, 1);
    return;
  }
  few_select(p, c, red0);
  __syncthreads();

  const uint32_t ring = smem_u32(smem) + warp * (kFewDepth * kFewStage) + lane * 16;
  FewStream<T> st(p, c, warp, lane);
  for (int s = 0; s < kFewDepth; ++s) st.issue(ring + s * kFewStage);
  int slot = 0, buf = 0, phase = 0;
  for (FewWalk<T> w(p, c);; w.next()) {
    if (w.phase != phase && phase == 0) {
      // H of every CTA is written; the copies of the first W2 chunks are already in flight
      phase = 1;
      if (!few_barrier(p, c, 1)) break;
    }
    if (w.phase == 2) break;
    const bool down = phase == 1;
    const int e = c.ent_e[w.ent], ntok = c.ent_n[w.ent], row0 = c.ent_row[w.ent];
    const uint8_t* tok = c.ent_tok[w.ent];
    const int f = e < 0 ? p.fs : p.f;
    T* H = (e < 0 ? p.Hs : p.H) + (int64_t)row0 * f;
    if (down && w.ent == 0) c.yacc[threadIdx.x >> 5][lane] = 0.f;
    float* red = red0 + buf * (kFewRed / 4);
    float* mine = red + warp * (kFewRowsW * kFewPitch);
    int a, b;
    w.span(warp, a, b);
    const T* rows = down ? H : p.x;
    const int64_t ld = down ? f : p.d;
    if (ntok <= 8) few_tile<T, 1>(st, ring, slot, a, b, down, rows, ld, down ? nullptr : tok, ntok, mine, lane);
    else few_tile<T, 2>(st, ring, slot, a, b, down, rows, ld, down ? nullptr : tok, ntok, mine, lane);
    __syncthreads();
    if (!down) {
      const int col = threadIdx.x & 15, n = threadIdx.x >> 4;
      if (n < ntok && col < w.n) {
        const int r = (col >> 3) * 16 + (col & 7);
        float gt = 0.f, up = 0.f;
#pragma unroll
        for (int i = 0; i < kFewWarps; ++i) {
          gt += red[(i * kFewRowsW + r) * kFewPitch + n];
          up += red[(i * kFewRowsW + r + 8) * kFewPitch + n];
        }
        H[(int64_t)n * f + w.col + col] = from_f32<T>(silu_mul(gt, up));
      }
    } else {
      const int n = warp;
      if (n < ntok && lane < w.n) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kFewWarps; ++i) v += red[(i * kFewRowsW + lane) * kFewPitch + n];
        const int t = tok[n];
        float wt = 1.f;
        if (e >= 0) {
          for (int j = 0; j < p.k; ++j)
            if (c.idx[t * p.k + j] == e) {
              wt = c.w[t * p.k + j];
              break;
            }
        }
        c.yacc[t][lane] = fmaf(wt, v, c.yacc[t][lane]);
      }
      if (w.ent == c.n_ent - 1) {
        __syncthreads();
        if (warp < p.T_ && lane < w.n) p.y[(int64_t)warp * p.d + w.col + lane] = from_f32<T>(c.yacc[warp][lane]);
      }
    }
    buf ^= 1;
  }
  cp_async_wait<0>();
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
