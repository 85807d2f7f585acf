// Device side of the vocabulary cross entropy (labels instead of a teacher
// cache): row selection by label, GEMM epilogues and per-row kernels around
// the shared GEMM core.
//
//   a = z / T,  z = W h,  q = softmax(a) over all V,  LSE = log sum exp a
//   l_r = (1 - e)(LSE - a_y) + e (LSE - mean_v a_v) + lam LSE^2
//   G_r = k_r [q (1 + 2 lam LSE) - (1 - e) 1_y - e / V]        (d / d a)
//   dH_r = G_r W / T,  dW = sum_r G_r^T h_r / T
// with e = label smoothing, lam = z-loss factor, k_r = the row's weight (or
// upstream gradient); 1 / (T D) is applied in the fp32 epilogues of dH and dW,
// so that the bf16 operand G stays O(k_r).  D = the number of kept rows (mean)
// or 1.
//
// The label's logit is a dot product of its own in fp32 (in the gather), and the
// tiles' sums leave the label out.  The tensor cores cut every partial sum to
// fp32 (256 of them at H = 4096), which moves a logit of 12 by up to 5e-5; in the
// difference LSE - a_y the label would carry that error in full.  So instead
//   nll = log(1 + R), R = sum_{v != y} exp(a_v - a_y),  q_y - 1 = -R / (1 + R),
// which also keeps its relative accuracy where the row is confident (R small).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogues.cuh"
#include "gemm.cuh"
#include "reduce.cuh"

namespace fckl {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kCeWarps = 8;  // rows per block of the warp-per-row kernels

// ---------------------------------------------------------------- rows by label
// A row is kept when its label is not ignore_index and lies in [0, V); another
// label outside [0, V) is recorded as a bad index and the row is left out.
template <class Label>
__device__ __forceinline__ bool ce_keep(const Label* __restrict__ labels, long long i,
                                        long long ignore, int V, bool& bad) {
  const long long y = (long long)labels[i];
  if (y == ignore) return false;
  if (y < 0 || y >= V) { bad = true; return false; }
  return true;
}

// Pass 1 of the two-pass row selection (more than one block): kept rows of
// block b's R rows into ctl->block_count[b].
template <class Label>
__global__ void __launch_bounds__(1024) k_ce_count(const Label* __restrict__ labels, long long N,
                                                   long long R, long long ignore, int V,
                                                   DeviceCtl* ctl) {
  pdl_wait();
  pdl_trigger();
  __shared__ int red[32];
  const long long r0 = blockIdx.x * R, r1 = (r0 + R < N) ? r0 + R : N;
  int c = 0;
  bool bad = false;
  for (long long i = r0 + threadIdx.x; i < r1; i += blockDim.x)
    c += ce_keep(labels, i, ignore, V, bad) ? 1 : 0;
  if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(&ctl->err, kErrBadIndex);
  c = warp_sum_int(c);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = c;
  __syncthreads();
  if (threadIdx.x < 32) {
    c = warp_sum_int(red[threadIdx.x]);
    if (threadIdx.x == 0) ctl->block_count[blockIdx.x] = c;
  }
}

// list = all N rows, the kept ones first (ascending, n of them), the others
// behind them (from the end downwards); n into ctl->n_rows, the divisor D
// (denom, or n when denom is 0) into ctl->n_valid.  One block also counts, and
// starts the control block (no memset ahead of it); several blocks start at
// the sum of pass 1's counts before them.
template <class Label>
__global__ void __launch_bounds__(1024) k_ce_list(const Label* __restrict__ labels, long long N,
                                                  long long R, long long ignore, int V, int denom,
                                                  int32_t* __restrict__ list, DeviceCtl* ctl) {
  pdl_wait();
  pdl_trigger();
  __shared__ int sh[32];
  __shared__ int s_base, s_total;
  const bool alone = gridDim.x == 1;
  if (threadIdx.x == 0) {
    int before = 0, all = 0;
    for (int b = 0; !alone && b < (int)gridDim.x; ++b) {
      const int cb = ctl->block_count[b];
      before += b < (int)blockIdx.x ? cb : 0;
      all += cb;
    }
    s_base = before;
    s_total = all;
  }
  __syncthreads();
  int base = s_base;
  bool bad = false;
  const long long r0 = blockIdx.x * R, r1 = (r0 + R < N) ? r0 + R : N;
  for (long long t0 = r0; t0 < r1; t0 += 4 * (long long)blockDim.x) {
    const long long i0 = t0 + 4 * (long long)threadIdx.x;
    int f = 0;  // bit k: row i0 + k is kept
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k < r1 && ce_keep(labels, i0 + k, ignore, V, bad)) f |= 1 << k;
    int tile_total;
    int pos = base + block_exclusive_scan(__popc(f), sh, &tile_total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long i = i0 + k;
      if (i >= r1) break;
      if (f & (1 << k)) list[pos++] = (int32_t)i;
      else list[N - 1 - (i - pos)] = (int32_t)i;  // i - pos rows before i are left out
    }
    base += tile_total;
  }
  const bool any_bad = __syncthreads_or(bad) != 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const int n = alone ? base : s_total;
    if (alone) {
      ctl->err = any_bad ? kErrBadIndex : 0u;
      ctl->timeout_site = 0u;
      ctl->ticket = 0u;
    }
    ctl->n_rows = n;
    ctl->n_valid = denom > 0 ? denom : n;
  }
}

// Copies H/8 vectors of a hidden row and returns, on thread 0, its dot product
// with the label's row of W, both by a block of 128 threads.
__device__ __forceinline__ float copy_and_dot(const __nv_bfloat16* __restrict__ src,
                                              const __nv_bfloat16* __restrict__ wrow,
                                              __nv_bfloat16* __restrict__ dst, int H) {
  __shared__ float red[4];
  float2 s = both(0.f);
  for (int j = threadIdx.x; j < H / 8; j += 128) {
    Raw8<__nv_bfloat16> a, b;
    a.load(src + 8 * j);
    b.load(wrow + 8 * j);
    reinterpret_cast<uint4*>(dst)[j] = a.a;
    float2 x[4], y[4];
    a.get(x);
    b.get(y);
#pragma unroll
    for (int k = 0; k < 4; ++k) s = fma2(x[k], y[k], s);
  }
  const float t = warp_sum(s.x + s.y);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// One chunk's kept rows, gathered: hidden row -> hst[i], label -> lab[i], the
// label's logit -> zlab[i], the row's factor (weight, upstream gradient, or 1) ->
// kw[i], and, when the caller gives the log-sum-exps, log2(e) times them ->
// lse2[i].  The 64 rows behind the last one get zero hidden rows: the dW GEMM
// reads whole blocks of 64 rows.  (Gathering, instead of masking in place, keeps
// what a left-out row holds -- NaN, say -- away from the products.)
template <class Label>
__global__ void __launch_bounds__(128)
    k_ce_gather(const int32_t* __restrict__ list, RowCount rc, int H,
                const __nv_bfloat16* __restrict__ hidden, const __nv_bfloat16* __restrict__ W,
                const Label* __restrict__ labels, const float* __restrict__ factor,
                const float* __restrict__ lse, __nv_bfloat16* __restrict__ hst,
                int* __restrict__ lab, float* __restrict__ zlab, float* __restrict__ kw,
                float* __restrict__ lse2) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int n = rc.get();
  if (i >= n + 64) return;
  __nv_bfloat16* dst = hst + (size_t)i * H;
  if (i >= n) {
    for (int j = threadIdx.x; j < H / 8; j += 128)
      reinterpret_cast<uint4*>(dst)[j] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int r = list[i], y = (int)labels[r];
  const float z = copy_and_dot(hidden + (size_t)r * H, W + (size_t)y * H, dst, H);
  if (threadIdx.x == 0) {
    lab[i] = y;
    zlab[i] = z;
    kw[i] = factor ? factor[r] : 1.f;
    if (lse) lse2[i] = lse[r] * kLog2e;
  }
}

// Selection and gathering in one launch, for calls of one chunk and few rows:
// block r counts the kept labels before its row, and all of them, by itself
// (N labels a block), so that row r's place in the list and in hst is known.
template <class Label>
__global__ void __launch_bounds__(128)
    k_ce_select(const Label* __restrict__ labels, int N, long long ignore, int V, int denom,
                int32_t* __restrict__ list, DeviceCtl* ctl, int H,
                const __nv_bfloat16* __restrict__ hidden, const __nv_bfloat16* __restrict__ W,
                const float* __restrict__ factor, const float* __restrict__ lse,
                __nv_bfloat16* __restrict__ hst, int* __restrict__ lab, float* __restrict__ zlab,
                float* __restrict__ kw, float* __restrict__ lse2) {
  __shared__ int red[2][4];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  int before = 0, n = 0;
  bool bad = false;
  for (int i = threadIdx.x; i < N; i += 128) {
    const int k = ce_keep(labels, i, ignore, V, bad) ? 1 : 0;
    n += k;
    before += i < r ? k : 0;
  }
  before = warp_sum_int(before);
  n = warp_sum_int(n);
  if ((threadIdx.x & 31) == 0) {
    red[0][threadIdx.x >> 5] = before;
    red[1][threadIdx.x >> 5] = n;
  }
  bad = __syncthreads_or(bad) != 0;
  before = red[0][0] + red[0][1] + red[0][2] + red[0][3];
  n = red[1][0] + red[1][1] + red[1][2] + red[1][3];
  const long long y = (long long)labels[r];
  bool unused = false;
  const bool keep = ce_keep(labels, r, ignore, V, unused);
  const int i = keep ? before : N - 1 - (r - before);
  if (threadIdx.x == 0) {
    list[i] = r;
    if (keep) {
      lab[i] = (int)y;
      kw[i] = factor ? factor[r] : 1.f;
      if (lse) lse2[i] = lse[r] * kLog2e;
    }
    if (r == 0) {
      ctl->err = bad ? kErrBadIndex : 0u;
      ctl->timeout_site = 0u;
      ctl->ticket = 0u;
      ctl->n_rows = n;
      ctl->n_valid = denom > 0 ? denom : n;
    }
  }
  if (i >= n + 64) return;
  __nv_bfloat16* dst = hst + (size_t)i * H;
  if (!keep) {
    for (int j = threadIdx.x; j < H / 8; j += 128)
      reinterpret_cast<uint4*>(dst)[j] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const float z = copy_and_dot(hidden + (size_t)r * H, W + (size_t)y * H, dst, H);
  if (threadIdx.x == 0) zlab[i] = z;
}

// ---------------------------------------------------------------- few rows
constexpr int kFewCols = 32;  // vocabulary columns per block of k_ce_few
constexpr int kFewRows = 2;   // rows of a chunk that take it

// 16 bytes that are read once: not kept in L1.
__device__ __forceinline__ uint4 load_once(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Forward of up to kRows rows: what EpiCe leaves, per 32 columns instead of 128.
// W is streamed once, a warp taking four of its rows at a time with kAhead
// 16-byte vectors of each on their way; the hidden rows come from L1.  The sums
// are fp32 products in pairs, so nothing is cut and scale2 is the plain log2(e) / T.
// W does not depend on the kernel ahead (which selects the rows): its first loads
// do not wait for it.  Bound by HBM: 4096 x 128256 in 153 us, 6.9 TB/s.  kAhead = 1, 2,
// 4: one row 162, 157, 159 us, two rows 175, 184, 170.
template <int kRows, int kAhead, bool kSum>
__global__ void __launch_bounds__(256)
    k_ce_few(RowCount rc, int cap, int H, int V, int NP, float scale2,
             const __nv_bfloat16* __restrict__ hst, const __nv_bfloat16* __restrict__ W,
             const int* __restrict__ lab, float2* __restrict__ partials,
             float* __restrict__ zsum) {
  constexpr int kCols = kFewCols / 8;
  __shared__ float z_sh[kRows][kFewCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kFewCols, nv = H / 8;
  const __nv_bfloat16* wr[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    wr[c] = W + (size_t)min((long long)n0 + warp * kCols + c, (long long)V - 1) * H;
  uint4 w[kAhead][kCols];
  auto fetch = [&](int u, int j) {
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      w[u][c] = j < nv ? load_once(wr[c] + 8 * (size_t)j) : make_uint4(0u, 0u, 0u, 0u);
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fetch(u, 32 * u + lane);
  pdl_wait();
  pdl_trigger();
  const int n = rc.get();
  if (n <= 0) return;
  float2 acc[kCols][kRows];
#pragma unroll
  for (int c = 0; c < kCols; ++c)
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[c][r] = both(0.f);
  for (int j0 = lane; j0 - lane < nv; j0 += 32 * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + 32 * u;
      float2 x[kCols][4];
#pragma unroll
      for (int c = 0; c < kCols; ++c) Raw8<__nv_bfloat16>{w[u][c]}.get(x[c]);
      fetch(u, j + 32 * kAhead);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        Raw8<__nv_bfloat16> h{make_uint4(0u, 0u, 0u, 0u)};
        if (j < nv) h.load(hst + (size_t)min(r, cap - 1) * H + 8 * (size_t)j);
        float2 y[4];
        h.get(y);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[c][r] = fma2(x[c][k], y[k], acc[c][r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const float t = warp_sum(acc[c][r].x + acc[c][r].y);
      if (lane == 0) z_sh[r][warp * kCols + c] = t;
    }
  __syncthreads();
  if (warp >= kRows || warp >= n) return;
  const long long col = (long long)n0 + lane;
  const float z = z_sh[warp][lane];
  const bool in = col < V, counts = in && col != lab[warp];  // the label's column is left out
  const float m = warp_max(counts ? z * scale2 : -INFINITY);
  const float ref = m == -INFINITY ? 0.f : m;
  const float s = warp_sum(counts ? ex2_approx(fmaf(z, scale2, -ref)) : 0.f);
  const float u = kSum ? warp_sum(in ? z : 0.f) : 0.f;
  if (lane == 0) {
    partials[(size_t)warp * NP + blockIdx.x] = make_float2(m, s);
    if (kSum) zsum[(size_t)warp * NP + blockIdx.x] = u;
  }
}

// ---------------------------------------------------------------- epilogues
// All with eight warps: a thread owns one accumulator row and one half (128
// columns) of the tile, so that two warps take turns on each SM quarter's
// special-function unit and hide each other's waits (a step of 1531 x 1024 x
// 50257: 498 us with four warps, 476 with eight).  What bounds a logits GEMM:
// the tensor cores from H = 512 on, below that this epilogue -- 4096 x 256 x 50257
// takes 109 us against 46 for its products and 61 for the main loop alone.  The
// half's results leave as partials of their own: [rows, NP], NP = 2 per vocab
// tile.  One 4 KB staging buffer a warp (as in epilogues.cuh) keeps the operand
// stages' room.

// Waits until the warp's staging buffer is no longer read by its last store.
__device__ __forceinline__ void stage_reuse(int lane) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
}

// max over the first `cols` of 32 values, in four chains.
__device__ __forceinline__ float max32(const float (&v)[32], int cols) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (cols >= 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j) m[j & 3] = fmaxf(m[j & 3], v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) m[j & 3] = j < cols ? fmaxf(m[j & 3], v[j]) : m[j & 3];
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// v = 2^(v scale2 - ref) for the first `cols` values, 0 behind; returns the sum.
__device__ __forceinline__ float exp32(float (&v)[32], float scale2, float ref, int cols) {
  const float2 sc = both(scale2), mr = both(-ref);
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float2 a = fma2(make_float2(v[j], v[j + 1]), sc, mr);
    v[j] = ex2_approx(a.x);
    v[j + 1] = ex2_approx(a.y);
  }
  if (cols < 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = j < cols ? v[j] : 0.f;
  }
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 32; ++j) s[j & 3] += v[j];
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ float sum32(const float (&v)[32], int cols) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (cols >= 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j & 3] += v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j & 3] += j < cols ? v[j] : 0.f;
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// The label's column out of the maximum and the sum: -inf in its place.
__device__ __forceinline__ void leave_out(float (&v)[32], int at) {
  if ((unsigned)at < 32u) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = j == at ? -INFINITY : v[j];
  }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Forward: per row and half tile, (max, sum 2^(a2 - max)) of a2 = z log2(e) / T
// over the columns but the label, and (kSum) the half's sum of z for label
// smoothing.  The logits are not written.
template <bool kSum>
struct EpiCe {
  static constexpr int kEpiWarps = 8;
  static constexpr uint32_t kSmemBytes = 0;
  static constexpr bool kUsesMapC = false;
  struct Params {
    int V, NP;
    float scale2;          // log2(e) / T (and the cut sums' share)
    const int* lab;        // [rows]
    float2* partials;      // [rows, NP]
    float* zsum;           // [rows, NP] (kSum)
  };
  struct State {};
  static __device__ void init(const Params&, State&, uint8_t*, int) {}
  static __device__ void tile(const Params& p, State&, const Work& w, uint32_t taddr, int r,
                              const CUtensorMap*, int, int) {
    const int row = w.m0 + r, n0 = w.n0 + w.half * 128;
    const bool rv = row < w.rows;
    const int y = rv ? __ldg(p.lab + row) - n0 : -1;  // the label's column in the half
    float m = -INFINITY, s = 0.f, u = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float v[32];
      tmem_ld32_conv(taddr + (uint32_t)(w.half * 128 + c * 32), v);
      const int cols = rv ? p.V - (n0 + c * 32) : 0;
      if (cols <= 0) continue;
      if (kSum) u += sum32(v, cols);
      leave_out(v, y - 32 * c);
      const float nm = fmaxf(m, max32(v, cols) * p.scale2);
      const float ref = nm == -INFINITY ? 0.f : nm;  // a slice of -inf only adds 0, not NaN
      s = s * ex2_approx(m - ref) + exp32(v, p.scale2, ref, cols);
      m = nm;
    }
    const int t = 2 * w.nt + w.half;
    if (rv) {
      p.partials[(size_t)row * p.NP + t] = make_float2(m, s);
      if (kSum) p.zsum[(size_t)row * p.NP + t] = u;
    }
  }
  static __device__ void finish(const Params&, State&, int) {}
};

// Forward of a call that also wants gradients: as EpiCe, and the exponentials
// themselves are kept, E = 2^(a2 - m) per half tile with m = (the row's maximum
// in it) - 15, as fp16 in the chunk's [rows, Vp] block; k_ce_dlogits turns them
// into dlogits in place once the row's LSE is known.  So the backward needs no
// second logits product (6 H V flops per row instead of 8, for 4 V more bytes:
// at H = 4096 the product costs about 10 times what the bytes do).
// fp16 because E is rounded here and G once more in k_ce_dlogits: 2^-11 against
// G's own 2^-8; in bf16 the two roundings would add up.  With the offset of 15
// the largest E is 2^15 and E stays normal down to 2^-29 of it.
// The accumulator is read twice (maximum, then exponentials).
template <bool kSum>
struct EpiCeStore {
  static constexpr int kEpiWarps = 8;
  static constexpr uint32_t kSmemBytes = 8 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: [rows, Vp] 16-bit, box {64, 32}
  struct Params {
    int V, NP;
    float scale2;
    const int* lab;
    float2* partials;      // [rows, NP] (m, sum of E before rounding)
    float* zsum;
    int store_rows;        // rows of the store map
  };
  struct State {
    uint8_t* buf;
  };
  static __device__ void init(const Params&, State& st, uint8_t* smem_warp, int) {
    st.buf = smem_warp;
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int r,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int row = w.m0 + r, n0 = w.n0 + w.half * 128;
    const uint32_t ta = taddr + (uint32_t)(w.half * 128);
    const bool rv = row < w.rows;
    const int y = rv ? __ldg(p.lab + row) - n0 : -1;
    float top = -INFINITY, u = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float v[32];
      tmem_ld32_conv(ta + (uint32_t)(c * 32), v);
      const int cols = rv ? p.V - (n0 + c * 32) : 0;
      if (kSum) u += sum32(v, cols);
      leave_out(v, y - 32 * c);
      top = fmaxf(top, max32(v, cols));
    }
    const float m = fmaf(top, p.scale2, -15.f);
    const float ref = m == -INFINITY ? 0.f : m;  // a half of -inf only adds 0, not NaN
    float s = 0.f;
    const int y0 = w.m0 + quarter * 32;
    // rows behind the last one, up to the next multiple of 64, are stored as
    // zeros (the dW GEMM reads whole blocks of 64 rows)
    const int y_end = min((w.rows + 63) & ~63, p.store_rows);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int base = n0 + c * 64;
      const int cols = rv ? p.V - base : 0;
      stage_reuse(lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_ld32_conv(ta + (uint32_t)(c * 64 + h * 32), v);
        leave_out(v, y - 64 * c - 32 * h);
        s += exp32(v, p.scale2, ref, cols - 32 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *stage_chunk(st.buf, lane, 4 * h + j) =
              make_uint4(pack_half2(v[8 * j], v[8 * j + 1]), pack_half2(v[8 * j + 2], v[8 * j + 3]),
                         pack_half2(v[8 * j + 4], v[8 * j + 5]),
                         pack_half2(v[8 * j + 6], v[8 * j + 7]));
      }
      stage_release();
      if (lane == 0) {  // one group per slice, empty when the slice lies outside the map
        if (base < p.V && y0 < y_end) tma_store_2d(mapC, smem_u32(st.buf), base, y0);
        bulk_commit();
      }
    }
    const int t = 2 * w.nt + w.half;
    if (rv) {
      p.partials[(size_t)row * p.NP + t] = make_float2(m, s);
      if (kSum) p.zsum[(size_t)row * p.NP + t] = u;
    }
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// k [q_y (1 + zl) - (1 - e) - e / V] from q1 = q_y - 1, zl = 2 lam LSE and
// base = k e / V.
__device__ __forceinline__ float ce_label_grad(float k, float q1, float zl, float smooth,
                                               float base) {
  return fmaf(k, fmaf(q1, 1.f + zl, zl + smooth), -base);
}

// What bf16 cuts off the label's entry.  That entry carries most of a row's
// gradient, so k_ce_dh_out adds the rest times the label's row of W in fp32.
__device__ __forceinline__ float bf16_rest(float g) {
  return g - __bfloat162float(__float2bfloat16_rn(g));
}

// Backward without the forward's exponentials (the row-gradient call):
// recomputed z tile -> G (see the top), rounded once to bf16 and TMA-stored to
// the chunk's [rows, Vp] block.  Columns in [V, Vp) and the rows behind the last
// one, up to the next multiple of 64, are stored as zeros.
struct EpiCeDlogits {
  static constexpr int kEpiWarps = 8;
  static constexpr uint32_t kSmemBytes = 8 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: [rows, Vp] bf16, box {64, 32}
  struct Params {
    int V;
    float scale2;          // log2(e) / T (and the cut sums' share)
    float label_scale2;    // log2(e) / T
    float smooth;          // label smoothing e
    float zloss2;          // 2 lam
    const int* lab;        // [rows]
    const float* kw;       // [rows] k_r
    const float* zlab;     // [rows] z at the label
    const float* lse2;     // [rows] log2(e) LSE
    float* rest;           // [rows] bf16_rest of the label's entry
    int store_rows;        // rows of the store map
  };
  struct State {
    uint8_t* buf;
  };
  static __device__ void init(const Params&, State& st, uint8_t* smem_warp, int) {
    st.buf = smem_warp;
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int r,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int row = w.m0 + r, n0 = w.n0 + w.half * 128;
    const uint32_t ta = taddr + (uint32_t)(w.half * 128);
    const bool rv = row < w.rows;
    const float kw = rv ? p.kw[row] : 0.f;
    const float lse2 = rv ? p.lse2[row] : 0.f;
    const int y = rv ? p.lab[row] - n0 : -1;
    const float kap = kw * fmaf(p.zloss2, lse2 * kLn2, 1.f);
    const float base_mass = kw * p.smooth / (float)p.V;
    float g_y = 0.f;  // the label's entry
    if ((unsigned)y < 128u) {
      const float q1 = expm1f(fmaf(p.zlab[row], p.label_scale2, -lse2) * kLn2);  // q_y - 1
      g_y = ce_label_grad(kw, q1, p.zloss2 * lse2 * kLn2, p.smooth, base_mass);
      p.rest[row] = bf16_rest(g_y);
    }
    const int y0 = w.m0 + quarter * 32;
    const int y_end = min((w.rows + 63) & ~63, p.store_rows);
    const float2 sc = both(p.scale2), ml = both(-lse2), kk = both(kap), nb = both(-base_mass);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int base = n0 + c * 64;
      stage_reuse(lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_ld32_conv(ta + (uint32_t)(c * 64 + h * 32), v);
        const int cols = rv ? p.V - base - 32 * h : 0, yc = y - c * 64 - 32 * h;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 a = fma2(make_float2(v[j], v[j + 1]), sc, ml);
          const float2 g = fma2(kk, make_float2(ex2_approx(a.x), ex2_approx(a.y)), nb);
          v[j] = g.x;
          v[j + 1] = g.y;
        }
        if ((unsigned)yc < 32u) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = j == yc ? g_y : v[j];
        }
        if (cols < 32) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = j < cols ? v[j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *stage_chunk(st.buf, lane, 4 * h + j) = make_uint4(
              pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
              pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
      }
      stage_release();
      if (lane == 0) {
        if (base < p.V && y0 < y_end) tma_store_2d(mapC, smem_u32(st.buf), base, y0);
        bulk_commit();
      }
    }
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// What the three gradient epilogues share: alpha = 1 / (T D) and the staging.
struct CeGradState {
  float alpha;
  uint8_t* buf;
  __device__ void init(float invT, const DeviceCtl* ctl, uint8_t* smem_warp) {
    const int nv = ctl->n_valid;
    alpha = nv > 0 ? invT / (float)nv : 0.f;
    buf = smem_warp;
  }
  // alpha * the half's accumulator as fp32, 32 columns at a time, to (x, y) of
  // the map (stored, or added in place).
  __device__ __forceinline__ void put_fp32(uint32_t ta, const CUtensorMap* map, bool add, int x0,
                                           int x_end, int y, bool y_ok, int lane) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float v[32];
      tmem_ld32_conv(ta + (uint32_t)(c * 32), v);
      stage_reuse(lane);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *stage_chunk(buf, lane, j) =
            make_uint4(__float_as_uint(alpha * v[4 * j]), __float_as_uint(alpha * v[4 * j + 1]),
                       __float_as_uint(alpha * v[4 * j + 2]), __float_as_uint(alpha * v[4 * j + 3]));
      stage_release();
      const int x = x0 + c * 32;
      if (lane == 0) {
        if (x < x_end && y_ok) {
          if (add) tma_reduce_add_2d(map, smem_u32(buf), x, y);
          else tma_store_2d(map, smem_u32(buf), x, y);
        }
        bulk_commit();
      }
    }
  }
};

// dH partials: the fp32 tile of k segment ks is stored to its own slab (rows
// [ks * 256 * MT, ...) of the slab array), not added in place, so that the sum
// over the segments has one order and repeated calls give the same bits.
struct EpiCeDH {
  static constexpr int kEpiWarps = 8;
  static constexpr uint32_t kSmemBytes = 8 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: slabs [S * 256 * MT, H] fp32, box {32, 32}
  struct Params {
    int H;
    float invT;
    const DeviceCtl* ctl;
  };
  using State = CeGradState;
  static __device__ void init(const Params& p, State& st, uint8_t* smem_warp, int) {
    st.init(p.invT, p.ctl, smem_warp);
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int y = w.m0 + quarter * 32, pitch = (w.rows + PM - 1) / PM * PM;
    st.put_fp32(taddr + (uint32_t)(w.half * 128), mapC, false, w.n0 + w.half * 128, p.H,
                w.ks * pitch + y, y < w.rows, lane);
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// dW of several chunks, summed in fp32: stored by the first chunk, added to in
// place by later ones (one tile a launch, so in the chunks' order).  For bf16
// gradients (out != nullptr) the last chunk that has rows -- the device knows
// which -- instead adds the sum so far to its accumulator, rounds once and writes
// dW; a pass of its own over the sum took 530 us at V = 128256, H = 4096.
struct EpiCeDWSum {
  static constexpr int kEpiWarps = 8;
  static constexpr uint32_t kSmemBytes = 8 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: the fp32 sum [V, H], box {32, 32}
  struct Params {
    int V, H;
    float invT;
    int accumulate;
    const DeviceCtl* ctl;
    int rows_end;               // rows of the call up to and with this chunk
    const float* sum;           // [V, H]
    __nv_bfloat16* out;         // [V, H], or nullptr
  };
  struct State : CeGradState {
    bool last;
  };
  static __device__ void init(const Params& p, State& st, uint8_t* smem_warp, int) {
    st.CeGradState::init(p.invT, p.ctl, smem_warp);
    st.last = p.out != nullptr && p.ctl->n_rows <= p.rows_end;
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int y = w.m0 + quarter * 32, x0 = w.n0 + w.half * 128;
    const uint32_t ta = taddr + (uint32_t)(w.half * 128);
    if (!st.last) {
      st.put_fp32(ta, mapC, p.accumulate != 0, x0, p.H, y, y < p.V, lane);
      return;
    }
    const bool have = p.accumulate && y + lane < p.V;
    const float* row = p.sum + (size_t)(have ? y + lane : 0) * p.H;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int x = x0 + c * 64;
      __syncwarp();  // the slice before has been read from the buffer
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float4 q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = x + h * 32 + 4 * j;
          q[j] = have && col < p.H ? *reinterpret_cast<const float4*>(row + col)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float v[32];
        tmem_ld32_conv(ta + (uint32_t)(c * 64 + h * 32), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[4 * j] = fmaf(st.alpha, v[4 * j], q[j].x);
          v[4 * j + 1] = fmaf(st.alpha, v[4 * j + 1], q[j].y);
          v[4 * j + 2] = fmaf(st.alpha, v[4 * j + 2], q[j].z);
          v[4 * j + 3] = fmaf(st.alpha, v[4 * j + 3], q[j].w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *stage_chunk(st.buf, lane, 4 * h + j) =
              make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                         pack_bf16x2(v[8 * j + 4], v[8 * j + 5]),
                         pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // 4 rows of 128 bytes per store
        const int rr = 4 * i + (lane >> 3), ch = lane & 7;
        const uint4 q = *reinterpret_cast<const uint4*>(st.buf + rr * 128 + ((ch ^ (rr & 7)) << 4));
        if (y + rr < p.V && x + 8 * ch < p.H)
          *reinterpret_cast<uint4*>(p.out + (size_t)(y + rr) * p.H + x + 8 * ch) = q;
      }
    }
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// dW written once, rounded once to bf16 (calls of one chunk).
struct EpiCeDW {
  static constexpr int kEpiWarps = 8;
  static constexpr uint32_t kSmemBytes = 8 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: dW [V, H] bf16, box {64, 32}
  struct Params {
    int V, H;
    float invT;
    const DeviceCtl* ctl;
  };
  using State = CeGradState;
  static __device__ void init(const Params& p, State& st, uint8_t* smem_warp, int) {
    st.init(p.invT, p.ctl, smem_warp);
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int y = w.m0 + quarter * 32;
    const float al = st.alpha;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int x = w.n0 + w.half * 128 + c * 64;
      stage_reuse(lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_ld32_conv(taddr + (uint32_t)(w.half * 128 + c * 64 + h * 32), v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *stage_chunk(st.buf, lane, 4 * h + j) =
              make_uint4(pack_bf16x2(al * v[8 * j], al * v[8 * j + 1]),
                         pack_bf16x2(al * v[8 * j + 2], al * v[8 * j + 3]),
                         pack_bf16x2(al * v[8 * j + 4], al * v[8 * j + 5]),
                         pack_bf16x2(al * v[8 * j + 6], al * v[8 * j + 7]));
      }
      stage_release();
      if (lane == 0) {
        if (x < p.H && y < p.V) tma_store_2d(mapC, smem_u32(st.buf), x, y);
        bulk_commit();
      }
    }
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// ---------------------------------------------------------------- row kernels
// loss = sum of the rows' shares / D, by whichever block of the call's row
// kernels finishes last (ctl->ticket counts them to `blocks`), in fp64 and in
// an order that does not depend on which it is.  Called by all 256 threads.
__device__ __forceinline__ void ce_finish_loss(const float* share, long long N, DeviceCtl* ctl,
                                               unsigned blocks, float* loss) {
  __shared__ double red[8];
  __shared__ bool s_last;
  __threadfence();  // this block's shares before its ticket
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&ctl->ticket, 1u) + 1u == blocks;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double s = 0.0;
#pragma unroll 8
  for (long long i = threadIdx.x; i < N; i += 256) s += (double)__ldcg(share + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) s += red[w];
    const int n = ctl->n_valid;
    *loss = ctl->n_rows > 0 && n > 0 ? (float)(s / (double)n) : 0.f;
  }
}

// A row from its merged partials over the columns but the label: S 2^M (base 2),
// the label's exponent a2 = z_y log2(e) / T, and the mean of a_v (smoothing).  The
// LSE is formed from the larger side: from a label far below the others it would
// take over ulp(a_y), 6e-5 at a_y = -1000, and no number at -inf, where only the
// loss is infinite.
struct CeRow {
  float L2, lse, nll, loss, q1;  // log2(e) LSE, LSE, LSE - a_y, l_r, q_y - 1
  __device__ __forceinline__ CeRow(float M, float S, float a2, float mean, float smooth,
                                   float zloss) {
    const float t = M + log2f(S), x = t - a2;  // log2 R; -inf when the label is alone
    // beyond 2^24 the 1 in 1 + R is below R's last bit
    const float R = exp2f(x);
    nll = x > 24.f ? x * kLn2 : log1pf(R);
    if (!(a2 < INFINITY)) nll = NAN;  // an overflowed label logit is no certainty
    q1 = x > 24.f ? exp2f(-x) - 1.f : -R / (1.f + R);
    const float big = x > 0.f ? t : a2, more = x > 0.f ? log1pf(exp2f(-x)) : nll;
    lse = fmaf(big, kLn2, more);
    L2 = fmaf(more, kLog2e, big);
    loss = smooth > 0.f ? fmaf(1.f - smooth, nll, smooth * (lse - mean)) : nll;
    if (zloss > 0.f) loss = fmaf(zloss * lse, lse, loss);
  }
};

// Max and sum of a row's partials (and its sum of z), on all threads of the row:
// a warp, or a block of 256 threads.
struct CeMerged {
  float M, S, Z;
};
template <bool kBlockRow>
__device__ __forceinline__ CeMerged ce_merge_row(const float2* __restrict__ pr,
                                                 const float* __restrict__ zr, int NP) {
  constexpr int kThreads = kBlockRow ? 256 : 32;
  const int tid = threadIdx.x % kThreads;
  float M = -INFINITY, S = 0.f, Z = 0.f;
#pragma unroll 4
  for (int t = tid; t < NP; t += kThreads) {
    const float2 q = pr[t];
    const float nm = fmaxf(M, q.x);
    const float ref = nm == -INFINITY ? 0.f : nm;
    S = S * exp2f(M - ref) + q.y * exp2f(q.x - ref);
    M = nm;
    if (zr) Z += zr[t];
  }
  const float Mw = warp_max(M);
  S = warp_sum(S * exp2f(M - (Mw == -INFINITY ? 0.f : Mw)));
  if (zr) Z = warp_sum(Z);
  if constexpr (!kBlockRow) return CeMerged{Mw, S, Z};
  __shared__ float red[3][8];
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) { red[0][warp] = Mw; red[1][warp] = S; red[2][warp] = Z; }
  __syncthreads();
  CeMerged m{red[0][0], 0.f, 0.f};
#pragma unroll
  for (int k = 1; k < 8; ++k) m.M = fmaxf(m.M, red[0][k]);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    m.S += red[1][k] * exp2f(red[0][k] - (m.M == -INFINITY ? 0.f : m.M));
    m.Z += red[2][k];
  }
  return m;
}

// Merges the tile partials of each row into its LSE and row loss.  All rows of
// the chunk's part of the list write the caller's row loss and LSE (0 for
// left-out rows) and their share k_r l_r of the loss (list order); lse2 (if
// given) is for the recompute GEMM.  One warp per row, or, when the rows are too
// few to fill the SMs so, one block.
template <bool kBlockRow>
__global__ void __launch_bounds__(256)
    k_ce_merge(const float2* __restrict__ partials, const float* __restrict__ zsum, int NP,
               RowCount rc, int cap, int V, float invT, float smooth, float zloss,
               const int32_t* __restrict__ list, const float* __restrict__ zlab,
               const float* __restrict__ kw, float* __restrict__ lse2,
               float* __restrict__ row_loss, float* __restrict__ lse_out,
               float* __restrict__ share, const float* __restrict__ all_shares, long long N,
               DeviceCtl* ctl, unsigned blocks, float* __restrict__ loss) {
  pdl_wait();
  pdl_trigger();
  const int row = kBlockRow ? blockIdx.x : blockIdx.x * kCeWarps + (threadIdx.x >> 5);
  const bool writes = kBlockRow ? threadIdx.x == 0 : (threadIdx.x & 31) == 0;
  if (row < cap) {
    float l = 0.f, lse = 0.f, part = 0.f;
    if (row < rc.get()) {
      const CeMerged m =
          ce_merge_row<kBlockRow>(partials + (size_t)row * NP,
                                  zsum ? zsum + (size_t)row * NP : nullptr, NP);
      const CeRow w(m.M, m.S, zlab[row] * (invT * kLog2e), m.Z / (float)V * invT, smooth, zloss);
      l = w.loss;
      lse = w.lse;
      part = kw[row] * l;
      if (lse2 && writes) lse2[row] = w.L2;
    }
    if (writes) {
      const int r = list[row];
      if (row_loss) row_loss[r] = l;
      if (lse_out) lse_out[r] = lse;
      share[row] = part;
    }
  }
  ce_finish_loss(all_shares, N, ctl, blocks, loss);
}

// Merge of EpiCeStore's partials, as k_ce_merge, and the row's dlogits from the
// stored exponentials, in place: fp16 E -> bf16 G = kap E 2^(m_t - L2) - targets,
// rounded once (the tensor cores take W and the rows as bf16 and their other operand
// alike; this rounding, 2^-9 of each entry, is most of the gradients' error); the
// label's entry, which E leaves out, from q_y - 1.  A row takes a
// warp (small vocabularies) or gridDim.y blocks (each merges the partials for
// itself), 16 bytes a thread at a time, four loads ahead.  Bound by HBM: 4 bytes
// per entry; 4096 x 128256 in 362 us, 5.8 TB/s (384 with the registers of 3 blocks
// an SM instead of 4).
template <bool kBlockRow>
__global__ void __launch_bounds__(256, 4)
    k_ce_dlogits(const float2* __restrict__ partials, const float* __restrict__ zsum, int NP,
                 RowCount rc, int cap, int V, long long Vp, float invT, float smooth, float zloss,
                 const int32_t* __restrict__ list, const int* __restrict__ lab,
                 const float* __restrict__ zlab, const float* __restrict__ kw,
                 uint4* __restrict__ dlog, float* __restrict__ rest, float* __restrict__ row_loss,
                 float* __restrict__ lse_out, float* __restrict__ share,
                 const float* __restrict__ all_shares, long long N, DeviceCtl* ctl,
                 unsigned blocks, float* __restrict__ loss) {
  pdl_wait();
  pdl_trigger();
  constexpr int kThreads = kBlockRow ? 256 : 32;
  const int row = kBlockRow ? blockIdx.x : blockIdx.x * kCeWarps + (threadIdx.x >> 5);
  const int tid = threadIdx.x % kThreads;
  const bool first = blockIdx.y == 0;  // of the row's blocks: writes the row's outputs
  if (row < rc.get()) {
    const float2* pr = partials + (size_t)row * NP;
    const CeMerged mg = ce_merge_row<kBlockRow>(pr, zsum ? zsum + (size_t)row * NP : nullptr, NP);
    const CeRow w(mg.M, mg.S, zlab[row] * (invT * kLog2e), mg.Z / (float)V * invT, smooth, zloss);
    const float L2 = w.L2, k0 = kw[row];
    if (first && tid == 0) {
      const int r = list[row];
      if (row_loss) row_loss[r] = w.loss;
      if (lse_out) lse_out[r] = w.lse;
      share[row] = k0 * w.loss;
    }
    const float zl = 2.f * zloss * w.lse, kap = fmaf(k0, zl, k0);
    const float base_mass = k0 * smooth / (float)V;
    const int y = lab[row];
    const float g_y = ce_label_grad(k0, w.q1, zl, smooth, base_mass);
    if (first && tid == 0) rest[row] = bf16_rest(g_y);
    uint4* dr = dlog + (size_t)row * (Vp / 8);
    const long long vecs = Vp / 8, step = (long long)kThreads * gridDim.y;
    constexpr int kAhead = 4;  // loads in flight per thread
    for (long long i0 = (long long)kThreads * blockIdx.y + tid; i0 < vecs; i0 += kAhead * step) {
      uint4 q[kAhead];
      float m[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const long long i = i0 + u * step;
        if (i < vecs) {
          q[u] = dr[i];
          m[u] = pr[i >> 4].x;  // 16 vectors to a half tile
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const long long i = i0 + u * step;
        if (i >= vecs) break;
        const float f = kap * ex2_approx(m[u] - L2);
        const uint32_t bits[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&bits[j]));
          v[2 * j] = fmaf(f, e.x, -base_mass);
          v[2 * j + 1] = fmaf(f, e.y, -base_mass);
        }
        const int at = y - 8 * (int)i;
        if ((unsigned)at < 8u) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = j == at ? g_y : v[j];
        }
        if (8 * i + 8 > V) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = 8 * i + j < V ? v[j] : 0.f;
        }
        dr[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      }
    }
  } else if (first && tid == 0 && row < cap) {
    const int r = list[row];
    if (row_loss) row_loss[r] = 0.f;
    if (lse_out) lse_out[r] = 0.f;
    share[row] = 0.f;
  }
  if (first) ce_finish_loss(all_shares, N, ctl, blocks, loss);
}

// dH rows of one chunk: the sum of the row's slabs, in segment order (the dH GEMM
// left their number in the control block), and the label's rest, to the caller's
// row (zeros for left-out rows), rounded once.  A block takes 512 columns
// (blockIdx.y) of a list entry (blockIdx.x).  When the whole call kept no row, no
// dW launch wrote anything: the blocks zero dW (dw_vecs vectors at dw, if given).
template <class Out>
__global__ void __launch_bounds__(128)
    k_ce_dh_out(const float* __restrict__ slabs, const int32_t* __restrict__ list, RowCount rc,
                int H, Out* __restrict__ dH,
                uint4* __restrict__ dw, long long dw_vecs, const DeviceCtl* ctl, float invT,
                const __nv_bfloat16* __restrict__ W, const int* __restrict__ lab,
                const float* __restrict__ rest) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int n = rc.get();
  if (dw != nullptr && ctl->n_rows == 0)
    for (long long j = ((long long)blockIdx.y * gridDim.x + i) * blockDim.x + threadIdx.x;
         j < dw_vecs; j += (long long)gridDim.x * gridDim.y * blockDim.x)
      dw[j] = make_uint4(0u, 0u, 0u, 0u);
  if (dH == nullptr) return;
  const int j = blockIdx.y * 512 + threadIdx.x * 4;
  Out* dst = dH + (size_t)list[i] * H;
  if (i >= n) {
    if (j < H) store4(dst + j, make_float4(0, 0, 0, 0));
    return;
  }
  if (j >= H) return;
  const int S = ctl->split;
  const size_t pitch = (size_t)((n + PM - 1) / PM) * PM * H;
  const float* src = slabs + (size_t)i * H + j;
  float4 a = *reinterpret_cast<const float4*>(src);
  const uint2 wy = *reinterpret_cast<const uint2*>(W + (size_t)lab[i] * H + j);
  const float f = rest[i] * (invT / (float)ctl->n_valid);
#pragma unroll 4
  for (int s = 1; s < S; ++s) {
    const float4 b = *reinterpret_cast<const float4*>(src + s * pitch);
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  a.x = fmaf(f, bf16_lo(wy.x), a.x);
  a.y = fmaf(f, bf16_hi(wy.x), a.y);
  a.z = fmaf(f, bf16_lo(wy.y), a.z);
  a.w = fmaf(f, bf16_hi(wy.y), a.w);
  store4(dst + j, a);
}

// g[0, n) *= *factor (n4 vectors of four and a tail), nothing when it is 1.
template <class T>
__global__ void __launch_bounds__(256)
    k_scale(T* __restrict__ g, long long n, const float* __restrict__ factor) {
  const float f = *factor;
  if (f == 1.f) return;
  const long long n4 = n / 4;
  const long long t0 = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long i = t0; i < n4; i += step) {
    float4 v;
    if constexpr (sizeof(T) == 4) {
      v = reinterpret_cast<const float4*>(g)[i];
    } else {
      const uint2 b = reinterpret_cast<const uint2*>(g)[i];
      const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&b.x));
      const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&b.y));
      v = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    store4(g + 4 * i, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
  }
  if (t0 < n - 4 * n4) g[4 * n4 + t0] = (T)((float)g[4 * n4 + t0] * f);
}

}  // namespace fckl
