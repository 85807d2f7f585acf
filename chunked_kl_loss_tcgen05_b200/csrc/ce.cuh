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
    }
    ctl->n_rows = n;
    ctl->n_valid = denom > 0 ? denom : n;
  }
}

// One chunk's kept rows, gathered: hidden row -> hst[i], label -> lab[i], the
// row's factor (weight, upstream gradient, or 1) -> kw[i], and, when the
// caller gives the log-sum-exps, log2(e) times them -> lse2[i].  The 64 rows
// behind the last one get zero hidden rows: the dW GEMM reads whole blocks of
// 64 rows.  (Gathering, instead of masking in place, keeps what a left-out row
// holds -- NaN, say -- away from the products.)
template <class Label>
__global__ void __launch_bounds__(128)
    k_ce_gather(const int32_t* __restrict__ list, RowCount rc, int H,
                const __nv_bfloat16* __restrict__ hidden, const Label* __restrict__ labels,
                const float* __restrict__ factor, const float* __restrict__ lse,
                __nv_bfloat16* __restrict__ hst, int* __restrict__ lab, float* __restrict__ kw,
                float* __restrict__ lse2) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int n = rc.get();
  if (i >= n + 64) return;
  uint4* dst = reinterpret_cast<uint4*>(hst + (size_t)i * H);
  if (i >= n) {
    for (int j = threadIdx.x; j < H / 8; j += blockDim.x) dst[j] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int r = list[i];
  const uint4* src = reinterpret_cast<const uint4*>(hidden + (size_t)r * H);
  for (int j = threadIdx.x; j < H / 8; j += blockDim.x) dst[j] = src[j];
  if (threadIdx.x == 0) {
    lab[i] = (int)labels[r];
    kw[i] = factor ? factor[r] : 1.f;
    if (lse) lse2[i] = lse[r] * kLog2e;
  }
}

// ---------------------------------------------------------------- epilogues
// Forward: per row and vocab tile of 256 columns, (max, sum 2^(a2 - max)) of
// a2 = z log2(e) / T, z at the row's label if it lies in the tile, and (kSum)
// the tile's sum of z for label smoothing.  The logits are not written.
template <bool kSum>
struct EpiCe {
  static constexpr uint32_t kSmemBytes = 0;
  static constexpr bool kUsesMapC = false;
  struct Params {
    int V, NT;
    float scale2;          // log2(e) / T
    const int* lab;        // [rows]
    float* zlab;           // [rows] z at the label
    float2* partials;      // [rows, NT]
    float* zsum;           // [rows, NT] (kSum)
  };
  struct State {};
  static __device__ void init(const Params&, State&, uint8_t*, int) {}
  static __device__ void tile(const Params& p, State&, const Work& w, uint32_t taddr, int r,
                              const CUtensorMap*, int, int) {
    const int row = w.m0 + r;
    const bool rv = row < w.rows;
    const int y = rv ? __ldg(p.lab + row) - w.n0 : -1;  // label's column in the tile
    float m = -INFINITY, s = 0.f, u = 0.f;
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      float v[32];
      tmem_ld32_conv(taddr + (uint32_t)(c * 32), v);
      if (!rv) continue;
      const int base = w.n0 + c * 32;
      if (base >= p.V) continue;
      if ((y >> 5) == c) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) z = (j == (y & 31)) ? v[j] : z;
        p.zlab[row] = z;
      }
      if (kSum) {
#pragma unroll
        for (int j = 0; j < 32; ++j) u += base + j < p.V ? v[j] : 0.f;
      }
      if (base + 32 > p.V) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = (base + j < p.V) ? v[j] : -INFINITY;
      }
      float cz = v[0];
#pragma unroll
      for (int j = 1; j < 32; ++j) cz = fmaxf(cz, v[j]);
      const float nm = fmaxf(m, cz * p.scale2);
      const float ref = nm == -INFINITY ? 0.f : nm;  // a slice of -inf only adds 0, not NaN
      float acc = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) acc += ex2_approx(fmaf(v[j], p.scale2, -ref));
      s = s * ex2_approx(m - ref) + acc;
      m = nm;
    }
    if (rv) {
      p.partials[(size_t)row * p.NT + w.nt] = make_float2(m, s);
      if (kSum) p.zsum[(size_t)row * p.NT + w.nt] = u;
    }
  }
  static __device__ void finish(const Params&, State&, int) {}
};

// Forward of a call that also wants gradients: as EpiCe, and the exponentials
// themselves are kept, E = 2^(a2 - m) per tile with m = (the row's tile maximum)
// - 15, as fp16 in the chunk's [rows, Vp] block; k_ce_dlogits turns them into
// dlogits in place once the row's LSE is known.  So the backward needs no second
// logits product (6 H V flops per row instead of 8, for 4 V more bytes: at
// H = 4096 the product costs about 10 times what the bytes do).
// fp16 because E is rounded here and G once more in k_ce_dlogits: 2^-11 against
// G's own 2^-8; in bf16 the two roundings would add up.  With the offset of 15
// the tile's largest E is 2^15 and E stays normal down to 2^-29 of it.
// The accumulator is read twice (maximum, then exponentials).
template <bool kSum>
struct EpiCeStore {
  static constexpr uint32_t kSmemBytes = 4 * 2 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: [rows, Vp] 16-bit, box {64, 32}
  struct Params {
    int V, NT;
    float scale2;
    const int* lab;
    float* zlab;
    float2* partials;      // [rows, NT] (m, sum of E before rounding)
    float* zsum;
    int store_rows;
  };
  struct State {
    int n;
    uint8_t* buf;
  };
  static __device__ void init(const Params&, State& st, uint8_t* smem_warp, int) {
    st.n = 0; st.buf = smem_warp;
  }
  static __device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void exps(float (&v)[32], float scale2, float ref, int cols,
                                              float& sum) {
    if (cols >= 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = ex2_approx(fmaf(v[j], scale2, -ref));
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = j < cols ? ex2_approx(fmaf(v[j], scale2, -ref)) : 0.f;
    }
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) acc += v[j];
    sum += acc;
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int r,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int row = w.m0 + r;
    const bool rv = row < w.rows;
    const int y = rv ? __ldg(p.lab + row) - w.n0 : -1;
    float top = -INFINITY, u = 0.f;
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      float v[32];
      tmem_ld32_conv(taddr + (uint32_t)(c * 32), v);
      const int cols = rv ? p.V - (w.n0 + c * 32) : 0;
      if ((y >> 5) == c) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) z = (j == (y & 31)) ? v[j] : z;
        p.zlab[row] = z;
      }
      if (kSum) {
#pragma unroll
        for (int j = 0; j < 32; ++j) u += j < cols ? v[j] : 0.f;
      }
      if (cols >= 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) top = fmaxf(top, v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) top = j < cols ? fmaxf(top, v[j]) : top;
      }
    }
    const float m = fmaf(top, p.scale2, -15.f);
    const float ref = m == -INFINITY ? 0.f : m;  // a tile of -inf only adds 0, not NaN
    float s = 0.f;
    const int y0 = w.m0 + quarter * 32;
    const int y_end = min((w.rows + 63) & ~63, p.store_rows);
#pragma unroll 1
    for (int c = 0; c < BN / 64; ++c) {
      const int base = w.n0 + c * 64;
      const int cols = rv ? p.V - base : 0;
      float v0[32], v1[32];
      tmem_ld32_conv(taddr + (uint32_t)(c * 64), v0);
      tmem_ld32_conv(taddr + (uint32_t)(c * 64 + 32), v1);
      exps(v0, p.scale2, ref, cols, s);
      exps(v1, p.scale2, ref, cols - 32, s);
      uint8_t* buf = st.buf + (st.n & 1) * 4096;
      stage_acquire(lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *stage_chunk(buf, lane, j) = make_uint4(
            pack_half2(v0[8 * j], v0[8 * j + 1]), pack_half2(v0[8 * j + 2], v0[8 * j + 3]),
            pack_half2(v0[8 * j + 4], v0[8 * j + 5]), pack_half2(v0[8 * j + 6], v0[8 * j + 7]));
        *stage_chunk(buf, lane, 4 + j) = make_uint4(
            pack_half2(v1[8 * j], v1[8 * j + 1]), pack_half2(v1[8 * j + 2], v1[8 * j + 3]),
            pack_half2(v1[8 * j + 4], v1[8 * j + 5]), pack_half2(v1[8 * j + 6], v1[8 * j + 7]));
      }
      stage_release();
      if (lane == 0) {
        if (base < p.V && y0 < y_end) tma_store_2d(mapC, smem_u32(buf), base, y0);
        bulk_commit();
      }
      ++st.n;
    }
    if (rv) {
      p.partials[(size_t)row * p.NT + w.nt] = make_float2(m, s);
      if (kSum) p.zsum[(size_t)row * p.NT + w.nt] = u;
    }
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// Backward without the forward's exponentials (the row-gradient call): recomputed z tile -> G (see the top), rounded once to bf16 and
// TMA-stored to the chunk's [rows, Vp] block.  Columns in [V, Vp) and the rows
// behind the last one, up to the next multiple of 64, are stored as zeros.
struct EpiCeDlogits {
  static constexpr uint32_t kSmemBytes = 4 * 2 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: [rows, Vp] bf16, box {64, 32}
  struct Params {
    int V;
    float scale2;          // log2(e) / T
    float smooth;          // label smoothing e
    float zloss2;          // 2 lam
    const int* lab;        // [rows]
    const float* kw;       // [rows] k_r
    const float* lse2;     // [rows] log2(e) LSE
    int store_rows;        // rows of the store map
  };
  struct State {
    int n;
    uint8_t* buf;
  };
  static __device__ void init(const Params&, State& st, uint8_t* smem_warp, int) {
    st.n = 0; st.buf = smem_warp;
  }
  static __device__ __forceinline__ void slice(float (&v)[32], float scale2, float lse2, float kap,
                                               float base_mass, float label_mass, int y, int cols) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float t = j == y ? base_mass + label_mass : base_mass;
      const float g = fmaf(kap, ex2_approx(fmaf(v[j], scale2, -lse2)), -t);
      v[j] = j < cols ? g : 0.f;
    }
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int r,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int row = w.m0 + r;
    const bool rv = row < w.rows;
    const float kw = rv ? p.kw[row] : 0.f;
    const float lse2 = rv ? p.lse2[row] : 0.f;
    const int y = rv ? p.lab[row] - w.n0 : -1;
    const float kap = kw * fmaf(p.zloss2, lse2 * kLn2, 1.f);
    const float label_mass = kw * (1.f - p.smooth), base_mass = kw * p.smooth / (float)p.V;
    const int y0 = w.m0 + quarter * 32;
    const int y_end = min((w.rows + 63) & ~63, p.store_rows);
#pragma unroll 1
    for (int s = 0; s < BN / 64; ++s) {
      const int base = w.n0 + s * 64;
      float v0[32], v1[32];
      tmem_ld32_conv(taddr + (uint32_t)(s * 64), v0);
      tmem_ld32_conv(taddr + (uint32_t)(s * 64 + 32), v1);
      slice(v0, p.scale2, lse2, kap, base_mass, label_mass, y - s * 64, rv ? p.V - base : 0);
      slice(v1, p.scale2, lse2, kap, base_mass, label_mass, y - s * 64 - 32,
            rv ? p.V - base - 32 : 0);
      uint8_t* buf = st.buf + (st.n & 1) * 4096;
      stage_acquire(lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *stage_chunk(buf, lane, j) = make_uint4(
            pack_bf16x2(v0[8 * j], v0[8 * j + 1]), pack_bf16x2(v0[8 * j + 2], v0[8 * j + 3]),
            pack_bf16x2(v0[8 * j + 4], v0[8 * j + 5]), pack_bf16x2(v0[8 * j + 6], v0[8 * j + 7]));
        *stage_chunk(buf, lane, 4 + j) = make_uint4(
            pack_bf16x2(v1[8 * j], v1[8 * j + 1]), pack_bf16x2(v1[8 * j + 2], v1[8 * j + 3]),
            pack_bf16x2(v1[8 * j + 4], v1[8 * j + 5]), pack_bf16x2(v1[8 * j + 6], v1[8 * j + 7]));
      }
      stage_release();
      if (lane == 0) {  // one group per slice, empty when the slice lies outside the map
        if (base < p.V && y0 < y_end) tma_store_2d(mapC, smem_u32(buf), base, y0);
        bulk_commit();
      }
      ++st.n;
    }
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// dH partials: the fp32 tile of k segment ks is stored to its own slab (rows
// [ks * 256 * MT, ...) of the slab array), not added in place, so that the sum
// over the segments has one order and repeated calls give the same bits.
struct EpiCeDH {
  static constexpr uint32_t kSmemBytes = 4 * 2 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: slabs [S * 256 * MT, H] fp32, box {32, 32}
  struct Params {
    int H;
    float invT;
    const DeviceCtl* ctl;
  };
  struct State {
    float alpha;
    int n;
    uint8_t* buf;
  };
  static __device__ void init(const Params& p, State& st, uint8_t* smem_warp, int) {
    const int nv = p.ctl->n_valid;
    st.alpha = nv > 0 ? p.invT / (float)nv : 0.f;
    st.n = 0;
    st.buf = smem_warp;
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int y = w.m0 + quarter * 32;
    const int pitch = (w.rows + PM - 1) / PM * PM;
    stage_fp32_slices<false>(st.buf, st.n, taddr, st.alpha, mapC, w.n0, p.H, w.ks * pitch + y,
                             y < w.rows, lane);
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// dW in fp32 over the chunks (a type of its own, so that the two translation
// units instantiate different kernels).
struct EpiCeDWSum : EpiDW {};

// dW written once, rounded once to bf16 (calls of one chunk).
struct EpiCeDW {
  static constexpr uint32_t kSmemBytes = 4 * 2 * 4096;
  static constexpr bool kUsesMapC = true;  // map C: dW [V, H] bf16, box {64, 32}
  struct Params {
    int V, H;
    float invT;
    const DeviceCtl* ctl;
  };
  struct State {
    float alpha;
    int n;
    uint8_t* buf;
  };
  static __device__ void init(const Params& p, State& st, uint8_t* smem_warp, int) {
    const int nv = p.ctl->n_valid;
    st.alpha = nv > 0 ? p.invT / (float)nv : 0.f;
    st.n = 0;
    st.buf = smem_warp;
  }
  static __device__ void tile(const Params& p, State& st, const Work& w, uint32_t taddr, int,
                              const CUtensorMap* mapC, int quarter, int lane) {
    const int y = w.m0 + quarter * 32;
#pragma unroll 1
    for (int s = 0; s < BN / 64; ++s) {
      float v0[32], v1[32];
      tmem_ld32_conv(taddr + (uint32_t)(s * 64), v0);
      tmem_ld32_conv(taddr + (uint32_t)(s * 64 + 32), v1);
      uint8_t* buf = st.buf + (st.n & 1) * 4096;
      stage_acquire(lane);
      const float al = st.alpha;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *stage_chunk(buf, lane, j) =
            make_uint4(pack_bf16x2(al * v0[8 * j], al * v0[8 * j + 1]),
                       pack_bf16x2(al * v0[8 * j + 2], al * v0[8 * j + 3]),
                       pack_bf16x2(al * v0[8 * j + 4], al * v0[8 * j + 5]),
                       pack_bf16x2(al * v0[8 * j + 6], al * v0[8 * j + 7]));
        *stage_chunk(buf, lane, 4 + j) =
            make_uint4(pack_bf16x2(al * v1[8 * j], al * v1[8 * j + 1]),
                       pack_bf16x2(al * v1[8 * j + 2], al * v1[8 * j + 3]),
                       pack_bf16x2(al * v1[8 * j + 4], al * v1[8 * j + 5]),
                       pack_bf16x2(al * v1[8 * j + 6], al * v1[8 * j + 7]));
      }
      stage_release();
      const int x = w.n0 + s * 64;
      if (lane == 0) {
        if (x < p.H && y < p.V) tma_store_2d(mapC, smem_u32(buf), x, y);
        bulk_commit();
      }
      ++st.n;
    }
  }
  static __device__ void finish(const Params&, State&, int lane) {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// ---------------------------------------------------------------- row kernels
// Merges the tile partials of each row into its LSE and row loss.  All rows of
// the chunk's part of the list write the caller's row loss and LSE (0 for
// left-out rows) and their share k_r l_r of the loss (list order).  One warp
// per row.
__global__ void __launch_bounds__(kCeWarps * 32)
    k_ce_merge(const float2* __restrict__ partials, const float* __restrict__ zsum, int NT,
               RowCount rc, int cap, int V, float invT, float smooth, float zloss,
               const int32_t* __restrict__ list, const float* __restrict__ zlab,
               const float* __restrict__ kw, float* __restrict__ row_loss,
               float* __restrict__ lse_out, float* __restrict__ share) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kCeWarps + (threadIdx.x >> 5);
  if (row >= cap) return;
  const int r = list[row];
  if (row >= rc.get()) {
    if (lane == 0) {
      if (row_loss) row_loss[r] = 0.f;
      if (lse_out) lse_out[r] = 0.f;
      share[row] = 0.f;
    }
    return;
  }
  const float2* pr = partials + (size_t)row * NT;
  float M = -INFINITY;
  for (int t = lane; t < NT; t += 32) M = fmaxf(M, pr[t].x);
  M = warp_max(M);
  float S = 0.f, Z = 0.f;
  for (int t = lane; t < NT; t += 32) {
    const float2 q = pr[t];
    S += q.y * exp2f(q.x - M);
    if (zsum) Z += zsum[(size_t)row * NT + t];
  }
  S = warp_sum(S);
  if (zsum) Z = warp_sum(Z);
  if (lane == 0) {
    const float L2 = M + log2f(S);
    const float lse = L2 * kLn2;
    const float nll = lse - zlab[row] * invT;
    float l = nll;
    if (smooth > 0.f) l += smooth * ((lse - Z / (float)V * invT) - nll);
    l = fmaf(zloss * lse, lse, l);
    if (row_loss) row_loss[r] = l;
    if (lse_out) lse_out[r] = lse;
    share[row] = kw[row] * l;
  }
}

// Merge of EpiCeStore's partials, as k_ce_merge, and the row's dlogits from the
// stored exponentials, in place: fp16 E -> bf16 G = kap E 2^(m_t - L2) - targets,
// rounded once.  The label's entry is formed from its fp32 logit: q_y - 1 would
// lose what E's rounding cuts off where the row is confident.  One block per
// row: 8 warps, a warp at a time on a tile of 256 columns (16 bytes a lane).
// Bound by HBM: 4 bytes per entry.
__global__ void __launch_bounds__(256)
    k_ce_dlogits(const float2* __restrict__ partials, const float* __restrict__ zsum, int NT,
                 RowCount rc, int V, long long Vp, float invT, float smooth, float zloss,
                 const int32_t* __restrict__ list, const int* __restrict__ lab,
                 const float* __restrict__ zlab, const float* __restrict__ kw,
                 uint4* __restrict__ dlog, float* __restrict__ row_loss,
                 float* __restrict__ lse_out, float* __restrict__ share) {
  __shared__ float red[3][8];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = list[row];
  if (row >= rc.get()) {
    if (threadIdx.x == 0) {
      if (row_loss) row_loss[r] = 0.f;
      if (lse_out) lse_out[r] = 0.f;
      share[row] = 0.f;
    }
    return;
  }
  const float2* pr = partials + (size_t)row * NT;
  float M = -INFINITY, S = 0.f, Z = 0.f;
  for (int t = threadIdx.x; t < NT; t += 256) {
    const float2 q = pr[t];
    const float nm = fmaxf(M, q.x);
    const float ref = nm == -INFINITY ? 0.f : nm;
    S = S * exp2f(M - ref) + q.y * exp2f(q.x - ref);
    M = nm;
    if (zsum) Z += zsum[(size_t)row * NT + t];
  }
  const float Mw = warp_max(M);
  S = warp_sum(S * exp2f(M - (Mw == -INFINITY ? 0.f : Mw)));
  if (zsum) Z = warp_sum(Z);
  if (lane == 0) { red[0][warp] = Mw; red[1][warp] = S; red[2][warp] = Z; }
  __syncthreads();
  M = red[0][0];
#pragma unroll
  for (int k = 1; k < 8; ++k) M = fmaxf(M, red[0][k]);
  S = Z = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    S += red[1][k] * exp2f(red[0][k] - (M == -INFINITY ? 0.f : M));
    Z += red[2][k];
  }
  const float L2 = M + log2f(S), lse = L2 * kLn2, k0 = kw[row], a_y = zlab[row] * invT;
  if (threadIdx.x == 0) {
    const float nll = lse - a_y;
    float l = nll;
    if (smooth > 0.f) l += smooth * ((lse - Z / (float)V * invT) - nll);
    l = fmaf(zloss * lse, lse, l);
    if (row_loss) row_loss[r] = l;
    if (lse_out) lse_out[r] = lse;
    share[row] = k0 * l;
  }
  const float kap = k0 * fmaf(2.f * zloss, lse, 1.f);
  const float label_mass = k0 * (1.f - smooth), base_mass = k0 * smooth / (float)V;
  const int y = lab[row];
  const float g_y = fmaf(kap, exp2f(fmaf(zlab[row], invT * kLog2e, -L2)), -(label_mass + base_mass));
  uint4* dr = dlog + (size_t)row * (Vp / 8);
#pragma unroll 4
  for (int t = warp; t < NT; t += 8) {
    const int col = t * BN + lane * 8;
    if (col >= Vp) continue;
    const float f = kap * ex2_approx(pr[t].x - L2);
    uint4 q = dr[col / 8];
    float v[8];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[2 * j] = fmaf(f, e.x, -base_mass);
      v[2 * j + 1] = fmaf(f, e.y, -base_mass);
    }
    if ((unsigned)(y - col) < 8u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j == y - col ? g_y : v[j];
    }
    if (col + 8 > V) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = col + j < V ? v[j] : 0.f;
    }
    dr[col / 8] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// loss = sum of the rows' shares / D, fp64 in a fixed order.
__global__ void __launch_bounds__(1024) k_ce_finalize(const float* __restrict__ share, long long N,
                                                      const DeviceCtl* ctl, float* loss) {
  pdl_wait();
  pdl_trigger();
  __shared__ double red[1024];
  double s = 0.0;
  for (long long i = threadIdx.x; i < N; i += blockDim.x) s += (double)share[i];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int w = blockDim.x >> 1; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int n = ctl->n_valid;
    *loss = ctl->n_rows > 0 && n > 0 ? (float)(red[0] / (double)n) : 0.f;
  }
}

// dH rows of one chunk: the sum of the row's slabs, in segment order, to the
// caller's row (zeros for left-out rows), rounded once.  One block per list
// entry.  The number of segments is the one the dH GEMM chose (same inputs).
// When the whole call kept no row, no dW launch wrote anything: the blocks zero
// the dw_bytes of dW (dw != nullptr) instead.
template <class Out>
__global__ void __launch_bounds__(128)
    k_ce_dh_out(const float* __restrict__ slabs, const int32_t* __restrict__ list, RowCount rc,
                int H, int NTh, int KB, int slots, int slab_units, Out* __restrict__ dH,
                uint4* __restrict__ dw, long long dw_vecs, const DeviceCtl* ctl) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int n = rc.get();
  if (dw != nullptr && ctl->n_rows == 0)
    for (long long j = i * (long long)blockDim.x + threadIdx.x; j < dw_vecs;
         j += (long long)gridDim.x * blockDim.x)
      dw[j] = make_uint4(0u, 0u, 0u, 0u);
  if (dH == nullptr) return;
  Out* dst = dH + (size_t)list[i] * H;
  if (i >= n) {
    for (int j = threadIdx.x * 4; j < H; j += blockDim.x * 4) store4(dst + j, make_float4(0, 0, 0, 0));
    return;
  }
  const int MT = (n + PM - 1) / PM;
  const int S = choose_split_warp(MT * NTh, KB, slots, slab_units);
  const size_t pitch = (size_t)MT * PM * H;
  const float* src = slabs + (size_t)i * H;
  for (int j = threadIdx.x * 4; j < H; j += blockDim.x * 4) {
    float4 a = *reinterpret_cast<const float4*>(src + j);
    for (int s = 1; s < S; ++s) {
      const float4 b = *reinterpret_cast<const float4*>(src + s * pitch + j);
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    store4(dst + j, a);
  }
}

// bf16 dW of a call of several chunks: the fp32 sum over the chunks, rounded once.
__global__ void __launch_bounds__(256)
    k_ce_dw_out(const float4* __restrict__ acc, long long n4, uint2* __restrict__ dW,
                const DeviceCtl* ctl) {
  pdl_wait();
  pdl_trigger();
  const bool none = ctl->n_rows == 0;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n4;
       i += (long long)gridDim.x * blockDim.x) {
    const float4 v = none ? make_float4(0, 0, 0, 0) : acc[i];
    dW[i] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
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
