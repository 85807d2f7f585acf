// The norms after and before a block, fused with the block's gate and residual
// scale, forward and backward, over rows of H values:
//   u = b rho_b w1 (post-norm)      v = x + s g u      y = v rho_v w2 (pre-norm)
//   rho_z = 1 / sqrt(mean(z^2) + eps)
//   t = w2 dy;  dx = dv = dv_in + rho_v t - v rho_v^3 mean(v t)
//   du = s g dv;  db = rho_b (w1 du) - b rho_b^3 mean(b w1 du)
//   dw2 = sum_r dy v rho_v;  dw1 = sum_r du b rho_b;  dg = sum_r s dv u
// With n = b rho_b (b without a post-norm), c = s g w1 and P = sum_r dv n:
//   v = x + c n,  dw1 = s g P,  dg = s w1 P,
// so the backward keeps two column sums, P and dw2, in registers.
// All in fp32 from the inputs on (v is not rounded before it is normed; the
// backward forms v again from x and b), each output rounded once.
//
// Bound by HBM: forward x, b in and v, y out; backward x, b, dy, dv in and dx,
// db out.  Rows go through a ring of shared-memory stages filled by 16-byte
// asynchronous copies, several rows ahead; a thread copies exactly the values
// it will read, so the data needs no barrier, and the waits are the copies'
// own.  A row of more than 512 values takes a block, a shorter one a warp
// (eight rows a block, and no barriers for the row sums either).
#pragma once

#include "ptx.cuh"
#include "reduce.cuh"
#include "vec.cuh"

namespace fckl {

constexpr int kNormHMax = 8192;
constexpr int kNormWarpH = 512;      // rows up to this length take one warp
constexpr int kNormRowWarps = 8;     // rows of a block then

struct NormArgs {
  long long N;
  int H;
  float scale, eps, offset;
  const void* x;
  const void* b;          // nullptr: v = x
  const void* w1;         // nullptr: ones (post only)
  const void* g;          // nullptr: ones
  const void* w2;         // nullptr: ones (pre only)
  int post, pre;
  int stages;             // ring stages
  // forward
  void* v;                // nullptr: not wanted
  void* y;
  // backward
  const void* dy;         // nullptr without pre
  const void* dv;         // nullptr: zeros
  void* dx;               // nullptr: not wanted, as the ones below
  void* db;
  float* part;            // [grid, 2, H]: P and dw2 over each block's rows
  float* dw1;
  float* dg;
  float* dw2;
};

// Sums of K values over the row's threads, the same on each of them.  `red` has
// room for two calls (`turn` alternates), so one barrier per call is enough.
template <bool kWarpRow, int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float* red, int& turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = warp_sum(s[k]);
  if (kWarpRow) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float* r = red + (turn & 1) * 64;
  ++turn;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) r[k * 32 + warp] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = warp_sum(lane < warps ? r[k * 32 + lane] : 0.f);
}

// Eight weights (+ offset), or ones.
template <class WT>
__device__ __forceinline__ void load_weight(const void* w, int col, float offset, float (&o)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 1.f;
    return;
  }
  Raw8<WT> r;
  r.load(static_cast<const WT*>(w) + col);
  r.get(o);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] += offset;
}

// Eight values of T, global -> shared, asynchronously.
template <class T>
__device__ __forceinline__ void copy8(uint8_t* dst, const T* src) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + 16 * i)),
                 "l"(reinterpret_cast<const uint8_t*>(src) + 16 * i)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The oldest of `stages` groups has landed.
__device__ __forceinline__ void copy_wait_oldest(int stages) {
  if (stages >= 4) copy_wait<3>();
  else if (stages == 3) copy_wait<2>();
  else copy_wait<1>();
}
constexpr int kNormStagesMax = 4;

// Where a thread's row begins and how the rows are dealt.
template <bool kWarpRow>
struct NormRows {
  int tid, threads;      // within the row
  long long r, step;
  __device__ __forceinline__ NormRows() {
    if (kWarpRow) {
      tid = threadIdx.x & 31; threads = 32;
      r = blockIdx.x * (long long)kNormRowWarps + (threadIdx.x >> 5);
      step = gridDim.x * (long long)kNormRowWarps;
    } else {
      tid = threadIdx.x; threads = blockDim.x;
      r = blockIdx.x; step = gridDim.x;
    }
  }
};

// NV vectors of eight per thread: columns 8 (tid + k threads).
template <bool kWarpRow, class XT, class WT, int NV>
__global__ void __launch_bounds__(512) k_norm_fwd(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[128];
  pdl_wait();
  pdl_trigger();
  const int nvec = a.H / 8;
  const float invH = 1.f / (float)a.H;
  const NormRows<kWarpRow> rows;
  const int row_bytes = a.H * ((int)sizeof(XT) + (a.b ? 2 : 0));
  uint8_t* mine = ring + (kWarpRow ? (threadIdx.x >> 5) * a.stages * row_bytes : 0);
  float c[NV][8], w2[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int j = rows.tid + k * rows.threads;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[k][i] = w2[k][i] = 0.f;
    if (j >= nvec) continue;
    float g[8];
    load_weight<WT>(a.post ? a.w1 : nullptr, 8 * j, a.offset, c[k]);
    load_weight<WT>(a.g, 8 * j, 0.f, g);
    load_weight<WT>(a.w2, 8 * j, a.offset, w2[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[k][i] *= a.scale * g[i];
  }
  auto fetch = [&](long long r, int stage) {
    if (r < a.N) {
      const long long o = r * a.H;
      uint8_t* s = mine + stage * row_bytes;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int j = rows.tid + k * rows.threads;
        if (j >= nvec) continue;
        copy8(s + j * 8 * sizeof(XT), static_cast<const XT*>(a.x) + o + 8 * j);
        if (a.b)
          copy8(s + a.H * sizeof(XT) + j * 16, static_cast<const __nv_bfloat16*>(a.b) + o + 8 * j);
      }
    }
    copy_commit();
  };
  int turn = 0, stage = 0;
  for (int i = 0; i < a.stages; ++i) fetch(rows.r + i * rows.step, i);
  for (long long r = rows.r; r < a.N; r += rows.step) {
    const long long o = r * a.H;
    copy_wait_oldest(a.stages);
    const uint8_t* s = mine + stage * row_bytes;
    float v[NV][8], b[NV][8], sb[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = b[k][i] = 0.f;
      if (j < nvec) {
        Raw8<XT> rx;
        rx.load(reinterpret_cast<const XT*>(s) + 8 * j);
        rx.get(v[k]);
        if (a.b) {
          Raw8<__nv_bfloat16> rb;
          rb.load(reinterpret_cast<const __nv_bfloat16*>(s + a.H * sizeof(XT)) + 8 * j);
          rb.get(b[k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sb[0] = fmaf(b[k][i], b[k][i], sb[0]);
    }
    fetch(r + a.stages * rows.step, stage);  // this thread has read its part of the stage
    stage = stage + 1 == a.stages ? 0 : stage + 1;
    if (a.b) {
      float rho = 1.f;
      if (a.post) {
        row_sums<kWarpRow>(sb, red, turn);
        rho = rsqrtf(fmaf(sb[0], invH, a.eps));
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int j = rows.tid + k * rows.threads;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = fmaf(c[k][i], b[k][i] * rho, v[k][i]);
        if (a.v && j < nvec) store8(static_cast<XT*>(a.v) + o + 8 * j, v[k]);
      }
    }
    if (!a.pre) continue;
    float sv[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sv[0] = fmaf(v[k][i], v[k][i], sv[0]);
    row_sums<kWarpRow>(sv, red, turn);
    const float rho = rsqrtf(fmaf(sv[0], invH, a.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
      if (j >= nvec) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] *= rho * w2[k][i];
      store8(static_cast<__nv_bfloat16*>(a.y) + o + 8 * j, v[k]);
    }
  }
  copy_wait<0>();
}

template <bool kWarpRow, class XT, class DT, class WT, int NV, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) k_norm_bwd(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[128];
  pdl_wait();
  pdl_trigger();
  const int nvec = a.H / 8;
  const float invH = 1.f / (float)a.H;
  const NormRows<kWarpRow> rows;
  const int off_b = a.H * (int)sizeof(XT), off_dv = off_b + (a.b ? a.H * 2 : 0);
  const int off_dy = off_dv + (a.dv ? a.H * (int)sizeof(XT) : 0);
  const int row_bytes = off_dy + (a.pre ? a.H * (int)sizeof(DT) : 0);
  uint8_t* mine = ring + (kWarpRow ? (threadIdx.x >> 5) * a.stages * row_bytes : 0);
  float c[NV][8], w2[NV][8], P[NV][8], D[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int j = rows.tid + k * rows.threads;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[k][i] = w2[k][i] = P[k][i] = D[k][i] = 0.f;
    if (j >= nvec) continue;
    float g[8];
    load_weight<WT>(a.post ? a.w1 : nullptr, 8 * j, a.offset, c[k]);
    load_weight<WT>(a.g, 8 * j, 0.f, g);
    load_weight<WT>(a.w2, 8 * j, a.offset, w2[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[k][i] *= a.scale * g[i];
  }
  auto fetch = [&](long long r, int stage) {
    if (r < a.N) {
      const long long o = r * a.H;
      uint8_t* s = mine + stage * row_bytes;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int j = rows.tid + k * rows.threads;
        if (j >= nvec) continue;
        copy8(s + j * 8 * sizeof(XT), static_cast<const XT*>(a.x) + o + 8 * j);
        if (a.b) copy8(s + off_b + j * 16, static_cast<const __nv_bfloat16*>(a.b) + o + 8 * j);
        if (a.dv)
          copy8(s + off_dv + j * 8 * sizeof(XT), static_cast<const XT*>(a.dv) + o + 8 * j);
        if (a.pre)
          copy8(s + off_dy + j * 8 * sizeof(DT), static_cast<const DT*>(a.dy) + o + 8 * j);
      }
    }
    copy_commit();
  };
  int turn = 0, stage = 0;
  for (int i = 0; i < a.stages; ++i) fetch(rows.r + i * rows.step, i);
  for (long long r = rows.r; r < a.N; r += rows.step) {
    const long long o = r * a.H;
    copy_wait_oldest(a.stages);
    const uint8_t* s = mine + stage * row_bytes;
    float v[NV][8], b[NV][8], d[NV][8];  // d: dy, then dv
    float sb[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[k][i] = 0.f;
      if (a.b && j < nvec) {
        Raw8<__nv_bfloat16> rb;
        rb.load(reinterpret_cast<const __nv_bfloat16*>(s + off_b) + 8 * j);
        rb.get(b[k]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sb[0] = fmaf(b[k][i], b[k][i], sb[0]);
    }
    float rho_b = 1.f;
    if (a.post) {
      row_sums<kWarpRow>(sb, red, turn);
      rho_b = rsqrtf(fmaf(sb[0], invH, a.eps));
    }
    float s2[2] = {0.f, 0.f};  // sum v^2, sum v t
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = d[k][i] = 0.f;
      if (j < nvec) {
        Raw8<XT> rx;
        rx.load(reinterpret_cast<const XT*>(s) + 8 * j);
        rx.get(v[k]);
        if (a.pre) {
          Raw8<DT> rd;
          rd.load(reinterpret_cast<const DT*>(s + off_dy) + 8 * j);
          rd.get(d[k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[k][i] *= rho_b;  // normed from here on
        v[k][i] = fmaf(c[k][i], b[k][i], v[k][i]);
        s2[0] = fmaf(v[k][i], v[k][i], s2[0]);
        s2[1] = fmaf(v[k][i], d[k][i] * w2[k][i], s2[1]);
      }
    }
    float rho_v = 0.f, corr = 0.f;
    if (a.pre) {
      row_sums<kWarpRow>(s2, red, turn);
      rho_v = rsqrtf(fmaf(s2[0], invH, a.eps));
      corr = s2[1] * invH * rho_v * rho_v;
    }
    float sbt[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
      float dv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.dv && j < nvec) {
        Raw8<XT> rv;
        rv.load(reinterpret_cast<const XT*>(s + off_dv) + 8 * j);
        rv.get(dv);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        D[k][i] = fmaf(d[k][i], v[k][i] * rho_v, D[k][i]);
        d[k][i] = fmaf(rho_v, fmaf(d[k][i], w2[k][i], -v[k][i] * corr), dv[i]);
        P[k][i] = fmaf(d[k][i], b[k][i], P[k][i]);
      }
      if (a.dx && j < nvec) store8(static_cast<XT*>(a.dx) + o + 8 * j, d[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[k][i] *= c[k][i];
        sbt[0] = fmaf(b[k][i], d[k][i], sbt[0]);
      }
    }
    fetch(r + a.stages * rows.step, stage);  // this thread has read its part of the stage
    stage = stage + 1 == a.stages ? 0 : stage + 1;
    if (!a.db) continue;
    float mean = 0.f;
    if (a.post) {
      row_sums<kWarpRow>(sbt, red, turn);
      mean = sbt[0] * invH;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
      if (j >= nvec) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[k][i] = rho_b * fmaf(-mean, b[k][i], d[k][i]);
      store8(static_cast<__nv_bfloat16*>(a.db) + o + 8 * j, d[k]);
    }
  }
  copy_wait<0>();
  if (!a.dw1 && !a.dg && !a.dw2) return;
  float* p = a.part + (size_t)blockIdx.x * 2 * a.H;
  if constexpr (kWarpRow) {  // the block's eight rows of sums become one, in warp order
    __syncthreads();
    float* sum = reinterpret_cast<float*>(ring);  // [8][2][H]
    float* w = sum + (threadIdx.x >> 5) * 2 * a.H;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
      if (j >= nvec) continue;
      store8(w + 8 * j, P[k]);
      store8(w + a.H + 8 * j, D[k]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.H; i += blockDim.x) {
      float t = sum[i];
      for (int k = 1; k < kNormRowWarps; ++k) t += sum[k * 2 * a.H + i];
      p[i] = t;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = rows.tid + k * rows.threads;
      if (j >= nvec) continue;
      store8(p + 8 * j, P[k]);
      store8(p + a.H + 8 * j, D[k]);
    }
  }
}

// Column sums of the blocks' partials, in block order: a block takes 64
// columns of P or dw2, each of its 16 warps every 16th partial.
template <class WT>
__global__ void __launch_bounds__(512) k_norm_sum(const NormArgs a, int blocks) {
  __shared__ float2 red[16][32];
  pdl_wait();
  pdl_trigger();
  const bool first = blockIdx.y == 0;
  if (first ? (!a.dw1 && !a.dg) : !a.dw2) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 64 + lane * 2;
  float2 s = make_float2(0.f, 0.f);
  if (col < a.H) {
    const float* p = a.part + (size_t)blockIdx.y * a.H + col;
#pragma unroll 8
    for (int i = warp; i < blocks; i += 16) {
      const float2 q = *reinterpret_cast<const float2*>(p + (size_t)i * 2 * a.H);
      s.x += q.x; s.y += q.y;
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= a.H) return;
  for (int w = 1; w < 16; ++w) {
    s.x += red[w][lane].x; s.y += red[w][lane].y;
  }
  if (!first) {
    *reinterpret_cast<float2*>(a.dw2 + col) = s;
    return;
  }
  s.x *= a.scale; s.y *= a.scale;
  auto at = [&](const void* w, int i, float off) {
    return w ? (float)static_cast<const WT*>(w)[col + i] + off : 1.f;
  };
  if (a.dw1)
    *reinterpret_cast<float2*>(a.dw1 + col) = make_float2(s.x * at(a.g, 0, 0.f), s.y * at(a.g, 1, 0.f));
  if (a.dg)
    *reinterpret_cast<float2*>(a.dg + col) =
        make_float2(s.x * at(a.post ? a.w1 : nullptr, 0, a.offset),
                    s.y * at(a.post ? a.w1 : nullptr, 1, a.offset));
}

}  // namespace fckl
