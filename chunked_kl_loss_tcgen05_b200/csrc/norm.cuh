// The norms after and before a block, fused with the block's gate and residual
// scale, forward and backward, over rows of H values:
//   u = b rho_b w1 (post-norm)      v = x + s g u      y = v rho_v w2 (pre-norm)
//   rho_z = 1 / sqrt(mean(z^2) + eps)
//   t = w2 dy;  dx = dv = dv_in + rho_v t - v rho_v^3 mean(v t)
//   du = s g dv;  db = rho_b (w1 du) - b rho_b^3 mean(b w1 du)
//   dw2 = sum_r dy v rho_v;  dw1 = sum_r du b rho_b;  dg = sum_r s dv u
// All in fp32 from the inputs on (v is not rounded before it is normed; the
// backward forms v again from x and b), each output rounded once.
//
// One row per block at a time, eight values per 16-byte vector, kept in
// registers between the reductions.  The bound is HBM: forward x, b in and v,
// y out; backward x, b, dy, dv in and dx, db out.
#pragma once

#include "ptx.cuh"
#include "reduce.cuh"
#include "vec.cuh"

namespace fckl {

constexpr int kNormHMax = 8192;
constexpr int kNormThreadsMax = 512;

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
  // forward
  void* v;                // nullptr: not wanted
  void* y;
  // backward
  const void* dy;         // nullptr without pre
  const void* dv;         // nullptr: zeros
  void* dx;               // nullptr: not wanted, as the ones below
  void* db;
  float* part;            // [grid, 3, H]: sums of dw1, dg, dw2 over each block's rows
  int want_w1, want_g, want_w2;
};

// Sums of K values over the block, the same on every thread.  `red` has room
// for two calls (`turn` alternates), so one barrier per call is enough.
template <int K>
__device__ __forceinline__ void block_sums(float (&s)[K], float* red, int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = warp_sum(s[k]);
  if (warps == 1) return;
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

// NV vectors per thread: columns 8 (threadIdx.x + k blockDim.x).
template <class XT, class WT, int NV>
__global__ void __launch_bounds__(kNormThreadsMax) k_norm_fwd(const NormArgs a) {
  __shared__ float red[128];
  pdl_wait();
  pdl_trigger();
  const int nvec = a.H / 8;
  const float invH = 1.f / (float)a.H;
  int turn = 0;
  for (long long r = blockIdx.x; r < a.N; r += gridDim.x) {
    const long long o = r * a.H;
    float v[NV][8], b[NV][8];
    float sb[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = threadIdx.x + k * blockDim.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = b[k][i] = 0.f;
      if (j < nvec) {
        Raw8<XT> rx;
        rx.load(static_cast<const XT*>(a.x) + o + 8 * j);
        rx.get(v[k]);
        if (a.b) {
          Raw8<__nv_bfloat16> rb;
          rb.load(static_cast<const __nv_bfloat16*>(a.b) + o + 8 * j);
          rb.get(b[k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sb[0] = fmaf(b[k][i], b[k][i], sb[0]);
    }
    if (a.b) {
      float rho = 1.f;
      if (a.post) {
        block_sums(sb, red, turn);
        rho = rsqrtf(fmaf(sb[0], invH, a.eps));
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int j = threadIdx.x + k * blockDim.x;
        if (j >= nvec) continue;
        float w[8], g[8];
        load_weight<WT>(a.post ? a.w1 : nullptr, 8 * j, a.offset, w);
        load_weight<WT>(a.g, 8 * j, 0.f, g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[k][i] = fmaf(a.scale * g[i], b[k][i] * rho * w[i], v[k][i]);
        if (a.v) store8(static_cast<XT*>(a.v) + o + 8 * j, v[k]);
      }
    }
    if (!a.pre) continue;
    float sv[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sv[0] = fmaf(v[k][i], v[k][i], sv[0]);
    block_sums(sv, red, turn);
    const float rho = rsqrtf(fmaf(sv[0], invH, a.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = threadIdx.x + k * blockDim.x;
      if (j >= nvec) continue;
      float w[8];
      load_weight<WT>(a.w2, 8 * j, a.offset, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= v[k][i] * rho;
      store8(static_cast<__nv_bfloat16*>(a.y) + o + 8 * j, w);
    }
  }
}

template <class XT, class DT, class WT, int NV>
__global__ void __launch_bounds__(kNormThreadsMax) k_norm_bwd(const NormArgs a) {
  __shared__ float red[128];
  pdl_wait();
  pdl_trigger();
  const int nvec = a.H / 8;
  const float invH = 1.f / (float)a.H;
  int turn = 0;
  float a1[NV][8] = {}, ag[NV][8] = {}, a2[NV][8] = {};
  for (long long r = blockIdx.x; r < a.N; r += gridDim.x) {
    const long long o = r * a.H;
    float v[NV][8], b[NV][8], d[NV][8];  // d: t = w2 dy, then dv, then w1 du
    float sb[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = threadIdx.x + k * blockDim.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = b[k][i] = 0.f;
      if (j < nvec) {
        Raw8<XT> rx;
        rx.load(static_cast<const XT*>(a.x) + o + 8 * j);
        rx.get(v[k]);
        if (a.b) {
          Raw8<__nv_bfloat16> rb;
          rb.load(static_cast<const __nv_bfloat16*>(a.b) + o + 8 * j);
          rb.get(b[k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sb[0] = fmaf(b[k][i], b[k][i], sb[0]);
    }
    float rho_b = 1.f;
    if (a.post) {
      block_sums(sb, red, turn);
      rho_b = rsqrtf(fmaf(sb[0], invH, a.eps));
    }
    float s2[2] = {0.f, 0.f};  // sum v^2, sum v t
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = threadIdx.x + k * blockDim.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[k][i] = 0.f;
      if (j >= nvec) continue;
      if (a.b) {
        float w[8], g[8];
        load_weight<WT>(a.post ? a.w1 : nullptr, 8 * j, a.offset, w);
        load_weight<WT>(a.g, 8 * j, 0.f, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          b[k][i] *= rho_b;  // normed from here on
          v[k][i] = fmaf(a.scale * g[i], b[k][i] * w[i], v[k][i]);
        }
      }
      if (a.pre) {
        float w[8];
        Raw8<DT> rd;
        rd.load(static_cast<const DT*>(a.dy) + o + 8 * j);
        rd.get(d[k]);
        load_weight<WT>(a.w2, 8 * j, a.offset, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s2[0] = fmaf(v[k][i], v[k][i], s2[0]);
          s2[1] = fmaf(v[k][i] * d[k][i], w[i], s2[1]);
        }
      }
    }
    float rho_v = 0.f, corr = 0.f;
    if (a.pre) {
      block_sums(s2, red, turn);
      rho_v = rsqrtf(fmaf(s2[0], invH, a.eps));
      corr = s2[1] * invH * rho_v * rho_v;
    }
    float sbt[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = threadIdx.x + k * blockDim.x;
      if (j >= nvec) continue;
      float dv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.dv) {
        Raw8<XT> rv;
        rv.load(static_cast<const XT*>(a.dv) + o + 8 * j);
        rv.get(dv);
      }
      if (a.pre) {
        float w[8];
        load_weight<WT>(a.w2, 8 * j, a.offset, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a2[k][i] = fmaf(d[k][i], v[k][i] * rho_v, a2[k][i]);
          dv[i] = fmaf(rho_v, fmaf(d[k][i], w[i], -v[k][i] * corr), dv[i]);
        }
      }
      if (a.dx) store8(static_cast<XT*>(a.dx) + o + 8 * j, dv);
      if (a.b) {
        float w[8], g[8];
        load_weight<WT>(a.post ? a.w1 : nullptr, 8 * j, a.offset, w);
        load_weight<WT>(a.g, 8 * j, 0.f, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float du = a.scale * dv[i];
          ag[k][i] = fmaf(du, b[k][i] * w[i], ag[k][i]);
          a1[k][i] = fmaf(du * g[i], b[k][i], a1[k][i]);
          d[k][i] = du * g[i] * w[i];
          sbt[0] = fmaf(b[k][i], d[k][i], sbt[0]);
        }
      }
    }
    if (!a.b || !a.db) continue;
    float mean = 0.f;
    if (a.post) {
      block_sums(sbt, red, turn);
      mean = sbt[0] * invH;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = threadIdx.x + k * blockDim.x;
      if (j >= nvec) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[k][i] = rho_b * fmaf(-mean, b[k][i], d[k][i]);
      store8(static_cast<__nv_bfloat16*>(a.db) + o + 8 * j, d[k]);
    }
  }
  float* p = a.part + (size_t)blockIdx.x * 3 * a.H;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int j = threadIdx.x + k * blockDim.x;
    if (j >= nvec) continue;
    if (a.want_w1) store8(p + 8 * j, a1[k]);
    if (a.want_g) store8(p + a.H + 8 * j, ag[k]);
    if (a.want_w2) store8(p + 2 * (size_t)a.H + 8 * j, a2[k]);
  }
}

// Column sums of the blocks' partials, in block order: gridDim.y picks dw1, dg
// or dw2; a block sums 128 columns, its eight warps every eighth partial.
__global__ void __launch_bounds__(256) k_norm_sum(const float* __restrict__ part, int blocks, int H,
                                                  float* dw1, float* dg, float* dw2) {
  __shared__ float4 red[8][32];
  pdl_wait();
  pdl_trigger();
  float* out = blockIdx.y == 0 ? dw1 : blockIdx.y == 1 ? dg : dw2;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 128 + lane * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < H) {
    const float* p = part + (size_t)blockIdx.y * H + col;
#pragma unroll 4
    for (int i = warp; i < blocks; i += 8) {
      const float4 q = *reinterpret_cast<const float4*>(p + (size_t)i * 3 * H);
      s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < H) {
    for (int w = 1; w < 8; ++w) {
      const float4 q = red[w][lane];
      s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
    }
    *reinterpret_cast<float4*>(out + col) = s;
  }
}

}  // namespace fckl
