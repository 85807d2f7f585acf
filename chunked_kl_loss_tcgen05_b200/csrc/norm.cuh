// The norms after and before a block, fused with the block's gate and residual
// scale, forward and backward, over rows of H values:
//   u = b rho_b w1 (post-norm)      v = x + s g u      y = v rho_v w2 (pre-norm)
//   rho_z = 1 / sqrt(mean(z^2) + eps)
//   t = w2 dy;  dx = dv = dv_in + rho_v t - v rho_v^3 mean(v t)
//   du = s g dv;  db = rho_b (w1 du) - b rho_b^3 mean(b w1 du)
//   dw2 = sum_r dy v rho_v;  dw1 = sum_r du b rho_b;  dg = sum_r s dv u
// With n = b rho_b (b without a post-norm), c = s g w1 and P = sum_r dv n:
//   v = x + c n,  dw1 = s g P,  dg = s w1 P,
// so the backward keeps two column sums, P and dw2, in registers; and, dv being
// dv_in + k1 t - k2 v for two scalars k1, k2 of the row, the mean that db needs is
// a combination of three sums that need neither:
//   sum c n dv = sum c n dv_in + k1 sum c n t - k2 sum c n v.
// All in fp32, two values to an instruction, from the inputs on (v is not
// rounded before it is normed; the backward forms v again from x and b), each
// output rounded once.
//
// Bound by HBM: forward x, b in and v, y out; backward x, b, dy, dv in and dx,
// db out.  16384 rows of 4096 in bf16, whole calls: 89 to 102 us (82 to 93% of a
// copy's speed) and 143 to 158 us (79 to 87%).  Rows go through a ring of
// shared-memory stages filled by 16-byte asynchronous copies, several rows ahead; a
// thread copies exactly the values it will read, so the data needs no barrier, and
// the waits are the copies' own.  A long row takes a block, a short one 32, 16 or 8 lanes of a warp (8, 16
// or 32 rows a block).  What limits the kernels below HBM speed is latency, of
// shuffles and barriers first: so all sums of a row go through one reduction,
// which also carries the next row's sum of b^2 (the only one that has to come
// before the others), and several values share a reduction's shuffles (three
// reductions a row took the backward 184 us).
#pragma once

#include "ptx.cuh"
#include "reduce.cuh"
#include "vec.cuh"

namespace fckl {

constexpr int kNormHMax = 8192;
constexpr int kNormLaneBlock = 256;  // threads of a block of rows shorter than a warp's reach

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

// Sums of K (2 or 8) values over the row's threads, the same on each of them.
// Lanes first split the values among them (xor 16, 8, 4: half of the values go
// to the partner), then finish one each.  `red` has room for two calls (`turn`
// alternates), so one barrier per call is enough; it starts zeroed, for the
// warps a block does not have.
constexpr int kNormRed = 2 * 8 * 16;
template <int kLanes, int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float* red, int& turn) {
  static_assert(K == 2 || K == 8, "values per reduction");
  constexpr int L = kLanes ? kLanes : 32;  // lanes that reduce by shuffles
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = K / 2, m = L / 2; n >= 1; n /= 2, m /= 2) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool up = lane & m;
      const float keep = up ? s[i + n] : s[i], give = up ? s[i] : s[i + n];
      s[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
  constexpr int kGroup = L / K;  // lanes that now share value (lane % L) / kGroup
  float x = s[0];
#pragma unroll
  for (int m = kGroup / 2; m >= 1; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
  if constexpr (kLanes == 0) {
    float* r = red + (turn & 1) * (kNormRed / 2);
    ++turn;
    if (lane % kGroup == 0) r[lane / kGroup * 16 + (threadIdx.x >> 5)] = x;
    __syncthreads();
    // value lane / kGroup: the group's lanes add its 16 warps' parts
    const float* q = r + lane / kGroup * 16;
    if constexpr (K == 8) {
      const float4 f = reinterpret_cast<const float4*>(q)[lane % kGroup];
      x = (f.x + f.y) + (f.z + f.w);
    } else {
      x = q[lane % kGroup];
    }
#pragma unroll
    for (int m = kGroup / 2; m >= 1; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = __shfl_sync(0xffffffffu, x, (lane & ~(L - 1)) + k * kGroup);
}

// Eight weights (+ offset), or ones.
template <class WT>
__device__ __forceinline__ void load_weight(const void* w, int col, float offset, float2 (&o)[4]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = both(1.f);
    return;
  }
  Raw8<WT> r;
  r.load(static_cast<const WT*>(w) + col);
  r.get(o);
#pragma unroll
  for (int i = 0; i < 4; ++i) { o[i].x += offset; o[i].y += offset; }
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
// All but the newest `stages` - 2 groups have landed.
__device__ __forceinline__ void copy_wait_two(int stages) {
  if (stages >= 4) copy_wait<2>();
  else if (stages == 3) copy_wait<1>();
  else copy_wait<0>();
}
constexpr int kNormStagesMax = 4;

// A thread's place in its row, and how the rows are dealt: kLanes lanes a row, or
// (0) a block.  The rows of one warp come and go together, so that its shuffles
// always meet; `on` tells whether this thread's row exists.
template <int kLanes>
struct NormRows {
  int tid, threads, place;  // within the row; the row's place in the block
  long long r, step, ahead; // row, rows per round, distance to the warp's first row
  __device__ __forceinline__ NormRows() {
    if (kLanes) {
      constexpr int L = kLanes ? kLanes : 32;
      tid = threadIdx.x % L; threads = L; place = threadIdx.x / L;
      r = blockIdx.x * (long long)(kNormLaneBlock / L) + place;
      step = gridDim.x * (long long)(kNormLaneBlock / L);
      ahead = place % (32 / L);
    } else {
      tid = threadIdx.x; threads = blockDim.x; place = 0;
      r = blockIdx.x; step = gridDim.x; ahead = 0;
    }
  }
};

// The ring: per stage the row's values of x, b, dv and dy one after another,
// each padded to all of the row's threads.  Threads past the row's end never
// copy; their places are zeroed once, so they read zeros.
template <class XT, class DT>
struct NormRing {
  uint8_t* base;
  int stages, off_b, off_dv, off_dy, bytes;
  __device__ __forceinline__ NormRing(uint8_t* ring, const NormArgs& a, int padded, int which)
      : stages(a.stages) {
    off_b = padded * (int)sizeof(XT);
    off_dv = off_b + (a.b ? padded * 2 : 0);
    off_dy = off_dv + (a.dv ? padded * (int)sizeof(XT) : 0);
    bytes = off_dy + (a.dy ? padded * (int)sizeof(DT) : 0);
    base = ring + which * stages * bytes;
  }
};

// Zeros for this thread's eight values at `col` of every stage.
template <class XT, class DT>
__device__ __forceinline__ void ring_zero(const NormRing<XT, DT>& g, const NormArgs& a, int col) {
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  for (int s = 0; s < g.stages; ++s) {
    uint8_t* p = g.base + s * g.bytes;
    for (int i = 0; i < (int)sizeof(XT) / 2; ++i) {
      reinterpret_cast<uint4*>(p + col * sizeof(XT))[i] = z;
      if (a.dv) reinterpret_cast<uint4*>(p + g.off_dv + col * sizeof(XT))[i] = z;
    }
    if (a.b) *reinterpret_cast<uint4*>(p + g.off_b + col * 2) = z;
    if (a.dy)
      for (int i = 0; i < (int)sizeof(DT) / 2; ++i)
        reinterpret_cast<uint4*>(p + g.off_dy + col * sizeof(DT))[i] = z;
  }
}

template <class T>
__device__ __forceinline__ void get8(const uint8_t* s, int col, float2 (&v)[4]) {
  Raw8<T> r;
  r.load(reinterpret_cast<const T*>(s) + col);
  r.get(v);
}
__device__ __forceinline__ void zero8(float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = both(0.f);
}

// What both directions keep per column: c = s g w1 and w2.
template <class WT, int NV>
__device__ __forceinline__ void norm_weights(const NormArgs& a, int tid, int threads,
                                             float2 (&c)[NV][4], float2 (&w2)[NV][4]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int col = 8 * (tid + k * threads);
    zero8(c[k]);
    zero8(w2[k]);
    if (col >= a.H) continue;
    float2 g[4];
    load_weight<WT>(a.post ? a.w1 : nullptr, col, a.offset, c[k]);
    load_weight<WT>(a.g, col, 0.f, g);
    load_weight<WT>(a.w2, col, a.offset, w2[k]);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[k][i] = mul2(c[k][i], mul2(both(a.scale), g[i]));
  }
}

// NV vectors of eight per thread: columns 8 (tid + k threads).
template <int kLanes, class XT, class WT, int NV>
__global__ void __launch_bounds__(kLanes ? 256 : 512, kLanes ? 2 : NV == 1 ? 2 : 1)
    k_norm_fwd(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float red[kNormRed];
  pdl_wait();
  pdl_trigger();
  const float invH = 1.f / (float)a.H;
  const NormRows<kLanes> rows;
  const NormRing<XT, float> g(ring, a, rows.threads * NV * 8, rows.place);
  float2 c[NV][4], w2[NV][4];
  norm_weights<WT, NV>(a, rows.tid, rows.threads, c, w2);
  for (int i = threadIdx.x; i < kNormRed; i += blockDim.x) red[i] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (8 * (rows.tid + k * rows.threads) >= a.H) ring_zero(g, a, 8 * (rows.tid + k * rows.threads));
  if constexpr (kLanes == 0) __syncthreads();
  auto fetch = [&](long long r, int stage) {
    if (r < a.N) {
      const long long o = r * a.H;
      uint8_t* s = g.base + stage * g.bytes;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = 8 * (rows.tid + k * rows.threads);
        if (col >= a.H) continue;
        copy8(s + col * sizeof(XT), static_cast<const XT*>(a.x) + o + col);
        if (a.b) copy8(s + g.off_b + col * 2, static_cast<const __nv_bfloat16*>(a.b) + o + col);
      }
    }
    copy_commit();
  };
  auto square_b = [&](int stage) {
    float2 q = both(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 b[4];
      get8<__nv_bfloat16>(g.base + stage * g.bytes + g.off_b, 8 * (rows.tid + k * rows.threads), b);
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(b[i], b[i], q);
    }
    return q.x + q.y;
  };
  int turn = 0, stage = 0;
  for (int i = 0; i < a.stages; ++i) fetch(rows.r + i * rows.step, i);
  float rho_b = 1.f;
  if (a.post && rows.r - rows.ahead < a.N) {
    copy_wait_two(a.stages);
    float s[2] = {square_b(0), 0.f};
    row_sums<kLanes>(s, red, turn);
    rho_b = rsqrtf(fmaf(s[0], invH, a.eps));
  }
  for (long long r = rows.r; r - rows.ahead < a.N; r += rows.step) {
    const bool on = r < a.N;
    copy_wait_two(a.stages);  // this row and the next one
    const uint8_t* s = g.base + stage * g.bytes;
    const long long o = r * a.H;
    const int next = stage + 1 == a.stages ? 0 : stage + 1;
    float2 v[NV][4], q = both(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = 8 * (rows.tid + k * rows.threads);
      get8<XT>(s, col, v[k]);
      if (a.b) {
        float2 b[4];
        get8<__nv_bfloat16>(s + g.off_b, col, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = fma2(c[k][i], mul2(b[i], both(rho_b)), v[k][i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(v[k][i], v[k][i], q);
    }
    float sums[2] = {q.x + q.y, a.post && r + rows.step < a.N ? square_b(next) : 0.f};
    fetch(r + a.stages * rows.step, stage);  // this thread has read its part of the stage
    stage = next;
    if (a.v) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = 8 * (rows.tid + k * rows.threads);
        if (on && col < a.H) store8(static_cast<XT*>(a.v) + o + col, v[k]);
      }
    }
    row_sums<kLanes>(sums, red, turn);
    rho_b = a.post ? rsqrtf(fmaf(sums[1], invH, a.eps)) : 1.f;
    if (!a.pre) continue;
    const float rho = rsqrtf(fmaf(sums[0], invH, a.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = 8 * (rows.tid + k * rows.threads);
      if (!on || col >= a.H) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k][i] = mul2(mul2(v[k][i], both(rho)), w2[k][i]);
      store8(static_cast<__nv_bfloat16*>(a.y) + o + col, v[k]);
    }
  }
  copy_wait<0>();
}

template <int kLanes, class XT, class DT, class WT, int NV>
__global__ void __launch_bounds__(kLanes ? 256 : 512, kLanes ? 2 : 1)
    k_norm_bwd(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float red[kNormRed];
  pdl_wait();
  pdl_trigger();
  const float invH = 1.f / (float)a.H;
  const NormRows<kLanes> rows;
  const NormRing<XT, DT> g(ring, a, rows.threads * NV * 8, rows.place);
  float2 c[NV][4], w2[NV][4], P[NV][4], D[NV][4];
  norm_weights<WT, NV>(a, rows.tid, rows.threads, c, w2);
  for (int i = threadIdx.x; i < kNormRed; i += blockDim.x) red[i] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    zero8(P[k]);
    zero8(D[k]);
    if (8 * (rows.tid + k * rows.threads) >= a.H) ring_zero(g, a, 8 * (rows.tid + k * rows.threads));
  }
  if constexpr (kLanes == 0) __syncthreads();
  auto fetch = [&](long long r, int stage) {
    if (r < a.N) {
      const long long o = r * a.H;
      uint8_t* s = g.base + stage * g.bytes;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = 8 * (rows.tid + k * rows.threads);
        if (col >= a.H) continue;
        copy8(s + col * sizeof(XT), static_cast<const XT*>(a.x) + o + col);
        if (a.b) copy8(s + g.off_b + col * 2, static_cast<const __nv_bfloat16*>(a.b) + o + col);
        if (a.dv) copy8(s + g.off_dv + col * sizeof(XT), static_cast<const XT*>(a.dv) + o + col);
        if (a.dy) copy8(s + g.off_dy + col * sizeof(DT), static_cast<const DT*>(a.dy) + o + col);
      }
    }
    copy_commit();
  };
  auto square_b = [&](int stage) {
    float2 q = both(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 b[4];
      get8<__nv_bfloat16>(g.base + stage * g.bytes + g.off_b, 8 * (rows.tid + k * rows.threads), b);
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(b[i], b[i], q);
    }
    return q.x + q.y;
  };
  int turn = 0, stage = 0;
  for (int i = 0; i < a.stages; ++i) fetch(rows.r + i * rows.step, i);
  float rho_b = 1.f;
  if (a.post && rows.r - rows.ahead < a.N) {
    copy_wait_two(a.stages);
    float s[2] = {square_b(0), 0.f};
    row_sums<kLanes>(s, red, turn);
    rho_b = rsqrtf(fmaf(s[0], invH, a.eps));
  }
  for (long long r = rows.r; r - rows.ahead < a.N; r += rows.step) {
    const bool on = r < a.N;
    copy_wait_two(a.stages);  // this row and the next one
    const uint8_t* s = g.base + stage * g.bytes;
    const long long o = r * a.H;
    const int next = stage + 1 == a.stages ? 0 : stage + 1;
    // With one vector a thread, the row's b, dy and dv stay in registers; with
    // two they are read from the ring again after the reduction (in registers
    // they would spill), which therefore refills the stage later.
    constexpr bool kKeep = NV == 1;
    float2 v[NV][4], n[kKeep ? NV : 1][4], dy[kKeep ? NV : 1][4], dv[kKeep ? NV : 1][4];
    float2 qv = both(0.f), qt = both(0.f), q1 = both(0.f), q2 = both(0.f), q3 = both(0.f);
    auto load = [&](int col, float2 (&bb)[4], float2 (&yy)[4], float2 (&vv)[4]) {
      if (a.b) get8<__nv_bfloat16>(s + g.off_b, col, bb); else zero8(bb);
      if (a.dy) get8<DT>(s + g.off_dy, col, yy); else zero8(yy);
      if (a.dv) get8<XT>(s + g.off_dv, col, vv); else zero8(vv);
#pragma unroll
      for (int i = 0; i < 4; ++i) bb[i] = mul2(bb[i], both(rho_b));
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = 8 * (rows.tid + k * rows.threads), h = kKeep ? k : 0;
      get8<XT>(s, col, v[k]);
      load(col, n[h], dy[h], dv[h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 m = mul2(c[k][i], n[h][i]), t = mul2(dy[h][i], w2[k][i]);
        v[k][i].x += m.x; v[k][i].y += m.y;
        qv = fma2(v[k][i], v[k][i], qv);
        qt = fma2(v[k][i], t, qt);
        q1 = fma2(m, dv[h][i], q1);
        q2 = fma2(m, t, q2);
        q3 = fma2(m, v[k][i], q3);
      }
    }
    float sums[8] = {qv.x + qv.y, qt.x + qt.y, q1.x + q1.y, q2.x + q2.y, q3.x + q3.y,
                     a.post && r + rows.step < a.N ? square_b(next) : 0.f, 0.f, 0.f};
    if (kKeep) fetch(r + a.stages * rows.step, stage);  // this thread's part has been read
    row_sums<kLanes>(sums, red, turn);
    float k1 = 0.f, k2 = 0.f;
    if (a.pre) {
      k1 = rsqrtf(fmaf(sums[0], invH, a.eps));
      k2 = sums[1] * invH * k1 * k1 * k1;
    }
    const float mean = a.post ? (sums[2] + k1 * sums[3] - k2 * sums[4]) * invH : 0.f;
    const float mb = -rho_b * mean;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = 8 * (rows.tid + k * rows.threads), h = kKeep ? k : 0;
      if (!on) continue;  // nothing of a row that is not there goes into P and D
      if (!kKeep) load(col, n[h], dy[h], dv[h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = mul2(dy[h][i], w2[k][i]);
        D[k][i] = fma2(dy[h][i], mul2(v[k][i], both(k1)), D[k][i]);
        dv[h][i] = fma2(both(-k2), v[k][i], fma2(both(k1), t, dv[h][i]));
        P[k][i] = fma2(dv[h][i], n[h][i], P[k][i]);
        n[h][i] = fma2(both(mb), n[h][i], mul2(both(rho_b), mul2(c[k][i], dv[h][i])));
      }
      if (col >= a.H) continue;
      if (a.dx) store8(static_cast<XT*>(a.dx) + o + col, dv[h]);
      if (a.db) store8(static_cast<__nv_bfloat16*>(a.db) + o + col, n[h]);
    }
    if (!kKeep) fetch(r + a.stages * rows.step, stage);
    stage = next;
    rho_b = a.post ? rsqrtf(fmaf(sums[5], invH, a.eps)) : 1.f;
  }
  copy_wait<0>();
  if (!a.dw1 && !a.dg && !a.dw2) return;
  float* p = a.part + (size_t)blockIdx.x * 2 * a.H;
  if constexpr (kLanes > 0) {  // the block's rows of sums become one, in order
    __syncthreads();
    float* sum = reinterpret_cast<float*>(ring);  // [rows of the block][2][H]
    float* w = sum + rows.place * 2 * a.H;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = 8 * (rows.tid + k * rows.threads);
      if (col >= a.H) continue;
      store8(w + col, P[k]);
      store8(w + a.H + col, D[k]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.H; i += blockDim.x) {
      float t = sum[i];
      for (int k = 1; k < kNormLaneBlock / (kLanes ? kLanes : 32); ++k) t += sum[k * 2 * a.H + i];
      p[i] = t;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = 8 * (rows.tid + k * rows.threads);
      if (col >= a.H) continue;
      store8(p + col, P[k]);
      store8(p + a.H + col, D[k]);
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
