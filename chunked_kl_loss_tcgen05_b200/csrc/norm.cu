// Host side of the fused norms: checks, launch shapes, workspace.
#include <algorithm>
#include <cmath>

#include "fckl.h"
#include "host.cuh"
#include "norm.cuh"

using namespace fckl;

namespace {

bool valid_norm(const fckl_norm_problem* p) {
  if (p == nullptr) return false;
  if (p->N < 1 || p->H < 1 || p->N > INT32_MAX || p->H > INT32_MAX) return false;
  if (!std::isfinite(p->scale) || !std::isfinite(p->weight_offset)) return false;
  if (!(p->eps >= 0.f && std::isfinite(p->eps))) return false;
  if (p->flags < 0 || p->flags > (FCKL_NORM_POST | FCKL_NORM_PRE)) return false;
  for (int t : {p->x_type, p->weight_type, p->dy_type})
    if (t != FCKL_FLOAT && t != FCKL_BFLOAT) return false;
  return true;
}
bool supported_norm(const fckl_norm_problem* p) { return p->H % 8 == 0 && p->H <= kNormHMax; }

// SMs of the current device if it is an sm_100, else 0.
int norm_sms() {
  static std::mutex mu;
  static int known[kMaxDevices];  // 0 unknown, -1 unusable
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0) {
    int major = 0, minor = 0, sms = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    known[dev] = major == 10 && minor == 0 && sms > 0 ? sms : -1;
  }
  return known[dev] > 0 ? known[dev] : 0;
}

constexpr int kSms = 148;             // of a B200: the workspace rule needs no GPU
constexpr size_t kRingBytes = 216 << 10;  // shared memory of an SM for the rings

// Launch shape.  A row takes 8, 16 or 32 lanes up to 64, 128 or 256 values, in
// the forward 32 lanes with two vectors each up to 512 (46 us for 65536 rows of
// 512; the backward would spill: 98 us, with blocks 75), else a block of as many
// threads as it has vectors (two vectors a thread beyond 4096 values).  `per_sm`
// blocks share an SM: 512 threads in the backward (at up to 128 registers), 1024
// in the forward; each gets its part of the ring memory, in 2 to 4 stages.
struct Shape {
  int lanes;  // 0: a block a row
  int threads, nv, per_sm, rows_per_block;
  int padded;  // values of a row in the ring (whole threads)
};
Shape norm_shape(long long H, bool bwd) {
  Shape s{};
  const int nvec = (int)(H / 8);
  s.lanes = H > (bwd ? 256 : 512) ? 0 : H <= 64 ? 8 : H <= 128 ? 16 : 32;
  if (s.lanes) {
    s.nv = nvec <= 32 ? 1 : 2;
    s.threads = kNormLaneBlock;
    s.rows_per_block = kNormLaneBlock / s.lanes;
  } else {
    s.nv = nvec <= 512 ? 1 : 2;
    s.threads = (int)align_up((size_t)cdiv(nvec, s.nv), 32);
    s.rows_per_block = 1;
  }
  s.padded = (s.lanes ? s.lanes : s.threads) * s.nv * 8;
  s.per_sm = std::max(1, (bwd || (s.nv == 2 && !s.lanes) ? 512 : 1024) / s.threads);
  return s;
}
int norm_grid(const Shape& s, long long N, int sms) {
  return (int)std::min<long long>(cdiv(N, s.rows_per_block), (long long)sms * s.per_sm);
}
// Ring stages that fit.
int norm_stages(const Shape& s, size_t row_bytes) {
  const size_t fit = kRingBytes / s.per_sm / (row_bytes * s.rows_per_block);
  return (int)std::max<size_t>(2, std::min<size_t>(kNormStagesMax, fit));
}

// The parts of the operation that the given arguments make impossible.
bool consistent(const fckl_norm_problem* p, const void* x, const void* block, const void* w1,
                const void* gate, const void* w2) {
  const bool post = p->flags & FCKL_NORM_POST, pre = p->flags & FCKL_NORM_PRE;
  if (!x || !aligned(x, 16) || !aligned(block, 16) || !aligned(w1, 16) || !aligned(gate, 16) ||
      !aligned(w2, 16))
    return false;
  if (!block && (post || gate || !pre)) return false;  // nothing to add: a plain pre-norm only
  if ((w1 && !post) || (w2 && !pre)) return false;
  return true;
}

NormArgs norm_args(const fckl_norm_problem* p, const void* x, const void* block, const void* w1,
                   const void* gate, const void* w2) {
  NormArgs a{};
  a.N = p->N; a.H = (int)p->H;
  a.scale = p->scale; a.eps = p->eps; a.offset = p->weight_offset;
  a.x = x; a.b = block; a.w1 = w1; a.g = gate; a.w2 = w2;
  a.post = (p->flags & FCKL_NORM_POST) ? 1 : 0;
  a.pre = (p->flags & FCKL_NORM_PRE) ? 1 : 0;
  return a;
}

using KernelFn = void (*)(const NormArgs);

template <class XT, class WT>
KernelFn pick_fwd(const Shape& s) {
  if (s.lanes == 8) return k_norm_fwd<8, XT, WT, 1>;
  if (s.lanes == 16) return k_norm_fwd<16, XT, WT, 1>;
  if (s.lanes == 32) return s.nv == 1 ? k_norm_fwd<32, XT, WT, 1> : k_norm_fwd<32, XT, WT, 2>;
  return s.nv == 1 ? k_norm_fwd<0, XT, WT, 1> : k_norm_fwd<0, XT, WT, 2>;
}
template <class XT, class DT, class WT>
KernelFn pick_bwd3(const Shape& s) {
  if (s.lanes == 8) return k_norm_bwd<8, XT, DT, WT, 1>;
  if (s.lanes == 16) return k_norm_bwd<16, XT, DT, WT, 1>;
  if (s.lanes == 32) return k_norm_bwd<32, XT, DT, WT, 1>;
  return s.nv == 1 ? k_norm_bwd<0, XT, DT, WT, 1> : k_norm_bwd<0, XT, DT, WT, 2>;
}
template <class XT, class DT>
KernelFn pick_bwd2(const fckl_norm_problem* p, const Shape& s) {
  return p->weight_type == FCKL_BFLOAT ? pick_bwd3<XT, DT, __nv_bfloat16>(s)
                                       : pick_bwd3<XT, DT, float>(s);
}
template <class XT>
KernelFn pick_bwd1(const fckl_norm_problem* p, const Shape& s) {
  return p->dy_type == FCKL_BFLOAT ? pick_bwd2<XT, __nv_bfloat16>(p, s) : pick_bwd2<XT, float>(p, s);
}

// Dynamic shared memory beyond 48 KB has to be allowed once per kernel and
// device.
bool allow_smem(KernelFn k) {
  static std::mutex mu;
  static std::vector<std::pair<KernelFn, int>> done;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lk(mu);
  for (const auto& d : done)
    if (d.first == k && d.second == dev) return true;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(SMEM_LIMIT - 1024)) != cudaSuccess)
    return false;
  done.emplace_back(k, dev);
  return true;
}

}  // namespace

extern "C" {

size_t fckl_block_norm_workspace_bytes(const fckl_norm_problem* prob) {
  if (!valid_norm(prob) || !supported_norm(prob)) return 0;
  const Shape s = norm_shape(prob->H, true);
  return align_up((size_t)norm_grid(s, prob->N, kSms) * 2 * prob->H * 4, kAlign);
}

fckl_status fckl_block_norm_fwd(const fckl_norm_problem* prob, const void* x, const void* block,
                                const void* post_weight, const void* gate, const void* pre_weight,
                                void* v, void* y, void* stream) {
  if (!valid_norm(prob) || !consistent(prob, x, block, post_weight, gate, pre_weight))
    return FCKL_ERR_INVALID_ARG;
  const bool pre = prob->flags & FCKL_NORM_PRE;
  if (pre != (y != nullptr) || (!pre && !v) || (!block && v) || !aligned(v, 16) || !aligned(y, 16))
    return FCKL_ERR_INVALID_ARG;
  if (!supported_norm(prob)) return FCKL_ERR_UNSUPPORTED;
  const int sms = norm_sms();
  if (sms == 0) return FCKL_ERR_UNSUPPORTED;
  NormArgs a = norm_args(prob, x, block, post_weight, gate, pre_weight);
  a.v = v; a.y = y;
  const Shape s = norm_shape(prob->H, false);
  const bool xb = prob->x_type == FCKL_BFLOAT, wb = prob->weight_type == FCKL_BFLOAT;
  const KernelFn k = xb ? (wb ? pick_fwd<__nv_bfloat16, __nv_bfloat16>(s)
                              : pick_fwd<__nv_bfloat16, float>(s))
                        : (wb ? pick_fwd<float, __nv_bfloat16>(s) : pick_fwd<float, float>(s));
  if (!allow_smem(k)) return FCKL_ERR_CUDA;
  const int grid = norm_grid(s, prob->N, sms);
  const size_t row_bytes = (size_t)s.padded * ((xb ? 2 : 4) + (block ? 2 : 0));
  a.stages = norm_stages(s, row_bytes);
  const bool pdl = pdl_enabled();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const double xs = xb ? 2.0 : 4.0, n = (double)prob->N * prob->H;
  ProfScope ps(K_NORM_FWD, st, 10.0 * n,
               n * (xs + (block ? 2.0 : 0.0) + (v ? xs : 0.0) + (y ? 2.0 : 0.0)));
  FCKL_LAUNCH(k, grid, s.threads, a.stages * row_bytes * s.rows_per_block, a);
  return FCKL_OK;
}

fckl_status fckl_block_norm_bwd(const fckl_norm_problem* prob, const void* x, const void* block,
                                const void* post_weight, const void* gate, const void* pre_weight,
                                const void* dy, const void* dv, void* dx, void* dblock,
                                float* dpost_weight, float* dgate, float* dpre_weight,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_norm(prob) || !consistent(prob, x, block, post_weight, gate, pre_weight))
    return FCKL_ERR_INVALID_ARG;
  const bool pre = prob->flags & FCKL_NORM_PRE;
  if (pre != (dy != nullptr) || (!pre && !dv) || !aligned(dy, 16) || !aligned(dv, 16) ||
      !aligned(dx, 16) || !aligned(dblock, 16) || !aligned(dpost_weight, 16) ||
      !aligned(dgate, 16) || !aligned(dpre_weight, 16))
    return FCKL_ERR_INVALID_ARG;
  if ((dblock && !block) || (dpost_weight && !post_weight) || (dgate && !gate) ||
      (dpre_weight && !pre_weight))
    return FCKL_ERR_INVALID_ARG;
  if (!dx && !dblock && !dpost_weight && !dgate && !dpre_weight) return FCKL_ERR_INVALID_ARG;
  if (!supported_norm(prob)) return FCKL_ERR_UNSUPPORTED;
  if (workspace == nullptr || !aligned(workspace, kAlign) ||
      workspace_bytes < fckl_block_norm_workspace_bytes(prob))
    return FCKL_ERR_WORKSPACE;
  const int sms = norm_sms();
  if (sms == 0) return FCKL_ERR_UNSUPPORTED;
  NormArgs a = norm_args(prob, x, block, post_weight, gate, pre_weight);
  a.dy = dy; a.dv = dv; a.dx = dx; a.db = dblock;
  a.part = static_cast<float*>(workspace);
  a.dw1 = dpost_weight; a.dg = dgate; a.dw2 = dpre_weight;
  const Shape s = norm_shape(prob->H, true);
  const bool xb = prob->x_type == FCKL_BFLOAT;
  const KernelFn k = xb ? pick_bwd1<__nv_bfloat16>(prob, s) : pick_bwd1<float>(prob, s);
  if (!allow_smem(k)) return FCKL_ERR_CUDA;
  const int grid = norm_grid(s, prob->N, std::min(sms, kSms));  // the workspace's partials
  const size_t row_bytes = (size_t)s.padded * ((xb ? 2 : 4) * (dv ? 2 : 1) + (block ? 2 : 0) +
                                              (dy ? (prob->dy_type == FCKL_BFLOAT ? 2 : 4) : 0));
  a.stages = norm_stages(s, row_bytes);
  size_t smem = a.stages * row_bytes * s.rows_per_block;
  if (s.lanes)  // the sums of the block's rows take its place at the end
    smem = std::max(smem, (size_t)s.rows_per_block * 2 * prob->H * 4);
  const bool pdl = pdl_enabled();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const double xs = xb ? 2.0 : 4.0, n = (double)prob->N * prob->H;
  {
    ProfScope ps(K_NORM_BWD, st, 30.0 * n,
                 n * (xs + (block ? 2.0 : 0.0) +
                      (dy ? (prob->dy_type == FCKL_BFLOAT ? 2.0 : 4.0) : 0.0) +
                      (dv ? xs : 0.0) + (dx ? xs : 0.0) + (dblock ? 2.0 : 0.0)));
    FCKL_LAUNCH(k, grid, s.threads, smem, a);
  }
  if (dpost_weight || dgate || dpre_weight) {
    ProfScope ps(K_NORM_SUM, st, 0.0, 8.0 * grid * prob->H);
    FCKL_LAUNCH(prob->weight_type == FCKL_BFLOAT ? k_norm_sum<__nv_bfloat16> : k_norm_sum<float>,
                dim3((unsigned)cdiv(prob->H, 64), 2), 512, 0, (const NormArgs)a, grid);
  }
  return FCKL_OK;
}

}  // extern "C"
