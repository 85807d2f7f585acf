// Host side of the fused norms: checks, launch shapes, workspace.
#include <algorithm>
#include <cmath>

#include "fckl.h"
#include "host.cuh"
#include "norm.cuh"

using namespace fckl;

namespace {

// Blocks whose weight-gradient partials the workspace has room for.
constexpr int kNormBlocks = 4 * 148;

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

int norm_blocks(const fckl_norm_problem* p) { return (int)std::min<long long>(p->N, kNormBlocks); }

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

// Threads per block and vectors of eight values per thread.
struct Shape {
  int threads, nv;
};
Shape norm_shape(long long H) {
  const int nvec = (int)(H / 8);
  const int nv = nvec <= 256 ? 1 : 2;
  return Shape{(int)align_up((size_t)cdiv(nvec, nv), 32), nv};
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
KernelFn pick_fwd(int nv) { return nv == 1 ? k_norm_fwd<XT, WT, 1> : k_norm_fwd<XT, WT, 2>; }
template <class XT, class DT, class WT>
KernelFn pick_bwd3(int nv) { return nv == 1 ? k_norm_bwd<XT, DT, WT, 1> : k_norm_bwd<XT, DT, WT, 2>; }
template <class XT, class DT>
KernelFn pick_bwd2(const fckl_norm_problem* p, int nv) {
  return p->weight_type == FCKL_BFLOAT ? pick_bwd3<XT, DT, __nv_bfloat16>(nv)
                                       : pick_bwd3<XT, DT, float>(nv);
}
template <class XT>
KernelFn pick_bwd1(const fckl_norm_problem* p, int nv) {
  return p->dy_type == FCKL_BFLOAT ? pick_bwd2<XT, __nv_bfloat16>(p, nv) : pick_bwd2<XT, float>(p, nv);
}

}  // namespace

extern "C" {

size_t fckl_block_norm_workspace_bytes(const fckl_norm_problem* prob) {
  if (!valid_norm(prob) || !supported_norm(prob)) return 0;
  return align_up((size_t)norm_blocks(prob) * 3 * prob->H * 4, kAlign);
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
  const Shape s = norm_shape(prob->H);
  const bool xb = prob->x_type == FCKL_BFLOAT, wb = prob->weight_type == FCKL_BFLOAT;
  const KernelFn k = xb ? (wb ? pick_fwd<__nv_bfloat16, __nv_bfloat16>(s.nv)
                              : pick_fwd<__nv_bfloat16, float>(s.nv))
                        : (wb ? pick_fwd<float, __nv_bfloat16>(s.nv) : pick_fwd<float, float>(s.nv));
  const int per_sm = std::max(1, std::min(16, 1536 / s.threads));
  const int grid = (int)std::min<long long>(prob->N, (long long)sms * per_sm);
  const bool pdl = pdl_enabled();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const double xs = xb ? 2.0 : 4.0, n = (double)prob->N * prob->H;
  ProfScope ps(K_NORM_FWD, st, 10.0 * n,
               n * (xs + (block ? 2.0 : 0.0) + (v ? xs : 0.0) + (y ? 2.0 : 0.0)));
  FCKL_LAUNCH(k, grid, s.threads, 0, a);
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
  a.want_w1 = dpost_weight != nullptr;
  a.want_g = dgate != nullptr;
  a.want_w2 = dpre_weight != nullptr;
  const Shape s = norm_shape(prob->H);
  const bool xb = prob->x_type == FCKL_BFLOAT;
  const KernelFn k = xb ? pick_bwd1<__nv_bfloat16>(prob, s.nv) : pick_bwd1<float>(prob, s.nv);
  const int grid = norm_blocks(prob);
  const bool pdl = pdl_enabled();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const double xs = xb ? 2.0 : 4.0, n = (double)prob->N * prob->H;
  {
    ProfScope ps(K_NORM_BWD, st, 30.0 * n,
                 n * (xs + (block ? 2.0 : 0.0) + (dy ? (prob->dy_type == FCKL_BFLOAT ? 2.0 : 4.0) : 0.0) +
                      (dv ? xs : 0.0) + (dx ? xs : 0.0) + (dblock ? 2.0 : 0.0)));
    FCKL_LAUNCH(k, grid, s.threads, 0, a);
  }
  if (dpost_weight || dgate || dpre_weight) {
    ProfScope ps(K_NORM_SUM, st, 0.0, 12.0 * grid * prob->H);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cdiv(prob->H, 128), 3, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, k_norm_sum, (const float*)a.part, grid, (int)prob->H, dpost_weight,
                           dgate, dpre_weight) != cudaSuccess)
      return FCKL_ERR_CUDA;
  }
  return FCKL_OK;
}

}  // extern "C"
