// Host-side pieces shared by the library's translation units: sizes and
// alignment, tensor maps, launch with programmatic dependent launch, the
// environment knobs that apply to every entry point, and the event profiler.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <utility>
#include <vector>

#include "fckl.h"
#include "gemm.cuh"

namespace fckl {

constexpr size_t kAlign = 256;
constexpr int kMaxDevices = 64;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows per chunk: the caller's (0: the largest multiple of 128 rows whose
// 16-bit [rows, V] block, V padded to 64 columns, fits in 1 GiB -- at V = 128K
// a 4096-row chunk, deep enough that one dW read-modify-write (V*H*8 bytes) per
// chunk stays well under the chunk's dW tensor-core time, with few launches and
// tail waves), at most N.
inline long long resolve_rows(long long N, long long V, long long chunk) {
  long long C = chunk;
  if (C == 0) {
    const long long budget = 1024ll << 20;
    C = budget / ((long long)align_up((size_t)V, 64) * 2) / 128 * 128;
    if (C < 128) C = 128;
    const long long Nr = (long long)align_up((size_t)N, 64);
    if (C > Nr) C = Nr;
  }
  return C < N ? C : N;
}

// ---------------------------------------------------------------- tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// 2-D map (bf16 or fp32): inner (contiguous) extent, outer extent, outer
// stride in bytes, box {box_inner, box_outer}, 128-byte swizzle, zero fill out
// of bounds.
inline bool make_map(CUtensorMap* m, const void* base, long long inner, long long outer,
              long long stride_bytes, int box_inner, int box_outer, bool fp32 = false) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)stride_bytes};
  cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D view of a row-major bf16 [outer, inner] matrix (inner % 64 == 0) for
// MN-major operand loads: dims {64, outer, inner / 64}, strides {row pitch,
// 128 B}; a box {64, box_outer, 2} brings two adjacent 64-wide column chunks,
// stored chunk after chunk in shared memory exactly as two 2-D boxes would be.
inline bool make_map_mn3(CUtensorMap* m, const void* base, long long inner, long long outer,
                  long long stride_bytes, int box_outer) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr || inner % 64 != 0) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)outer, (cuuint64_t)(inner / 64)};
  cuuint64_t strides[2] = {(cuuint64_t)stride_bytes, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_outer, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// MN-major operand map: the 3-D form when the column count allows it and the
// driver accepts it (sets *is3d), else the 2-D form with 64-column boxes.
inline bool make_map_mn(CUtensorMap* m, const void* base, long long inner, long long outer,
                 long long stride_bytes, int* is3d) {
  *is3d = 0;
  if (inner % 64 == 0 && make_map_mn3(m, base, inner, outer, stride_bytes, BK)) {
    *is3d = 1;
    return true;
  }
  return make_map(m, base, inner, outer, stride_bytes, 64, BK);
}

// ---------------------------------------------------------------- knobs
inline uint64_t wait_timeout_ns() {
  const char* s = std::getenv("FCKL_WAIT_TIMEOUT_MS");
  long long ms = s ? std::atoll(s) : 2000;
  if (ms < 1) ms = 1;
  if (ms > 60000) ms = 60000;
  return (uint64_t)ms * 1000000ull;
}
// Programmatic dependent launch for the kernels of a call (FCKL_NO_PDL=1 turns
// it off: every kernel then starts after the previous one has completed).
inline bool pdl_enabled() {
  const char* s = std::getenv("FCKL_NO_PDL");
  return !(s && std::atoi(s) > 0);
}

// Launches `kernel` on `st`, with programmatic stream serialization when
// `pdl`: the kernel may start once every CTA of the previous kernel has
// called pdl_trigger() (or exited); it calls pdl_wait() before it touches what
// that kernel produces.  Kernels with compile-time cluster dimensions keep them.
template <typename... KArgs, typename... Args>
cudaError_t launch(bool pdl, void (*kernel)(KArgs...), dim3 grid, int block, size_t smem,
                   cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Ends the enclosing call with FCKL_ERR_CUDA when the launch fails.
#define FCKL_LAUNCH(kernel, grid, block, smem, ...)                                          \
  do {                                                                                       \
    if (::fckl::launch(pdl, kernel, dim3(grid), (int)(block), (size_t)(smem), st, __VA_ARGS__) != \
        cudaSuccess)                                                                         \
      return FCKL_ERR_CUDA;                                                                  \
  } while (0)

// ---------------------------------------------------------------- profiling
enum Kind {
  K_COUNT, K_PREP, K_FWD, K_MERGE, K_BWD, K_DH, K_DW, K_FINAL, K_ENT, K_ENT_MERGE, K_GATHER,
  K_SCATTER, K_SELECT, K_ZERO_DW, K_CE_FWD, K_CE_DLOGITS, K_DH_OUT,
  K_NORM_FWD, K_NORM_BWD, K_NORM_SUM, K_CE_SCALE, K_DHW, K_NKINDS
};
inline const char* const kKindName[K_NKINDS] = {
    "count_valid", "prep_teacher", "fwd_logits_lse", "merge_loss", "bwd_dlogits",
    "dH_gemm",     "dW_gemm",      "finalize",       "entropy_gemm", "merge_entropy",
    "gather_rows", "scatter_rows", "select_rows", "zero_dw", "ce_logits", "ce_dlogits",
    "dH_rows", "norm_fwd", "norm_bwd", "norm_sum",
    "ce_scale", "dH_dW_gemm"};
struct ProfRec {
  int kind;
  cudaEvent_t a, b;
  double flops, bytes;
};
struct Profiler {
  bool on = false;
  uint32_t mask = 0xFFFFFFFFu;
  std::vector<ProfRec> recs;
  std::vector<cudaEvent_t> pool;
  size_t used = 0;
  cudaEvent_t next() {
    if (used == pool.size()) {
      cudaEvent_t e = nullptr;
      if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
      pool.push_back(e);
    }
    return pool[used++];
  }
};
inline Profiler g_prof;

struct ProfScope {
  int kind;
  cudaStream_t st;
  double flops, bytes;
  cudaEvent_t a = nullptr;
  ProfScope(int k, cudaStream_t s, double f, double b) : kind(k), st(s), flops(f), bytes(b) {
    if (g_prof.on && ((g_prof.mask >> k) & 1u) && (a = g_prof.next()) != nullptr)
      cudaEventRecord(a, st);
  }
  ~ProfScope() {
    if (!g_prof.on || a == nullptr) return;
    cudaEvent_t b = g_prof.next();
    if (b == nullptr) return;
    cudaEventRecord(b, st);
    g_prof.recs.push_back(ProfRec{kind, a, b, flops, bytes});
  }
};

}  // namespace fckl
