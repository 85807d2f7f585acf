// Host side of the vocabulary cross entropy: checks, workspace layout and the
// chunk loop.  Per chunk of C kept rows, on the caller's stream:
//   gather rows -> logits GEMM (log-sum-exp epilogue), or W streamed past one or
//   two rows -> merge (row losses; the last block adds up the loss),
// with gradients
//   gather rows -> logits GEMM (and its exponentials) -> merge and dlogits, or,
//   for given log-sum-exps, gather rows -> logits GEMM (dlogits epilogue),
//   -> dH GEMM -> dW GEMM -> dH rows.  (Short hidden rows take the forward's steps
//   and then those of given log-sum-exps.)
#include <algorithm>
#include <cmath>

#include "ce.cuh"
#include "fckl.h"
#include "host.cuh"

using namespace fckl;

namespace {

// Sleep of an epilogue between polls, per k-block of its unit.  A k-block takes
// a pair about 280 ns, so this is a tenth of the main loop; 2 us regardless of
// it, as long loops can afford, cost 476 us against 417 in a step of
// 1531 x 1024 x 50257.
constexpr int kPollNs = 30;

// The tensor cores add 16 products at a time to an fp32 accumulator and cut the
// sum instead of rounding it, H / 16 times: the logits come out too small in
// magnitude, by how much depends on how the sum grows.  In units of (H / 16) 2^-23
// of the logit, measured for H from 1024 to 16384 and logits from 12 to 30: 0.13 to
// 0.17 where the products are noise around a mean (what a hidden row and a row of W
// that it has learned make), 0.25 to 0.67 where all have one sign, nothing where the
// partial sums are exact (a few nonzero values).  The scale that the epilogues
// multiply the logits with makes up for 0.14 of it, the first kind, and so leaves a
// logit off by -0.55 to +0.14 units of itself instead of -0.67 to 0 (one unit is 3e-5
// at H = 4096).  The label's logit and the streamed rows are rounded sums and not
// scaled, so a column equal to the label's is off against it by that much.
constexpr double kCutShare = 0.14;

// Calls of one row tile run their dH GEMM (which reads W) and their dW GEMM (which
// writes as much) side by side, on 3/8 and 5/8 of the CTA pairs, unless W is large:
// small ones are bound by launches and tails, large ones by memory, and with 5/8 of
// the pairs dW does not reach its rate.  More rows carry it further with bf16
// gradients, where the products grow and dW's bytes do not; fp32 ones cost more when
// dH goes first.
// Graph-timed steps with L2 flushed, us, one after the other and side by side; bf16
// gradients: 256 x 256 x 4096 37 and 35, 16 x 512 x 32000 55 and 51, 256 x 1024 x 32000 96
// and 86, 16 x 2880 x 8192 66 and 70, 64 x 1024 x 50257 96 and 107, 128 x 4096 x 128256
// 721 and 862; fp32: 64 x 1024 x 50257 119 and 115, 64 x 2048 x 32000 both 137, 128 x 4096 x
// 128256 919 and 1001.  Two row tiles: 384 x 2880 x 8192 92 and 98.
constexpr int kTwoRows = PM;
bool ce_two(long long rows, long long V, long long H, bool bf16_grads) {
  if (rows > kTwoRows) return false;
  return V * H <= (bf16_grads ? (1ll << 24) + rows * (1ll << 17) : 1ll << 26);
}

// Room for the k segments of a chunk's dH GEMM: four units for every CTA pair
// of a B200 (more would mean more slabs to sum than waves to balance), 256 KB
// each, or one segment of every tile; and no more than the GEMM can choose, which
// has a k-block of the vocabulary at least in a segment and at most 128 segments.
constexpr int kSlabUnits = 4 * 74;

enum class CeMode { kFwd, kFwdBwd, kBwd };

struct CeLayout {
  long long C, Vp, NT, NTh, nchunks;
  int slab_units;
  size_t off_list, off_share, off_lab, off_kw, off_zlab, off_lse2, off_rest, off_part, off_zsum,
      off_h, off_dlog, off_slab, off_dw, total;
};

bool valid_ce(const fckl_ce_problem* p) {
  if (p == nullptr) return false;
  if (p->N < 1 || p->H < 1 || p->V < 1 || p->chunk < 0) return false;
  if (p->N > INT32_MAX || p->H > INT32_MAX || p->V > INT32_MAX) return false;
  if (!(std::isfinite(p->T) && p->T > 0.f)) return false;
  if (!(p->label_smoothing >= 0.f && p->label_smoothing <= 1.f)) return false;
  if (!(p->z_loss >= 0.f && std::isfinite(p->z_loss))) return false;
  if (p->label_type != FCKL_LABELS_INT && p->label_type != FCKL_LABELS_LONG) return false;
  if (p->reduction != FCKL_REDUCE_MEAN && p->reduction != FCKL_REDUCE_SUM) return false;
  if (p->grad_type != FCKL_GRAD_FLOAT && p->grad_type != FCKL_GRAD_BFLOAT) return false;
  if (p->n_valid_total < 0 || p->n_valid_total > INT32_MAX) return false;
  return true;
}

bool supported_ce(const fckl_ce_problem* p) { return p->H % 8 == 0; }

// Rows per chunk: the caller's, or the library's automatic rows (resolve_rows)
// but no fewer than 4096 and no more than 32768, spread evenly over the nearest
// number of chunks, so that no chunk is a remainder (3/4 to 3/2 of that number,
// then): every chunk beyond the first reads W twice and reads and writes dW once
// more.  Measured with bf16 gradients, us per step: 4096 x 2880 x 201088 (2660 kept
// rows) 10430 at the 2560 rows of 1 GiB, 7900 at 4096; 16384 x 4096 x 128256 43700 at
// 4096 rows, 45900 at 8192, 49000 at 16384 (there the gathered rows no longer stay in
// L2 beside W).
// The upper end is for accuracy: dW sums a chunk's rows on the tensor cores, which
// cut every partial sum, and a sum of one sign comes out short by 0.7 to 0.8 (rows /
// 16) 2^-23 of itself; the chunks' sums are rounded.  262144 x 1024 x 1000 (small
// vocabularies would fit far more rows into 1 GiB): 1.6e-3 short in one chunk, 3490
// us, 1.8e-4 and 3580 at 32768 rows, 8e-5 and 3730 at 16384.
constexpr long long kAutoRowsMin = 4096, kAutoRowsMax = 32768;
long long ce_rows(const fckl_ce_problem* p) {
  if (p->chunk > 0) return std::min<long long>(p->chunk, p->N);
  const long long want =
      std::clamp<long long>(resolve_rows(INT32_MAX, p->V, 0), kAutoRowsMin, kAutoRowsMax);
  const long long chunks = std::max<long long>(1, (p->N + want / 2) / want);
  return std::min<long long>(p->N, (long long)align_up((size_t)cdiv(p->N, chunks), 128));
}

// Scoring calls of one or two rows stream W past them instead of multiplying
// tiles of 256 rows, whose products alone take 157 us at 4096 x 128256 (W's bytes: 163
// at a copy's rate, which a read alone beats).
// Graph-timed, us, tiles and streamed: one row 4096 x 128256 184 and 157, 2048 x 32000
// 38 and 28, 1344 x 583 19 and 10; two rows of 4096 x 128256 184 and 170.  Four rows
// (184 and 188) and eight (184 and 373) are bound by the sums' arithmetic.
bool ce_few(long long C) { return C <= kFewRows; }

template <int kRows, int kAhead>
auto ce_few_kernel(bool smooth) {
  return smooth ? k_ce_few<kRows, kAhead, true> : k_ce_few<kRows, kAhead, false>;
}

CeLayout ce_layout(const fckl_ce_problem* p, bool grads) {
  CeLayout L{};
  L.C = ce_rows(p);
  L.Vp = (long long)align_up((size_t)p->V, 64);
  L.NT = cdiv(p->V, BN);
  L.NTh = cdiv(p->H, BN);
  L.nchunks = cdiv(p->N, L.C);
  const long long tiles = cdiv(L.C, PM) * L.NTh;
  const long long segments = std::min<long long>(cdiv(p->V, BK), kMaxSplit);
  L.slab_units = (int)std::min<long long>(
      {std::max<long long>(tiles, kSlabUnits), tiles * segments, INT32_MAX});
  size_t off = align_up(sizeof(DeviceCtl), kAlign);
  auto take = [&](size_t bytes) { size_t o = off; off = align_up(off + bytes, kAlign); return o; };
  const size_t C = (size_t)L.C;
  L.off_list = take((size_t)p->N * 4);
  L.off_share = take((size_t)p->N * 4);
  L.off_lab = take(C * 4);
  L.off_kw = take(C * 4);
  L.off_zlab = take(C * 4);
  L.off_lse2 = take(C * 4);
  L.off_rest = take(C * 4);
  const size_t NP = (size_t)std::max(2 * L.NT, ce_few(L.C) ? cdiv(p->V, kFewCols) : 0);
  L.off_part = take(C * NP * sizeof(float2));
  L.off_zsum = take(p->label_smoothing > 0.f ? C * NP * 4 : 0);
  L.off_h = take(align_up(C, CM) * p->H * 2);
  L.off_dlog = take(grads ? C * L.Vp * 2 : 0);
  // S segments of MT row tiles fit when S * MT * NTh <= slab_units
  L.off_slab = take(grads ? (size_t)(L.slab_units / L.NTh) * PM * p->H * 4 : 0);
  // bf16 gradients of several chunks are summed in fp32 first
  L.off_dw = take(grads && L.nchunks > 1 && p->grad_type == FCKL_GRAD_BFLOAT
                      ? (size_t)p->V * p->H * 4 : 0);
  L.total = off;
  return L;
}

// Chunks of so few rows that a warp a row would leave SMs idle merge them with a
// block each (one row against 128256 columns: 9.6 us with a warp, 6.5 with a block).
bool ce_block_rows(long long cap) { return cap <= 148 * kCeWarps; }

struct CeRequest {
  CeMode mode = CeMode::kFwd;
  const fckl_ce_problem* prob = nullptr;
  const void* hidden = nullptr;
  const void* W = nullptr;
  const void* labels = nullptr;
  const float* factor = nullptr;  // row weight, or the upstream row gradient
  const float* lse_in = nullptr;
  float* loss = nullptr;
  float* row_loss = nullptr;
  float* lse_out = nullptr;
  void* dH = nullptr;
  void* dW = nullptr;
  void* workspace = nullptr;
  size_t ws_bytes = 0;
  void* stream = nullptr;
};

// The dlogits kernel gives a row to a warp instead of blocks where the vocabulary
// is too small to keep 256 threads busy and the rows fill the SMs.
bool ce_warp_dlogits(long long V, long long cap) { return V <= 8192 && !ce_block_rows(cap); }

// Whether a training call computes the logits twice after all: with short hidden
// rows the second product costs less than keeping the exponentials (written,
// read, written as dlogits), as long as those do not stay in L2.  Graph-timed
// steps, us, kept and recomputed: 1531 x 384 x 50257 258 and 245, 4096 x 256 x 128256
// 1260 and 1150, 4096 x 512 x 50257 694 and 693, 1024 x 256 x 32000 102 and 108.
bool ce_recompute(CeMode mode, const fckl_ce_problem* p, const CeLayout& L) {
  return mode == CeMode::kFwdBwd && p->H <= 384 && L.C * L.Vp >= (1ll << 26);
}

template <class E2>
bool allow_smem_two() {
  return cudaFuncSetAttribute(gemm_two_kernel<EpiCeDH, false, true, E2, true, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)std::max(pair_smem_bytes<EpiCeDH>(), pair_smem_bytes<E2>())) ==
         cudaSuccess;
}

template <class Epi, bool A_MN, bool B_MN>
bool allow_smem() {
  return cudaFuncSetAttribute(gemm_pair_kernel<Epi, A_MN, B_MN>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)pair_smem_bytes<Epi>()) == cudaSuccess;
}

struct CeDevice {
  bool ready = false, ok = false;
  int sms = 0;
};
CeDevice g_ce_dev[kMaxDevices];
std::mutex g_ce_mu;

const CeDevice* ce_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_ce_mu);
  CeDevice& d = g_ce_dev[dev];
  if (!d.ready) {
    d.ready = true;
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    d.ok = major == 10 && minor == 0 && d.sms > 1 && allow_smem<EpiCe<false>, false, false>() &&
           allow_smem<EpiCe<true>, false, false>() &&
           allow_smem<EpiCeStore<false>, false, false>() &&
           allow_smem<EpiCeStore<true>, false, false>() &&
           allow_smem<EpiCeDlogits, false, false>() &&
           allow_smem<EpiCeDH, false, true>() && allow_smem<EpiCeDW, true, true>() &&
           allow_smem<EpiCeDWSum, true, true>() && allow_smem_two<EpiCeDW>() &&
           allow_smem_two<EpiCeDWSum>();
  }
  return &d;
}

template <class Label>
fckl_status enqueue_ce(const CeRequest& q, const CeLayout& L, const CeDevice* dev) {
  const fckl_ce_problem* prob = q.prob;
  const bool grads = q.mode != CeMode::kFwd;
  const bool bf16_grads = prob->grad_type == FCKL_GRAD_BFLOAT;
  const int H = (int)prob->H, V = (int)prob->V;
  const long long N = prob->N;
  const Label* labels = static_cast<const Label*>(q.labels);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(q.stream);
  const bool pdl = pdl_enabled();
  uint8_t* ws = static_cast<uint8_t*>(q.workspace);
  DeviceCtl* ctl = reinterpret_cast<DeviceCtl*>(ws);
  auto at = [&](size_t off) { return static_cast<void*>(ws + off); };
  int32_t* list = static_cast<int32_t*>(at(L.off_list));
  float* share = static_cast<float*>(at(L.off_share));
  int* lab = static_cast<int*>(at(L.off_lab));
  float* kw = static_cast<float*>(at(L.off_kw));
  float* zlab = static_cast<float*>(at(L.off_zlab));
  float* lse2 = static_cast<float*>(at(L.off_lse2));
  float* rest = static_cast<float*>(at(L.off_rest));
  float2* part = static_cast<float2*>(at(L.off_part));
  float* zsum = static_cast<float*>(at(L.off_zsum));
  __nv_bfloat16* hst = static_cast<__nv_bfloat16*>(at(L.off_h));
  __nv_bfloat16* dlog = static_cast<__nv_bfloat16*>(at(L.off_dlog));
  float* slab = static_cast<float*>(at(L.off_slab));
  const float invT = 1.f / prob->T;
  const float scale2 = (float)(1.4426950408889634 / prob->T *
                               (1.0 + kCutShare * (H / 16.0) / 8388608.0));
  const CtlArgs ca{ctl, wait_timeout_ns(), 0};
  const int pairs = dev->sms / 2;
  const int NT = (int)L.NT, NTh = (int)L.NTh, NP = 2 * NT;  // log-sum-exp partials of 128 columns
  const int KBh = (int)cdiv(H, BK), KBv = (int)cdiv(V, BK);
  const int narrow_h = (H % BN != 0 && H % BN <= 128) ? 1 : 0;
  const bool smooth = prob->label_smoothing > 0.f;

  // Rows by label.  Few rows of one chunk are selected and gathered at once (a
  // block a row, each reading all labels: up to 1024 of them cost less than a
  // launch); else one block selects up to 8192 rows (more passes of 4096 rows
  // would cost more than the second launch and the memset they save).
  const bool at_once = N <= 1024 && L.nchunks == 1;
  {
    const int denom = q.mode == CeMode::kBwd || prob->reduction == FCKL_REDUCE_SUM
                          ? 1 : (int)prob->n_valid_total;
    const long long R =
        N <= 8192 ? 8192
                  : std::max<long long>(4096, cdiv(cdiv(N, kCompactBlocks), 4096) * 4096);
    const int nb = (int)cdiv(N, R);
    ProfScope ps(K_COUNT, st, 0.0, (double)N * (sizeof(Label) * (nb > 1 ? 2 : 1) + 4));
    if (at_once) {
      FCKL_LAUNCH(k_ce_select<Label>, N, 128, 0, labels, (int)N, (long long)prob->ignore_index, V,
                  denom, list, ctl, H, static_cast<const __nv_bfloat16*>(q.hidden),
                  static_cast<const __nv_bfloat16*>(q.W), q.factor, q.lse_in, hst, lab, zlab, kw,
                  lse2);
    } else {
      if (nb > 1) {
        if (cudaMemsetAsync(ctl, 0, sizeof(DeviceCtl), st) != cudaSuccess) return FCKL_ERR_CUDA;
        FCKL_LAUNCH(k_ce_count<Label>, nb, 1024, 0, labels, N, R, (long long)prob->ignore_index, V,
                    ctl);
      }
      FCKL_LAUNCH(k_ce_list<Label>, nb, 1024, 0, labels, N, R, (long long)prob->ignore_index, V,
                  denom, list, ctl);
    }
  }
  const bool recompute = ce_recompute(q.mode, prob, L);
  // Blocks of the row kernels that leave loss shares, over all chunks.
  unsigned blocks = 0;
  for (long long c = 0; c < L.nchunks; ++c) {
    const long long cap = std::min(L.C, N - c * L.C);
    const bool warps = q.mode == CeMode::kFwd || recompute ? !ce_block_rows(cap)
                                                           : ce_warp_dlogits(prob->V, cap);
    blocks += (unsigned)(warps ? cdiv(cap, kCeWarps) : cap);
  }

  CUtensorMap mapW_k, mapW_mn, mapdW, mapSlab;
  int w3d = 0;
  if (!make_map(&mapW_k, q.W, H, V, (long long)H * 2, BK, BN / 2)) return FCKL_ERR_CUDA;
  // dW goes to the caller (fp32 always; bf16 when one chunk computes all of
  // it) or to the fp32 sum in the workspace.
  void* dw_dst = bf16_grads && L.nchunks > 1 ? at(L.off_dw) : q.dW;
  const bool dw_direct16 = bf16_grads && L.nchunks == 1;
  if (q.dW) {
    if (dw_direct16 ? !make_map(&mapdW, dw_dst, H, V, (long long)H * 2, 64, 32)
                    : !make_map(&mapdW, dw_dst, H, V, (long long)H * 4, 32, 32, true))
      return FCKL_ERR_CUDA;
  }
  if (q.dH) {
    if (!make_map_mn(&mapW_mn, q.W, H, V, (long long)H * 2, &w3d)) return FCKL_ERR_CUDA;
    if (!make_map(&mapSlab, slab, H, (long long)(L.slab_units / NTh) * PM, (long long)H * 4, 32, 32,
                  true))
      return FCKL_ERR_CUDA;
  }
  auto grid_for = [&](long long units) {
    return (int)(2 * std::max<long long>(1, std::min<long long>(pairs, units)));
  };

  for (long long c = 0; c < L.nchunks; ++c) {
    const long long row0 = c * L.C;
    const int cap = (int)std::min(L.C, N - row0);
    const int32_t* clist = list + row0;
    const RowCount rc{-1, ctl, (int)row0, cap};
    const double nr = (double)cap, flops = 2.0 * nr * V * H;
    const long long MT = cdiv(cap, PM);
    if (!at_once) {
      ProfScope ps(K_GATHER, st, 0.0, nr * (H * 6.0 + 20.0));
      FCKL_LAUNCH(k_ce_gather<Label>, cap, 128, 0, clist, rc, H,
                  static_cast<const __nv_bfloat16*>(q.hidden),
                  static_cast<const __nv_bfloat16*>(q.W), labels, q.factor, q.lse_in, hst, lab,
                  zlab, kw, lse2);
    }
    CUtensorMap mapH_k;
    // whole boxes of 128 rows: a box that reaches past the map's end loads more
    // slowly (one row against a 128K vocabulary: 280 us, with whole boxes 220);
    // what the rows behind the last one hold only reaches their own logits
    if (!make_map(&mapH_k, hst, H, (long long)align_up(cap, CM), (long long)H * 2, BK, CM))
      return FCKL_ERR_CUDA;
    SchedArgs sa_v{SCHED_VOCAB_MAJOR, NT, KBh, 1, 0, rc, 0, 0};
    sa_v.poll_ns = kPollNs;
    sa_v.fresh_rows = at_once ? 1 : 0;
    const int Gv = grid_for(MT * NT);
    CUtensorMap mapD_st, mapD_k, mapD_mn, mapH_mn;
    if (grads && !make_map(&mapD_st, dlog, L.Vp, cap, L.Vp * 2, 64, 32)) return FCKL_ERR_CUDA;
    const float* zs = smooth ? zsum : nullptr;
    // The GEMM over h W^T: its row count, hence its work, is read on the device.
#define FCKL_CE_GEMM(Epi, map, params)                                        \
  FCKL_LAUNCH((gemm_pair_kernel<Epi, false, false>), Gv, gemm_threads<Epi>(), \
              pair_smem_bytes<Epi>(), mapH_k, mapW_k, map, params, sa_v, ca)
    if (q.mode == CeMode::kFwd || recompute) {
      const bool few = q.mode == CeMode::kFwd && ce_few(L.C);
      const int NPm = few ? (int)cdiv(V, kFewCols) : NP;
      if (few) {
        ProfScope ps(K_CE_FWD, st, flops, 2.0 * (nr + V) * H + nr * NPm * 8.0);
        auto few_kernel = cap == 1 ? ce_few_kernel<1, 2>(smooth) : ce_few_kernel<2, 4>(smooth);
        FCKL_LAUNCH(few_kernel, (int)cdiv(V, kFewCols), 256, 0, rc, cap, H, V, NPm,
                    (float)(1.4426950408889634 / prob->T), (const __nv_bfloat16*)hst,
                    static_cast<const __nv_bfloat16*>(q.W), (const int*)lab, part, zsum);
      } else {
        ProfScope ps(K_CE_FWD, st, flops, 2.0 * (nr + V) * H + nr * NT * 8.0);
        if (smooth) {
          EpiCe<true>::Params pf{V, NP, scale2, lab, part, zsum};
          FCKL_CE_GEMM(EpiCe<true>, mapW_k, pf);
        } else {
          EpiCe<false>::Params pf{V, NP, scale2, lab, part, nullptr};
          FCKL_CE_GEMM(EpiCe<false>, mapW_k, pf);
        }
      }
      ProfScope ps(K_MERGE, st, 0.0, nr * (NT * 8.0 + 28.0));
      const bool block_row = ce_block_rows(cap);
      FCKL_LAUNCH(block_row ? k_ce_merge<true> : k_ce_merge<false>,
                  block_row ? cap : (int)cdiv(cap, kCeWarps), 256, 0, (const float2*)part, zs, NPm,
                  rc, cap, V, invT, prob->label_smoothing, prob->z_loss, clist, (const float*)zlab,
                  (const float*)kw, recompute ? lse2 : nullptr, q.row_loss, q.lse_out, share + row0,
                  (const float*)share, N, ctl, blocks, q.loss);
    }
    if (q.mode == CeMode::kFwd) continue;
    if (q.mode == CeMode::kFwdBwd && !recompute) {
      {
        ProfScope ps(K_CE_FWD, st, flops, 2.0 * (nr + V) * H + 2.0 * nr * V);
        if (smooth) {
          EpiCeStore<true>::Params pf{V, NP, scale2, lab, part, zsum, cap};
          FCKL_CE_GEMM(EpiCeStore<true>, mapD_st, pf);
        } else {
          EpiCeStore<false>::Params pf{V, NP, scale2, lab, part, nullptr, cap};
          FCKL_CE_GEMM(EpiCeStore<false>, mapD_st, pf);
        }
      }
      ProfScope ps(K_CE_SCALE, st, 0.0, nr * (V * 4.0 + NT * 16.0));
      const bool warp_row = ce_warp_dlogits(prob->V, cap);
      // blocks that share a row, so that few rows still fill the SMs
      const unsigned parts = (unsigned)std::max<long long>(
          1, std::min<long long>(cdiv(L.Vp, 2048), cdiv(4ll * dev->sms, cap)));
      FCKL_LAUNCH(warp_row ? k_ce_dlogits<false> : k_ce_dlogits<true>,
                  warp_row ? dim3((unsigned)cdiv(cap, kCeWarps)) : dim3(cap, parts), 256, 0,
                  (const float2*)part, zs, NP, rc, cap, V, L.Vp, invT, prob->label_smoothing,
                  prob->z_loss, clist, (const int*)lab, (const float*)zlab, (const float*)kw,
                  reinterpret_cast<uint4*>(dlog), rest, q.row_loss, q.lse_out, share + row0,
                  (const float*)share, N, ctl, blocks, q.loss);
    } else {
      EpiCeDlogits::Params pb{V, scale2, invT * kLog2e, prob->label_smoothing,
                              2.f * prob->z_loss, lab, kw, zlab, lse2, rest, cap};
      ProfScope ps(K_CE_DLOGITS, st, flops, 2.0 * (nr + V) * H + 2.0 * nr * V);
      if (recompute) {  // the operands and the count were complete before the merge launched
        sa_v.early = 1;
        sa_v.fresh_rows = 0;
      }
      FCKL_CE_GEMM(EpiCeDlogits, mapD_st, pb);
    }
#undef FCKL_CE_GEMM
    // dH = dlogits W / (T D), k segments to slabs; dW (+)= dlogits^T h / (T D).
    SchedArgs sa_h{SCHED_SPLIT_K, NTh, KBv, 0, 0, rc, 0, w3d, 0, narrow_h, 0, 2, 1,
                   L.slab_units, kPollNs};
    const EpiCeDH::Params ph{H, invT, ctl};
    if (q.dH && !make_map(&mapD_k, dlog, V, cap, L.Vp * 2, BK, CM)) return FCKL_ERR_CUDA;
    const int MTv = (int)cdiv(V, PM);
    int d3d = 0, h3d = 0;
    if (q.dW && (!make_map_mn(&mapD_mn, dlog, L.Vp, cap, L.Vp * 2, &d3d) ||
                 !make_map_mn(&mapH_mn, hst, H, cap, (long long)H * 2, &h3d)))
      return FCKL_ERR_CUDA;
    SchedArgs sa_w{SCHED_TILES, NTh, 0, 1, MTv, rc, d3d, h3d, 0, narrow_h, 0};
    sa_w.poll_ns = kPollNs;
    const EpiCeDW::Params pw{V, H, invT, ctl};
    const EpiCeDWSum::Params ps_w{V, H, invT, c > 0 ? 1 : 0, ctl, (int)(row0 + cap),
                                  static_cast<const float*>(dw_dst),
                                  bf16_grads ? static_cast<__nv_bfloat16*>(q.dW) : nullptr};
    const double dh_bytes = 2.0 * nr * V + 2.0 * (double)V * H + 4.0 * nr * H;
    const double dw_bytes = 2.0 * nr * (V + H) + (dw_direct16 ? 2.0 : c > 0 ? 8.0 : 4.0) * V * H;
    const bool two = q.dH && q.dW && L.nchunks == 1 && ce_two(cap, V, H, bf16_grads);
    const int dh_pairs = two ? std::max(1, pairs * 3 / 8) : pairs;
    if (two) {
      ProfScope ps(K_DHW, st, 2.0 * flops, dh_bytes + dw_bytes);
      constexpr size_t smem = std::max({pair_smem_bytes<EpiCeDH>(), pair_smem_bytes<EpiCeDW>(),
                                        pair_smem_bytes<EpiCeDWSum>()});
      if (dw_direct16)
        FCKL_LAUNCH((gemm_two_kernel<EpiCeDH, false, true, EpiCeDW, true, true>), 2 * pairs,
                    gemm_threads<EpiCeDH>(), smem, mapD_k, mapW_mn, mapSlab, mapD_mn, mapH_mn,
                    mapdW, ph, pw, sa_h, sa_w, ca, dh_pairs);
      else
        FCKL_LAUNCH((gemm_two_kernel<EpiCeDH, false, true, EpiCeDWSum, true, true>), 2 * pairs,
                    gemm_threads<EpiCeDH>(), smem, mapD_k, mapW_mn, mapSlab, mapD_mn, mapH_mn,
                    mapdW, ph, ps_w, sa_h, sa_w, ca, dh_pairs);
    } else {
      if (q.dH) {
        ProfScope ps(K_DH, st, flops, dh_bytes);
        FCKL_LAUNCH((gemm_pair_kernel<EpiCeDH, false, true>), 2 * pairs, gemm_threads<EpiCeDH>(),
                    pair_smem_bytes<EpiCeDH>(), mapD_k, mapW_mn, mapSlab, ph, sa_h, ca);
      }
      if (q.dW) {
        // dlogits and the gathered rows were complete before the dH GEMM
        // launched, so this main loop starts at once (without a dH GEMM it
        // follows the kernel that wrote dlogits)
        sa_w.early = q.dH ? 1 : 0;
        ProfScope ps(K_DW, st, flops, dw_bytes);
        if (dw_direct16)
          FCKL_LAUNCH((gemm_pair_kernel<EpiCeDW, true, true>), grid_for((long long)MTv * NTh),
                      gemm_threads<EpiCeDW>(), pair_smem_bytes<EpiCeDW>(), mapD_mn, mapH_mn, mapdW,
                      pw, sa_w, ca);
        else
          FCKL_LAUNCH((gemm_pair_kernel<EpiCeDWSum, true, true>), grid_for((long long)MTv * NTh),
                      gemm_threads<EpiCeDWSum>(), pair_smem_bytes<EpiCeDWSum>(), mapD_mn, mapH_mn,
                      mapdW, ps_w, sa_w, ca);
      }
    }
    // the last chunk's blocks zero dW when no row was kept
    const bool last = c + 1 == L.nchunks && q.dW;
    if (q.dH || last) {
      uint4* zdw = last ? static_cast<uint4*>(q.dW) : nullptr;
      const long long vecs = (long long)V * H * (bf16_grads ? 2 : 4) / 16;
      ProfScope ps(K_DH_OUT, st, 0.0, nr * H * (bf16_grads ? 8.0 : 10.0));
      if (bf16_grads)
        FCKL_LAUNCH(k_ce_dh_out<__nv_bfloat16>, dim3(cap, (unsigned)cdiv(H, 512)), 128, 0,
                    (const float*)slab, clist, rc, H, static_cast<__nv_bfloat16*>(q.dH), zdw, vecs,
                    (const DeviceCtl*)ctl, invT, static_cast<const __nv_bfloat16*>(q.W),
                    (const int*)lab, (const float*)rest);
      else
        FCKL_LAUNCH(k_ce_dh_out<float>, dim3(cap, (unsigned)cdiv(H, 512)), 128, 0,
                    (const float*)slab, clist, rc, H, static_cast<float*>(q.dH), zdw, vecs,
                    (const DeviceCtl*)ctl, invT, static_cast<const __nv_bfloat16*>(q.W),
                    (const int*)lab, (const float*)rest);
    }
  }
  return cudaGetLastError() == cudaSuccess ? FCKL_OK : FCKL_ERR_CUDA;
}

fckl_status run_ce(const CeRequest& q) {
  const fckl_ce_problem* prob = q.prob;
  const bool grads = q.mode != CeMode::kFwd;
  if (!valid_ce(prob)) return FCKL_ERR_INVALID_ARG;
  if (!q.hidden || !q.W || !q.labels || !aligned(q.hidden, 16) || !aligned(q.W, 16) ||
      !aligned(q.labels, prob->label_type == FCKL_LABELS_LONG ? 8 : 4))
    return FCKL_ERR_INVALID_ARG;
  if (!aligned(q.factor, 4) || !aligned(q.row_loss, 4) || !aligned(q.lse_out, 4))
    return FCKL_ERR_INVALID_ARG;
  if (q.mode == CeMode::kBwd ? (!q.lse_in || !q.factor || !aligned(q.lse_in, 4))
                             : (!q.loss || !aligned(q.loss, 4)))
    return FCKL_ERR_INVALID_ARG;
  if (grads && ((!q.dH && !q.dW) || !aligned(q.dH, 16) || !aligned(q.dW, 16)))
    return FCKL_ERR_INVALID_ARG;
  if (!supported_ce(prob)) return FCKL_ERR_UNSUPPORTED;
  const CeLayout L = ce_layout(prob, grads);
  if (q.workspace == nullptr || !aligned(q.workspace, kAlign) || q.ws_bytes < L.total)
    return FCKL_ERR_WORKSPACE;
  const CeDevice* dev = ce_device();
  if (dev == nullptr || !dev->ok) return FCKL_ERR_UNSUPPORTED;
  if (get_encode_fn() == nullptr) return FCKL_ERR_CUDA;
  return prob->label_type == FCKL_LABELS_LONG ? enqueue_ce<int64_t>(q, L, dev)
                                              : enqueue_ce<int32_t>(q, L, dev);
}

}  // namespace

extern "C" {

size_t fckl_ce_workspace_bytes(const fckl_ce_problem* prob, int32_t gradients) {
  if (!valid_ce(prob) || !supported_ce(prob)) return 0;
  return ce_layout(prob, gradients != 0).total;
}

fckl_status fckl_ce_fwd(const fckl_ce_problem* prob, const void* hidden, const void* W,
                        const void* labels, const float* row_weight, float* loss, float* row_loss,
                        float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  CeRequest q;
  q.mode = CeMode::kFwd;
  q.prob = prob; q.hidden = hidden; q.W = W; q.labels = labels; q.factor = row_weight;
  q.loss = loss; q.row_loss = row_loss; q.lse_out = lse;
  q.workspace = workspace; q.ws_bytes = workspace_bytes; q.stream = stream;
  return run_ce(q);
}

fckl_status fckl_ce_fwd_bwd(const fckl_ce_problem* prob, const void* hidden, const void* W,
                            const void* labels, const float* row_weight, float* loss,
                            float* row_loss, float* lse, void* dH, void* dW, void* workspace,
                            size_t workspace_bytes, void* stream) {
  CeRequest q;
  q.mode = CeMode::kFwdBwd;
  q.prob = prob; q.hidden = hidden; q.W = W; q.labels = labels; q.factor = row_weight;
  q.loss = loss; q.row_loss = row_loss; q.lse_out = lse; q.dH = dH; q.dW = dW;
  q.workspace = workspace; q.ws_bytes = workspace_bytes; q.stream = stream;
  return run_ce(q);
}

fckl_status fckl_ce_bwd(const fckl_ce_problem* prob, const void* hidden, const void* W,
                        const void* labels, const float* lse, const float* row_grad, void* dH,
                        void* dW, void* workspace, size_t workspace_bytes, void* stream) {
  CeRequest q;
  q.mode = CeMode::kBwd;
  q.prob = prob; q.hidden = hidden; q.W = W; q.labels = labels; q.lse_in = lse;
  q.factor = row_grad; q.dH = dH; q.dW = dW;
  q.workspace = workspace; q.ws_bytes = workspace_bytes; q.stream = stream;
  return run_ce(q);
}

fckl_status fckl_scale_gradient(void* grad, int64_t n, int32_t grad_type, const float* factor,
                                void* stream) {
  if (!grad || !factor || n < 1 || !aligned(grad, 16) || !aligned(factor, 4) ||
      (grad_type != FCKL_GRAD_FLOAT && grad_type != FCKL_GRAD_BFLOAT))
    return FCKL_ERR_INVALID_ARG;
  const CeDevice* dev = ce_device();
  if (dev == nullptr || !dev->ok) return FCKL_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int grid = (int)std::min<long long>(cdiv(cdiv(n, 4), 256), (long long)dev->sms * 8);
  if (grad_type == FCKL_GRAD_BFLOAT)
    k_scale<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<__nv_bfloat16*>(grad), n, factor);
  else
    k_scale<float><<<grid, 256, 0, st>>>(static_cast<float*>(grad), n, factor);
  return cudaGetLastError() == cudaSuccess ? FCKL_OK : FCKL_ERR_CUDA;
}

}  // extern "C"
