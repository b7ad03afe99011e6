// C ABI of libda.so: argument checks, workspace layout and kernel launches.
// Every check happens before the first launch, so a call that returns an error launched nothing.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "da.h"
#include "da_common.cuh"
#include "da_internal.h"

using namespace da;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

namespace da {

da_status check_dims(const da_dims* dims, Dims* g) {
  if (!dims) return DA_ERR_INVALID_ARG;
  if (dims->B <= 0 || dims->H <= 0 || dims->N <= 0 || dims->d <= 0 || dims->C <= 0 || dims->block <= 0)
    return DA_ERR_INVALID_ARG;
  if (dims->dtype != DA_BF16 && dims->dtype != DA_F32) return DA_ERR_DTYPE;
  if (dims->d != 64 && dims->d != 128) return DA_ERR_UNSUPPORTED;
  if (dims->block != 64 && dims->block != 128) return DA_ERR_UNSUPPORTED;
  if (dims->C % 32 != 0 || dims->C > 1024) return DA_ERR_UNSUPPORTED;
  g->B = dims->B;
  g->H = dims->H;
  g->N = dims->N;
  g->d = dims->d;
  g->C = dims->C;
  g->block = dims->block;
  g->nB = (dims->N + dims->block - 1) / dims->block;
  g->bf16 = dims->dtype == DA_BF16;
  const long long BH = (long long)dims->B * dims->H;
  // work items and block-row indices are int32 on the device
  if (BH * g->nB >= (1LL << 31) || BH * dims->N >= (1LL << 31)) return DA_ERR_SHAPE;
  // a head's lookup rows (seg_idx, blk_hist: nB x C) are indexed in 32 bits
  if ((long long)g->nB * dims->C >= (1LL << 31)) return DA_ERR_SHAPE;
  // the tensor-core path addresses block entries (block row x block + entry) in 32 bits
  if (g->bf16 && BH * g->nB * g->block >= (1LL << 32)) return DA_ERR_SHAPE;
  return DA_OK;
}

da_status check_stats(const da_cluster_stats* st, StatsPtrs* p) {
  if (!st) return DA_ERR_INVALID_ARG;
  if (!st->assign || !st->blk_hist || !st->seg_idx || !st->seg_n || !st->seg_c || !st->seg_cnt ||
      !st->seg_vsum || !st->n_tot || !st->S_tot)
    return DA_ERR_INVALID_ARG;
  if (!aligned16(st->assign) || !aligned16(st->blk_hist) || !aligned16(st->seg_idx) || !aligned16(st->seg_n) ||
      !aligned16(st->seg_c) || !aligned16(st->seg_cnt) || !aligned16(st->seg_vsum) || !aligned16(st->n_tot) ||
      !aligned16(st->S_tot))
    return DA_ERR_ALIGNMENT;
  *p = StatsPtrs{st->assign, st->blk_hist, st->seg_idx, st->seg_n, st->seg_c,
                 st->seg_cnt, st->seg_vsum, st->n_tot, st->S_tot};
  return DA_OK;
}

}  // namespace da

namespace {

// An NVTX range around the host side of a call (argument checks and launches), named after the
// call, so that a profiler's timeline groups each call's kernels; header-only NVTX costs next to
// nothing without a profiler attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

da_status check_ws(const Dims& g, void* ws, size_t ws_bytes) {
  if (!ws) return DA_ERR_INVALID_ARG;
  if (!aligned16(ws)) return DA_ERR_ALIGNMENT;
  if (ws_bytes < ws_layout(g).total) return DA_ERR_WORKSPACE;
  return DA_OK;
}

da_status check_mask(const Dims& g, const da_block_mask* mask) {
  if (!mask || !mask->kv_idx || !mask->kv_cnt) return DA_ERR_INVALID_ARG;
  if (mask->max_sel < 1) return DA_ERR_SHAPE;
  if ((long long)g.B * g.H * g.nB * mask->max_sel >= (1LL << 40)) return DA_ERR_SHAPE;
  if (!aligned16(mask->kv_idx) || !aligned16(mask->kv_cnt)) return DA_ERR_ALIGNMENT;
  if (mask->schedule && !aligned16(mask->schedule)) return DA_ERR_ALIGNMENT;
  return DA_OK;
}

da_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DA_OK : DA_ERR_CUDA; }

// Rows, tokens and the like stay this far below 2^31, so that a grid's last blocks index beyond them in 32 bits.
constexpr long long kMaxTokens = (1LL << 31) - 65536;

// Strides of dimensions of one entry are never used: zero, so that no check takes offence at them.
da_head_strides used_strides(int B, int H, int N, const da_head_strides& s) {
  return da_head_strides{B > 1 ? s.batch : 0, H > 1 ? s.head : 0, N > 1 ? s.token : 0};
}

// A strided tensor of the layer operators: up to three outer dimensions over `inner` contiguous
// elements of `size` bytes.
struct View {
  const void* p;
  long long inner;
  int size;
  long long n[3], stride[3];

  bool fits() const {   // strides and extents whose offsets stay far inside 64 bits
    __int128 s = inner;
    for (int i = 0; i < 3; ++i) {
      if (stride[i] < 0 || stride[i] > (1LL << 40) || n[i] > kMaxTokens) return false;
      if (n[i] > 1) s += (__int128)(n[i] - 1) * stride[i];
    }
    return s < (__int128)1 << 46;
  }
  long long span() const {   // elements from the first to the last, both included; of a view that fits
    long long s = inner;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1) s += (n[i] - 1) * stride[i];
    return s;
  }
  // No element twice: each outer dimension, from the smallest stride up, steps over what lies below it.
  bool distinct() const {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
      for (int j = i + 1; j < 3; ++j)
        if (stride[order[j]] < stride[order[i]]) { const int t = order[i]; order[i] = order[j]; order[j] = t; }
    long long s = inner;
    for (int i = 0; i < 3; ++i) {
      const int k = order[i];
      if (n[k] <= 1) continue;
      if (stride[k] < s) return false;
      s += (n[k] - 1) * stride[k];
    }
    return true;
  }
  bool element_aligned() const { return reinterpret_cast<uintptr_t>(p) % size == 0; }
  bool aligned16() const {   // every run of `inner` elements starts on 16 bytes
    bool ok = reinterpret_cast<uintptr_t>(p) % 16 == 0 && inner * size % 16 == 0;
    for (int i = 0; i < 3; ++i) ok = ok && (n[i] <= 1 || stride[i] * size % 16 == 0);
    return ok;
  }
};

View matrix(const void* p, int size, long long rows, long long width, long long stride) {
  return View{p, width, size, {1, 1, rows}, {0, 0, stride}};
}

View heads(const void* p, int size, int B, int H, int N, int d, const da_head_strides& s) {
  return View{p, d, size, {B, H, N}, {s.batch, s.head, s.token}};
}

// An output and another tensor: apart in memory, or (in_place) the very same elements.
bool apart(const View& o, const View& v, bool in_place) {
  if (!v.p) return true;
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(o.p), v0 = reinterpret_cast<uintptr_t>(v.p);
  const uintptr_t o1 = o0 + (uintptr_t)(o.span() * o.size), v1 = v0 + (uintptr_t)(v.span() * v.size);
  if (o1 <= v0 || v1 <= o0) return true;
  if (!in_place || o0 != v0 || o.inner != v.inner || o.size != v.size) return false;
  for (int i = 0; i < 3; ++i)
    if (o.n[i] > 1 && o.stride[i] != v.stride[i]) return false;
  return true;
}

constexpr int kMaxRowWidth = 16384;   // a row is held in one block's registers

da_status check_dtype(da_dtype t) { return t == DA_BF16 || t == DA_F32 ? DA_OK : DA_ERR_DTYPE; }
int element_size(da_dtype t) { return t == DA_BF16 ? 2 : 4; }

// Shared by da_rms_norm and da_rms_norm_i8 (scale non-null): out and its rows are elements or codes.
da_status rms_norm(int64_t rows, int width, da_dtype dtype, const void* x, int64_t x_stride, const void* residual,
                   int64_t residual_stride, const void* weight, float eps, void* sum_out, int64_t sum_stride,
                   void* out, int64_t out_stride, float* scale, bool codes, da_stream stream) {
  if (rows <= 0 || width <= 0 || !x || !out || (codes && !scale) || (sum_out && !residual)) return DA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || eps > 3e38f) return DA_ERR_INVALID_ARG;
  da_status st = check_dtype(dtype);
  if (st != DA_OK) return st;
  if (width > kMaxRowWidth) return DA_ERR_UNSUPPORTED;
  const int size = element_size(dtype);
  const View vx = matrix(x, size, rows, width, x_stride), vr = matrix(residual, size, rows, width, residual_stride);
  const View vw = matrix(weight, size, 1, width, 0), vs = matrix(sum_out, size, rows, width, sum_stride);
  const View vo = matrix(out, codes ? 1 : size, rows, width, out_stride), vc = matrix(scale, 4, rows, 1, 1);
  if (!vx.fits() || !vo.fits() || (residual && !vr.fits()) || (sum_out && !vs.fits())) return DA_ERR_SHAPE;
  if (!vo.distinct() || (sum_out && !vs.distinct())) return DA_ERR_SHAPE;
  if (!vx.element_aligned() || !vr.element_aligned() || !vw.element_aligned() || !vs.element_aligned() ||
      !vo.element_aligned() || !vc.element_aligned())
    return DA_ERR_ALIGNMENT;
  const bool ok = apart(vo, vx, !codes) && apart(vo, vr, !codes) && apart(vo, vw, false) && apart(vo, vs, false) &&
                  apart(vo, vc, false) &&
                  (!sum_out || (apart(vs, vx, true) && apart(vs, vr, true) && apart(vs, vw, false) && apart(vs, vc, false))) &&
                  (!codes || (apart(vc, vx, false) && apart(vc, vr, false) && apart(vc, vw, false)));
  if (!ok) return DA_ERR_INVALID_ARG;
  return cuda_status(launch_rms_norm(dtype == DA_BF16, rows, width, x, x_stride, residual, residual_stride, weight, eps,
                                     sum_out, sum_stride, out, out_stride, codes ? scale : nullptr,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int da_version(void) { return 103; }

size_t da_workspace_bytes(const da_dims* dims) {
  Dims g;
  if (check_dims(dims, &g) != DA_OK) return 0;
  return ws_layout(g).total;
}

size_t da_schedule_bytes(const da_dims* dims) {
  Dims g;
  if (check_dims(dims, &g) != DA_OK) return 0;
  return (size_t)g.B * g.H * g.nB * sizeof(int32_t);
}

da_status da_reassign(const da_dims* dims, const void* K, const void* V, const void* centroids,
                      const da_cluster_stats* out, void* ws, size_t ws_bytes, da_stream stream) {
  NvtxRange nvtx("da_reassign");
  Dims g;
  da_status st = check_dims(dims, &g);
  if (st != DA_OK) return st;
  if (!K || !V || !centroids) return DA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !aligned16(centroids)) return DA_ERR_ALIGNMENT;
  StatsPtrs sp;
  if ((st = check_stats(out, &sp)) != DA_OK) return st;
  if ((st = check_ws(g, ws, ws_bytes)) != DA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const WsLayout L = ws_layout(g);
  int* status = reinterpret_cast<int*>(static_cast<char*>(ws) + L.status);
  float* norms = reinterpret_cast<float*>(static_cast<char*>(ws) + L.norms);
  cudaError_t e;
  if (reassign_tc_supported(g)) {
    e = launch_centroid_norms(g, centroids, norms, s);
    if (e == cudaSuccess) e = launch_reassign_tc(g, K, V, centroids, norms, sp, status, s);
  } else {
    e = g.bf16 ? launch_assign_simt_bf16(g, K, centroids, sp.assign, s)
               : launch_assign_simt_f32(g, K, centroids, sp.assign, s);
    if (e == cudaSuccess) e = launch_block_stats(g, V, sp, s);
  }
  if (e == cudaSuccess) e = launch_totals(g, sp, s);
  return cuda_status(e);
}

da_status da_mask_prepare(const da_dims* dims, const da_block_mask* mask, int32_t* schedule,
                          size_t schedule_bytes, void* ws, size_t ws_bytes, da_stream stream) {
  NvtxRange nvtx("da_mask_prepare");
  Dims g;
  da_status st = check_dims(dims, &g);
  if (st != DA_OK) return st;
  if ((st = check_mask(g, mask)) != DA_OK) return st;
  if (!schedule) return DA_ERR_INVALID_ARG;
  if (!aligned16(schedule)) return DA_ERR_ALIGNMENT;
  if (schedule_bytes < (size_t)g.B * g.H * g.nB * sizeof(int32_t)) return DA_ERR_WORKSPACE;
  if ((st = check_ws(g, ws, ws_bytes)) != DA_OK) return st;
  const WsLayout L = ws_layout(g);
  int* status = reinterpret_cast<int*>(static_cast<char*>(ws) + L.status);
  return cuda_status(launch_schedule(g, mask->kv_idx, mask->kv_cnt, mask->max_sel, schedule, status,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

// Validation shared by da_compensation, da_attention_prebuilt and da_attention.
static da_status attention_common(const da_dims* dims, const da_block_mask* mask, const da_cluster_stats* stats,
                                  void* ws, size_t ws_bytes, Dims* g, StatsPtrs* sp) {
  da_status st = check_dims(dims, g);
  if (st != DA_OK) return st;
  if ((st = check_mask(*g, mask)) != DA_OK) return st;
  if ((st = check_stats(stats, sp)) != DA_OK) return st;
  return check_ws(*g, ws, ws_bytes);
}

static da_status check_attention_ptrs(const void* Q, const void* K, const void* V, const void* centroids,
                                      const void* O, const float* lse) {
  if (!Q || !K || !V || !centroids || !O) return DA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(centroids) || !aligned16(O) ||
      (lse && !aligned16(lse)))
    return DA_ERR_ALIGNMENT;
  return DA_OK;
}

static cudaError_t compensation_launch(const Dims& g, const da_block_mask* mask, const StatsPtrs& sp, void* ws,
                                       cudaStream_t s) {
  if (!attention_tc_supported(g)) return cudaSuccess;   // the CUDA-core path compensates in-kernel
  const WsLayout L = ws_layout(g);
  return launch_comp_build(g, mask->kv_idx, mask->kv_cnt, mask->max_sel, sp, static_cast<char*>(ws) + L.comp, s);
}

static da_status attention_launch(const Dims& g, const void* Q, const void* K, const void* V,
                                  const da_block_mask* mask, const void* centroids, const StatsPtrs& sp, float scale,
                                  void* O, float* lse, void* ws, cudaStream_t s) {
  const da_status pst = check_attention_ptrs(Q, K, V, centroids, O, lse);
  if (pst != DA_OK) return pst;
  if (!(scale > 0.f)) scale = 1.0f / sqrtf((float)g.d);
  const WsLayout L = ws_layout(g);
  int* status = reinterpret_cast<int*>(static_cast<char*>(ws) + L.status);
  const int32_t* sched = mask->schedule;
  cudaError_t e = cudaSuccess;
  if (!sched) {
    int32_t* own = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + L.sched);
    e = launch_schedule(g, mask->kv_idx, mask->kv_cnt, mask->max_sel, own, status, s);
    sched = own;
  }
  if (e == cudaSuccess) {
    if (attention_tc_supported(g))
      e = launch_attention_tc(g, Q, K, V, mask->kv_idx, mask->kv_cnt, mask->max_sel, sched, centroids, sp, scale, O,
                              lse, status, static_cast<char*>(ws) + L.comp, nullptr, nullptr, s);
    else
      e = (g.bf16 ? launch_attention_simt_bf16 : launch_attention_simt_f32)(
          g, Q, K, V, mask->kv_idx, mask->kv_cnt, mask->max_sel, sched, centroids, sp, nullptr, scale, O, lse, status,
          s);
  }
  return cuda_status(e);
}

da_status da_compensation(const da_dims* dims, const da_block_mask* mask, const da_cluster_stats* stats, void* ws,
                          size_t ws_bytes, da_stream stream) {
  NvtxRange nvtx("da_compensation");
  Dims g;
  StatsPtrs sp;
  da_status st = attention_common(dims, mask, stats, ws, ws_bytes, &g, &sp);
  if (st != DA_OK) return st;
  return cuda_status(compensation_launch(g, mask, sp, ws, reinterpret_cast<cudaStream_t>(stream)));
}

da_status da_attention_prebuilt(const da_dims* dims, const void* Q, const void* K, const void* V,
                                const da_block_mask* mask, const void* centroids, const da_cluster_stats* stats,
                                float scale, void* O, float* lse, void* ws, size_t ws_bytes, da_stream stream) {
  NvtxRange nvtx("da_attention_prebuilt");
  Dims g;
  StatsPtrs sp;
  da_status st = attention_common(dims, mask, stats, ws, ws_bytes, &g, &sp);
  if (st != DA_OK) return st;
  return attention_launch(g, Q, K, V, mask, centroids, sp, scale, O, lse, ws, reinterpret_cast<cudaStream_t>(stream));
}

da_status da_attention(const da_dims* dims, const void* Q, const void* K, const void* V,
                       const da_block_mask* mask, const void* centroids, const da_cluster_stats* stats,
                       float scale, void* O, float* lse, void* ws, size_t ws_bytes, da_stream stream) {
  NvtxRange nvtx("da_attention");
  Dims g;
  StatsPtrs sp;
  da_status st = attention_common(dims, mask, stats, ws, ws_bytes, &g, &sp);
  if (st != DA_OK) return st;
  if ((st = check_attention_ptrs(Q, K, V, centroids, O, lse)) != DA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = compensation_launch(g, mask, sp, ws, s);
  if (e != cudaSuccess) return cuda_status(e);
  return attention_launch(g, Q, K, V, mask, centroids, sp, scale, O, lse, ws, s);
}

da_status da_centroid_update(const da_dims* dims, const da_cluster_stats* stats, void* centroids,
                             da_stream stream) {
  NvtxRange nvtx("da_centroid_update");
  Dims g;
  da_status st = check_dims(dims, &g);
  if (st != DA_OK) return st;
  if (!centroids) return DA_ERR_INVALID_ARG;
  if (!aligned16(centroids)) return DA_ERR_ALIGNMENT;
  StatsPtrs sp;
  if ((st = check_stats(stats, &sp)) != DA_OK) return st;
  return cuda_status(launch_centroid_update(g, sp, centroids, reinterpret_cast<cudaStream_t>(stream)));
}

da_status da_cluster_spread(const da_dims* dims, const void* K, const void* centroids, const da_cluster_stats* stats,
                            float* spread, da_stream stream) {
  NvtxRange nvtx("da_cluster_spread");
  Dims g;
  da_status st = check_dims(dims, &g);
  if (st != DA_OK) return st;
  if (!K || !centroids || !spread) return DA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(centroids) || !aligned16(spread)) return DA_ERR_ALIGNMENT;
  StatsPtrs sp;
  if ((st = check_stats(stats, &sp)) != DA_OK) return st;
  return cuda_status(launch_cluster_spread(g, K, centroids, sp, spread, reinterpret_cast<cudaStream_t>(stream)));
}

da_status da_attention_spread(const da_dims* dims, const void* Q, const void* K, const void* V,
                              const da_block_mask* mask, const void* centroids, const da_cluster_stats* stats,
                              const float* spread, float scale, void* O, float* lse, void* ws, size_t ws_bytes,
                              da_stream stream) {
  NvtxRange nvtx("da_attention_spread");
  Dims g;
  StatsPtrs sp;
  da_status st = attention_common(dims, mask, stats, ws, ws_bytes, &g, &sp);
  if (st != DA_OK) return st;
  if ((st = check_attention_ptrs(Q, K, V, centroids, O, lse)) != DA_OK) return st;
  if (!spread) return DA_ERR_INVALID_ARG;
  if (!aligned16(spread)) return DA_ERR_ALIGNMENT;
  if (!(scale > 0.f)) scale = 1.0f / sqrtf((float)g.d);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const WsLayout L = ws_layout(g);
  int* status = reinterpret_cast<int*>(static_cast<char*>(ws) + L.status);
  const int32_t* sched = mask->schedule;
  cudaError_t e = cudaSuccess;
  if (!sched) {
    int32_t* own = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + L.sched);
    e = launch_schedule(g, mask->kv_idx, mask->kv_cnt, mask->max_sel, own, status, s);
    sched = own;
  }
  if (e == cudaSuccess && attention_tc_supported(g)) {
    // tensor cores: the compensation pre-pass, Dh = (s/2) D in bf16, then the fused kernel in its
    // variance-corrected mode
    void* dh = static_cast<char*>(ws) + L.spread;
    e = launch_comp_build(g, mask->kv_idx, mask->kv_cnt, mask->max_sel, sp, static_cast<char*>(ws) + L.comp, s);
    if (e == cudaSuccess) e = launch_spread_half(g, spread, scale, dh, s);
    if (e == cudaSuccess)
      e = launch_attention_tc(g, Q, K, V, mask->kv_idx, mask->kv_cnt, mask->max_sel, sched, centroids, sp, scale, O,
                              lse, status, static_cast<char*>(ws) + L.comp, nullptr, dh, s);
  } else if (e == cudaSuccess) {
    e = (g.bf16 ? launch_attention_simt_bf16 : launch_attention_simt_f32)(
        g, Q, K, V, mask->kv_idx, mask->kv_cnt, mask->max_sel, sched, centroids, sp, spread, scale, O, lse, status,
        s);
  }
  return cuda_status(e);
}

da_status da_attention_sip(const da_dims* dims, const void* Q, const void* K, const void* V,
                           const da_block_mask* mask, const float* incl, float scale, void* O, float* lse, void* ws,
                           size_t ws_bytes, da_stream stream) {
  NvtxRange nvtx("da_attention_sip");
  Dims g;
  da_status st = check_dims(dims, &g);
  if (st != DA_OK) return st;
  if (!attention_tc_supported(g)) return DA_ERR_UNSUPPORTED;
  if ((st = check_mask(g, mask)) != DA_OK) return st;
  if ((st = check_ws(g, ws, ws_bytes)) != DA_OK) return st;
  if ((st = check_attention_ptrs(Q, K, V, K, O, lse)) != DA_OK) return st;
  if (!incl) return DA_ERR_INVALID_ARG;
  if (!aligned16(incl)) return DA_ERR_ALIGNMENT;
  if (!(scale > 0.f)) scale = 1.0f / sqrtf((float)g.d);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const WsLayout L = ws_layout(g);
  int* status = reinterpret_cast<int*>(static_cast<char*>(ws) + L.status);
  const int32_t* sched = mask->schedule;
  cudaError_t e = cudaSuccess;
  if (!sched) {
    int32_t* own = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + L.sched);
    e = launch_schedule(g, mask->kv_idx, mask->kv_cnt, mask->max_sel, own, status, s);
    sched = own;
  }
  // no cluster steps: the centroid map is never read (K stands in for it), nor are the statistics
  if (e == cudaSuccess)
    e = launch_attention_tc(g, Q, K, V, mask->kv_idx, mask->kv_cnt, mask->max_sel, sched, K, StatsPtrs{}, scale, O,
                            lse, status, static_cast<char*>(ws) + L.comp, incl, nullptr, s);
  return cuda_status(e);
}

da_status da_rms_norm(int64_t rows, int width, da_dtype dtype, const void* x, int64_t x_stride, const void* residual,
                      int64_t residual_stride, const void* weight, float eps, void* sum_out, int64_t sum_stride,
                      void* out, int64_t out_stride, da_stream stream) {
  NvtxRange nvtx("da_rms_norm");
  return rms_norm(rows, width, dtype, x, x_stride, residual, residual_stride, weight, eps, sum_out, sum_stride, out,
                  out_stride, nullptr, false, stream);
}

da_status da_rms_norm_i8(int64_t rows, int width, da_dtype dtype, const void* x, int64_t x_stride,
                         const void* residual, int64_t residual_stride, const void* weight, float eps, void* sum_out,
                         int64_t sum_stride, int8_t* q, int64_t q_stride, float* scale, da_stream stream) {
  NvtxRange nvtx("da_rms_norm_i8");
  return rms_norm(rows, width, dtype, x, x_stride, residual, residual_stride, weight, eps, sum_out, sum_stride, q,
                  q_stride, scale, true, stream);
}

da_status da_quantize_i8(int B, int H, int N, int d, da_dtype dtype, const void* x, const da_head_strides* x_strides,
                         int8_t* q, int64_t q_stride, float* scale, da_stream stream) {
  NvtxRange nvtx("da_quantize_i8");
  if (B <= 0 || H <= 0 || N <= 0 || d <= 0 || !x || !x_strides || !q || !scale) return DA_ERR_INVALID_ARG;
  const da_status st = check_dtype(dtype);
  if (st != DA_OK) return st;
  if ((long long)H * d > kMaxRowWidth) return DA_ERR_UNSUPPORTED;
  const long long rows = (long long)B * N;
  const da_head_strides xs = used_strides(B, H, N, *x_strides);
  const View vx = heads(x, element_size(dtype), B, H, N, d, xs);
  const View vq = matrix(q, 1, rows, H * d, q_stride), vc = matrix(scale, 4, rows, 1, 1);
  if (B > 65535 || rows > kMaxTokens || !vx.fits() || !vq.fits() || !vq.distinct()) return DA_ERR_SHAPE;
  if (!vx.element_aligned() || !vc.element_aligned()) return DA_ERR_ALIGNMENT;
  if (!apart(vq, vx, false) || !apart(vq, vc, false) || !apart(vc, vx, false)) return DA_ERR_INVALID_ARG;
  return cuda_status(launch_quantize_i8(dtype == DA_BF16, B, H, N, d, x, xs, q, q_stride, scale,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

da_status da_linear_i8(int B, int N, int H, int d, int K, const int8_t* x, int64_t x_stride, const float* x_scale,
                       const int8_t* w, int64_t w_stride, const float* w_scale, const float* bias, da_dtype out_dtype,
                       void* out, const da_head_strides* out_strides, void* ws, size_t ws_bytes, da_stream stream) {
  NvtxRange nvtx("da_linear_i8");
  if (B <= 0 || N <= 0 || H <= 0 || d <= 0 || K <= 0 || !x || !x_scale || !w || !w_scale || !out || !out_strides || !ws)
    return DA_ERR_INVALID_ARG;
  const da_status st = check_dtype(out_dtype);
  if (st != DA_OK) return st;
  // 128 * 128 * K has to stay below 2^31
  if (K > 131071) return DA_ERR_UNSUPPORTED;
  const long long M = (long long)B * N, channels = (long long)H * d;
  if (M > kMaxTokens || channels > (1 << 22) - 64) return DA_ERR_SHAPE;
  const View vx = matrix(x, 1, M, K, x_stride), vw = matrix(w, 1, channels, K, w_stride);
  const View vsx = matrix(x_scale, 4, M, 1, 1), vsw = matrix(w_scale, 4, channels, 1, 1);
  const View vb = matrix(bias, 4, channels, 1, 1);
  const da_head_strides os = used_strides(B, H, N, *out_strides);
  const View vo = heads(out, element_size(out_dtype), B, H, N, d, os);
  if (!vx.fits() || !vw.fits() || !vo.fits() || !vo.distinct()) return DA_ERR_SHAPE;
  if (!vsx.element_aligned() || !vsw.element_aligned() || !vb.element_aligned() || !vo.element_aligned() || !aligned16(ws))
    return DA_ERR_ALIGNMENT;
  if (ws_bytes < kStatusWords * sizeof(int)) return DA_ERR_WORKSPACE;
  if (!apart(vo, vx, false) || !apart(vo, vw, false) || !apart(vo, vsx, false) || !apart(vo, vsw, false) ||
      !apart(vo, vb, false) || !apart(vo, matrix(ws, 1, 1, kStatusWords * sizeof(int), 0), false))
    return DA_ERR_INVALID_ARG;
  const LinearArgs a{x, w, x_scale, w_scale, bias, out, M, (int)channels, K, d, N,
                     x_stride, w_stride, os.batch, os.head, os.token};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = out_dtype == DA_BF16;
  if (!linear_i8_tc_supported(a)) return cuda_status(launch_linear_i8_bytes(bf16, a, static_cast<int*>(ws), s));
  if (linear_i8_rows_supported(a)) return cuda_status(launch_linear_i8_rows(bf16, a, s));
  return cuda_status(launch_linear_i8_tc(bf16, a, static_cast<int*>(ws), s));
}

da_status da_rope(const da_rope_plan* plan, int B, int H, int N, int d, da_dtype dtype, const void* x,
                  const da_head_strides* x_strides, const int32_t* positions, int64_t positions_batch,
                  const void* weight, int weight_width, float eps, void* out, const da_head_strides* out_strides,
                  da_stream stream) {
  NvtxRange nvtx("da_rope");
  if (!plan || B <= 0 || H <= 0 || N <= 0 || d <= 0 || !x || !x_strides || !out || !out_strides)
    return DA_ERR_INVALID_ARG;
  da_status st = check_dtype(dtype);
  if (st != DA_OK) return st;
  if (d != 64 && d != 128) return DA_ERR_UNSUPPORTED;
  if (plan->pairing != DA_ROPE_ADJACENT && plan->pairing != DA_ROPE_HALVES) return DA_ERR_INVALID_ARG;
  if (!(plan->theta >= 1.0) || !(plan->theta < 1e30)) return DA_ERR_INVALID_ARG;
  long long dims = 0, cells = 1;
  for (int u = 0; u < 3; ++u) {
    if (plan->axis_dims[u] < 0 || plan->axis_dims[u] % 2 != 0) return DA_ERR_SHAPE;
    dims += plan->axis_dims[u];
    if (!positions) {
      if (plan->grid[u] <= 0) return DA_ERR_SHAPE;
      if ((cells *= plan->grid[u]) >= (1LL << 31)) return DA_ERR_SHAPE;
    }
  }
  if (dims != d) return DA_ERR_SHAPE;
  if (weight && ((weight_width != d && weight_width != (long long)H * d) || !(eps >= 0.f) || eps > 3e38f))
    return weight_width != d && weight_width != (long long)H * d ? DA_ERR_SHAPE : DA_ERR_INVALID_ARG;
  if (weight && weight_width != d && weight_width > kMaxRowWidth) return DA_ERR_UNSUPPORTED;
  const int size = element_size(dtype);
  const da_head_strides xs = used_strides(B, H, N, *x_strides), os = used_strides(B, H, N, *out_strides);
  const View vx = heads(x, size, B, H, N, d, xs), vo = heads(out, size, B, H, N, d, os);
  const View vw = matrix(weight, size, 1, weight ? weight_width : 1, 0);
  const View vp = View{positions, 3, 4, {1, B, N}, {0, positions_batch, 3}};
  if (B > 65535 || H > 65535 || (long long)B * N > kMaxTokens) return DA_ERR_SHAPE;
  if (!vx.fits() || !vo.fits() || !vo.distinct()) return DA_ERR_SHAPE;
  if (positions && (!vp.fits() || (positions_batch != 0 && positions_batch < 3LL * N))) return DA_ERR_SHAPE;
  if (!vx.aligned16() || !vo.aligned16() || reinterpret_cast<uintptr_t>(weight) % 16 != 0 || !vp.element_aligned())
    return DA_ERR_ALIGNMENT;
  if (!apart(vo, vx, true) || !apart(vo, vw, false) || !apart(vo, vp, false)) return DA_ERR_INVALID_ARG;
  return cuda_status(launch_rope(dtype == DA_BF16, *plan, B, H, N, d, x, xs, positions, positions_batch, weight,
                                 weight_width, eps, out, os, reinterpret_cast<cudaStream_t>(stream)));
}

da_status da_device_status(void* ws, da_stream stream) {
  if (!ws) return DA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int word = 0;
  if (cudaStreamSynchronize(s) != cudaSuccess) return DA_ERR_CUDA;
  if (cudaMemcpyAsync(&word, ws, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return DA_ERR_CUDA;
  if (cudaMemsetAsync(ws, 0, sizeof(int), s) != cudaSuccess) return DA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return DA_ERR_CUDA;
  switch (word) {
    case 0: return DA_OK;
    case DA_ERR_TIMEOUT: return DA_ERR_TIMEOUT;
    case DA_ERR_DEVICE_INDEX: return DA_ERR_DEVICE_INDEX;
    case DA_ERR_RANGE: return DA_ERR_RANGE;
    default: return DA_ERR_CUDA;
  }
}

const char* da_status_string(da_status s) {
  switch (s) {
    case DA_OK: return "ok";
    case DA_ERR_INVALID_ARG: return "invalid argument (NULL pointer or non-positive size)";
    case DA_ERR_SHAPE: return "inconsistent or too large shape";
    case DA_ERR_DTYPE: return "unknown dtype";
    case DA_ERR_ALIGNMENT: return "tensor base pointer not 16-byte aligned";
    case DA_ERR_UNSUPPORTED: return "sizes not supported by this library (d, block or C)";
    case DA_ERR_CUDA: return "CUDA runtime or driver call failed";
    case DA_ERR_TIMEOUT: return "a bounded device wait gave up";
    case DA_ERR_DEVICE_INDEX: return "malformed block plan seen on the device";
    case DA_ERR_WORKSPACE: return "workspace or schedule buffer too small";
    case DA_ERR_RANGE: return "logits beyond the attention kernel's range (a later step's max far above the first's)";
  }
  return "unknown status";
}

}  // extern "C"
