// C ABI of libkvevict: argument validation, workspace layout, dispatch.
// Every check here runs on the host before anything is enqueued.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "kv_internal.cuh"

namespace kv {

int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

int num_sms() {
  static std::atomic<int> slot[kMaxDevices];
  return per_device(slot, []() {
    int v = 0;
    const int dev = current_device();
    if (dev >= 0 && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
        v > 0)
      return v;
    return 148;
  });
}

size_t max_smem_optin() {
  static std::atomic<int> slot[kMaxDevices];
  return (size_t)per_device(slot, []() {
    int v = 0;
    const int dev = current_device();
    if (dev >= 0 &&
        cudaDeviceGetAttribute(&v, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) == cudaSuccess &&
        v > 0)
      return v;
    return 48 * 1024;
  });
}

static std::atomic<unsigned long long> g_launches{0};
void count_launches(int n) { g_launches.fetch_add((unsigned long long)n); }

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks common to every op.  Returns false on an invalid shape.
static bool shape_ok(const kv_shape* sh, Shape* out) {
  if (sh == nullptr) return false;
  Shape s{sh->batch, sh->layers, sh->hq, sh->hkv, sh->d, sh->n, sh->w, sh->pool, sh->dtype};
  if (s.B < 0 || s.L < 0 || s.Hq <= 0 || s.Hkv <= 0 || s.d <= 0 || s.n < 0 || s.w < 0) return false;
  if (s.Hq % s.Hkv != 0) return false;
  if (s.d % 8 != 0) return false;
  if (s.w > s.n) return false;
  if (s.pool < 1 || s.pool % 2 == 0) return false;
  if (s.dtype != KV_BF16 && s.dtype != KV_F32) return false;
  *out = s;
  return true;
}

// Limits of the kernels as built (valid shapes outside them are KV_ERR_UNSUPPORTED).
static bool shape_supported(const Shape& s) {
  if (s.G() > 8) return false;
  if (s.d > 128) return false;
  if (s.R() > 256) return false;
  if (s.Hkv > 256) return false;
  if ((int64_t)s.Hkv * s.n >= (int64_t)1 << 31) return false;
  return true;
}

// Shape checks of the paged cache: KV_OK (with *out filled), invalid or unsupported.
static kv_status paged_shape_check(const kv_paged_shape* sh, PagedShape* out) {
  if (sh == nullptr) return KV_ERR_INVALID_ARG;
  PagedShape s{sh->seqs, sh->hq, sh->hkv, sh->d, sh->tables, sh->page, sh->max_pages, sh->dtype,
               sh->num_pages, sh->page_stride};
  if (s.seqs < 0 || s.Hq <= 0 || s.Hkv <= 0 || s.d <= 0 || s.page <= 0 || s.max_pages <= 0 ||
      s.num_pages <= 0 || s.page_stride < 0)
    return KV_ERR_INVALID_ARG;
  if (s.Hq % s.Hkv != 0 || s.d % 8 != 0) return KV_ERR_INVALID_ARG;
  if (s.tables != 1 && s.tables != s.Hkv) return KV_ERR_INVALID_ARG;
  if (s.dtype != KV_BF16 && s.dtype != KV_F32) return KV_ERR_INVALID_ARG;
  if (s.G() > 8 || s.d > 128 || s.Hkv > 256) return KV_ERR_UNSUPPORTED;
  if (s.page < 8 || s.page > 256 || (s.page & (s.page - 1)) != 0) return KV_ERR_UNSUPPORTED;
  if ((int64_t)s.max_pages * s.page > INT32_MAX || s.num_pages > INT32_MAX)
    return KV_ERR_UNSUPPORTED;
  if ((int64_t)s.seqs * s.Hkv > INT32_MAX) return KV_ERR_UNSUPPORTED;
  const int64_t dense = (int64_t)s.Hp() * s.page * s.d;
  if (s.page_stride == 0) s.page_stride = dense;
  if (s.page_stride < dense || s.page_stride % (16 / s.esize()) != 0) return KV_ERR_INVALID_ARG;
  if (s.page_stride >= ((int64_t)1 << 40) / s.esize()) return KV_ERR_UNSUPPORTED;
  *out = s;
  return KV_OK;
}

static bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// The same for the cache in 8 bits, whose pages are bytes.
static kv_status quant_shape_check(const kv_paged_shape* sh, PagedShape* out) {
  if (sh == nullptr) return KV_ERR_INVALID_ARG;
  kv_paged_shape dense = *sh;
  dense.page_stride = 0;
  const kv_status st = paged_shape_check(&dense, out);
  if (st != KV_OK) return st;
  if (out->page < KV_QUANT_BLOCK || out->d % 16 != 0) return KV_ERR_UNSUPPORTED;
  if (sh->page_stride == 0) return KV_OK;
  if (sh->page_stride < out->page_stride || sh->page_stride % 16 != 0) return KV_ERR_INVALID_ARG;
  if (sh->page_stride >= (int64_t)1 << 40) return KV_ERR_UNSUPPORTED;
  out->page_stride = sh->page_stride;
  return KV_OK;
}

static kv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KV_OK : KV_ERR_CUDA; }

// The shape of a model-wide selection (kv_allocate layer_entropy_mode 2): the L layers of a
// sequence as one layer of L * Hkv heads.  Scores [B][L][Hkv][C] and head budgets
// [B][L][Hkv] already have that layout.  False when it exceeds the kernels' limits.
static bool model_wide_shape(const Shape& s, Shape* m) {
  *m = s;
  m->L = 1;
  m->Hq = s.Hq * s.L;
  m->Hkv = s.Hkv * s.L;
  return s.L > 0 && shape_supported(*m);
}

// Scratch of flat_decode_attn_noalloc: one fixed array per device, never allocated at run
// time.  Host code must not pass the symbol itself to a kernel (on the host it names a
// host-side stand-in); the device address comes from cudaGetSymbolAddress, looked up once
// per device with that device current.
static __device__ __align__(256) char g_decode_noalloc_scratch[KV_DECODE_NOALLOC_SCRATCH_BYTES];

static std::mutex g_noalloc_mu;
static void* g_noalloc_ptr[256] = {};

static cudaError_t noalloc_scratch(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 256) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_decode_noalloc_scratch);
    if (e != cudaSuccess) return e;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return cudaSuccess;
}

}  // namespace kv

using namespace kv;

extern "C" {

size_t kv_workspace_size(int op, const kv_shape* shape) {
  Shape s;
  if (!shape_ok(shape, &s)) return 0;
  switch (op) {
    case KV_OP_SCORE: {
      const ScorePlan a = score_plan(s, KV_SCORE_LAVA);
      const ScorePlan b = score_plan(s, KV_SCORE_CRITICAL);
      return a.off_end > b.off_end ? a.off_end : b.off_end;
    }
    case KV_OP_ALLOCATE: {
      size_t need = alloc_plan(s).off_end;
      Shape m;
      if (model_wide_shape(s, &m)) {   // room for layer_entropy_mode 2 as well
        const size_t w2 = alloc_plan(m).off_end + align_up((size_t)s.B * sizeof(int32_t), 256);
        if (w2 > need) need = w2;
      }
      return need;
    }
    case KV_OP_COMPACT: return compact_plan(s, true).off_end;
    case KV_OP_DECODE: return decode_plan(s).off_end;
    default: return 0;
  }
}

kv_status kv_score(const kv_shape* shape, int mode, int group, const void* q_win, const void* k,
                   const void* v, const void* w_o, int32_t model_dim, float* scores,
                   float* crit_norm, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (mode < KV_SCORE_ADA || mode > KV_SCORE_CRITICAL) return KV_ERR_INVALID_ARG;
  if (group != KV_GROUP_MEAN && group != KV_GROUP_MAX) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  if (s.n == 0 || s.w == 0) return KV_ERR_INVALID_ARG;
  if (q_win == nullptr || k == nullptr || scores == nullptr) return KV_ERR_INVALID_ARG;
  if (!aligned16(q_win) || !aligned16(k) || !aligned16(scores)) return KV_ERR_INVALID_ARG;
  if (mode != KV_SCORE_ADA && (v == nullptr || !aligned16(v))) return KV_ERR_INVALID_ARG;
  if (mode == KV_SCORE_CRITICAL) {
    if (w_o == nullptr || crit_norm == nullptr || !aligned16(w_o) || !aligned16(crit_norm))
      return KV_ERR_INVALID_ARG;
    if (model_dim <= 0 || model_dim % 8 != 0) return KV_ERR_INVALID_ARG;
  }
  if (!shape_supported(s)) return KV_ERR_UNSUPPORTED;
  const ScorePlan p = score_plan(s, mode);
  if (ws_bytes < p.off_end) return KV_ERR_WORKSPACE;
  return cuda_status(launch_score(s, mode, group, q_win, k, v, w_o, model_dim, scores,
                                  crit_norm, static_cast<char*>(ws), p,
                                  static_cast<cudaStream_t>(stream)));
}

kv_status kv_crit_norm(const kv_shape* shape, const void* v, const void* w_o, int32_t model_dim,
                       float* crit_norm, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (s.units() == 0 || s.C() <= 0) return KV_OK;
  if (v == nullptr || w_o == nullptr || crit_norm == nullptr) return KV_ERR_INVALID_ARG;
  if (!aligned16(v) || !aligned16(w_o) || !aligned16(crit_norm)) return KV_ERR_INVALID_ARG;
  if (model_dim <= 0 || model_dim % 8 != 0) return KV_ERR_INVALID_ARG;
  if (!shape_supported(s)) return KV_ERR_UNSUPPORTED;
  if (ws_bytes < kWsHeader) return KV_ERR_WORKSPACE;
  return cuda_status(launch_crit_norm(s, v, w_o, model_dim, crit_norm, static_cast<char*>(ws),
                                      static_cast<cudaStream_t>(stream)));
}

kv_status kv_allocate(const kv_shape* shape, const float* scores, const int64_t* budget,
                      int layer_entropy_mode, uint32_t alpha_num, uint32_t alpha_den,
                      int32_t* layer_budget, int32_t* head_budget, void* ws, size_t ws_bytes,
                      void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (layer_entropy_mode < 0 || layer_entropy_mode > 2) return KV_ERR_INVALID_ARG;
  if (alpha_den == 0 || alpha_num > alpha_den || alpha_den > 65536u) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  if (scores == nullptr || budget == nullptr || layer_budget == nullptr || head_budget == nullptr)
    return KV_ERR_INVALID_ARG;
  if (!aligned16(scores) || !aligned16(budget) || !aligned16(layer_budget) ||
      !aligned16(head_budget))
    return KV_ERR_INVALID_ARG;
  if (layer_entropy_mode == 2) {
    // one selection over every layer of a sequence, then each layer's sum of head budgets
    Shape m;
    if (!shape_supported(s) || !model_wide_shape(s, &m)) return KV_ERR_UNSUPPORTED;
    const AllocPlan pm = alloc_plan(m);
    if (ws_bytes < pm.off_end + align_up((size_t)s.B * sizeof(int32_t), 256))
      return KV_ERR_WORKSPACE;
    char* w = static_cast<char*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_allocate(m, scores, budget, 0, nullptr, alpha_num, alpha_den,
                                    reinterpret_cast<int32_t*>(w + pm.off_end), head_budget, w,
                                    pm, st);
    if (e == cudaSuccess) e = launch_layer_sums(head_budget, s.segments(), s.Hkv, layer_budget, st);
    return cuda_status(e);
  }
  if (!shape_supported(s) || (layer_entropy_mode && s.L > 1024)) return KV_ERR_UNSUPPORTED;
  const AllocPlan p = alloc_plan(s);
  if (ws_bytes < p.off_end) return KV_ERR_WORKSPACE;
  return cuda_status(launch_allocate(s, scores, budget, layer_entropy_mode, nullptr, alpha_num,
                                     alpha_den, layer_budget, head_budget,
                                     static_cast<char*>(ws), p,
                                     static_cast<cudaStream_t>(stream)));
}

kv_status kv_allocate_capped(const kv_shape* shape, const float* scores, const int64_t* budget,
                             const int32_t* layer_cap, uint32_t alpha_num, uint32_t alpha_den,
                             int32_t* layer_budget, int32_t* head_budget, void* ws,
                             size_t ws_bytes, void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (alpha_den == 0 || alpha_num > alpha_den || alpha_den > 65536u) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  if (scores == nullptr || budget == nullptr || layer_cap == nullptr || layer_budget == nullptr ||
      head_budget == nullptr)
    return KV_ERR_INVALID_ARG;
  if (!aligned16(scores) || !aligned16(budget) || !aligned16(layer_cap) ||
      !aligned16(layer_budget) || !aligned16(head_budget))
    return KV_ERR_INVALID_ARG;
  if (!shape_supported(s) || s.L > 1024) return KV_ERR_UNSUPPORTED;
  const AllocPlan p = alloc_plan(s);
  if (ws_bytes < p.off_end) return KV_ERR_WORKSPACE;
  return cuda_status(launch_allocate(s, scores, budget, 1, layer_cap, alpha_num, alpha_den,
                                     layer_budget, head_budget, static_cast<char*>(ws), p,
                                     static_cast<cudaStream_t>(stream)));
}

// Argument checks of a compaction (kv_compact, kv_compact_kappa): KV_OK or the error.
static kv_status kv_compact_check(const Shape& s, const void* k, const void* v,
                                  const float* scores, const float* crit_norm,
                                  uint32_t crit_alpha_num, uint32_t crit_alpha_den,
                                  float crit_eps, const int32_t* head_budget, int32_t reserve,
                                  int32_t* kept_idx, int64_t* cu_off, int32_t* lens,
                                  void* k_flat, void* v_flat, int64_t flat_capacity_rows,
                                  void* ws) {
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (reserve < 0 || flat_capacity_rows < 0) return KV_ERR_INVALID_ARG;
  if (k == nullptr || v == nullptr || scores == nullptr || head_budget == nullptr ||
      kept_idx == nullptr || cu_off == nullptr || lens == nullptr || k_flat == nullptr ||
      v_flat == nullptr)
    return KV_ERR_INVALID_ARG;
  const void* ptrs[] = {k, v, scores, head_budget, kept_idx, cu_off, lens, k_flat, v_flat};
  for (const void* q : ptrs)
    if (!aligned16(q)) return KV_ERR_INVALID_ARG;
  if (crit_norm != nullptr) {
    if (!aligned16(crit_norm)) return KV_ERR_INVALID_ARG;
    if (crit_alpha_den == 0 || crit_alpha_num > crit_alpha_den || crit_alpha_den > 65536u)
      return KV_ERR_INVALID_ARG;
    if (!(crit_eps >= 0.0f) || std::isinf(crit_eps)) return KV_ERR_INVALID_ARG;
  }
  // The smallest flat buffer any valid budgets can need: every head keeps its window.
  if (flat_capacity_rows < s.units() * (int64_t)(s.w + reserve)) return KV_ERR_CAPACITY;
  if (!shape_supported(s)) return KV_ERR_UNSUPPORTED;
  return KV_OK;
}

kv_status kv_compact(const kv_shape* shape, const void* k, const void* v, const float* scores,
                     const float* crit_norm, uint32_t crit_alpha_num, uint32_t crit_alpha_den,
                     float crit_eps, const int32_t* head_budget, int32_t reserve,
                     int32_t* kept_idx, int64_t* cu_off, int32_t* lens, void* k_flat,
                     void* v_flat, int64_t flat_capacity_rows, void* ws, size_t ws_bytes,
                     void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (reserve < 0 || flat_capacity_rows < 0) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  const kv_status st = kv_compact_check(s, k, v, scores, crit_norm, crit_alpha_num,
                                        crit_alpha_den, crit_eps, head_budget, reserve, kept_idx,
                                        cu_off, lens, k_flat, v_flat, flat_capacity_rows, ws);
  if (st != KV_OK) return st;
  const CompactPlan p = compact_plan(s, crit_norm != nullptr);
  if (ws_bytes < p.off_end) return KV_ERR_WORKSPACE;
  return cuda_status(launch_compact(s, k, v, scores, crit_norm, crit_alpha_num, crit_alpha_den,
                                    crit_eps, false, head_budget, reserve, kept_idx, cu_off,
                                    lens, k_flat, v_flat, flat_capacity_rows,
                                    static_cast<char*>(ws), p,
                                    static_cast<cudaStream_t>(stream)));
}

kv_status kv_compact_streaming(const kv_shape* shape, const void* k, const void* v,
                               int32_t sinks, const int32_t* head_budget, int32_t reserve,
                               int32_t* kept_idx, int64_t* cu_off, int32_t* lens, void* k_flat,
                               void* v_flat, int64_t flat_capacity_rows, void* ws,
                               size_t ws_bytes, void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (sinks < 0) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (reserve < 0 || flat_capacity_rows < 0) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  // the checks of kv_compact; the scores are not read (any aligned pointer will do)
  const kv_status st = kv_compact_check(s, k, v, reinterpret_cast<const float*>(head_budget),
                                        nullptr, 1, 2, 0.0f, head_budget, reserve, kept_idx,
                                        cu_off, lens, k_flat, v_flat, flat_capacity_rows, ws);
  if (st != KV_OK) return st;
  if (ws_bytes < kWsHeader) return KV_ERR_WORKSPACE;
  return cuda_status(launch_compact_streaming(s, k, v, sinks, head_budget, reserve, kept_idx,
                                              cu_off, lens, k_flat, v_flat, flat_capacity_rows,
                                              static_cast<char*>(ws),
                                              static_cast<cudaStream_t>(stream)));
}

kv_status kv_compact_kappa(const kv_shape* shape, const void* k, const void* v,
                           const float* scores, const float* kappa, uint32_t crit_alpha_num,
                           uint32_t crit_alpha_den, const int32_t* head_budget, int32_t reserve,
                           int32_t* kept_idx, int64_t* cu_off, int32_t* lens, void* k_flat,
                           void* v_flat, int64_t flat_capacity_rows, void* ws, size_t ws_bytes,
                           void* stream) {
  if (kappa == nullptr) return KV_ERR_INVALID_ARG;
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  // the argument checks of kv_compact, with kappa in the norm's place
  const kv_status st = kv_compact_check(s, k, v, scores, kappa, crit_alpha_num, crit_alpha_den,
                                        0.0f, head_budget, reserve, kept_idx, cu_off, lens,
                                        k_flat, v_flat, flat_capacity_rows, ws);
  if (st != KV_OK) return st;
  const CompactPlan p = compact_plan(s, true);
  if (ws_bytes < p.off_end) return KV_ERR_WORKSPACE;
  return cuda_status(launch_compact(s, k, v, scores, kappa, crit_alpha_num, crit_alpha_den, 0.0f,
                                    true, head_budget, reserve, kept_idx, cu_off, lens, k_flat,
                                    v_flat, flat_capacity_rows, static_cast<char*>(ws), p,
                                    static_cast<cudaStream_t>(stream)));
}

kv_status kv_window_terms(const kv_shape* shape, int kind, const void* q_win, const void* k,
                          float* terms, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (kind != KV_TERMS_MEAN_POOLED && kind != KV_TERMS_L2) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  if (s.n == 0 || s.w == 0) return KV_ERR_INVALID_ARG;
  if (q_win == nullptr || k == nullptr || terms == nullptr) return KV_ERR_INVALID_ARG;
  if (!aligned16(q_win) || !aligned16(k) || !aligned16(terms)) return KV_ERR_INVALID_ARG;
  if (!shape_supported(s)) return KV_ERR_UNSUPPORTED;
  const ScorePlan p = score_plan(s, KV_SCORE_ADA);
  if (ws_bytes < p.off_end) return KV_ERR_WORKSPACE;
  return cuda_status(launch_window_terms(s, kind, q_win, k, terms, static_cast<char*>(ws), p,
                                         static_cast<cudaStream_t>(stream)));
}

kv_status kv_proj_score(const kv_shape* shape, int kind, const void* v, const void* w_o,
                        int32_t model_dim, const float* terms, float eps, float* out, void* ws,
                        size_t ws_bytes, void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (kind != KV_PROJ_CRIT_GQA && kind != KV_PROJ_LAPROX) return KV_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || std::isinf(eps)) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (s.units() == 0 || s.C() <= 0) return KV_OK;
  if (v == nullptr || w_o == nullptr || terms == nullptr || out == nullptr)
    return KV_ERR_INVALID_ARG;
  if (!aligned16(v) || !aligned16(w_o) || !aligned16(terms) || !aligned16(out))
    return KV_ERR_INVALID_ARG;
  if (model_dim <= 0 || model_dim % 8 != 0) return KV_ERR_INVALID_ARG;
  if (!shape_supported(s) || !crit_tc_supported(s, model_dim)) return KV_ERR_UNSUPPORTED;
  if (ws_bytes < kWsHeader) return KV_ERR_WORKSPACE;
  return cuda_status(launch_proj_tc(s, kind == KV_PROJ_CRIT_GQA ? 1 : 2, v, w_o, model_dim,
                                    terms, kind == KV_PROJ_CRIT_GQA ? eps : 0.0f, out,
                                    static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
}

// Argument checks of a decode step; on KV_OK, `s` and `p` hold its shape and workspace plan.
static kv_status decode_check(const kv_shape* shape, const void* q, const void* k_new,
                              const void* v_new, const void* k_flat, const void* v_flat,
                              const int64_t* cu_off, const int32_t* lens,
                              int64_t flat_capacity_rows, float softmax_scale, const void* out,
                              Shape* s, DecodePlan* p) {
  if (!shape_ok(shape, s)) return KV_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return KV_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale)) return KV_ERR_INVALID_ARG;
  if (flat_capacity_rows < 0) return KV_ERR_INVALID_ARG;
  if (s->units() == 0) {
    *p = DecodePlan{};
    return KV_OK;
  }
  if (q == nullptr || k_flat == nullptr || v_flat == nullptr || cu_off == nullptr ||
      lens == nullptr || out == nullptr)
    return KV_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k_flat, v_flat, cu_off, lens, out};
  for (const void* x : ptrs)
    if (!aligned16(x)) return KV_ERR_INVALID_ARG;
  if (k_new != nullptr && (!aligned16(k_new) || !aligned16(v_new))) return KV_ERR_INVALID_ARG;
  if (!shape_supported(*s) || s->G() * s->d > 1024) return KV_ERR_UNSUPPORTED;
  *p = decode_plan(*s);
  return KV_OK;
}

size_t kv_recompact_workspace_size(int64_t src_capacity_rows) {
  if (src_capacity_rows < 0) return 0;
  return recompact_ws_bytes(src_capacity_rows);
}

kv_status kv_recompact(const kv_shape* shape, const float* scores, const int32_t* head_budget,
                       const int32_t* src_kept, const int64_t* src_cu, const int32_t* src_lens,
                       const void* src_k, const void* src_v, int64_t src_capacity_rows,
                       int32_t reserve, const int64_t* row_base, int32_t* kept_idx,
                       int64_t* cu_off, int32_t* lens, void* k_flat, void* v_flat,
                       int64_t flat_capacity_rows, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  if (!shape_ok(shape, &s)) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (reserve < 0 || flat_capacity_rows < 0 || src_capacity_rows < 0) return KV_ERR_INVALID_ARG;
  if (s.units() == 0) return KV_OK;
  const bool full = src_kept == nullptr;   // the source is the uncompacted K/V
  if (full != (src_cu == nullptr) || full != (src_lens == nullptr)) return KV_ERR_INVALID_ARG;
  if (scores == nullptr || head_budget == nullptr || src_k == nullptr || src_v == nullptr ||
      kept_idx == nullptr || cu_off == nullptr || lens == nullptr || k_flat == nullptr ||
      v_flat == nullptr)
    return KV_ERR_INVALID_ARG;
  // the rows move as 16-byte vectors; every table is read and written element by element,
  // so slices of per-layer tables need only their element's alignment
  const void* rows[] = {src_k, src_v, k_flat, v_flat};
  for (const void* x : rows)
    if (!aligned16(x)) return KV_ERR_INVALID_ARG;
  auto al = [](const void* x, uintptr_t a) {
    return x == nullptr || (reinterpret_cast<uintptr_t>(x) & (a - 1)) == 0;
  };
  if (!al(scores, 4) || !al(head_budget, 4) || !al(src_kept, 4) || !al(src_cu, 8) ||
      !al(src_lens, 4) || !al(row_base, 8) || !al(kept_idx, 4) || !al(cu_off, 8) ||
      !al(lens, 4))
    return KV_ERR_INVALID_ARG;
  if (src_k == k_flat || src_v == v_flat) return KV_ERR_INVALID_ARG;
  if (!shape_supported(s)) return KV_ERR_UNSUPPORTED;
  const int64_t src_rows = full ? s.units() * (int64_t)s.n : src_capacity_rows;
  if (src_rows >= ((int64_t)1 << 31)) return KV_ERR_UNSUPPORTED;
  if (ws_bytes < recompact_ws_bytes(src_rows)) return KV_ERR_WORKSPACE;
  return cuda_status(launch_recompact(s, scores, head_budget, src_kept, src_cu, src_lens, src_k,
                                      src_v, src_rows, reserve, row_base, kept_idx, cu_off, lens,
                                      k_flat, v_flat, flat_capacity_rows,
                                      static_cast<char*>(ws),
                                      static_cast<cudaStream_t>(stream)));
}

kv_status flat_decode_attn(const kv_shape* shape, const void* q, const void* k_new,
                           const void* v_new, void* k_flat, void* v_flat, const int64_t* cu_off,
                           int32_t* lens, int64_t flat_capacity_rows, float softmax_scale,
                           void* out, void* ws, size_t ws_bytes, void* stream) {
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  Shape s;
  DecodePlan p;
  const kv_status st = decode_check(shape, q, k_new, v_new, k_flat, v_flat, cu_off, lens,
                                    flat_capacity_rows, softmax_scale, out, &s, &p);
  if (st != KV_OK || s.units() == 0) return st;
  if (ws_bytes < p.off_end) return KV_ERR_WORKSPACE;
  return cuda_status(launch_decode(s, q, k_new, v_new, k_flat, v_flat, cu_off, lens,
                                   flat_capacity_rows, softmax_scale, out,
                                   static_cast<char*>(ws), p, static_cast<cudaStream_t>(stream)));
}

size_t kv_paged_workspace_size(int op, const kv_paged_shape* shape) {
  PagedShape s;
  if (op >= KV_OP_QUANT_WRITE && op <= KV_OP_QUANT_DECODE) {
    if (quant_shape_check(shape, &s) != KV_OK) return 0;
    return op == KV_OP_QUANT_DECODE ? quant_decode_ws_bytes(s) : kWsHeader;
  }
  if (paged_shape_check(shape, &s) != KV_OK) return 0;
  switch (op) {
    case KV_OP_PAGE_MAP: return kPageMapWsBytes;
    case KV_OP_PAGED_WRITE: return kWsHeader;
    case KV_OP_PAGED_DECODE: return paged_decode_ws_bytes(s);
    default: return 0;
  }
}

kv_status kv_page_map(const kv_paged_shape* shape, const int32_t* lens, const int32_t* add,
                      int32_t* free_ring, const int64_t* free_state, int64_t slot_capacity,
                      int32_t* block_table, int32_t* lens_out, int64_t* free_out, int64_t* cu_add,
                      int64_t* slot_map, void* ws, size_t ws_bytes, void* stream) {
  PagedShape s;
  const kv_status st = paged_shape_check(shape, &s);
  if (st != KV_OK) return st;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (slot_capacity < 0 || slot_capacity >= INT32_MAX) return KV_ERR_INVALID_ARG;
  if (s.seqs == 0) return KV_OK;
  if (lens == nullptr || add == nullptr || free_ring == nullptr || free_state == nullptr ||
      block_table == nullptr || lens_out == nullptr || free_out == nullptr || cu_add == nullptr ||
      (slot_map == nullptr && slot_capacity > 0))
    return KV_ERR_INVALID_ARG;
  if (!aligned_to(lens, 4) || !aligned_to(add, 4) || !aligned_to(free_ring, 4) ||
      !aligned_to(free_state, 8) || !aligned_to(block_table, 4) || !aligned_to(lens_out, 4) ||
      !aligned_to(free_out, 8) || !aligned_to(cu_add, 8) || !aligned_to(slot_map, 8))
    return KV_ERR_INVALID_ARG;
  if (s.U() > KV_PAGE_MAP_MAX_TABLES) return KV_ERR_UNSUPPORTED;
  // lens_out is lens, or apart from lens and add; free_out likewise
  auto apart = [](const void* x, const void* y, int64_t bytes) {
    const char *p = static_cast<const char*>(x), *q = static_cast<const char*>(y);
    return p + bytes <= q || q + bytes <= p;
  };
  if (!apart(lens_out, add, s.U() * 4) || (lens_out != lens && !apart(lens_out, lens, s.U() * 4)) ||
      (free_out != free_state && !apart(free_out, free_state, 16)))
    return KV_ERR_INVALID_ARG;
  if (ws_bytes < kPageMapWsBytes) return KV_ERR_WORKSPACE;
  return cuda_status(launch_page_map(s, lens, add, free_ring, free_state, slot_capacity,
                                     block_table, lens_out, free_out, cu_add, slot_map,
                                     static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
}

kv_status kv_paged_write(const kv_paged_shape* shape, const void* k, const void* v,
                         int64_t src_stride, const int64_t* slot_map, int64_t rows,
                         const int64_t* n_rows, void* k_pages, void* v_pages, void* ws,
                         size_t ws_bytes, void* stream) {
  PagedShape s;
  const kv_status st = paged_shape_check(shape, &s);
  if (st != KV_OK) return st;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (rows < 0 || rows > INT32_MAX || src_stride < 0) return KV_ERR_INVALID_ARG;
  if (s.seqs == 0 || rows == 0) return KV_OK;
  if (k == nullptr || v == nullptr || slot_map == nullptr || k_pages == nullptr ||
      v_pages == nullptr)
    return KV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) ||
      !aligned_to(slot_map, 8) || !aligned_to(n_rows, 8))
    return KV_ERR_INVALID_ARG;
  const int64_t dense = (int64_t)s.Hp() * s.d;
  if (src_stride == 0) src_stride = dense;
  if (src_stride < dense || src_stride % (16 / s.esize()) != 0 ||
      src_stride > ((int64_t)1 << 31))
    return KV_ERR_INVALID_ARG;
  if (ws_bytes < kWsHeader) return KV_ERR_WORKSPACE;
  return cuda_status(launch_paged_write(s, k, v, src_stride, slot_map, rows, n_rows, k_pages,
                                        v_pages, static_cast<WsHeader*>(ws),
                                        static_cast<cudaStream_t>(stream)));
}

// What paged_decode_attn and quant_decode_attn check alike, after the shape.  *work is false where
// there is nothing to do.
static kv_status paged_decode_check(const PagedShape& s, const void* q, const void* k_new,
                                    const void* v_new, const int64_t* cu_add,
                                    const int64_t* slot_map, int64_t slot_capacity,
                                    const void* k_pages, const void* v_pages,
                                    const int32_t* block_table, const int32_t* lens,
                                    float softmax_scale, const void* out, const void* ws,
                                    size_t ws_bytes, size_t ws_needed, bool* work) {
  *work = false;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return KV_ERR_INVALID_ARG;
  if (!(std::fabs(softmax_scale) < 0x1p127f)) return KV_ERR_INVALID_ARG;   // times log2 e is finite
  if (slot_capacity < 0 || slot_capacity > INT32_MAX) return KV_ERR_INVALID_ARG;
  if (s.seqs == 0) return KV_OK;
  if (q == nullptr || k_pages == nullptr || v_pages == nullptr || block_table == nullptr ||
      lens == nullptr || out == nullptr)
    return KV_ERR_INVALID_ARG;
  if (k_new != nullptr && (cu_add == nullptr || (slot_map == nullptr && slot_capacity > 0)))
    return KV_ERR_INVALID_ARG;
  const void* rows[] = {q, k_new, v_new, k_pages, v_pages, out};
  for (const void* x : rows)
    if (!aligned16(x)) return KV_ERR_INVALID_ARG;
  if (!aligned_to(cu_add, 8) || !aligned_to(slot_map, 8) || !aligned_to(block_table, 4) ||
      !aligned_to(lens, 4))
    return KV_ERR_INVALID_ARG;
  // every CTA reads all lengths; the kernel counts tiles of at least 8 rows in 31 bits
  if (s.U() > KV_PAGED_DECODE_MAX_TABLES ||
      (int64_t)s.seqs * s.Hkv > (((int64_t)1 << 34) - 1) / ((int64_t)s.max_pages * s.page))
    return KV_ERR_UNSUPPORTED;
  if (ws_bytes < ws_needed) return KV_ERR_WORKSPACE;
  *work = true;
  return KV_OK;
}

kv_status paged_decode_attn(const kv_paged_shape* shape, const void* q, const void* k_new,
                            const void* v_new, const int64_t* cu_add, const int64_t* slot_map,
                            int64_t slot_capacity, void* k_pages, void* v_pages,
                            const int32_t* block_table, const int32_t* lens, float softmax_scale,
                            void* out, void* ws, size_t ws_bytes, void* stream) {
  PagedShape s;
  bool work;
  kv_status st = paged_shape_check(shape, &s);
  if (st != KV_OK) return st;
  st = paged_decode_check(s, q, k_new, v_new, cu_add, slot_map, slot_capacity, k_pages, v_pages,
                          block_table, lens, softmax_scale, out, ws, ws_bytes,
                          paged_decode_ws_bytes(s), &work);
  if (st != KV_OK || !work) return st;
  return cuda_status(launch_paged_decode(s, q, k_new, v_new, cu_add, slot_map, slot_capacity,
                                         k_pages, v_pages, block_table, lens, softmax_scale, out,
                                         static_cast<char*>(ws),
                                         static_cast<cudaStream_t>(stream)));
}

kv_status quant_decode_attn(const kv_paged_shape* shape, int format, const void* q,
                            const void* k_new, const void* v_new, const int64_t* cu_add,
                            const int64_t* slot_map, int64_t slot_capacity, void* k_pages,
                            void* v_pages, float* k_scale, float* v_scale,
                            const int32_t* block_table, const int32_t* lens, float softmax_scale,
                            void* out, void* ws, size_t ws_bytes, void* stream) {
  PagedShape s;
  bool work;
  kv_status st = quant_shape_check(shape, &s);
  if (st != KV_OK) return st;
  if (format != KV_E4M3 && format != KV_INT8) return KV_ERR_INVALID_ARG;
  if (s.seqs > 0 && (k_scale == nullptr || v_scale == nullptr)) return KV_ERR_INVALID_ARG;
  if (!aligned_to(k_scale, 4) || !aligned_to(v_scale, 4)) return KV_ERR_INVALID_ARG;
  st = paged_decode_check(s, q, k_new, v_new, cu_add, slot_map, slot_capacity, k_pages, v_pages,
                          block_table, lens, softmax_scale, out, ws, ws_bytes,
                          quant_decode_ws_bytes(s), &work);
  if (st != KV_OK || !work) return st;
  return cuda_status(launch_quant_decode(s, format, q, k_new, v_new, cu_add, slot_map,
                                         slot_capacity, k_pages, v_pages, k_scale, v_scale,
                                         block_table, lens, softmax_scale, out,
                                         static_cast<char*>(ws),
                                         static_cast<cudaStream_t>(stream)));
}

// What kv_quant_write and kv_quant_read check alike.  `rows_stride` becomes that of dense rows
// where it is 0; *work is false where there is nothing to do.
static kv_status quant_rows_check(const kv_paged_shape* shape, int format, const void* k,
                                  const void* v, int64_t* rows_stride, const int64_t* slot_map,
                                  int64_t rows, const int64_t* n_rows, const void* k_pages,
                                  const void* v_pages, const float* k_scale, const float* v_scale,
                                  const void* ws, size_t ws_bytes, PagedShape* s, bool* work) {
  *work = false;
  const kv_status st = quant_shape_check(shape, s);
  if (st != KV_OK) return st;
  if (format != KV_E4M3 && format != KV_INT8) return KV_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  if (rows < 0 || rows > INT32_MAX || *rows_stride < 0) return KV_ERR_INVALID_ARG;
  if (s->seqs == 0 || rows == 0) return KV_OK;
  if (k == nullptr || v == nullptr || slot_map == nullptr || k_pages == nullptr ||
      v_pages == nullptr || k_scale == nullptr || v_scale == nullptr)
    return KV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) ||
      !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) || !aligned_to(slot_map, 8) ||
      !aligned_to(n_rows, 8))
    return KV_ERR_INVALID_ARG;
  const int64_t dense = (int64_t)s->Hp() * s->d;
  if (*rows_stride == 0) *rows_stride = dense;
  if (*rows_stride < dense || *rows_stride % (16 / s->esize()) != 0 ||
      *rows_stride > ((int64_t)1 << 31))
    return KV_ERR_INVALID_ARG;
  if (ws_bytes < kWsHeader) return KV_ERR_WORKSPACE;
  *work = true;
  return KV_OK;
}

kv_status kv_quant_write(const kv_paged_shape* shape, int format, const void* k, const void* v,
                         int64_t src_stride, const int64_t* slot_map, int64_t rows,
                         const int64_t* n_rows, void* k_pages, void* v_pages, float* k_scale,
                         float* v_scale, void* ws, size_t ws_bytes, void* stream) {
  PagedShape s;
  bool work;
  const kv_status st = quant_rows_check(shape, format, k, v, &src_stride, slot_map, rows, n_rows,
                                        k_pages, v_pages, k_scale, v_scale, ws, ws_bytes, &s,
                                        &work);
  if (st != KV_OK || !work) return st;
  return cuda_status(launch_quant_write(s, format, k, v, src_stride, slot_map, rows, n_rows,
                                        k_pages, v_pages, k_scale, v_scale,
                                        static_cast<WsHeader*>(ws),
                                        static_cast<cudaStream_t>(stream)));
}

kv_status kv_quant_read(const kv_paged_shape* shape, int format, const void* k_pages,
                        const void* v_pages, const float* k_scale, const float* v_scale,
                        const int64_t* slot_map, int64_t rows, const int64_t* n_rows, void* k,
                        void* v, int64_t dst_stride, void* ws, size_t ws_bytes, void* stream) {
  PagedShape s;
  bool work;
  const kv_status st = quant_rows_check(shape, format, k, v, &dst_stride, slot_map, rows, n_rows,
                                        k_pages, v_pages, k_scale, v_scale, ws, ws_bytes, &s,
                                        &work);
  if (st != KV_OK || !work) return st;
  return cuda_status(launch_quant_read(s, format, k_pages, v_pages, k_scale, v_scale, slot_map,
                                       rows, n_rows, k, v, dst_stride, static_cast<WsHeader*>(ws),
                                       static_cast<cudaStream_t>(stream)));
}

kv_status kv_rotary(const kv_rotary_shape* shape, int back, const void* q, int64_t q_stride,
                    const void* k, int64_t k_stride, const int32_t* positions,
                    const double* inv_freq, int64_t rows, const int64_t* n_rows, void* q_out,
                    int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  if (shape == nullptr) return KV_ERR_INVALID_ARG;
  const RotaryShape s{shape->hq, shape->hkv, shape->d, shape->rot, shape->layout, shape->dtype,
                      shape->magnitude};
  if (s.hq < 0 || s.hkv < 0 || s.hq + (int64_t)s.hkv == 0 || s.d <= 0 || s.rot <= 0 || s.rot > s.d)
    return KV_ERR_INVALID_ARG;
  if (s.d % 8 != 0 || s.rot % 2 != 0) return KV_ERR_INVALID_ARG;
  if (s.layout != KV_ROTARY_HALF && s.layout != KV_ROTARY_INTERLEAVED) return KV_ERR_INVALID_ARG;
  if (s.dtype != KV_BF16 && s.dtype != KV_F32) return KV_ERR_INVALID_ARG;
  if (!std::isfinite(s.magnitude)) return KV_ERR_INVALID_ARG;
  if (s.d > 256 || s.rot % 8 != 0 || s.hq > 4096 || s.hkv > 4096) return KV_ERR_UNSUPPORTED;
  if (rows < 0 || rows > INT32_MAX) return KV_ERR_INVALID_ARG;
  struct Side {
    int heads;
    const void* in;
    const void* out;
    int64_t *in_stride, *out_stride;
  } sides[2] = {{s.hq, q, q_out, &q_stride, &q_out_stride},
                {s.hkv, k, k_out, &k_stride, &k_out_stride}};
  for (const Side& x : sides) {
    const int64_t dense = (int64_t)x.heads * s.d;
    for (int64_t* stride : {x.in_stride, x.out_stride}) {
      if (*stride == 0) *stride = dense;
      if (*stride < dense || *stride % (16 / s.esize()) != 0 || *stride > ((int64_t)1 << 31))
        return KV_ERR_INVALID_ARG;
    }
  }
  if (rows == 0) return KV_OK;
  if (positions == nullptr || inv_freq == nullptr) return KV_ERR_INVALID_ARG;
  if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 8) || !aligned_to(n_rows, 8))
    return KV_ERR_INVALID_ARG;
  for (const Side& x : sides) {
    if (x.heads == 0) continue;
    if (x.in == nullptr || x.out == nullptr || !aligned16(x.in) || !aligned16(x.out))
      return KV_ERR_INVALID_ARG;
    // in place, or apart from the rows that are read (counted in elements: no overflow)
    const int64_t row = (int64_t)x.heads * s.d;
    const int64_t in_rows = (rows - 1) * *x.in_stride + row;
    const int64_t out_rows = (rows - 1) * *x.out_stride + row;
    const int64_t ahead = ((int64_t)reinterpret_cast<uintptr_t>(x.out) -
                           (int64_t)reinterpret_cast<uintptr_t>(x.in)) / s.esize();
    if (ahead == 0 ? *x.in_stride != *x.out_stride && rows > 1 : ahead < in_rows && -ahead < out_rows)
      return KV_ERR_INVALID_ARG;
  }
  return cuda_status(launch_rotary(s, back != 0, q, q_stride, k, k_stride, positions, inv_freq,
                                   rows, n_rows, q_out, q_out_stride, k_out, k_out_stride,
                                   static_cast<cudaStream_t>(stream)));
}

kv_status kv_check_device_status(void* ws, void* stream, uint32_t* info) {
  if (ws == nullptr || !aligned16(ws)) return KV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  WsHeader h;
  if (cudaMemcpyAsync(&h, ws, 8, cudaMemcpyDeviceToHost, st) != cudaSuccess) return KV_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return KV_ERR_CUDA;
  if (h.err == 0) {
    if (info) *info = 0;
    return KV_OK;
  }
  if (info) *info = h.err;
  if (cudaMemsetAsync(ws, 0, 8, st) != cudaSuccess) return KV_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return KV_ERR_CUDA;
  return KV_ERR_DEVICE_CHECK;
}

kv_status flat_decode_attn_noalloc(const kv_shape* shape, const void* q, const void* k_new,
                                   const void* v_new, void* k_flat, void* v_flat,
                                   const int64_t* cu_off, int32_t* lens,
                                   int64_t flat_capacity_rows, float softmax_scale, void* out,
                                   void* stream) {
  Shape s;
  DecodePlan p;
  const kv_status st = decode_check(shape, q, k_new, v_new, k_flat, v_flat, cu_off, lens,
                                    flat_capacity_rows, softmax_scale, out, &s, &p);
  if (st != KV_OK || s.units() == 0) return st;
  // A decode whose plan needs more than the fixed array is refused before anything is
  // enqueued.
  if (p.off_end > (size_t)KV_DECODE_NOALLOC_SCRATCH_BYTES) return KV_ERR_WORKSPACE;
  void* scratch = nullptr;
  if (noalloc_scratch(&scratch) != cudaSuccess) return KV_ERR_CUDA;
  char* ws = static_cast<char*>(scratch);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // The array starts at zero when the library is loaded, but it is shared by every call and
  // no caller reads its error word back.  So each call clears, on its own stream, what the
  // decode kernels need at zero: the error word (a check that fired in an earlier call must
  // not linger) and the tickets and counter of the one-launch kernels (the split and the
  // heads in parts), which share one region.  Those return to zero at the end of every
  // complete launch; clearing them here also undoes a launch that was cut short or raced
  // with an overlapping call.  The partials, the chunk map and the work counter are written
  // before they are read in every launch.  A memset allocates nothing.
  if (cudaMemsetAsync(ws, 0, kWsHeader, cs) != cudaSuccess ||
      cudaMemsetAsync(ws + p.off_tick, 0, p.off_end - p.off_tick, cs) != cudaSuccess)
    return KV_ERR_CUDA;
  return cuda_status(launch_decode(s, q, k_new, v_new, k_flat, v_flat, cu_off, lens,
                                   flat_capacity_rows, softmax_scale, out, ws, p, cs));
}

uint64_t kv_kernel_launches(void) { return (uint64_t)g_launches.load(); }

const char* kv_status_string(kv_status status) {
  switch (status) {
    case KV_OK: return "ok";
    case KV_ERR_INVALID_ARG: return "invalid argument";
    case KV_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case KV_ERR_WORKSPACE: return "workspace too small";
    case KV_ERR_CAPACITY: return "flat buffer capacity too small";
    case KV_ERR_CUDA: return "CUDA error";
    case KV_ERR_DEVICE_CHECK: return "device-side check failed";
    default: return "unknown status";
  }
}

}  // extern "C"
