// C ABI of libfva: argument validation, workspace carving and kernel dispatch.
// Every check that can be made on the host is made here, before anything is enqueued.
#include <math.h>
#include <string.h>

#include "cache.cuh"
#include "fva_internal.cuh"

namespace fva {

bool route_shape_supported(const Dims& D);

bool make_dims(const fva_shape* s, Dims* out) {
  if (!s) return false;
  if (s->B < 1 || s->H < 1 || s->d < 1 || s->T < 1 || s->Hg < 1 || s->Wg < 1) return false;
  if (s->block != kBlock) return false;
  if (s->dtype != FVA_F32 && s->dtype != FVA_BF16) return false;
  Dims D;
  D.B = s->B;
  D.H = s->H;
  D.d = s->d;
  D.N = static_cast<int64_t>(s->T) * s->Hg * s->Wg;
  D.nB = (D.N + kBlock - 1) / kBlock;
  D.nPairs = (D.nB + 1) / 2;
  D.BH = D.B * D.H;
  D.rows = D.BH * D.nB;
  D.tiles = D.BH * D.nPairs;
  D.nWords = (D.nB + 31) / 32;
  D.esize = s->dtype == FVA_BF16 ? 2 : 4;
  if (D.N > 0x7fffffffLL || D.rows > 0x7fffffffLL) return false;
  const int64_t row_bytes = D.d * D.esize;
  if (row_bytes != 64 && row_bytes != 128 && row_bytes != 256 && row_bytes != 512 && row_bytes != 1024) return false;
  if (s->Hg > 65536 || s->Wg > 65536) return false;
  if (D.BH > 65535 || D.nB > 65535 * 8) return false;
  *out = D;
  return true;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int cuda_status(cudaError_t e) { return e == cudaSuccess ? FVA_OK : FVA_ERR_CUDA; }

struct Carver {
  uint8_t* base;
  size_t off;
  template <typename T>
  T* take(size_t bytes) {
    T* p = reinterpret_cast<T*>(base ? base + off : nullptr);
    off = align_up(off + bytes, 256);
    return p;
  }
};

static size_t route_scratch_layout(const Dims& D, int need_pool, void* ws, RouteScratch* rs, double** pq,
                                   double** pk, bool with_scores) {
  Carver c{static_cast<uint8_t*>(ws), 0};
  RouteScratch r;
  r.scores = with_scores ? c.take<double>(static_cast<size_t>(D.BH * D.nB * D.nB) * 8) : nullptr;
  r.bits = c.take<uint32_t>(static_cast<size_t>(D.rows * D.nWords) * 4);
  r.row_cnt = c.take<int32_t>(static_cast<size_t>(D.rows) * 4);
  r.head_load = c.take<int64_t>(static_cast<size_t>(D.BH) * 8);
  double* q = nullptr;
  double* k = nullptr;
  if (need_pool) {
    q = c.take<double>(static_cast<size_t>(D.rows * D.d) * 8);
    k = c.take<double>(static_cast<size_t>(D.rows * D.d) * 8);
  }
  if (rs) *rs = r;
  if (pq) *pq = q;
  if (pk) *pk = k;
  return c.off;
}

}  // namespace fva

using namespace fva;

extern "C" {

const char* fva_status_string(int status) {
  switch (status) {
    case FVA_OK: return "ok";
    case FVA_ERR_INVALID_ARG: return "invalid argument";
    case FVA_ERR_UNSUPPORTED_SHAPE: return "unsupported shape or dtype";
    case FVA_ERR_CAPACITY: return "mask buffer capacity too small";
    case FVA_ERR_CUDA: return "CUDA error";
    case FVA_ERR_DEVICE_TIMEOUT: return "device-side wait timed out";
    case FVA_ERR_WORKSPACE: return "workspace too small";
    case FVA_ERR_ALIGNMENT: return "device pointer not 16-byte aligned";
    case FVA_ERR_TOO_LARGE: return "shape needs more scratch than the fixed no-alloc array holds";
    default: return "unknown status";
  }
}

int fva_version(void) { return 100; }

void fva_set_diagnostics(uint64_t wait_limit_ns, int flags) {
  set_attn_diagnostics(wait_limit_ns, static_cast<uint32_t>(flags));
}

int fva_set_cta_trace(int64_t* trace_dev, int64_t capacity_ctas) {
  if ((trace_dev == nullptr) != (capacity_ctas == 0) || capacity_ctas < 0) return FVA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(trace_dev) % 8 != 0) return FVA_ERR_ALIGNMENT;
  set_attn_cta_trace(trace_dev, capacity_ctas);
  return FVA_OK;
}

int64_t fva_num_tokens(const fva_shape* s) {
  Dims D;
  return make_dims(s, &D) ? D.N : -1;
}
int64_t fva_num_blocks(const fva_shape* s) {
  Dims D;
  return make_dims(s, &D) ? D.nB : -1;
}
int64_t fva_num_tiles(const fva_shape* s) {
  Dims D;
  return make_dims(s, &D) ? D.tiles : -1;
}
int64_t fva_mask_capacity(const fva_shape* s) {
  Dims D;
  return make_dims(s, &D) ? D.BH * D.nB * D.nB : -1;
}
int64_t fva_tile_capacity(const fva_shape* s) {
  Dims D;
  return make_dims(s, &D) ? D.BH * D.nPairs * D.nB : -1;
}

size_t fva_route_workspace_bytes(const fva_shape* s, int need_pool) {
  Dims D;
  if (!make_dims(s, &D) || !route_shape_supported(D)) return 0;
  return route_scratch_layout(D, need_pool, nullptr, nullptr, nullptr, nullptr, true);
}

size_t fva_tiles_workspace_bytes(const fva_shape* s) {
  Dims D;
  if (!make_dims(s, &D)) return 0;
  return route_scratch_layout(D, 0, nullptr, nullptr, nullptr, nullptr, false);
}

int fva_hilbert_perm(const fva_shape* s, int32_t* perm_dev, int32_t* inv_dev, fva_stream_t stream) {
  Dims D;
  if (!s || !perm_dev || !inv_dev) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  return cuda_status(launch_hilbert_perm(D, s->T, s->Hg, s->Wg, perm_dev, inv_dev, stream));
}

int fva_curve_perm(const fva_shape* s, int curve, int32_t* perm_dev, int32_t* inv_dev, int32_t* dev_status,
                   fva_stream_t stream) {
  Dims D;
  if (!s || !perm_dev || !inv_dev) return FVA_ERR_INVALID_ARG;
  if (curve != FVA_CURVE_HILBERT && curve != FVA_CURVE_RECT) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (curve == FVA_CURVE_HILBERT) return cuda_status(launch_hilbert_perm(D, s->T, s->Hg, s->Wg, perm_dev, inv_dev, stream));
  return cuda_status(launch_rect_curve_perm(D, s->Hg, s->Wg, perm_dev, inv_dev, dev_status, stream));
}

int fva_reorder(const fva_shape* s, const void* x_in_dev, void* x_out_dev, double* pooled_dev,
                const int32_t* perm_dev, int direction, fva_stream_t stream) {
  Dims D;
  if (!s || !x_in_dev || !x_out_dev || !perm_dev) return FVA_ERR_INVALID_ARG;
  if (direction != FVA_FWD && direction != FVA_INV && direction != FVA_FWD_F16) return FVA_ERR_INVALID_ARG;
  if (direction != FVA_FWD && pooled_dev) return FVA_ERR_INVALID_ARG;
  if (direction == FVA_FWD_F16 && s->dtype != FVA_BF16) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x_in_dev) || !aligned16(x_out_dev) || (pooled_dev && !aligned16(pooled_dev)))
    return FVA_ERR_ALIGNMENT;
  if (x_in_dev == x_out_dev) return FVA_ERR_INVALID_ARG;
  return cuda_status(launch_reorder(D, x_in_dev, x_out_dev, pooled_dev, perm_dev, direction, stream));
}

int fva_pool(const fva_shape* s, const void* x_bhnd_dev, double* pooled_dev, fva_stream_t stream) {
  Dims D;
  if (!s || !x_bhnd_dev || !pooled_dev) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x_bhnd_dev) || !aligned16(pooled_dev)) return FVA_ERR_ALIGNMENT;
  return cuda_status(launch_pool(D, x_bhnd_dev, pooled_dev, stream));
}

static int check_mask_outputs(const Dims& D, const fva_mask* m) {
  if (!m || !m->row_ptr || !m->col_idx || !m->head_kept || !m->tile_ptr || !m->tile_col || !m->tile_cost ||
      !m->worklist)
    return FVA_ERR_INVALID_ARG;
  if (m->capacity < D.BH * D.nB * D.nB || m->tile_capacity < D.BH * D.nPairs * D.nB) return FVA_ERR_CAPACITY;
  if (D.BH * D.nB * D.nB > 0x7fffffffLL) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (m->logits && !aligned16(m->logits)) return FVA_ERR_ALIGNMENT;
  return FVA_OK;
}

int fva_route(const fva_shape* s, const void* q_bhnd_dev, const void* k_bhnd_dev, const double* pooled_q_dev,
              const double* pooled_k_dev, double p, int k_floor, int order, const fva_mask* mask,
              void* workspace_dev, size_t workspace_bytes, int32_t* dev_status, fva_stream_t stream) {
  Dims D;
  if (!s) return FVA_ERR_INVALID_ARG;
  if (!(p > 0.0 && p <= 1.0)) return FVA_ERR_INVALID_ARG;
  if (k_floor < 0) return FVA_ERR_INVALID_ARG;
  if (order != FVA_ORDER_NATURAL && order != FVA_ORDER_LPT && order != FVA_ORDER_HEAD_LPT) return FVA_ERR_INVALID_ARG;
  const bool have_pooled = pooled_q_dev && pooled_k_dev;
  if ((pooled_q_dev == nullptr) != (pooled_k_dev == nullptr)) return FVA_ERR_INVALID_ARG;
  if (!have_pooled && (!q_bhnd_dev || !k_bhnd_dev)) return FVA_ERR_INVALID_ARG;
  if (!workspace_dev) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!route_shape_supported(D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  int rc = check_mask_outputs(D, mask);
  if (rc != FVA_OK) return rc;
  const int need_pool = have_pooled ? 0 : 1;
  if (workspace_bytes < route_scratch_layout(D, need_pool, nullptr, nullptr, nullptr, nullptr, true))
    return FVA_ERR_WORKSPACE;
  if (!aligned16(workspace_dev)) return FVA_ERR_ALIGNMENT;
  RouteScratch rs;
  double* pq = const_cast<double*>(pooled_q_dev);
  double* pk = const_cast<double*>(pooled_k_dev);
  double* wq = nullptr;
  double* wk = nullptr;
  route_scratch_layout(D, need_pool, workspace_dev, &rs, &wq, &wk, true);
  if (need_pool) {
    if (!aligned16(q_bhnd_dev) || !aligned16(k_bhnd_dev)) return FVA_ERR_ALIGNMENT;
    cudaError_t e = launch_pool(D, q_bhnd_dev, wq, stream);
    if (e == cudaSuccess) e = launch_pool(D, k_bhnd_dev, wk, stream);
    if (e != cudaSuccess) return FVA_ERR_CUDA;
    pq = wq;
    pk = wk;
  }
  if (mask->logits) rs.scores = mask->logits;  // the logits go to the caller's buffer
  return cuda_status(launch_route(D, pq, pk, p, k_floor, order, mask, rs, dev_status, stream));
}

int fva_copy_strided(void* dst, size_t dst_pitch_bytes, const void* src, size_t src_pitch_bytes, size_t width_bytes,
                     int64_t rows, fva_stream_t stream) {
  if (!dst || !src || rows < 0) return FVA_ERR_INVALID_ARG;
  if (width_bytes > dst_pitch_bytes || width_bytes > src_pitch_bytes) return FVA_ERR_INVALID_ARG;
  if (rows == 0 || width_bytes == 0) return FVA_OK;
  return cuda_status(cudaMemcpy2DAsync(dst, dst_pitch_bytes, src, src_pitch_bytes, width_bytes,
                                       static_cast<size_t>(rows), cudaMemcpyDefault, stream));
}

size_t fva_sasa_workspace_bytes(const fva_shape* s) {
  Dims D;
  if (!make_dims(s, &D) || !route_shape_supported(D)) return 0;
  return route_scratch_layout(D, 0, nullptr, nullptr, nullptr, nullptr, true) + sasa_extra_bytes(D);
}

int fva_sasa_augment(const fva_shape* s, const double* pooled_q_dev, const double* pooled_k_dev,
                     const int32_t* rank_of_head_dev, int n_ranks, const int64_t* budget_dev, int order,
                     const fva_mask* mask, void* workspace_dev, size_t workspace_bytes, int64_t* added_dev,
                     int32_t* dev_status, fva_stream_t stream) {
  Dims D;
  if (!s || !rank_of_head_dev || !budget_dev || !workspace_dev) return FVA_ERR_INVALID_ARG;
  if (!mask) return FVA_ERR_INVALID_ARG;
  if (!mask->logits && (!pooled_q_dev || !pooled_k_dev)) return FVA_ERR_INVALID_ARG;
  if (n_ranks < 1 || n_ranks > FVA_SASA_MAX_RANKS) return FVA_ERR_INVALID_ARG;
  if (order != FVA_ORDER_NATURAL && order != FVA_ORDER_LPT && order != FVA_ORDER_HEAD_LPT) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!route_shape_supported(D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  int rc = check_mask_outputs(D, mask);
  if (rc != FVA_OK) return rc;
  const size_t base = route_scratch_layout(D, 0, nullptr, nullptr, nullptr, nullptr, true);
  if (workspace_bytes < base + sasa_extra_bytes(D)) return FVA_ERR_WORKSPACE;
  if (!aligned16(workspace_dev)) return FVA_ERR_ALIGNMENT;
  if (!mask->logits && (!aligned16(pooled_q_dev) || !aligned16(pooled_k_dev))) return FVA_ERR_ALIGNMENT;
  RouteScratch rs;
  route_scratch_layout(D, 0, workspace_dev, &rs, nullptr, nullptr, true);
  return cuda_status(launch_sasa(D, pooled_q_dev, pooled_k_dev, rank_of_head_dev, n_ranks, budget_dev, order, mask,
                                 rs, static_cast<uint8_t*>(workspace_dev) + base, added_dev, dev_status, stream));
}

int fva_sasa_budgets(const double* rank_load_ms, int n_ranks, double block_ms, double n1, double n2,
                     int64_t* budget_out) {
  if (!rank_load_ms || !budget_out || n_ranks < 1) return FVA_ERR_INVALID_ARG;
  if (!(block_ms > 0.0) || !(n1 >= 0.0) || !(n2 >= 0.0)) return FVA_ERR_INVALID_ARG;
  double crit = 0.0;
  for (int r = 0; r < n_ranks; ++r) {
    if (!(rank_load_ms[r] >= 0.0) || isinf(rank_load_ms[r])) return FVA_ERR_INVALID_ARG;
    if (rank_load_ms[r] > crit) crit = rank_load_ms[r];
  }
  for (int r = 0; r < n_ranks; ++r) {
    const double slack = crit - rank_load_ms[r];
    budget_out[r] = (crit > 0.0 && slack >= n2 * crit) ? static_cast<int64_t>(floor(n1 * slack / block_ms)) : 0;
  }
  return FVA_OK;
}

int fva_build_tiles(const fva_shape* s, const fva_mask* mask, int order, void* workspace_dev, size_t workspace_bytes,
                    int32_t* dev_status, fva_stream_t stream) {
  Dims D;
  if (!s || !workspace_dev) return FVA_ERR_INVALID_ARG;
  if (order != FVA_ORDER_NATURAL && order != FVA_ORDER_LPT && order != FVA_ORDER_HEAD_LPT) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  int rc = check_mask_outputs(D, mask);
  if (rc != FVA_OK) return rc;
  if (workspace_bytes < route_scratch_layout(D, 0, nullptr, nullptr, nullptr, nullptr, false)) return FVA_ERR_WORKSPACE;
  if (!aligned16(workspace_dev)) return FVA_ERR_ALIGNMENT;
  if (D.nPairs * 4 > 200 * 1024) return FVA_ERR_UNSUPPORTED_SHAPE;
  RouteScratch rs;
  route_scratch_layout(D, 0, workspace_dev, &rs, nullptr, nullptr, false);
  return cuda_status(launch_build_tiles(D, mask, order, rs, dev_status, stream));
}

static int attn_common(const fva_shape* s, const void* q, const void* k, const void* v, int v_dtype,
                       const fva_mask* m, void* o, float* lse, float scale, bool dense, int64_t first_slot,
                       int64_t n_slots, bool whole, int32_t* dev_status, fva_stream_t stream) {
  Dims D;
  if (!s || !q || !k || !v || !o) return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FVA_ERR_ALIGNMENT;
  if (o == q || o == k || o == v) return FVA_ERR_INVALID_ARG;
  if (lse && !aligned16(lse)) return FVA_ERR_ALIGNMENT;
  if (whole) {
    first_slot = 0;
    n_slots = D.tiles;
  }
  if (first_slot < 0 || n_slots < 0 || first_slot + n_slots > D.tiles) return FVA_ERR_INVALID_ARG;
  if (!(scale > 0.0f)) scale = 1.0f / sqrtf(static_cast<float>(D.d));
  if (s->dtype == FVA_BF16) {
    if (v_dtype != FVA_BF16 && v_dtype != FVA_F16) return FVA_ERR_INVALID_ARG;
    if (D.d != 64 && D.d != 128) return FVA_ERR_UNSUPPORTED_SHAPE;
    if (!dense && (!m || !m->tile_ptr || !m->tile_col || !m->worklist)) return FVA_ERR_INVALID_ARG;
    if (!attn_cta_trace_fits(D.tiles)) return FVA_ERR_CAPACITY;
    return cuda_status(launch_attn_bf16(D, q, k, v, v_dtype == FVA_F16, m, dense, o, lse, scale, first_slot, n_slots,
                                        dev_status, stream));
  }
  if (v_dtype != FVA_F32) return FVA_ERR_INVALID_ARG;
  if (D.d != 32 && D.d != 64 && D.d != 128) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!whole) return FVA_ERR_UNSUPPORTED_SHAPE;  // the fp32 path reads the CSR, not the work list
  if (!dense && (!m || !m->row_ptr || !m->col_idx)) return FVA_ERR_INVALID_ARG;
  return cuda_status(launch_attn_f32(D, static_cast<const float*>(q), static_cast<const float*>(k),
                                     static_cast<const float*>(v), dense ? nullptr : m->row_ptr,
                                     dense ? nullptr : m->col_idx, dense, static_cast<float*>(o), lse, scale, stream));
}

int fva_sparse_attn(const fva_shape* s, const void* q_dev, const void* k_dev, const void* v_dev, int v_dtype,
                    const fva_mask* mask, void* o_dev, float scale, int32_t* dev_status, fva_stream_t stream) {
  return attn_common(s, q_dev, k_dev, v_dev, v_dtype, mask, o_dev, nullptr, scale, false, 0, 0, true, dev_status, stream);
}

int fva_sparse_attn_range(const fva_shape* s, const void* q_dev, const void* k_dev, const void* v_dev, int v_dtype,
                          const fva_mask* mask, void* o_dev, float scale, int64_t first_slot, int64_t n_slots,
                          int32_t* dev_status, fva_stream_t stream) {
  return attn_common(s, q_dev, k_dev, v_dev, v_dtype, mask, o_dev, nullptr, scale, false, first_slot, n_slots, false,
                     dev_status, stream);
}

int fva_dense_attn(const fva_shape* s, const void* q_dev, const void* k_dev, const void* v_dev, int v_dtype,
                   void* o_dev, float scale, int32_t* dev_status, fva_stream_t stream) {
  return attn_common(s, q_dev, k_dev, v_dev, v_dtype, nullptr, o_dev, nullptr, scale, true, 0, 0, true, dev_status, stream);
}

int fva_sparse_attn_lse(const fva_shape* s, const void* q_dev, const void* k_dev, const void* v_dev, int v_dtype,
                        const fva_mask* mask, void* o_dev, float* lse_dev, float scale, int32_t* dev_status,
                        fva_stream_t stream) {
  if (!lse_dev) return FVA_ERR_INVALID_ARG;
  return attn_common(s, q_dev, k_dev, v_dev, v_dtype, mask, o_dev, lse_dev, scale, false, 0, 0, true, dev_status,
                     stream);
}

// Shapes that the gradient takes: the attention's head dims, int32 list offsets, and in shared
// memory one int32 per tile of a head (order) and 64 bit rows of nB bits (transposition).
static bool bwd_shape_supported(const Dims& D) {
  if (D.d != 64 && D.d != 128 && !(D.esize == 4 && D.d == 32)) return false;
  return D.BH * D.nB * D.nB <= 0x7fffffffLL && D.nB <= 25600;
}

static size_t bwd_scratch_layout(const Dims& D, void* ws, BwdScratch* out) {
  Carver c{static_cast<uint8_t*>(ws), 0};
  BwdScratch b{};
  b.stats = c.take<float>(static_cast<size_t>(D.rows) * 2 * kBlock * 4);
  b.lists.cost = c.take<int32_t>(static_cast<size_t>(D.tiles) * 4);
  b.worklist = c.take<int32_t>(static_cast<size_t>(D.tiles) * 4);
  b.lists.col = c.take<int32_t>(static_cast<size_t>(D.tiles * D.nB) * 4);
  if (out) *out = b;
  return c.off;
}

size_t fva_sparse_attn_bwd_workspace_bytes(const fva_shape* s) {
  Dims D;
  if (!make_dims(s, &D) || !bwd_shape_supported(D)) return 0;
  return bwd_scratch_layout(D, nullptr, nullptr);
}

int fva_sparse_attn_bwd(const fva_shape* s, const void* q_dev, const void* k_dev, const void* v_dev, const void* o_dev,
                        const void* d_o_dev, const float* lse_dev, const fva_mask* mask, void* dq_dev, void* dk_dev,
                        void* dv_dev, float scale, void* workspace_dev, size_t workspace_bytes, int32_t* dev_status,
                        fva_stream_t stream) {
  Dims D;
  const void* in[5] = {q_dev, k_dev, v_dev, o_dev, d_o_dev};
  void* out[3] = {dq_dev, dk_dev, dv_dev};
  if (!s || !lse_dev || !mask || !workspace_dev) return FVA_ERR_INVALID_ARG;
  for (const void* p : in)
    if (!p) return FVA_ERR_INVALID_ARG;
  for (const void* p : out)
    if (!p) return FVA_ERR_INVALID_ARG;
  if (!mask->row_ptr || !mask->col_idx || !mask->tile_ptr || !mask->tile_col || !mask->worklist)
    return FVA_ERR_INVALID_ARG;
  if (!make_dims(s, &D) || !bwd_shape_supported(D)) return FVA_ERR_UNSUPPORTED_SHAPE;
  for (int i = 0; i < 3; ++i) {
    for (const void* p : in)
      if (p == out[i]) return FVA_ERR_INVALID_ARG;
    if (out[i] == out[(i + 1) % 3]) return FVA_ERR_INVALID_ARG;
  }
  for (const void* p : in)
    if (!aligned16(p)) return FVA_ERR_ALIGNMENT;
  for (const void* p : out)
    if (!aligned16(p)) return FVA_ERR_ALIGNMENT;
  if (!aligned16(lse_dev) || !aligned16(workspace_dev)) return FVA_ERR_ALIGNMENT;
  if (workspace_bytes < bwd_scratch_layout(D, nullptr, nullptr)) return FVA_ERR_WORKSPACE;
  BwdScratch ws;
  bwd_scratch_layout(D, workspace_dev, &ws);
  if (!(scale > 0.0f)) scale = 1.0f / sqrtf(static_cast<float>(D.d));
  const BwdArgs x = {q_dev, k_dev, v_dev, o_dev, d_o_dev, lse_dev, dq_dev, dk_dev, dv_dev, scale};
  return cuda_status(launch_attn_bwd(D, x, mask, ws, dev_status, stream));
}

// ---------------------------------------------------------------------------------
// Paged cache
// ---------------------------------------------------------------------------------
static int check_cache(const fva_cache* c, const fva_seqs* q) {
  if (!c || !q || !c->k || !c->v || !c->key_mean || !q->table || !q->len) return FVA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->Hkv < 1 || q->B < 1 || q->max_blocks < 1) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (c->dtype != FVA_F32 && c->dtype != FVA_BF16 && c->dtype != FVA_F16) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (c->d != 64 && c->d != 128 && !(c->dtype == FVA_F32 && c->d == 32)) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (c->Hkv > 65535 || q->B > 65535 || q->max_blocks > kMaxCacheBlocks) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->key_mean) || !aligned16(c->mass)) return FVA_ERR_ALIGNMENT;
  return FVA_OK;
}

// Query rows: H a multiple of Hkv, rows that start on 16 bytes.
static int check_query(const fva_cache* c, const fva_seqs* q, const void* q_dev, int H, int64_t q_stride) {
  if (!q_dev) return FVA_ERR_INVALID_ARG;
  if (H < 1 || H > 65535 || H % c->Hkv != 0 || H / c->Hkv > kMaxCacheGroup) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<int64_t>(q->B) * H > 0x7fffffffLL) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (q_stride < static_cast<int64_t>(H) * c->d) return FVA_ERR_INVALID_ARG;
  if (!aligned16(q_dev) || q_stride * (c->dtype == FVA_F32 ? 4 : 2) % 16 != 0) return FVA_ERR_ALIGNMENT;
  return FVA_OK;
}

int fva_cache_append(const fva_cache* cache, const fva_seqs* seqs, const void* k_new_dev, const void* v_new_dev,
                     int64_t n_tokens, int64_t token_stride, const int32_t* new_ptr_dev, int max_new,
                     int32_t* dev_status, fva_stream_t stream) {
  const int rc = check_cache(cache, seqs);
  if (rc != FVA_OK) return rc;
  if (!new_ptr_dev || n_tokens < 0 || max_new < 0 || max_new > kMaxCacheBlocks * kBlock) return FVA_ERR_INVALID_ARG;
  if (max_new == 0) return FVA_OK;
  if (!k_new_dev || !v_new_dev || token_stride < static_cast<int64_t>(cache->Hkv) * cache->d) return FVA_ERR_INVALID_ARG;
  if (!aligned16(k_new_dev) || !aligned16(v_new_dev) || token_stride * (cache->dtype == FVA_F32 ? 4 : 2) % 16 != 0)
    return FVA_ERR_ALIGNMENT;
  return cuda_status(launch_cache_append(cache, seqs, k_new_dev, v_new_dev, n_tokens, token_stride, new_ptr_dev, max_new,
                                         dev_status, stream));
}

static bool batch_sizes_ok(const fva_cache* c, int B, int max_blocks) {
  return c && c->Hkv >= 1 && c->Hkv <= 65535 && c->d >= 1 && B >= 1 && B <= 65535 && max_blocks >= 1 &&
         max_blocks <= kMaxCacheBlocks;
}

size_t fva_cache_route_workspace_bytes(const fva_cache* cache, int B, int max_blocks, int H) {
  if (!batch_sizes_ok(cache, B, max_blocks) || H < 1) return 0;
  return align_up(static_cast<size_t>(B) * H * max_blocks * sizeof(double), 256);
}

int fva_cache_route(const fva_cache* cache, const fva_seqs* seqs, const void* q_dev, int H, int64_t q_stride, double p,
                    int k_floor, int n_recent, float scale, int32_t* kept_dev, int32_t* n_kept_dev,
                    void* workspace_dev, size_t workspace_bytes, int32_t* dev_status, fva_stream_t stream) {
  int rc = check_cache(cache, seqs);
  if (rc == FVA_OK) rc = check_query(cache, seqs, q_dev, H, q_stride);
  if (rc != FVA_OK) return rc;
  if (!(p > 0.0 && p <= 1.0) || k_floor < 0 || n_recent < 0 || !kept_dev || !n_kept_dev || !workspace_dev)
    return FVA_ERR_INVALID_ARG;
  if (workspace_bytes < fva_cache_route_workspace_bytes(cache, seqs->B, seqs->max_blocks, H)) return FVA_ERR_WORKSPACE;
  if (!aligned16(workspace_dev) || !aligned16(kept_dev) || !aligned16(n_kept_dev)) return FVA_ERR_ALIGNMENT;
  const double sc = scale > 0.0f ? static_cast<double>(scale) : 1.0 / sqrt(static_cast<double>(cache->d));
  return cuda_status(launch_cache_route(cache, seqs, q_dev, H, q_stride, p, k_floor, n_recent, sc, kept_dev, n_kept_dev,
                                        static_cast<double*>(workspace_dev), dev_status, stream));
}

static size_t cache_attn_layout(const fva_cache* c, int B, int max_blocks, int H, int accumulate, void* ws,
                                CacheAttnScratch* out) {
  Carver k{static_cast<uint8_t*>(ws), 0};
  CacheAttnScratch a{};
  a.part = k.take<float>(cache_attn_part_floats(c->d) * sizeof(float));
  a.per = k.take<int64_t>(sizeof(int64_t));
  a.start = k.take<int64_t>(static_cast<size_t>(B) * H * sizeof(int64_t));  // at most a unit per query head
  if (accumulate) {
    a.lse = k.take<float>(static_cast<size_t>(B) * H * sizeof(float));
    a.scores = k.take<float>(static_cast<size_t>(B) * H * max_blocks * kBlock * sizeof(float));
  }
  if (out) *out = a;
  return k.off;
}

size_t fva_cache_attn_workspace_bytes(const fva_cache* cache, int B, int max_blocks, int H, int accumulate) {
  if (!batch_sizes_ok(cache, B, max_blocks) || H < 1) return 0;
  return cache_attn_layout(cache, B, max_blocks, H, accumulate, nullptr, nullptr);
}

int fva_cache_attn(const fva_cache* cache, const fva_seqs* seqs, const void* q_dev, int H, int64_t q_stride,
                   const int32_t* kept_dev, const int32_t* n_kept_dev, void* o_dev, float* lse_dev, float scale,
                   int accumulate, void* workspace_dev, size_t workspace_bytes, int32_t* dev_status,
                   fva_stream_t stream) {
  int rc = check_cache(cache, seqs);
  if (rc == FVA_OK) rc = check_query(cache, seqs, q_dev, H, q_stride);
  if (rc != FVA_OK) return rc;
  if ((kept_dev == nullptr) != (n_kept_dev == nullptr) || !o_dev || !workspace_dev || (accumulate && !cache->mass) ||
      o_dev == q_dev)
    return FVA_ERR_INVALID_ARG;
  if (workspace_bytes < cache_attn_layout(cache, seqs->B, seqs->max_blocks, H, accumulate, nullptr, nullptr))
    return FVA_ERR_WORKSPACE;
  if (!aligned16(workspace_dev) || !aligned16(kept_dev) || !aligned16(n_kept_dev) || !aligned16(o_dev) || !aligned16(lse_dev))
    return FVA_ERR_ALIGNMENT;
  CacheAttnScratch ws;
  cache_attn_layout(cache, seqs->B, seqs->max_blocks, H, accumulate, workspace_dev, &ws);
  if (!(scale > 0.0f)) scale = 1.0f / sqrtf(static_cast<float>(cache->d));
  return cuda_status(launch_cache_attn(cache, seqs, q_dev, H, q_stride, kept_dev, n_kept_dev, o_dev, lse_dev, scale,
                                       accumulate, ws, dev_status, stream));
}

size_t fva_cache_evict_workspace_bytes(const fva_cache* cache, int B, int max_blocks) {
  return batch_sizes_ok(cache, B, max_blocks) ? cache_evict_clash_words(B) * sizeof(uint32_t) : 0;
}

int fva_cache_evict(const fva_cache* cache, const fva_seqs* seqs, int keep, int n_sink, int n_recent,
                    const int32_t* dst_table_dev, int dst_max_blocks, int32_t* kept_dev, int32_t* new_len_dev,
                    void* workspace_dev, size_t workspace_bytes, int32_t* dev_status, fva_stream_t stream) {
  const int rc = check_cache(cache, seqs);
  if (rc != FVA_OK) return rc;
  if (cache->Hkv > 65534) return FVA_ERR_UNSUPPORTED_SHAPE;
  if (!cache->mass || !dst_table_dev || !kept_dev || !new_len_dev || !workspace_dev) return FVA_ERR_INVALID_ARG;
  if (keep < 1 || keep > kMaxCacheBlocks * kBlock || n_sink < 0 || n_recent < 0 ||
      static_cast<int64_t>(n_sink) + n_recent > keep)
    return FVA_ERR_INVALID_ARG;
  if (dst_max_blocks < (keep + kBlock - 1) / kBlock) return FVA_ERR_CAPACITY;
  if (workspace_bytes < fva_cache_evict_workspace_bytes(cache, seqs->B, seqs->max_blocks)) return FVA_ERR_WORKSPACE;
  if (!aligned16(workspace_dev)) return FVA_ERR_ALIGNMENT;
  return cuda_status(launch_cache_evict(cache, seqs, keep, n_sink, n_recent, dst_table_dev, dst_max_blocks, kept_dev,
                                        new_len_dev, static_cast<uint32_t*>(workspace_dev), dev_status, stream));
}

}  // extern "C"
