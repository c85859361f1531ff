// Paged key/value cache: what its kernels share.
#pragma once

#include <cuda_fp16.h>

#include "fva_internal.cuh"

namespace fva {

constexpr int kMaxCacheBlocks = 16384;  // one CTA's shared memory holds a float64 per block
constexpr int kMaxCacheGroup = 128;     // query heads per key head

// Pointers of one cache and one batch of sequences, as the kernels take them.
template <typename T>
struct CacheView {
  T* k;
  T* v;
  float* key_mean;
  float* mass;
  const int32_t* table;
  const int32_t* len;
  int B, Hkv, n_pages, max_blocks;
};

template <typename T>
inline CacheView<T> cache_view(const fva_cache* c, const fva_seqs* q) {
  return {static_cast<T*>(c->k), static_cast<T*>(c->v), c->key_mean, c->mass, q->table,
          q->len,                q->B,                  c->Hkv,      c->n_pages, q->max_blocks};
}

// Sequence length, kept inside [0, 64 max_blocks]; a length outside is reported.
template <typename T>
__device__ __forceinline__ int seq_len(const CacheView<T>& c, int b, int32_t* dev_status) {
  const int n = c.len[b];
  if (n < 0 || n > c.max_blocks * kBlock) {
    report(dev_status, FVA_DEVERR_BAD_LIST);
    return n < 0 ? 0 : c.max_blocks * kBlock;
  }
  return n;
}

// Page of a sequence's block; -1, reported, when the table names no page.
template <typename T>
__device__ __forceinline__ int page_of(const CacheView<T>& c, int b, int block, int32_t* dev_status) {
  const int p = c.table[static_cast<int64_t>(b) * c.max_blocks + block];
  if (p >= 0 && p < c.n_pages) return p;
  report(dev_status, FVA_DEVERR_BAD_LIST);
  return -1;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float x, float* o) { *o = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* o) { *o = __float2bfloat16(x); }
__device__ __forceinline__ void from_f32(float x, __half* o) { *o = __float2half_rn(x); }

// Calls f with the element type and the head dim as template arguments.
template <typename F>
inline cudaError_t by_cache_type(const fva_cache* c, const F& f) {
  if (c->dtype == FVA_BF16)
    return c->d == 128 ? f.template operator()<__nv_bfloat16, 128>() : f.template operator()<__nv_bfloat16, 64>();
  if (c->dtype == FVA_F16) return c->d == 128 ? f.template operator()<__half, 128>() : f.template operator()<__half, 64>();
  if (c->d == 128) return f.template operator()<float, 128>();
  return c->d == 64 ? f.template operator()<float, 64>() : f.template operator()<float, 32>();
}

cudaError_t launch_cache_append(const fva_cache* c, const fva_seqs* q, const void* k_new, const void* v_new,
                                int64_t n_tokens, int64_t token_stride, const int32_t* new_ptr, int max_new, int32_t* dev_status,
                                cudaStream_t st);
cudaError_t launch_cache_route(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride, double p,
                               int k_floor, int n_recent, double scale, int32_t* kept, int32_t* n_kept, double* scores,
                               int32_t* dev_status, cudaStream_t st);
struct CacheAttnScratch {
  float* part;     // [2 * shares][16][d + 2]: unfinished rows' O, maximum and sum
  int64_t* start;  // [units] first block of a unit among all units' blocks
  int64_t* per;    // blocks of a share
  float* scores;   // [B, H, 64 * max_blocks], log2 units; only when weights are accumulated
  float* lse;      // [B, H] log2 units, likewise
};
size_t cache_attn_part_floats(int d);
cudaError_t launch_cache_attn(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride,
                              const int32_t* kept, const int32_t* n_kept, void* o, float* lse, float scale,
                              int accumulate, const CacheAttnScratch& ws, int32_t* dev_status, cudaStream_t st);
// clash: cache_evict_clash_words(B) words of workspace.
size_t cache_evict_clash_words(int B);
cudaError_t launch_cache_evict(const fva_cache* c, const fva_seqs* s, int keep, int n_sink, int n_recent,
                               const int32_t* dst_table, int dst_blocks, int32_t* kept, int32_t* new_len, uint32_t* clash,
                               int32_t* dev_status, cudaStream_t st);

}  // namespace fva
