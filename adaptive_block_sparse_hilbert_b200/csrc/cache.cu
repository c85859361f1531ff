// Paged key/value cache: append, routing of single queries, eviction by accumulated weight.
#include <math.h>

#include "cache.cuh"

namespace fva {

// Mean of a page's first n keys, one thread per channel: the sum in float64 in token order
// (exact for 16-bit keys of a usual range, so it does not depend on how the tokens came),
// divided, rounded once.
template <typename T>
__device__ __forceinline__ void write_mean(const T* page_k, int n, int d, float* mean) {
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    double s = 0.0;
    for (int r = 0; r < n; ++r) s += static_cast<double>(to_f32(page_k[r * d + c]));
    mean[c] = static_cast<float>(s / n);
  }
}

// ---------------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------------
// One CTA per (touched block, key head, sequence): its share of the new rows is copied in
// 16-byte pieces, then the page's mean is taken from the page itself.
template <typename T>
__global__ void __launch_bounds__(128) append_kernel(CacheView<T> c, const T* __restrict__ k_new,
                                                     const T* __restrict__ v_new, int64_t token_stride, int d,
                                                     const int32_t* __restrict__ new_ptr, int max_new,
                                                     int32_t* dev_status) {
  const int b = blockIdx.z, h = blockIdx.y;
  const int len = seq_len(c, b, dev_status);
  const int from = new_ptr[b], n_new = new_ptr[b + 1] - from;
  if (n_new <= 0 || n_new > max_new || n_new > len) {
    if (n_new != 0 && threadIdx.x == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
    return;
  }
  const int first = len - n_new;                     // position of the first new token
  const int block = first / kBlock + blockIdx.x;
  if (block * kBlock >= len) return;
  const int page = page_of(c, b, block, dev_status);
  if (page < 0) return;
  const int r0 = max(first - block * kBlock, 0), r1 = min(len - block * kBlock, kBlock);
  const int64_t base = (static_cast<int64_t>(page) * c.Hkv + h) * kBlock;
  const int vecs = d * static_cast<int>(sizeof(T)) / 16;  // 16-byte pieces of a row
  for (int i = threadIdx.x; i < (r1 - r0) * vecs; i += blockDim.x) {
    const int r = r0 + i / vecs, p = i % vecs;
    const int64_t src = (static_cast<int64_t>(from) + block * kBlock + r - first) * token_stride + static_cast<int64_t>(h) * d;
    reinterpret_cast<uint4*>(c.k + (base + r) * d)[p] = reinterpret_cast<const uint4*>(k_new + src)[p];
    reinterpret_cast<uint4*>(c.v + (base + r) * d)[p] = reinterpret_cast<const uint4*>(v_new + src)[p];
  }
  if (c.mass)
    for (int r = r0 + threadIdx.x; r < r1; r += blockDim.x) c.mass[base + r] = 0.0f;
  __syncthreads();
  write_mean(c.k + base * d, r1, d, c.key_mean + (static_cast<int64_t>(page) * c.Hkv + h) * d);
}

// ---------------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------------
// Block scores: one warp per block, lanes over the channels, one query head after another.
template <typename T>
__global__ void __launch_bounds__(128) cache_scores_kernel(CacheView<T> c, const T* __restrict__ q, int64_t q_stride,
                                                           int H, int d, double scale, double* __restrict__ scores,
                                                           int32_t* dev_status) {
  const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
  const int block = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int len = seq_len(c, b, dev_status);
  if (block * kBlock >= len) return;
  const int page = page_of(c, b, block, dev_status);
  const int G = H / c.Hkv;
  const float* mean = c.key_mean + (static_cast<int64_t>(page < 0 ? 0 : page) * c.Hkv + h) * d;
  for (int g = 0; g < G; ++g) {
    const T* qh = q + b * q_stride + static_cast<int64_t>(h * G + g) * d;
    double s = 0.0;
    if (page >= 0)
      for (int i = lane; i < d; i += 32) s = fma(static_cast<double>(to_f32(qh[i])), static_cast<double>(mean[i]), s);
    s = warp_sum_d(s) * scale;
    if (page < 0) s = -INFINITY;  // a block without a page is never chosen for its score
    if (lane == 0) scores[(static_cast<int64_t>(b) * H + h * G + g) * c.max_blocks + block] = s;
  }
}

constexpr double kMassUnit = 4503599627370496.0;  // 2^52: fixed-point unit of a block's share

__device__ __forceinline__ double block_reduce(double v, bool take_max, double* sm) {
  v = take_max ? warp_max_d(v) : warp_sum_d(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  const int n = blockDim.x >> 5;
  double r = sm[0];
  for (int i = 1; i < n; ++i) r = take_max ? fmax(r, sm[i]) : r + sm[i];
  return r;
}

// One CTA per (key head, sequence). Shares P_b in shared memory; the threshold is found
// digit by digit (8 bits of the float64 pattern, which orders non-negative values): a digit's
// bins hold their blocks' count and fixed-point mass, and the walk stops in the bin in which
// the prefix first has both the mass and the count it needs. Integer sums: any order of the
// atomics gives the same bins.
__global__ void __launch_bounds__(512) cache_select_kernel(const double* __restrict__ scores, int H, int Hkv,
                                                           int max_blocks, const int32_t* __restrict__ len_dev, double p,
                                                           int k_floor, int n_recent, int32_t* __restrict__ kept,
                                                           int32_t* __restrict__ n_kept) {
  extern __shared__ __align__(16) double prob[];  // [max_blocks]
  __shared__ double red[16];
  __shared__ unsigned long long bin_mass[256];
  __shared__ int bin_cnt[256];
  __shared__ unsigned long long s_prefix, s_mass_above;
  __shared__ int s_cnt_above, s_done, warp_cnt[16], s_nan;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int len = min(max(len_dev[b], 0), max_blocks * kBlock);
  const int nB = (len + kBlock - 1) / kBlock;
  int32_t* out = kept + (static_cast<int64_t>(b) * Hkv + h) * max_blocks;
  const int G = H / Hkv;

  if (tid == 0) s_nan = 0;
  for (int i = tid; i < nB; i += nt) prob[i] = 0.0;
  for (int g = 0; g < G; ++g) {
    const double* s = scores + (static_cast<int64_t>(b) * H + h * G + g) * max_blocks;
    double m = -INFINITY;
    bool bad = false;
    for (int i = tid; i < nB; i += nt) {
      m = fmax(m, s[i]);
      bad |= isnan(s[i]);
    }
    m = block_reduce(m, true, red);
    double z = 0.0;
    for (int i = tid; i < nB; i += nt) z += exp(s[i] - m);
    z = block_reduce(z, false, red);
    if (bad || !(z > 0.0) || isinf(z)) s_nan = 1;
    for (int i = tid; i < nB; i += nt) prob[i] += exp(s[i] - m) / (z * G);
  }
  __syncthreads();

  unsigned long long threshold = 0;  // blocks with a larger pattern are kept, `ties` of the equal ones
  int ties = 0;
  const bool all = p >= 1.0 || s_nan || nB == 0;
  if (!all) {
    const unsigned long long need_mass = static_cast<unsigned long long>(ceil(p * kMassUnit));
    const int need_cnt = min(k_floor, nB);
    if (tid == 0) {
      s_prefix = 0;
      s_mass_above = 0;
      s_cnt_above = 0;
    }
    for (int shift = 56; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += nt) {
        bin_mass[i] = 0;
        bin_cnt[i] = 0;
      }
      __syncthreads();
      const unsigned long long prefix = s_prefix;
      for (int i = tid; i < nB; i += nt) {
        const unsigned long long bits = __double_as_longlong(prob[i]);
        if (shift == 56 || (bits >> (shift + 8)) == (prefix >> (shift + 8))) {
          const int bin = static_cast<int>((bits >> shift) & 255);
          atomicAdd(&bin_mass[bin], static_cast<unsigned long long>(rint(prob[i] * kMassUnit)));
          atomicAdd(&bin_cnt[bin], 1);
        }
      }
      __syncthreads();
      if (tid == 0) {
        unsigned long long mass = s_mass_above;
        int cnt = s_cnt_above, bin = 255, last = -1;
        for (; bin >= 0; --bin) {
          if (bin_cnt[bin] == 0) continue;
          last = bin;
          if (mass + bin_mass[bin] >= need_mass && cnt + bin_cnt[bin] >= need_cnt) break;
          mass += bin_mass[bin];
          cnt += bin_cnt[bin];
        }
        if (bin < 0) {  // rounding left the total below p: the smallest block ends the prefix
          bin = last;
          mass -= bin_mass[bin];
          cnt -= bin_cnt[bin];
        }
        s_prefix = prefix | (static_cast<unsigned long long>(bin) << shift);
        s_mass_above = mass;
        s_cnt_above = cnt;
        s_done = bin_cnt[bin];
      }
      __syncthreads();
    }
    threshold = s_prefix;
    const double v = __longlong_as_double(threshold);
    const unsigned long long one = static_cast<unsigned long long>(rint(v * kMassUnit));
    ties = max(need_cnt - s_cnt_above, 1);
    if (s_mass_above < need_mass) {
      const unsigned long long lack = need_mass - s_mass_above;
      const unsigned long long n = one ? (lack + one - 1) / one : static_cast<unsigned long long>(s_done);
      if (n > static_cast<unsigned long long>(ties)) ties = n > static_cast<unsigned long long>(nB) ? nB : static_cast<int>(n);
    }
  }
  // emission in block order, 512 blocks at a time
  int written = 0, tied = 0;
  for (int base = 0; base < nB; base += nt) {
    const int i = base + tid;
    const unsigned long long bits = i < nB ? __double_as_longlong(prob[i]) : 0ull;
    const bool eq = !all && i < nB && bits == threshold;
    // rank among the equal ones
    const unsigned eqm = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) warp_cnt[warp] = __popc(eqm);
    __syncthreads();
    int before = tied + __popc(eqm & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < (nt >> 5); ++w) {
      if (w < warp) before += warp_cnt[w];
      total += warp_cnt[w];
    }
    tied += total;
    const bool keep = i < nB && (all || bits > threshold || (eq && before < ties) || i >= nB - n_recent);
    const unsigned km = __ballot_sync(0xffffffffu, keep);
    __syncthreads();
    if (lane == 0) warp_cnt[warp] = __popc(km);
    __syncthreads();
    int at = written + __popc(km & ((1u << lane) - 1u));
    total = 0;
    for (int w = 0; w < (nt >> 5); ++w) {
      if (w < warp) at += warp_cnt[w];
      total += warp_cnt[w];
    }
    if (keep) out[at] = i;
    written += total;
  }
  for (int i = written + tid; i < max_blocks; i += nt) out[i] = -1;
  if (tid == 0) n_kept[static_cast<int64_t>(b) * Hkv + h] = written;
}

// ---------------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------------
// Order-preserving pattern of a weight: larger weight, larger pattern; -0 as 0, NaN lowest.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (isnan(x)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One CTA per (key head, sequence): radix selection of the threshold over the middle tokens,
// then the kept positions in order.
template <typename T>
__global__ void __launch_bounds__(1024) evict_select_kernel(CacheView<T> c, int keep, int n_sink, int n_recent,
                                                            int32_t* __restrict__ kept, int32_t* __restrict__ new_len,
                                                            int32_t* dev_status) {
  __shared__ int bins[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, warp_cnt[32];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int len = seq_len(c, b, dev_status);
  int32_t* out = kept + (static_cast<int64_t>(b) * c.Hkv + h) * keep;
  if (h == 0 && tid == 0) new_len[b] = min(len, keep);
  auto key = [&](int t) -> uint32_t {
    const int page = page_of(c, b, t / kBlock, dev_status);
    return page < 0 ? 0u : mass_key(c.mass[(static_cast<int64_t>(page) * c.Hkv + h) * kBlock + t % kBlock]);
  };
  if (len <= keep) {
    for (int i = tid; i < keep; i += nt) out[i] = i < len ? i : -1;
    return;
  }
  const int lo = n_sink, hi = len - n_recent;
  int need = keep - n_sink - n_recent;  // of the tokens lo .. hi - 1, of which there are more
  uint32_t prefix = 0;
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    for (int i = tid; i < 256; i += nt) bins[i] = 0;
    __syncthreads();
    for (int t = lo + tid; t < hi; t += nt) {
      const uint32_t u = key(t);
      if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&bins[(u >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int bin = 255, left = need;
      while (bin > 0 && bins[bin] < left) left -= bins[bin--];
      s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // keys above the threshold, `need` of the equal ones (the earliest), the ends
  const bool some = keep > n_sink + n_recent;
  int written = 0, tied = 0;
  for (int base = 0; base < len; base += nt) {
    const int t = base + tid;
    const bool middle = t >= lo && t < hi;
    const uint32_t u = middle && some ? key(t) : 0u;
    const bool eq = middle && some && u == prefix;
    const unsigned eqm = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) warp_cnt[warp] = __popc(eqm);
    __syncthreads();
    int before = tied + __popc(eqm & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < (nt >> 5); ++w) {
      if (w < warp) before += warp_cnt[w];
      total += warp_cnt[w];
    }
    tied += total;
    const bool take = t < len && (!middle || (some && (u > prefix || (eq && before < need))));
    const unsigned km = __ballot_sync(0xffffffffu, take);
    __syncthreads();
    if (lane == 0) warp_cnt[warp] = __popc(km);
    __syncthreads();
    int at = written + __popc(km & ((1u << lane) - 1u));
    total = 0;
    for (int w = 0; w < (nt >> 5); ++w) {
      if (w < warp) at += warp_cnt[w];
      total += warp_cnt[w];
    }
    if (take) out[at] = t;
    written += total;
  }
}

// One CTA per (destination block, key head, sequence): gathers its 64 kept tokens.
template <typename T>
__global__ void __launch_bounds__(128) evict_copy_kernel(CacheView<T> c, int d, int keep,
                                                         const int32_t* __restrict__ dst_table, int dst_blocks,
                                                         const int32_t* __restrict__ kept, int32_t* dev_status) {
  const int b = blockIdx.z, h = blockIdx.y, block = blockIdx.x;
  const int len = seq_len(c, b, nullptr);
  const int n = min(min(len, keep) - block * kBlock, kBlock);
  if (n <= 0) return;
  const int dst = dst_table[static_cast<int64_t>(b) * dst_blocks + block];
  bool clash = false;
  for (int i = threadIdx.x; i * kBlock < len; i += blockDim.x)
    clash |= c.table[static_cast<int64_t>(b) * c.max_blocks + i] == dst;
  if (__syncthreads_or(clash) || dst < 0 || dst >= c.n_pages) {
    if (threadIdx.x == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
    return;
  }
  const int32_t* src_at = kept + (static_cast<int64_t>(b) * c.Hkv + h) * keep + block * kBlock;
  const int64_t to = (static_cast<int64_t>(dst) * c.Hkv + h) * kBlock;
  const int vecs = d * static_cast<int>(sizeof(T)) / 16;
  for (int i = threadIdx.x; i < n * vecs; i += blockDim.x) {
    const int r = i / vecs, p = i % vecs, t = src_at[r];
    const int page = page_of(c, b, t / kBlock, dev_status);
    const int64_t from = (static_cast<int64_t>(page < 0 ? dst : page) * c.Hkv + h) * kBlock + (page < 0 ? r : t % kBlock);
    reinterpret_cast<uint4*>(c.k + (to + r) * d)[p] = reinterpret_cast<const uint4*>(c.k + from * d)[p];
    reinterpret_cast<uint4*>(c.v + (to + r) * d)[p] = reinterpret_cast<const uint4*>(c.v + from * d)[p];
    if (p == 0) c.mass[to + r] = c.mass[from];
  }
  __syncthreads();
  write_mean(c.k + to * d, n, d, c.key_mean + (static_cast<int64_t>(dst) * c.Hkv + h) * d);
}

// ---------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------
template <typename T>
static cudaError_t append_t(const fva_cache* c, const fva_seqs* s, const void* k_new, const void* v_new, int64_t stride,
                            const int32_t* new_ptr, int max_new, int32_t* dev_status, cudaStream_t st) {
  // a sequence's new tokens touch at most this many blocks
  const dim3 grid(static_cast<unsigned>((max_new + kBlock - 2) / kBlock + 1), static_cast<unsigned>(c->Hkv), static_cast<unsigned>(s->B));
  append_kernel<T><<<grid, 128, 0, st>>>(cache_view<T>(c, s), static_cast<const T*>(k_new), static_cast<const T*>(v_new),
                                         stride, c->d, new_ptr, max_new, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const fva_cache* c, const fva_seqs* s, const void* k_new, const void* v_new,
                                int64_t stride, const int32_t* new_ptr, int max_new, int32_t* dev_status,
                                cudaStream_t st) {
  if (c->dtype == FVA_BF16) return append_t<__nv_bfloat16>(c, s, k_new, v_new, stride, new_ptr, max_new, dev_status, st);
  if (c->dtype == FVA_F16) return append_t<__half>(c, s, k_new, v_new, stride, new_ptr, max_new, dev_status, st);
  return append_t<float>(c, s, k_new, v_new, stride, new_ptr, max_new, dev_status, st);
}

template <typename T>
static cudaError_t scores_t(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride, double scale,
                            double* scores, int32_t* dev_status, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((s->max_blocks + 3) / 4), static_cast<unsigned>(c->Hkv), static_cast<unsigned>(s->B));
  cache_scores_kernel<T><<<grid, 128, 0, st>>>(cache_view<T>(c, s), static_cast<const T*>(q), q_stride, H, c->d, scale,
                                               scores, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_cache_route(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride, double p,
                               int k_floor, int n_recent, double scale, int32_t* kept, int32_t* n_kept, double* scores,
                               int32_t* dev_status, cudaStream_t st) {
  cudaError_t e = c->dtype == FVA_BF16  ? scores_t<__nv_bfloat16>(c, s, q, H, q_stride, scale, scores, dev_status, st)
                  : c->dtype == FVA_F16 ? scores_t<__half>(c, s, q, H, q_stride, scale, scores, dev_status, st)
                                        : scores_t<float>(c, s, q, H, q_stride, scale, scores, dev_status, st);
  if (e != cudaSuccess) return e;
  const size_t smem = static_cast<size_t>(s->max_blocks) * sizeof(double);
  e = cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cache_select_kernel<<<dim3(static_cast<unsigned>(c->Hkv), static_cast<unsigned>(s->B)), 512, smem, st>>>(
      scores, H, c->Hkv, s->max_blocks, s->len, p, k_floor, n_recent, kept, n_kept);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t evict_t(const fva_cache* c, const fva_seqs* s, int keep, int n_sink, int n_recent,
                           const int32_t* dst_table, int dst_blocks, int32_t* kept, int32_t* new_len,
                           int32_t* dev_status, cudaStream_t st) {
  const CacheView<T> v = cache_view<T>(c, s);
  const unsigned Hkv = static_cast<unsigned>(c->Hkv), B = static_cast<unsigned>(s->B);
  evict_select_kernel<T><<<dim3(Hkv, B), 1024, 0, st>>>(v, keep, n_sink, n_recent, kept, new_len, dev_status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_copy_kernel<T><<<dim3(static_cast<unsigned>((keep + kBlock - 1) / kBlock), Hkv, B), 128, 0, st>>>(
      v, c->d, keep, dst_table, dst_blocks, kept, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const fva_cache* c, const fva_seqs* s, int keep, int n_sink, int n_recent,
                               const int32_t* dst_table, int dst_blocks, int32_t* kept, int32_t* new_len,
                               int32_t* dev_status, cudaStream_t st) {
  if (c->dtype == FVA_BF16)
    return evict_t<__nv_bfloat16>(c, s, keep, n_sink, n_recent, dst_table, dst_blocks, kept, new_len, dev_status, st);
  if (c->dtype == FVA_F16)
    return evict_t<__half>(c, s, keep, n_sink, n_recent, dst_table, dst_blocks, kept, new_len, dev_status, st);
  return evict_t<float>(c, s, keep, n_sink, n_recent, dst_table, dst_blocks, kept, new_len, dev_status, st);
}

}  // namespace fva
