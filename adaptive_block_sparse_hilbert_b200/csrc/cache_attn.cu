// Attention of single query tokens over kept blocks of a paged key/value cache.
//
// A unit is one (sequence, key head, group of up to 16 query heads). All units' kept blocks,
// laid end to end, are cut into equal shares, one per CTA, so a long sequence spreads over
// many SMs and short ones share one: the work is a read of the kept keys and values, and every
// SM reads the same amount. A unit inside one CTA's share is finished there; one that crosses
// shares leaves each share's unnormalised O with its running maximum and sum in the workspace,
// and a second kernel joins them in share order (a fixed order: equal inputs, equal bits).
#include <math.h>

#include "cache.cuh"

namespace fva {

constexpr int kShares = 296;      // CTAs of the split kernel: two per SM
constexpr int kGroup = 16;        // query heads of a unit at most
constexpr int kSplitThreads = 128;

template <typename T>
struct AttnView {
  CacheView<T> c;
  const T* q;
  int64_t q_stride;
  const int32_t* kept;
  const int32_t* n_kept;
  int H, G, GS, units;  // G query heads per key head, GS units per (sequence, key head)
  float scale_log2;
  float* part;
  float* scores;
  float* lse2;
};

// Kept blocks of a unit (its list's length, or every block of the sequence).
template <typename T>
__device__ __forceinline__ int unit_count(const AttnView<T>& a, int u, int32_t* dev_status) {
  const int bh = u / a.GS, b = bh / a.c.Hkv;
  const int nB = (seq_len(a.c, b, dev_status) + kBlock - 1) / kBlock;
  if (!a.n_kept) return nB;
  const int n = a.n_kept[bh];
  if (n < 0 || n > nB) {
    report(dev_status, FVA_DEVERR_BAD_LIST);
    return n < 0 ? 0 : nB;
  }
  return n;
}

struct Share {
  int64_t total, per;  // blocks of all units, blocks of a share
  int unit;            // unit that holds this share's first block
  int64_t unit_start;  // first block of that unit
};

// Every thread of the CTA calls this; `at`: the block (of all units' blocks) to look up, in
// units of shares when by_share.
template <typename T>
__device__ Share find_share(const AttnView<T>& a, int share, int32_t* dev_status) {
  __shared__ int64_t warp_sum[32];
  __shared__ Share found;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (a.units + nt - 1) / nt;
  const int u0 = min(tid * chunk, a.units), u1 = min(u0 + chunk, a.units);
  int64_t mine = 0;
  for (int u = u0; u < u1; ++u) mine += unit_count(a, u, dev_status);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = inc - mine, total = 0;
  for (int w = 0; w < (nt >> 5); ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t per = (total + kShares - 1) / kShares;
  const int64_t at = share * per;
  if (at >= before && at < before + mine) {
    int64_t s = before;
    int u = u0;
    for (; u < u1; ++u) {
      const int n = unit_count(a, u, nullptr);
      if (at < s + n) break;
      s += n;
    }
    found.unit = u;
    found.unit_start = s;
  }
  if (tid == 0) {
    found.total = total;
    found.per = per;
  }
  __syncthreads();
  return found;
}

// Sums v[i] over the warp for N values at once (N a power of two <= 32): lanes i, i + N, ..
// end with value i. Each halving step keeps half of the values, so N - 1 + log2(32 / N)
// shuffles do what 5 N would.
template <int N>
__device__ __forceinline__ float warp_sum_many(float (&v)[N], int lane) {
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      const float keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, n);
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = to_f32(p[i]);
}

// One CTA per share. Each of the four warps takes 16 keys of every block with softmax
// statistics and an O of its own: lanes hold d / 32 channels each.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kSplitThreads) split_kernel(AttnView<T> a, T* __restrict__ o, float* __restrict__ lse,
                                                              int32_t* dev_status) {
  constexpr int V = D / 32;
  __shared__ float s_p[4][G][16];
  __shared__ float s_o[4][G][D];
  __shared__ float s_m[4][G], s_l[4][G];
  const int share = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Share sh = find_share(a, share, dev_status);
  int64_t at = share * sh.per;
  const int64_t end = min(sh.total, at + sh.per);
  if (at >= end) return;
  int u = sh.unit;
  int64_t start = sh.unit_start;
  bool first = true;
  while (at < end) {
    const int n = unit_count(a, u, nullptr);
    if (n == 0) {
      ++u;
      continue;
    }
    const int64_t stop = min(end, start + n);
    const int bh = u / a.GS, b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
    const int g0 = (u - bh * a.GS) * kGroup, ng = min(a.G - g0, kGroup);
    const int len = seq_len(a.c, b, nullptr);
    float q[G][V], acc[G][V], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g < ng)
        load_vec<T, V>(a.q + b * a.q_stride + static_cast<int64_t>(h * a.G + g0 + g) * D + lane * V, q[g]);
      m[g] = -INFINITY;
      l[g] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc[g][i] = 0.0f;
        q[g][i] = g < ng ? q[g][i] * a.scale_log2 : 0.0f;
      }
    }
    for (; at < stop; ++at) {
      const int pos = static_cast<int>(at - start);
      int block = pos;
      if (a.kept) {
        block = a.kept[static_cast<int64_t>(bh) * a.c.max_blocks + pos];
        if (block < 0 || block * static_cast<int64_t>(kBlock) >= len) {
          report(dev_status, FVA_DEVERR_BAD_LIST);
          block = -1;
        }
      }
      const int page = block < 0 ? -1 : page_of(a.c, b, block, dev_status);
      const int valid = page < 0 ? 0 : min(len - block * kBlock, kBlock);
      const int64_t base = (static_cast<int64_t>(page < 0 ? 0 : page) * a.c.Hkv + h) * kBlock;
      const int r0 = warp * 16, nk = max(0, min(valid - r0, 16));
      __syncwarp();
      for (int r = 0; r < 16; ++r) {
        float v[G];
        if (r < nk) {
          float k[V];
          load_vec<T, V>(a.c.k + (base + r0 + r) * D + lane * V, k);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            v[g] = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) v[g] = fmaf(q[g][i], k[i], v[g]);
          }
          const float s = warp_sum_many<G>(v, lane);
          if (lane < G) s_p[warp][lane][r] = s;
        } else if (lane < G) {
          s_p[warp][lane][r] = -INFINITY;
        }
      }
      __syncwarp();
      if (a.scores) {  // kept for the accumulation: raw scores, -inf behind the last key
        for (int i = lane; i < ng * 16; i += 32)
          a.scores[(static_cast<int64_t>(b) * a.H + h * a.G + g0 + i / 16) * a.c.max_blocks * kBlock +
                   static_cast<int64_t>(pos) * kBlock + r0 + i % 16] = s_p[warp][i / 16][i % 16];
      }
      if (nk > 0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float s = s_p[warp][g][lane & 15];
          float mx = s;
#pragma unroll
          for (int k = 8; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
          const float m_new = fmaxf(m[g], mx);
          const float corr = m_new == -INFINITY ? 1.0f : exp2f(m[g] - m_new);
          const float p = m_new == -INFINITY ? 0.0f : exp2f(s - m_new);
          m[g] = m_new;
          l[g] = l[g] * corr + (lane < 16 ? p : 0.0f);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[g][i] *= corr;
          __syncwarp();
          if (lane < 16) s_p[warp][g][lane] = p;
        }
        __syncwarp();
        for (int r = 0; r < nk; ++r) {
          float v[V];
          load_vec<T, V>(a.c.v + (base + r0 + r) * D + lane * V, v);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float p = s_p[warp][g][r];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[g][i] = fmaf(p, v[i], acc[g][i]);
          }
        }
      }
    }
    // join the four warps
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = l[g];
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      if (lane == 0) {
        s_m[warp][g] = m[g];
        s_l[warp][g] = sum;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s_o[warp][g][lane * V + i] = acc[g][i];
    }
    __syncthreads();
    const bool whole = stop == start + n && (!first || share * sh.per == start);
    float* part = a.part + (static_cast<int64_t>(share) * 2 + (first ? 0 : 1)) * kGroup * (D + 2);
    for (int i = threadIdx.x; i < ng * D; i += kSplitThreads) {
      const int g = i / D, ch = i % D;
      float mx = -INFINITY;
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, s_m[w][g]);
      float sum = 0.0f, x = 0.0f;
      for (int w = 0; w < 4; ++w) {
        const float f = s_m[w][g] == -INFINITY ? 0.0f : exp2f(s_m[w][g] - mx);
        sum = fmaf(s_l[w][g], f, sum);
        x = fmaf(s_o[w][g][ch], f, x);
      }
      const int64_t row = static_cast<int64_t>(b) * a.H + h * a.G + g0 + g;
      if (whole) {
        from_f32(sum > 0.0f ? x / sum : 0.0f, o + row * D + ch);
        if (ch == 0) {
          const float l2 = sum > 0.0f ? mx + log2f(sum) : -INFINITY;
          if (lse) lse[row] = l2 * 0.6931471805599453f;
          if (a.scores) a.lse2[row] = l2;
        }
      } else {
        part[g * (D + 2) + ch] = x;
        if (ch == 0) {
          part[g * (D + 2) + D] = mx;
          part[g * (D + 2) + D + 1] = sum;
        }
      }
    }
    __syncthreads();
    first = false;
    if (stop == start + n) {
      start += n;
      ++u;
    }
  }
}

// One CTA per unit: joins the shares of a unit that crosses them; rows without keys get 0.
template <typename T, int D>
__global__ void __launch_bounds__(kSplitThreads) join_kernel(AttnView<T> a, T* __restrict__ o, float* __restrict__ lse) {
  __shared__ int64_t s_start;
  __shared__ int64_t warp_sum[4], warp_before[4];
  const int u = blockIdx.x, tid = threadIdx.x;
  int64_t before = 0, total = 0;
  for (int i = tid; i < a.units; i += kSplitThreads) {
    const int n = unit_count(a, i, nullptr);
    total += n;
    if (i < u) before += n;
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, k);
    before += __shfl_xor_sync(0xffffffffu, before, k);
  }
  if ((tid & 31) == 0) {
    warp_sum[tid >> 5] = total;
    warp_before[tid >> 5] = before;
  }
  __syncthreads();
  total = warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3];
  if (tid == 0) s_start = warp_before[0] + warp_before[1] + warp_before[2] + warp_before[3];
  __syncthreads();
  const int64_t start = s_start, per = (total + kShares - 1) / kShares;
  const int n = unit_count(a, u, nullptr);
  const int bh = u / a.GS, b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
  const int g0 = (u - bh * a.GS) * kGroup, ng = min(a.G - g0, kGroup);
  const int64_t c0 = n ? start / per : 0, c1 = n ? (start + n - 1) / per : -1;
  if (n && c0 == c1) return;  // finished by the split kernel
  for (int i = tid; i < ng * D; i += kSplitThreads) {
    const int g = i / D, ch = i % D;
    float mx = -INFINITY, sum = 0.0f, x = 0.0f;
    for (int64_t s = c0; s <= c1; ++s) {
      const float* part = a.part + (s * 2 + (s * per >= start ? 0 : 1)) * kGroup * (D + 2) + g * (D + 2);
      const float m = part[D];
      if (m == -INFINITY) continue;
      const float m_new = fmaxf(mx, m), f0 = mx == -INFINITY ? 0.0f : exp2f(mx - m_new), f1 = exp2f(m - m_new);
      sum = sum * f0 + part[D + 1] * f1;
      x = x * f0 + part[ch] * f1;
      mx = m_new;
    }
    const int64_t row = static_cast<int64_t>(b) * a.H + h * a.G + g0 + g;
    from_f32(sum > 0.0f ? x / sum : 0.0f, o + row * D + ch);
    if (ch == 0) {
      const float l2 = sum > 0.0f ? mx + log2f(sum) : -INFINITY;
      if (lse) lse[row] = l2 * 0.6931471805599453f;
      if (a.scores) a.lse2[row] = l2;
    }
  }
}

// Adds exp(s - lse), summed over a key head's query heads, to the tokens' masses. One CTA per
// 4 listed blocks of a (sequence, key head); one thread per token.
template <typename T>
__global__ void __launch_bounds__(256) mass_kernel(AttnView<T> a) {
  const int b = blockIdx.z, h = blockIdx.y;
  const int pos = blockIdx.x * 4 + (threadIdx.x >> 6), r = threadIdx.x & 63;
  const int64_t bh = static_cast<int64_t>(b) * a.c.Hkv + h;
  if (pos >= unit_count(a, static_cast<int>(bh) * a.GS, nullptr)) return;
  const int block = a.kept ? a.kept[bh * a.c.max_blocks + pos] : pos;
  const int len = seq_len(a.c, b, nullptr);
  if (block < 0 || static_cast<int64_t>(block) * kBlock + r >= len) return;
  const int page = page_of(a.c, b, block, nullptr);
  if (page < 0) return;
  float w = 0.0f;
  for (int g = 0; g < a.G; ++g) {
    const int64_t row = static_cast<int64_t>(b) * a.H + h * a.G + g;
    w += exp2f(a.scores[row * a.c.max_blocks * kBlock + static_cast<int64_t>(pos) * kBlock + r] - a.lse2[row]);
  }
  atomicAdd(a.c.mass + (static_cast<int64_t>(page) * a.c.Hkv + h) * kBlock + r, w);
}

// ---------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------
size_t cache_attn_part_floats(int d) { return static_cast<size_t>(kShares) * 2 * kGroup * (d + 2); }

template <typename T, int D>
static cudaError_t attn_d(const AttnView<T>& a, void* o, float* lse, int accumulate, int32_t* dev_status,
                          cudaStream_t st) {
  T* out = static_cast<T*>(o);
  const int g = a.G < kGroup ? a.G : kGroup;
  if (g <= 1) split_kernel<T, D, 1><<<kShares, kSplitThreads, 0, st>>>(a, out, lse, dev_status);
  else if (g <= 4) split_kernel<T, D, 4><<<kShares, kSplitThreads, 0, st>>>(a, out, lse, dev_status);
  else if (g <= 8) split_kernel<T, D, 8><<<kShares, kSplitThreads, 0, st>>>(a, out, lse, dev_status);
  else split_kernel<T, D, 16><<<kShares, kSplitThreads, 0, st>>>(a, out, lse, dev_status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  join_kernel<T, D><<<static_cast<unsigned>(a.units), kSplitThreads, 0, st>>>(a, out, lse);
  e = cudaGetLastError();
  if (e != cudaSuccess || !accumulate) return e;
  mass_kernel<T><<<dim3(static_cast<unsigned>((a.c.max_blocks + 3) / 4), static_cast<unsigned>(a.c.Hkv),
                        static_cast<unsigned>(a.c.B)), 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t attn_t(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride,
                          const int32_t* kept, const int32_t* n_kept, void* o, float* lse, float scale, int accumulate,
                          const CacheAttnScratch& ws, int32_t* dev_status, cudaStream_t st) {
  const int G = H / c->Hkv, GS = (G + kGroup - 1) / kGroup;
  const AttnView<T> a = {cache_view<T>(c, s), static_cast<const T*>(q), q_stride, kept, n_kept, H, G, GS,
                         s->B * c->Hkv * GS, scale * 1.4426950408889634f, ws.part, accumulate ? ws.scores : nullptr,
                         ws.lse};
  if (c->d == 128) return attn_d<T, 128>(a, o, lse, accumulate, dev_status, st);
  if (c->d == 64) return attn_d<T, 64>(a, o, lse, accumulate, dev_status, st);
  if constexpr (sizeof(T) == 4) return attn_d<T, 32>(a, o, lse, accumulate, dev_status, st);
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_attn(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride,
                              const int32_t* kept, const int32_t* n_kept, void* o, float* lse, float scale,
                              int accumulate, const CacheAttnScratch& ws, int32_t* dev_status, cudaStream_t st) {
  if (c->dtype == FVA_BF16)
    return attn_t<__nv_bfloat16>(c, s, q, H, q_stride, kept, n_kept, o, lse, scale, accumulate, ws, dev_status, st);
  if (c->dtype == FVA_F16)
    return attn_t<__half>(c, s, q, H, q_stride, kept, n_kept, o, lse, scale, accumulate, ws, dev_status, st);
  return attn_t<float>(c, s, q, H, q_stride, kept, n_kept, o, lse, scale, accumulate, ws, dev_status, st);
}

}  // namespace fva
