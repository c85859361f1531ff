// Paged key/value cache: append, routing of single queries, eviction by accumulated weight.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "cache.cuh"

namespace fva {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------------
// Rows of a page: copy and mean (append, eviction)
// ---------------------------------------------------------------------------------
// A CTA holds the 64 rows of one (page, key head), 16 bytes a thread and row: thread = (row
// lane, 16-byte piece), rows row lane, row lane + kLanes, ... All of a thread's loads are issued
// before its first store, so a CTA has up to 32 KB in flight. (16 prompts, d = 128, on 128 / 256
// / 512 threads: 41 / 44 / 50 us of kernel. The gather of an eviction, while values still went through
// registers, took 3% longer on 128 and 5% longer on 512 threads than on 256.)
constexpr int kAppendThreads = 128, kEvictCopyThreads = 256;

template <typename T, int D, int kPageThreads>
struct PageRows {
  static constexpr int kPieces = D * static_cast<int>(sizeof(T)) / 16;
  static constexpr int kLanes = kPageThreads / kPieces;
  static constexpr int kRows = kBlock / kLanes;
  static constexpr int kPer = 16 / static_cast<int>(sizeof(T));  // values of a piece
};

// key_mean of the page from its rows' keys in registers (rows >= n are not counted): sums in
// float64 (exact for 16-bit keys of a usual range), divided, rounded once. A row's place in
// the sum depends on the row alone, so the mean does not depend on how the tokens came.
template <typename T, int D, int kPageThreads>
__device__ __forceinline__ void write_mean(const uint4 (&k)[PageRows<T, D, kPageThreads>::kRows], int n, float* mean) {
  using P = PageRows<T, D, kPageThreads>;
  __shared__ double sums[P::kLanes][D];
  const int lane = threadIdx.x / P::kPieces, piece = threadIdx.x % P::kPieces;
  double s[P::kPer];
#pragma unroll
  for (int i = 0; i < P::kPer; ++i) s[i] = 0.0;
#pragma unroll
  for (int r = 0; r < P::kRows; ++r) {
    const T* x = reinterpret_cast<const T*>(&k[r]);
    if (lane + r * P::kLanes < n) {
#pragma unroll
      for (int i = 0; i < P::kPer; ++i) s[i] += static_cast<double>(to_f32(x[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < P::kPer; ++i) sums[lane][piece * P::kPer + i] = s[i];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kPageThreads) {
    double t = 0.0;
#pragma unroll
    for (int l = 0; l < P::kLanes; ++l) t += sums[l][c];
    mean[c] = static_cast<float>(t / n);
  }
}

// ---------------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------------
// One CTA per (touched block, key head, sequence). Bound by the copy: 16 prompts of 1 to 4001
// tokens, 8 key heads, d = 128, take 41 us of kernel, the copy rate (a call among others 48).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(CacheView<T> c, const T* __restrict__ k_new,
                                                              const T* __restrict__ v_new, int64_t n_tokens,
                                                              int64_t token_stride,
                                                              const int32_t* __restrict__ new_ptr, int max_new,
                                                              int32_t* dev_status) {
  using P = PageRows<T, D, kAppendThreads>;
  const int b = blockIdx.z, h = blockIdx.y;
  const int len = seq_len(c, b, dev_status);
  const int from = new_ptr[b], to = new_ptr[b + 1], n_new = to - from;
  if (from < 0 || to <= from || to > n_tokens || n_new > max_new || n_new > len) {
    if (to != from && threadIdx.x == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
    return;
  }
  const int first = len - n_new;  // position of the first new token
  const int block = first / kBlock + blockIdx.x;
  if (block * kBlock >= len) return;
  const int page = page_of(c, b, block, dev_status);
  if (page < 0) return;
  const int r0 = max(first - block * kBlock, 0), r1 = min(len - block * kBlock, kBlock);
  const int64_t base = (static_cast<int64_t>(page) * c.Hkv + h) * kBlock;
  const int lane = threadIdx.x / P::kPieces, piece = threadIdx.x % P::kPieces;
  uint4 k[P::kRows], v[P::kRows];
#pragma unroll
  for (int i = 0; i < P::kRows; ++i) {
    const int r = lane + i * P::kLanes;
    const int64_t src = (static_cast<int64_t>(from) + block * kBlock + r - first) * token_stride + static_cast<int64_t>(h) * D;
    k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < r0) {
      k[i] = reinterpret_cast<const uint4*>(c.k + (base + r) * D)[piece];  // older, for the mean
    } else if (r < r1) {
      k[i] = reinterpret_cast<const uint4*>(k_new + src)[piece];
      v[i] = reinterpret_cast<const uint4*>(v_new + src)[piece];
    }
  }
#pragma unroll
  for (int i = 0; i < P::kRows; ++i) {
    const int r = lane + i * P::kLanes;
    if (r >= r0 && r < r1) {
      reinterpret_cast<uint4*>(c.k + (base + r) * D)[piece] = k[i];
      reinterpret_cast<uint4*>(c.v + (base + r) * D)[piece] = v[i];
      if (c.mass && piece == 0) c.mass[base + r] = 0.0f;
    }
  }
  write_mean<T, D, kAppendThreads>(k, r1, c.key_mean + (static_cast<int64_t>(page) * c.Hkv + h) * D);
}

// ---------------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------------
// A cluster of CTAs per (key head, sequence), each with a contiguous share of the blocks:
// scores in float64 (a share of the softmax next to the p border decides), the heads' maxima
// and sums joined over the cluster, then every block's share P_b, gathered in the shared
// memory of the cluster's first CTA, which selects. Bound by latencies: 32 sequences of 2 to 9
// thousand tokens, 32 query on 8 key heads, d = 128, take 23 us, of which the scores are a fifth;
// 131 and 250 thousand tokens, 40 on 8 heads, 35 us: scores 9, softmaxes 6, selection 6, emission 3.
constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRankMost = 256;    // this many blocks are ranked against one another (4 us)
constexpr int kDigitBits = 11, kDigitBins = 1 << kDigitBits;
constexpr double kMassUnit = 4503599627370496.0;  // 2^52: fixed-point unit of a block's share
constexpr int kHeads = 8;         // query heads of one pass over the means
constexpr int kMaxCluster = 8;

struct RouteShared {
  double part[2][kRouteWarps];                  // maxima, then sums, of a head's warps
  double top[kHeads], sum[kHeads];              // this CTA's maximum and sum of each head
  double cta_top[kMaxCluster][kHeads], cta_sum[kMaxCluster][kHeads];  // every CTA's
  double all_top[kHeads], inv[kHeads];          // the cluster's maximum, 1 / (sum G)
  double cand_p[kRankMost];
  unsigned long long cand_mass[kRankMost];
  int cand_at[kRankMost];
  unsigned long long warp_mass[kRouteWarps];
  int warp_cnt[kRouteWarps];
  unsigned long long prefix, mass_above;
  int cnt_above, in_bin, n_cand, bad;
  // a bin's fixed-point mass in three 18-bit parts (16384 of them fit 32 bits: plain atomics)
  // and its count
  unsigned int bin[4][kDigitBins];
};

__device__ __forceinline__ unsigned long long fixed_mass(double p) {
  return static_cast<unsigned long long>(__double2ll_rn(p * kMassUnit));
}

// Scores of up to 8 heads for the blocks [lo, hi): a warp takes eight blocks at a time through
// the float64 tensor cores (8 heads x 8 blocks x 4 channels an instruction), their means all on
// their way before the first is used. (Dot products by lanes and shuffles took 42 thousand
// cycles for a CTA's 488 blocks and 5 heads.) Lane (row, t) of a warp holds channels 16 i + 4 t
// .. + 3 of its head or block: the four products of 16 channels pair them in that order.
template <typename T, int D>
__device__ __forceinline__ void block_scores(const CacheView<T>& c, const double (*s_q)[D + 1], int ng, int b, int h,
                                             int lo, int hi, double scale, double* scores, int64_t stride,
                                             int32_t* dev_status) {
  constexpr int V = D / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane >> 2, t = lane & 3;
  auto find_page = [&](int at) { return at < hi ? page_of(c, b, at, dev_status) : 0; };
  int next = find_page(lo + warp * 8 + row);
#pragma unroll 1
  for (int base = lo + warp * 8; base < hi; base += kRouteWarps * 8) {
    const int page = next;
    const float* mean = c.key_mean + (static_cast<int64_t>(page < 0 ? 0 : page) * c.Hkv + h) * D + 4 * t;
    float4 m[V];
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = *reinterpret_cast<const float4*>(mean + 16 * i);
    next = find_page(base + kRouteWarps * 8 + row);
    double x[2] = {0.0, 0.0}, y[2] = {0.0, 0.0};  // two chains of products
    const double* q = s_q[row] + 4 * t;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dmma_8x8x4(x[0], x[1], q[16 * i], static_cast<double>(m[i].x));
      dmma_8x8x4(y[0], y[1], q[16 * i + 1], static_cast<double>(m[i].y));
      dmma_8x8x4(x[0], x[1], q[16 * i + 2], static_cast<double>(m[i].z));
      dmma_8x8x4(y[0], y[1], q[16 * i + 3], static_cast<double>(m[i].w));
    }
    x[0] += y[0];
    x[1] += y[1];
    // lane (head, t) holds blocks 2 t and 2 t + 1 of the eight
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool gone = __shfl_sync(0xffffffffu, page, (2 * t + k) * 4) < 0;  // no page: never chosen for its score
      if (row < ng && base + 2 * t + k < hi) scores[row * stride + base + 2 * t + k] = gone ? -INFINITY : x[k] * scale;
    }
  }
}

// The selection, by the cluster's first CTA. Block i is kept when the blocks before it (larger
// share, or equal and a lower index) lack the mass or the count the prefix needs. Up to 256
// blocks are ranked against one another. Of more, a histogram finds the bin in which the prefix
// ends: its key is the float64 pattern of 1 less that of the share, which orders shares from the
// largest down, and its first digit key >> 47, 32 bins an octave over 64 octaves, so that as a
// rule one pass leaves a few blocks to rank. Blocks of a bin that holds too many are told apart
// by the key's next 11 bits, and so on; shares below 2^-64 (all in the last bin) by the digits
// from the top. The sums are of integers: any order gives the same.
// Returns the key below which blocks are kept; a ranked block's share is set to 2 if it is kept,
// else to -1.
constexpr unsigned long long kOnePattern = 0x3ff0000000000000ull;
constexpr int kFirstShift = 47;
__device__ __forceinline__ unsigned long long share_key(double share) {
  return kOnePattern - static_cast<unsigned long long>(__double_as_longlong(share));
}
__device__ unsigned long long select_blocks(RouteShared& sm, double* prob, int nB, double p, int k_floor) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned long long need_mass = static_cast<unsigned long long>(ceil(p * kMassUnit));
  const int need_cnt = min(k_floor, nB);
  bool ranged = true;  // the first, logarithmic digit
  int shift = 64;
  if (tid == 0) {
    sm.prefix = 0;
    sm.mass_above = 0;
    sm.cnt_above = 0;
    sm.in_bin = nB;
    sm.n_cand = 0;
  }
  __syncthreads();
  while (sm.in_bin > kRankMost && shift > 0) {
    const int up = shift, width = shift >= kDigitBits ? kDigitBits : shift;
    shift = ranged ? kFirstShift : shift - width;
    for (int i = tid; i < kDigitBins; i += kRouteThreads) sm.bin[0][i] = sm.bin[1][i] = sm.bin[2][i] = sm.bin[3][i] = 0u;
    __syncthreads();
    const unsigned long long prefix = sm.prefix;
    for (int base = 0; base < nB; base += kRouteThreads) {
      const int i = base + tid;
      const unsigned long long key = i < nB ? share_key(prob[i]) : 0ull;
      const bool in = i < nB && (up == 64 || (key >> up) == (prefix >> up));
      const int d = !in      ? -1
                    : ranged ? static_cast<int>(min(key >> kFirstShift, static_cast<unsigned long long>(kDigitBins - 1)))
                             : static_cast<int>((key >> shift) & ((1 << width) - 1));
      int same;
      __match_all_sync(0xffffffffu, d, &same);
      const unsigned long long m = in ? fixed_mass(prob[i]) : 0ull;
      unsigned int part[4] = {static_cast<unsigned int>(m & 0x3ffff), static_cast<unsigned int>((m >> 18) & 0x3ffff),
                              static_cast<unsigned int>(m >> 36), in ? 1u : 0u};
      if (same) {  // one digit in the whole warp (blocks of equal shares): one addition for it
#pragma unroll
        for (int k = 0; k < 4; ++k) part[k] = __reduce_add_sync(0xffffffffu, part[k]);
      }
      if (d >= 0 && (!same || lane == 0)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (part[k]) atomicAdd(&sm.bin[k][d], part[k]);
      }
    }
    __syncthreads();
    // bins in order: four a thread, then a scan over the threads
    constexpr int kPer = kDigitBins / kRouteThreads;
    unsigned long long m[kPer], tm = 0;
    int n[kPer], tn = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int d = tid * kPer + k;
      m[k] = sm.bin[0][d] + (static_cast<unsigned long long>(sm.bin[1][d]) << 18) +
             (static_cast<unsigned long long>(sm.bin[2][d]) << 36);
      n[k] = static_cast<int>(sm.bin[3][d]);
      tm += m[k];
      tn += n[k];
    }
    unsigned long long im = tm;
    int in = tn;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long a = __shfl_up_sync(0xffffffffu, im, o);
      const int e = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) {
        im += a;
        in += e;
      }
    }
    if (lane == 31) {
      sm.warp_mass[warp] = im;
      sm.warp_cnt[warp] = in;
    }
    __syncthreads();
    unsigned long long mass = sm.mass_above + im - tm, total = sm.mass_above;
    int cnt = sm.cnt_above + in - tn;
    const int in_bin = sm.in_bin, cnt_before = sm.cnt_above;
    for (int w = 0; w < kRouteWarps; ++w) {
      if (w < warp) {
        mass += sm.warp_mass[w];
        cnt += sm.warp_cnt[w];
      }
      total += sm.warp_mass[w];
    }
    __syncthreads();
    // the bin in which the prefix first has both; where rounding leaves the total below p, the
    // last one that holds a block
    const bool short_of = total < need_mass;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const bool before = mass < need_mass || cnt < need_cnt;
      const bool after = mass + m[k] < need_mass || cnt + n[k] < need_cnt;
      const bool here = n[k] > 0 && before && (!after || (short_of && cnt + n[k] == cnt_before + in_bin));
      if (here) {
        const int d = tid * kPer + k;
        if (ranged && d == kDigitBins - 1) {  // shares below 2^-64: all digits from the top
          sm.prefix = ~0ull;
        } else {
          sm.prefix = prefix | (static_cast<unsigned long long>(d) << shift);
          sm.mass_above = mass;
          sm.cnt_above = cnt;
          sm.in_bin = n[k];
        }
      }
      mass += m[k];
      cnt += n[k];
    }
    __syncthreads();
    if (ranged && sm.prefix == ~0ull) {
      __syncthreads();
      if (tid == 0) sm.prefix = 0;
      shift = 64;
      __syncthreads();
    }
    ranged = false;
  }
  const unsigned long long prefix = sm.prefix;
  if (sm.in_bin <= kRankMost) {
    for (int i = tid; i < nB; i += kRouteThreads) {
      if (shift == 64 || (share_key(prob[i]) >> shift) == (prefix >> shift)) {
        const int at = atomicAdd(&sm.n_cand, 1);
        sm.cand_p[at] = prob[i];
        sm.cand_mass[at] = fixed_mass(prob[i]);
        sm.cand_at[at] = i;
      }
    }
    __syncthreads();
    const int n = sm.n_cand;
    int w = 1;  // lanes of a candidate
    while (w < 32 && n * w * 2 <= kRouteThreads) w *= 2;
    const int i = tid / w;
    const bool on = i < n;
    const double mine = on ? sm.cand_p[i] : 0.0;
    const int at = on ? sm.cand_at[i] : 0;
    unsigned long long mass = 0;
    int cnt = 0;
    if (on) {
      for (int j = tid % w; j < n; j += w) {
        const double o = sm.cand_p[j];
        const bool first = o > mine || (o == mine && sm.cand_at[j] < at);
        mass += first ? sm.cand_mass[j] : 0ull;
        cnt += first;
      }
    }
    for (int o = w / 2; o > 0; o >>= 1) {
      mass += __shfl_xor_sync(0xffffffffu, mass, o);
      cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
    }
    mass += sm.mass_above;
    cnt += sm.cnt_above;
    if (on && tid % w == 0) prob[at] = mass < need_mass || cnt < need_cnt ? 2.0 : -1.0;
    __syncthreads();
    return shift == 64 ? 0ull : prefix;  // the bins before the candidates' own
  }
  // more than 256 blocks of one and the same share: the first ones of them, by index
  const unsigned long long one = fixed_mass(__longlong_as_double(static_cast<long long>(kOnePattern - prefix)));
  long long ties = max(need_cnt - sm.cnt_above, 1);
  if (sm.mass_above < need_mass) {
    const unsigned long long lack = need_mass - sm.mass_above;
    const unsigned long long n = one ? (lack + one - 1) / one : static_cast<unsigned long long>(sm.in_bin);
    if (n > static_cast<unsigned long long>(ties)) ties = n > static_cast<unsigned long long>(nB) ? nB : static_cast<long long>(n);
  }
  int before = 0;  // equal ones at lower indices
  for (int base = 0; base < nB; base += kRouteThreads) {
    const int i = base + tid;
    const bool eq = i < nB && share_key(prob[i]) == prefix;
    const unsigned mask = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) sm.warp_cnt[warp] = __popc(mask);
    __syncthreads();
    int at = before + __popc(mask & ((1u << lane) - 1u));
    for (int w = 0; w < kRouteWarps; ++w) {
      if (w < warp) at += sm.warp_cnt[w];
      before += sm.warp_cnt[w];
    }
    if (eq) prob[i] = at < ties ? 2.0 : -1.0;
  }
  __syncthreads();
  return prefix;
}

// `score_cap`: blocks of a share whose scores (kHeads heads) fit shared memory behind prob, or
// 0: they go through the workspace.
template <typename T, int D>
__global__ void __launch_bounds__(kRouteThreads, 2) route_kernel(CacheView<T> c, const T* __restrict__ q, int64_t q_stride,
                                                              int H, double scale, double p, int k_floor, int n_recent,
                                                              int score_cap, double* __restrict__ scores,
                                                              int32_t* __restrict__ kept, int32_t* __restrict__ n_kept,
                                                              int32_t* dev_status) {
  extern __shared__ __align__(16) double prob[];  // [max_blocks], used in the cluster's first CTA
  __shared__ RouteShared sm;
  __shared__ double s_q[kHeads][D + 1];  // (the odd stride spreads the lanes' reads over the banks)
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_wait();
  grid_release();
  const int len = seq_len(c, b, dev_status);
  const int nB = (len + kBlock - 1) / kBlock, G = H / c.Hkv;
  const int per = (nB + C - 1) / C, lo = min(rank * per, nB), hi = min(lo + per, nB);
  double* const gathered = C > 1 ? cluster.map_shared_rank(prob, 0) : prob;
  auto sync_all = [&] {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  if (tid == 0) sm.bad = 0;

  for (int g0 = 0; g0 < G; g0 += kHeads) {
    const int ng = min(G - g0, kHeads);
    const T* qg = q + b * q_stride + static_cast<int64_t>(h * G + g0) * D;
    const int64_t stride = score_cap ? score_cap : c.max_blocks;
    // score of head g and block i at sg[g * stride + i]
    double* sg = score_cap ? prob + c.max_blocks - lo : scores + (static_cast<int64_t>(b) * H + h * G + g0) * c.max_blocks;
    for (int i = tid; i < kHeads * D; i += kRouteThreads)
      s_q[i / D][i % D] = i / D < ng ? static_cast<double>(to_f32(qg[i])) : 0.0;
    __syncthreads();
    block_scores<T, D>(c, s_q, ng, b, h, lo, hi, scale, sg, stride, dev_status);
    __syncthreads();
    // maxima and sums, 16 / ng warps a head (their order is fixed: equal inputs, equal bits)
    const int wph = kRouteWarps / ng, g = warp / wph, first = lo + (warp % wph) * 32 + lane;
    const double* s = sg + g * stride;
    double m = -INFINITY;
    bool nan = false;
    if (g < ng)
      for (int i = first; i < hi; i += wph * 32) {
        m = fmax(m, s[i]);
        nan |= isnan(s[i]);
      }
    if (nan) sm.bad = 1;
    m = warp_max_d(m);
    if (lane == 0) sm.part[0][warp] = m;
    __syncthreads();
    for (int k = 0; k < wph && g < ng; ++k) m = fmax(m, sm.part[0][g * wph + k]);
    double z = 0.0;
    if (g < ng)
      for (int i = first; i < hi; i += wph * 32) z += exp(s[i] - m);
    z = warp_sum_d(z);
    if (lane == 0) {
      sm.part[1][warp] = z;
      if (warp % wph == 0 && g < ng) sm.top[g] = m;
    }
    __syncthreads();
    if (tid < ng) {
      double t = 0.0;
      for (int k = 0; k < wph; ++k) t += sm.part[1][tid * wph + k];
      sm.sum[tid] = t;
    }
    sync_all();
    if (tid < C * kHeads) {  // a thread per CTA of the cluster and head
      const int r = tid / kHeads, k = tid % kHeads;
      const bool far = C > 1;
      sm.cta_top[r][k] = k < ng ? (far ? cluster.map_shared_rank(sm.top, r)[k] : sm.top[k]) : 0.0;
      sm.cta_sum[r][k] = k < ng ? (far ? cluster.map_shared_rank(sm.sum, r)[k] : sm.sum[k]) : 1.0;
    }
    __syncthreads();
    if (tid < C * kHeads) {
      const int r = tid / kHeads, k = tid % kHeads;
      double top = -INFINITY;
      for (int i = 0; i < C; ++i) top = fmax(top, sm.cta_top[i][k]);
      const double t = sm.cta_top[r][k];
      if (r == 0) sm.all_top[k] = top;
      // a CTA without a finite score (none of its own, or none at all) adds nothing
      sm.cta_sum[r][k] = t > -INFINITY ? sm.cta_sum[r][k] * exp(t - top) : 0.0;
    }
    __syncthreads();
    if (tid < ng) {
      double sum = 0.0;
      for (int i = 0; i < C; ++i) sum += sm.cta_sum[i][tid];
      if (!(sum > 0.0) || isinf(sum)) sm.bad = 1;  // no finite score, or a NaN
      sm.inv[tid] = 1.0 / (sum * G);
    }
    __syncthreads();
    // a block's share is a function of its scores alone (the cluster-wide maximum and sum), so
    // blocks of equal scores have equal shares whichever CTA holds them
    for (int i = lo + tid; i < hi; i += kRouteThreads) {
      double x = g0 > 0 ? gathered[i] : 0.0;
#pragma unroll 1
      for (int k = 0; k < ng; ++k) x += exp(sg[k * stride + i] - sm.all_top[k]) * sm.inv[k];
      gathered[i] = fmin(x, 1.0);  // (a share is at most 1 but for its last bit)
    }
    sync_all();  // the next heads overwrite the maxima; at the end, the shares are complete
  }
  bool bad = sm.bad != 0;
  if (C > 1) {
    for (int r = 0; r < C; ++r) bad |= *cluster.map_shared_rank(&sm.bad, r) != 0;
    cluster.sync();  // nobody leaves while its shared memory is read
  }
  if (rank != 0) return;

  const bool all = p >= 1.0 || bad || nB == 0;
  const unsigned long long border = all ? 0ull : select_blocks(sm, prob, nB, p, k_floor);
  // emission in block order, a contiguous piece a warp
  int32_t* out = kept + (static_cast<int64_t>(b) * c.Hkv + h) * c.max_blocks;
  const int piece = ((nB + kRouteWarps - 1) / kRouteWarps + 31) / 32 * 32, w0 = warp * piece;
  auto keep = [&](int i) -> bool {
    if (i >= nB) return false;
    const double x = prob[i];
    return all || i >= nB - n_recent || x > 1.0 || (x >= 0.0 && share_key(x) < border);
  };
  int n = 0;
  for (int i = w0; i < w0 + piece && i < nB; i += 32) n += __popc(__ballot_sync(0xffffffffu, keep(i + lane)));
  __syncthreads();
  if (lane == 0) sm.warp_cnt[warp] = n;
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < kRouteWarps; ++w) {
    if (w < warp) at += sm.warp_cnt[w];
    total += sm.warp_cnt[w];
  }
  for (int i = w0; i < w0 + piece && i < nB; i += 32) {
    const bool k = keep(i + lane);
    const unsigned mask = __ballot_sync(0xffffffffu, k);
    if (k) out[at + __popc(mask & ((1u << lane) - 1u))] = i + lane;
    at += __popc(mask);
  }
  for (int i = total + tid; i < c.max_blocks; i += kRouteThreads) out[i] = -1;
  if (tid == 0) n_kept[static_cast<int64_t>(b) * c.Hkv + h] = total;
}

// ---------------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------------
// Order-preserving pattern of a weight: larger weight, larger pattern; -0 as 0, NaN lowest.
constexpr uint32_t kZeroMass = 0x80000000u;
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (isnan(x)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A cluster of CTAs per (key head, sequence), each with a contiguous share of the tokens. The
// threshold among the middle tokens is found in three digits (11, 11, 10 bits) from the
// cluster-wide histograms; then the shares' counts place every share's kept tokens. The
// patterns stay in shared memory between the passes while a share fits (`hold` tokens); a
// thread takes four consecutive tokens at a time, since what bounds the passes is the number of
// instructions a token (250 thousand tokens, 8 key heads, 64 CTAs: 34 us; 16 sequences of 3 to 9
// thousand: 14). One further cluster a sequence (blockIdx.y = Hkv) marks the destination
// pages that are pages of the sequence itself.
constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kClashWords = kMaxCacheBlocks / 32;
constexpr uint32_t kAlways = ~0u;  // a token of either end, above every pattern; or none, behind the share

// Bit i of `clash`: destination i is one of the sequence's own pages. The pages' bits stand in
// `bits`, as many of them at a time as `words` hold.
template <typename T>
__device__ void mark_clashes(const CacheView<T>& c, int b, int nB, const int32_t* __restrict__ dst, int n_dst, uint32_t* bits,
                             int words, uint32_t* __restrict__ clash) {
  const int tid = threadIdx.x;
  for (int i = tid; i < (n_dst + 31) / 32; i += kEvictThreads) clash[i] = 0u;
  const int64_t most = static_cast<int64_t>(words) * 32;
  for (int64_t first = 0; first < c.n_pages; first += most) {
    const int n = static_cast<int>(min(most, c.n_pages - first));
    for (int i = tid; i < (n + 31) / 32; i += kEvictThreads) bits[i] = 0u;
    __syncthreads();
    for (int i = tid; i < nB; i += kEvictThreads) {
      const int64_t at = c.table[static_cast<int64_t>(b) * c.max_blocks + i] - first;
      if (at >= 0 && at < n) atomicOr(&bits[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    for (int i = tid; i < n_dst; i += kEvictThreads) {
      const int64_t at = dst[i] - first;
      if (at >= 0 && at < n && ((bits[at >> 5] >> (at & 31)) & 1u)) atomicOr(&clash[i >> 5], 1u << (i & 31));
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kEvictThreads)
    evict_select_kernel(CacheView<T> c, int keep, int n_sink, int n_recent, int hold, int words,
                        const int32_t* __restrict__ dst_table, int dst_blocks, uint32_t* __restrict__ clash,
                        int32_t* __restrict__ kept, int32_t* __restrict__ new_len, int32_t* dev_status) {
  extern __shared__ __align__(16) uint32_t held[];  // [words], hold of them for patterns
  __shared__ __align__(16) uint32_t bins[3][2048];  // of each pass
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, warp_n[3][kEvictWarps], warp_a[kEvictWarps], warp_e[kEvictWarps], mine[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * 2048 / 4; i += kEvictThreads)
    reinterpret_cast<uint4*>(&bins[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
  grid_wait();
  grid_release();
  const int len = seq_len(c, b, dev_status);
  if (h == c.Hkv) {
    if (rank > 0) return;
    if (tid == 0) new_len[b] = min(len, keep);
    mark_clashes(c, b, (len + kBlock - 1) / kBlock, dst_table + static_cast<int64_t>(b) * dst_blocks,
                 (min(len, keep) + kBlock - 1) / kBlock, held, words, clash + static_cast<int64_t>(b) * kClashWords);
    return;
  }
  int32_t* out = kept + (static_cast<int64_t>(b) * c.Hkv + h) * keep;
  if (len <= keep) {
    for (int i = rank * kEvictThreads + tid; i < keep; i += C * kEvictThreads) out[i] = i < len ? i : -1;
    return;
  }
  auto sync_all = [&] {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  // shares end on block borders, so a warp's loads lie in one page
  const int per = ((len + C - 1) / C + kBlock - 1) / kBlock * kBlock, t0 = min(rank * per, len), t1 = min(t0 + per, len);
  const bool fits = per <= hold;
  const int lo = n_sink, hi = min(len - n_recent, t1);  // the middle, as far as this share goes
  auto load_key = [&](int t) -> uint32_t {
    if (t < lo || t >= hi) return kAlways;
    const int page = page_of(c, b, t / kBlock, dev_status);
    return page < 0 ? 0u : mass_key(c.mass[(static_cast<int64_t>(page) * c.Hkv + h) * kBlock + t % kBlock]);
  };
  if (fits) {  // a warp takes whole pages, 16 on their way at a time
    const int nb = (t1 - t0 + kBlock - 1) / kBlock, b0 = t0 / kBlock;
    for (int base = warp; base < nb; base += 32 * kEvictWarps) {
      const int mine_at = base + lane * kEvictWarps;
      const int pages = mine_at < nb ? page_of(c, b, b0 + mine_at, dev_status) : -1;
      const int cnt = min(32, (nb - base + kEvictWarps - 1) / kEvictWarps);
      for (int k0 = 0; k0 < cnt; k0 += 16) {
        float2 x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int page = __shfl_sync(0xffffffffu, pages, min(k0 + k, cnt - 1));
          x[k] = page < 0 ? make_float2(NAN, NAN)
                          : reinterpret_cast<const float2*>(c.mass + (static_cast<int64_t>(page) * c.Hkv + h) * kBlock)[lane];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (k0 + k < cnt) {
            const int at = (base + (k0 + k) * kEvictWarps) * kBlock + 2 * lane, t = t0 + at;
            *reinterpret_cast<uint2*>(held + at) = make_uint2(t < lo || t >= hi ? kAlways : mass_key(x[k].x),
                                                              t + 1 < lo || t + 1 >= hi ? kAlways : mass_key(x[k].y));
          }
      }
    }
  }
  __syncthreads();
  // patterns of t .. t + 3 (t - t0 a multiple of 4, t < t1: the share's last block is held whole)
  auto four = [&](int t, uint32_t (&u)[4]) {
    if (fits) {
      const uint4 x = *reinterpret_cast<const uint4*>(held + (t - t0));
      u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = load_key(t + k);
    }
  };
  int need = keep - n_sink - n_recent;  // of the middle tokens so many stay
  const bool some = need > 0;
  uint32_t prefix = 0, same = 0;  // the digits found so far, and their bits
  int shift = 32;
  for (int pass = 0; pass < 3 && some; ++pass) {
    const int width = pass < 2 ? 11 : 10;
    shift -= width;
    uint32_t zeros = 0;  // tokens that were never attended to, often many: counted aside
    const uint32_t mask = (1u << width) - 1u;
#pragma unroll 2
    for (int t = t0 + 4 * tid; t < t1; t += 4 * kEvictThreads) {
      uint32_t u[4];
      four(t, u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (((u[k] ^ prefix) & same) != 0u || u[k] == kAlways) continue;
        if (u[k] == kZeroMass) ++zeros;
        else atomicAdd(&bins[pass][(u[k] >> shift) & mask], 1u);
      }
    }
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros) atomicAdd(&bins[pass][(kZeroMass >> shift) & mask], zeros);
    sync_all();
    // two bins a thread, from the highest down; every CTA finds the same one
    const int d0 = 2047 - 2 * tid;
    uint32_t n0 = 0, n1 = 0;
    if (C > 1) {
      uint2 x[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        x[r] = r < C ? *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&bins[pass][0], r) + d0 - 1) : make_uint2(0u, 0u);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        n1 += x[r].x;
        n0 += x[r].y;
      }
    } else {
      n1 = bins[pass][d0 - 1];
      n0 = bins[pass][d0];
    }
    int inc = static_cast<int>(n0 + n1);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_n[pass][warp] = inc;
    __syncthreads();
    const int before = inc - static_cast<int>(n0 + n1) + __reduce_add_sync(0xffffffffu, lane < warp ? warp_n[pass][lane] : 0);
    if (before < need && need <= before + static_cast<int>(n0 + n1)) {
      const bool first = need <= before + static_cast<int>(n0);
      s_prefix = prefix | (static_cast<uint32_t>(first ? d0 : d0 - 1) << shift);
      s_need = need - before - (first ? 0 : static_cast<int>(n0));
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    same |= mask << shift;
  }
  // patterns above the threshold and both ends stay, and the first `need` of the equal ones. A
  // warp takes a contiguous piece, a lane four tokens of each 128.
  const uint32_t border = some ? prefix : kAlways - 1u;  // (no token has the pattern kAlways - 1)
  const int piece = (per / kEvictWarps + 127) / 128 * 128, w0 = t0 + warp * piece, w1 = min(w0 + piece, t1);
  auto classify = [&](int t, unsigned& above, unsigned& equal) {  // a bit a token
    above = equal = 0u;
    if (t >= w1) return;
    uint32_t u[4];
    four(t, u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      above |= u[k] > border ? 1u << k : 0u;
      equal |= u[k] == border ? 1u << k : 0u;
    }
    if (t + 4 > w1) above &= (1u << (w1 - t)) - 1u;  // (behind the share: kAlways, never equal)
  };
  int na = 0, ne = 0;
  unsigned held_a = 0, held_e = 0;  // the bits of the first 1024 tokens of the piece
  for (int base = w0; base < w1; base += 128) {
    unsigned a, e;
    classify(base + 4 * lane, a, e);
    const int at = (base - w0) / 32;
    if (at < 32) {
      held_a |= a << at;
      held_e |= e << at;
    }
    na += __popc(a);
    ne += __popc(e);
  }
  na = __reduce_add_sync(0xffffffffu, na);
  ne = __reduce_add_sync(0xffffffffu, ne);
  if (lane == 0) {
    warp_a[warp] = na;
    warp_e[warp] = ne;
  }
  __syncthreads();
  if (warp == 0) {
    const int all_a = __reduce_add_sync(0xffffffffu, warp_a[lane]), all_e = __reduce_add_sync(0xffffffffu, warp_e[lane]);
    if (lane == 0) {
      mine[0] = all_a;
      mine[1] = all_e;
    }
  }
  if (C > 1) cluster.sync();
  int above = lane < warp ? warp_a[lane] : 0, equal = lane < warp ? warp_e[lane] : 0;
  if (lane < rank) {
    const int* theirs = cluster.map_shared_rank(mine, lane);
    above += theirs[0];
    equal += theirs[1];
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  for (int base = w0; base < w1; base += 128) {
    const int at = (base - w0) / 32, t = base + 4 * lane;
    unsigned a, e;
    if (at < 32) {
      a = (held_a >> at) & 15u;
      e = (held_e >> at) & 15u;
    } else {
      classify(t, a, e);
    }
    const int count = __popc(a) | (__popc(e) << 16);
    int inc = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int total = __shfl_sync(0xffffffffu, inc, 31), before = inc - count;
    int pa = above + (before & 0xffff), pe = equal + (before >> 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool is_a = (a >> k) & 1u, is_e = (e >> k) & 1u;
      if (is_a || (is_e && pe < need)) out[pa + min(pe, need)] = t + k;
      pa += is_a;
      pe += is_e;
    }
    above += total & 0xffff;
    equal += total >> 16;
  }
  if (C > 1) cluster.sync();  // nobody leaves while its counts are read
}

// One CTA per (destination block, key head, sequence): gathers its 64 kept tokens. What bounds it
// are the rows in flight, so a CTA holds little: the keys pass through registers, for their mean,
// the values through shared memory, and six CTAs fit an SM. (62500 of 250 thousand tokens, 8 key
// heads, d = 128: 91 us, 5.9 TB/s; with the values in registers too, four CTAs an SM, 95.)
template <typename T, int D>
__global__ void __launch_bounds__(kEvictCopyThreads, sizeof(T) == 2 ? 6 : 4)
    evict_copy_kernel(CacheView<T> c, int keep, const int32_t* __restrict__ dst_table, int dst_blocks,
                      const uint32_t* __restrict__ clash, const int32_t* __restrict__ kept, int32_t* dev_status) {
  using P = PageRows<T, D, kEvictCopyThreads>;
  __shared__ __align__(128) uint4 s_v[kBlock * P::kPieces];
  const int b = blockIdx.z, h = blockIdx.y, block = blockIdx.x;
  grid_wait();
  const int len = seq_len(c, b, nullptr);
  const int n = min(min(len, keep) - block * kBlock, kBlock);
  if (n <= 0) return;
  const int lane = threadIdx.x / P::kPieces, piece = threadIdx.x % P::kPieces;
  const int32_t* src_at = kept + (static_cast<int64_t>(b) * c.Hkv + h) * keep + block * kBlock;
  const int dst = dst_table[static_cast<int64_t>(b) * dst_blocks + block];
  const bool own = (clash[static_cast<int64_t>(b) * kClashWords + block / 32] >> (block % 32)) & 1u;
  uint4 k[P::kRows];
  float mass[P::kRows];
#pragma unroll
  for (int i = 0; i < P::kRows; ++i) {
    const int r = lane + i * P::kLanes;
    k[i] = make_uint4(0u, 0u, 0u, 0u);
    mass[i] = 0.0f;
    const int t = r < n ? src_at[r] : -1;
    const int page = t >= 0 ? page_of(c, b, t / kBlock, dev_status) : -1;
    const int64_t from = (static_cast<int64_t>(max(page, 0)) * c.Hkv + h) * kBlock + (t & (kBlock - 1));
    copy16(s_v + r * P::kPieces + piece, reinterpret_cast<const uint4*>(c.v + from * D) + piece, page >= 0);
    if (page >= 0) {
      k[i] = __ldcs(reinterpret_cast<const uint4*>(c.k + from * D) + piece);
      if (piece == 0) mass[i] = c.mass[from];
    }
  }
  if (own || dst < 0 || dst >= c.n_pages) {
    if (threadIdx.x == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  const int64_t to = (static_cast<int64_t>(dst) * c.Hkv + h) * kBlock;
#pragma unroll
  for (int i = 0; i < P::kRows; ++i) {
    const int r = lane + i * P::kLanes;
    if (r < n) {
      __stcs(reinterpret_cast<uint4*>(c.k + (to + r) * D) + piece, k[i]);
      if (piece == 0) c.mass[to + r] = mass[i];
    }
  }
  asm volatile("cp.async.wait_all;\n\tfence.proxy.async.shared::cta;" ::: "memory");
  write_mean<T, D, kEvictCopyThreads>(k, n, c.key_mean + (static_cast<int64_t>(dst) * c.Hkv + h) * D);  // (a barrier in it)
  if (threadIdx.x == kEvictCopyThreads - 1) bulk_store(c.v + to * D, s_v, n * D * static_cast<int>(sizeof(T)));
}

// ---------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------
// CTAs of a unit's cluster: doubled while the units leave SMs idle and every CTA keeps at
// least `least` items, up to 8 (clusters of 16 found too few places at a time: an earlier version of
// the eviction's selection, over 250 thousand tokens and 8 key heads, took 2.5 times as long with them).
static int cluster_size(int64_t units, int64_t items, int64_t least) {
  int n = 1;
  while (n < 8 && units * n * 2 <= 148 && items / (2 * n) >= least) n *= 2;
  return n;
}

template <typename... Params, typename... Args>
static cudaError_t launch_cluster(void (*kernel)(Params...), dim3 grid, int threads, int cluster, size_t smem,
                                  cudaStream_t st, const Args&... args) {
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_chained(kernel, grid, threads, cluster, smem, st, args...);
}

struct AppendCall {
  const fva_cache* c;
  const fva_seqs* s;
  const void *k_new, *v_new;
  int64_t n_tokens, stride;
  const int32_t* new_ptr;
  int max_new;
  int32_t* dev_status;
  cudaStream_t st;
  template <typename T, int D>
  cudaError_t operator()() const {
    // a sequence's new tokens touch at most this many blocks
    const dim3 grid(static_cast<unsigned>((max_new + kBlock - 2) / kBlock + 1), static_cast<unsigned>(c->Hkv),
                    static_cast<unsigned>(s->B));
    append_kernel<T, D><<<grid, kAppendThreads, 0, st>>>(cache_view<T>(c, s), static_cast<const T*>(k_new),
                                                       static_cast<const T*>(v_new), n_tokens, stride, new_ptr, max_new,
                                                       dev_status);
    return cudaGetLastError();
  }
};

cudaError_t launch_cache_append(const fva_cache* c, const fva_seqs* s, const void* k_new, const void* v_new,
                                int64_t n_tokens, int64_t stride, const int32_t* new_ptr, int max_new,
                                int32_t* dev_status, cudaStream_t st) {
  return by_cache_type(c, AppendCall{c, s, k_new, v_new, n_tokens, stride, new_ptr, max_new, dev_status, st});
}

struct RouteCall {
  const fva_cache* c;
  const fva_seqs* s;
  const void* q;
  int H;
  int64_t q_stride;
  double p, scale;
  int k_floor, n_recent;
  int32_t *kept, *n_kept;
  double* scores;
  int32_t* dev_status;
  cudaStream_t st;
  template <typename T, int D>
  cudaError_t operator()() const {
    const int C = cluster_size(static_cast<int64_t>(s->B) * c->Hkv, s->max_blocks, 64);
    // Two CTAs share an SM where there are many units. Clusters are made only where SMs are to
    // spare: their CTAs ask for more than half of an SM's shared memory, or pairs of them would
    // share one while others idle.
    const int per = (s->max_blocks + C - 1) / C, most = (C > 1 ? 170 : 60) * 1024 / 8;
    const int cap = s->max_blocks + kHeads * per <= most ? per : 0;
    size_t smem = static_cast<size_t>(s->max_blocks + kHeads * cap) * sizeof(double);
    if (C > 1 && smem < 116 * 1024) smem = 116 * 1024;
    return launch_cluster(route_kernel<T, D>,
                          dim3(static_cast<unsigned>(C), static_cast<unsigned>(c->Hkv), static_cast<unsigned>(s->B)),
                          kRouteThreads, C, smem, st, cache_view<T>(c, s), static_cast<const T*>(q), q_stride, H, scale, p,
                          k_floor, n_recent, cap, scores, kept, n_kept, dev_status);
  }
};

cudaError_t launch_cache_route(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride, double p,
                               int k_floor, int n_recent, double scale, int32_t* kept, int32_t* n_kept, double* scores,
                               int32_t* dev_status, cudaStream_t st) {
  return by_cache_type(c, RouteCall{c, s, q, H, q_stride, p, scale, k_floor, n_recent, kept, n_kept, scores, dev_status, st});
}

struct EvictCall {
  const fva_cache* c;
  const fva_seqs* s;
  int keep, n_sink, n_recent;
  const int32_t* dst_table;
  int dst_blocks;
  int32_t *kept, *new_len;
  uint32_t* clash;
  int32_t* dev_status;
  cudaStream_t st;
  template <typename T, int D>
  cudaError_t operator()() const {
    const CacheView<T> v = cache_view<T>(c, s);
    const unsigned Hkv = static_cast<unsigned>(c->Hkv), B = static_cast<unsigned>(s->B);
    const int tokens = s->max_blocks * kBlock, C = cluster_size(static_cast<int64_t>(B) * Hkv, tokens, 4096);
    const int per = ((tokens + C - 1) / C + kBlock - 1) / kBlock * kBlock, most = 200 * 1024 / 4;
    const int hold = per <= most ? per : 0, page_words = (c->n_pages - 1) / 32 + 1;
    const int words = std::max(hold, std::min(page_words, 16384));
    cudaError_t e = launch_cluster(evict_select_kernel<T>, dim3(static_cast<unsigned>(C), Hkv + 1, B), kEvictThreads, C,
                                   static_cast<size_t>(words) * 4, st, v, keep, n_sink, n_recent, hold, words, dst_table,
                                   dst_blocks, clash, kept, new_len, dev_status);
    if (e != cudaSuccess) return e;
    return launch_chained(evict_copy_kernel<T, D>, dim3(static_cast<unsigned>((keep + kBlock - 1) / kBlock), Hkv, B),
                          kEvictCopyThreads, 0, 0, st, v, keep, dst_table, dst_blocks, clash, kept, dev_status);
  }
};

cudaError_t launch_cache_evict(const fva_cache* c, const fva_seqs* s, int keep, int n_sink, int n_recent,
                               const int32_t* dst_table, int dst_blocks, int32_t* kept, int32_t* new_len,
                               uint32_t* clash, int32_t* dev_status, cudaStream_t st) {
  return by_cache_type(c, EvictCall{c, s, keep, n_sink, n_recent, dst_table, dst_blocks, kept, new_len, clash, dev_status, st});
}

size_t cache_evict_clash_words(int B) { return static_cast<size_t>(B) * kClashWords; }

}  // namespace fva
