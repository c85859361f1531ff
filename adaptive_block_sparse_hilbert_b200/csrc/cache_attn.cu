// Attention of single query tokens over kept blocks of a paged key/value cache.
//
// A unit is one (sequence, key head, group of up to 16 query heads). All units' kept blocks,
// laid end to end, are cut into equal shares, one per CTA, so a long sequence spreads over
// many SMs and short ones share one: the work is a read of the kept keys and values, and every
// SM reads the same amount. A unit inside one CTA's share is finished there; one that crosses
// shares leaves each share's unnormalised O with its running maximum and sum in the workspace,
// and a second kernel joins them in share order (a fixed order: equal inputs, equal bits) and
// accumulates the weights. Small calls have a cluster of CTAs per unit instead, a part of its list
// each, that joins through shared memory: the second launch then only accumulates, if at all.
#include <cooperative_groups.h>
#include <math.h>

#include "cache.cuh"

namespace fva {

namespace cg = cooperative_groups;

constexpr int kShares = 296;  // CTAs of the split kernels at most: two per SM
constexpr int kGroup = 16;    // query heads of a unit at most
constexpr int kMaxParts = 8;  // CTAs of a cluster at most
constexpr int kPartBlocks = 24;  // blocks that a CTA of a cluster takes at most

template <typename T>
struct AttnView {
  CacheView<T> c;
  const T* q;
  int64_t q_stride;
  const int32_t* kept;
  const int32_t* n_kept;
  int H, G, GS, units;  // G query heads per key head, GS units per (sequence, key head)
  float scale_log2;
  CacheAttnScratch ws;
  T* o;
  float* lse;
  int32_t* dev_status;
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

// Block of a unit's list entry; -1, reported, when it lies outside the sequence.
template <typename T>
__device__ __forceinline__ int unit_block(const AttnView<T>& a, int bh, int pos, int len, int32_t* dev_status) {
  if (!a.kept) return pos;
  const int block = a.kept[static_cast<int64_t>(bh) * a.c.max_blocks + pos];
  if (block >= 0 && static_cast<int64_t>(block) * kBlock < len) return block;
  report(dev_status, FVA_DEVERR_BAD_LIST);
  return -1;
}

struct Share {
  int64_t total, per;  // blocks of all units, blocks of a share
  int unit;            // unit that holds this share's first block
  int64_t unit_start;  // first block of that unit
};

// Every thread of the CTA calls this. Share 0 leaves `per` in the workspace.
template <typename T>
__device__ Share find_share(const AttnView<T>& a, int share) {
  __shared__ int64_t warp_sum[32];
  __shared__ Share found;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (a.units + nt - 1) / nt;
  const int u0 = min(tid * chunk, a.units), u1 = min(u0 + chunk, a.units);
  int64_t mine = 0;
  for (int u = u0; u < u1; ++u) mine += unit_count(a, u, a.dev_status);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = inc - mine, total = 0;
  for (int w = 0; w < (nt >> 5); ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
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
    if (share == 0) *a.ws.per = per;
  }
  __syncthreads();
  return found;
}

// A share's walk over its units: segment by segment, the same in every thread.
template <typename T>
struct Walk {
  int64_t at, end, start;  // next block, end of the share, first block of the unit
  int64_t first_at;
  int u, n;
  __device__ Walk(const Share& sh, int share) {
    first_at = at = share * sh.per;
    end = min(sh.total, at + sh.per);
    u = sh.unit - 1;
    start = sh.unit_start;
    n = 0;
  }
  // Moves to the next segment: unit u, blocks [at - start, stop() - start) of it.
  __device__ bool next(const AttnView<T>& a) {
    if (at >= end) return false;
    start += n;
    do {
      ++u;
      n = unit_count(a, u, nullptr);
    } while (n == 0);
    return true;
  }
  __device__ int64_t stop() const { return min(end, start + n); }
  __device__ bool whole() const { return at == start && stop() == start + n; }
  __device__ int slot() const { return at == first_at ? 0 : 1; }
};

// A cluster's walk: its one unit, this CTA's part of the list, which may be empty.
template <typename T>
struct PartWalk {
  int64_t at, end, start = 0;
  int u, n;
  bool taken = false;
  __device__ PartWalk(const AttnView<T>& a, int rank, int parts) {
    u = static_cast<int>(blockIdx.x) / parts;
    n = unit_count(a, u, a.dev_status);
    const int per = (n + parts - 1) / parts;
    at = min(rank * per, n);
    end = min(static_cast<int>(at) + per, n);
  }
  __device__ bool next(const AttnView<T>&) {
    const bool first = !taken;
    taken = true;
    return first;
  }
  __device__ int64_t stop() const { return end; }
};

template <typename T, bool kCluster>
__device__ __forceinline__ auto make_walk(const AttnView<T>& a) {
  if constexpr (kCluster) {
    cg::cluster_group cluster = cg::this_cluster();
    __syncthreads();  // publishes the mbarriers
    return PartWalk<T>(a, static_cast<int>(cluster.block_rank()), static_cast<int>(cluster.num_blocks()));
  } else {
    const Share sh = find_share(a, blockIdx.x);  // (its barriers publish the mbarriers too)
    return Walk<T>(sh, blockIdx.x);
  }
}

// The log-sum-exp of a finished row.
template <typename T>
__device__ __forceinline__ void put_lse(const AttnView<T>& a, int64_t row, float mx, float sum) {
  const float l2 = sum == 0.0f ? -INFINITY : mx + log2f(sum);
  if (a.lse) a.lse[row] = l2 * 0.6931471805599453f;
  if (a.ws.scores) a.ws.lse[row] = l2;
}

// Rows of a unit from its cluster's parts ([row][D + 2] in every CTA's `part`: unnormalised O,
// maximum, sum), in their order; a warp per row. Every thread of the CTA calls this.
template <typename T, int D>
__device__ void join_cluster(const AttnView<T>& a, int u, float* part) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), parts = static_cast<int>(cluster.num_blocks());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int bh = u / a.GS, b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
  const int g0 = (u - bh * a.GS) * kGroup, ng = min(a.G - g0, kGroup);
  cluster.sync();
  for (int r = rank + parts * warp; r < ng; r += parts * warps) {
    constexpr int V = D / 32;
    float m[kMaxParts], l[kMaxParts], x[kMaxParts][V];
#pragma unroll
    for (int c = 0; c < kMaxParts; ++c) {
      const float* from = c < parts ? cluster.map_shared_rank(part, c) + r * (D + 2) : nullptr;
      m[c] = from ? from[D] : -INFINITY;
      l[c] = from ? from[D + 1] : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) x[c][i] = from ? from[lane * V + i] : 0.0f;
    }
    float mx = -INFINITY, sum = 0.0f, acc[V];
#pragma unroll
    for (int c = 0; c < kMaxParts; ++c) mx = fmaxf(mx, m[c]);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < kMaxParts; ++c) {
      const float f = m[c] == -INFINITY ? 0.0f : exp2f(m[c] - mx);
      sum = fmaf(f, l[c], sum);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(f, x[c][i], acc[i]);
    }
    const int64_t row = static_cast<int64_t>(b) * a.H + h * a.G + g0 + r;
#pragma unroll
    for (int i = 0; i < V; ++i) from_f32(sum == 0.0f ? 0.0f : acc[i] / sum, a.o + row * D + lane * V + i);
    if (lane == 0) put_lse(a, row, mx, sum);
  }
  cluster.sync();  // nobody leaves while its part is read
}

struct SplitWaits {
  uint64_t limit_ns;
  uint32_t diag_flags;
};

// The loading warp of a split kernel: walks its share's lists and the page table 32 entries at
// a time and has `load(stage, page, head)` request the pages, as the ring's stages come free.
// `valid` of a stage: its keys that count, 0 for a page that is skipped.
template <typename T, typename W, typename Load>
__device__ __forceinline__ void feed_pages(const AttnView<T>& a, W& w, uint64_t* full, uint64_t* empty, int* valid_of,
                                           volatile int* abort_flag, const SplitWaits& waits, int stages,
                                           const Load& load) {
  if (waits.diag_flags & FVA_DIAG_WITHHOLD_Q) return;  // nothing ever arrives: the waits run out
  const int lane = threadIdx.x & 31;
  const bool leader = elect_one();
  int stage = 0, phase = 0, issued = 0;
  bool ok = true;
  while (ok && w.next(a)) {
    const int bh = w.u / a.GS, b = bh / a.c.Hkv, h = bh - b * a.c.Hkv, len = seq_len(a.c, b, nullptr);
    for (int64_t base = w.at; base < w.stop() && ok; base += 32) {
      const int cnt = static_cast<int>(min(static_cast<int64_t>(32), w.stop() - base));
      int page = -1, valid = 0;
      if (lane < cnt) {
        const int block = unit_block(a, bh, static_cast<int>(base - w.start) + lane, len, a.dev_status);
        if (block >= 0) page = page_of(a.c, b, block, a.dev_status);
        if (page >= 0) valid = min(len - block * kBlock, kBlock);
      }
      for (int k = 0; k < cnt; ++k) {
        const int pg = __shfl_sync(0xffffffffu, page, k), va = __shfl_sync(0xffffffffu, valid, k);
        if (!warp_wait_spin(&empty[stage], phase ^ 1, abort_flag, waits.limit_ns)) {
          ok = false;
          break;
        }
        if (leader) {
          valid_of[stage] = va;
          if (pg >= 0) load(stage, pg, h);
          else mbar_arrive(&full[stage]);
        }
        ++issued;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    w.at = w.stop();
  }
  if (!ok) {
    report(a.dev_status, FVA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  }
  __syncwarp();
  // wait (bounded) for the loads in flight: a CTA that gives up must not leave them behind
  volatile int never = 0;
  for (int j = issued > stages ? issued - stages : 0; j < issued; ++j)
    mbar_wait(&full[j % stages], (j / stages) & 1, &never, 100000000ull);
}

// ---------------------------------------------------------------------------------
// 16-bit caches
// ---------------------------------------------------------------------------------
// Four warps take 16 keys each of every block, with softmax statistics and an O of their own
// (joined at a unit's end); a fifth walks the lists and page table and keeps TMA loads of whole
// pages in flight. The reads bound it, so the products are the small mma.sync ones (16 query
// heads x 8 keys), whose operands stay in registers between the two products, and a weight is
// kept in two 16-bit parts (its head and the rest, 2^-16 of it or less is lost), which costs
// tensor time that the loads hide. (32 sequences of 2 to 9 thousand tokens, a quarter of the
// blocks kept, 32 query on 8 key heads, d = 128: 33 us, about 23 of it at the copy rate.)
template <int D>
struct SplitCfg {
  static constexpr int kTile = kBlock * D * 2;  // K or V of one page and key head
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kSmem = 1024 + kStages * 2 * kTile;
};
constexpr int kSplitThreads = 160;

template <typename T>
struct Frag;
template <>
struct Frag<__nv_bfloat16> {
  static constexpr float kLift = 0.0f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Frag<__half> {
  // fp16 weights are held 2^14 times as large: the small ones of a long list stay out of the
  // subnormal range's coarse steps
  static constexpr float kLift = 14.0f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Byte offset of 16-byte piece `piece` of row `row` in a page tile as TMA lays it down: chunks
// of 64 channels, rows of 128 bytes, pieces swizzled by the row.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return static_cast<uint32_t>((piece >> 3) * (kBlock * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

template <typename T, int D, bool kCluster>
__global__ void __launch_bounds__(kSplitThreads, 2)
    split_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, AttnView<T> a,
                 SplitWaits waits) {
  using Cfg = SplitCfg<D>;
  using F = Frag<T>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float2 s_o[2][8][D / 2 + 4];  // (the padding spreads the rows over the banks)
  __shared__ float s_m[4][kGroup], s_l[4][kGroup];
  __shared__ uint64_t full[Cfg::kStages], empty[Cfg::kStages];
  __shared__ int s_valid[Cfg::kStages], s_abort;
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int share = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  grid_wait();
  grid_release();
  auto w = make_walk<T, kCluster>(a);
  const int unit = w.u;
  volatile int* abort_flag = &s_abort;
  if (warp == 4) {
    feed_pages(a, w, full, empty, s_valid, abort_flag, waits, Cfg::kStages, [&](int stage, int page, int h) {
      uint8_t* dst = ring + stage * 2 * Cfg::kTile;
      mbar_arrive_expect_tx(&full[stage], 2 * Cfg::kTile);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        tma_load_3d(dst + c * (kBlock * 128), &tmk, &full[stage], c * 64, h * kBlock, page);
        tma_load_3d(dst + Cfg::kTile + c * (kBlock * 128), &tmv, &full[stage], c * 64, h * kBlock, page);
      }
    });
    if constexpr (kCluster) join_cluster<T, D>(a, unit, reinterpret_cast<float*>(ring));
    return;
  }

  // -------------------------------------------------------------------- products and softmax
  // A warp whose wait runs out takes no further data but goes through its units' joins: the
  // four warps meet at barriers there.
  bool ok = true;
  int stage = 0, phase = 0;
  const int rg = lane >> 2, ct = lane & 3;  // fragment rows rg, rg + 8; columns 2 ct, 2 ct + 1
  const int lm = lane >> 3, lr = lane & 7;  // ldmatrix: matrix and row of this lane's address
  while (w.next(a)) {
    const int bh = w.u / a.GS, b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
    const int g0 = (w.u - bh * a.GS) * kGroup, ng = min(a.G - g0, kGroup);
    const int64_t row0 = static_cast<int64_t>(b) * a.H + h * a.G + g0;
    uint32_t qa[D / 16][4];
    {
      const T* q = a.q + b * a.q_stride + static_cast<int64_t>(h * a.G + g0) * D;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = rg + (i & 1) * 8, ch = kk * 16 + ct * 2 + (i >> 1) * 8;
          qa[kk][i] = r < ng ? *reinterpret_cast<const uint32_t*>(q + r * D + ch) : 0u;
        }
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int64_t stop = w.stop();
    const int first_pos = static_cast<int>(w.at - w.start), n_pos = static_cast<int>(stop - w.at);
    for (int j = 0; j < n_pos; ++j) {
      ok = ok && warp_wait_spin(&full[stage], phase, abort_flag, waits.limit_ns);
      if (!ok) {
        *abort_flag = 1;
        break;
      }
      const int nk = s_valid[stage] - warp * 16;  // this warp's keys that count
      const uint32_t sk = smem_u32(ring + stage * 2 * Cfg::kTile), sv = sk + Cfg::kTile;
      float s[2][4], s1[2][4];  // sums over the even and the odd steps: two chains of products
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = s1[n][i] = 0.0f;
      if (nk > 0) {
        if (nk < 16) {  // values behind the sequence's end may be NaN, and 0 NaN is NaN: clear them
          for (int i = lane; i < (16 - nk) * (D / 8); i += 32) {
            const int r = warp * 16 + nk + i / (D / 8);
            *reinterpret_cast<uint4*>(ring + stage * 2 * Cfg::kTile + Cfg::kTile + tile_at(r, i % (D / 8))) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t kb[4];
          ldmatrix4(kb, sk + tile_at(warp * 16 + (lm >> 1) * 8 + lr, kk * 2 + (lm & 1)));
          F::mma(kk & 1 ? s1[0] : s[0], qa[kk], kb[0], kb[1]);
          F::mma(kk & 1 ? s1[1] : s[1], qa[kk], kb[2], kb[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = n * 8 + ct * 2 + (i & 1);
          s[n][i] = key < nk ? (s[n][i] + s1[n][i]) * a.scale_log2 : -INFINITY;
        }
      if (a.ws.scores) {  // kept for the accumulation: -inf behind the last key
        float* out = a.ws.scores + row0 * a.c.max_blocks * kBlock + static_cast<int64_t>(first_pos + j) * kBlock + warp * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (rg + i * 8 < ng)
#pragma unroll
            for (int n = 0; n < 2; ++n)
              *reinterpret_cast<float2*>(out + static_cast<int64_t>(rg + i * 8) * a.c.max_blocks * kBlock + n * 8 + ct * 2) =
                  make_float2(s[n][2 * i], s[n][2 * i + 1]);
      }
      if (nk > 0) {
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // fragment rows rg and rg + 8
          float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float m_new = fmaxf(m[i], mx);
          if (__any_sync(0xffffffffu, m_new > m[i])) {
            const float f = m[i] == -INFINITY ? 0.0f : exp2f(m[i] - m_new);
            l[i] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * i] *= f;
              o[n][2 * i + 1] *= f;
            }
          }
          m[i] = m_new;
          const float ref = m_new == -INFINITY ? 0.0f : m_new - F::kLift;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = exp2f(s[n][2 * i] - ref), p1 = exp2f(s[n][2 * i + 1] - ref);
            l[i] += p0 + p1;
            const uint32_t hi = F::pack(p0, p1);
            const float2 x = F::unpack(hi);
            ph[n * 2 + i] = hi;
            pl[n * 2 + i] = F::pack(p0 - x.x, p1 - x.y);
          }
        }
#pragma unroll
        for (int n0 = 0; n0 < D / 16; n0 += 2) {  // two pieces at a time: a product between dependent ones
          uint32_t vb[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            ldmatrix4_trans(vb[k], sv + tile_at(warp * 16 + (lm & 1) * 8 + lr, (n0 + k) * 2 + (lm >> 1)));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            F::mma(o[2 * (n0 + k)], ph, vb[k][0], vb[k][1]);
            F::mma(o[2 * (n0 + k) + 1], ph, vb[k][2], vb[k][3]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            F::mma(o[2 * (n0 + k)], pl, vb[k][0], vb[k][1]);
            F::mma(o[2 * (n0 + k) + 1], pl, vb[k][2], vb[k][3]);
          }
        }
        if (nk < 16) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the next load overwrites them
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == Cfg::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // ---- join the four warps: 2 and 3 hand over to 0 and 1, then 1 to 0, eight rows at a time
    auto sync4 = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[i];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (ct == 0) {
        s_m[warp][rg + i * 8] = m[i] - F::kLift;
        s_l[warp][rg + i * 8] = sum;
      }
    }
    sync4();
    bool whole = false;  // finished here; else the sums go to `parts`, rows of D + 2
    float* parts = reinterpret_cast<float*>(ring);
    if constexpr (!kCluster) {
      whole = w.whole();
      parts = a.ws.part + (static_cast<int64_t>(share) * 2 + w.slot()) * kGroup * (D + 2);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // fragment rows rg, then rg + 8
      if (i * 8 >= ng) break;
      const int r = rg + i * 8;
      const float mx = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
      const float f = m[i] == -INFINITY ? 0.0f : exp2f(s_m[warp][r] - mx);
#pragma unroll
      for (int step = 2; step > 0; step >>= 1) {
        if (warp >= step && warp < 2 * step) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            s_o[warp - step][rg][n * 4 + ct] = step == 2 ? make_float2(o[n][2 * i] * f, o[n][2 * i + 1] * f)
                                                         : make_float2(o[n][2 * i], o[n][2 * i + 1]);
        }
        sync4();
        if (warp < step) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const float2 x = s_o[warp][rg][n * 4 + ct];
            o[n][2 * i] = (step == 2 ? o[n][2 * i] * f : o[n][2 * i]) + x.x;
            o[n][2 * i + 1] = (step == 2 ? o[n][2 * i + 1] * f : o[n][2 * i + 1]) + x.y;
          }
        }
        if (step == 2) sync4();
      }
      if (warp == 0 && r < ng) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) sum += s_l[v][r] * (s_m[v][r] == -INFINITY ? 0.0f : exp2f(s_m[v][r] - mx));
        const int64_t row = row0 + r;
        if (whole) {
          const float inv = 1.0f / sum;  // (a row without weight is 0 even where 0 times its values is NaN)
          uint32_t* out = reinterpret_cast<uint32_t*>(a.o + row * D);
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            out[n * 4 + ct] = sum == 0.0f ? 0u : F::pack(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
        } else {
          float2* part = reinterpret_cast<float2*>(parts + r * (D + 2));
#pragma unroll
          for (int n = 0; n < D / 8; ++n) part[n * 4 + ct] = make_float2(o[n][2 * i], o[n][2 * i + 1]);
        }
        if (ct == 0 && whole) put_lse(a, row, mx, sum);
        if (ct == 0 && !whole) parts[r * (D + 2) + D] = mx, parts[r * (D + 2) + D + 1] = sum;
      }
      sync4();  // the buffers are rewritten by the next rows, s_m and s_l by the next unit
    }
    if (!kCluster && tid == 0) a.ws.start[w.u] = w.start;
    w.at = stop;
  }
  if (!ok) report(a.dev_status, FVA_DEVERR_TIMEOUT);
  if constexpr (kCluster) join_cluster<T, D>(a, unit, reinterpret_cast<float*>(ring));
}

// ---------------------------------------------------------------------------------
// fp32 caches
// ---------------------------------------------------------------------------------
// CUDA cores, the same division of work: four warps with 16 keys each of every block, a fifth
// that keeps bulk loads of whole pages in flight. Scores: two lanes a key, half of the channels
// each, in an order rotated by the key so that the lanes' 16-byte reads of a page's rows fall
// into different banks; the query sits in shared memory. Values: lanes hold D / 32 channels. (8
// sequences of 500 to 2900 tokens, 12 heads, d = 64: 14 us, launch and lists included.)
// Sums are short: a score's error is a relative one of its weight, and one chain of D / 2 products
// made it the larger part of the result's (9 sequences of 6 to 19 thousand tokens, d = 128, 8 heads: 1.3e-6 of
// the outputs' norm; in two chains 7.8e-7, in four 5.9e-7). Four cost nothing up to 4 heads, but 3.5
// of 43.5 us at 8 heads and d = 64, where two cost nothing (1 of 50 us at d = 128) and leave 5.9e-7 (four
// 5.3e-7). Values are added four keys at a time (lists of 20 thousand tokens in one CTA: 5.6e-7 in place of 1.1e-6).
template <int D>
struct SplitF32Cfg {
  static constexpr int kTile = kBlock * D * 4;
  static constexpr int kStages = D == 32 ? 6 : 3;
  static constexpr int kSmem = 128 + kStages * 2 * kTile;
  static constexpr int kUseShares = D == 128 ? kShares / 2 : kShares;  // CTAs that are resident at once
};

template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[V]) {
  if constexpr (V == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
  } else if constexpr (V == 2) {
    const float2 t = *reinterpret_cast<const float2*>(p);
    x[0] = t.x, x[1] = t.y;
  } else {
    x[0] = p[0];
  }
}

template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[V]) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else if constexpr (V == 2) *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  else p[0] = x[0];
}

template <int D, int G, bool kCluster>
__global__ void __launch_bounds__(kSplitThreads) split_f32_kernel(AttnView<float> a, SplitWaits waits) {
  using Cfg = SplitF32Cfg<D>;
  constexpr int V = D / 32, kHalf = D / 8;  // kHalf: 16-byte pieces of half a row
  constexpr int kChains = G > 4 ? 2 : 4;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) float s_q[G][D];
  __shared__ __align__(16) float s_p[4][G][16];
  __shared__ __align__(16) float s_o[2][G][D];
  __shared__ float s_m[4][G], s_l[4][G];
  __shared__ uint64_t full[Cfg::kStages], empty[Cfg::kStages];
  __shared__ int s_valid[Cfg::kStages], s_abort;
  uint8_t* ring = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  const int share = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  grid_wait();
  grid_release();
  auto w = make_walk<float, kCluster>(a);
  const int unit = w.u;
  volatile int* abort_flag = &s_abort;
  if (warp == 4) {
    feed_pages(a, w, full, empty, s_valid, abort_flag, waits, Cfg::kStages, [&](int stage, int page, int h) {
      const int64_t at = (static_cast<int64_t>(page) * a.c.Hkv + h) * kBlock * D;
      mbar_arrive_expect_tx(&full[stage], 2 * Cfg::kTile);
      bulk_load(ring + stage * 2 * Cfg::kTile, a.c.k + at, Cfg::kTile, &full[stage]);
      bulk_load(ring + stage * 2 * Cfg::kTile + Cfg::kTile, a.c.v + at, Cfg::kTile, &full[stage]);
    });
    if constexpr (kCluster) join_cluster<float, D>(a, unit, reinterpret_cast<float*>(ring));
    return;
  }

  bool ok = true;  // (a warp whose wait runs out still meets the others at the joins' barriers)
  int stage = 0, phase = 0;
  const int key = lane & 15, part = lane >> 4;
  auto sync4 = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
  while (w.next(a)) {
    const int bh = w.u / a.GS, b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
    const int g0 = (w.u - bh * a.GS) * kGroup, ng = min(a.G - g0, kGroup);
    const int64_t row0 = static_cast<int64_t>(b) * a.H + h * a.G + g0;
    for (int i = tid; i < G * D; i += 128)
      s_q[i / D][i % D] = i / D < ng ? a.q[b * a.q_stride + static_cast<int64_t>(h * a.G + g0) * D + i] * a.scale_log2 : 0.0f;
    sync4();
    float acc[G][V], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[g][i] = 0.0f;
    }
    const int64_t stop = w.stop();
    const int first_pos = static_cast<int>(w.at - w.start), n_pos = static_cast<int>(stop - w.at);
    for (int j = 0; j < n_pos; ++j) {
      ok = ok && warp_wait_spin(&full[stage], phase, abort_flag, waits.limit_ns);
      if (!ok) {
        *abort_flag = 1;
        break;
      }
      const int nk = min(s_valid[stage] - warp * 16, 16);  // this warp's keys that count
      const float* tk = reinterpret_cast<const float*>(ring + stage * 2 * Cfg::kTile) + warp * 16 * D;
      const float* tv = tk + kBlock * D;
      float s[G], sc[G][kChains];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < kChains; ++i) sc[g][i] = 0.0f;
      if (nk > 0) {
#pragma unroll 4
        for (int c = 0; c < kHalf; ++c) {
          const int at = 4 * (part * kHalf + ((c + key) & (kHalf - 1)));
          const float4 k = *reinterpret_cast<const float4*>(tk + key * D + at);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float4 q = *reinterpret_cast<const float4*>(&s_q[g][at]);
            sc[g][0] = fmaf(q.x, k.x, sc[g][0]);
            sc[g][1] = fmaf(q.y, k.y, sc[g][1]);
            sc[g][2 % kChains] = fmaf(q.z, k.z, sc[g][2 % kChains]);
            sc[g][3 % kChains] = fmaf(q.w, k.w, sc[g][3 % kChains]);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        s[g] = kChains == 4 ? (sc[g][0] + sc[g][1]) + (sc[g][2] + sc[g][3]) : sc[g][0] + sc[g][1];
        s[g] += __shfl_xor_sync(0xffffffffu, s[g], 16);
        if (key >= nk) s[g] = -INFINITY;  // also what lies behind the sequence's end, NaN included
      }
      if (a.ws.scores && part == 0) {  // kept for the accumulation
        float* out = a.ws.scores + row0 * a.c.max_blocks * kBlock + static_cast<int64_t>(first_pos + j) * kBlock + warp * 16 + key;
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (g < ng) out[static_cast<int64_t>(g) * a.c.max_blocks * kBlock] = s[g];
      }
      if (nk > 0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float mx = s[g];
#pragma unroll
          for (int k = 8; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
          const float m_new = fmaxf(m[g], mx);
          const float corr = m_new == -INFINITY ? 1.0f : exp2f(m[g] - m_new);
          const float p = exp2f(s[g] - (m_new == -INFINITY ? 0.0f : m_new));
          m[g] = m_new;
          l[g] = l[g] * corr + (part == 0 ? p : 0.0f);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[g][i] *= corr;
          if (part == 0) s_p[warp][g][key] = p;
        }
        __syncwarp();
        const int groups = (nk + 3) / 4;
        for (int r4 = 0; r4 < groups; ++r4) {
          float v[4][V];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            load_vec<V>(tv + (4 * r4 + r) * D + lane * V, v[r]);
            if (4 * r4 + r >= nk) {  // 0 times what lies behind the end may be NaN
#pragma unroll
              for (int i = 0; i < V; ++i) v[r][i] = 0.0f;
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float4 p = *reinterpret_cast<const float4*>(&s_p[warp][g][4 * r4]);
#pragma unroll
            for (int i = 0; i < V; ++i)
              acc[g][i] += fmaf(p.x, v[0][i], fmaf(p.y, v[1][i], fmaf(p.z, v[2][i], p.w * v[3][i])));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == Cfg::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // ---- join the four warps: 2 and 3 hand over to 0 and 1, then 1 to 0
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = l[g];
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      if (lane == 0) {
        s_m[warp][g] = m[g];
        s_l[warp][g] = sum;
      }
    }
    sync4();
    bool whole = false;  // finished here; else the sums go to `parts`, rows of D + 2
    float* parts = reinterpret_cast<float*>(ring);
    if constexpr (!kCluster) {
      whole = w.whole();
      parts = a.ws.part + (static_cast<int64_t>(share) * 2 + w.slot()) * kGroup * (D + 2);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float mx = fmaxf(fmaxf(s_m[0][g], s_m[1][g]), fmaxf(s_m[2][g], s_m[3][g]));
      const float f = m[g] == -INFINITY ? 0.0f : exp2f(m[g] - mx);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[g][i] *= f;
      m[g] = mx;
    }
#pragma unroll
    for (int step = 2; step > 0; step >>= 1) {
      if (warp >= step && warp < 2 * step) {
#pragma unroll
        for (int g = 0; g < G; ++g) store_vec<V>(&s_o[warp - step][g][lane * V], acc[g]);
      }
      sync4();
      if (warp < step) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float x[V];
          load_vec<V>(&s_o[warp][g][lane * V], x);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[g][i] += x[i];
        }
      }
      if (step == 2) sync4();
    }
    if (warp == 0) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (g >= ng) continue;
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) sum += s_l[v][g] * (s_m[v][g] == -INFINITY ? 0.0f : exp2f(s_m[v][g] - m[g]));
        const float inv = 1.0f / sum;  // (a row without weight is 0 even where 0 times its values is NaN)
        float* out = whole ? a.o + (row0 + g) * D : parts + g * (D + 2);
#pragma unroll
        for (int i = 0; i < V; ++i) out[lane * V + i] = !whole ? acc[g][i] : sum == 0.0f ? 0.0f : acc[g][i] * inv;
        if (lane == 0 && whole) put_lse(a, row0 + g, m[g], sum);
        if (lane == 0 && !whole) out[D] = m[g], out[D + 1] = sum;
      }
    }
    if (!kCluster && tid == 0) a.ws.start[w.u] = w.start;
    sync4();  // the next unit rewrites what was read here
    w.at = stop;
  }
  if (!ok) report(a.dev_status, FVA_DEVERR_TIMEOUT);
  if constexpr (kCluster) join_cluster<float, D>(a, unit, reinterpret_cast<float*>(ring));
}

// ---------------------------------------------------------------------------------
// Join and accumulation
// ---------------------------------------------------------------------------------
// CTA (x, key head, sequence), 0 < x: forms the heads' log-sum-exp from the shares' maxima and
// sums and adds exp(s - lse), summed over the heads, to the masses of pieces x - 1, x - 1 + (the
// grid's x less one), .. of 16 listed blocks. x = 0 joins the shares' O, a warp per head. Little
// is moved: what such a CTA takes is its chain of dependent loads. `joined`: the clusters of the
// split kernel have finished every row. (32 sequences of 2 to 9 thousand tokens: 12 us.)
constexpr int kJoinThreads = 256, kMassBlocks = 16;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnView<T> a, bool joined) {
  __shared__ float s_lse[kMaxCacheGroup];
  __shared__ int s_page[kMassBlocks], s_valid[kMassBlocks];
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = b * a.c.Hkv + h;
  const bool joins = blockIdx.x == 0;
  grid_wait();
  grid_release();
  const int len = seq_len(a.c, b, nullptr), n = unit_count(a, bh * a.GS, nullptr);
  const int first = joins ? 0 : (blockIdx.x - 1) * kMassBlocks;
  if (joins ? joined : first >= n) return;
  auto find_pages = [&](int pos0) {
    if (tid < kMassBlocks) {
      const int pos = pos0 + tid;
      int page = -1, valid = 0;
      if (pos < n) {
        const int block = unit_block(a, bh, pos, len, nullptr);
        if (block >= 0) page = page_of(a.c, b, block, nullptr);
        if (page >= 0) valid = min(len - block * kBlock, kBlock);
      }
      s_page[tid] = page;
      s_valid[tid] = valid;
    }
  };
  if (!joins) find_pages(first);
  // A head without a finite score weighs nothing: exp2(-inf - inf) is 0, -inf - -inf is NaN.
  auto weightless = [](float l2) { return l2 == -INFINITY ? INFINITY : l2; };
  const int64_t per = n && !joined ? *a.ws.per : 1;
  for (int g = warp; g < a.G; g += kJoinThreads / 32) {
    const int64_t row = static_cast<int64_t>(b) * a.H + h * a.G + g;
    if (joined) {
      if (lane == 0) s_lse[g] = weightless(a.ws.lse[row]);
      continue;
    }
    const int64_t start = n ? a.ws.start[bh * a.GS + g / kGroup] : 0;
    const int c0 = static_cast<int>(start / per), c1 = n ? static_cast<int>((start + n - 1) / per) : c0;
    if (c0 < 0 || c1 < c0 || c1 >= kShares) continue;  // (never: whatever the workspace holds, no access leaves it)
    if (n && c0 == c1) {  // finished by the split kernel
      if (!joins && lane == 0) s_lse[g] = weightless(a.ws.lse[row]);
      continue;
    }
    constexpr int V = D / 32;
    float mx = -INFINITY, sum = 0.0f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int s0 = c0; n && s0 <= c1; s0 += 32) {  // 32 shares at a time, a lane each
      const int s = s0 + lane;
      auto part_of = [&](int share) -> const float* {
        const int slot = share * per >= start ? 0 : 1;
        return a.ws.part + ((static_cast<int64_t>(share) * 2 + slot) * kGroup + g % kGroup) * (D + 2);
      };
      const float m = s <= c1 ? part_of(s)[D] : -INFINITY, l = s <= c1 ? part_of(s)[D + 1] : 0.0f;
      float m_new = fmaxf(mx, m);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, k));
      const float f0 = mx == -INFINITY ? 0.0f : exp2f(mx - m_new), f = m == -INFINITY ? 0.0f : exp2f(m - m_new);
      float t = l * f;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
      sum = sum * f0 + t;
      mx = m_new;
      if (joins) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= f0;
        const int cnt = min(32, c1 - s0 + 1);
        for (int k0 = 0; k0 < cnt; k0 += 8) {  // eight shares' rows on their way at a time
          float x[8][V];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float* from = part_of(s0 + min(k0 + k, cnt - 1)) + lane * V;
#pragma unroll
            for (int i = 0; i < V; ++i) x[k][i] = from[i];
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = k0 + k < cnt ? fmaf(fk, x[k][i], acc[i]) : acc[i];
          }
        }
      }
    }
    // (a row without keys has a sum of 0; a NaN in its scores makes the sum one)
    const float l2 = sum == 0.0f ? -INFINITY : mx + log2f(sum);
    if (joins) {
#pragma unroll
      for (int i = 0; i < V; ++i) from_f32(sum == 0.0f ? 0.0f : acc[i] / sum, a.o + row * D + lane * V + i);
      if (lane == 0 && a.lse) a.lse[row] = l2 * 0.6931471805599453f;
    } else if (lane == 0) {
      s_lse[g] = weightless(l2);
    }
  }
  if (joins) return;
  const int64_t head_stride = static_cast<int64_t>(a.c.max_blocks) * kBlock;
  for (int pos0 = first; pos0 < n;) {
    __syncthreads();  // s_lse and the pages are there
    // scores behind a sequence's end and of skipped pages are -inf; entries behind the list's
    // end were not written
    const float* s = a.ws.scores + (static_cast<int64_t>(b) * a.H + h * a.G) * head_stride + static_cast<int64_t>(pos0) * kBlock;
    constexpr int kPer = kMassBlocks * kBlock / kJoinThreads;
    float w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = 0.0f;
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int k = tid + i * kJoinThreads;
        const float x = k % kBlock < s_valid[k / kBlock] ? s[g * head_stride + k] : -INFINITY;
        w[i] += exp2f(x - s_lse[g]);
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int k = tid + i * kJoinThreads, j = k / kBlock;
      if (k % kBlock < s_valid[j])
        atomicAdd(a.c.mass + (static_cast<int64_t>(s_page[j]) * a.c.Hkv + h) * kBlock + k % kBlock, w[i]);
    }
    pos0 += (gridDim.x - 1) * kMassBlocks;
    __syncthreads();  // the pages are rewritten
    find_pages(pos0);
  }
}

// ---------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------
size_t cache_attn_part_floats(int d) { return static_cast<size_t>(kShares) * 2 * kGroup * (d + 2); }

// 3-D map over a cache's [n_pages, Hkv * 64, d] 16-bit tensor, box = 64 channels x 64 rows.
static bool make_page_map(CUtensorMap* map, const void* base, const fva_cache* c) {
  return make_rows_map(map, base, c->n_pages, static_cast<int64_t>(c->Hkv) * kBlock, c->d, c->dtype == FVA_F16);
}

// CTAs of a unit's cluster, or 0: shares and a second launch. A cluster saves the launch and the
// trip through global memory, but leaves CTAs unused where there are few units and balances
// nothing between them. Routing and attention of one sequence (bf16, d = 128, 8 key heads of 4
// query heads, all blocks kept) take, with clusters / shares, 28 / 29 us at 119 blocks, 35 / 36 at
// 172, 42 / 39 at 235; of 8 sequences (fp32, d = 64, 12 heads, all kept) 25 / 30 us at 24 blocks,
// 37 / 42 at 47.
static int cluster_parts(int units, int max_blocks, int resident) {
  int parts = 1;
  while (parts < kMaxParts && units * parts * 2 <= resident) parts *= 2;
  return units * parts <= resident && (max_blocks + parts - 1) / parts <= kPartBlocks ? parts : 0;
}

template <typename... Params, typename... Args>
static cudaError_t launch_split_grid(void (*kernel)(Params...), int grid, int parts, size_t smem, cudaStream_t st,
                                     const Args&... args) {
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_chained(kernel, dim3(static_cast<unsigned>(grid)), kSplitThreads, parts, smem, st, args...);
}

template <int D, int G>
static cudaError_t launch_f32(const AttnView<float>& a, int parts, cudaStream_t st) {
  using Cfg = SplitF32Cfg<D>;
  return launch_split_grid(parts ? split_f32_kernel<D, G, true> : split_f32_kernel<D, G, false>,
                           parts ? a.units * parts : Cfg::kUseShares, parts, Cfg::kSmem, st, a,
                           SplitWaits{attn_wait_limit_ns(), attn_diag_flags()});
}

// parts: of a cluster per unit; 0: shares.
template <typename T, int D>
static cudaError_t launch_split(const fva_cache* c, const AttnView<T>& a, int parts, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    CUtensorMap mk, mv;
    if (!make_page_map(&mk, c->k, c) || !make_page_map(&mv, c->v, c)) return cudaErrorInvalidValue;
    return launch_split_grid(parts ? split_kernel<T, D, true> : split_kernel<T, D, false>, parts ? a.units * parts : kShares,
                             parts, SplitCfg<D>::kSmem, st, mk, mv, a, SplitWaits{attn_wait_limit_ns(), attn_diag_flags()});
  } else {
    const int g = a.G < kGroup ? a.G : kGroup;
    return g <= 1   ? launch_f32<D, 1>(a, parts, st)
           : g <= 2 ? launch_f32<D, 2>(a, parts, st)
           : g <= 4 ? launch_f32<D, 4>(a, parts, st)
           : g <= 8 ? launch_f32<D, 8>(a, parts, st)
                    : launch_f32<D, 16>(a, parts, st);
  }
}

struct AttnCall {
  const fva_cache* c;
  const fva_seqs* s;
  const void* q;
  int H;
  int64_t q_stride;
  const int32_t *kept, *n_kept;
  void* o;
  float* lse;
  float scale;
  int accumulate;
  CacheAttnScratch ws;
  int32_t* dev_status;
  cudaStream_t st;
  template <typename T, int D>
  cudaError_t operator()() const {
    const int G = H / c->Hkv, GS = (G + kGroup - 1) / kGroup;
    const AttnView<T> a = {cache_view<T>(c, s), static_cast<const T*>(q), q_stride, kept, n_kept, H, G, GS,
                           s->B * c->Hkv * GS, scale * 1.4426950408889634f, ws, static_cast<T*>(o), lse, dev_status};
    const int resident = sizeof(T) == 4 && D == 128 ? kShares / 2 : kShares;
    const int parts = cluster_parts(a.units, s->max_blocks, resident);
    const cudaError_t e = launch_split<T, D>(c, a, parts, st);
    if (e != cudaSuccess || (parts && !accumulate)) return e;
    // pieces of the accumulation: about eight CTAs an SM, were every list of full length
    unsigned chunks = 0;
    if (accumulate) {
      const int64_t units = static_cast<int64_t>(s->B) * c->Hkv, pieces = (s->max_blocks + kMassBlocks - 1) / kMassBlocks;
      const int64_t most = (8 * 148 + units - 1) / units;
      chunks = static_cast<unsigned>(pieces < most ? pieces : most);
    }
    return launch_chained(join_kernel<T, D>, dim3(1 + chunks, static_cast<unsigned>(c->Hkv), static_cast<unsigned>(s->B)),
                          kJoinThreads, 0, 0, st, a, parts > 0);
  }
};

cudaError_t launch_cache_attn(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride,
                              const int32_t* kept, const int32_t* n_kept, void* o, float* lse, float scale,
                              int accumulate, const CacheAttnScratch& ws, int32_t* dev_status, cudaStream_t st) {
  return by_cache_type(c, AttnCall{c, s, q, H, q_stride, kept, n_kept, o, lse, scale, accumulate, ws, dev_status, st});
}

}  // namespace fva
