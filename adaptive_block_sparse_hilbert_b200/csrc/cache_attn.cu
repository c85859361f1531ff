// Attention of single query tokens over kept blocks of a paged key/value cache.
//
// A unit is one (sequence, key head, group of up to 16 query heads). All units' kept blocks,
// laid end to end, are cut into equal shares, one per CTA, so a long sequence spreads over
// many SMs and short ones share one: the work is a read of the kept keys and values, and every
// SM reads the same amount. A unit inside one CTA's share is finished there; one that crosses
// shares leaves each share's unnormalised O with its running maximum and sum in the workspace,
// and a second kernel joins them in share order (a fixed order: equal inputs, equal bits) and
// accumulates the weights.
#include <math.h>

#include "cache.cuh"

namespace fva {

constexpr int kShares = 296;  // CTAs of the split kernels: two per SM
constexpr int kGroup = 16;    // query heads of a unit at most

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

// Writes a finished row, or its unnormalised parts for the join. x: this thread's channel.
template <typename T, int D>
__device__ __forceinline__ void put_row(const AttnView<T>& a, bool whole, int share, int slot, int64_t row, int g, int ch,
                                        float x, float mx, float sum) {
  if (whole) {
    from_f32(sum > 0.0f ? x / sum : 0.0f, a.o + row * D + ch);
    if (ch == 0) {
      const float l2 = sum > 0.0f ? mx + log2f(sum) : -INFINITY;
      if (a.lse) a.lse[row] = l2 * 0.6931471805599453f;
      if (a.ws.scores) a.ws.lse[row] = l2;
    }
  } else {
    float* part = a.ws.part + ((static_cast<int64_t>(share) * 2 + slot) * kGroup + g) * (D + 2);
    part[ch] = x;
    if (ch == 0) {
      part[D] = mx;
      part[D + 1] = sum;
    }
  }
}

// ---------------------------------------------------------------------------------
// 16-bit caches
// ---------------------------------------------------------------------------------
// Four warps take 16 keys each of every block, with softmax statistics and an O of their own
// (joined at a unit's end); a fifth walks the lists and page table and keeps TMA loads of whole
// pages in flight. The reads bound it, so the products are the small mma.sync ones (16 query
// heads x 8 keys), whose operands stay in registers between the two products, and a weight is
// kept in two 16-bit parts (its head and the rest, 2^-16 of it or less is lost), which costs
// tensor time that the loads hide.
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

template <typename T, int D>
__global__ void __launch_bounds__(kSplitThreads, 2)
    split_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, AttnView<T> a,
                 uint64_t wait_limit_ns) {
  using Cfg = SplitCfg<D>;
  using F = Frag<T>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float s_o[kGroup][D];
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
  const Share sh = find_share(a, share);  // (its barriers publish the mbarriers too)
  Walk<T> w(sh, share);
  volatile int* abort_flag = &s_abort;
  bool ok = true;
  int stage = 0, phase = 0;

  if (warp == 4) {
    // ------------------------------------------------------------------ loads
    const bool leader = elect_one();
    int issued = 0;
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
          if (!warp_wait_spin(&empty[stage], phase ^ 1, abort_flag, wait_limit_ns)) {
            ok = false;
            break;
          }
          if (leader) {
            s_valid[stage] = va;
            if (pg >= 0) {
              uint8_t* dst = ring + stage * 2 * Cfg::kTile;
              mbar_arrive_expect_tx(&full[stage], 2 * Cfg::kTile);
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                tma_load_3d(dst + c * (kBlock * 128), &tmk, &full[stage], c * 64, h * kBlock, pg);
                tma_load_3d(dst + Cfg::kTile + c * (kBlock * 128), &tmv, &full[stage], c * 64, h * kBlock, pg);
              }
            } else {
              mbar_arrive(&full[stage]);
            }
          }
          ++issued;
          if (++stage == Cfg::kStages) {
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
    // a CTA that gives up waits (bounded) for its loads in flight
    if (*abort_flag) {
      volatile int never = 0;
      for (int j = issued > Cfg::kStages ? issued - Cfg::kStages : 0; j < issued; ++j)
        mbar_wait(&full[j % Cfg::kStages], (j / Cfg::kStages) & 1, &never, 100000000ull);
    }
    return;
  }

  // -------------------------------------------------------------------- products and softmax
  const int rg = lane >> 2, ct = lane & 3;  // fragment rows rg, rg + 8; columns 2 ct, 2 ct + 1
  const int lm = lane >> 3, lr = lane & 7;  // ldmatrix: matrix and row of this lane's address
  while (ok && w.next(a)) {
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
      if (!warp_wait_spin(&full[stage], phase, abort_flag, wait_limit_ns)) {
        ok = false;
        break;
      }
      const int nk = s_valid[stage] - warp * 16;  // this warp's keys that count
      const uint32_t sk = smem_u32(ring + stage * 2 * Cfg::kTile), sv = sk + Cfg::kTile;
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
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
          F::mma(s[0], qa[kk], kb[0], kb[1]);
          F::mma(s[1], qa[kk], kb[2], kb[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = n * 8 + ct * 2 + (i & 1);
          s[n][i] = key < nk ? s[n][i] * a.scale_log2 : -INFINITY;
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
        for (int n = 0; n < D / 16; ++n) {
          uint32_t vb[4];
          ldmatrix4_trans(vb, sv + tile_at(warp * 16 + (lm & 1) * 8 + lr, n * 2 + (lm >> 1)));
          F::mma(o[2 * n], ph, vb[0], vb[1]);
          F::mma(o[2 * n + 1], ph, vb[2], vb[3]);
          F::mma(o[2 * n], pl, vb[0], vb[1]);
          F::mma(o[2 * n + 1], pl, vb[2], vb[3]);
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
    if (!ok) break;
    // ---- join the four warps, one after the other, in shared memory
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
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rg + i * 8;
      const float mx = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
      f[i] = m[i] == -INFINITY ? 0.0f : exp2f(s_m[warp][r] - mx);
    }
    for (int turn = 0; turn < 4; ++turn) {
      if (turn == warp) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = rg + (i >> 1) * 8;
            if (r < ng) {
              float* at = &s_o[r][n * 8 + ct * 2 + (i & 1)];
              const float x = o[n][i] * f[i >> 1];
              *at = turn == 0 ? x : *at + x;
            }
          }
      }
      sync4();
    }
    const bool whole = w.whole();
    for (int i = tid; i < ng * D; i += 128) {
      const int g = i / D, ch = i % D;
      const float mx = fmaxf(fmaxf(s_m[0][g], s_m[1][g]), fmaxf(s_m[2][g], s_m[3][g]));
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) sum += s_m[v][g] == -INFINITY ? 0.0f : s_l[v][g] * exp2f(s_m[v][g] - mx);
      put_row<T, D>(a, whole, share, w.slot(), row0 + g, g, ch, s_o[g][ch], mx, sum);
    }
    if (tid == 0) a.ws.start[w.u] = w.start;
    sync4();  // s_m, s_l and s_o are rewritten by the next unit
    w.at = stop;
  }
  if (!ok) {
    report(a.dev_status, FVA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  }
}

// ---------------------------------------------------------------------------------
// fp32 caches
// ---------------------------------------------------------------------------------
// CUDA cores, one CTA per share: each of four warps takes 16 keys of every block, lanes hold
// D / 32 channels each, with softmax statistics and an O of their own.
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

template <int D, int G>
__global__ void __launch_bounds__(128) split_f32_kernel(AttnView<float> a) {
  constexpr int V = D / 32;
  __shared__ float s_p[4][G][16];
  __shared__ float s_o[4][G][D];
  __shared__ float s_m[4][G], s_l[4][G];
  const int share = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Share sh = find_share(a, share);
  Walk<float> w(sh, share);
  while (w.next(a)) {
    const int bh = w.u / a.GS, b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
    const int g0 = (w.u - bh * a.GS) * kGroup, ng = min(a.G - g0, kGroup);
    const int64_t row0 = static_cast<int64_t>(b) * a.H + h * a.G + g0;
    const int len = seq_len(a.c, b, nullptr);
    float q[G][V], acc[G][V], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g < ng) load_vec<V>(a.q + b * a.q_stride + static_cast<int64_t>(h * a.G + g0 + g) * D + lane * V, q[g]);
      m[g] = -INFINITY;
      l[g] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc[g][i] = 0.0f;
        q[g][i] = g < ng ? q[g][i] * a.scale_log2 : 0.0f;
      }
    }
    const int64_t stop = w.stop();
    for (int64_t at = w.at; at < stop; ++at) {
      const int pos = static_cast<int>(at - w.start);
      const int block = unit_block(a, bh, pos, len, a.dev_status);
      const int page = block < 0 ? -1 : page_of(a.c, b, block, a.dev_status);
      const int valid = page < 0 ? 0 : min(len - block * kBlock, kBlock);
      const int r0 = warp * 16, nk = max(0, min(valid - r0, 16));
      const int64_t base = (static_cast<int64_t>(page < 0 ? 0 : page) * a.c.Hkv + h) * kBlock + r0;
      __syncwarp();
#pragma unroll 4
      for (int r = 0; r < 16; ++r) {
        float v[G];
        if (r < nk) {
          float k[V];
          load_vec<V>(a.c.k + (base + r) * D + lane * V, k);
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
      if (a.ws.scores) {  // kept for the accumulation: -inf behind the last key
        for (int i = lane; i < ng * 16; i += 32)
          a.ws.scores[(row0 + i / 16) * a.c.max_blocks * kBlock + static_cast<int64_t>(pos) * kBlock + r0 + i % 16] =
              s_p[warp][i / 16][i % 16];
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
#pragma unroll 4
        for (int r = 0; r < 16; ++r) {
          if (r >= nk) break;
          float v[V];
          load_vec<V>(a.c.v + (base + r) * D + lane * V, v);
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
    const bool whole = w.whole();
    for (int i = threadIdx.x; i < ng * D; i += 128) {
      const int g = i / D, ch = i % D;
      float mx = -INFINITY;
      for (int v = 0; v < 4; ++v) mx = fmaxf(mx, s_m[v][g]);
      float sum = 0.0f, x = 0.0f;
      for (int v = 0; v < 4; ++v) {
        const float f = s_m[v][g] == -INFINITY ? 0.0f : exp2f(s_m[v][g] - mx);
        sum = fmaf(s_l[v][g], f, sum);
        x = fmaf(s_o[v][g][ch], f, x);
      }
      put_row<float, D>(a, whole, share, w.slot(), row0 + g, g, ch, x, mx, sum);
    }
    if (threadIdx.x == 0) a.ws.start[w.u] = w.start;
    __syncthreads();
    w.at = stop;
  }
}

// ---------------------------------------------------------------------------------
// Join and accumulation
// ---------------------------------------------------------------------------------
// CTA (x, key head, sequence): every CTA forms the heads' log-sum-exp from the shares' maxima
// and sums; x = 0 also joins their O (a warp per head), and, where weights are accumulated,
// each adds exp(s - lse), summed over the heads, to the masses of 32 listed blocks.
constexpr int kJoinThreads = 256, kMassBlocks = 32;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnView<T> a, int accumulate) {
  __shared__ float s_lse[kMaxCacheGroup];
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = b * a.c.Hkv + h;
  const int n = unit_count(a, bh * a.GS, nullptr);
  const int pos0 = blockIdx.x * kMassBlocks;
  if (blockIdx.x > 0 && pos0 >= n) return;
  const int64_t per = n ? *a.ws.per : 1;
  for (int g = warp; g < a.G; g += kJoinThreads / 32) {
    const int64_t row = static_cast<int64_t>(b) * a.H + h * a.G + g;
    const int64_t start = n ? a.ws.start[bh * a.GS + g / kGroup] : 0;
    const int c0 = static_cast<int>(start / per), c1 = n ? static_cast<int>((start + n - 1) / per) : c0;
    if (n && c0 == c1) {  // finished by the split kernel
      if (lane == 0 && accumulate) s_lse[g] = a.ws.lse[row];
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
      if (blockIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= f0;
        const int cnt = min(32, c1 - s0 + 1);
#pragma unroll 4
        for (int k = 0; k < cnt; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, k);
          const float* x = part_of(s0 + k) + lane * V;
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fk == 0.0f ? acc[i] : fmaf(fk, x[i], acc[i]);
        }
      }
    }
    const float l2 = sum > 0.0f ? mx + log2f(sum) : -INFINITY;
    if (blockIdx.x == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) from_f32(sum > 0.0f ? acc[i] / sum : 0.0f, a.o + row * D + lane * V + i);
      if (lane == 0 && a.lse) a.lse[row] = l2 * 0.6931471805599453f;
    }
    if (lane == 0) s_lse[g] = l2;
  }
  if (!accumulate) return;
  __syncthreads();
  const int len = seq_len(a.c, b, nullptr);
  for (int i = tid; i < kMassBlocks * kBlock; i += kJoinThreads) {
    const int pos = pos0 + i / kBlock, r = i % kBlock;
    if (pos >= n) break;
    const int block = a.kept ? a.kept[static_cast<int64_t>(bh) * a.c.max_blocks + pos] : pos;
    if (block < 0 || static_cast<int64_t>(block) * kBlock + r >= len) continue;
    const int page = page_of(a.c, b, block, nullptr);
    if (page < 0) continue;
    const float* s = a.ws.scores + ((static_cast<int64_t>(b) * a.H + h * a.G) * a.c.max_blocks + pos) * kBlock + r;
    float w = 0.0f;
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) w += exp2f(s[static_cast<int64_t>(g) * a.c.max_blocks * kBlock] - s_lse[g]);
    atomicAdd(a.c.mass + (static_cast<int64_t>(page) * a.c.Hkv + h) * kBlock + r, w);
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

template <typename T, int D>
static cudaError_t launch_split(const fva_cache* c, const AttnView<T>& a, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    CUtensorMap mk, mv;
    if (!make_page_map(&mk, c->k, c) || !make_page_map(&mv, c->v, c)) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(split_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               SplitCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    split_kernel<T, D><<<kShares, kSplitThreads, SplitCfg<D>::kSmem, st>>>(mk, mv, a, attn_wait_limit_ns());
  } else {
    const int g = a.G < kGroup ? a.G : kGroup;
    if (g <= 1) split_f32_kernel<D, 1><<<kShares, 128, 0, st>>>(a);
    else if (g <= 4) split_f32_kernel<D, 4><<<kShares, 128, 0, st>>>(a);
    else if (g <= 8) split_f32_kernel<D, 8><<<kShares, 128, 0, st>>>(a);
    else split_f32_kernel<D, 16><<<kShares, 128, 0, st>>>(a);
  }
  return cudaGetLastError();
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
    const cudaError_t e = launch_split<T, D>(c, a, st);
    if (e != cudaSuccess) return e;
    const unsigned chunks = accumulate ? static_cast<unsigned>((s->max_blocks + kMassBlocks - 1) / kMassBlocks) : 1u;
    join_kernel<T, D><<<dim3(chunks, static_cast<unsigned>(c->Hkv), static_cast<unsigned>(s->B)), kJoinThreads, 0, st>>>(
        a, accumulate);
    return cudaGetLastError();
  }
};

cudaError_t launch_cache_attn(const fva_cache* c, const fva_seqs* s, const void* q, int H, int64_t q_stride,
                              const int32_t* kept, const int32_t* n_kept, void* o, float* lse, float scale,
                              int accumulate, const CacheAttnScratch& ws, int32_t* dev_status, cudaStream_t st) {
  return by_cache_type(c, AttnCall{c, s, q, H, q_stride, kept, n_kept, o, lse, scale, accumulate, ws, dev_status, st});
}

}  // namespace fva
