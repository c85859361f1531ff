// Gradient of block-sparse attention on sm_100a tensor cores (bf16, d in {64, 128}).
//
// Two kernels of one shape. A CTA owns 128 rows (two adjacent blocks) and walks its tile's
// list of 64-row blocks of the other side:
//   KV = false  owns query rows; streams K, V.   S = Q K^T, dP = dO V^T, dQ += dS K
//   KV = true   owns key rows; streams Q, dO.    S^T = K Q^T, dP^T = V dO^T,
//                                                dV += P^T dO, dK += dS^T Q
// with P = 2^(scale log2(e) S - lse2) and dS = P (dP - D), both rounded to bf16 as operands of
// the second products (their relative error, 2^-9 on average, is the size of the gradients'
// own rounding); sums stay in fp32 in TMEM. One owner per output row: no atomics.
//
//   * Warp 8 issues TMA loads into a ring of stages, warp 9 issues tcgen05.mma; warps 0-7 form
//     P and dS, each thread one row (TMEM lane) and half of a step's 64 columns. S and dP sit
//     in 2 (d = 128) or 3 (d = 64) TMEM buffers, so the tensor cores run the next step's first
//     products while the warps work; P and dS overwrite them as packed bf16 and are the A
//     operands, from TMEM, of the second products.
//   * M = 128, N = 64 products with A in shared memory read 6 KB per 32 tensor cycles, above
//     the 128 B a cycle that shared memory gives. The query kernel therefore keeps Q and dO
//     in TMEM (columns: dQ d, Q d/2, dO d/2, buffers: 512 in all). The key kernel has no room
//     for both K and V there beside dK and dV.
//   * The statistics of a 64-row block, -lse2 and -D, are one 512-byte piece (see
//     row_stats_kernel): the key kernel streams it with Q and dO. Rows without keys and rows
//     past N have -lse2 = -infinity, so their P is 0.
//   * Every wait is bounded; on expiry the CTA reports FVA_DEVERR_TIMEOUT, drains its own
//     loads and products, frees TMEM and exits.
#include <math.h>

#include "fva_internal.cuh"

namespace fva {

constexpr int kBwdThreads = 320;
constexpr uint32_t kBwdTmemCols = 512;

template <int D, bool KV>
struct BwdCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = kChunks * 64 * 128;                  // 64 rows x D bf16
  static constexpr int kOwn = KV ? 2 * kChunks * 128 * 128 : 0;     // K and V of the owned rows
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = D == 128 ? (KV ? 4 : 6) : 8;
  static constexpr int kStats = KV ? kStages * 512 : 0;
  static constexpr int kBufs = D == 128 ? 2 : 3;
  static constexpr uint32_t kBufCol = 2 * D;  // buffer i: S at kBufCol + 128 i, dP 64 columns on
  static constexpr int kSmemData = kOwn + kStages * kStage + kStats;
};

template <int D, bool KV>
struct __align__(8) BwdBars {
  uint64_t own_full;
  uint64_t full[BwdCfg<D, KV>::kStages];
  uint64_t empty[BwdCfg<D, KV>::kStages];
  uint64_t s_full[BwdCfg<D, KV>::kBufs];
  uint64_t p_full[BwdCfg<D, KV>::kBufs];
  uint64_t out_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int D, bool KV>
constexpr size_t bwd_smem_bytes() {
  return 1024 /*alignment slack*/ + BwdCfg<D, KV>::kSmemData + sizeof(BwdBars<D, KV>);
}

// own0, own1: Q and dO (KV = false, read by the threads) -- maps of the streamed pair in
// tm0 / tm1, of the owned pair (KV) in tmo0 / tmo1.
template <int D, bool KV>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmo0, const __grid_constant__ CUtensorMap tmo1,
                       const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                       const __nv_bfloat16* __restrict__ own0, const __nv_bfloat16* __restrict__ own1,
                       const float* __restrict__ stats, __nv_bfloat16* __restrict__ out0,
                       __nv_bfloat16* __restrict__ out1, const int32_t* __restrict__ tile_ptr,
                       const int32_t* __restrict__ tile_col, const int32_t* __restrict__ worklist, int ntiles, int N,
                       int nB, int nPairs, float scale, float scale_log2, uint64_t wait_limit_ns, uint32_t diag_flags,
                       int32_t* dev_status) {
  using Cfg = BwdCfg<D, KV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_own = smem;
  uint8_t* s_ring = smem + Cfg::kOwn;
  uint8_t* s_stats = s_ring + Cfg::kStages * Cfg::kStage;
  BwdBars<D, KV>& bar = *reinterpret_cast<BwdBars<D, KV>*>(smem + Cfg::kSmemData);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int tile = worklist[blockIdx.x];
  const bool tile_ok = tile >= 0 && tile < ntiles;
  if (!tile_ok) {
    if (threadIdx.x == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
    tile = 0;
  }
  const int bh = tile / nPairs, t = tile - bh * nPairs;
  const int list_base = tile_ptr[tile];
  const int n_iter = tile_ok ? tile_ptr[tile + 1] - list_base : 0;

  if (threadIdx.x == 256) {
    tma_prefetch_desc(&tm0);
    tma_prefetch_desc(&tm1);
    mbar_init(&bar.own_full, 1);
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
    }
    for (int i = 0; i < Cfg::kBufs; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 256);
    }
    mbar_init(&bar.out_full, 1);
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&bar.tmem_base, kBwdTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;
  volatile int* abort_flag = &bar.abort;
  const int row = (warp & 3) * 32 + lane;  // warps 0-7: row of the tile, and column half
  const int grow = t * 128 + row;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  if (!KV) {
    // the owned rows become A operands: warps 0-3 store Q, warps 4-7 dO
    if (warp < 8) {
      const uint4* src = reinterpret_cast<const uint4*>((warp < 4 ? own0 : own1) + (static_cast<int64_t>(bh) * N + grow) * D);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 x = grow < N ? src[c * 8 + i] : make_uint4(0u, 0u, 0u, 0u);
          r[4 * i] = x.x;
          r[4 * i + 1] = x.y;
          r[4 * i + 2] = x.z;
          r[4 * i + 3] = x.w;
        }
        tmem_st32(lane_base + D + (warp < 4 ? 0 : D / 2) + c * 32, r);
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      bool ok = true;
      int uses[Cfg::kStages];
      for (int s = 0; s < Cfg::kStages; ++s) uses[s] = 0;
      const bool withhold = diag_flags & FVA_DIAG_WITHHOLD_Q;
      if (KV && !withhold && n_iter > 0) {
        mbar_arrive_expect_tx(&bar.own_full, Cfg::kOwn);
        for (int c = 0; c < Cfg::kChunks; ++c)
          for (int hf = 0; hf < 2; ++hf) {
            const int at = c * (128 * 128) + hf * (64 * 128);
            tma_load_3d(s_own + at, &tmo0, &bar.own_full, c * 64, t * 128 + hf * 64, bh);
            tma_load_3d(s_own + Cfg::kOwn / 2 + at, &tmo1, &bar.own_full, c * 64, t * 128 + hf * 64, bh);
          }
      }
      for (int j = 0; j < n_iter; ++j) {
        const int blk = tile_col[list_base + j] >> 2;
        if (blk < 0 || blk >= nB) {
          report(dev_status, FVA_DEVERR_BAD_LIST);
          *abort_flag = 1;
          break;
        }
        const int s = j % Cfg::kStages;
        if (j >= Cfg::kStages &&
            !mbar_wait(&bar.empty[s], ((j / Cfg::kStages) - 1) & 1, abort_flag, wait_limit_ns)) {
          ok = false;
          break;
        }
        if (!KV && withhold) break;  // nothing ever arrives: the waits behind it run out
        mbar_arrive_expect_tx(&bar.full[s], Cfg::kStage + (KV ? 512 : 0));
        uint8_t* dst = s_ring + s * Cfg::kStage;
        for (int c = 0; c < Cfg::kChunks; ++c) {
          tma_load_3d(dst + c * (64 * 128), &tm0, &bar.full[s], c * 64, blk * 64, bh);
          tma_load_3d(dst + Cfg::kTile + c * (64 * 128), &tm1, &bar.full[s], c * 64, blk * 64, bh);
        }
        if (KV) bulk_load(s_stats + s * 512, stats + (static_cast<int64_t>(bh) * nB + blk) * 128, 512, &bar.full[s]);
        ++uses[s];
      }
      if (!ok) {
        report(dev_status, FVA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (*abort_flag) {  // wait (bounded) for the last load into every buffer
        volatile int never = 0;
        if (KV && !withhold && n_iter > 0) mbar_wait(&bar.own_full, 0, &never, 100000000ull);
        for (int s = 0; s < Cfg::kStages; ++s)
          if (uses[s] > 0) mbar_wait(&bar.full[s], (uses[s] - 1) & 1, &never, 100000000ull);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_iter > 0) {
      constexpr uint32_t idesc_first = idesc_f16kind_f32(128, 64, 0, 0, kFmtBF16);
      constexpr uint32_t idesc_second = idesc_f16kind_f32(128, D, 0, 1, kFmtBF16);
      bool ok = KV ? mbar_wait(&bar.own_full, 0, abort_flag, wait_limit_ns) : true;
      bool issued = false;
      constexpr int kLag = Cfg::kBufs - 1;
      // x(buffer) = own (A) * streamed^T, over the D channels
      auto first = [&](uint32_t d_col, uint32_t own_smem, uint32_t own_col, uint32_t b_base) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int c = kk >> 2;
          const uint32_t ko = (kk & 3) * 32;
          const uint64_t bdesc = sdesc_sw128(b_base + c * (64 * 128) + ko, 16, 1024);
          if (KV)
            mma_ss(tmem + d_col, sdesc_sw128(own_smem + c * (128 * 128) + ko, 16, 1024), bdesc, idesc_first, kk > 0);
          else
            mma_ts(tmem + d_col, tmem + own_col + kk * 8, bdesc, idesc_first, kk > 0);
        }
      };
      // out += x (A, packed bf16 in the buffer) * streamed, over the block's 64 rows. The two
      // column halves of x were stored 32 columns apart (each warp inside its own columns).
      auto second = [&](uint32_t out_col, uint32_t x_col, uint32_t b_base, bool add) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(tmem + out_col, tmem + x_col + (kk >> 1) * 32 + (kk & 1) * 8,
                 sdesc_sw128(b_base + kk * 2048, 64 * 128, 1024), idesc_second, add || kk > 0);
      };
      auto finish = [&](int i) -> bool {
        const int sb = i % Cfg::kBufs, s = i % Cfg::kStages;
        if (!mbar_wait(&bar.p_full[sb], (i / Cfg::kBufs) & 1, abort_flag, wait_limit_ns)) return false;
        tc_fence_after();
        const uint32_t b0 = smem_u32(s_ring + s * Cfg::kStage);
        const uint32_t col = Cfg::kBufCol + sb * 128;
        if (KV) second(D, col, b0 + Cfg::kTile, i > 0);  // dV += P^T dO
        second(0, col + 64, b0, i > 0);                  // dK += dS^T Q, or dQ += dS K
        tc_commit(&bar.empty[s]);
        return true;
      };
      if (ok) tc_fence_after();
      for (int j = 0; j < n_iter && ok; ++j) {
        const int s = j % Cfg::kStages, sb = j % Cfg::kBufs;
        if (!mbar_wait(&bar.full[s], (j / Cfg::kStages) & 1, abort_flag, wait_limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the products are executed in the order of issue, so the buffer's last reader, step
        // j - kBufs, is done with it when these write
        const uint32_t b0 = smem_u32(s_ring + s * Cfg::kStage);
        const uint32_t col = Cfg::kBufCol + sb * 128;
        first(col, smem_u32(s_own), D, b0);
        first(col + 64, smem_u32(s_own) + Cfg::kOwn / 2, D + D / 2, b0 + Cfg::kTile);
        issued = true;
        tc_commit(&bar.s_full[sb]);
        if (j >= kLag && !finish(j - kLag)) ok = false;
      }
      for (int i = n_iter > kLag ? n_iter - kLag : 0; i < n_iter && ok; ++i) ok = finish(i);
      if (ok) {
        tc_commit(&bar.out_full);
      } else {
        report(dev_status, FVA_DEVERR_TIMEOUT);
        *abort_flag = 1;
        if (issued) {
          volatile int never = 0;
          tc_commit(&bar.drain);
          mbar_wait(&bar.drain, 0, &never, 100000000ull);
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ P and dS
    const int half = (warp & 3) >> 1, ch = warp >> 2;
    float nl_row = 0.0f, nd_row = 0.0f;  // KV = false: this row's -lse2 and -D
    if (!KV) {
      const bool in = 2 * t + (row >> 6) < nB;
      const float* st = stats + (static_cast<int64_t>(bh) * nB + 2 * t + (row >> 6)) * 128 + (row & 63);
      nl_row = in ? st[0] : -INFINITY;
      nd_row = in ? st[64] : 0.0f;
    }
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    bool ok = true;
    for (int j = 0; j < n_iter; ++j) {
      const int entry = tile_col[list_base + j];
      const int blk = entry >> 2;
      const int sb = j % Cfg::kBufs;
      // (KV: these threads read the stage's statistics too, which S only implies have landed)
      if (!warp_wait(&bar.s_full[sb], (j / Cfg::kBufs) & 1, abort_flag, wait_limit_ns) ||
          (KV && !warp_wait(&bar.full[j % Cfg::kStages], (j / Cfg::kStages) & 1, abort_flag, wait_limit_ns))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t col = lane_base + Cfg::kBufCol + sb * 128 + ch * 32;
      uint32_t pp[16], pd[16];
      if ((entry >> half) & 1) {
        uint32_t x[32], y[32];
        tmem_ld32_pair(col, x, col + 64, y);
        const ulonglong2* nl4 = nullptr;
        const ulonglong2* nd4 = nullptr;
        if (KV) {
          nl4 = reinterpret_cast<const ulonglong2*>(s_stats + (j % Cfg::kStages) * 512 + ch * 128);
          nd4 = reinterpret_cast<const ulonglong2*>(s_stats + (j % Cfg::kStages) * 512 + 256 + ch * 128);
        }
        const uint64_t nlr = f2_pack(nl_row, nl_row), ndr = f2_pack(nd_row, nd_row);
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          ulonglong2 nl, nd;
          if (KV) {
            nl = nl4[c / 2];
            nd = nd4[c / 2];
          } else {
            nl = make_ulonglong2(nlr, nlr);
            nd = make_ulonglong2(ndr, ndr);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int e = 2 * (c + i);
            const float2 a = f2_unpack(f2_fma(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sc2, i ? nl.y : nl.x));
            float p0 = ex2_approx(a.x), p1 = ex2_approx(a.y);
            if (!KV && blk == nB - 1) {  // keys past N: zero rows, not -inf scores
              const int nvalid = N - blk * 64 - ch * 32;
              if (e >= nvalid) p0 = 0.0f;
              if (e + 1 >= nvalid) p1 = 0.0f;
            }
            const uint64_t g = f2_add(f2_pack(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), i ? nd.y : nd.x);
            const float2 ds = f2_unpack(f2_mul(f2_pack(p0, p1), g));
            if (KV) pp[c + i] = pack_bf16x2(p0, p1);
            pd[c + i] = pack_bf16x2(ds.x, ds.y);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) pp[c] = pd[c] = 0u;
      }
      if (KV) tmem_st16(col, pp);
      tmem_st16(col + 64, pd);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bar.p_full[sb]);
    }
    // ------------------------------------------------------------------ epilogue
    if (ok && n_iter > 0 && !warp_wait(&bar.out_full, 0, abort_flag, wait_limit_ns)) ok = false;
    if (!ok) {
      report(dev_status, FVA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    } else if (tile_ok) {
      tc_fence_after();
      // KV: warps 0-3 write dK, warps 4-7 dV; else the halves of dQ
      constexpr int kCols = KV ? D : D / 2;
      const float f = KV && ch == 1 ? 1.0f : scale;
      __nv_bfloat16* dst = (KV && ch == 1 ? out1 : out0) + (static_cast<int64_t>(bh) * N + grow) * D + (KV ? 0 : ch * kCols);
#pragma unroll
      for (int cc = 0; cc < kCols / 32; ++cc) {
        uint32_t o[32];
        if (n_iter > 0) {
          tmem_ld32(lane_base + (KV ? ch * D : ch * kCols) + cc * 32, o);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
        if (grow < N) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * i]) * f, __uint_as_float(o[8 * q + 2 * i + 1]) * f);
            reinterpret_cast<uint4*>(dst)[cc * 4 + q] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kBwdTmemCols);
  }
}

template <int D, bool KV>
static cudaError_t launch_tc_t(const Dims& Dm, const BwdArgs& x, const CUtensorMap& mq, const CUtensorMap& mk,
                               const CUtensorMap& mv, const CUtensorMap& mdo, const fva_mask* m, const float* stats,
                               int32_t* dev_status, cudaStream_t st) {
  const size_t smem = bwd_smem_bytes<D, KV>();
  const cudaError_t e = cudaFuncSetAttribute(attn_bwd_tc_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  using bf = __nv_bfloat16;
  attn_bwd_tc_kernel<D, KV><<<static_cast<unsigned>(Dm.tiles), kBwdThreads, smem, st>>>(
      KV ? mk : mq, KV ? mv : mdo, KV ? mq : mk, KV ? mdo : mv, static_cast<const bf*>(x.q),
      static_cast<const bf*>(x.d_o), stats, static_cast<bf*>(KV ? x.dk : x.dq), static_cast<bf*>(KV ? x.dv : nullptr),
      m->tile_ptr, m->tile_col, m->worklist, static_cast<int>(Dm.tiles), static_cast<int>(Dm.N),
      static_cast<int>(Dm.nB), static_cast<int>(Dm.nPairs), x.scale, x.scale * 1.4426950408889634f,
      attn_wait_limit_ns(), attn_diag_flags(), dev_status);
  return cudaGetLastError();
}

cudaError_t launch_attn_bwd_tc(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const fva_mask* m_t,
                               const float* stats, int32_t* dev_status, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mdo;
  if (!make_bhnd_map(&mq, x.q, Dm.BH, Dm.N, Dm.d, false) || !make_bhnd_map(&mk, x.k, Dm.BH, Dm.N, Dm.d, false) ||
      !make_bhnd_map(&mv, x.v, Dm.BH, Dm.N, Dm.d, false) || !make_bhnd_map(&mdo, x.d_o, Dm.BH, Dm.N, Dm.d, false))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (Dm.d == 128) {
    e = launch_tc_t<128, true>(Dm, x, mq, mk, mv, mdo, m_t, stats, dev_status, st);
    return e != cudaSuccess ? e : launch_tc_t<128, false>(Dm, x, mq, mk, mv, mdo, m, stats, dev_status, st);
  }
  e = launch_tc_t<64, true>(Dm, x, mq, mk, mv, mdo, m_t, stats, dev_status, st);
  return e != cudaSuccess ? e : launch_tc_t<64, false>(Dm, x, mq, mk, mv, mdo, m, stats, dev_status, st);
}

}  // namespace fva
