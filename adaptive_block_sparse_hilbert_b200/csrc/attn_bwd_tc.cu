// Gradient of block-sparse attention on sm_100a tensor cores (bf16, d in {64, 128}).
//
// Two passes of one shape, one launch. A CTA owns 128 rows (two adjacent blocks) and walks its tile's
// list of 64-row blocks of the other side:
//   KV = false  owns query rows; streams K, V.   S = Q K^T, dP = dO V^T, dQ += dS K
//   KV = true   owns key rows; streams Q, dO.    S^T = K Q^T, dP^T = V dO^T,
//                                                dV += P^T dO, dK += dS^T Q
// with P = 2^(scale log2(e) S - lse2) and dS = P (dP - D), both rounded to bf16 as operands of
// the second products. That moves the gradients by 1.7e-3 of their norm, as much as their own
// rounding does, so the two together by 2.4e-3; two parts of 16 bits, as the decoding attention keeps
// its weights in, would make two products of each second one. Sums stay in fp32 in TMEM. One
// owner per output row: no atomics.
//
//   * Warp 16 issues TMA loads into two rings of stages, warp 17 the products S, warp 18 dP and
//     the second products. (One thread's waits and commits for all three took longer than the
//     products: 1130 cycles a step where the dQ kernel's take 800. dP and the second products
//     stay in one thread because products execute in the order of issue: dP needs no wait for
//     its buffer's last readers.) Warps 0-15 form P and dS: two groups of eight take alternate
//     steps, each thread one row (TMEM lane) and half of the step's 64 columns.
//   * S runs ahead: its buffers are free again once the warps have read them, so the exponentials
//     of a step overlap the products of the one before. P and dS (packed bf16) share the
//     columns of the dP buffer they came from and are A operands from TMEM.
//   * M = 128, N = 64 products with A in shared memory read 6 KB per 32 tensor cycles, above
//     the 128 B a cycle that shared memory gives, so the owned operands (A) go to TMEM where
//     its 512 columns have room (outputs, owned operands, S buffers, dP buffers):
//       dQ     d = 128: 128 + Q 64 + dO 64 + 2 x 64 + 2 x 64    d = 64: 64 + 32 + 32 + 3 x 64 + 3 x 64
//       dK, dV d = 128: 256 (K, V in smem) + 2 x 64 + 2 x 64    d = 64: 128 + 32 + 32 + 2 x 64 + 3 x 64
//     (dK, dV at d = 128 with K in TMEM and one S buffer: 5.3 ms where this takes 5.2.)
//   * The statistics of a 64-row block, -lse2 and -D, are one 512-byte piece (see
//     prepare_kernel): the key kernel streams it with Q and dO. Rows without keys and rows
//     past N have -lse2 = -infinity, so their P is 0.
//   * Measured: 21 x 30 x 52 tokens, 16 heads, d = 128, a quarter of the blocks: 9.0 ms in a
//     stream of calls, 1.35 PFLOP/s of executed products under the power cap, 7.8 alone (tensor
//     pipe 72% of a small case's cycles); 13 x 30 x 45 tokens, 32 heads, d = 64: 4.0 and 3.5 ms,
//     bound by the warps that form P and dS (issue 52%).
//   * Every wait is bounded; on expiry the CTA reports FVA_DEVERR_TIMEOUT, drains its own
//     loads and products, frees TMEM and exits.
#include <math.h>

#include "fva_internal.cuh"

namespace fva {

constexpr int kBwdThreads = 608;
constexpr uint32_t kBwdTmemCols = 512;

template <int D, bool KV>
struct BwdCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = kChunks * 64 * 128;                  // 64 rows x D bf16
  static constexpr bool kOwnSmem = KV && D == 128;                  // K and V stay in shared memory
  static constexpr int kOwnTile = kChunks * 128 * 128;
  static constexpr int kOwn = kOwnSmem ? 2 * kOwnTile : 0;
  // ring 0 holds Q or K (read by the first product of a step and by its second ones), ring 1
  // dO or V, which are needed later or for less long
  static constexpr int kS0 = D == 128 ? (KV ? 5 : 6) : 8;
  static constexpr int kS1 = D == 128 ? (KV ? 4 : 5) : 8;
  static constexpr int kStats = KV ? kS0 * 512 : 0;  // statistics travel with Q
  // S and dP buffers, 64 columns each
  static constexpr int kSBufs = D == 128 || KV ? 2 : 3;
  static constexpr int kDPBufs = D == 128 ? 2 : 3;
  static constexpr int kLag = kDPBufs - 1;
  static constexpr uint32_t kOwn0Col = (KV ? 2 : 1) * D, kOwn1Col = kOwn0Col + D / 2;
  static constexpr uint32_t kSCol = kOwnSmem ? kOwn0Col : kOwn1Col + D / 2, kDPCol = kSCol + 64 * kSBufs;
  static_assert(kDPCol + 64 * kDPBufs <= kBwdTmemCols, "TMEM columns");
  static constexpr int kSmemData = kOwn + (kS0 + kS1) * kTile + kStats;
};

template <int D, bool KV>
struct __align__(8) BwdBars {
  using Cfg = BwdCfg<D, KV>;
  uint64_t own_full;
  uint64_t full0[Cfg::kS0], empty0[Cfg::kS0];
  uint64_t full1[Cfg::kS1], empty1[Cfg::kS1];
  uint64_t s_full[Cfg::kSBufs];    // S is in the buffer
  uint64_t s_free[Cfg::kSBufs];    // the warps have read it
  uint64_t dp_full[Cfg::kDPBufs];  // dP is in the buffer
  uint64_t p_full[Cfg::kDPBufs];   // P and dS have replaced it
  uint64_t out_full;
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
};

// Position in a ring: index and parity of the pass, stepped without divisions.
template <int kSize>
struct RingPos {
  int i = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == kSize) {
      i = 0;
      phase ^= 1;
    }
  }
};

// Entries of a tile's list, 32 at a time in a warp's lanes, the next 32 on their way: a
// per-step load's latency stays off the warp's path. Called by whole warps, j ascending, no 32
// consecutive steps left out.
struct ListReader {
  const int32_t* list;
  int n, batch, cur, next;
  __device__ __forceinline__ ListReader(const int32_t* l, int count, int lane) : list(l), n(count), batch(0) {
    cur = lane < n ? list[lane] : 0;
    next = 32 + lane < n ? list[32 + lane] : 0;
  }
  __device__ __forceinline__ int get(int j, int lane) {
    if ((j >> 5) != batch) {
      batch = j >> 5;
      cur = next;
      const int at = 32 * (batch + 1) + lane;
      next = at < n ? list[at] : 0;
    }
    return __shfl_sync(0xffffffffu, cur, j & 31);
  }
};

template <int D, bool KV>
constexpr size_t bwd_smem_bytes() {
  return 1024 /*alignment slack*/ + BwdCfg<D, KV>::kSmemData + sizeof(BwdBars<D, KV>);
}

struct BwdTcArgs {
  const __nv_bfloat16 *q, *k, *v, *d_o;
  const float* stats;
  __nv_bfloat16 *dq, *dk, *dv;
  const int32_t *tile_ptr, *tile_col, *worklist;  // of the query rows
  BwdLists lists;                                 // of the key rows
  const int32_t* worklist_t;                      // or null: their own order
  int ntiles, N, nB, nPairs;
  float scale, scale_log2;
  uint64_t wait_limit_ns;
  uint32_t diag_flags;
  int32_t* dev_status;
};

// tmo0, tmo1: maps of the owned pair; tm0, tm1: maps of the streamed pair.
template <int D, bool KV>
__device__ __forceinline__ void bwd_tile(const BwdTcArgs& x, const CUtensorMap& tmo0, const CUtensorMap& tmo1,
                                         const CUtensorMap& tm0, const CUtensorMap& tm1, int slot) {
  using Cfg = BwdCfg<D, KV>;
  const __nv_bfloat16 *own0 = KV ? x.k : x.q, *own1 = KV ? x.v : x.d_o;
  __nv_bfloat16 *out0 = KV ? x.dk : x.dq, *out1 = x.dv;
  const float* stats = x.stats;
  const int N = x.N, nB = x.nB, nPairs = x.nPairs;
  const float scale = x.scale, scale_log2 = x.scale_log2;
  const uint64_t wait_limit_ns = x.wait_limit_ns;
  const uint32_t diag_flags = x.diag_flags;
  int32_t* dev_status = x.dev_status;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_own = smem;
  uint8_t* s_ring0 = smem + Cfg::kOwn;
  uint8_t* s_ring1 = s_ring0 + Cfg::kS0 * Cfg::kTile;
  uint8_t* s_stats = s_ring1 + Cfg::kS1 * Cfg::kTile;
  BwdBars<D, KV>& bar = *reinterpret_cast<BwdBars<D, KV>*>(smem + Cfg::kSmemData);

  // (through a shuffle: the compiler then knows that the warp takes each role as a whole)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  int tile = KV ? (x.worklist_t ? x.worklist_t[slot] : slot) : x.worklist[slot];
  const bool tile_ok = tile >= 0 && tile < x.ntiles;
  if (!tile_ok) {
    if (threadIdx.x == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
    tile = 0;
  }
  const int32_t* list = KV ? x.lists.col + static_cast<int64_t>(tile) * nB : x.tile_col + x.tile_ptr[tile];
  const int n_iter = !tile_ok ? 0 : KV ? x.lists.cost[tile] : x.tile_ptr[tile + 1] - x.tile_ptr[tile];
  const int bh = tile / nPairs, t = tile - bh * nPairs;
  if (threadIdx.x == 512) {
    tma_prefetch_desc(&tm0);
    tma_prefetch_desc(&tm1);
    mbar_init(&bar.own_full, 1);
    for (int s = 0; s < Cfg::kS0; ++s) {
      mbar_init(&bar.full0[s], 1);
      mbar_init(&bar.empty0[s], 1);
    }
    for (int s = 0; s < Cfg::kS1; ++s) {
      mbar_init(&bar.full1[s], 1);
      mbar_init(&bar.empty1[s], 1);
    }
    for (int i = 0; i < Cfg::kSBufs; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.s_free[i], 8);
    }
    for (int i = 0; i < Cfg::kDPBufs; ++i) {
      mbar_init(&bar.dp_full[i], 1);
      mbar_init(&bar.p_full[i], 8);
    }
    mbar_init(&bar.out_full, 1);
    mbar_init(&bar.drain[0], 1);
    mbar_init(&bar.drain[1], 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(&bar.tmem_base, kBwdTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;
  volatile int* abort_flag = &bar.abort;
  const int row = (warp & 3) * 32 + lane;  // warps 0-15: row of the tile; warp / 4: a quarter of the work
  const int part = warp >> 2;
  const int grow = t * 128 + row;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  // the owned rows become A operands in TMEM: own0 by parts 0 and 1, own1 by 2 and 3, 64 channels each
  if (!Cfg::kOwnSmem && warp < 16 && (D == 128 || (part & 1) == 0)) {
    const uint4* src = reinterpret_cast<const uint4*>((part < 2 ? own0 : own1) + (static_cast<int64_t>(bh) * N + grow) * D) +
                       (part & 1) * 8;
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 x = grow < N ? src[i] : make_uint4(0u, 0u, 0u, 0u);
      r[4 * i] = x.x;
      r[4 * i + 1] = x.y;
      r[4 * i + 2] = x.z;
      r[4 * i + 3] = x.w;
    }
    tmem_st32(lane_base + (part < 2 ? Cfg::kOwn0Col : Cfg::kOwn1Col) + (part & 1) * 32, r);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 16) {
    // ------------------------------------------------------------------ TMA producer
    const bool leader = elect_one();
    const bool withhold = diag_flags & FVA_DIAG_WITHHOLD_Q;
    ListReader entries(list, n_iter, lane);
    if (Cfg::kOwnSmem && !withhold && n_iter > 0 && leader) {
      mbar_arrive_expect_tx(&bar.own_full, Cfg::kOwn);
      for (int c = 0; c < Cfg::kChunks; ++c)
        for (int hf = 0; hf < 2; ++hf) {
          const int at = c * (128 * 128) + hf * (64 * 128);
          tma_load_3d(s_own + at, &tmo0, &bar.own_full, c * 64, t * 128 + hf * 64, bh);
          tma_load_3d(s_own + Cfg::kOwnTile + at, &tmo1, &bar.own_full, c * 64, t * 128 + hf * 64, bh);
        }
    }
    RingPos<Cfg::kS0> r0;
    RingPos<Cfg::kS1> r1;
    bool ok = true;
    int n0 = 0, n1 = 0;  // loads issued into each ring
    for (int j = 0; j < n_iter; ++j) {
      const int blk = entries.get(j, lane) >> 2;
      if (blk < 0 || blk >= nB) {
        report(dev_status, FVA_DEVERR_BAD_LIST);
        *abort_flag = 1;
        break;
      }
      if (withhold) break;  // nothing ever arrives: the waits behind it run out
      // a ring's first pass finds its stages empty: the parity before the first phase passes
      if (!warp_wait_spin(&bar.empty0[r0.i], r0.phase ^ 1, abort_flag, wait_limit_ns)) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(&bar.full0[r0.i], Cfg::kTile + (KV ? 512 : 0));
#pragma unroll
        for (int c = 0; c < Cfg::kChunks; ++c)
          tma_load_3d(s_ring0 + r0.i * Cfg::kTile + c * (64 * 128), &tm0, &bar.full0[r0.i], c * 64, blk * 64, bh);
        if (KV)
          bulk_load(s_stats + r0.i * 512, stats + (static_cast<int64_t>(bh) * nB + blk) * 128, 512, &bar.full0[r0.i]);
      }
      ++n0;
      if (!warp_wait_spin(&bar.empty1[r1.i], r1.phase ^ 1, abort_flag, wait_limit_ns)) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(&bar.full1[r1.i], Cfg::kTile);
#pragma unroll
        for (int c = 0; c < Cfg::kChunks; ++c)
          tma_load_3d(s_ring1 + r1.i * Cfg::kTile + c * (64 * 128), &tm1, &bar.full1[r1.i], c * 64, blk * 64, bh);
      }
      ++n1;
      r0.next();
      r1.next();
    }
    if (!ok) {
      report(dev_status, FVA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
    __syncwarp();
    // wait (bounded) for the last load into every stage: whichever warp gives up, no load
    // outlives the CTA
    volatile int never = 0;
    if (Cfg::kOwnSmem && !withhold && n_iter > 0) mbar_wait(&bar.own_full, 0, &never, 100000000ull);
    for (int j = n0 > Cfg::kS0 ? n0 - Cfg::kS0 : 0; j < n0; ++j)
      mbar_wait(&bar.full0[j % Cfg::kS0], (j / Cfg::kS0) & 1, &never, 100000000ull);
    for (int j = n1 > Cfg::kS1 ? n1 - Cfg::kS1 : 0; j < n1; ++j)
      mbar_wait(&bar.full1[j % Cfg::kS1], (j / Cfg::kS1) & 1, &never, 100000000ull);
  } else if (warp >= 17) {
    // ------------------------------------------------------------------ products
    // An elected lane, not `lane == 0`: the compiler keeps the descriptors in uniform registers
    // then. An M = 128, N = 64, K = 16 product issues every 34 (A in TMEM) or 48 cycles (A in
    // shared memory: its bandwidth) instead of every 57 to 61.
    if (n_iter > 0 && elect_one()) {
      constexpr uint32_t idesc_first = idesc_f16kind_f32(128, 64, 0, 0, kFmtBF16);
      constexpr uint32_t idesc_second = idesc_f16kind_f32(128, D, 0, 1, kFmtBF16);
      // x(buffer) = own (A) * streamed^T, over the D channels; A in TMEM or shared memory
      auto first = [&](uint32_t d_col, uint32_t own_col, uint32_t own_smem, uint32_t b_base) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int c = kk >> 2;
          const uint32_t ko = (kk & 3) * 32;
          const uint64_t bdesc = sdesc_sw128(b_base + c * (64 * 128) + ko, 16, 1024);
          if (Cfg::kOwnSmem)
            mma_ss(tmem + d_col, sdesc_sw128(own_smem + c * (128 * 128) + ko, 16, 1024), bdesc, idesc_first, kk > 0);
          else
            mma_ts(tmem + d_col, tmem + own_col + kk * 8, bdesc, idesc_first, kk > 0);
        }
      };
      // out += x (A, packed bf16 in the dP buffer) * streamed, over the block's 64 rows. The
      // two column halves of x were stored 32 columns apart (each warp inside its own columns).
      auto second = [&](uint32_t out_col, uint32_t x_col, uint32_t b_base, bool add) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(tmem + out_col, tmem + x_col + (kk >> 1) * 32 + (kk & 1) * 8,
                 sdesc_sw128(b_base + kk * 2048, 64 * 128, 1024), idesc_second, add || kk > 0);
      };
      bool ok = Cfg::kOwnSmem ? mbar_wait(&bar.own_full, 0, abort_flag, wait_limit_ns) : true;
      if (warp == 17) {
        RingPos<Cfg::kSBufs> buf;
        RingPos<Cfg::kS0> r;
        for (int j = 0; j < n_iter && ok; ++j) {
          ok = mbar_wait_spin(&bar.full0[r.i], r.phase, abort_flag, wait_limit_ns);
          ok = ok && mbar_wait_spin(&bar.s_free[buf.i], buf.phase ^ 1, abort_flag, wait_limit_ns);
          if (!ok) break;
          tc_fence_after();
          first(Cfg::kSCol + buf.i * 64, Cfg::kOwn0Col, smem_u32(s_own), smem_u32(s_ring0) + r.i * Cfg::kTile);
          tc_commit(&bar.s_full[buf.i]);
          buf.next();
          r.next();
        }
      } else {
        RingPos<Cfg::kDPBufs> db, pb;  // buffers of the next dP and of the next second products
        RingPos<Cfg::kS0> q0;
        RingPos<Cfg::kS1> r1, q1;
        // turn j: dP(j), then the second products of step j - kLag
        for (int j = 0; j < n_iter + Cfg::kLag && ok; ++j) {
          if (j < n_iter) {
            ok = mbar_wait_spin(&bar.full1[r1.i], r1.phase, abort_flag, wait_limit_ns);
            if (!ok) break;
            tc_fence_after();
            first(Cfg::kDPCol + db.i * 64, Cfg::kOwn1Col, smem_u32(s_own) + Cfg::kOwnTile,
                  smem_u32(s_ring1) + r1.i * Cfg::kTile);
            tc_commit(&bar.dp_full[db.i]);
            if (!KV) tc_commit(&bar.empty1[r1.i]);
            db.next();
            r1.next();
          }
          if (j >= Cfg::kLag) {
            ok = mbar_wait_spin(&bar.p_full[pb.i], pb.phase, abort_flag, wait_limit_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t x = Cfg::kDPCol + pb.i * 64;
            if (KV) second(D, x + 16, smem_u32(s_ring1) + q1.i * Cfg::kTile, j > Cfg::kLag);  // dV += P^T dO
            second(0, x, smem_u32(s_ring0) + q0.i * Cfg::kTile, j > Cfg::kLag);  // dK += dS^T Q, or dQ += dS K
            tc_commit(&bar.empty0[q0.i]);
            if (KV) tc_commit(&bar.empty1[q1.i]);
            pb.next();
            q0.next();
            q1.next();
          }
        }
        if (ok) tc_commit(&bar.out_full);
      }
      if (!ok) {
        report(dev_status, FVA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else {
    // ------------------------------------------------------------------ P and dS
    const int half = (warp & 3) >> 1, ch = part & 1, group = part >> 1;
    float nl_row = 0.0f, nd_row = 0.0f;  // KV = false: this row's -lse2 and -D
    if (!KV) {
      const bool in = 2 * t + (row >> 6) < nB;
      const float* st = stats + (static_cast<int64_t>(bh) * nB + 2 * t + (row >> 6)) * 128 + (row & 63);
      nl_row = in ? st[0] : -INFINITY;
      nd_row = in ? st[64] : 0.0f;
    }
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    ListReader entries(list, n_iter, lane);
    bool ok = true;
    RingPos<Cfg::kSBufs> sb;
    RingPos<Cfg::kDPBufs> db;
    RingPos<Cfg::kS0> stage;
    if (group == 1) {
      sb.next();
      db.next();
      stage.next();
    }
    for (int j = group; j < n_iter; j += 2) {
      const int entry = entries.get(j, lane);
      const int blk = entry >> 2;
      // (KV: these threads read the stage's statistics too, which S only implies have landed)
      if (!warp_wait_spin(&bar.s_full[sb.i], sb.phase, abort_flag, wait_limit_ns) ||
          (KV && !warp_wait_spin(&bar.full0[stage.i], stage.phase, abort_flag, wait_limit_ns))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_col = lane_base + Cfg::kSCol + sb.i * 64 + ch * 32;
      const uint32_t dp_col = lane_base + Cfg::kDPCol + db.i * 64 + ch * 32;
      const bool keep = (entry >> half) & 1;
      float p[32];
      if (keep) {
        uint32_t x[32];
        tmem_ld32(s_col, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.s_free[sb.i]);
        const ulonglong2* nl4 = reinterpret_cast<const ulonglong2*>(s_stats + stage.i * 512 + ch * 128);
        const uint64_t nlr = f2_pack(nl_row, nl_row);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const ulonglong2 nl = KV ? nl4[c / 4] : make_ulonglong2(nlr, nlr);
          const float2 a = f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, nl.x));
          const float2 b = f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc2, nl.y));
          p[c] = ex2_approx(a.x);
          p[c + 1] = ex2_approx(a.y);
          p[c + 2] = ex2_approx(b.x);
          p[c + 3] = ex2_approx(b.y);
        }
        if (!KV && blk == nB - 1) {  // keys past N: zero rows, not -inf scores
          const int nvalid = N - blk * 64 - ch * 32;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c >= nvalid) p[c] = 0.0f;
        }
      } else if (lane == 0) {
        mbar_arrive(&bar.s_free[sb.i]);
      }
      if (!warp_wait_spin(&bar.dp_full[db.i], db.phase, abort_flag, wait_limit_ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t w[16];
      if (keep) {
        uint32_t y[32];
        tmem_ld32(dp_col, y);
        if (KV) {
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
          tmem_st16(dp_col + 16, w);
        }
        const ulonglong2* nd4 = reinterpret_cast<const ulonglong2*>(s_stats + stage.i * 512 + 256 + ch * 128);
        const uint64_t ndr = f2_pack(nd_row, nd_row);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const ulonglong2 nd = KV ? nd4[c / 4] : make_ulonglong2(ndr, ndr);
          const float2 a = f2_unpack(f2_mul(f2_pack(p[c], p[c + 1]),
                                            f2_add(f2_pack(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), nd.x)));
          const float2 b = f2_unpack(f2_mul(f2_pack(p[c + 2], p[c + 3]),
                                            f2_add(f2_pack(__uint_as_float(y[c + 2]), __uint_as_float(y[c + 3])), nd.y)));
          w[c / 2] = pack_bf16x2(a.x, a.y);
          w[c / 2 + 1] = pack_bf16x2(b.x, b.y);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = 0u;
        if (KV) tmem_st16(dp_col + 16, w);
      }
      tmem_st16(dp_col, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[db.i]);
      sb.next();
      sb.next();
      db.next();
      db.next();
      stage.next();
      stage.next();
    }
    // ------------------------------------------------------------------ epilogue
    if (ok && n_iter > 0 && !warp_wait(&bar.out_full, 0, abort_flag, wait_limit_ns)) ok = false;
    if (!ok) {
      report(dev_status, FVA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    } else if (tile_ok) {
      tc_fence_after();
      // the outputs' columns (KV: dK, then dV) in pieces of 32, a quarter of them a part
      constexpr int kPieces = (KV ? 2 * D : D) / 32;
#pragma unroll
      for (int pc = part; pc < kPieces; pc += 4) {
        const bool second = KV && pc >= D / 32;
        const float f = second ? 1.0f : scale;
        uint32_t o[32];
        if (n_iter > 0) {
          tmem_ld32(lane_base + pc * 32, o);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
        if (grow < N) {
          uint4* dst = reinterpret_cast<uint4*>((second ? out1 : out0) + (static_cast<int64_t>(bh) * N + grow) * D +
                                                (second ? pc * 32 - D : pc * 32));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * i]) * f, __uint_as_float(o[8 * q + 2 * i + 1]) * f);
            dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (bar.abort) {  // products may be in flight that nobody waited for
    if (warp >= 17 && n_iter > 0 && elect_one()) {
      volatile int never = 0;
      tc_commit(&bar.drain[warp - 17]);
      mbar_wait(&bar.drain[warp - 17], 0, &never, 100000000ull);
    }
    __syncthreads();
  }
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, kBwdTmemCols);
  }
}

// Both passes in one launch: CTAs 0 .. tiles - 1 own key rows (the longer work), the others
// query rows, so the second pass fills the SMs that the first one's tail leaves idle.
template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmdo,
                       const __grid_constant__ BwdTcArgs x) {
  const int slot = static_cast<int>(blockIdx.x);
  grid_wait();
  if (slot < x.ntiles) bwd_tile<D, true>(x, tmk, tmv, tmq, tmdo, slot);
  else bwd_tile<D, false>(x, tmq, tmdo, tmk, tmv, slot - x.ntiles);
}

template <int D>
static cudaError_t launch_tc_d(const BwdTcArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                               const CUtensorMap& mdo, cudaStream_t st) {
  constexpr size_t kKv = bwd_smem_bytes<D, true>(), kQ = bwd_smem_bytes<D, false>(), smem = kKv > kQ ? kKv : kQ;
  const cudaError_t e = cudaFuncSetAttribute(attn_bwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_chained(attn_bwd_tc_kernel<D>, dim3(2 * static_cast<unsigned>(a.ntiles)), kBwdThreads, 0, smem, st, mq, mk,
                        mv, mdo, a);
}

cudaError_t launch_attn_bwd_tc(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const BwdScratch& ws,
                               const int32_t* worklist, int32_t* dev_status, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mdo;
  if (!make_rows_map(&mq, x.q, Dm.BH, Dm.N, Dm.d, false) || !make_rows_map(&mk, x.k, Dm.BH, Dm.N, Dm.d, false) ||
      !make_rows_map(&mv, x.v, Dm.BH, Dm.N, Dm.d, false) || !make_rows_map(&mdo, x.d_o, Dm.BH, Dm.N, Dm.d, false))
    return cudaErrorInvalidValue;
  using bf = __nv_bfloat16;
  const BwdTcArgs a = {static_cast<const bf*>(x.q), static_cast<const bf*>(x.k), static_cast<const bf*>(x.v),
                       static_cast<const bf*>(x.d_o), ws.stats, static_cast<bf*>(x.dq), static_cast<bf*>(x.dk),
                       static_cast<bf*>(x.dv), m->tile_ptr, m->tile_col, m->worklist, ws.lists, worklist,
                       static_cast<int>(Dm.tiles), static_cast<int>(Dm.N), static_cast<int>(Dm.nB),
                       static_cast<int>(Dm.nPairs), x.scale, x.scale * 1.4426950408889634f, attn_wait_limit_ns(),
                       attn_diag_flags(), dev_status};
  return Dm.d == 128 ? launch_tc_d<128>(a, mq, mk, mv, mdo, st) : launch_tc_d<64>(a, mq, mk, mv, mdo, st);
}

}  // namespace fva
