// Gradient of block-sparse attention: the parts that both element types share (transposed
// block lists, row statistics) and the CUDA-core kernel for fp32.
//
// With P = exp(scale Q K^T - lse) on the kept blocks:
//   dP = dO V^T,  dS = P (dP - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// The gradient runs as two passes over the kept blocks, one that owns query rows (dQ) and
// walks the rows' lists, one that owns key rows (dK, dV) and walks the transposed lists. Each
// output row has one owner, so nothing is summed with atomics and equal inputs give equal
// bits; the price is that Q K^T and dO V^T are computed twice (7 products instead of 5). Both
// passes are one launch.
#include <cooperative_groups.h>
#include <math.h>

#include "fva_internal.cuh"

namespace fva {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------------
// Transposed lists and row statistics
// ---------------------------------------------------------------------------------
// One launch: the first CTAs build lists, the others statistics.
//
// Lists: a CTA has 64 key blocks of one (b, h) as bit rows in shared memory (bit a of row b:
// query block a keeps key block b), reads the head's whole CSR, four rows and up to 128 entries
// of each at a time, and writes the lists of its 32 tiles (pairs of key blocks): ascending, the
// entry's low bits saying which of the two keep the query block, as in tile_col. Tile t's list
// starts at t * nB, so no counts have to be summed first.
//
// Statistics: -lse in log2 units and -D, D_i = sum_c dO_ic O_ic, 64 rows as one 512-byte piece.
// d * sizeof(T) / 16 lanes per row, 16 bytes each; a row without keys (lse = -inf) and the rows
// past N of the last block get -infinity and 0, so that their P is 0. O is the stored one, of a
// bf16 layer rounded to bf16: that moves dQ and dK by 2e-4 of their norm, the rounding of dS by
// 1.7e-3.
//
// Bound by the CSR's reads, once per 64 key blocks: 77 us of 9 ms (21 x 30 x 52 tokens, 16 heads,
// a quarter of the blocks), 7 us at 2 x 6 heads of 612 tokens.
constexpr int kPrepThreads = 512;
constexpr int kListRows = 64, kStatRows = 4;

__device__ __forceinline__ float dot16(const uint4& a, const uint4& b, float) {
  const float* x = reinterpret_cast<const float*>(&a);
  const float* y = reinterpret_cast<const float*>(&b);
  return fmaf(x[0], y[0], fmaf(x[1], y[1], fmaf(x[2], y[2], x[3] * y[3])));
}
__device__ __forceinline__ float dot16(const uint4& a, const uint4& b, __nv_bfloat16) {
  const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&a);
  const __nv_bfloat162* y = reinterpret_cast<const __nv_bfloat162*>(&b);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = __bfloat1622float2(x[i]), v = __bfloat1622float2(y[i]);
    s = fmaf(u.x, v.x, fmaf(u.y, v.y, s));
  }
  return s;
}

__device__ void build_lists(int chunk, int bh, const int32_t* __restrict__ row_ptr, const int32_t* __restrict__ col_idx,
                            int nB, int nWords, int nPairs, const BwdLists& out, uint32_t* bits, int32_t* dev_status) {
  constexpr int kWarps = kPrepThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = chunk * kListRows;
  for (int i = tid; i < kListRows * nWords; i += kPrepThreads) bits[i] = 0u;
  __syncthreads();
  auto set = [&](int a, int c) {
    if (c < 0 || c >= nB) report(dev_status, FVA_DEVERR_BAD_LIST);
    else if (c >= c0 && c < c0 + kListRows) atomicOr(&bits[(c - c0) * nWords + (a >> 5)], 1u << (a & 31));
  };
  for (int a0 = warp * 4; a0 < nB; a0 += kWarps * 4) {
    const int64_t r0 = static_cast<int64_t>(bh) * nB;
    const int p = a0 + lane <= nB && lane < 5 ? row_ptr[r0 + a0 + lane] : 0;
    int lo[4], hi[4], most = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      lo[r] = __shfl_sync(0xffffffffu, p, r);
      hi[r] = __shfl_sync(0xffffffffu, p, r + 1);
      if (a0 + r >= nB) hi[r] = lo[r] = 0;
      most = max(most, hi[r] - lo[r]);
    }
    for (int off = lane; off - lane < most; off += 128) {
      int c[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) c[r][k] = lo[r] + off + k * 32 < hi[r] ? col_idx[lo[r] + off + k * 32] : -1;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (lo[r] + off + k * 32 < hi[r]) set(a0 + r, c[r][k]);
    }
  }
  __syncthreads();
  const uint32_t below = (1u << lane) - 1u;
  for (int t = warp; t < kListRows / 2; t += kWarps) {
    const int pair = chunk * (kListRows / 2) + t;
    if (pair >= nPairs) break;
    const int64_t tile = static_cast<int64_t>(bh) * nPairs + pair;
    int32_t* list = out.col + tile * nB;
    const uint32_t* wa = bits + 2 * t * nWords;
    const uint32_t* wb = wa + nWords;  // past the last key block: all 0
    int n = 0;
    for (int k = 0; k < nWords; ++k) {
      const uint32_t a = wa[k], b = wb[k], u = a | b;
      if ((u >> lane) & 1u)
        list[n + __popc(u & below)] = ((32 * k + lane) << 2) | static_cast<int>((a >> lane) & 1u) |
                                      (static_cast<int>((b >> lane) & 1u) << 1);
      n += __popc(u);
    }
    if (lane == 0) out.cost[tile] = n;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const int32_t* __restrict__ row_ptr,
                                                               const int32_t* __restrict__ col_idx, int nB, int nWords,
                                                               int nPairs, int chunks, int list_ctas, BwdLists lists,
                                                               const T* __restrict__ o, const T* __restrict__ d_o,
                                                               const float* __restrict__ lse, int64_t rows, int N,
                                                               float* __restrict__ stats, int32_t* dev_status) {
  extern __shared__ uint32_t bits[];  // [kListRows][nWords]
  grid_wait();
  grid_release();
  if (static_cast<int>(blockIdx.x) < list_ctas) {
    build_lists(blockIdx.x % chunks, blockIdx.x / chunks, row_ptr, col_idx, nB, nWords, nPairs, lists, bits, dev_status);
    return;
  }
  // four rows a thread, their loads all on the way before the first is used
  constexpr int kLanes = D * static_cast<int>(sizeof(T)) / 16;  // 8, 16 or 32
  constexpr int kRowsAtOnce = kPrepThreads / kLanes;
  const int l = threadIdx.x % kLanes;
  const int64_t first = static_cast<int64_t>(blockIdx.x - list_ctas) * (kStatRows * kRowsAtOnce) + threadIdx.x / kLanes;
  uint4 x[kStatRows], y[kStatRows];
  int64_t at[kStatRows];  // row of [BH, N]; -1: past N
#pragma unroll
  for (int k = 0; k < kStatRows; ++k) {
    const int64_t r = first + k * kRowsAtOnce, bh = r / (static_cast<int64_t>(nB) * kBlock), n = r - bh * nB * kBlock;
    at[k] = r < rows && n < N ? bh * N + n : -1;
    if (at[k] >= 0) {
      x[k] = reinterpret_cast<const uint4*>(o)[at[k] * kLanes + l];
      y[k] = reinterpret_cast<const uint4*>(d_o)[at[k] * kLanes + l];
    }
  }
#pragma unroll
  for (int k = 0; k < kStatRows; ++k) {
    const int64_t r = first + k * kRowsAtOnce;
    float s = at[k] >= 0 ? dot16(x[k], y[k], T()) : 0.0f;
#pragma unroll
    for (int i = kLanes / 2; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    if (l == 0 && r < rows) {
      const float e = at[k] >= 0 ? lse[at[k]] : -INFINITY;
      float* out = stats + (r / kBlock) * 128 + r % kBlock;
      out[0] = e == -INFINITY ? -INFINITY : -1.4426950408889634f * e;
      out[64] = -s;
    }
  }
}

// Order of the transposed tiles: head by head, the longest list first. One CTA per head.
__global__ void __launch_bounds__(512) order_kernel(const int32_t* __restrict__ cost, int nPairs,
                                                    int32_t* __restrict__ worklist) {
  extern __shared__ int32_t sc[];
  grid_wait();
  grid_release();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * nPairs;
  for (int i = threadIdx.x; i < nPairs; i += 512) sc[i] = cost[base + i];
  __syncthreads();
  for (int t = threadIdx.x; t < nPairs; t += 512) {
    const int32_t ct = sc[t];
    int r = 0;
    for (int i = 0; i < nPairs; ++i) r += (sc[i] > ct) || (sc[i] == ct && i < t);
    worklist[base + r] = static_cast<int32_t>(base + t);
  }
}

// ---------------------------------------------------------------------------------
// CUDA-core gradient
// ---------------------------------------------------------------------------------
// A cluster of four CTAs owns 32 rows (half a block) and takes the blocks of its list in turn, so
// that a small layer has CTAs for every SM and its longest list is a quarter as long; their sums
// are added in the first's order at the end. Blocks stream through two shared-memory buffers.
//   KV = false: owns query rows (a0 = Q, a1 = dO), streams K and V:  out0 = dQ = scale dS K
//   KV = true:  owns key rows   (a0 = K, a1 = V), streams Q and dO:  out0 = dK = scale dS^T Q,
//                                                                     out1 = dV = P^T dO
// Warps 0-3 form X = a0 b0^T and P, warps 4-7 Y = a1 b1^T and dS (scores and dP, transposed when
// KV), 4 x 4 values a thread; then the two groups accumulate P b1 and dS b0 (KV) or half of the
// block's rows of dS b0 each, 4 rows x D / 16 channels a thread. Measured (4 x 16 x 16 tokens, 2
// heads, d = 64, 0.4 of the blocks): 47 us, 49 with the preparation; FMA pipes 31% and shared memory
// 40% of the time; what bounds it are a step's three barriers with two CTAs an SM, and the last CTAs.
// Tried, with the preparation: 8 x 8 values a thread 53; one stream buffer and three CTAs 53; packed
// FMAs the same.
struct F32Args {
  const float *q, *k, *v, *d_o, *stats;
  float *dq, *dk, *dv;
};
constexpr int kF32Rows = 32, kF32Split = 4;

template <int D>
struct F32Cfg {
  static constexpr int kLD = D + 4, kLP = kBlock + 4;  // row strides: 16-byte pieces fall into different banks
  static constexpr int kA = kF32Rows * kLD, kB = kBlock * kLD, kP = kF32Rows * kLP;
  static constexpr int kSmem = 4 * (2 * kA + 4 * kB + 2 * kP + 4 * kBlock);
  static_assert(2 * kF32Rows * D <= 4 * kB, "the sums of both groups fit the stream's buffers");
};

template <int D, bool KV>
__device__ __forceinline__ void bwd_f32(const F32Args& x, int64_t bh, int own, const int32_t* list, int n_list, int N,
                                        int nB, float scale, float* smem, int32_t* dev_status) {
  using Cfg = F32Cfg<D>;
  constexpr int LD = Cfg::kLD, LP = Cfg::kLP, NC = D / 16;
  constexpr int kW = NC >= 4 ? 4 : NC, kG = NC / kW;  // channels of a vector, vectors of a thread
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  float* sA0 = smem;
  float* sA1 = sA0 + Cfg::kA;
  float* sB = sA1 + Cfg::kA;        // two buffers of b0, b1
  float* sP = sB + 4 * Cfg::kB;
  float* sDS = sP + Cfg::kP;
  float* sStat = sDS + Cfg::kP;     // two buffers of -lse2, -D (64 each)
  const int tid = threadIdx.x, group = tid >> 7, tr = (tid & 127) >> 4, tc = tid & 15;
  const int block = own / (kBlock / kF32Rows), r0 = own * kF32Rows, half = block & 1;
  const int64_t base = bh * N;
  const float *a0 = KV ? x.k : x.q, *a1 = KV ? x.v : x.d_o, *b0 = KV ? x.q : x.k, *b1 = KV ? x.d_o : x.v;

  auto load = [&](float* dst, const float* src, int row, int rows) {
    for (int i = tid; i < rows * (D / 4); i += 256) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      const bool in = row + r < N;
      copy16(dst + r * LD + c, src + (base + (in ? row + r : 0)) * D + c, in);
    }
  };
  auto load_stats = [&](float* dst, int blk) {
    if (tid < 32) copy16(dst + 4 * tid, x.stats + (bh * nB + blk) * 128 + 4 * tid, true);
  };
  int nth = 0;  // kept entries so far: this CTA takes every fourth
  auto next_of = [&](int e) {
    for (; e < n_list; ++e) {
      const int entry = list[e];
      if (!((entry >> half) & 1)) continue;
      if ((entry >> 2) < 0 || (entry >> 2) >= nB) {
        if (tid == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
        continue;
      }
      if (nth++ % kF32Split == rank) break;
    }
    return e;
  };
  auto fetch = [&](int e, int buf) {
    if (e < n_list) {
      const int blk = list[e] >> 2;
      load(sB + buf * 2 * Cfg::kB, b0, blk * kBlock, kBlock);
      load(sB + buf * 2 * Cfg::kB + Cfg::kB, b1, blk * kBlock, kBlock);
      if (KV) load_stats(sStat + buf * 128, blk);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int e = next_of(0);
  if (rank > 0 && e >= n_list) return;  // nothing to add: its SM takes another CTA
  load(sA0, a0, r0, kF32Rows);
  load(sA1, a1, r0, kF32Rows);
  if (!KV) load_stats(sStat, block);
  float acc[4][NC];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[i][j] = 0.0f;
  const float scale_log2 = scale * 1.4426950408889634f;

  fetch(e, 0);
  for (int buf = 0; e < n_list; buf ^= 1) {
    const int blk = list[e] >> 2;
    const int following = next_of(e + 1);
    fetch(following, buf ^ 1);  // (its last readers are behind the barrier that ended the step before)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float* sB0 = sB + buf * 2 * Cfg::kB;
    const float* sB1 = sB0 + Cfg::kB;
    const float* st = sStat + (KV ? buf * 128 : (block * kBlock == r0 ? 0 : kF32Rows));
    const float* pa = (group == 0 ? sA0 : sA1) + tr * LD;
    const float* pb = (group == 0 ? sB0 : sB1) + tc * LD;
    float u[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) u[i][j] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(pa + 8 * i * LD + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w = *reinterpret_cast<const float4*>(pb + 16 * j * LD + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i][j] = fmaf(a[i].x, w.x, fmaf(a[i].y, w.y, fmaf(a[i].z, w.z, fmaf(a[i].w, w.w, u[i][j]))));
      }
    }
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = tr + 8 * i, s = tc + 16 * j, key = KV ? r0 + r : blk * kBlock + s;
          // keys past N hold zero scores, not -inf: their weight is forced to 0
          sP[r * LP + s] = key < N ? exp2f(fmaf(u[i][j], scale_log2, st[KV ? s : r])) : 0.0f;
        }
    }
    __syncthreads();
    if (group == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = tr + 8 * i, s = tc + 16 * j;
          sDS[r * LP + s] = sP[r * LP + s] * (u[i][j] + st[64 + (KV ? s : r)]);
        }
    }
    __syncthreads();
    const float* px = (KV && group == 0 ? sP : sDS) + tr * LP;
    const float* pw = KV && group == 0 ? sB1 : sB0;
    const int s0 = KV ? 0 : group * (kBlock / 2), s1 = KV ? kBlock : s0 + kBlock / 2;
#pragma unroll 4
    for (int s = s0; s < s1; s += 4) {
      float4 d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<const float4*>(px + 8 * i * LP + s);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          float w[kW];
          const float* at = pw + (s + k) * LD + (g * 16 + tc) * kW;
          if constexpr (kW == 4) *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(at);
          else *reinterpret_cast<float2*>(w) = *reinterpret_cast<const float2*>(at);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y = reinterpret_cast<const float*>(&d[i])[k];
#pragma unroll
            for (int j = 0; j < kW; ++j) acc[i][g * kW + j] = fmaf(y, w[j], acc[i][g * kW + j]);
          }
        }
      }
    }
    __syncthreads();
    e = following;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  // every CTA leaves its sums in the stream's buffers as [2][32][D] (KV: dV and dK; else dQ of the
  // groups), and the CTAs add a share of them each
  float* sum = sB + group * kF32Rows * D;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) sum[(tr + 8 * i) * D + ((j / kW) * 16 + tc) * kW + j % kW] = acc[i][j];
  cluster.sync();
  const int active = min(max(nth, 1), kF32Split);  // the list has been read to its end
  constexpr int kHalf = kF32Rows * D / 4;          // 16-byte pieces of a group
  for (int at = rank * 256 + tid; at < (KV ? 2 : 1) * kHalf; at += active * 256) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float4 x) {
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    };
#pragma unroll
    for (int r = 0; r < kF32Split; ++r) {
      if (r < active) {
        const float4* far = reinterpret_cast<const float4*>(cluster.map_shared_rank(sB, r));
        add(far[at]);
        if (!KV) add(far[kHalf + at]);
      }
    }
    const bool second = KV && at >= kHalf;
    const int in = second ? at - kHalf : at;
    const float f = KV && !second ? 1.0f : scale;
    float* out = KV ? (second ? x.dk : x.dv) : x.dq;
    if (r0 + in / (D / 4) < N)
      reinterpret_cast<float4*>(out + (base + r0) * D)[in] = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
  cluster.sync();  // nobody leaves while its buffers are read
}

// Clusters of a head: those of the key rows, then those of the query rows.
template <int D>
__global__ void __launch_bounds__(256)
    attn_bwd_f32_kernel(F32Args x, const int32_t* __restrict__ tile_ptr, const int32_t* __restrict__ tile_col,
                        BwdLists lists, int N, int nB, int nPairs, int owners, float scale, int32_t* dev_status) {
  extern __shared__ __align__(16) float smem_bwd[];
  grid_wait();
  const int at_x = static_cast<int>(blockIdx.x) / kF32Split;
  const bool kv = at_x < owners;
  const int own = at_x - (kv ? 0 : owners);
  const int64_t bh = blockIdx.y, tile = bh * nPairs + own / (2 * kBlock / kF32Rows);
  if (kv) {
    bwd_f32<D, true>(x, bh, own, lists.col + tile * nB, lists.cost[tile], N, nB, scale, smem_bwd, dev_status);
  } else {
    const int at = tile_ptr[tile];
    bwd_f32<D, false>(x, bh, own, tile_col + at, tile_ptr[tile + 1] - at, N, nB, scale, smem_bwd, dev_status);
  }
}

template <int D>
static cudaError_t launch_f32(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const BwdScratch& ws,
                              int32_t* dev_status, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(attn_bwd_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             F32Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  const F32Args a = {static_cast<const float*>(x.q),   static_cast<const float*>(x.k), static_cast<const float*>(x.v),
                     static_cast<const float*>(x.d_o), ws.stats,                       static_cast<float*>(x.dq),
                     static_cast<float*>(x.dk),        static_cast<float*>(x.dv)};
  const int owners = static_cast<int>((Dm.N + kF32Rows - 1) / kF32Rows);
  return launch_chained(attn_bwd_f32_kernel<D>, dim3(static_cast<unsigned>(2 * kF32Split * owners), static_cast<unsigned>(Dm.BH)),
                        256, kF32Split, F32Cfg<D>::kSmem, st, a, m->tile_ptr, m->tile_col, ws.lists, static_cast<int>(Dm.N),
                        static_cast<int>(Dm.nB), static_cast<int>(Dm.nPairs), owners, x.scale, dev_status);
}

template <typename T, int D>
static cudaError_t launch_prepare(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const BwdScratch& ws,
                                  int32_t* dev_status, cudaStream_t st) {
  const int chunks = static_cast<int>((Dm.nB + kListRows - 1) / kListRows);
  const int64_t list_ctas = chunks * Dm.BH, rows = Dm.rows * kBlock;
  const int64_t per_cta = kStatRows * kPrepThreads * 16 / (D * static_cast<int>(sizeof(T)));
  const size_t smem = static_cast<size_t>(kListRows) * Dm.nWords * 4;
  const cudaError_t e = cudaFuncSetAttribute(prepare_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_chained(prepare_kernel<T, D>, dim3(static_cast<unsigned>(list_ctas + (rows + per_cta - 1) / per_cta)),
                        kPrepThreads, 0, smem, st, m->row_ptr, m->col_idx, static_cast<int>(Dm.nB),
                        static_cast<int>(Dm.nWords), static_cast<int>(Dm.nPairs), chunks, static_cast<int>(list_ctas),
                        ws.lists, static_cast<const T*>(x.o), static_cast<const T*>(x.d_o), x.lse, rows,
                        static_cast<int>(Dm.N), ws.stats, dev_status);
}

cudaError_t launch_attn_bwd(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const BwdScratch& ws,
                            int32_t* dev_status, cudaStream_t st) {
  cudaError_t e;
  if (Dm.esize == 4) {
    switch (Dm.d) {
      case 32:
        e = launch_prepare<float, 32>(Dm, x, m, ws, dev_status, st);
        return e != cudaSuccess ? e : launch_f32<32>(Dm, x, m, ws, dev_status, st);
      case 64:
        e = launch_prepare<float, 64>(Dm, x, m, ws, dev_status, st);
        return e != cudaSuccess ? e : launch_f32<64>(Dm, x, m, ws, dev_status, st);
      default:
        e = launch_prepare<float, 128>(Dm, x, m, ws, dev_status, st);
        return e != cudaSuccess ? e : launch_f32<128>(Dm, x, m, ws, dev_status, st);
    }
  }
  e = Dm.d == 128 ? launch_prepare<__nv_bfloat16, 128>(Dm, x, m, ws, dev_status, st)
                  : launch_prepare<__nv_bfloat16, 64>(Dm, x, m, ws, dev_status, st);
  if (e != cudaSuccess) return e;
  // where every tile is resident at once (one CTA an SM) their order does not matter
  const bool ordered = 2 * Dm.tiles > 148;
  if (ordered) {
    const size_t smem = static_cast<size_t>(Dm.nPairs) * 4;
    e = cudaFuncSetAttribute(order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    e = launch_chained(order_kernel, dim3(static_cast<unsigned>(Dm.BH)), 512, 0, smem, st, ws.lists.cost,
                       static_cast<int>(Dm.nPairs), ws.worklist);
    if (e != cudaSuccess) return e;
  }
  return launch_attn_bwd_tc(Dm, x, m, ws, ordered ? ws.worklist : nullptr, dev_status, st);
}

}  // namespace fva
