// Gradient of block-sparse attention: the parts that both element types share (transposed
// block lists, row statistics) and the CUDA-core kernel for fp32.
//
// With P = exp(scale Q K^T - lse) on the kept blocks:
//   dP = dO V^T,  dS = P (dP - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// The gradient runs as two passes over the kept blocks, one that owns query rows (dQ) and
// walks the rows' lists, one that owns key rows (dK, dV) and walks the transposed lists. Each
// output row has one owner, so nothing is summed with atomics and equal inputs give equal
// bits; the price is that Q K^T and dO V^T are computed twice (7 products instead of 5).
#include <math.h>

#include "fva_internal.cuh"

namespace fva {

// ---------------------------------------------------------------------------------
// Transposed lists: bit a of key row b = bit b of query row a
// ---------------------------------------------------------------------------------
// One warp per 32 x 32 bit tile: lane i holds query row 32 i0 + i's word, and 32 ballots
// give the 32 key rows' words.
__global__ void __launch_bounds__(256) transpose_bits_kernel(const uint32_t* __restrict__ bits, int nB, int nWords,
                                                             int64_t n_tiles, uint32_t* __restrict__ bits_t) {
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= n_tiles) return;
  const int64_t per_head = static_cast<int64_t>(nWords) * nWords;
  const int64_t bh = w / per_head;
  const int a0 = static_cast<int>((w - bh * per_head) / nWords), b0 = static_cast<int>((w - bh * per_head) % nWords);
  const int a = 32 * a0 + lane;
  const uint32_t word = a < nB ? bits[(bh * nB + a) * nWords + b0] : 0u;
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint32_t col = __ballot_sync(0xffffffffu, (word >> j) & 1u);
    if (lane == j) mine = col;
  }
  const int b = 32 * b0 + lane;
  if (b < nB) bits_t[(bh * nB + b) * nWords + a0] = mine;
}

// One warp per key row: how many query blocks keep it.
__global__ void __launch_bounds__(256) count_bits_kernel(const uint32_t* __restrict__ bits, int64_t rows, int nWords,
                                                         int32_t* __restrict__ cnt) {
  const int lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= rows) return;
  int n = 0;
  for (int k = lane; k < nWords; k += 32) n += __popc(bits[r * nWords + k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) cnt[r] = n;
}

// ---------------------------------------------------------------------------------
// Row statistics: -lse in log2 units and -D, D_i = sum_c dO_ic O_ic
// ---------------------------------------------------------------------------------
// d * sizeof(T) / 16 lanes per row, 16 bytes each; a row without keys (lse = -inf) and the rows
// past N of the last block get -infinity and 0, so that their P is 0.
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

template <typename T, int D>
__global__ void __launch_bounds__(256) row_stats_kernel(const T* __restrict__ o, const T* __restrict__ d_o,
                                                        const float* __restrict__ lse, int64_t rows, int N, int nB,
                                                        float* __restrict__ stats) {
  constexpr int kLanes = D * static_cast<int>(sizeof(T)) / 16;  // 8, 16 or 32
  const int64_t r = (blockIdx.x * 256ll + threadIdx.x) / kLanes;  // row of the padded [BH, nB * 64]
  const int l = threadIdx.x % kLanes;
  const int64_t bh = r / (static_cast<int64_t>(nB) * kBlock);
  const int64_t n = r - bh * nB * kBlock;
  const bool in = r < rows && n < N;
  float s = 0.0f;
  if (in) {
    const int64_t at = (bh * N + n) * kLanes + l;
    s = dot16(reinterpret_cast<const uint4*>(o)[at], reinterpret_cast<const uint4*>(d_o)[at], T());
  }
#pragma unroll
  for (int k = kLanes / 2; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  if (l == 0 && r < rows) {
    const float x = in ? lse[bh * N + n] : -INFINITY;
    float* out = stats + (r / kBlock) * 128 + r % kBlock;
    out[0] = x == -INFINITY ? -INFINITY : -1.4426950408889634f * x;
    out[64] = -s;
  }
}

// ---------------------------------------------------------------------------------
// CUDA-core gradient
// ---------------------------------------------------------------------------------
// One CTA owns one 64-row block and streams the blocks of its list through shared memory.
//   KV = false: owns query rows (a0 = Q, a1 = dO), streams K and V:  out0 = dQ = scale dS K
//   KV = true:  owns key rows   (a0 = K, a1 = V), streams Q and dO:  out0 = dK = scale dS^T Q,
//                                                                     out1 = dV = P^T dO
// Both form X = a0 b0^T and Y = a1 b1^T (scores and dP, transposed when KV), 4 x 4 values a
// thread, then accumulate out0 += dS b0 (and out1 += P b1) from the 64 x 64 tiles.
template <int D, bool KV>
__global__ void __launch_bounds__(256) attn_bwd_f32_kernel(const float* __restrict__ a0, const float* __restrict__ a1,
                                                           const float* __restrict__ b0, const float* __restrict__ b1,
                                                           const float* __restrict__ stats,
                                                           const int32_t* __restrict__ tile_ptr,
                                                           const int32_t* __restrict__ tile_col,
                                                           float* __restrict__ out0, float* __restrict__ out1, int N,
                                                           int nB, int nPairs, float scale, int32_t* dev_status) {
  constexpr int LD = D + 4, LP = kBlock + 1, NC = D / 16;
  extern __shared__ __align__(16) float smem_bwd[];
  float* sA0 = smem_bwd;
  float* sA1 = sA0 + kBlock * LD;
  float* sB0 = sA1 + kBlock * LD;
  float* sB1 = sB0 + kBlock * LD;
  float* sP = sB1 + kBlock * LD;  // only used when KV
  float* sDS = sP + kBlock * LP;
  float* sL = sDS + kBlock * LP;
  float* sD = sL + kBlock;
  const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15;
  const int a = blockIdx.x;
  const int64_t bh = blockIdx.y;
  const int64_t base = bh * N;
  const int64_t tile = bh * nPairs + (a >> 1);
  const int half = a & 1;
  const float scale_log2 = scale * 1.4426950408889634f;

  auto load = [&](float* dst, const float* src, int block) {
    for (int i = tid; i < kBlock * D; i += 256) {
      const int r = i / D, c = i % D;
      const int n = block * kBlock + r;
      dst[r * LD + c] = n < N ? src[(base + n) * D + c] : 0.0f;
    }
  };
  auto load_rows = [&](int block) {
    if (tid < kBlock) {
      const float* st = stats + (bh * nB + block) * 128 + tid;
      sL[tid] = st[0];
      sD[tid] = st[64];
    }
  };
  load(sA0, a0, a);
  load(sA1, a1, a);
  if (!KV) load_rows(a);
  float acc0[4][NC], acc1[4][NC];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) acc0[i][j] = acc1[i][j] = 0.0f;

  const int lo = tile_ptr[tile], hi = tile_ptr[tile + 1];
  for (int e = lo; e < hi; ++e) {
    const int entry = tile_col[e];
    if (!((entry >> half) & 1)) continue;  // uniform over the CTA
    const int blk = entry >> 2;
    if (blk < 0 || blk >= nB) {
      if (tid == 0) report(dev_status, FVA_DEVERR_BAD_LIST);
      continue;
    }
    __syncthreads();
    load(sB0, b0, blk);
    load(sB1, b1, blk);
    if (KV) load_rows(blk);
    __syncthreads();
    float x[4][4], y[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = y[i][j] = 0.0f;
    for (int c = 0; c < D; c += 4) {
      float4 u0[4], u1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u0[i] = *reinterpret_cast<const float4*>(sA0 + (tr + 16 * i) * LD + c);
        u1[i] = *reinterpret_cast<const float4*>(sA1 + (tr + 16 * i) * LD + c);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w0 = *reinterpret_cast<const float4*>(sB0 + (tc + 16 * j) * LD + c);
        const float4 w1 = *reinterpret_cast<const float4*>(sB1 + (tc + 16 * j) * LD + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i][j] = fmaf(u0[i].x, w0.x, fmaf(u0[i].y, w0.y, fmaf(u0[i].z, w0.z, fmaf(u0[i].w, w0.w, x[i][j]))));
          y[i][j] = fmaf(u1[i].x, w1.x, fmaf(u1[i].y, w1.y, fmaf(u1[i].z, w1.z, fmaf(u1[i].w, w1.w, y[i][j]))));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = tr + 16 * i, s = tc + 16 * j;
        const int qi = KV ? s : r, key = (KV ? a : blk) * kBlock + (KV ? r : s);
        // keys past N hold zero scores, not -inf: their weight is forced to 0
        const float p = key < N ? exp2f(fmaf(x[i][j], scale_log2, sL[qi])) : 0.0f;
        if (KV) sP[r * LP + s] = p;
        sDS[r * LP + s] = p * (y[i][j] + sD[qi]);
      }
    }
    __syncthreads();
    for (int s = 0; s < kBlock; ++s) {
      float w0[NC], w1[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        w0[j] = sB0[s * LD + tc + 16 * j];
        if (KV) w1[j] = sB1[s * LD + tc + 16 * j];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ds = sDS[(tr + 16 * i) * LP + s];
        const float p = KV ? sP[(tr + 16 * i) * LP + s] : 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          acc0[i][j] = fmaf(ds, w0[j], acc0[i][j]);
          if (KV) acc1[i][j] = fmaf(p, w1[j], acc1[i][j]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = a * kBlock + tr + 16 * i;
    if (n >= N) continue;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      out0[(base + n) * D + tc + 16 * j] = acc0[i][j] * scale;
      if (KV) out1[(base + n) * D + tc + 16 * j] = acc1[i][j];
    }
  }
}

template <int D, bool KV>
static cudaError_t launch_f32_t(const Dims& Dm, const void* a0, const void* a1, const void* b0, const void* b1,
                                const float* stats, const fva_mask* m, void* out0, void* out1, float scale,
                                int32_t* dev_status, cudaStream_t st) {
  const size_t smem = sizeof(float) * (4 * kBlock * (D + 4) + 2 * kBlock * (kBlock + 1) + 2 * kBlock);
  const cudaError_t e = cudaFuncSetAttribute(attn_bwd_f32_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(Dm.nB), static_cast<unsigned>(Dm.BH));
  attn_bwd_f32_kernel<D, KV><<<grid, 256, smem, st>>>(
      static_cast<const float*>(a0), static_cast<const float*>(a1), static_cast<const float*>(b0),
      static_cast<const float*>(b1), stats, m->tile_ptr, m->tile_col, static_cast<float*>(out0),
      static_cast<float*>(out1), static_cast<int>(Dm.N), static_cast<int>(Dm.nB), static_cast<int>(Dm.nPairs), scale,
      dev_status);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_f32_d(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const BwdScratch& ws,
                                int32_t* dev_status, cudaStream_t st) {
  const cudaError_t e = launch_f32_t<D, true>(Dm, x.k, x.v, x.q, x.d_o, ws.stats, &ws.mask_t, x.dk, x.dv, x.scale,
                                              dev_status, st);
  if (e != cudaSuccess) return e;
  return launch_f32_t<D, false>(Dm, x.q, x.d_o, x.k, x.v, ws.stats, m, x.dq, nullptr, x.scale, dev_status, st);
}

template <typename T, int D>
static cudaError_t launch_stats(const Dims& Dm, const BwdArgs& x, float* stats, cudaStream_t st) {
  const int64_t rows = Dm.rows * kBlock, per_cta = 256 * 16 / (D * static_cast<int>(sizeof(T)));
  row_stats_kernel<T, D><<<static_cast<unsigned>((rows + per_cta - 1) / per_cta), 256, 0, st>>>(
      static_cast<const T*>(x.o), static_cast<const T*>(x.d_o), x.lse, rows, static_cast<int>(Dm.N),
      static_cast<int>(Dm.nB), stats);
  return cudaGetLastError();
}

// The transposed mask's tile lists (tiles of two key blocks over the union of the query
// blocks that keep them) and work list, longest first within a head.
static cudaError_t launch_transposed_lists(const Dims& Dm, const fva_mask* m, const BwdScratch& ws,
                                           int32_t* dev_status, cudaStream_t st) {
  cudaError_t e = launch_csr_to_bits(Dm, m, ws.bits, dev_status, st);
  if (e != cudaSuccess) return e;
  const int64_t n = Dm.BH * Dm.nWords * Dm.nWords;
  transpose_bits_kernel<<<static_cast<unsigned>((n + 7) / 8), 256, 0, st>>>(
      ws.bits, static_cast<int>(Dm.nB), static_cast<int>(Dm.nWords), n, ws.route_t.bits);
  count_bits_kernel<<<static_cast<unsigned>((Dm.rows + 7) / 8), 256, 0, st>>>(
      ws.route_t.bits, Dm.rows, static_cast<int>(Dm.nWords), ws.route_t.row_cnt);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_tiles_from_bits(Dm, &ws.mask_t, FVA_ORDER_HEAD_LPT, ws.route_t, ws.route_t.row_cnt, 0, dev_status, st);
}

cudaError_t launch_attn_bwd(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const BwdScratch& ws,
                            int32_t* dev_status, cudaStream_t st) {
  cudaError_t e = launch_transposed_lists(Dm, m, ws, dev_status, st);
  if (e != cudaSuccess) return e;
  if (Dm.esize == 2) {
    e = Dm.d == 128 ? launch_stats<__nv_bfloat16, 128>(Dm, x, ws.stats, st)
                    : launch_stats<__nv_bfloat16, 64>(Dm, x, ws.stats, st);
    return e != cudaSuccess ? e : launch_attn_bwd_tc(Dm, x, m, &ws.mask_t, ws.stats, dev_status, st);
  }
  switch (Dm.d) {
    case 32:
      e = launch_stats<float, 32>(Dm, x, ws.stats, st);
      return e != cudaSuccess ? e : launch_f32_d<32>(Dm, x, m, ws, dev_status, st);
    case 64:
      e = launch_stats<float, 64>(Dm, x, ws.stats, st);
      return e != cudaSuccess ? e : launch_f32_d<64>(Dm, x, m, ws, dev_status, st);
    default:
      e = launch_stats<float, 128>(Dm, x, ws.stats, st);
      return e != cudaSuccess ? e : launch_f32_d<128>(Dm, x, m, ws, dev_status, st);
  }
}

}  // namespace fva
