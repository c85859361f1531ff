// Gradient of block-sparse attention: the parts that every element type shares (transposed
// block lists, D = rowsum(dO O)) and the CUDA-core gradient kernel.
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
// D_i = sum_c dO_ic O_ic: one warp per row
// ---------------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* o) { *o = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* o) { *o = __float2bfloat16(x); }

template <typename T>
__global__ void __launch_bounds__(256) row_dot_kernel(const T* __restrict__ o, const T* __restrict__ d_o, int64_t rows,
                                                      int d, float* __restrict__ delta) {
  const int lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= rows) return;
  float s = 0.0f;
  for (int c = lane; c < d; c += 32) s = fmaf(to_f32(o[r * d + c]), to_f32(d_o[r * d + c]), s);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  if (lane == 0) delta[r] = s;
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
template <typename T, int D, bool KV>
__global__ void __launch_bounds__(256) attn_bwd_kernel(const T* __restrict__ a0, const T* __restrict__ a1,
                                                       const T* __restrict__ b0, const T* __restrict__ b1,
                                                       const float* __restrict__ lse, const float* __restrict__ delta,
                                                       const int32_t* __restrict__ tile_ptr,
                                                       const int32_t* __restrict__ tile_col, T* __restrict__ out0,
                                                       T* __restrict__ out1, int N, int nB, int nPairs, float scale,
                                                       int32_t* dev_status) {
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

  auto load = [&](float* dst, const T* src, int block) {
    for (int i = tid; i < kBlock * D; i += 256) {
      const int r = i / D, c = i % D;
      const int n = block * kBlock + r;
      dst[r * LD + c] = n < N ? to_f32(src[(base + n) * D + c]) : 0.0f;
    }
  };
  auto load_rows = [&](int block) {
    if (tid < kBlock) {
      const int n = block * kBlock + tid;
      // a row without keys (lse = -inf) and a row past N contribute nothing
      const float l = n < N ? lse[base + n] : INFINITY;
      sL[tid] = l == -INFINITY ? INFINITY : l;
      sD[tid] = n < N ? delta[base + n] : 0.0f;
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
        const float p = key < N ? expf(x[i][j] * scale - sL[qi]) : 0.0f;
        if (KV) sP[r * LP + s] = p;
        sDS[r * LP + s] = p == 0.0f ? 0.0f : p * (y[i][j] - sD[qi]);
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
      from_f32(acc0[i][j] * scale, out0 + (base + n) * D + tc + 16 * j);
      if (KV) from_f32(acc1[i][j], out1 + (base + n) * D + tc + 16 * j);
    }
  }
}

template <typename T, int D, bool KV>
static cudaError_t launch_bwd_t(const Dims& Dm, const void* a0, const void* a1, const void* b0, const void* b1,
                                const float* lse, const float* delta, const int32_t* tile_ptr, const int32_t* tile_col,
                                void* out0, void* out1, float scale, int32_t* dev_status, cudaStream_t st) {
  const size_t smem = sizeof(float) * (4 * kBlock * (D + 4) + 2 * kBlock * (kBlock + 1) + 2 * kBlock);
  const cudaError_t e = cudaFuncSetAttribute(attn_bwd_kernel<T, D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(Dm.nB), static_cast<unsigned>(Dm.BH));
  attn_bwd_kernel<T, D, KV><<<grid, 256, smem, st>>>(
      static_cast<const T*>(a0), static_cast<const T*>(a1), static_cast<const T*>(b0), static_cast<const T*>(b1), lse,
      delta, tile_ptr, tile_col, static_cast<T*>(out0), static_cast<T*>(out1), static_cast<int>(Dm.N),
      static_cast<int>(Dm.nB), static_cast<int>(Dm.nPairs), scale, dev_status);
  return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t launch_bwd_d(const Dims& Dm, const BwdArgs& x, const fva_mask* m, const BwdScratch& ws,
                                int32_t* dev_status, cudaStream_t st) {
  cudaError_t e = launch_bwd_t<T, D, true>(Dm, x.k, x.v, x.q, x.d_o, x.lse, ws.delta, ws.mask_t.tile_ptr,
                                           ws.mask_t.tile_col, x.dk, x.dv, x.scale, dev_status, st);
  if (e != cudaSuccess) return e;
  return launch_bwd_t<T, D, false>(Dm, x.q, x.d_o, x.k, x.v, x.lse, ws.delta, m->tile_ptr, m->tile_col, x.dq, nullptr,
                                   x.scale, dev_status, st);
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
  const int64_t rows = Dm.BH * Dm.N;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (Dm.esize == 2)
    row_dot_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x.o),
                                                        static_cast<const __nv_bfloat16*>(x.d_o), rows,
                                                        static_cast<int>(Dm.d), ws.delta);
  else
    row_dot_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(x.o), static_cast<const float*>(x.d_o), rows,
                                                static_cast<int>(Dm.d), ws.delta);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (Dm.esize == 2) {
    if (Dm.d == 128) return launch_bwd_d<__nv_bfloat16, 128>(Dm, x, m, ws, dev_status, st);
    return launch_bwd_d<__nv_bfloat16, 64>(Dm, x, m, ws, dev_status, st);
  }
  switch (Dm.d) {
    case 32: return launch_bwd_d<float, 32>(Dm, x, m, ws, dev_status, st);
    case 64: return launch_bwd_d<float, 64>(Dm, x, m, ws, dev_status, st);
    default: return launch_bwd_d<float, 128>(Dm, x, m, ws, dev_status, st);
  }
}

}  // namespace fva
