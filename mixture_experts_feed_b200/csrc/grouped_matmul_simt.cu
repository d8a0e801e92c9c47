// Grouped matrix products (moe_grouped_matmul and its two gradients) on the
// CUDA cores: out[i, j] = sum_r P[i, r] Q[j, r] in fp32 FFMA, for fp32
// operands (tf32 inputs would lose 13 of their bits) and for 16-bit operands
// whose row lengths are not whole 16-byte vectors, which TMA cannot address.
//
//   forward  P = a [R, k]    (r contiguous), Q = W[e] [n, k] (r contiguous)
//   dgrad    P = dout [R, n] (r contiguous), Q = W[e]        (j contiguous)
//   wgrad    P = dout        (i contiguous), Q = a           (j contiguous)
//
// Tiles of 64 x 64 outputs, 16 of r at a time through shared memory, 256
// threads with 4 x 4 outputs each.  The reduction runs in one fixed order, so
// results repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "grouping.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int TB = 64, TR = 16, NT = 256;

__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ float elem_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_f32(__half v) { return __half2float(v); }
template <typename O> __device__ __forceinline__ O elem_from(float v);
template <> __device__ __forceinline__ float elem_from<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 elem_from<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half elem_from<__half>(float v) { return __float2half_rn(v); }

// tile[r][x] = M[x0 + x, r0 + r], zero outside nx x nr.  RED: r contiguous
// (element x * ld + r), else x contiguous (r * ld + x).
template <bool RED, typename T>
__device__ __forceinline__ void load_tile(const T* __restrict__ m, int64_t ld, int64_t x0, int64_t nx,
                                          int64_t r0, int64_t nr, float (*tile)[TB + 4]) {
  const int tid = threadIdx.x;
  if (RED) {
    const int x = tid >> 2, r = (tid & 3) * 4;
    const bool ok = x0 + x < nx;
    const T* src = m + (ok ? (x0 + x) * ld : 0) + r0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      tile[r + q][x] = ok && r0 + r + q < nr ? elem_f32(src[r + q]) : 0.0f;
  } else {
    const int r = tid >> 4, x = (tid & 15) * 4;
    const bool ok = r0 + r < nr;
    const T* src = m + (ok ? (r0 + r) * ld : 0) + x0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      tile[r][x + q] = ok && x0 + x + q < nx ? elem_f32(src[x + q]) : 0.0f;
  }
}

struct SimtProduct {
  const void *p, *q;
  void* out;
  const int32_t* offsets;
  int32_t* status;
  int E, n, k, rows_cap, accumulate;
};

template <int FORM, typename T, typename O>
__global__ void __launch_bounds__(NT) grouped_matmul_simt_kernel(const SimtProduct g) {
  __shared__ __align__(16) float Ps[TR][TB + 4];
  __shared__ __align__(16) float Qs[TR][TB + 4];
  __shared__ int s_bad;
  extern __shared__ int s_tables[];
  int* s_off = s_tables;
  int* s_tile = s_tables + g.E + 1;
  const int tid = threadIdx.x;
  // outputs across a row (j) and the tiles over them
  const int cols = FORM == kForward ? g.n : g.k;
  const int j_tiles = (cols + TB - 1) / TB;
  const int i_tiles = (g.n + TB - 1) / TB;     // kWgrad: tiles over i of each expert
  if (tid == 0) s_bad = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (tid < 32)
    build_tile_prefix(g.offsets, g.E, 0, 0, kAllTiles, TB, j_tiles, g.rows_cap, s_off, s_tile, &s_bad);
  __syncthreads();
  if (tid == 0 && s_bad) record_status(g.status, DEV_BAD_ROW);
  const int64_t total = FORM == kWgrad ? static_cast<int64_t>(g.E) * i_tiles * j_tiles : s_tile[g.E];
  const int tx = tid & 15, ty = tid >> 4;

  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int e, it, jt;
    if (FORM == kWgrad) {
      e = static_cast<int>(tile / (static_cast<int64_t>(i_tiles) * j_tiles));
      const int local = static_cast<int>(tile - static_cast<int64_t>(e) * i_tiles * j_tiles);
      it = local / j_tiles;
      jt = local - it * j_tiles;
    } else {
      decode_tile(static_cast<int>(tile), s_tile, g.E, s_off, g.E, 0, kAllTiles, TB, e, it, jt);
    }
    const int64_t row0 = s_off[e];
    const int rows = s_off[e + 1] - s_off[e];
    if (FORM == kWgrad && g.accumulate && rows == 0) continue;
    const T* P = static_cast<const T*>(g.p);
    const T* Q = static_cast<const T*>(g.q);
    const int64_t i0 = static_cast<int64_t>(it) * TB, j0 = static_cast<int64_t>(jt) * TB;
    const int64_t ni = FORM == kWgrad ? g.n : rows;
    const int64_t nr = FORM == kForward ? g.k : (FORM == kDgrad ? g.n : rows);
    if (FORM == kWgrad) {
      P += row0 * g.n;
      Q += row0 * g.k;
    } else {
      P += row0 * (FORM == kForward ? g.k : g.n);
      Q += static_cast<int64_t>(e) * g.n * g.k;
    }
    float acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = 0.0f;
    for (int64_t r0 = 0; r0 < nr; r0 += TR) {
      load_tile<FORM != kWgrad>(P, FORM == kForward ? g.k : g.n, i0, ni, r0, nr, Ps);
      load_tile<FORM == kForward>(Q, g.k, j0, cols, r0, nr, Qs);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < TR; ++r) {
        const float4 pv = *reinterpret_cast<const float4*>(&Ps[r][ty * 4]);
        const float4 qv = *reinterpret_cast<const float4*>(&Qs[r][tx * 4]);
        const float pa[4] = {pv.x, pv.y, pv.z, pv.w}, qa[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(pa[a], qa[b], acc[a][b]);
      }
      __syncthreads();
    }
    O* out = static_cast<O*>(g.out) + (FORM == kWgrad ? static_cast<int64_t>(e) * g.n : row0) * cols;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int64_t i = i0 + ty * 4 + a;
      if (i >= ni) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t j = j0 + tx * 4 + b;
        if (j >= cols) continue;
        O* dst = out + i * cols + j;
        float v = acc[a][b];
        if (FORM == kWgrad && g.accumulate) v += elem_f32(*dst);
        *dst = elem_from<O>(v);
      }
    }
  }
}

template <int FORM, typename T, typename O>
cudaError_t launch_form(const GroupedProduct& g, int num_sms, cudaStream_t stream) {
  SimtProduct s{g.p, g.q, g.out, g.offsets, g.status, g.E, g.n, g.k, static_cast<int>(g.rows), g.accumulate};
  const size_t smem = sizeof(int) * (2 * static_cast<size_t>(g.E) + 2);
  const int cols = FORM == kForward ? g.n : g.k;
  const int64_t j_tiles = ceil_div(cols, TB);
  // at most this many tiles (each group may end in a partial row tile)
  const int64_t tiles = FORM == kWgrad ? g.E * ceil_div(g.n, TB) * j_tiles
                                       : (ceil_div(g.rows, TB) + g.E) * j_tiles;
  const unsigned grid = static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>(tiles, static_cast<int64_t>(num_sms) * 4)));
  return launch_chained(grouped_matmul_simt_kernel<FORM, T, O>, grid, NT, smem, stream, s);
}

template <typename T, typename O>
cudaError_t launch_types(const GroupedProduct& g, int num_sms, cudaStream_t stream) {
  return g.form == kForward ? launch_form<kForward, T, O>(g, num_sms, stream)
         : g.form == kDgrad ? launch_form<kDgrad, T, O>(g, num_sms, stream)
                            : launch_form<kWgrad, T, O>(g, num_sms, stream);
}

}  // namespace

cudaError_t launch_grouped_matmul_simt(const GroupedProduct& g, int num_sms, cudaStream_t stream) {
  const bool f32 = g.out_dtype == MOE_ELEM_F32;
  if (g.dtype == MOE_ELEM_F32) return launch_types<float, float>(g, num_sms, stream);
  if (g.dtype == MOE_ELEM_BF16)
    return f32 ? launch_types<__nv_bfloat16, float>(g, num_sms, stream)
               : launch_types<__nv_bfloat16, __nv_bfloat16>(g, num_sms, stream);
  return f32 ? launch_types<__half, float>(g, num_sms, stream)
             : launch_types<__half, __half>(g, num_sms, stream);
}

}  // namespace moe
