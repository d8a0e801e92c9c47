// Grouped matrix products (moe_grouped_matmul and its two gradients) on the
// CUDA cores: out[i, j] = sum_r P[i, r] Q[j, r] in fp32 FFMA, for fp32
// operands (tf32 inputs would lose 13 of their bits) and for 16-bit operands
// whose row lengths are not whole 16-byte vectors, which TMA cannot address.
//
//   forward  P = a [R, k]    (r contiguous), Q = W[e] [n, k] (r contiguous)
//   dgrad    P = dout [R, n] (r contiguous), Q = W[e]        (j contiguous)
//   wgrad    P = dout        (i contiguous), Q = a           (j contiguous)
//
// Three kernels.  Tiles of TB x TB outputs, 16 of r at a time through shared
// memory in two buffers (the next step's operands are in flight while this one
// is used), 256 threads with (TB / 16)^2 outputs each: TB = 128 reads 64 bytes
// of shared memory for 64 FMAs a thread and step, TB = 64 32 bytes for 16, the
// larger tile where its tiles fill the SMs.  Where 64 x 64 tiles do not, or
// would be half empty, tiles of 32 x 32 whose sum the block's warps share; and
// for a handful of rows no tiles at all (below, with the figures of both).
// Products go two at a time (packed fp32 FMAs): the same rate from the FMA pipe
// for half the issue slots, which the loads need.  Every reduction runs in one
// fixed order, so results repeat bit for bit.  Bound by shared memory at TB = 64
// (2048 rows, n = k = 640, fp32: 75 us) and by latency on smaller batches; 2048
// rows of 4 experts, n = k = 1024: dW 106 us (40 TFLOP/s).
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

constexpr int NT = 256;
// r of a step
__host__ __device__ constexpr int step_r(int tb) { return tb == 32 ? 64 : 16; }

__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ float elem_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_f32(__half v) { return __half2float(v); }
template <typename O> __device__ __forceinline__ O elem_from(float v);
template <> __device__ __forceinline__ float elem_from<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 elem_from<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half elem_from<__half>(float v) { return __float2half_rn(v); }

// Four consecutive elements; `vec`: 16-byte (fp32) or 8-byte aligned.
template <typename T> __device__ __forceinline__ float4 load4(const T* p) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  const T* t = reinterpret_cast<const T*>(&q);
  return make_float4(elem_f32(t[0]), elem_f32(t[1]), elem_f32(t[2]), elem_f32(t[3]));
}
template <> __device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <typename O> __device__ __forceinline__ void store4(O* p, float4 v) {
  const O t[4] = {elem_from<O>(v.x), elem_from<O>(v.y), elem_from<O>(v.z), elem_from<O>(v.w)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(t);
}
template <> __device__ __forceinline__ void store4<float>(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// One operand's tile of TB x TR, as M[x0 + x, r0 + r] with zeros outside
// nx x nr.  RED: r contiguous (element x * ld + r), else x contiguous
// (r * ld + x).  A thread carries G groups of 4 elements from global
// memory (fetch) to shared memory (place: tile[r][x]).
template <bool RED, int TB, typename T> struct Operand {
  static constexpr int TR = step_r(TB), G = TB * TR / (4 * NT);
  const T* m;
  int64_t ld, x0, nx, nr;
  bool vec;
  float4 v[G];
  __device__ __forceinline__ void where(int g, int& x, int& r) const {
    const int i = static_cast<int>(threadIdx.x) + g * NT;
    if (RED && TB == 32) {               // a warp: 8 of x, 16 of r (two lanes a bank in place())
      const int lane = i & 31, run = i >> 5;
      x = (run & 3) * 8 + (lane >> 2);
      r = ((run >> 2) * 4 + (lane & 3)) * 4;
      return;
    }
    x = RED ? i / (TR / 4) : (i % (TB / 4)) * 4;
    r = RED ? (i % (TR / 4)) * 4 : i / (TB / 4);
  }
  __device__ __forceinline__ void fetch(int64_t r0) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      int x, r;
      where(g, x, r);
      const int64_t xx = x0 + x, rr = r0 + r;
      const int64_t left = RED ? (xx < nx ? nr - rr : 0) : (rr < nr ? nx - xx : 0);   // of the 4
      const T* p = m + (RED ? xx * ld + rr : rr * ld + xx);
      if (left >= 4 && vec) {
        v[g] = load4(p);
      } else {
        v[g].x = left > 0 ? elem_f32(p[0]) : 0.0f;
        v[g].y = left > 1 ? elem_f32(p[1]) : 0.0f;
        v[g].z = left > 2 ? elem_f32(p[2]) : 0.0f;
        v[g].w = left > 3 ? elem_f32(p[3]) : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void place(float (*tile)[TB + 4]) const {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      int x, r;
      where(g, x, r);
      if (RED) {
        tile[r][x] = v[g].x;
        tile[r + 1][x] = v[g].y;
        tile[r + 2][x] = v[g].z;
        tile[r + 3][x] = v[g].w;
      } else {
        *reinterpret_cast<float4*>(&tile[r][x]) = v[g];
      }
    }
  }
};

struct SimtProduct {
  const void *p, *q;
  void* out;
  const int32_t* offsets;
  int32_t* status;
  int E, n, k, rows_cap, accumulate;
  int vec_p, vec_q;      // rows of whole 4-element vectors
};

template <int FORM, int TB, typename T, typename O>
__global__ void __launch_bounds__(NT, TB == 64 ? 3 : 2) grouped_matmul_simt_kernel(const SimtProduct g) {
  constexpr int M = TB / 16, TR = step_r(TB);   // outputs a thread, each way
  __shared__ __align__(16) float Ps[2][TR][TB + 4];
  __shared__ __align__(16) float Qs[2][TR][TB + 4];
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
    f32x2 acc[M][M / 2];                 // neighbouring columns as packed pairs
#pragma unroll
    for (int a = 0; a < M; ++a)
#pragma unroll
      for (int b = 0; b < M / 2; ++b) acc[a][b] = 0;
    Operand<FORM != kWgrad, TB, T> op{P, FORM == kForward ? g.k : g.n, i0, ni, nr, g.vec_p != 0};
    Operand<FORM == kForward, TB, T> oq{Q, g.k, j0, cols, nr, g.vec_q != 0};
    int buf = 0;
    __syncthreads();                     // the previous tile's last buffer is free
    if (nr > 0) {
      op.fetch(0);
      oq.fetch(0);
      op.place(Ps[0]);
      oq.place(Qs[0]);
      __syncthreads();
    }
    for (int64_t r0 = 0; r0 < nr; r0 += TR) {
      const bool more = r0 + TR < nr;
      if (more) {
        op.fetch(r0 + TR);
        oq.fetch(r0 + TR);
      }
#pragma unroll
      for (int r = 0; r < TR; ++r) {
        float pa[M];
        f32x2 qa[M / 2];
        // thread (ty, tx) holds rows 4 ty + 64 h.. and columns 4 tx + 64 h..
#pragma unroll
        for (int h = 0; h < M / 4; ++h) {
          const float4 pv = *reinterpret_cast<const float4*>(&Ps[buf][r][ty * 4 + 64 * h]);
          const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(&Qs[buf][r][tx * 4 + 64 * h]);
          pa[4 * h] = pv.x; pa[4 * h + 1] = pv.y; pa[4 * h + 2] = pv.z; pa[4 * h + 3] = pv.w;
          qa[2 * h] = qv.x; qa[2 * h + 1] = qv.y;
        }
#pragma unroll
        for (int a = 0; a < M; ++a) {
          const f32x2 p2 = pack2(pa[a], pa[a]);
#pragma unroll
          for (int b = 0; b < M / 2; ++b) acc[a][b] = fma2(p2, qa[b], acc[a][b]);
        }
      }
      if (more) {
        op.place(Ps[buf ^ 1]);
        oq.place(Qs[buf ^ 1]);
        __syncthreads();
        buf ^= 1;
      }
    }
    O* out = static_cast<O*>(g.out) + (FORM == kWgrad ? static_cast<int64_t>(e) * g.n : row0) * cols;
#pragma unroll
    for (int a = 0; a < M; ++a) {
      const int64_t i = i0 + ty * 4 + 64 * (a / 4) + a % 4;
      if (i >= ni) continue;
      float v[M];
#pragma unroll
      for (int b = 0; b < M / 2; ++b) {
        const float2 pr = unpack2(acc[a][b]);
        v[2 * b] = pr.x, v[2 * b + 1] = pr.y;
      }
      if (FORM == kWgrad && g.accumulate) {          // a row's loads together, ahead of its stores
#pragma unroll
        for (int b = 0; b < M; ++b) {
          const int64_t j = j0 + tx * 4 + 64 * (b / 4) + b % 4;
          v[b] += j < cols ? elem_f32(out[i * cols + j]) : 0.0f;
        }
      }
#pragma unroll
      for (int b = 0; b < M; ++b) {
        const int64_t j = j0 + tx * 4 + 64 * (b / 4) + b % 4;
        if (j < cols) out[i * cols + j] = elem_from<O>(v[b]);
      }
    }
  }
}

// Tiles of 32 x 32 outputs, 64 of r at a time, of which every warp takes eight:
// a lane sums 4 x 8 outputs over its warp's part of r, the eight warps' sums are
// added at the end, in order.  Four times the tiles and a quarter of the steps of
// TB = 64 (and 4 loads in flight a thread), for twice its operand bytes: faster
// where 64 x 64 tiles do not fill the SMs (us, against them): dW of 2048 rows, 128 x 128,
// 33 / 98; of 2048 rows, 640 x 640 (100 tiles), 68 / 92; 500 rows of 8 experts,
// n = 1024, k = 256, input gradient 23 / 56.  With more of them: 2048 rows
// of 16 experts, n = k = 512 (256 tiles), 61 / 44.  Also for up to 32 rows an
// expert: 128 rows of 8, n = k = 1024, 29 / 57; 1024 of 32, 98 / 157.  Bound by
// latency.
template <int FORM, typename T, typename O>
__global__ void __launch_bounds__(NT, 2) grouped_matmul_sliced_kernel(const SimtProduct g) {
  constexpr int TB = 32, TR = step_r(TB), W = NT / 32;
  using Tile = float[TR][TB + 4];
  __shared__ __align__(16) Tile s_ops[4];              // P and Q, two buffers each; then the warps' sums
  static_assert(sizeof(s_ops) == sizeof(float) * W * TB * (TB + 4), "the sums take the operands' place");
  float (*s_sum)[TB][TB + 4] = reinterpret_cast<float (*)[TB][TB + 4]>(&s_ops[0][0][0]);
  __shared__ int s_bad;
  extern __shared__ int s_tables[];
  int* s_off = s_tables;
  int* s_tile = s_tables + g.E + 1;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int cols = FORM == kForward ? g.n : g.k;
  const int j_tiles = (cols + TB - 1) / TB;
  const int i_tiles = (g.n + TB - 1) / TB;
  if (tid == 0) s_bad = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (tid < 32)
    build_tile_prefix(g.offsets, g.E, 0, 0, kAllTiles, TB, j_tiles, g.rows_cap, s_off, s_tile, &s_bad);
  __syncthreads();
  if (tid == 0 && s_bad) record_status(g.status, DEV_BAD_ROW);
  const int64_t total = FORM == kWgrad ? static_cast<int64_t>(g.E) * i_tiles * j_tiles : s_tile[g.E];
  const int tx = tid & 3, ty = (tid & 31) >> 2;

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
    f32x2 acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = 0;
    Operand<FORM != kWgrad, TB, T> op{P, FORM == kForward ? g.k : g.n, i0, ni, nr, g.vec_p != 0};
    Operand<FORM == kForward, TB, T> oq{Q, g.k, j0, cols, nr, g.vec_q != 0};
    int buf = 0;
    __syncthreads();                     // the previous tile's sums are read
    if (nr > 0) {
      op.fetch(0);
      oq.fetch(0);
      op.place(s_ops[0]);
      oq.place(s_ops[2]);
      __syncthreads();
    }
    for (int64_t r0 = 0; r0 < nr; r0 += TR) {
      const bool more = r0 + TR < nr;
      if (more) {
        op.fetch(r0 + TR);
        oq.fetch(r0 + TR);
      }
#pragma unroll
      for (int x = 0; x < TR / W; ++x) {
        const int r = warp * (TR / W) + x;
        const float4 pv = *reinterpret_cast<const float4*>(&s_ops[buf][r][ty * 4]);
        const ulonglong2 q0 = *reinterpret_cast<const ulonglong2*>(&s_ops[2 + buf][r][tx * 8]);
        const ulonglong2 q1 = *reinterpret_cast<const ulonglong2*>(&s_ops[2 + buf][r][tx * 8 + 4]);
        const float pa[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const f32x2 p2 = pack2(pa[a], pa[a]);
          acc[a][0] = fma2(p2, q0.x, acc[a][0]);
          acc[a][1] = fma2(p2, q0.y, acc[a][1]);
          acc[a][2] = fma2(p2, q1.x, acc[a][2]);
          acc[a][3] = fma2(p2, q1.y, acc[a][3]);
        }
      }
      if (more) {
        op.place(s_ops[buf ^ 1]);
        oq.place(s_ops[2 + (buf ^ 1)]);
        __syncthreads();
        buf ^= 1;
      }
    }
    __syncthreads();                     // the last operands are read
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        *reinterpret_cast<ulonglong2*>(&s_sum[warp][ty * 4 + a][tx * 8 + 4 * b]) =
            make_ulonglong2(acc[a][2 * b], acc[a][2 * b + 1]);
    __syncthreads();
    const int ii = tid >> 3, jj = (tid & 7) * 4;         // four outputs a thread
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(&s_sum[w][ii][jj]);
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    const int64_t left = i0 + ii < ni ? cols - (j0 + jj) : 0;
    O* out = static_cast<O*>(g.out) +
             ((FORM == kWgrad ? static_cast<int64_t>(e) * g.n : row0) + i0 + ii) * cols + j0 + jj;
    if (left >= 4 && cols % 4 == 0) {
      if (FORM == kWgrad && g.accumulate) {
        const float4 old = load4(out);
        v.x += old.x;
        v.y += old.y;
        v.z += old.z;
        v.w += old.w;
      }
      store4(out, v);
    } else {
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b < left) out[b] = elem_from<O>(FORM == kWgrad && g.accumulate ? f[b] + elem_f32(out[b]) : f[b]);
    }
  }
}

// Forward and dgrad of few rows, where tiles would be mostly padding and each
// of their steps a wait for memory: W goes straight to registers, four to eight
// loads of a thread in flight, against up to eight rows of P, which L1 serves.
//   forward  a warp per two n: its lanes walk k, then add up
//   dgrad    a block per 32 k: eight lanes of 4 k each for a row of W, 32 rows of
//            W at a time, then the 32 partial sums add up
// Each sum has one fixed order.  Against the 32 x 32 tiles, us:
//   4 rows, n = k = 1024, fp32                  16 / 23, 8 rows 23 / 23
//   128 rows of 64 experts, n = k = 1024, fp32  76 / 170
//   256 of 64, n = k = 512, fp32                45 / 57, 512 rows 61 / 57
//   32 rows, n = 1001, k = 999, bf16            forward 18 / 47, dgrad 35 / 49
//   64 of 8, n = 1001, k = 999, bf16            forward 29 / 49, dgrad 39 / 51
// so it takes calls of up to 4 rows an expert; where rows are no whole vectors,
// whose elements the tiles fetch one by one, of up to 8 an expert or 64 in all.
// Bound by the loads of P from L1 and by latency (128 of 64: 3.5 TB/s of weights).
constexpr int kFewRows = 64;
constexpr int kRowsAtOnce = 8;
constexpr int kFewNs = 2;         // n of a warp of the forward product
template <int R, typename T, typename O>
__device__ __forceinline__ void few_rows_forward(const T* __restrict__ p, const T* __restrict__ w, int rows, int nr,
                                                 int cols, int j0, int vec, O* __restrict__ out) {
  constexpr int N = kFewNs, U = 2;                   // 4 loads of W in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = j0 + N * warp;
  if (j >= cols) return;                             // uniform over the warp
  float acc[R][N];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int q = 0; q < N; ++q) acc[r][q] = 0.0f;
  const T* wr[N];
#pragma unroll
  for (int q = 0; q < N; ++q) wr[q] = w + static_cast<int64_t>(min(j + q, cols - 1)) * nr;
  if (vec) {                                         // nr is a multiple of 4: all four inside or none
    for (int c0 = 4 * lane; c0 < nr; c0 += U * 128) {
      float4 wv[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < N; ++q)
          wv[u][q] = c0 + u * 128 < nr ? load4(wr[q] + c0 + u * 128) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rows)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (c0 + u * 128 >= nr) continue;
            const float4 v = load4(p + static_cast<int64_t>(r) * nr + c0 + u * 128);
#pragma unroll
            for (int q = 0; q < N; ++q)
              acc[r][q] = fmaf(v.x, wv[u][q].x,
                               fmaf(v.y, wv[u][q].y, fmaf(v.z, wv[u][q].z, fmaf(v.w, wv[u][q].w, acc[r][q]))));
          }
    }
  } else {
#pragma unroll 4
    for (int c = lane; c < nr; c += 32) {
      float wv[N];
#pragma unroll
      for (int q = 0; q < N; ++q) wv[q] = elem_f32(wr[q][c]);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rows) {
          const float v = elem_f32(p[static_cast<int64_t>(r) * nr + c]);
#pragma unroll
          for (int q = 0; q < N; ++q) acc[r][q] = fmaf(v, wv[q], acc[r][q]);
        }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int q = 0; q < N; ++q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][q] += __shfl_xor_sync(0xffffffffu, acc[r][q], o);
      if (lane == 0 && r < rows && j + q < cols) out[static_cast<int64_t>(r) * cols + j + q] = elem_from<O>(acc[r][q]);
    }
}

constexpr int kFewCols = 32;      // columns of a dgrad tile
template <int R, typename T, typename O>
__device__ __forceinline__ void few_rows_dgrad(const T* __restrict__ p, const T* __restrict__ w, int rows, int nr,
                                               int cols, int j0, int vec, float (*s_acc)[kRowsAtOnce][kFewCols],
                                               O* __restrict__ out) {
  constexpr int U = 8;                               // loads of W in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane >> 3, jl = 4 * (lane & 7);
  const int j = j0 + jl;
  float acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[r][q] = 0.0f;
  for (int c0 = 4 * warp + part; c0 < nr; c0 += U * (NT / 8)) {
    float wv[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * (NT / 8);
      const T* wr = w + static_cast<int64_t>(c) * cols + j;
      if (vec) {                                     // cols is a multiple of 4: all four inside or none
        const float4 v = c < nr && j < cols ? load4(wr) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        wv[u][0] = v.x, wv[u][1] = v.y, wv[u][2] = v.z, wv[u][3] = v.w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) wv[u][q] = c < nr && j + q < cols ? elem_f32(wr[q]) : 0.0f;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < rows) {
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * (NT / 8);
          d[u] = c < nr ? elem_f32(p[static_cast<int64_t>(r) * nr + c]) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[r][q] = fmaf(d[u], wv[u][q], acc[r][q]);
      }
  }
  __syncthreads();                                   // the previous tile's sums are read
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[r][q] += __shfl_xor_sync(0xffffffffu, acc[r][q], 8);
      acc[r][q] += __shfl_xor_sync(0xffffffffu, acc[r][q], 16);
    }
    if (part == 0)
      *reinterpret_cast<float4*>(&s_acc[warp][r][jl]) = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
  __syncthreads();
  const int r = threadIdx.x / kFewCols, c = threadIdx.x % kFewCols;   // NT = 8 rows of 32
  if (r < rows && j0 + c < cols) {
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < NT / 32; ++q) v += s_acc[q][r][c];
    out[static_cast<int64_t>(r) * cols + j0 + c] = elem_from<O>(v);
  }
}

template <int FORM, typename T, typename O>
__global__ void __launch_bounds__(NT) grouped_matmul_few_rows_kernel(const SimtProduct g) {
  constexpr int R = kRowsAtOnce, COLS = FORM == kForward ? kFewNs * NT / 32 : kFewCols;   // columns of a tile
  __shared__ __align__(16) float s_acc[FORM == kForward ? 1 : NT / 32][R][kFewCols];
  __shared__ int s_bad;
  extern __shared__ int s_tables[];
  int* s_off = s_tables;
  int* s_tile = s_tables + g.E + 1;
  const int cols = FORM == kForward ? g.n : g.k, nr = FORM == kForward ? g.k : g.n;
  if (threadIdx.x == 0) s_bad = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (threadIdx.x < 32)
    build_tile_prefix(g.offsets, g.E, 0, 0, kAllTiles, R, (cols + COLS - 1) / COLS, g.rows_cap, s_off, s_tile, &s_bad);
  __syncthreads();
  if (threadIdx.x == 0 && s_bad) record_status(g.status, DEV_BAD_ROW);
  const int total = s_tile[g.E];
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int e, it, jt;
    decode_tile(tile, s_tile, g.E, s_off, g.E, 0, kAllTiles, R, e, it, jt);
    const int64_t row0 = static_cast<int64_t>(s_off[e]) + it * R;
    const int rows = min(R, s_off[e + 1] - static_cast<int>(row0));
    const T* p = static_cast<const T*>(g.p) + row0 * nr;
    const T* w = static_cast<const T*>(g.q) + static_cast<int64_t>(e) * g.n * g.k;
    O* out = static_cast<O*>(g.out) + row0 * cols;
    if (FORM == kForward) {
      if (rows <= 2)
        few_rows_forward<2>(p, w, rows, nr, cols, jt * COLS, g.vec_q, out);
      else
        few_rows_forward<R>(p, w, rows, nr, cols, jt * COLS, g.vec_q, out);
    } else {
      if (rows <= 2)
        few_rows_dgrad<2>(p, w, rows, nr, cols, jt * COLS, g.vec_q, s_acc, out);
      else
        few_rows_dgrad<R>(p, w, rows, nr, cols, jt * COLS, g.vec_q, s_acc, out);
    }
  }
}

// tiles of TB x TB at most (each group may end in a partial row tile)
template <int FORM> int64_t tile_bound(const GroupedProduct& g, int tb) {
  const int64_t j_tiles = ceil_div(FORM == kForward ? g.n : g.k, tb);
  return FORM == kWgrad ? g.E * ceil_div(g.n, tb) * j_tiles : (ceil_div(g.rows, tb) + g.E) * j_tiles;
}

template <int FORM, int TB, typename T, typename O>
cudaError_t launch_tile(const GroupedProduct& g, int num_sms, cudaStream_t stream) {
  SimtProduct s{g.p, g.q, g.out, g.offsets, g.status, g.E, g.n, g.k, static_cast<int>(g.rows), g.accumulate, 0, 0};
  // rows start on vector boundaries (the operands are 16-byte aligned)
  s.vec_p = (FORM == kForward ? g.k : g.n) % 4 == 0;
  s.vec_q = g.k % 4 == 0;
  const size_t smem = sizeof(int) * (2 * static_cast<size_t>(g.E) + 2);
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(
      1, std::min<int64_t>(tile_bound<FORM>(g, TB), static_cast<int64_t>(num_sms) * (TB == 64 ? 4 : 2))));
  return launch_chained(grouped_matmul_simt_kernel<FORM, TB, T, O>, grid, NT, smem, stream, s);
}

template <int FORM, typename T, typename O>
cudaError_t launch_sliced(const GroupedProduct& g, int num_sms, cudaStream_t stream) {
  SimtProduct s{g.p, g.q, g.out, g.offsets, g.status, g.E, g.n, g.k, static_cast<int>(g.rows), g.accumulate, 0, 0};
  s.vec_p = (FORM == kForward ? g.k : g.n) % 4 == 0;
  s.vec_q = g.k % 4 == 0;
  const size_t smem = sizeof(int) * (2 * static_cast<size_t>(g.E) + 2);
  const unsigned grid = static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>(tile_bound<FORM>(g, 32), static_cast<int64_t>(num_sms) * 2)));
  return launch_chained(grouped_matmul_sliced_kernel<FORM, T, O>, grid, NT, smem, stream, s);
}

template <int FORM, typename T, typename O>
cudaError_t launch_few_rows(const GroupedProduct& g, int num_sms, cudaStream_t stream) {
  SimtProduct s{g.p, g.q, g.out, g.offsets, g.status, g.E, g.n, g.k, static_cast<int>(g.rows), 0, 0, 0};
  s.vec_q = g.k % 4 == 0;
  const size_t smem = sizeof(int) * (2 * static_cast<size_t>(g.E) + 2);
  const int64_t tiles = std::min<int64_t>(g.rows, ceil_div(g.rows, kRowsAtOnce) + g.E) *
                        (FORM == kForward ? ceil_div(g.n, kFewNs * NT / 32) : ceil_div(g.k, kFewCols));
  const unsigned grid = static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>(tiles, static_cast<int64_t>(num_sms) * 8)));
  return launch_chained(grouped_matmul_few_rows_kernel<FORM, T, O>, grid, NT, smem, stream, s);
}

template <int FORM, typename T, typename O>
cudaError_t launch_form(const GroupedProduct& g, int num_sms, cudaStream_t stream) {
  if constexpr (FORM != kWgrad) {
    const int64_t E = g.E;
    const bool vec = g.n % 4 == 0 && g.k % 4 == 0;
    if (vec ? g.rows <= 4 * E : g.rows <= std::max<int64_t>(kFewRows, kRowsAtOnce * E))
      return launch_few_rows<FORM, T, O>(g, num_sms, stream);
    if (g.rows <= 32 * E) return launch_sliced<FORM, T, O>(g, num_sms, stream);   // tiles of 64 half empty
  }
  // rows / 128 + E bounds the tiles from above by E: full tiles alone count
  const int64_t full = FORM == kWgrad ? tile_bound<FORM>(g, 128)
                                      : g.rows / 128 * ceil_div(FORM == kForward ? g.n : g.k, 128);
  if (full >= num_sms) return launch_tile<FORM, 128, T, O>(g, num_sms, stream);
  const int64_t tiles = FORM == kWgrad ? tile_bound<FORM>(g, 64)
                                       : std::max<int64_t>(ceil_div(g.rows, 64), std::min<int64_t>(g.rows, g.E)) *
                                             ceil_div(FORM == kForward ? g.n : g.k, 64);
  return 4 * tiles < 3 * num_sms ? launch_sliced<FORM, T, O>(g, num_sms, stream)
                                 : launch_tile<FORM, 64, T, O>(g, num_sms, stream);
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
