// Layer norm's forward pass, and the backward passes of layer norm and
// RMSNorm with the reduction of the weight's (and bias's) gradient.
//
//   x^ = (x - mean) r,  r = 1 / sqrt(var + eps)     (RMSNorm: x^ = x r,
//                                                   r = 1 / sqrt(mean x^2 + eps))
//   out = x^ weight + bias
//   gy = dout weight,  dx = r (gy - mean(gy) - x^ mean(gy x^)) + dres
//                                                   (RMSNorm: no mean(gy))
//   dweight = sum_t dout x^,  dbias = sum_t dout
//
// Row sums are fp32 and the variance is summed around the mean.  Each block
// takes row groups blockIdx.x, + gridDim.x, ... and adds its rows' dout x^ and
// dout, column by column always by the same thread, into one partial row; a
// second kernel adds the blocks' partial rows in a fixed order.  No atomics:
// the same bits on every run.
//
// All passes are bound by HBM (backward: read x, dout and dres, write dx).
// Rows of whole 16-byte vectors run in the *_rows kernels: a team of threads
// holds a row in registers, 16 elements (8 to 32) a thread, so x and dout are
// read once although the statistics need the whole row first.  Each thread
// copies its own vectors of the rows to come into shared memory with cp.async,
// one or two row groups ahead, and reads back only what it copied itself: the
// loads stay in flight across the reductions with no barrier between them.
// The reductions (RMSNorm one, layer norm two: the mean first) cost one block
// barrier each, none when a team is one warp.  Other rows take the *_any
// kernels, which stream them several times.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// sum over the block of two values, in every thread (fixed order)
__device__ __forceinline__ float2 block_sum2(float a, float b) {
  __shared__ float2 s_part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    t.x += s_part[i].x;
    t.y += s_part[i].y;
  }
  __syncthreads();
  return t;
}

// mean (RMSNorm: 0) and r of a row of any length, streamed
template <typename T, bool LAYER>
__device__ __forceinline__ float2 row_stats(const T* row, int H, float eps) {
  float mean = 0.0f;
  if (LAYER) {
    float s = 0.0f;
    for (int c = threadIdx.x; c < H; c += kThreads) s += to_f32(row[c]);
    mean = block_sum2(s, 0.0f).x / H;
  }
  float v = 0.0f;
  for (int c = threadIdx.x; c < H; c += kThreads) {
    const float d = to_f32(row[c]) - mean;
    v = fmaf(d, d, v);
  }
  const float var = block_sum2(v, 0.0f).x / H;
  return make_float2(mean, 1.0f / sqrtf(var + eps));
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_any_kernel(const T* x, const T* __restrict__ weight, const T* __restrict__ bias, T* out,
                          int64_t rows, int H, float eps) {
  pdl_wait();
  pdl_trigger();
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    const T* row = x + t * H;
    const float2 st = row_stats<T, true>(row, H, eps);
    for (int c = threadIdx.x; c < H; c += kThreads) {
      const float y = (to_f32(row[c]) - st.x) * st.y * to_f32(weight[c]);
      store_elem(out + t * H + c, bias != nullptr ? y + to_f32(bias[c]) : y);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- row teams
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int V = 8;
  __device__ static void get(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 put(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};
template <> struct Vec<float> {
  static constexpr int V = 4;
  __device__ static void get(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
  __device__ static uint4 put(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

__device__ __forceinline__ void copy16_async(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kMaxTeam = 512;
constexpr int kMaxRing = 224 * 1024;
// row groups in shared memory, the current one included
__host__ __device__ constexpr int stages_of(int vpt) { return vpt == 4 ? 2 : 3; }

// Sums of N values over the `tpr` threads of a team (whole warps), in every
// thread: butterflies, then the warps' sums in order.  Two buffers in turn,
// so one barrier a call is enough.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int tpr, float (*s_red)[kMaxTeam / 32][4], int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (tpr == 32) return;            // uniform over the block
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s_red[buf][warp][i] = v[i];
  __syncthreads();
  const int first = static_cast<int>(threadIdx.x) / tpr * (tpr >> 5);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = 0; w < tpr >> 5; ++w) {
    const float4 q = *reinterpret_cast<const float4*>(s_red[buf][first + w]);
    const float a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += a[i];
  }
  buf ^= 1;
}

// One thread's share of the row ring: ARR arrays of VPT vectors a row group.
template <int VPT, int ARR> struct Ring {
  uint4* base;
  int threads;
  __device__ __forceinline__ uint4* at(int stage, int arr, int j) const {
    return base + ((stage * ARR + arr) * VPT + j) * threads + threadIdx.x;
  }
};

template <typename T, int VPT>
__global__ void __launch_bounds__(kMaxTeam)
    layer_norm_rows_kernel(const T* x_, const T* __restrict__ w_, const T* __restrict__ b_, T* out_,
                           int64_t rows, int H, float eps, int tpr) {
  constexpr int V = Vec<T>::V, kStages = stages_of(VPT);
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ __align__(16) float s_red[2][kMaxTeam / 32][4];
  pdl_wait();
  pdl_trigger();
  const Ring<VPT, 1> ring{reinterpret_cast<uint4*>(s_dyn), static_cast<int>(blockDim.x)};
  const uint4* x = reinterpret_cast<const uint4*>(x_);
  const uint4* w = reinterpret_cast<const uint4*>(w_);
  const uint4* bias = reinterpret_cast<const uint4*>(b_);
  uint4* out = reinterpret_cast<uint4*>(out_);
  const int nv = H / V, team = static_cast<int>(threadIdx.x) / tpr, me = static_cast<int>(threadIdx.x) - team * tpr;
  const int rpb = static_cast<int>(blockDim.x) / tpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
  const float inv_h = 1.0f / static_cast<float>(H);
  auto fetch = [&](int64_t t, int stage) {
    if (t < rows)
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (me + j * tpr < nv) copy16_async(ring.at(stage, 0, j), x + t * nv + me + j * tpr);
    copy_commit();
  };
  int64_t base = static_cast<int64_t>(blockIdx.x) * rpb;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(base + s * step + team, s);
  int stage = 0, buf = 0;
  for (; base < rows; base += step) {
    const int64_t t = base + team;
    fetch(t + (kStages - 1) * step, (stage + kStages - 1) % kStages);
    copy_wait<kStages - 1>();
    float xv[VPT][V];
    float s1[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool mine = t < rows && me + j * tpr < nv;
      const uint4 q = mine ? *ring.at(stage, 0, j) : make_uint4(0, 0, 0, 0);
      Vec<T>::get(q, xv[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) s1[0] += xv[j][i];
    }
    team_sum<1>(s1, tpr, s_red, buf);
    const float mean = s1[0] * inv_h;
    float s2[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (me + j * tpr < nv)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xv[j][i] -= mean;
          s2[0] = fmaf(xv[j][i], xv[j][i], s2[0]);
        }
    team_sum<1>(s2, tpr, s_red, buf);
    const float r = 1.0f / sqrtf(s2[0] * inv_h + eps);
    if (t < rows)
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = me + j * tpr;
        if (c >= nv) continue;
        float wv[V], bv[V];
        Vec<T>::get(w[c], wv);
        Vec<T>::get(bias != nullptr ? bias[c] : make_uint4(0, 0, 0, 0), bv);
#pragma unroll
        for (int i = 0; i < V; ++i) xv[j][i] = fmaf(xv[j][i] * r, wv[i], bv[i]);
        out[t * nv + c] = Vec<T>::put(xv[j]);
      }
    stage = (stage + 1) % kStages;
  }
  copy_wait<0>();
}

template <typename T, int VPT, bool LAYER, bool RES>
__global__ void __launch_bounds__(kMaxTeam)
    norm_backward_rows_kernel(const T* x_, const T* __restrict__ w_, const T* dout_, const T* dres_, T* dx_,
                              float* __restrict__ part_w, float* __restrict__ part_b, int64_t rows, int H,
                              float eps, int tpr) {
  constexpr int V = Vec<T>::V, ARR = RES ? 3 : 2, kStages = stages_of(VPT);
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ __align__(16) float s_red[2][kMaxTeam / 32][4];
  pdl_wait();
  pdl_trigger();
  const Ring<VPT, ARR> ring{reinterpret_cast<uint4*>(s_dyn), static_cast<int>(blockDim.x)};
  const uint4* src[3] = {reinterpret_cast<const uint4*>(x_), reinterpret_cast<const uint4*>(dout_),
                         reinterpret_cast<const uint4*>(dres_)};
  uint4* dx = reinterpret_cast<uint4*>(dx_);
  const int nv = H / V, team = static_cast<int>(threadIdx.x) / tpr, me = static_cast<int>(threadIdx.x) - team * tpr;
  const int rpb = static_cast<int>(blockDim.x) / tpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
  const float inv_h = 1.0f / static_cast<float>(H);
  auto fetch = [&](int64_t t, int stage) {
    if (t < rows)
#pragma unroll
      for (int a = 0; a < ARR; ++a)
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          if (me + j * tpr < nv) copy16_async(ring.at(stage, a, j), src[a] + t * nv + me + j * tpr);
    copy_commit();
  };
  int64_t base = static_cast<int64_t>(blockIdx.x) * rpb;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(base + s * step + team, s);
  uint4 wq[VPT];
  float aw[VPT][V], ab[VPT][V];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    wq[j] = me + j * tpr < nv ? reinterpret_cast<const uint4*>(w_)[me + j * tpr] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < V; ++i) aw[j][i] = ab[j][i] = 0.0f;
  }
  int stage = 0, buf = 0;
  for (; base < rows; base += step) {
    const int64_t t = base + team;
    fetch(t + (kStages - 1) * step, (stage + kStages - 1) % kStages);
    copy_wait<kStages - 1>();
    // vectors past the row, and rows past the last, read as zeros: they add
    // nothing to any sum (the mean is taken off live elements alone)
    uint4 xq[VPT], gq[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool mine = t < rows && me + j * tpr < nv;
      xq[j] = mine ? *ring.at(stage, 0, j) : make_uint4(0, 0, 0, 0);
      gq[j] = mine ? *ring.at(stage, 1, j) : make_uint4(0, 0, 0, 0);
    }
    float mean = 0.0f;
    if (LAYER) {
      float s1[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float xv[V];
        Vec<T>::get(xq[j], xv);
#pragma unroll
        for (int i = 0; i < V; ++i) s1[0] += xv[i];
      }
      team_sum<1>(s1, tpr, s_red, buf);
      mean = s1[0] * inv_h;
    }
    float s[LAYER ? 3 : 2] = {};          // x'^2, gy x', and gy (x' = x - mean)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (me + j * tpr >= nv) continue;
      float xv[V], gv[V], wv[V];
      Vec<T>::get(xq[j], xv);
      Vec<T>::get(gq[j], gv);
      Vec<T>::get(wq[j], wv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xc = xv[i] - mean, gy = gv[i] * wv[i];
        s[0] = fmaf(xc, xc, s[0]);
        s[1] = fmaf(gy, xc, s[1]);
        if (LAYER) s[LAYER ? 2 : 0] += gy;
      }
    }
    team_sum<LAYER ? 3 : 2>(s, tpr, s_red, buf);
    const float r = 1.0f / sqrtf(s[0] * inv_h + eps);
    const float m1 = LAYER ? s[LAYER ? 2 : 0] * inv_h : 0.0f, m2 = s[1] * r * inv_h;
    if (t < rows)
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = me + j * tpr;
        if (c >= nv) continue;
        float xv[V], gv[V], wv[V], dv[V];
        Vec<T>::get(xq[j], xv);
        Vec<T>::get(gq[j], gv);
        Vec<T>::get(wq[j], wv);
        if (RES) Vec<T>::get(*ring.at(stage, ARR - 1, j), dv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (xv[i] - mean) * r;
          aw[j][i] = fmaf(gv[i], xh, aw[j][i]);
          if (LAYER) ab[j][i] += gv[i];
          const float d = r * (gv[i] * wv[i] - m1 - xh * m2);
          dv[i] = RES ? dv[i] + d : d;
        }
        dx[t * nv + c] = Vec<T>::put(dv);
      }
    stage = (stage + 1) % kStages;
  }
  copy_wait<0>();
  // the teams' sums, in order, through shared memory (the ring is done)
  const int64_t at = static_cast<int64_t>(blockIdx.x) * H;
  float* s_sum = reinterpret_cast<float*>(s_dyn);
#pragma unroll
  for (int pass = 0; pass < (LAYER ? 2 : 1); ++pass) {
    float* part = pass == 0 ? part_w : part_b;
    if (part == nullptr) continue;        // uniform
    for (int turn = 0; turn < rpb; ++turn) {
      __syncthreads();
      if (team == turn)
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int c = (me + j * tpr) * V;
          if (c >= H) continue;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float v = pass == 0 ? aw[j][i] : ab[j][i];
            if (turn > 0) v = s_sum[c + i] + v;
            if (turn + 1 < rpb) s_sum[c + i] = v;
            else part[at + c + i] = v;
          }
        }
    }
  }
}

template <typename T, bool LAYER>
__global__ void __launch_bounds__(kThreads)
    norm_backward_any_kernel(const T* x, const T* __restrict__ weight, const T* dout, const T* dres,
                             T* dx, float* __restrict__ part_w, float* __restrict__ part_b,
                             int64_t rows, int H, float eps) {
  pdl_wait();
  pdl_trigger();
  float* pw = part_w + static_cast<int64_t>(blockIdx.x) * H;
  float* pb = part_b == nullptr ? nullptr : part_b + static_cast<int64_t>(blockIdx.x) * H;
  bool first = true;
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    const T* row = x + t * H;
    const T* grow = dout + t * H;
    const float2 st = row_stats<T, LAYER>(row, H, eps);
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < H; c += kThreads) {
      const float gy = to_f32(grow[c]) * to_f32(weight[c]);
      s1 += gy;
      s2 = fmaf(gy, (to_f32(row[c]) - st.x) * st.y, s2);
    }
    const float2 m = block_sum2(s1, s2);
    const float m1 = LAYER ? m.x / H : 0.0f, m2 = m.y / H;
    for (int c = threadIdx.x; c < H; c += kThreads) {
      const float g = to_f32(grow[c]);
      const float xh = (to_f32(row[c]) - st.x) * st.y;
      float d = st.y * (g * to_f32(weight[c]) - m1 - xh * m2);
      if (dres != nullptr) d += to_f32(dres[t * H + c]);
      pw[c] = first ? g * xh : fmaf(g, xh, pw[c]);
      if (pb != nullptr) pb[c] = first ? g : pb[c] + g;
      store_elem(dx + t * H + c, d);
    }
    first = false;
    __syncthreads();
  }
}

// out[c] = sum over blocks of part[block][c]: 32 columns a block of threads,
// warp w adds the partial rows w, w + 8, ... in order, then the warps' sums
// are added in order.
__global__ void __launch_bounds__(kThreads)
    norm_partials_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, int blocks,
                         int H, float* __restrict__ dweight, float* __restrict__ dbias) {
  constexpr int W = kThreads / 32;
  __shared__ float s_sum[W][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float s = 0.0f;
  if (c < H) {
    int b = warp;
    for (; b + 7 * W < blocks; b += 8 * W) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[static_cast<int64_t>(b + i * W) * H + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; b < blocks; b += W) s += part[static_cast<int64_t>(b) * H + c];
  }
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < H) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += s_sum[w][lane];
    (blockIdx.y == 0 ? dweight : dbias)[c] = t;
  }
}

// Threads of a team and the vectors each holds; 0 vectors: the row has no
// whole 16-byte vectors or is too long for a team.
struct TeamShape {
  int vpt, tpr, threads;
};
template <typename T> TeamShape team_shape(int H) {
  constexpr int V = Vec<T>::V, want = 16 / V;        // 16 elements a thread
  TeamShape s{0, 0, 0};
  if (H % V != 0 || H / V > 4 * kMaxTeam) return s;
  const int nv = H / V;
  s.vpt = nv <= 32 ? 1 : nv <= want * kMaxTeam ? want : 4;
  s.tpr = (static_cast<int>(ceil_div(nv, s.vpt)) + 31) / 32 * 32;
  s.threads = s.tpr >= 256 ? s.tpr : 256 / s.tpr * s.tpr;
  return s;
}

// more than 48 KB of shared memory (some of it static) has to be asked for,
// once a device
template <auto Kernel> cudaError_t allow_smem(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  if (bytes <= 40 * 1024) return cudaSuccess;
  cudaGetDevice(&dev);
  const bool cached = dev >= 0 && dev < 64;
  if (cached && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRing);
  if (e == cudaSuccess && cached) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <typename T, int VPT>
cudaError_t forward_rows(const TeamShape& s, int64_t rows, int H, float eps, const void* x, const void* w,
                         const void* b, void* out, int num_sms, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(stages_of(VPT)) * VPT * s.threads * 16;
  const cudaError_t e = allow_smem<layer_norm_rows_kernel<T, VPT>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t groups = ceil_div(rows, s.threads / s.tpr);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(groups, static_cast<int64_t>(num_sms) * (1024 / s.threads)));
  return launch_chained(layer_norm_rows_kernel<T, VPT>, grid, s.threads, smem, stream, static_cast<const T*>(x), static_cast<const T*>(w),
                        static_cast<const T*>(b), static_cast<T*>(out), rows, H, eps, s.tpr);
}

template <typename T, int VPT, bool LAYER, bool RES>
cudaError_t backward_rows(const TeamShape& s, const NormBackwardArgs& a, float* part_b, int blocks,
                          cudaStream_t stream) {
  size_t smem = static_cast<size_t>(stages_of(VPT)) * (RES ? 3 : 2) * VPT * s.threads * 16;
  smem = std::max(smem, static_cast<size_t>(a.H) * sizeof(float));
  const cudaError_t e = allow_smem<norm_backward_rows_kernel<T, VPT, LAYER, RES>>(smem);
  if (e != cudaSuccess) return e;
  return launch_chained(norm_backward_rows_kernel<T, VPT, LAYER, RES>, static_cast<unsigned>(blocks), s.threads,
                        smem, stream, static_cast<const T*>(a.x), static_cast<const T*>(a.weight),
                        static_cast<const T*>(a.dout), static_cast<const T*>(a.dres), static_cast<T*>(a.dx),
                        a.partials, part_b, a.T, a.H, a.eps, s.tpr);
}

template <typename T, int VPT>
cudaError_t backward_rows_of(const TeamShape& s, const NormBackwardArgs& a, float* part_b, int blocks,
                             cudaStream_t stream) {
  if (a.layer)
    return a.dres != nullptr ? backward_rows<T, VPT, true, true>(s, a, part_b, blocks, stream)
                             : backward_rows<T, VPT, true, false>(s, a, part_b, blocks, stream);
  return a.dres != nullptr ? backward_rows<T, VPT, false, true>(s, a, part_b, blocks, stream)
                           : backward_rows<T, VPT, false, false>(s, a, part_b, blocks, stream);
}

template <typename T>
cudaError_t backward_any(const NormBackwardArgs& a, int blocks, float* part_b, cudaStream_t stream) {
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.weight);
  const T* g = static_cast<const T*>(a.dout);
  const T* r = static_cast<const T*>(a.dres);
  auto* kernel = a.layer ? norm_backward_any_kernel<T, true> : norm_backward_any_kernel<T, false>;
  return launch_chained(kernel, static_cast<unsigned>(blocks), kThreads, 0, stream, x, w, g, r,
                        static_cast<T*>(a.dx), a.partials, part_b, a.T, a.H, a.eps);
}

template <typename T>
cudaError_t forward_of(int64_t rows, int H, float eps, const void* x, const void* w, const void* b, void* out,
                       int num_sms, cudaStream_t stream) {
  const TeamShape s = team_shape<T>(H);
  if (s.vpt == 1) return forward_rows<T, 1>(s, rows, H, eps, x, w, b, out, num_sms, stream);
  if (s.vpt == 2) return forward_rows<T, 2>(s, rows, H, eps, x, w, b, out, num_sms, stream);
  if (s.vpt == 4) return forward_rows<T, 4>(s, rows, H, eps, x, w, b, out, num_sms, stream);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(rows, static_cast<int64_t>(num_sms) * 8));
  return launch_chained(layer_norm_any_kernel<T>, grid, kThreads, 0, stream, static_cast<const T*>(x),
                        static_cast<const T*>(w), static_cast<const T*>(b), static_cast<T*>(out), rows, H, eps);
}

// blocks of the partial sums, and the launch that writes them
template <typename T>
cudaError_t backward_of(const NormBackwardArgs& a, float* part_b, int num_sms, int* blocks, cudaStream_t stream) {
  const TeamShape s = team_shape<T>(a.H);
  const int64_t groups = s.vpt == 0 ? a.T : ceil_div(a.T, s.threads / s.tpr);
  const int64_t resident = static_cast<int64_t>(num_sms) * (s.vpt == 0 ? 4 : s.threads <= 384 ? 2 : 1);
  *blocks = static_cast<int>(std::min<int64_t>(groups, std::min<int64_t>(resident, kNormMaxBlocks)));
  if (*blocks == 0) return cudaSuccess;
  if (s.vpt == 1) return backward_rows_of<T, 1>(s, a, part_b, *blocks, stream);
  if (s.vpt == 2) return backward_rows_of<T, 2>(s, a, part_b, *blocks, stream);
  if (s.vpt == 4) return backward_rows_of<T, 4>(s, a, part_b, *blocks, stream);
  return backward_any<T>(a, *blocks, part_b, stream);
}

}  // namespace

cudaError_t launch_layer_norm(int64_t T, int H, int dtype, float eps, const void* x,
                              const void* weight, const void* bias, void* out, int num_sms,
                              cudaStream_t stream) {
  return dtype == MOE_BF16 ? forward_of<__nv_bfloat16>(T, H, eps, x, weight, bias, out, num_sms, stream)
                           : forward_of<float>(T, H, eps, x, weight, bias, out, num_sms, stream);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& a, int num_sms, cudaStream_t stream) {
  float* part_b = a.dbias != nullptr ? a.partials + static_cast<int64_t>(kNormMaxBlocks) * a.H : nullptr;
  int blocks = 0;
  const cudaError_t e = a.dtype == MOE_BF16 ? backward_of<__nv_bfloat16>(a, part_b, num_sms, &blocks, stream)
                                            : backward_of<float>(a, part_b, num_sms, &blocks, stream);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.H, 32)), a.dbias != nullptr ? 2 : 1);
  return launch_chained(norm_partials_kernel, grid, dim3(kThreads), 0, stream,
                        static_cast<const float*>(a.partials), static_cast<const float*>(part_b), blocks,
                        a.H, a.dweight, a.dbias);
}

}  // namespace moe
