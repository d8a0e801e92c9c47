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
// takes rows blockIdx.x, + gridDim.x, ... and adds its rows' dout x^ and dout
// into one partial row of its own, column by column always by the same
// thread; a second kernel adds the blocks' partial rows in block order.  No
// atomics: the same bits on every run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

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

// out[c] = sum over blocks of part[block][c], in block order
__global__ void __launch_bounds__(kThreads)
    norm_partials_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, int blocks,
                         int H, float* __restrict__ dweight, float* __restrict__ dbias) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= H) return;
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float s = 0.0f;
  for (int b = 0; b < blocks; ++b) s += part[static_cast<int64_t>(b) * H + c];
  (blockIdx.y == 0 ? dweight : dbias)[c] = s;
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

}  // namespace

cudaError_t launch_layer_norm(int64_t T, int H, int dtype, float eps, const void* x,
                              const void* weight, const void* bias, void* out, int num_sms,
                              cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(T, static_cast<int64_t>(num_sms) * 8));
  if (dtype == MOE_BF16)
    return launch_chained(layer_norm_any_kernel<__nv_bfloat16>, grid, kThreads, 0, stream,
                          static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(weight),
                          static_cast<const __nv_bfloat16*>(bias), static_cast<__nv_bfloat16*>(out), T, H,
                          eps);
  return launch_chained(layer_norm_any_kernel<float>, grid, kThreads, 0, stream,
                        static_cast<const float*>(x), static_cast<const float*>(weight),
                        static_cast<const float*>(bias), static_cast<float*>(out), T, H, eps);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& a, int num_sms, cudaStream_t stream) {
  const int blocks = static_cast<int>(
      std::min<int64_t>(a.T, std::min<int64_t>(static_cast<int64_t>(num_sms) * 4, kNormMaxBlocks)));
  float* part_b = a.dbias != nullptr ? a.partials + static_cast<int64_t>(kNormMaxBlocks) * a.H : nullptr;
  if (blocks > 0) {
    const cudaError_t e = a.dtype == MOE_BF16 ? backward_any<__nv_bfloat16>(a, blocks, part_b, stream)
                                              : backward_any<float>(a, blocks, part_b, stream);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(ceil_div(a.H, kThreads)), a.dbias != nullptr ? 2 : 1);
  return launch_chained(norm_partials_kernel, grid, dim3(kThreads), 0, stream,
                        static_cast<const float*>(a.partials), static_cast<const float*>(part_b), blocks,
                        a.H, a.dweight, a.dbias);
}

}  // namespace moe
