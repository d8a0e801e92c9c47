// The experts' SwiGLU over gate_up rows with an 8-bit checkpoint of those
// rows, and its backward pass from the checkpoint.
//
// Checkpoint: every 32 consecutive columns of gu [R, 2I] (16 gate/up pairs,
// columns interleaved) share one power of two s = 2^(b - 127), b the least
// byte in [0, 254] with amax <= 448 s, and hold x / s as e4m3 rounded to
// nearest even.  Dividing by a power of two is exact, so the stored value is
// the one nearest to x on its grid (half a step: 2^-4 of |x|, or 2^-10 s for
// the smallest), the same bits on every device, and q s is exact in bf16.
// With amax = 1.m 2^(E - 127), 448 = 1.75 2^8: b = E - 8, plus one when
// 1.m > 1.75.
//
// Backward, for a row of weight w:  s = 1 / (1 + e^-g), a = g s,
//   dg = w dh u s (1 + g (1 - s)),  du = w dh a,  dw = sum_j dh a u,
// all in fp32, each output rounded once.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 32;      // columns of one scale

template <typename T> __device__ __forceinline__ void load16(const T* p, float (&v)[16]);
template <> __device__ __forceinline__ void load16<float>(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
  }
}
template <> __device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 f = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
template <typename T> __device__ __forceinline__ void store16(T* p, const float (&v)[16]);
template <> __device__ __forceinline__ void store16<float>(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <> __device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                   pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}

// 2^(b - 127) as fp32 for b in [0, 254]: b = 0 is the subnormal 2^-127
__device__ __forceinline__ float pow2_of_byte(int b) {
  return __uint_as_float(b > 0 ? static_cast<uint32_t>(b) << 23 : 0x00400000u);
}

// scale byte of a block whose largest finite magnitude is amax
__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int b = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return b > 0 ? b : 0;
}

__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) <= FLT_MAX; }

// e4m3 bits of two scaled values (|v| <= 448, or not finite: NaN)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi, float inv) {
  const float2 v = make_float2(is_finite(lo) ? lo * inv : __int_as_float(0x7FC00000),
                               is_finite(hi) ? hi * inv : __int_as_float(0x7FC00000));
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

// two e4m3 values as fp32 (exact)
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t bits) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(bits), __NV_E4M3);
  return __half22float2(__half2(h));
}

// 1 / (1 + e^-g) from t = e^-|g|: both forms divide by a number in [1, 2], so
// no exponential overflows and the fast division (2 ulp) keeps even the
// smallest results (it returns 0 for divisors past 2^126).
__device__ __forceinline__ float sigmoid(float g) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g >= 0.0f ? 1.0f : t, 1.0f + t);
}

struct RowWeight {
  const int32_t* perm_slot;
  const float* topk_w;
  int64_t rows;
  int32_t* status;
  // slot of row r (-1: out of range, recorded) and its weight
  __device__ __forceinline__ int64_t slot(int64_t r) const {
    if (perm_slot == nullptr) return r;
    const int s = perm_slot[r];
    if (s >= 0 && s < rows) return s;
    record_status(status, DEV_BAD_ROW);
    return -1;
  }
  __device__ __forceinline__ float weight(int64_t s) const {
    return topk_w == nullptr ? 1.0f : (s < 0 ? 0.0f : topk_w[s]);
  }
};

__device__ __forceinline__ int64_t live_rows(const int32_t* live, int64_t rows) {
  if (live == nullptr) return rows;
  const int64_t n = *live;
  return n < 0 ? 0 : (n > rows ? rows : n);
}

// one thread per block of 32 columns
template <typename T>
__global__ void __launch_bounds__(kThreads)
    swiglu_checkpoint_kernel(const int32_t* live_ptr, RowWeight rw, int I, const T* __restrict__ gu,
                             T* __restrict__ h, uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const int nb = I / 16;
  const int64_t n = live_rows(live_ptr, rw.rows) * nb;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / nb;
    const float w = rw.weight(rw.slot(r));
    float a[16], b[16], out[16];
    load16(gu + i * kBlock, a);
    load16(gu + i * kBlock + 16, b);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (is_finite(a[j])) amax = fmaxf(amax, fabsf(a[j]));
      if (is_finite(b[j])) amax = fmaxf(amax, fabsf(b[j]));
    }
    const int byte = scale_byte(amax);
    const float inv = pow2_of_byte(254 - byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      out[j] = w * (a[2 * j] * sigmoid(a[2 * j])) * a[2 * j + 1];
      out[8 + j] = w * (b[2 * j] * sigmoid(b[2 * j])) * b[2 * j + 1];
    }
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = e4m3x2(a[4 * j], a[4 * j + 1], inv) | e4m3x2(a[4 * j + 2], a[4 * j + 3], inv) << 16;
      p[4 + j] = e4m3x2(b[4 * j], b[4 * j + 1], inv) | e4m3x2(b[4 * j + 2], b[4 * j + 3], inv) << 16;
    }
    store16(h + i * 16, out);
    uint4* dst = reinterpret_cast<uint4*>(q + i * kBlock);
    dst[0] = make_uint4(p[0], p[1], p[2], p[3]);
    dst[1] = make_uint4(p[4], p[5], p[6], p[7]);
    scale[i] = static_cast<uint8_t>(byte);
  }
}

// one warp per row, a block of 32 columns a lane at a time
template <typename T>
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(const int32_t* live_ptr, RowWeight rw, int I, const uint8_t* __restrict__ q,
                           const uint8_t* __restrict__ scale, const T* __restrict__ dh,
                           T* __restrict__ dgu, float* __restrict__ d_topk_w, T* __restrict__ h) {
  pdl_wait();
  pdl_trigger();
  const int nb = I / 16;
  const int lane = threadIdx.x & 31;
  const int64_t live = live_rows(live_ptr, rw.rows);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); r < live;
       r += warps) {
    const int64_t slot = rw.slot(r);
    const float w = rw.weight(slot);
    float dw = 0.0f;
    for (int b = lane; b < nb; b += 32) {
      const int64_t i = r * nb + b;
      const float s2 = pow2_of_byte(scale[i]);
      const uint4 q0 = reinterpret_cast<const uint4*>(q + i * kBlock)[0];
      const uint4 q1 = reinterpret_cast<const uint4*>(q + i * kBlock)[1];
      const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
      float d[16], o0[16], o1[16], hv[16];
      load16(dh + i * 16, d);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 gu = e4m3x2_f32((qw[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
        const float g = gu.x * s2, u = gu.y * s2;
        const float s = sigmoid(g);
        const float a = g * s;
        dw = fmaf(d[j], a * u, dw);
        const float wd = w * d[j];
        const float dg = wd * u * s * (1.0f + g * (1.0f - s)), du = wd * a;
        if (j < 8) { o0[2 * j] = dg; o0[2 * j + 1] = du; }
        else { o1[2 * j - 16] = dg; o1[2 * j - 15] = du; }
        hv[j] = w * a * u;
      }
      store16(dgu + i * kBlock, o0);
      store16(dgu + i * kBlock + 16, o1);
      if (h != nullptr) store16(h + i * 16, hv);
    }
    if (d_topk_w != nullptr) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dw += __shfl_xor_sync(0xffffffffu, dw, o);
      if (lane == 0 && slot >= 0) d_topk_w[slot] = dw;
    }
  }
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const SwigluArgs& a, const void* gu, void* h, void* q,
                                     uint8_t* scale, int num_sms, cudaStream_t stream) {
  const RowWeight rw{a.perm_slot, a.topk_w, a.rows, a.status};
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(ceil_div(a.rows * (a.I / 16), kThreads), static_cast<int64_t>(num_sms) * 8));
  if (a.dtype == MOE_BF16)
    return launch_chained(swiglu_checkpoint_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, a.live,
                          rw, a.I, static_cast<const __nv_bfloat16*>(gu),
                          static_cast<__nv_bfloat16*>(h), static_cast<uint8_t*>(q), scale);
  return launch_chained(swiglu_checkpoint_kernel<float>, grid, kThreads, 0, stream, a.live, rw, a.I,
                        static_cast<const float*>(gu), static_cast<float*>(h),
                        static_cast<uint8_t*>(q), scale);
}

cudaError_t launch_swiglu_backward(const SwigluArgs& a, const void* q, const uint8_t* scale,
                                   const void* dh, void* dgu, float* d_topk_w, void* h,
                                   int num_sms, cudaStream_t stream) {
  // slots that hold no row get 0: with no row map and every row live there
  // are none
  if (d_topk_w != nullptr && (a.live != nullptr || a.perm_slot != nullptr)) {
    const cudaError_t e = cudaMemsetAsync(d_topk_w, 0, static_cast<size_t>(a.rows) * 4, stream);
    if (e != cudaSuccess) return e;
  }
  const RowWeight rw{a.perm_slot, a.topk_w, a.rows, a.status};
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(ceil_div(a.rows, kThreads / 32), static_cast<int64_t>(num_sms) * 8));
  const uint8_t* qb = static_cast<const uint8_t*>(q);
  if (a.dtype == MOE_BF16)
    return launch_chained(swiglu_backward_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, a.live, rw,
                          a.I, qb, scale, static_cast<const __nv_bfloat16*>(dh),
                          static_cast<__nv_bfloat16*>(dgu), d_topk_w, static_cast<__nv_bfloat16*>(h));
  return launch_chained(swiglu_backward_kernel<float>, grid, kThreads, 0, stream, a.live, rw, a.I, qb,
                        scale, static_cast<const float*>(dh), static_cast<float*>(dgu), d_topk_w,
                        static_cast<float*>(h));
}

}  // namespace moe
