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
//
// Both passes are HBM-bound with little to spare for arithmetic (70 to 80
// instructions a vector of 8 columns).  A lane takes 8 columns (4 pairs) at a
// time, so that every load and store of a warp is one run of memory, and four
// of them are in flight before any is used.  A team of lanes owns a row, so
// that its weight is looked up once.  Measured on a B200 (65536 rows, I = 2048,
// bf16): checkpoint 194 us (5.5 TB/s, 84% of the measured copy bandwidth; a
// thread per 32 columns took 218 us), backward 224 us (6.0 TB/s, 91%; 310 us);
// fp32: 293 us (6.4 TB/s, 99%) and 394 us (6.2 TB/s, 95%).  Narrow rows stay
// below that, with fewer loads in flight a lane and a row's look-ups and sums for
// few columns: I = 64, bf16, 15 us and 19 us (2.3 TB/s).
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

// 8 columns (or 4: the h side) of a row as they lie in memory
template <typename T> struct Cols;
template <> struct Cols<__nv_bfloat16> {
  using Eight = uint4;
  using Four = uint2;
  __device__ static void get(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static void get(const uint2& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x << 16);
    v[1] = __uint_as_float(q.x & 0xFFFF0000u);
    v[2] = __uint_as_float(q.y << 16);
    v[3] = __uint_as_float(q.y & 0xFFFF0000u);
  }
  __device__ static uint4 put(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
  __device__ static uint2 put(const float (&v)[4]) {
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
  // largest magnitude as fp32 bits (at or past an infinity's: not finite)
  __device__ static uint32_t top(const uint4& q, const float (&)[8]) {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t t = __vmaxu2(__vmaxu2(q.x & m, q.y & m), __vmaxu2(q.z & m, q.w & m));
    return max(t & 0xFFFF0000u, t << 16);
  }
};
struct alignas(16) F32x8 { float4 a, b; };
template <> struct Cols<float> {
  using Eight = F32x8;
  using Four = float4;
  __device__ static void get(const F32x8& q, float (&v)[8]) {
    v[0] = q.a.x; v[1] = q.a.y; v[2] = q.a.z; v[3] = q.a.w;
    v[4] = q.b.x; v[5] = q.b.y; v[6] = q.b.z; v[7] = q.b.w;
  }
  __device__ static void get(const float4& q, float (&v)[4]) { v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w; }
  __device__ static F32x8 put(const float (&v)[8]) {
    return F32x8{make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
  }
  __device__ static float4 put(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
  __device__ static uint32_t top(const F32x8&, const float (&v)[8]) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return t;
  }
};

// 2^(b - 127) as fp32 for b in [0, 254]: b = 0 is the subnormal 2^-127
__device__ __forceinline__ float pow2_of_byte(int b) {
  return __uint_as_float(b > 0 ? static_cast<uint32_t>(b) << 23 : 0x00400000u);
}

// scale byte of a block whose largest finite magnitude has these bits
__device__ __forceinline__ int scale_byte(uint32_t bits) {
  const int b = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return b > 0 ? b : 0;
}

__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) <= FLT_MAX; }

// e4m3 bits of 8 finite scaled values (|v inv| <= 448)
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// two e4m3 values as fp32 (exact)
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t bits) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(bits), __NV_E4M3);
  return __half22float2(__half2(h));
}

// s = 1 / (1 + e^-g) and c = 1 - s from t = e^-|g|: every quotient divides by a
// number in [1, 2], so no exponential overflows and even the smallest results
// keep their digits.
//   bf16 rows  the fast exponential and division: (12 + 1.2 |g|) 2^-23 relative at
//              most, far below a bf16 step
//   fp32 rows  expf (2 ulp): 5 x 2^-23 whatever g is.  The passes have the time
//              for it, with twice the bytes for the same arithmetic; a division
//              that rounds correctly would save 3 units of 2^-24 more and take 5%
//              on the forward pass (65536 rows, I = 2048: 308 us against 293)
template <typename T> struct Sigmoid {
  float s, c;
  __device__ __forceinline__ explicit Sigmoid(float g) {
    const float t = __expf(-fabsf(g));
    s = __fdividef(g >= 0.0f ? 1.0f : t, 1.0f + t);
    c = 1.0f - s;
  }
};
template <> struct Sigmoid<float> {
  float s, c;
  __device__ __forceinline__ explicit Sigmoid(float g) {
    const float t = expf(-fabsf(g)), inv = __fdividef(1.0f, 1.0f + t);   // 2 ulp
    s = g >= 0.0f ? inv : t * inv;
    c = g >= 0.0f ? t * inv : inv;
  }
};

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

// rows that are live; a count outside [0, rows] is recorded and read as the
// nearer end
__device__ __forceinline__ int64_t live_rows(const int32_t* live, const RowWeight& rw) {
  if (live == nullptr) return rw.rows;
  const int64_t n = *live;
  if (n >= 0 && n <= rw.rows) return n;
  if (blockIdx.x == 0 && threadIdx.x == 0) record_status(rw.status, DEV_BAD_ROW);
  return n < 0 ? 0 : rw.rows;
}

constexpr int kBatch = 4;       // vectors of 8 columns a thread has in flight

// A team of `lanes` lanes (4..32) or, WIDE, a whole block per row; the 4 lanes
// that hold a block of 32 columns agree on its scale.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads)
    swiglu_checkpoint_kernel(const int32_t* live_ptr, RowWeight rw, int I, int lanes, const T* __restrict__ gu,
                             T* __restrict__ h, uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  using C = Cols<T>;
  pdl_wait();
  pdl_trigger();
  const int nv = I / 4;                                      // vectors of 8 columns a row
  const int team_size = WIDE ? kThreads : lanes;
  const int me = static_cast<int>(threadIdx.x) & (team_size - 1);
  const int64_t live_n = live_rows(live_ptr, rw);
  const int teams = kThreads / team_size;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * teams; base < live_n; base += step) {
    const int64_t r = base + static_cast<int>(threadIdx.x) / team_size;
    const bool mine = r < live_n;
    const float w = mine ? rw.weight(rw.slot(r)) : 0.0f;
    const int64_t row = (mine ? r : 0) * nv;
    // every lane of a warp runs the same rounds (the shuffles)
    for (int vb = 0; vb < nv; vb += kBatch * team_size) {
      typename C::Eight in[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = vb + b * team_size + me;
        if (mine && v < nv) in[b] = reinterpret_cast<const typename C::Eight*>(gu)[row + v];
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = vb + b * team_size + me;
        const bool live = mine && v < nv;                    // nv is a multiple of 4: a block's lanes agree
        float x[8];
        uint32_t top = 0;
        if (live) {
          C::get(in[b], x);
          top = C::top(in[b], x);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float out[4];
        if (live)
#pragma unroll
          for (int j = 0; j < 4; ++j) out[j] = w * (x[2 * j] * Sigmoid<T>(x[2 * j]).s) * x[2 * j + 1];
        if (__any_sync(0xffffffffu, top >= 0x7F800000u)) {   // rare: the finite values' top, NaN for the others
          uint32_t t = 0;
          if (live)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (is_finite(x[j])) t = max(t, __float_as_uint(x[j]) & 0x7FFFFFFFu);
              else x[j] = __int_as_float(0x7FC00000);        // e4m3 has no infinity
            }
          t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
          top = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
        }
        if (!live) continue;
        const int byte = scale_byte(top);
        reinterpret_cast<typename C::Four*>(h)[row + v] = C::put(out);
        reinterpret_cast<uint2*>(q)[row + v] = e4m3x8(x, pow2_of_byte(254 - byte));
        if ((me & 3) == 0) scale[(row + v) >> 2] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// A team of `lanes` lanes (4..32) or, WIDE, a whole block per row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(const int32_t* live_ptr, RowWeight rw, int I, int lanes,
                           const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                           const T* __restrict__ dh, T* __restrict__ dgu, float* __restrict__ d_topk_w,
                           T* __restrict__ h) {
  using C = Cols<T>;
  __shared__ float s_part[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int nv = I / 4;
  const int team_size = WIDE ? kThreads : lanes;
  const int me = static_cast<int>(threadIdx.x) & (team_size - 1);
  const int64_t live = live_rows(live_ptr, rw);
  const int teams = kThreads / team_size;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  // every lane of a warp runs the same number of rounds (the shuffles below)
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * teams; base < live; base += step) {
    const int64_t r = base + static_cast<int>(threadIdx.x) / team_size;
    const bool mine = r < live;
    const int64_t slot = mine ? rw.slot(r) : -1;
    const float w = rw.weight(slot);
    const int64_t row = (mine ? r : 0) * nv;
    float dw = 0.0f;
    for (int v0 = me; v0 < nv && mine; v0 += kBatch * team_size) {
      uint2 qv[kBatch];
      typename C::Four dv[kBatch];
      uint32_t sb[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = v0 + b * team_size;
        if (v >= nv) continue;
        qv[b] = reinterpret_cast<const uint2*>(q)[row + v];
        dv[b] = reinterpret_cast<const typename C::Four*>(dh)[row + v];
        sb[b] = scale[(row + v) >> 2];
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = v0 + b * team_size;
        if (v >= nv) continue;
        const float s2 = pow2_of_byte(static_cast<int>(sb[b]));
        float d[4], o[8], hv[4];
        C::get(dv[b], d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 gu = e4m3x2_f32(((j < 2 ? qv[b].x : qv[b].y) >> (16 * (j & 1))) & 0xFFFFu);
          const float g = gu.x * s2, u = gu.y * s2;
          const Sigmoid<T> sg(g);
          const float s = sg.s, a = g * s, au = a * u, wd = w * d[j];
          dw = fmaf(d[j], au, dw);
          o[2 * j] = wd * u * (s * fmaf(g, sg.c, 1.0f));
          o[2 * j + 1] = wd * a;
          hv[j] = w * au;
        }
        reinterpret_cast<typename C::Eight*>(dgu)[row + v] = C::put(o);
        if (h != nullptr) reinterpret_cast<typename C::Four*>(h)[row + v] = C::put(hv);
      }
    }
    if (d_topk_w == nullptr) continue;                       // uniform
    for (int o = min(team_size, 32) >> 1; o > 0; o >>= 1) dw += __shfl_xor_sync(0xffffffffu, dw, o);
    if (WIDE) {
      if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = dw;
      __syncthreads();
      if (threadIdx.x == 0) {
        dw = 0.0f;
        for (int i = 0; i < kThreads / 32; ++i) dw += s_part[i];
      }
      __syncthreads();
    }
    if (me == 0 && slot >= 0) d_topk_w[slot] = dw;
  }
}

// The fewest lanes (4..32) that cover a row; with too few rows for that many
// teams, and long ones, a block per row.
struct TeamShape {
  int lanes;
  bool wide;
  unsigned grid;
};
TeamShape team_shape(const SwigluArgs& a, int num_sms) {
  TeamShape s{4, false, 1};
  const int nv = a.I / 4;
  while (s.lanes < nv && s.lanes < 32) s.lanes <<= 1;
  s.wide = nv >= 2 * kThreads / kBatch && a.rows < static_cast<int64_t>(num_sms) * 16;
  const int64_t blocks = s.wide ? a.rows : ceil_div(a.rows, kThreads / s.lanes);
  s.grid = static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * 16));
  return s;
}

template <typename T>
cudaError_t checkpoint_of(const SwigluArgs& a, const void* gu, void* h, void* q, uint8_t* scale, int num_sms,
                          cudaStream_t stream) {
  const RowWeight rw{a.perm_slot, a.topk_w, a.rows, a.status};
  const TeamShape s = team_shape(a, num_sms);
  return launch_chained(s.wide ? swiglu_checkpoint_kernel<T, true> : swiglu_checkpoint_kernel<T, false>, s.grid,
                        kThreads, 0, stream, a.live, rw, a.I, s.lanes, static_cast<const T*>(gu),
                        static_cast<T*>(h), static_cast<uint8_t*>(q), scale);
}

template <typename T>
cudaError_t backward_of(const SwigluArgs& a, const void* q, const uint8_t* scale, const void* dh, void* dgu,
                        float* d_topk_w, void* h, int num_sms, cudaStream_t stream) {
  const RowWeight rw{a.perm_slot, a.topk_w, a.rows, a.status};
  const TeamShape s = team_shape(a, num_sms);
  return launch_chained(s.wide ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>, s.grid,
                        kThreads, 0, stream, a.live, rw, a.I, s.lanes, static_cast<const uint8_t*>(q), scale,
                        static_cast<const T*>(dh), static_cast<T*>(dgu), d_topk_w, static_cast<T*>(h));
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const SwigluArgs& a, const void* gu, void* h, void* q,
                                     uint8_t* scale, int num_sms, cudaStream_t stream) {
  return a.dtype == MOE_BF16 ? checkpoint_of<__nv_bfloat16>(a, gu, h, q, scale, num_sms, stream)
                             : checkpoint_of<float>(a, gu, h, q, scale, num_sms, stream);
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
  return a.dtype == MOE_BF16 ? backward_of<__nv_bfloat16>(a, q, scale, dh, dgu, d_topk_w, h, num_sms, stream)
                             : backward_of<float>(a, q, scale, dh, dgu, d_topk_w, h, num_sms, stream);
}

}  // namespace moe
