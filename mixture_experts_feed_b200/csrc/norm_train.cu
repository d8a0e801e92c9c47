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
// owns a row, 8 to 32 elements a thread.  Each thread copies its own vectors
// of the rows to come into shared memory with cp.async, two row groups ahead,
// and reads back only what it copied itself: x and dout are read once although
// the statistics need the whole row first, and the loads stay in flight across
// the reductions with no barrier between them.  A row costs one reduction with
// one block barrier (none when a team is one warp): layer norm's mean of the
// next row is summed with the current row's other sums.  Other rows take the
// *_any kernels, which stream them several times.
//
// bf16 rows run into the issue rate before HBM, so the arithmetic is packed two
// fp32 values at a time, the row is read from shared memory in each pass (80
// registers a thread keep two blocks of 384 threads on an SM; fewer, fuller
// threads measured slower: 142 us where this takes 74), and layer norm's four
// sums are scattered over the lanes as they are added.  Measured on a B200:
// RMSNorm backward with residual, 8192 x 6144 bf16, 74 us (5.4 TB/s, 83% of the
// measured copy bandwidth); layer norm backward 80 to 84 us there (3.7 TB/s: 30
// instructions an element) and 21 us on 4096 x 2048; 8192 x 4096 fp32 66 us
// (6.1 TB/s), with residual 84 us (6.4 TB/s); layer norm forward 8192 x 6144 bf16
// 45 us (4.4 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
// RMSNorm rows whose squares pass the fp32 range (moe_rmsnorm sums in fp64) are
// summed again at this scale: values to 2^128 then have squares to 2^116.
constexpr float kDown = 0x1p-70f;

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
  if (!LAYER && !(var <= FLT_MAX)) {        // uniform over the block
    v = 0.0f;
    for (int c = threadIdx.x; c < H; c += kThreads) {
      const float d = to_f32(row[c]) * kDown;
      v = fmaf(d, d, v);
    }
    return make_float2(0.0f, kDown / sqrtf(block_sum2(v, 0.0f).x / H + eps * kDown * kDown));
  }
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
// A 16-byte vector as P pairs
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int V = 8, P = 4;
  __device__ static f32x2 pair(const uint4& q, int i) {
    const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ static uint4 put(const f32x2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(v[i]);
      w[i] = pack_bf16x2(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec<float> {
  static constexpr int V = 4, P = 2;
  __device__ static f32x2 pair(const uint4& q, int i) {
    return i == 0 ? pack2(__uint_as_float(q.x), __uint_as_float(q.y))
                  : pack2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
  __device__ static uint4 put(const f32x2 (&v)[2]) {
    const float2 a = unpack2(v[0]), b = unpack2(v[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};

__device__ __forceinline__ void copy16_async(uint32_t dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kMaxTeam = 512;
// The backward kernels hide their reductions behind other warps: with one or
// two vectors a thread an SM holds 768 threads (80 registers each), as one
// block or two.  fp32 rows of 4 vectors a thread, and bf16 rows of more than
// 6144 values, run up to 512 threads with 128 registers.
__host__ __device__ constexpr int max_threads(int vpt) { return vpt == 4 ? kMaxTeam : vpt == 1 ? 768 : 384; }
__host__ __device__ constexpr int min_blocks(int vpt) { return vpt == 2 ? 2 : 1; }
constexpr int kMaxWarps = 32;
constexpr int kMaxRing = 224 * 1024;
// row groups in shared memory, the current one included (layer norm also reads
// the next one; with three arrays a fourth would not leave room for two blocks)
__host__ __device__ constexpr int stages_of(bool layer, int arrays) { return layer && arrays < 3 ? 4 : 3; }

// Sums of N values (1, 2 or 4) over the `tpr` threads of a team (whole warps;
// at most 16 for two values), in every thread: in each warp, then, past one
// barrier, over the warps' sums.  Two buffers in turn, so one barrier a call is
// enough.  One or two values go by butterflies; four are scattered over the
// lanes as they are summed (the first exchange leaves each lane 2 of them, the
// second 1, three more steps finish: 6 shuffles instead of 20), summed over
// the warps side by side, and broadcast.  ONE: a call that this team alone makes,
// past a barrier of its own.
template <int N, bool ONE = false>
__device__ __forceinline__ void team_sum(float (&v)[N], int tpr, float (*s_red)[4 * kMaxWarps], int& buf) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wpr = tpr >> 5;
  if (N <= 2) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (tpr == 32) return;          // uniform over the block
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s_red[buf][warp * N + i] = v[i];
    if (ONE) asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / tpr), "r"(tpr) : "memory");
    else __syncthreads();
    constexpr int W = kMaxWarps / N;
    const int w = lane & (W - 1);
    const float* part = s_red[buf] + (warp - warp % wpr + w) * N;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = w < wpr ? part[i] : 0.0f;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    buf ^= 1;
    return;
  }
  const bool b0 = lane & 1, b1 = lane & 2;
  const int id = (b0 ? 2 : 0) + (b1 ? 1 : 0);   // the value this lane ends up with
  const float k0 = b0 ? v[N > 2 ? 2 : 0] : v[0], k1 = b0 ? v[N > 3 ? 3 : 0] : v[N > 1 ? 1 : 0];
  const float g0 = b0 ? v[0] : v[N > 2 ? 2 : 0], g1 = b0 ? v[N > 1 ? 1 : 0] : v[N > 3 ? 3 : 0];
  const float c0 = k0 + __shfl_xor_sync(0xffffffffu, g0, 1), c1 = k1 + __shfl_xor_sync(0xffffffffu, g1, 1);
  float a = (b1 ? c1 : c0) + __shfl_xor_sync(0xffffffffu, b1 ? c0 : c1, 2);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (tpr > 32) {                   // uniform over the block
    if (lane < 4) s_red[buf][warp * 4 + id] = a;
    __syncthreads();
    const float* part = s_red[buf] + (warp - warp % wpr) * 4 + id;
    a = 0.0f;
#pragma unroll
    for (int w = 0; w < kMaxWarps; w += 8)
      if (w + (lane >> 2) < wpr) a += part[(w + (lane >> 2)) * 4];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    buf ^= 1;
  }
  v[0] = __shfl_sync(0xffffffffu, a, 0);
  v[N > 1 ? 1 : 0] = __shfl_sync(0xffffffffu, a, 2);
  v[N > 2 ? 2 : 0] = __shfl_sync(0xffffffffu, a, 1);
  v[N > 3 ? 3 : 0] = __shfl_sync(0xffffffffu, a, 3);
}

// What the row kernels share: this thread's place, and its own slots of the
// ring ([stage][ARR * VPT][thread] vectors: a warp's copies and reads are runs
// of 512 bytes).
template <typename T, int VPT, int ARR, int STAGES> struct Team {
  static constexpr int SLOTS = ARR * VPT;
  int nv, tpr, team, me, rpb;
  int64_t rows, step;
  uint4* mine;                 // stage 0
  uint32_t mine_smem;
  int stage_vecs;              // vectors of a stage
  __device__ __forceinline__ Team(int H, int tpr_, int64_t rows_, uint8_t* s_dyn)
      : nv(H / Vec<T>::V), tpr(tpr_), rows(rows_) {
    team = static_cast<int>(threadIdx.x) / tpr;
    me = static_cast<int>(threadIdx.x) - team * tpr;
    rpb = static_cast<int>(blockDim.x) / tpr;
    step = static_cast<int64_t>(gridDim.x) * rpb;
    mine = reinterpret_cast<uint4*>(s_dyn) + threadIdx.x;
    mine_smem = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
    stage_vecs = static_cast<int>(blockDim.x) * SLOTS;
    // vectors past the row's end stay zero: they add nothing to any sum
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) mine[s * stage_vecs + i * static_cast<int>(blockDim.x)] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ bool has(int j) const { return me + j * tpr < nv; }
  __device__ __forceinline__ void fetch(const uint4* const (&src)[3], int64_t t, int stage) const {
    if (t < rows) {
      const int64_t at = t * nv + me;
      const uint32_t dst = mine_smem + static_cast<uint32_t>(stage * stage_vecs) * 16;
#pragma unroll
      for (int a = 0; a < ARR; ++a)
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          if (has(j)) copy16_async(dst + (a * VPT + j) * blockDim.x * 16, src[a] + at + j * tpr);
    }
    copy_commit();
  }
  __device__ __forceinline__ const uint4* slot(int stage) const { return mine + stage * stage_vecs; }
  // this thread's share of the sum of the row in a stage
  __device__ __forceinline__ float row_sum(int stage) const {
    f32x2 acc = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const uint4 q = slot(stage)[j * static_cast<int>(blockDim.x)];
#pragma unroll
      for (int i = 0; i < Vec<T>::P; ++i) acc = add2(acc, Vec<T>::pair(q, i));
    }
    return sum2(acc);
  }
};

template <typename T, int VPT>
__global__ void __launch_bounds__(kMaxTeam, 2)
    layer_norm_rows_kernel(const T* x_, const T* __restrict__ w_, const T* __restrict__ b_, T* out_,
                           int64_t rows, int H, float eps, int tpr) {
  constexpr int P = Vec<T>::P;
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float s_red[2][4 * kMaxWarps];
  pdl_wait();
  pdl_trigger();
  constexpr int STAGES = stages_of(true, 1);
  const Team<T, VPT, 1, STAGES> tm(H, tpr, rows, s_dyn);
  const uint4* const src[3] = {reinterpret_cast<const uint4*>(x_), nullptr, nullptr};
  const uint4* w = reinterpret_cast<const uint4*>(w_);
  const uint4* bias = reinterpret_cast<const uint4*>(b_);
  uint4* out = reinterpret_cast<uint4*>(out_);
  const float inv_h = 1.0f / static_cast<float>(H);
  int64_t base = static_cast<int64_t>(blockIdx.x) * tm.rpb;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) tm.fetch(src, base + s * tm.step + tm.team, s);
  // the mean of the first row; every later one comes with the reduction of
  // the row before it
  int stage = 0, buf = 0;
  copy_wait<STAGES - 2>();
  float s1[1] = {tm.row_sum(0)};
  team_sum<1>(s1, tpr, s_red, buf);
  float mean = s1[0] * inv_h;
  for (; base < rows; base += tm.step) {
    const int64_t t = base + tm.team;
    const int after = stage == STAGES - 1 ? 0 : stage + 1;
    tm.fetch(src, t + (STAGES - 1) * tm.step, stage == 0 ? STAGES - 1 : stage - 1);
    copy_wait<STAGES - 2>();
    const f32x2 neg_mean = pack2(-mean, -mean);
    f32x2 xc[VPT][P], acc = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (tm.has(j)) {
        const uint4 q = tm.slot(stage)[j * static_cast<int>(blockDim.x)];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          xc[j][i] = add2(Vec<T>::pair(q, i), neg_mean);
          acc = fma2(xc[j][i], xc[j][i], acc);
        }
      }
    float s2[2] = {sum2(acc), tm.row_sum(after)};
    team_sum<2>(s2, tpr, s_red, buf);
    mean = s2[1] * inv_h;
    const float r = rsqrtf(s2[0] * inv_h + eps);
    const f32x2 r2 = pack2(r, r);
    if (t < rows)
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (tm.has(j)) {
          const int c = tm.me + j * tpr;
          const uint4 wq = w[c], bq = bias != nullptr ? bias[c] : make_uint4(0, 0, 0, 0);
          f32x2 y[P];
#pragma unroll
          for (int i = 0; i < P; ++i)
            y[i] = fma2(mul2(xc[j][i], r2), Vec<T>::pair(wq, i), Vec<T>::pair(bq, i));
          out[t * tm.nv + c] = Vec<T>::put(y);
        }
    stage = after;
  }
  copy_wait<0>();
}

// A thread's slots of a row (x, then dout, each VPT vectors `stride` apart):
// b += its sums of (x 2^-70)^2 and gy x 2^-70; and x times a power of two.
template <typename T, int VPT>
__device__ __forceinline__ void scaled_sums(const uint4* slots, const uint4 (&wq)[VPT], int stride, float (&b)[2]) {
  f32x2 sxx = 0, sgx = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const uint4 xq = slots[j * stride], gq = slots[(VPT + j) * stride];
#pragma unroll
    for (int i = 0; i < Vec<T>::P; ++i) {
      const f32x2 x = mul2(Vec<T>::pair(xq, i), pack2(kDown, kDown));
      sxx = fma2(x, x, sxx);
      sgx = fma2(mul2(Vec<T>::pair(gq, i), Vec<T>::pair(wq[j], i)), x, sgx);
    }
  }
  b[0] += sum2(sxx);
  b[1] += sum2(sgx);
}
template <typename T, int VPT> __device__ __forceinline__ void scale_slots(uint4* slots, int stride, float by) {
#pragma unroll 1
  for (int j = 0; j < VPT; ++j) {
    const uint4 q = slots[j * stride];
    f32x2 x[Vec<T>::P];
#pragma unroll
    for (int i = 0; i < Vec<T>::P; ++i) x[i] = mul2(Vec<T>::pair(q, i), pack2(by, by));
    slots[j * stride] = Vec<T>::put(x);
  }
}

template <typename T, int VPT, bool LAYER, bool RES>
__global__ void __launch_bounds__(max_threads(VPT), min_blocks(VPT))
    norm_backward_rows_kernel(const T* x_, const T* __restrict__ w_, const T* dout_, const T* dres_, T* dx_,
                              float* __restrict__ part_w, float* __restrict__ part_b, int64_t rows, int H,
                              float eps, int tpr) {
  constexpr int P = Vec<T>::P, ARR = RES ? 3 : 2, STAGES = stages_of(LAYER, ARR);
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float s_red[2][4 * kMaxWarps];
  pdl_wait();
  pdl_trigger();
  const Team<T, VPT, ARR, STAGES> tm(H, tpr, rows, s_dyn);
  const uint4* const src[3] = {reinterpret_cast<const uint4*>(x_), reinterpret_cast<const uint4*>(dout_),
                               reinterpret_cast<const uint4*>(dres_)};
  uint4* dx = reinterpret_cast<uint4*>(dx_);
  const float inv_h = 1.0f / static_cast<float>(H);
  int64_t base = static_cast<int64_t>(blockIdx.x) * tm.rpb;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) tm.fetch(src, base + s * tm.step + tm.team, s);
  uint4 wq[VPT];
  f32x2 aw[VPT][P], ab[VPT][P];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    wq[j] = tm.has(j) ? reinterpret_cast<const uint4*>(w_)[tm.me + j * tpr] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < P; ++i) aw[j][i] = ab[j][i] = 0;
  }
  int stage = 0, buf = 0;
  float mean = 0.0f;                      // of the current row
  if (LAYER) {
    // of the first row; every later one comes with the sums of the row before
    copy_wait<STAGES - 2>();
    float s1[1] = {tm.row_sum(0)};
    team_sum<1>(s1, tpr, s_red, buf);
    mean = s1[0] * inv_h;
  }
  for (; base < rows; base += tm.step) {
    const int64_t t = base + tm.team;
    const int after = stage == STAGES - 1 ? 0 : stage + 1;
    tm.fetch(src, t + (STAGES - 1) * tm.step, stage == 0 ? STAGES - 1 : stage - 1);
    copy_wait<LAYER ? STAGES - 2 : STAGES - 1>();
    const uint4* ring = tm.slot(stage);
    // each pass reads the row from shared memory again: registers for 16 more
    // fp32 values would cost the second block of the SM
    auto read = [&](int a, int j) { return ring[(a * VPT + j) * static_cast<int>(blockDim.x)]; };
    const f32x2 neg_mean = pack2(-mean, -mean);
    f32x2 sxx = 0, sgx = 0, sg = 0;       // x'^2, gy x', gy   (x' = x - mean)
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (!LAYER || tm.has(j)) {
        const uint4 xq = read(0, j), gq = read(1, j);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          f32x2 xc = Vec<T>::pair(xq, i);
          if (LAYER) xc = add2(xc, neg_mean);
          const f32x2 gy = mul2(Vec<T>::pair(gq, i), Vec<T>::pair(wq[j], i));
          sxx = fma2(xc, xc, sxx);
          sgx = fma2(gy, xc, sgx);
          if (LAYER) sg = add2(sg, gy);
        }
      }
    float s[LAYER ? 4 : 2];
    s[0] = sum2(sxx);
    s[1] = sum2(sgx);
    if (LAYER) {
      s[LAYER ? 2 : 0] = sum2(sg);
      s[LAYER ? 3 : 0] = tm.row_sum(after);
    }
    team_sum<LAYER ? 4 : 2>(s, tpr, s_red, buf);
    // dx = r gy - r mean(gy) + k x',  k = -r^3 mean(gy x')
    float r = rsqrtf(s[0] * inv_h + eps), rx = r;
    float k = -r * (r * (r * (s[1] * inv_h)));
    if (!LAYER && !(s[0] <= FLT_MAX)) {     // uniform over the team
      // RMSNorm, squares past the fp32 range: summed again at 2^-70.  The thread's
      // own slots of the row are then scaled to values around 1 (by a power of two,
      // so exactly), x^ = rx x', and k keeps its digits.
      uint4* x_slots = tm.mine + stage * tm.stage_vecs;
      float b[2] = {0.0f, 0.0f};
      scaled_sums<T, VPT>(x_slots, wq, static_cast<int>(blockDim.x), b);
      team_sum<2, true>(b, tpr, s_red, buf);
      if (b[0] <= FLT_MAX) {                // else an infinity or NaN in the row
        const float rs = rsqrtf(b[0] * inv_h + eps * kDown * kDown);
        const float p = __uint_as_float(__float_as_uint(rs) & 0x7F800000u);
        r = rs * kDown;
        rx = rs / p;
        k = -r * (rx * (rs * (b[1] * inv_h)));
        scale_slots<T, VPT>(x_slots, static_cast<int>(blockDim.x), kDown * p);
      }
    }
    const float m1 = LAYER ? -r * (s[LAYER ? 2 : 0] * inv_h) : 0.0f;
    const f32x2 r2 = pack2(r, r), rx2 = LAYER ? r2 : pack2(rx, rx), k2 = pack2(k, k), m12 = pack2(m1, m1);
    if (t < rows)
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (tm.has(j)) {
          const uint4 xq = read(0, j), gq = read(1, j);
          uint4 dq = make_uint4(0, 0, 0, 0);
          if (RES) dq = read(ARR - 1, j);
          f32x2 d[P];
#pragma unroll
          for (int i = 0; i < P; ++i) {
            f32x2 xc = Vec<T>::pair(xq, i);
            if (LAYER) xc = add2(xc, neg_mean);
            const f32x2 g = Vec<T>::pair(gq, i);
            aw[j][i] = fma2(g, mul2(xc, rx2), aw[j][i]);
            if (LAYER) ab[j][i] = add2(ab[j][i], g);
            f32x2 v = LAYER ? fma2(xc, k2, m12) : mul2(xc, k2);
            v = fma2(mul2(g, Vec<T>::pair(wq[j], i)), r2, v);
            d[i] = RES ? add2(v, Vec<T>::pair(dq, i)) : v;
          }
          dx[t * tm.nv + tm.me + j * tpr] = Vec<T>::put(d);
        }
    if (LAYER) mean = s[LAYER ? 3 : 0] * inv_h;
    stage = after;
  }
  copy_wait<0>();
  // the teams' sums, in order, through shared memory (the ring is done)
  float* s_sum = reinterpret_cast<float*>(s_dyn);
#pragma unroll
  for (int pass = 0; pass < (LAYER ? 2 : 1); ++pass) {
    float* part = pass == 0 ? part_w : part_b;
    if (part == nullptr) continue;        // uniform
    part += static_cast<int64_t>(blockIdx.x) * H;
    for (int turn = 0; turn < tm.rpb; ++turn) {
      __syncthreads();
      if (tm.team == turn)
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          if (tm.has(j))
#pragma unroll
            for (int i = 0; i < P; ++i) {
              const int c = (tm.me + j * tpr) * Vec<T>::V + 2 * i;
              float2 v = unpack2(pass == 0 ? aw[j][i] : ab[j][i]);
              if (turn > 0) {
                v.x = s_sum[c] + v.x;
                v.y = s_sum[c + 1] + v.y;
              }
              *reinterpret_cast<float2*>((turn + 1 < tm.rpb ? s_sum : part) + c) = v;
            }
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

// out[c] = sum over blocks of part[block][c]: 64 columns a block of threads (so
// that both gradients of a wide row fit one wave), warp w adds the partial
// rows w, w + 32, ... in order, then the warps' sums are added in a fixed tree.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_partials_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, int blocks,
                         int H, float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float s_sum[kSumWarps][66];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 64 + 2 * lane;
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float2 s = make_float2(0.0f, 0.0f);
  if (H % 2 == 0) {
    if (c < H) {
#pragma unroll 4
      for (int b = warp; b < blocks; b += kSumWarps) {
        const float2 v = *reinterpret_cast<const float2*>(part + static_cast<int64_t>(b) * H + c);
        s.x += v.x;
        s.y += v.y;
      }
    }
  } else {
    for (int b = warp; b < blocks; b += kSumWarps) {
      if (c < H) s.x += part[static_cast<int64_t>(b) * H + c];
      if (c + 1 < H) s.y += part[static_cast<int64_t>(b) * H + c + 1];
    }
  }
  s_sum[warp][2 * lane] = s.x;
  s_sum[warp][2 * lane + 1] = s.y;
  __syncthreads();
  // warp w: columns w and w + 32, over the warps' sums
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int col = warp + 32 * half;
    float t = s_sum[lane][col];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int cw = blockIdx.x * 64 + col;
    if (lane == 0 && cw < H) (blockIdx.y == 0 ? dweight : dbias)[cw] = t;
  }
}

// Threads of a team and the vectors each holds; 0 vectors: the row has no
// whole 16-byte vectors or is too long for a team.
struct TeamShape {
  int vpt, tpr, threads;
  int rows_a_block() const { return threads / tpr; }
};
// 16 elements a thread, which halve what a thread spends on a row whatever its
// length (copies, reductions, loop) against 8; layer norm's backward pass keeps
// two sums a column and takes 8 bf16 elements, where 16 spilled registers
// (8192 x 6144: 88 us against 110).
template <typename T> TeamShape team_shape(int H, bool two_sums) {
  constexpr int V = Vec<T>::V;
  TeamShape s{0, 0, 0};
  if (H % V != 0 || H / V > 4 * kMaxTeam) return s;
  const int nv = H / V;
  s.vpt = nv <= 32 || (two_sums && V == 8 && nv <= 768) ? 1 : V == 8 && nv <= 2 * 384 ? 2 : V == 4 && nv <= 64 ? 2 : 4;
  s.tpr = static_cast<int>(ceil_div(ceil_div(nv, s.vpt), 32) * 32);
  const int full = s.vpt == 4 ? 256 : 384;
  s.threads = s.tpr >= full ? s.tpr : full / s.tpr * s.tpr;
  return s;
}
// shared memory of a block, and the blocks an SM holds
size_t ring_bytes(const TeamShape& s, bool layer, int arrays) {
  return static_cast<size_t>(stages_of(layer, arrays)) * arrays * s.vpt * s.threads * 16;
}
int resident_blocks(int threads_by_regs, const TeamShape& s, size_t smem) {
  return std::max(1, std::min(static_cast<int>(kMaxRing / (smem + 2048)), threads_by_regs / s.threads));
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
  const size_t smem = ring_bytes(s, true, 1);
  const cudaError_t e = allow_smem<layer_norm_rows_kernel<T, VPT>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t groups = ceil_div(rows, s.rows_a_block());
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(groups, static_cast<int64_t>(num_sms) * resident_blocks(2 * kMaxTeam, s, smem)));
  return launch_chained(layer_norm_rows_kernel<T, VPT>, grid, s.threads, smem, stream, static_cast<const T*>(x),
                        static_cast<const T*>(w), static_cast<const T*>(b), static_cast<T*>(out), rows, H, eps,
                        s.tpr);
}

template <typename T, int VPT, bool LAYER, bool RES>
cudaError_t backward_rows(const TeamShape& s, const NormBackwardArgs& a, float* part_b, int blocks, size_t smem,
                          cudaStream_t stream) {
  const cudaError_t e = allow_smem<norm_backward_rows_kernel<T, VPT, LAYER, RES>>(smem);
  if (e != cudaSuccess) return e;
  return launch_chained(norm_backward_rows_kernel<T, VPT, LAYER, RES>, static_cast<unsigned>(blocks), s.threads,
                        smem, stream, static_cast<const T*>(a.x), static_cast<const T*>(a.weight),
                        static_cast<const T*>(a.dout), static_cast<const T*>(a.dres), static_cast<T*>(a.dx),
                        a.partials, part_b, a.T, a.H, a.eps, s.tpr);
}

template <typename T, int VPT>
cudaError_t backward_rows_of(const TeamShape& s, const NormBackwardArgs& a, float* part_b, int blocks, size_t smem,
                             cudaStream_t stream) {
  if (a.layer)
    return a.dres != nullptr ? backward_rows<T, VPT, true, true>(s, a, part_b, blocks, smem, stream)
                             : backward_rows<T, VPT, true, false>(s, a, part_b, blocks, smem, stream);
  return a.dres != nullptr ? backward_rows<T, VPT, false, true>(s, a, part_b, blocks, smem, stream)
                           : backward_rows<T, VPT, false, false>(s, a, part_b, blocks, smem, stream);
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
  const TeamShape s = team_shape<T>(H, false);
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
  const TeamShape s = team_shape<T>(a.H, a.layer);
  const size_t smem = s.vpt == 0 ? 0 : std::max(ring_bytes(s, a.layer, a.dres != nullptr ? 3 : 2),
                                                static_cast<size_t>(a.H) * sizeof(float));
  const bool team = s.vpt != 0 && smem <= kMaxRing;
  const int64_t groups = team ? ceil_div(a.T, s.rows_a_block()) : a.T;
  const int64_t resident = static_cast<int64_t>(num_sms) * (team ? resident_blocks(max_threads(s.vpt) * min_blocks(s.vpt), s, smem) : 4);
  *blocks = static_cast<int>(std::min<int64_t>(groups, std::min<int64_t>(resident, kNormMaxBlocks)));
  if (*blocks == 0) return cudaSuccess;
  if (team && s.vpt == 1) return backward_rows_of<T, 1>(s, a, part_b, *blocks, smem, stream);
  if (team && s.vpt == 2) return backward_rows_of<T, 2>(s, a, part_b, *blocks, smem, stream);
  if (team && s.vpt == 4) return backward_rows_of<T, 4>(s, a, part_b, *blocks, smem, stream);
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
  const dim3 grid(static_cast<unsigned>(ceil_div(a.H, 64)), a.dbias != nullptr ? 2 : 1);
  return launch_chained(norm_partials_kernel, grid, dim3(32 * kSumWarps), 0, stream,
                        static_cast<const float*>(a.partials), static_cast<const float*>(part_b), blocks,
                        a.H, a.dweight, a.dbias);
}

}  // namespace moe
