// The C ABI of the training operators (declared in include/inkling_moe.h):
// argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "inkling_moe.h"
#include "internal.h"

namespace moe {
namespace {

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// a workspace that holds at least the status region (and `bytes`)
moe_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return MOE_ERR_INVALID_ARG;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status_t check_grouped(const moe_grouped_desc_t* d) {
  if (d == nullptr) return MOE_ERR_INVALID_ARG;
  if (d->rows < 0 || d->n_groups <= 0 || d->n <= 0 || d->k <= 0) return MOE_ERR_INVALID_ARG;
  if (d->dtype != MOE_ELEM_F32 && d->dtype != MOE_ELEM_BF16 && d->dtype != MOE_ELEM_F16)
    return MOE_ERR_INVALID_ARG;
  if (d->out_dtype != d->dtype && d->out_dtype != MOE_ELEM_F32) return MOE_ERR_INVALID_ARG;
  // past 2^24 features the kernels' tile counts (the fewest rows and columns a
  // tile has: 1 x 16) would leave 32 bits
  if (d->rows >= (int64_t{1} << 31) || d->n_groups > 1024 || d->n > (1 << 24) || d->k > (1 << 24))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

GroupedProduct grouped_sizes(const moe_grouped_desc_t* d) {
  GroupedProduct g{};
  g.rows = d->rows;
  g.E = d->n_groups;
  g.n = d->n;
  g.k = d->k;
  g.dtype = d->dtype;
  g.out_dtype = d->out_dtype;
  return g;
}

moe_status_t run_grouped(const moe_grouped_desc_t* d, int form, const void* p, const void* q,
                         const int32_t* offsets, void* out, int accumulate, void* ws,
                         size_t ws_bytes, void* stream) {
  moe_status_t st = check_grouped(d);
  if (st != MOE_OK) return st;
  if (accumulate && d->out_dtype != MOE_ELEM_F32) return MOE_ERR_INVALID_ARG;
  if (form != kWgrad && d->rows == 0) return MOE_OK;
  // row operands may be absent when there are no rows
  if (d->rows > 0 && !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if ((form != kWgrad || d->rows > 0) && !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!aligned4(offsets) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  GroupedProduct g = grouped_sizes(d);
  g.form = form;
  st = check_workspace(ws, ws_bytes, kStatusBytes);
  if (st != MOE_OK) return st;
  // a workspace of another product, or of the layer, may be too small for the pieces: uncut then
  if (ws_bytes - kStatusBytes >= grouped_matmul_sm100_parts_bytes(g, form))
    g.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes);
  g.p = p;
  g.q = q;
  g.offsets = offsets;
  g.out = out;
  g.accumulate = accumulate ? 1 : 0;
  g.status = static_cast<int32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!grouped_matmul_sm100_takes(g)) return cuda_status(launch_grouped_matmul_simt(g, device_sm_count(), s));
  bool map_error = false;
  const cudaError_t e = launch_grouped_matmul_sm100(g, device_sm_count(), s, &map_error);
  return map_error ? MOE_ERR_INVALID_ARG : cuda_status(e);
}

moe_status_t check_swiglu(int64_t rows, int32_t I, moe_dtype_t dtype, int32_t n_groups,
                          const int32_t* offsets, const int32_t* perm_slot, const float* topk_w) {
  if (rows < 0 || I <= 0 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (offsets != nullptr && (n_groups <= 0 || !aligned4(offsets))) return MOE_ERR_INVALID_ARG;
  if (perm_slot != nullptr && (topk_w == nullptr || !aligned4(perm_slot))) return MOE_ERR_INVALID_ARG;
  if (topk_w != nullptr && !aligned4(topk_w)) return MOE_ERR_INVALID_ARG;
  if (I % 16 != 0 || I > (1 << 24) || rows >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

SwigluArgs swiglu_args(int64_t rows, int32_t I, moe_dtype_t dtype, int32_t n_groups,
                       const int32_t* offsets, const int32_t* perm_slot, const float* topk_w,
                       void* ws) {
  SwigluArgs a{};
  a.rows = rows;
  a.I = I;
  a.dtype = dtype;
  a.live = offsets != nullptr ? offsets + n_groups : nullptr;
  a.perm_slot = perm_slot;
  a.topk_w = topk_w;
  a.status = static_cast<int32_t*>(ws);
  return a;
}

moe_status_t check_norm(int64_t T, int32_t H, moe_dtype_t dtype, float eps) {
  if (T < 0 || H <= 0 || (dtype != MOE_F32 && dtype != MOE_BF16) || !isfinite(eps) || eps < 0.0f)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

size_t norm_workspace(int32_t H) {
  return 2 * static_cast<size_t>(kNormMaxBlocks) * static_cast<size_t>(H) * sizeof(float);
}

moe_status_t run_norm_backward(bool layer, int64_t T, int32_t H, moe_dtype_t dtype, float eps,
                               const void* x, const void* weight, const void* dout,
                               const void* dres, void* dx, float* dweight, float* dbias, void* ws,
                               size_t ws_bytes, void* stream) {
  moe_status_t st = check_norm(T, H, dtype, eps);
  if (st != MOE_OK) return st;
  if (T > 0 && (!aligned16(x) || !aligned16(weight) || !aligned16(dout) || !aligned16(dx)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dweight) || (dbias != nullptr && !aligned16(dbias)) ||
      (dres != nullptr && !aligned16(dres)))
    return MOE_ERR_INVALID_ARG;
  st = check_workspace(ws, ws_bytes, norm_workspace(H));
  if (st != MOE_OK) return st;
  NormBackwardArgs a{};
  a.T = T;
  a.H = H;
  a.dtype = dtype;
  a.layer = layer;
  a.eps = eps;
  a.x = x;
  a.weight = weight;
  a.dout = dout;
  a.dres = dres;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partials = static_cast<float*>(ws);
  return cuda_status(launch_norm_backward(a, device_sm_count(), static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_grouped_workspace_size(const moe_grouped_desc_t* desc, size_t* bytes) {
  const moe_status_t st = check_grouped(desc);
  if (st != MOE_OK) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const GroupedProduct g = grouped_sizes(desc);
  size_t parts = 0;
  for (const int form : {kForward, kDgrad, kWgrad})
    parts = std::max(parts, grouped_matmul_sm100_parts_bytes(g, form));
  *bytes = kStatusBytes + parts;
  return MOE_OK;
}

moe_status_t moe_grouped_matmul(const moe_grouped_desc_t* desc, const void* a, const void* w,
                                const int32_t* expert_offsets, void* out, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return run_grouped(desc, kForward, a, w, expert_offsets, out, 0, workspace, workspace_bytes, stream);
}

moe_status_t moe_grouped_matmul_dgrad(const moe_grouped_desc_t* desc, const void* dout,
                                      const void* w, const int32_t* expert_offsets, void* da,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  return run_grouped(desc, kDgrad, dout, w, expert_offsets, da, 0, workspace, workspace_bytes, stream);
}

moe_status_t moe_grouped_matmul_wgrad(const moe_grouped_desc_t* desc, const void* dout,
                                      const void* a, const int32_t* expert_offsets, void* dw,
                                      int32_t accumulate, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  return run_grouped(desc, kWgrad, dout, a, expert_offsets, dw, accumulate, workspace,
                     workspace_bytes, stream);
}

moe_status_t moe_swiglu_checkpoint(int64_t rows, int32_t intermediate, moe_dtype_t dtype,
                                   const void* gu, int32_t n_groups, const int32_t* expert_offsets,
                                   const int32_t* perm_slot, const float* topk_w, void* h, void* q,
                                   uint8_t* scale, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  moe_status_t st = check_swiglu(rows, intermediate, dtype, n_groups, expert_offsets, perm_slot, topk_w);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!aligned16(gu) || !aligned16(h) || !aligned16(q) || !aligned16(scale)) return MOE_ERR_INVALID_ARG;
  st = check_workspace(workspace, workspace_bytes, kStatusBytes);
  if (st != MOE_OK) return st;
  const SwigluArgs a = swiglu_args(rows, intermediate, dtype, n_groups, expert_offsets, perm_slot,
                                   topk_w, workspace);
  return cuda_status(launch_swiglu_checkpoint(a, gu, h, q, scale, device_sm_count(),
                                              static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_swiglu_backward(int64_t rows, int32_t intermediate, moe_dtype_t dtype,
                                 const void* q, const uint8_t* scale, const void* dh,
                                 int32_t n_groups, const int32_t* expert_offsets,
                                 const int32_t* perm_slot, const float* topk_w, void* dgu,
                                 float* d_topk_w, void* h, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  moe_status_t st = check_swiglu(rows, intermediate, dtype, n_groups, expert_offsets, perm_slot, topk_w);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!aligned16(q) || !aligned16(scale) || !aligned16(dh) || !aligned16(dgu) ||
      (h != nullptr && !aligned16(h)) || (d_topk_w != nullptr && !aligned4(d_topk_w)))
    return MOE_ERR_INVALID_ARG;
  st = check_workspace(workspace, workspace_bytes, kStatusBytes);
  if (st != MOE_OK) return st;
  const SwigluArgs a = swiglu_args(rows, intermediate, dtype, n_groups, expert_offsets, perm_slot,
                                   topk_w, workspace);
  return cuda_status(launch_swiglu_backward(a, q, scale, dh, dgu, d_topk_w, h, device_sm_count(),
                                            static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_layer_norm(int64_t num_tokens, int32_t hidden, moe_dtype_t dtype, float eps,
                            const void* x, const void* weight, const void* bias, void* out,
                            void* stream) {
  const moe_status_t st = check_norm(num_tokens, hidden, dtype, eps);
  if (st != MOE_OK) return st;
  if (num_tokens == 0) return MOE_OK;
  if (!aligned16(x) || !aligned16(weight) || !aligned16(out) || (bias != nullptr && !aligned16(bias)))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_layer_norm(num_tokens, hidden, dtype, eps, x, weight, bias, out,
                                       device_sm_count(), static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_norm_workspace_size(int64_t num_tokens, int32_t hidden, size_t* bytes) {
  if (num_tokens < 0 || hidden <= 0 || bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = norm_workspace(hidden);
  return MOE_OK;
}

moe_status_t moe_layer_norm_backward(int64_t num_tokens, int32_t hidden, moe_dtype_t dtype,
                                     float eps, const void* x, const void* weight,
                                     const void* dout, const void* dres, void* dx, float* dweight,
                                     float* dbias, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  return run_norm_backward(true, num_tokens, hidden, dtype, eps, x, weight, dout, dres, dx, dweight,
                           dbias, workspace, workspace_bytes, stream);
}

moe_status_t moe_rmsnorm_backward(int64_t num_tokens, int32_t hidden, moe_dtype_t dtype, float eps,
                                  const void* x, const void* weight, const void* dout,
                                  const void* dres, void* dx, float* dweight, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return run_norm_backward(false, num_tokens, hidden, dtype, eps, x, weight, dout, dres, dx, dweight,
                           nullptr, workspace, workspace_bytes, stream);
}

}  // extern "C"
