// Entry points of shared-prefix attention (declared in include/te_attn.h): argument
// checks, workspace layout and launch sequence.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/te_attn.h"
#include "api_internal.h"
#include "attn_prefix.cuh"
#include "launch.h"

namespace teattn {
namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_prefix(const void* const* tensors, int n_tensors, const int32_t* prefix_len, int batch,
                 int total_q, int total_kv, int prefix_rows, int hq, int hkv, int d, float attn_scale,
                 int mask_type, int dtype, const int32_t* cu_q, const int32_t* cu_kv,
                 const int32_t* cu_q_pad, const int32_t* cu_kv_pad) {
  const int rc = api_check_common(batch, total_q, total_kv, hq, hkv, d, attn_scale, mask_type, dtype,
                                  cu_q, cu_kv, cu_q_pad, cu_kv_pad);
  if (rc != TE_OK) return rc;
  if (prefix_rows < 0) return api_fail(TE_ERR_INVALID_ARG, "prefix_rows must be >= 0");
  if (static_cast<long long>(prefix_rows) * hkv * d >= (1ll << 40) ||
      static_cast<long long>(total_q) * hq > INT32_MAX)
    return api_fail(TE_ERR_UNSUPPORTED, "tensor too large");
  for (int i = 0; i < n_tensors; ++i)
    if (!aligned(tensors[i], 16)) return api_fail(TE_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  const void* words[] = {prefix_len, cu_q, cu_kv, cu_q_pad, cu_kv_pad};
  for (const void* w : words)
    if (!aligned(w, 4)) return api_fail(TE_ERR_INVALID_ARG, "int32 arrays need their natural alignment");
  return TE_OK;
}

PrefixParams base_params(const void* q, const void* k, const void* v, const void* kp, const void* vp,
                         const int32_t* cu_q, const int32_t* cu_kv, const int32_t* cu_q_pad,
                         const int32_t* cu_kv_pad, const int32_t* prefix_len, int batch, int total_q,
                         int total_kv, int prefix_rows, int hq, int hkv, int d, float scale,
                         int mask_type) {
  PrefixParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.kp = kp;
  p.vp = vp;
  p.cu_q = cu_q;
  p.cu_kv = cu_kv;
  p.cu_q_pad = cu_q_pad;
  p.cu_kv_pad = cu_kv_pad;
  p.prefix_len = prefix_len;
  p.prefix_rows = prefix_rows;
  p.batch = batch;
  p.total_q = total_q;
  p.total_kv = total_kv;
  p.hq = hq;
  p.hkv = hkv;
  p.d = d;
  p.group = hq / hkv;
  p.rs = 1;
  p.causal = mask_type == TE_MASK_PADDING_CAUSAL ? 1 : mask_type == TE_MASK_PADDING_CAUSAL_BOTTOM_RIGHT ? 2 : 0;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  return p;
}

}  // namespace
}  // namespace teattn

using namespace teattn;

extern "C" {

size_t te_attn_prefix_fwd_workspace_size(int batch, int total_q, int total_kv, int prefix_rows,
                                         int hq, int hkv, int d) {
  if (batch < 1 || total_q < 0 || total_kv < 0 || prefix_rows < 0 || hq < 1 || hkv < 1 || hq % hkv != 0 ||
      d < 8 || d > 256)
    return 0;
  return kHdrWords * sizeof(int);
}

size_t te_attn_prefix_bwd_workspace_size(int batch, int total_q, int total_kv, int prefix_rows,
                                         int hq, int hkv, int d) {
  return te_attn_prefix_fwd_workspace_size(batch, total_q, total_kv, prefix_rows, hq, hkv, d);
}

int te_attn_prefix_fwd_thd(const void* q, const void* k, const void* v, const void* k_prefix,
                           const void* v_prefix, void* out, float* lse, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_kv, const int32_t* cu_seqlens_q_padded,
                           const int32_t* cu_seqlens_kv_padded, const int32_t* prefix_len, int batch,
                           int total_q, int total_kv, int prefix_rows, int hq, int hkv, int d,
                           float attn_scale, int mask_type, int dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const void* tensors[] = {q, k, v, k_prefix, v_prefix, out, workspace};
  const int rc = check_prefix(tensors, 7, prefix_len, batch, total_q, total_kv, prefix_rows, hq, hkv, d,
                              attn_scale, mask_type, dtype, cu_seqlens_q, cu_seqlens_kv,
                              cu_seqlens_q_padded, cu_seqlens_kv_padded);
  if (rc != TE_OK) return rc;
  if (!workspace) return api_fail(TE_ERR_INVALID_ARG, "workspace must not be NULL");
  if (total_q > 0 && (!q || !out || !lse))
    return api_fail(TE_ERR_INVALID_ARG, "q, out and lse must not be NULL");
  if (total_kv > 0 && (!k || !v)) return api_fail(TE_ERR_INVALID_ARG, "k and v must not be NULL");
  if (prefix_rows > 0 && (!k_prefix || !v_prefix))
    return api_fail(TE_ERR_INVALID_ARG, "k_prefix and v_prefix must not be NULL");
  if (workspace_bytes < te_attn_prefix_fwd_workspace_size(batch, total_q, total_kv, prefix_rows, hq, hkv, d))
    return api_fail(TE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than te_attn_prefix_fwd_workspace_size()");
  const int sms = api_num_sms();
  if (sms <= 0) return api_fail(TE_ERR_CUDA, "no CUDA device");
  PrefixParams p = base_params(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_kv,
                               cu_seqlens_q_padded, cu_seqlens_kv_padded, prefix_len, batch, total_q,
                               total_kv, prefix_rows, hq, hkv, d, attn_scale, mask_type);
  p.out = out;
  p.lse = lse;
  p.header = static_cast<int*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      api_timed(TE_KERNEL_FWD, st, [&] { return launch_prefix_fwd(p, dtype == TE_DTYPE_BF16, sms, st); });
  return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "shared-prefix forward");
}

int te_attn_prefix_bwd_thd(const void* q, const void* k, const void* v, const void* k_prefix,
                           const void* v_prefix, const void* out, const void* dout, const float* lse,
                           void* dq, void* dk, void* dv, void* dk_prefix, void* dv_prefix,
                           const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv,
                           const int32_t* cu_seqlens_q_padded, const int32_t* cu_seqlens_kv_padded,
                           const int32_t* prefix_len, int batch, int total_q, int total_kv,
                           int prefix_rows, int hq, int hkv, int d, float attn_scale, int mask_type,
                           int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const void* tensors[] = {q, k, v, k_prefix, v_prefix, out, dout, dq, dk, dv, dk_prefix, dv_prefix, workspace};
  const int rc = check_prefix(tensors, 13, prefix_len, batch, total_q, total_kv, prefix_rows, hq, hkv, d,
                              attn_scale, mask_type, dtype, cu_seqlens_q, cu_seqlens_kv,
                              cu_seqlens_q_padded, cu_seqlens_kv_padded);
  if (rc != TE_OK) return rc;
  if (!workspace) return api_fail(TE_ERR_INVALID_ARG, "workspace must not be NULL");
  if (total_q > 0 && (!q || !out || !dout || !lse || !dq))
    return api_fail(TE_ERR_INVALID_ARG, "q, out, dout, lse and dq must not be NULL");
  if (total_kv > 0 && (!k || !v || !dk || !dv))
    return api_fail(TE_ERR_INVALID_ARG, "k, v, dk and dv must not be NULL");
  if (prefix_rows > 0 && (!k_prefix || !v_prefix || !dk_prefix || !dv_prefix))
    return api_fail(TE_ERR_INVALID_ARG, "k_prefix, v_prefix, dk_prefix and dv_prefix must not be NULL");
  if (workspace_bytes < te_attn_prefix_bwd_workspace_size(batch, total_q, total_kv, prefix_rows, hq, hkv, d))
    return api_fail(TE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than te_attn_prefix_bwd_workspace_size()");
  const int sms = api_num_sms();
  if (sms <= 0) return api_fail(TE_ERR_CUDA, "no CUDA device");
  PrefixParams p = base_params(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_kv,
                               cu_seqlens_q_padded, cu_seqlens_kv_padded, prefix_len, batch, total_q,
                               total_kv, prefix_rows, hq, hkv, d, attn_scale, mask_type);
  p.out_in = out;
  p.dout = dout;
  p.lse_in = lse;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.dkp = dk_prefix;
  p.dvp = dv_prefix;
  p.header = static_cast<int*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      api_timed(TE_KERNEL_DKDV, st, [&] { return launch_prefix_bwd(p, dtype == TE_DTYPE_BF16, sms, st); });
  return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "shared-prefix backward");
}

}  // extern "C"
