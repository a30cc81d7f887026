// Entry points of attention over a paged cache (declared in include/te_attn.h): argument
// checks, workspace layout and launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/te_attn.h"
#include "api_internal.h"
#include "attn_paged.cuh"

namespace teattn {
namespace {

// Workspace, 256-byte aligned sections: header, a status word a slice, and for each of the two
// kernels prefix sums of the sequences' work and partial rows (maximum and sum; d fp32 columns),
// two slots of a row tile for every slice.
struct PagedLayout {
  size_t warp_status, pref[2], ml[2], o[2], total;
  int rows, slices[2], wide_rows;
};

bool paged_layout(int batch, int total_q, int hq, int hkv, int d, bool four, PagedLayout* L) {
  if (batch < 1 || batch > kPagedMaxBatch || total_q < 0 || hq < 1 || hkv < 1 || hq % hkv != 0 || d < 8 || d > 256 || d % 8 != 0 ||
      static_cast<long long>(total_q) * hq > INT32_MAX - 256)
    return false;
  L->rows = paged_rows(batch, total_q, hq / hkv, d, four);
  L->wide_rows = paged_wide_rows(batch, total_q, hq, hkv, d, four);
  L->slices[0] = paged_warps(d, four, L->rows);
  L->slices[1] = L->wide_rows > 0 ? kPagedSMs : 0;
  size_t off = kHdrWords * sizeof(int);
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  L->warp_status = take((L->slices[0] + L->slices[1]) * sizeof(int));
  for (int k = 0; k < 2; ++k) {
    const size_t rows = 2 * static_cast<size_t>(L->slices[k]) * (k ? kWideRows : L->rows);
    L->pref[k] = take((static_cast<size_t>(batch) + 1) * sizeof(long long));
    L->ml[k] = take(rows * sizeof(float2));
    L->o[k] = take(rows * d * sizeof(float));
  }
  L->total = off;
  return true;
}

}  // namespace
}  // namespace teattn

using namespace teattn;

extern "C" {

size_t te_attn_paged_fwd_workspace_size(int batch, int total_q, int hq, int hkv, int d, int bits) {
  PagedLayout L;
  if (bits != 4 && bits != 16) return 0;
  return paged_layout(batch, total_q, hq, hkv, d, bits == 4, &L) ? L.total : 0;
}

int te_attn_paged_fwd_thd(const te_attn_paged_cache* cache, const void* q, void* out, float* lse,
                          const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_q_padded, const int32_t* past,
                          int batch, int total_q, int hq, float attn_scale, int window, int sinks, void* workspace,
                          size_t workspace_bytes, void* stream) {
  PagedParams p{};
  int rc = api_paged_cache(cache, &p.cache);
  if (rc != TE_OK) return rc;
  rc = api_check_common(batch, total_q, 0, hq, cache->hkv, cache->d, attn_scale, TE_MASK_PADDING_CAUSAL_BOTTOM_RIGHT,
                        cache->dtype, cu_seqlens_q, past, cu_seqlens_q_padded, past);
  if (rc != TE_OK) return rc;
  if (window < 0) return api_fail(TE_ERR_INVALID_ARG, "window must be >= 0");
  if (sinks < 0 || (sinks > 0 && window == 0)) return api_fail(TE_ERR_INVALID_ARG, "sinks must be >= 0 and go with a window");
  auto aligned = [](const void* x, unsigned n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0; };
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16))
    return api_fail(TE_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  for (const void* x : {static_cast<const void*>(cu_seqlens_q), static_cast<const void*>(cu_seqlens_q_padded),
                        static_cast<const void*>(past), static_cast<const void*>(lse)})
    if (!aligned(x, 4)) return api_fail(TE_ERR_INVALID_ARG, "int32 arrays and lse need their natural alignment");
  if (batch > kPagedMaxBatch) return api_fail(TE_ERR_UNSUPPORTED, "at most 4096 sequences");
  if (!workspace) return api_fail(TE_ERR_INVALID_ARG, "workspace must not be NULL");
  if (total_q > 0 && (!q || !out || !lse)) return api_fail(TE_ERR_INVALID_ARG, "q, out and lse must not be NULL");
  PagedLayout L;
  const bool four = cache->k_meta != nullptr;
  if (!paged_layout(batch, total_q, hq, cache->hkv, cache->d, four, &L)) return api_fail(TE_ERR_UNSUPPORTED, "tensor too large");
  if (workspace_bytes < L.total)
    return api_fail(TE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than te_attn_paged_fwd_workspace_size()");
  const int sms = api_num_sms();
  if (sms <= 0) return api_fail(TE_ERR_CUDA, "no CUDA device");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  p.header = static_cast<int*>(workspace);
  if (total_q == 0) {
    const cudaError_t e = cudaMemsetAsync(p.header, 0, kHdrWords * sizeof(int), st);
    return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "paged attention");
  }
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.cu_q = cu_seqlens_q;
  p.cu_q_pad = cu_seqlens_q_padded;
  p.past = past;
  p.batch = batch;
  p.total_q = total_q;
  p.hq = hq;
  p.hkv = cache->hkv;
  p.d = cache->d;
  p.group = hq / cache->hkv;
  // (a window, or sinks, of 2^30 leave every key)
  p.window = window < (1 << 30) ? window : 1 << 30;
  p.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
  p.scale_log2 = attn_scale * 1.4426950408889634f;
  p.warp_status = reinterpret_cast<int*>(ws + L.warp_status);
  p.wide_rows = L.wide_rows;
  // one slice for each warp, or block, of as many SMs as there are
  const int use = sms < kPagedSMs ? sms : kPagedSMs;
  PagedParts parts[2];
  for (int k = 0; k < 2; ++k)
    parts[k] = PagedParts{reinterpret_cast<long long*>(ws + L.pref[k]), reinterpret_cast<float2*>(ws + L.ml[k]),
                          reinterpret_cast<float*>(ws + L.o[k]), L.slices[k] / kPagedSMs * use, kLeastWideUnits};
  const bool bf16 = cache->dtype == TE_DTYPE_BF16;
  PagedCut cut{};
  cudaError_t e = api_timed(TE_KERNEL_FWD, st, [&] { return launch_paged_rows(p, parts[0], bf16, four, L.rows, &cut, st); });
  if (e != cudaSuccess) return api_cuda_fail(e, "paged attention");
  parts[0].least = kLeastKeys / cut.unit;
  if (L.wide_rows > 0) {
    e = api_timed(TE_KERNEL_FWD, st, [&] { return launch_paged_tiles(p, parts[1], parts[0].slices, bf16, four, st); });
    if (e != cudaSuccess) return api_cuda_fail(e, "paged attention of long pieces");
  }
  e = api_timed(TE_KERNEL_FWD, st, [&] { return launch_paged_join(p, cut, parts[0], parts[1], bf16, st); });
  return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "paged join");
}

}  // extern "C"
