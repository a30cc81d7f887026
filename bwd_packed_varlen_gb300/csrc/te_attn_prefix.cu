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

// Lengths are rounded up to whole tiles (of at most 256 rows) in 32 bits.
bool too_long(int total_q, int total_kv, int prefix_rows, int hq) {
  constexpr int kMost = INT32_MAX - 256;
  return static_cast<long long>(total_q) * hq > kMost || total_kv > kMost || prefix_rows > kMost;
}

int check_prefix(const void* const* tensors, int n_tensors, const int32_t* prefix_len, int batch,
                 int total_q, int total_kv, int prefix_rows, int hq, int hkv, int d, float attn_scale,
                 int mask_type, int dtype, const int32_t* cu_q, const int32_t* cu_kv,
                 const int32_t* cu_q_pad, const int32_t* cu_kv_pad) {
  const int rc = api_check_common(batch, total_q, total_kv, hq, hkv, d, attn_scale, mask_type, dtype,
                                  cu_q, cu_kv, cu_q_pad, cu_kv_pad);
  if (rc != TE_OK) return rc;
  if (prefix_rows < 0) return api_fail(TE_ERR_INVALID_ARG, "prefix_rows must be >= 0");
  if (static_cast<long long>(prefix_rows) * hkv * d >= (1ll << 40) || too_long(total_q, total_kv, prefix_rows, hq))
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

// Forward workspace, 256-byte aligned sections: header, per-sequence records, compact
// tokens, long row tiles, entries, partial rows (maximum and sum; d fp32 columns). The
// capacities follow from sum_b Lq_b <= total_q: with T chunks aimed at and row tiles of R rows,
//   long row tiles <= total_q G / R + batch,   entries <= T + 2 (total_q G / R + batch + 1)
//   partial rows of a kv head <= 2 R T + 2 min(total_q G, 128 batch):
// a row tile of n key tiles has at most n / len + 1 chunks, sum n / len <= T, a chunk leaves
// at most R partial rows, rows of short sequences (at most 128 each) are in a compact row
// tile and in one of their own, and a long row tile leaves partial rows only with two chunks
// or more, when n / len + 1 <= 2 n / len.
struct FwdLayout {
  size_t seqs, short_tok, longs, entries, part_ml, part_o, total;
  int parts_target;
  long long cap_longs, cap_entries, cap_rows;
};

bool fwd_layout(int batch, int total_q, int total_kv, int prefix_rows, int hq, int hkv, int d, FwdLayout* L) {
  if (batch < 1 || total_q < 0 || total_kv < 0 || prefix_rows < 0 || hq < 1 || hkv < 1 || hq % hkv != 0 ||
      d < 8 || d > 256 || d % 8 != 0 || too_long(total_q, total_kv, prefix_rows, hq))
    return false;
  const long long rows = static_cast<long long>(total_q) * (hq / hkv), rt = prefix_row_tile(d);
  L->parts_target = (kPartsTarget + hkv - 1) / hkv;
  L->cap_longs = rows / rt + batch;
  L->cap_entries = L->parts_target + 2 * (L->cap_longs + 1);
  const long long few = static_cast<long long>(kShortRows) * batch;
  L->cap_rows = hkv * (2 * rt * L->parts_target + 2 * (rows < few ? rows : few));
  if (L->cap_rows > INT32_MAX || L->cap_entries * hkv > INT32_MAX) return false;
  size_t off = kHdrWords * sizeof(int);
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  L->seqs = take(static_cast<size_t>(batch) * sizeof(int4));
  L->short_tok = take(static_cast<size_t>(total_q) * sizeof(int));
  L->longs = take(static_cast<size_t>(L->cap_longs) * sizeof(int4));
  L->entries = take(static_cast<size_t>(L->cap_entries) * 3 * sizeof(int4));
  L->part_ml = take(static_cast<size_t>(L->cap_rows) * sizeof(float2));
  L->part_o = take(static_cast<size_t>(L->cap_rows) * d * sizeof(float));
  L->total = off;
  return true;
}

// Backward workspace, 256-byte aligned sections: header, prefix sums of row tiles, lists of
// row and key tiles (of packed rows), lse and D of those tiles and of
// the whole tensor's rows, and with splits > 1 the parts of the prefix's gradients.
struct BwdLayout {
  size_t pref_q, q_pairs, k_pairs, lse_t, delta_t, lse_lin, delta_lin, part_dk, part_dv, total;
  int pack_shift, splits;
  long long cap_q, cap_k, rows_lin;
};

bool bwd_layout(int batch, int total_q, int total_kv, int prefix_rows, int hq, int hkv, int d, BwdLayout* L) {
  if (batch < 1 || total_q < 0 || total_kv < 0 || prefix_rows < 0 || hq < 1 || hkv < 1 || hq % hkv != 0 ||
      d < 8 || d > 256 || d % 8 != 0 || too_long(total_q, total_kv, prefix_rows, hq))
    return false;
  const int group = hq / hkv;
  int sh = 0;  // a 64-row tile holds whole tokens
  while (sh < 6 && group % (2 << sh) == 0) ++sh;
  L->pack_shift = sh;
  const long long rows = static_cast<long long>(total_q) << sh;
  L->cap_q = rows / kBlockM + batch + 1;
  L->cap_k = total_kv / kBlockN + static_cast<long long>(batch) + 1;
  L->rows_lin = (rows + kBlockM - 1) / kBlockM * kBlockM;
  const int halves = d > 128 ? 2 : 1;
  const long long steps = (group >> sh) * (L->rows_lin / (d > 128 ? 64 : 128));
  const long long items = (static_cast<long long>(prefix_rows) + kBlockN - 1) / kBlockN * hkv * halves;
  // Parts of a sweep: the number that ends the dK/dV launch soonest by this estimate. Its
  // units are about microseconds, but its coefficients are those of a fit, not measured times
  // of a step: a step (a row tile against a key tile) counts 0.8, 2 and 0.8 at head dims to 64,
  // 128 and 256 (where 64-row steps take longer than that), an item 8 more. The sequences'
  // own items, here all of mean length, come after the prefix's and fill what those leave
  // idle. The tail is 0.4 of the longest item, or of an own one if those are many and the
  // prefix's fill the SMs without being cut. Summing parts costs 3, and their bytes at 2.5 MB
  // a microsecond. The rates were fitted to 58 problems: the chosen number came within 1.7 %
  // of the best one's backward pass on average, with counting whole rounds of the prefix's
  // items alone within 6.6 % (16 sequences of 38 to 192 tokens, 8 heads of 80, prefix 615: 85
  // -> 67 us).
  const double step = d <= 64 ? 0.8 : d <= 128 ? 2.0 : 0.8;
  const long long row_tile = d > 128 ? 64 : 128;
  const long long seq_steps = (rows / batch + row_tile - 1) / row_tile, seq_tiles = (total_kv / batch + kBlockN - 1) / kBlockN;
  const double own = total_kv > 0 ? static_cast<double>(hkv) * halves * batch * (seq_tiles > 1 ? seq_tiles : 1) : 0;
  const double own_us = (group >> sh) * (seq_steps > 1 ? seq_steps : 1) * step + 8;
  const double part_mb = static_cast<double>(prefix_rows) * hkv * d * 2 * sizeof(float) / 1e6;
  double best = 0;
  L->splits = 1;
  for (long long n = 1; items > 0 && n <= 64 && n <= (steps > 3 ? steps / 2 : 1); ++n) {
    const double part_us = static_cast<double>((steps + n - 1) / n) * step + 8;
    const double own_share = own * own_us / kSMs;
    const double tail = items >= kSMs && own_share >= 0.5 * part_us ? own_us : part_us > own_us ? part_us : own_us;
    const double area = items * n * part_us / kSMs + own_share + 0.4 * tail;
    const double rounds = static_cast<double>((items * n + kSMs - 1) / kSMs) * part_us;
    double cost = area > rounds ? area : rounds;
    if (cost < own_us) cost = own_us;
    if (n > 1) cost += 3 + n * part_mb / 2.5;
    if (best == 0 || cost < best) {
      best = cost;
      L->splits = static_cast<int>(n);
    }
  }
  // (an item's steps have 24 bits; those of own keys are not cut into parts, and come to
  // all of them where one sequence holds all queries)
  if (steps >= (1 << 24) - 1 || L->cap_q * hq > INT32_MAX || L->cap_k * hkv * halves > INT32_MAX) return false;
  size_t off = kHdrWords * sizeof(int);
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  L->pref_q = take((static_cast<size_t>(batch) + 1) * sizeof(int));
  L->q_pairs = take(static_cast<size_t>(L->cap_q) * sizeof(int2));
  L->k_pairs = take(static_cast<size_t>(L->cap_k) * sizeof(int2));
  const size_t tiled = static_cast<size_t>(L->cap_q) * (hq >> sh) * kBlockM * sizeof(float);
  L->lse_t = take(tiled);
  L->delta_t = take(tiled);
  const size_t lin = static_cast<size_t>(L->rows_lin) * (hq >> sh) * sizeof(float);
  L->lse_lin = take(lin);
  L->delta_lin = take(lin);
  const size_t part = L->splits > 1 ? static_cast<size_t>(L->splits) * prefix_rows * hkv * d * sizeof(float) : 0;
  L->part_dk = take(part);
  L->part_dv = take(part);
  L->total = off;
  return true;
}

}  // namespace
}  // namespace teattn

using namespace teattn;

extern "C" {

size_t te_attn_prefix_fwd_workspace_size(int batch, int total_q, int total_kv, int prefix_rows,
                                         int hq, int hkv, int d) {
  FwdLayout L;
  return fwd_layout(batch, total_q, total_kv, prefix_rows, hq, hkv, d, &L) ? L.total : 0;
}

size_t te_attn_prefix_bwd_workspace_size(int batch, int total_q, int total_kv, int prefix_rows,
                                         int hq, int hkv, int d) {
  BwdLayout L;
  return bwd_layout(batch, total_q, total_kv, prefix_rows, hq, hkv, d, &L) ? L.total : 0;
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
  FwdLayout L;
  if (!fwd_layout(batch, total_q, total_kv, prefix_rows, hq, hkv, d, &L))
    return api_fail(TE_ERR_UNSUPPORTED, "problem too large for its work lists");
  if (workspace_bytes < L.total)
    return api_fail(TE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than te_attn_prefix_fwd_workspace_size()");
  const int sms = api_num_sms();
  if (sms <= 0) return api_fail(TE_ERR_CUDA, "no CUDA device");
  PrefixParams p = base_params(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_kv,
                               cu_seqlens_q_padded, cu_seqlens_kv_padded, prefix_len, batch, total_q,
                               total_kv, prefix_rows, hq, hkv, d, attn_scale, mask_type);
  p.out = out;
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.header = static_cast<int*>(workspace);
  p.seqs = reinterpret_cast<int4*>(ws + L.seqs);
  p.short_tok = reinterpret_cast<int*>(ws + L.short_tok);
  p.longs = reinterpret_cast<int4*>(ws + L.longs);
  p.entries = reinterpret_cast<int4*>(ws + L.entries);
  p.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + L.part_o);
  p.parts_target = L.parts_target;
  p.cap_longs = static_cast<int>(L.cap_longs);
  p.cap_entries = static_cast<int>(L.cap_entries);
  p.cap_rows = static_cast<int>(L.cap_rows);
  const bool bf16 = dtype == TE_DTYPE_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = api_timed(TE_KERNEL_SCHEDULE, st, [&] { return launch_prefix_schedule(p, st); });
  if (e != cudaSuccess) return api_cuda_fail(e, "shared-prefix schedule");
  if (total_q == 0) return api_ok();
  if (total_kv > 0 || prefix_rows > 0) {
    e = api_timed(TE_KERNEL_FWD, st, [&] { return launch_prefix_fwd(p, bf16, sms, st); });
    if (e != cudaSuccess) return api_cuda_fail(e, "shared-prefix forward");
  }
  e = api_timed(TE_KERNEL_FWD, st, [&] { return launch_prefix_join(p, bf16, sms, st); });
  return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "shared-prefix join");
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
  BwdLayout L;
  if (!bwd_layout(batch, total_q, total_kv, prefix_rows, hq, hkv, d, &L))
    return api_fail(TE_ERR_UNSUPPORTED, "problem too large for its work lists");
  if (workspace_bytes < L.total)
    return api_fail(TE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than te_attn_prefix_bwd_workspace_size()");
  const int sms = api_num_sms();
  if (sms <= 0) return api_fail(TE_ERR_CUDA, "no CUDA device");
  PrefixBwd p{};
  static_cast<PrefixParams&>(p) =
      base_params(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded,
                  prefix_len, batch, total_q, total_kv, prefix_rows, hq, hkv, d, attn_scale, mask_type);
  p.out_in = out;
  p.dout = dout;
  p.lse_in = lse;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.dkp = dk_prefix;
  p.dvp = dv_prefix;
  char* ws = static_cast<char*>(workspace);
  p.header = static_cast<int*>(workspace);
  int* pref_q = reinterpret_cast<int*>(ws + L.pref_q);
  p.pref_q = pref_q;
  p.q_pairs = reinterpret_cast<int2*>(ws + L.q_pairs);
  p.k_pairs = reinterpret_cast<int2*>(ws + L.k_pairs);
  p.pair_cap_q = static_cast<int>(L.cap_q);
  p.pair_cap_k = static_cast<int>(L.cap_k);
  p.lse_t = reinterpret_cast<float*>(ws + L.lse_t);
  p.delta_t = reinterpret_cast<float*>(ws + L.delta_t);
  p.lse_lin = reinterpret_cast<float*>(ws + L.lse_lin);
  p.delta_lin = reinterpret_cast<float*>(ws + L.delta_lin);
  p.part_dk = reinterpret_cast<float*>(ws + L.part_dk);
  p.part_dv = reinterpret_cast<float*>(ws + L.part_dv);
  p.pack_shift = L.pack_shift;
  p.vheads = hq >> L.pack_shift;
  p.vgroup = p.group >> L.pack_shift;
  p.rows_lin = L.rows_lin;
  p.splits = L.splits;
  const bool bf16 = dtype == TE_DTYPE_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = api_timed(TE_KERNEL_SCHEDULE, st, [&] { return launch_prefix_bwd_schedule(p, pref_q, st); });
  if (e != cudaSuccess) return api_cuda_fail(e, "shared-prefix schedule");
  e = api_timed(TE_KERNEL_DELTA, st, [&] { return launch_prefix_prep(p, bf16, sms, st); });
  if (e != cudaSuccess) return api_cuda_fail(e, "shared-prefix rows");
  if (total_q > 0 && (total_kv > 0 || prefix_rows > 0)) {
    e = api_timed(TE_KERNEL_DQ, st, [&] { return launch_prefix_bwd_dq(p, bf16, sms, st); });
    if (e != cudaSuccess) return api_cuda_fail(e, "shared-prefix dQ");
    e = api_timed(TE_KERNEL_DKDV, st, [&] { return launch_prefix_bwd_dkdv(p, bf16, sms, st); });
    if (e != cudaSuccess) return api_cuda_fail(e, "shared-prefix dK/dV");
  }
  // with one part and every row seen, the dK/dV kernel wrote all of it
  if (prefix_rows > 0 && (p.splits > 1 || prefix_len || total_q == 0)) {
    e = api_timed(TE_KERNEL_DKDV, st, [&] { return launch_prefix_sum(p, bf16, sms, st); });
    if (e != cudaSuccess) return api_cuda_fail(e, "shared-prefix gradient sum");
  }
  return api_ok();
}

}  // extern "C"
