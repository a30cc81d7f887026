// Shared-prefix attention, backward, one warp per row.
//
//   P = exp(S - LSE),  dS = P (dO V^T - rowsum(dO O)),  dQ = scale dS K,
//   dK = scale dS^T Q and dV = P^T dO, summed over the group's heads and, for the
//   prefix, over every sequence.
//
// The plainest form that is right for every size: lanes hold a row's elements
// (c = lane + 32 i), a dot product is a warp sum, all in fp32.
#include <cuda_runtime.h>

#include <cmath>

#include "attn_prefix.cuh"
#include "sm103_ptx.cuh"

namespace teattn {

constexpr int kMaxPer = 8;  // ceil(256 / 32)

template <bool kBF16>
__device__ __forceinline__ float ld16(const void* base, size_t i) {
  if constexpr (kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  else return __half2float(static_cast<const __half*>(base)[i]);
}
template <bool kBF16>
__device__ __forceinline__ void st16(void* base, size_t i, float v) {
  if constexpr (kBF16) static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(base)[i] = __float2half_rn(v);
}

template <bool kBF16>
__device__ __forceinline__ void load_row(const void* base, size_t row, int d, float (&f)[kMaxPer]) {
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const int c = (threadIdx.x & 31) + 32 * i;
    f[i] = c < d ? ld16<kBF16>(base, row * d + c) : 0.f;
  }
}
template <bool kBF16>
__device__ __forceinline__ void store_row(void* base, size_t row, int d, const float (&f)[kMaxPer]) {
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const int c = (threadIdx.x & 31) + 32 * i;
    if (c < d) st16<kBF16>(base, row * d + c, f[i]);
  }
}
__device__ __forceinline__ float dot_row(const float (&a)[kMaxPer], const float (&b)[kMaxPer]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Token i of sequence b at packed query row r, or false for a row that is no token.
__device__ __forceinline__ bool query_of_row(const PrefixParams& p, int r, SeqInfo* s, int* i) {
  const int b = locate_row(p, p.cu_q_pad, r, i);
  if (b < 0) return false;
  *s = load_seq(p, b);
  return *i < s->len_q;
}

template <bool kBF16>
__global__ void prefix_dq_rows(PrefixParams p) {
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= static_cast<long long>(p.total_q) * p.hq) return;
  const int r = static_cast<int>(w / p.hq), h = static_cast<int>(w % p.hq), g = h / p.group;
  SeqInfo s;
  int i;
  float dq[kMaxPer] = {};
  if (query_of_row(p, r, &s, &i)) {
    float q[kMaxPer], g0[kMaxPer], k[kMaxPer], v[kMaxPer];
    load_row<kBF16>(p.q, w, p.d, q);
    load_row<kBF16>(p.dout, w, p.d, g0);
    load_row<kBF16>(p.out_in, w, p.d, v);
    const float delta = dot_row(g0, v), lse = p.lse_in[w];
    const int np = prefix_keys(p), n = np + row_keys(s, i, p.causal != 0);
    for (int j = 0; j < n; ++j) {
      const size_t row = j < np ? j : k_row(p, s, j - np);
      load_row<kBF16>(j < np ? p.kp : p.k, row * p.hkv + g, p.d, k);
      load_row<kBF16>(j < np ? p.vp : p.v, row * p.hkv + g, p.d, v);
      const float e = expf(dot_row(q, k) * p.scale - lse);
      const float ds = e * (dot_row(g0, v) - delta) * p.scale;
#pragma unroll
      for (int c = 0; c < kMaxPer; ++c) dq[c] = fmaf(ds, k[c], dq[c]);
    }
  }
  store_row<kBF16>(p.dq, w, p.d, dq);
}

// One warp per (key row, kv head): own keys first, then the prefix's.
template <bool kBF16>
__global__ void prefix_dkv_rows(PrefixParams p) {
  long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const long long own = static_cast<long long>(p.total_kv) * p.hkv;
  if (w >= own + static_cast<long long>(p.prefix_rows) * p.hkv) return;
  const bool pre = w >= own;
  if (pre) w -= own;
  const int r = static_cast<int>(w / p.hkv), g = static_cast<int>(w % p.hkv);
  float k[kMaxPer], v[kMaxPer], dk[kMaxPer] = {}, dv[kMaxPer] = {};
  int b0 = 0, b1 = p.batch, j = 0;
  bool real = true;
  if (pre) {
    real = r < prefix_keys(p);
  } else {
    b0 = locate_row(p, p.cu_kv_pad, r, &j);
    b1 = b0 + 1;
    real = b0 >= 0;
  }
  if (real) {
    load_row<kBF16>(pre ? p.kp : p.k, w, p.d, k);
    load_row<kBF16>(pre ? p.vp : p.v, w, p.d, v);
    for (int b = b0; b < b1; ++b) {
      const SeqInfo s = load_seq(p, b);
      if (!pre && j >= s.len_k) continue;
      for (int i = pre ? 0 : first_query(s, j, p.causal != 0); i < s.len_q; ++i) {
        for (int e = 0; e < p.group; ++e) {
          const size_t qr = q_row(p, s, i) * p.hq + g * p.group + e;
          float q[kMaxPer], g0[kMaxPer], o[kMaxPer];
          load_row<kBF16>(p.q, qr, p.d, q);
          load_row<kBF16>(p.dout, qr, p.d, g0);
          load_row<kBF16>(p.out_in, qr, p.d, o);
          const float pr = expf(dot_row(q, k) * p.scale - p.lse_in[qr]);
          const float ds = pr * (dot_row(g0, v) - dot_row(g0, o)) * p.scale;
#pragma unroll
          for (int c = 0; c < kMaxPer; ++c) {
            dv[c] = fmaf(pr, g0[c], dv[c]);
            dk[c] = fmaf(ds, q[c], dk[c]);
          }
        }
      }
    }
  }
  store_row<kBF16>(pre ? p.dkp : p.dk, w, p.d, dk);
  store_row<kBF16>(pre ? p.dvp : p.dv, w, p.d, dv);
}

// Status word of the call: inconsistent lengths (the sequences concerned, or the prefix,
// count as empty).
__global__ void prefix_status(PrefixParams p) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
    if (!load_seq(p, b).ok) bad = 1;
  if (threadIdx.x == 0 && p.prefix_len && (*p.prefix_len < 0 || *p.prefix_len > p.prefix_rows)) bad = 1;
  __syncthreads();
  if (threadIdx.x == 0) p.header[kHdrStatus] = bad ? kStatusBadSeqlens : 0;
}

static unsigned blocks_for(long long warps) { return static_cast<unsigned>((warps + 3) / 4); }

cudaError_t launch_prefix_bwd(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.total_q) * p.hq;
  const long long keys = (static_cast<long long>(p.total_kv) + p.prefix_rows) * p.hkv;
  prefix_status<<<1, 256, 0, st>>>(p);
  if (rows > 0) {
    if (bf16) prefix_dq_rows<true><<<blocks_for(rows), 128, 0, st>>>(p);
    else prefix_dq_rows<false><<<blocks_for(rows), 128, 0, st>>>(p);
  }
  if (keys > 0) {
    if (bf16) prefix_dkv_rows<true><<<blocks_for(keys), 128, 0, st>>>(p);
    else prefix_dkv_rows<false><<<blocks_for(keys), 128, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace teattn
