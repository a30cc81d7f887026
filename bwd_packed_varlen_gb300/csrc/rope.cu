// Rotary positions on packed or sequence-major queries and keys.
//
// A pair (x1, x2) of a head's first `rot` elements is turned by the angle of its token,
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a),  a = pos * w_c,
// with pos = start_b + i for token i of sequence b; the rest of the head is copied.
// The backward pass is the same with -a.
//
// Angles. pos * w_c reaches 1e6 and more, where fp32 has lost the fraction of a turn.
// w_c / 2 pi, taken to 64 bits, is reduced to its fraction and kept as a 64-bit
// fixed-point number of turns per position; pos times it, wrapping modulo 2^64, is then
// the fraction of a turn at pos, and only that is rounded to fp32 (for sincospif). The
// few fp64 operations are per block and pair, not per element.
//
// Memory-bound: each element is read once and written once, 16 bytes per access where
// sizes and alignment allow it. A block takes kTokens tokens, computes their angles into
// shared memory once and applies them to every query and key head.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/te_attn.h"
#include "api_internal.h"
#include "common.cuh"
#include "sm103_ptx.cuh"

namespace teattn {

struct RopeParams {
  const void* x[2];      // queries, keys (keys may be absent: heads[1] = 0)
  void* y[2];
  long long stride_t[2], stride_h[2];  // elements; outputs are contiguous
  int heads[2];
  const double* inv_freq;
  const int* cu;
  const int* cu_pad;
  const int* start;      // may be null
  int batch, total, d, rot;
  int sbhd;              // rows i * batch + b instead of cu_pad[b] + i
  float mscale, sign;    // sign -1: the inverse rotation
};

constexpr int kRopeThreads = 256;

// Position of row r, or *real = false for a row that holds no token.
__device__ __forceinline__ long long rope_position(const RopeParams& p, int r, bool* real) {
  int b = 0, i;
  *real = false;
  if (p.sbhd) {
    b = r % p.batch;
    i = r / p.batch;
  } else {
    if (r < p.cu_pad[0] || r >= p.cu_pad[p.batch]) return 0;
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu_pad[mid] <= r) lo = mid; else hi = mid - 1;
    }
    b = lo;
    i = r - p.cu_pad[b];
    // a sequence whose real length does not fit its slot, or whose slot does not fit
    // the tensor, is treated as empty
    if (p.cu[b + 1] - p.cu[b] > p.cu_pad[b + 1] - p.cu_pad[b] || p.cu_pad[b] < 0 ||
        p.cu_pad[b + 1] > p.total)
      return 0;
  }
  if (i < 0 || i >= p.cu[b + 1] - p.cu[b]) return 0;
  if (p.sbhd && p.cu[b + 1] - p.cu[b] > p.total / p.batch) return 0;
  *real = true;
  return static_cast<long long>(p.start ? p.start[b] : 0) + i;
}

// V consecutive 16-bit elements.
template <int V>
struct Vec;
template <>
struct Vec<8> { using type = uint4; };
template <>
struct Vec<4> { using type = uint2; };
template <>
struct Vec<2> { using type = uint32_t; };
template <>
struct Vec<1> { using type = uint16_t; };

template <int V, bool kBF16>
__device__ __forceinline__ void load_vec(const uint16_t* src, float (&f)[V]) {
  using T = typename Vec<V>::type;
  union {
    T v;
    uint16_t h[V];
  } u;
  u.v = *reinterpret_cast<const T*>(src);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (kBF16)
      f[i] = __uint_as_float(static_cast<uint32_t>(u.h[i]) << 16);
    else
      f[i] = __half2float(__ushort_as_half(u.h[i]));
  }
}

template <int V, bool kBF16>
__device__ __forceinline__ void store_vec(uint16_t* dst, const float (&f)[V]) {
  using T = typename Vec<V>::type;
  union {
    T v;
    uint16_t h[V];
  } u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (kBF16)
      u.h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
    else
      u.h[i] = __half_as_ushort(__float2half_rn(f[i]));
  }
  *reinterpret_cast<T*>(dst) = u.v;
}

// kHalf: pairs (c, c + rot/2), a unit is V pairs; otherwise pairs (2c, 2c + 1), a unit
// is V elements. The units of a head are its rotated ones, then V-element pieces of the
// rest. V = 1 with interleaved pairs takes one pair per unit.
template <int V, bool kHalf, bool kBF16>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p,
                                                            int tokens_per_block) {
  extern __shared__ float2 s_cs[];  // [tokens][rot / 2]
  __shared__ long long s_pos[16];
  __shared__ bool s_real[16];
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * tokens_per_block;
  const int nt = min(tokens_per_block, p.total - r0);
  const int half = p.rot / 2;
  if (tid < nt) {
    bool real;
    s_pos[tid] = rope_position(p, r0 + tid, &real);
    s_real[tid] = real;
  }
  __syncthreads();
  for (int c = tid; c < half; c += kRopeThreads) {
    const double turns = p.inv_freq[c] * 0.15915494309189535;  // 1 / (2 pi)
    const unsigned long long step =
        static_cast<unsigned long long>((turns - floor(turns)) * 18446744073709551616.0);
    for (int t = 0; t < nt; ++t) {
      const long long frac = static_cast<long long>(static_cast<unsigned long long>(s_pos[t]) * step);
      float sn, cs;
      sincospif(static_cast<float>(frac) * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63: half turns
      s_cs[t * half + c] = make_float2(cs * p.mscale, sn * p.mscale * p.sign);
    }
  }
  __syncthreads();

  constexpr int kPairElems = kHalf ? V : (V == 1 ? 2 : V);  // elements a rotated unit reads at once
  const int rot_units = kHalf ? half / V : p.rot / kPairElems;
  const int units = rot_units + (p.d - p.rot) / V;
  const int heads = p.heads[0] + p.heads[1];
  const int per_token = heads * units;
  for (int w = tid; w < nt * per_token; w += kRopeThreads) {
    const int t = w / per_token, rem = w - t * per_token;
    const int hh = rem / units, u = rem - hh * units;
    const int which = hh >= p.heads[0] ? 1 : 0;
    const int h = which ? hh - p.heads[0] : hh;
    const long long r = r0 + t;
    const uint16_t* x = static_cast<const uint16_t*>(p.x[which]) + r * p.stride_t[which] + h * p.stride_h[which];
    uint16_t* y = static_cast<uint16_t*>(p.y[which]) + (r * p.heads[which] + h) * p.d;
    const bool real = s_real[t];
    if (u >= rot_units) {
      const int c = p.rot + (u - rot_units) * V;
      float f[V];
      load_vec<V, kBF16>(x + c, f);
      if (!real) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 0.f;
      }
      store_vec<V, kBF16>(y + c, f);
      continue;
    }
    const float2* cs = s_cs + t * half;
    if constexpr (kHalf) {
      const int c = u * V;
      float a[V], b[V];
      load_vec<V, kBF16>(x + c, a);
      load_vec<V, kBF16>(x + half + c, b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 w2 = cs[c + i];
        const float y1 = a[i] * w2.x - b[i] * w2.y, y2 = b[i] * w2.x + a[i] * w2.y;
        a[i] = real ? y1 : 0.f;
        b[i] = real ? y2 : 0.f;
      }
      store_vec<V, kBF16>(y + c, a);
      store_vec<V, kBF16>(y + half + c, b);
    } else {
      const int c = u * kPairElems;
      float f[kPairElems];
      if constexpr (V == 1) {
        float a[1], b[1];
        load_vec<1, kBF16>(x + c, a);
        load_vec<1, kBF16>(x + c + 1, b);
        f[0] = a[0];
        f[1] = b[0];
      } else {
        load_vec<V, kBF16>(x + c, f);
      }
#pragma unroll
      for (int i = 0; i < kPairElems; i += 2) {
        const float2 w2 = cs[c / 2 + i / 2];
        const float y1 = f[i] * w2.x - f[i + 1] * w2.y, y2 = f[i + 1] * w2.x + f[i] * w2.y;
        f[i] = real ? y1 : 0.f;
        f[i + 1] = real ? y2 : 0.f;
      }
      if constexpr (V == 1) {
        const float a[1] = {f[0]}, b[1] = {f[1]};
        store_vec<1, kBF16>(y + c, a);
        store_vec<1, kBF16>(y + c + 1, b);
      } else {
        store_vec<V, kBF16>(y + c, f);
      }
    }
  }
}

template <int V, bool kHalf>
static cudaError_t launch_rope_v(const RopeParams& p, bool bf16, cudaStream_t st) {
  const int tokens = 4;
  const int grid = (p.total + tokens - 1) / tokens;
  const size_t smem = static_cast<size_t>(tokens) * (p.rot / 2) * sizeof(float2);
  if (bf16)
    rope_kernel<V, kHalf, true><<<grid, kRopeThreads, smem, st>>>(p, tokens);
  else
    rope_kernel<V, kHalf, false><<<grid, kRopeThreads, smem, st>>>(p, tokens);
  return cudaGetLastError();
}

// The widest access that the rotated part's split, every stride and every pointer allow.
static int rope_vector(const RopeParams& p, bool half_layout) {
  const int split = half_layout ? p.rot / 2 : p.rot;
  int v = 8;
  auto fits = [&](int n) {
    if (split % n != 0) return false;
    for (int w = 0; w < 2; ++w) {
      if (p.heads[w] == 0) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(p.x[w]) | reinterpret_cast<uintptr_t>(p.y[w]);
      if (a % (2 * n) != 0 || p.stride_t[w] % n != 0 || p.stride_h[w] % n != 0) return false;
    }
    return true;
  };
  while (v > 1 && !fits(v)) v /= 2;
  return v;
}

static cudaError_t launch_rope(const RopeParams& p, bool half_layout, bool bf16, cudaStream_t st) {
  switch (rope_vector(p, half_layout)) {
    case 8:
      return half_layout ? launch_rope_v<8, true>(p, bf16, st) : launch_rope_v<8, false>(p, bf16, st);
    case 4:
      return half_layout ? launch_rope_v<4, true>(p, bf16, st) : launch_rope_v<4, false>(p, bf16, st);
    case 2:
      return half_layout ? launch_rope_v<2, true>(p, bf16, st) : launch_rope_v<2, false>(p, bf16, st);
    default:
      return half_layout ? launch_rope_v<1, true>(p, bf16, st) : launch_rope_v<1, false>(p, bf16, st);
  }
}

static int rope_impl(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
                     int n_freq, const int32_t* cu, const int32_t* cu_pad, const int32_t* start,
                     int batch, long long rows, int hq, int hkv, int d, int64_t q_stride_t,
                     int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h, int interleaved,
                     float mscale, int inverse, int dtype, void* stream, bool sbhd) {
  if (!cu || !cu_pad) return api_fail(TE_ERR_INVALID_ARG, "cu_seqlens pointers must not be NULL");
  if (batch < 1) return api_fail(TE_ERR_INVALID_ARG, "batch must be >= 1");
  if (rows < 0 || rows > INT32_MAX) return api_fail(TE_ERR_INVALID_ARG, "rows must lie in [0, 2^31)");
  if (hq < 1 || hkv < 0) return api_fail(TE_ERR_INVALID_ARG, "hq must be >= 1 and hkv >= 0");
  if (hq > 65535 || hkv > 65535) return api_fail(TE_ERR_UNSUPPORTED, "at most 65535 heads");
  if (d < 8 || d > 256 || d % 8 != 0)
    return api_fail(TE_ERR_UNSUPPORTED, "head dim must be a multiple of 8 in [8, 256]");
  if (n_freq < 1 || 2 * n_freq > d)
    return api_fail(TE_ERR_INVALID_ARG, "n_freq must lie in [1, d / 2]");
  if (dtype != TE_DTYPE_FP16 && dtype != TE_DTYPE_BF16)
    return api_fail(TE_ERR_UNSUPPORTED, "dtype must be TE_DTYPE_FP16 or TE_DTYPE_BF16");
  if (!(mscale - mscale == 0.f)) return api_fail(TE_ERR_INVALID_ARG, "mscale must be finite");
  if (!inv_freq) return api_fail(TE_ERR_INVALID_ARG, "inv_freq must not be NULL");
  if (rows > 0 && (!q || !q_out || (hkv > 0 && (!k || !k_out))))
    return api_fail(TE_ERR_INVALID_ARG, "q, q_out and, with hkv > 0, k and k_out must not be NULL");
  const void* two[] = {q, k, q_out, k_out};
  for (const void* x : two)
    if (reinterpret_cast<uintptr_t>(x) & 1u)
      return api_fail(TE_ERR_INVALID_ARG, "tensors must be 2-byte aligned");
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) || (reinterpret_cast<uintptr_t>(cu) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_pad) & 3u) || (reinterpret_cast<uintptr_t>(start) & 3u))
    return api_fail(TE_ERR_INVALID_ARG, "inv_freq and the int32 arrays need their natural alignment");
  constexpr int64_t kMaxStride = int64_t(1) << 31;
  for (int64_t s : {q_stride_t, q_stride_h, k_stride_t, k_stride_h})
    if (s < 0 || s > kMaxStride) return api_fail(TE_ERR_INVALID_ARG, "strides must lie in [0, 2^31]");
  if (rows == 0) return api_ok();
  RopeParams p{};
  p.x[0] = q;
  p.x[1] = k;
  p.y[0] = q_out;
  p.y[1] = k_out;
  p.stride_t[0] = q_stride_t;
  p.stride_h[0] = q_stride_h;
  p.stride_t[1] = k_stride_t;
  p.stride_h[1] = k_stride_h;
  p.heads[0] = hq;
  p.heads[1] = hkv;
  p.inv_freq = inv_freq;
  p.cu = cu;
  p.cu_pad = cu_pad;
  p.start = start;
  p.batch = batch;
  p.total = static_cast<int>(rows);
  p.d = d;
  p.rot = 2 * n_freq;
  p.sbhd = sbhd ? 1 : 0;
  p.mscale = mscale;
  p.sign = inverse ? -1.f : 1.f;
  const cudaError_t e = launch_rope(p, !interleaved, dtype == TE_DTYPE_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "rotary positions");
}

}  // namespace teattn

extern "C" {

int te_attn_rope_thd(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
                     int n_freq, const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                     const int32_t* start_positions, int batch, int total, int hq, int hkv, int d,
                     int64_t q_stride_t, int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h,
                     int interleaved, float mscale, int inverse, int dtype, void* stream) {
  return teattn::rope_impl(q, k, q_out, k_out, inv_freq, n_freq, cu_seqlens, cu_seqlens_padded,
                           start_positions, batch, total, hq, hkv, d, q_stride_t, q_stride_h,
                           k_stride_t, k_stride_h, interleaved, mscale, inverse, dtype, stream, false);
}

int te_attn_rope_sbhd(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
                      int n_freq, const int32_t* cu_seqlens, const int32_t* start_positions, int batch,
                      int seq, int hq, int hkv, int d, int64_t q_stride_t, int64_t q_stride_h,
                      int64_t k_stride_t, int64_t k_stride_h, int interleaved, float mscale, int inverse,
                      int dtype, void* stream) {
  const long long rows = batch < 1 || seq < 0 ? -1 : static_cast<long long>(batch) * seq;
  if (rows < 0)
    return teattn::api_fail(TE_ERR_INVALID_ARG, "batch must be >= 1 and seq >= 0");
  return teattn::rope_impl(q, k, q_out, k_out, inv_freq, n_freq, cu_seqlens, cu_seqlens,
                           start_positions, batch, rows, hq, hkv, d, q_stride_t, q_stride_h, k_stride_t,
                           k_stride_h, interleaved, mscale, inverse, dtype, stream, true);
}

}  // extern "C"
