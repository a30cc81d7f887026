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
// sizes and alignment allow it. A block takes a few tokens (and, with few tokens, a part of
// the heads), issues its first loads, works out the tokens' angles into shared memory while
// they are on their way, and applies them to every query and key head. What it took:
// bytes in flight from many small blocks (a thread keeps one access in 32-40 registers;
// unrolled, or with a warp on its own, it was slower), few instructions per access (one
// loop over rotated and copied units took 43 us where two take 34), and angles laid out so
// that neighbouring lanes read neighbouring words. 34656 tokens of 40 heads of 128, all of
// each head rotated: 113 us, 6.3 TB/s; a token each of 48 sequences: 6 us.
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
  int tokens, heads_per; // tokens and heads (of q, then k) of a block
  int units[2];          // of a head: rotated, copied
  uint32_t units_inv[2], heads_inv;  // ceil(2^32 / n) of those
};

constexpr int kRopeThreads = 256, kRopeTokens = 4;
constexpr int kRopeSMs = 152;  // of the GPU that work is cut for

// n / d with inv = ceil(2^32 / d), exact for n d < 2^32.
__device__ __forceinline__ int div_by(int n, uint32_t inv, int d) {
  return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), inv));
}

// Position of row r, or *real = false for a row that holds no token. A whole warp works on
// one row: the lanes count the sequences that start at or before it, one trip to memory
// instead of a search's several.
__device__ __forceinline__ long long rope_position(const RopeParams& p, int r, bool* real) {
  int b, i;
  *real = false;
  if (p.sbhd) {
    b = r % p.batch;
    i = r / p.batch;
    if (p.cu[b + 1] - p.cu[b] > p.total / p.batch) return 0;
  } else {
    int before = 0;
    for (int k = threadIdx.x & 31; k < p.batch; k += 32) before += p.cu_pad[k] <= r ? 1 : 0;
    b = __reduce_add_sync(0xffffffffu, before) - 1;
    if (b < 0) return 0;
    i = r - p.cu_pad[b];
    // a sequence whose real length does not fit its slot, or whose slot does not fit
    // the tensor, is treated as empty
    if (p.cu[b + 1] - p.cu[b] > p.cu_pad[b + 1] - p.cu_pad[b] || p.cu_pad[b] < 0 ||
        p.cu_pad[b + 1] > p.total)
      return 0;
  }
  if (i < 0 || i >= p.cu[b + 1] - p.cu[b]) return 0;
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
__device__ __forceinline__ void widen(typename Vec<V>::type v, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = kBF16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 x = unpack2<kBF16>(w[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
}

template <int V, bool kBF16>
__device__ __forceinline__ typename Vec<V>::type narrow(const float (&f)[V]) {
  typename Vec<V>::type v;
  if constexpr (V == 1) {
    v = kBF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f[0])) : __half_as_ushort(__float2half_rn(f[0]));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack2<kBF16>(f[2 * i], f[2 * i + 1]);
  }
  return v;
}

// kHalf: pairs (c, c + rot/2), a rotated unit is V pairs in two accesses; otherwise pairs
// (2c, 2c + 1), a unit is V elements in one (V = 1: one pair in two). A copied unit is V
// elements of the rest of the head. The two kinds are loops of their own, so that no warp
// goes through both.
template <int V, bool kHalf, bool kBF16>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  // (cos, sin) of pair i of rotated unit u at [token][i][u]: neighbouring lanes hold
  // neighbouring units, and read neighbouring words
  extern __shared__ float2 s_cs[];
  __shared__ long long s_pos[kRopeTokens];
  __shared__ bool s_real[kRopeTokens];
  using T = typename Vec<V>::type;
  constexpr bool kTwo = kHalf || V == 1;                // two accesses per rotated unit
  constexpr int kPair = kHalf ? V : (V == 1 ? 2 : V);  // elements from one unit to the next
  const int tid = threadIdx.x, warp = tid >> 5;
  const int r0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.total - r0);
  const int half = p.rot / 2, units = p.units[0], second = kHalf ? half : 1;
  const int h0 = blockIdx.y * p.heads_per, nh = min(p.heads_per, p.heads[0] + p.heads[1] - h0);
  // unit n of one kind: (token, head, unit) = (n / (heads_per units), .., n % units); its
  // elements' places in the input and output, or false past the block's last one
  auto locate = [&](int n, int kind, const uint16_t** x, uint16_t** y, int* t, int* u) {
    const int th = div_by(n, p.units_inv[kind], p.units[kind]);
    *u = n - th * p.units[kind];
    *t = div_by(th, p.heads_inv, p.heads_per);
    const int k = th - *t * p.heads_per;
    if (*t >= nt || k >= nh) return false;
    const int head = h0 + k, which = head >= p.heads[0] ? 1 : 0, h = which ? head - p.heads[0] : head;
    const long long r = r0 + *t;
    const int e = kind ? p.rot + *u * V : *u * kPair;
    *x = static_cast<const uint16_t*>(p.x[which]) + r * p.stride_t[which] + h * p.stride_h[which] + e;
    *y = static_cast<uint16_t*>(p.y[which]) + (r * p.heads[which] + h) * p.d + e;
    return true;
  };
  struct Unit {
    T a, b;
    uint16_t* y;
    int t, u;
    bool in;
  };
  auto load = [&](int n, int kind, Unit& w) {
    const uint16_t* x;
    w.in = locate(n, kind, &x, &w.y, &w.t, &w.u);
    if (!w.in) return;
    w.a = *reinterpret_cast<const T*>(x);
    if (kTwo && kind == 0) w.b = *reinterpret_cast<const T*>(x + second);
  };
  const int n_rot = nt * p.heads_per * units, n_copy = nt * p.heads_per * p.units[1];
  Unit w;
  load(tid, 0, w);

  if (warp < nt) {
    bool real;
    const long long pos = rope_position(p, r0 + warp, &real);
    s_pos[warp] = pos;
    s_real[warp] = real;
  }
  __syncthreads();
  const int per = half / units;  // pairs of a unit
  for (int c = tid; c < half; c += kRopeThreads) {
    const double turns = p.inv_freq[c] * 0.15915494309189535;  // 1 / (2 pi)
    const unsigned long long step =
        static_cast<unsigned long long>((turns - floor(turns)) * 18446744073709551616.0);
    const int u = c / per, at = (c - u * per) * units + u;
    for (int t = 0; t < nt; ++t) {
      const long long frac = static_cast<long long>(static_cast<unsigned long long>(s_pos[t]) * step);
      float sn, cs;
      sincospif(static_cast<float>(frac) * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63: half turns
      s_cs[t * half + at] = make_float2(cs * p.mscale, sn * p.mscale * p.sign);
    }
  }
  __syncthreads();

  for (int n = tid; n < n_rot; n += kRopeThreads) {
    if (n != tid) load(n, 0, w);
    if (!w.in) continue;
    const bool real = s_real[w.t];
    const float2* cs = s_cs + w.t * half + w.u;
    float f[V];
    widen<V, kBF16>(w.a, f);
    if constexpr (kTwo) {
      float g[V];
      widen<V, kBF16>(w.b, g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 z = cs[i * units];
        const float y1 = f[i] * z.x - g[i] * z.y, y2 = g[i] * z.x + f[i] * z.y;
        f[i] = y1;
        g[i] = y2;
      }
      *reinterpret_cast<T*>(w.y + second) = real ? narrow<V, kBF16>(g) : T{};
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 z = cs[i / 2 * units];
        const float y1 = f[i] * z.x - f[i + 1] * z.y, y2 = f[i + 1] * z.x + f[i] * z.y;
        f[i] = y1;
        f[i + 1] = y2;
      }
    }
    *reinterpret_cast<T*>(w.y) = real ? narrow<V, kBF16>(f) : T{};
  }
  for (int n = tid; n < n_copy; n += kRopeThreads) {
    load(n, 1, w);
    if (w.in) *reinterpret_cast<T*>(w.y) = s_real[w.t] ? w.a : T{};
  }
}

template <int V, bool kHalf>
static cudaError_t launch_rope_v(RopeParams p, bool bf16, cudaStream_t st) {
  p.units[0] = kHalf ? p.rot / 2 / V : p.rot / (V == 1 ? 2 : V);
  p.units[1] = (p.d - p.rot) / V;
  const int heads = p.heads[0] + p.heads[1], all = heads * (p.units[0] + p.units[1]);
  // A block takes up to four tokens, which share the work on the frequencies, while that is
  // no more than five passes of its threads: many small blocks overlap one's angles with
  // another's copies. With few tokens a block takes a part of a token's heads, half a pass at
  // least, to fill the SMs; and never more units than the divisions allow.
  const int share = 5 * kRopeThreads / all;
  p.tokens = p.total < 16 * kRopeSMs || share < 1 ? 1 : share < kRopeTokens ? share : kRopeTokens;
  const int blocks = (p.total + p.tokens - 1) / p.tokens;
  const int want = blocks < 2 * kRopeSMs ? (2 * kRopeSMs + blocks - 1) / blocks : 1;
  const int most = (all + kRopeThreads / 2 - 1) / (kRopeThreads / 2), least = (all + 8191) / 8192;
  int parts = want > most ? most : want > least ? want : least;
  parts = parts < heads ? parts : heads;
  p.heads_per = (heads + parts - 1) / parts;
  auto inverse = [](int n) { return n > 0 ? static_cast<uint32_t>(((1ull << 32) + n - 1) / n) : 0u; };
  p.units_inv[0] = inverse(p.units[0]);
  p.units_inv[1] = inverse(p.units[1]);
  p.heads_inv = inverse(p.heads_per);
  const size_t smem = static_cast<size_t>(p.tokens) * (p.rot / 2) * sizeof(float2);
  const dim3 grid(blocks, (heads + p.heads_per - 1) / p.heads_per);
  if (bf16)
    rope_kernel<V, kHalf, true><<<grid, kRopeThreads, smem, st>>>(p);
  else
    rope_kernel<V, kHalf, false><<<grid, kRopeThreads, smem, st>>>(p);
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
  // (rounded up to whole blocks of tokens in 32 bits)
  if (rows < 0 || rows > INT32_MAX - 256) return api_fail(TE_ERR_INVALID_ARG, "rows must lie in [0, 2^31 - 256)");
  if (hq < 1 || hkv < 0) return api_fail(TE_ERR_INVALID_ARG, "hq must be >= 1 and hkv >= 0");
  if (hq > 4096 || hkv > 4096) return api_fail(TE_ERR_UNSUPPORTED, "at most 4096 heads");
  if (d < 8 || d > 256 || d % 8 != 0)
    return api_fail(TE_ERR_UNSUPPORTED, "head dim must be a multiple of 8 in [8, 256]");
  if (n_freq < 1 || n_freq > d / 2)
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
