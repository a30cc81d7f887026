// Appending keys and values to a paged cache, with rotary positions put in on the way, and
// reading them back.
//
// One pass: queries and keys are turned as in rope.cu (the angle of a token as a 64-bit
// fraction of a turn, pairs in fp32, one rounding), queries go to their output, keys and values
// to the place of their position. Memory-bound: each element is read once and written once,
// 16 bytes per access where sizes and alignment allow it. Prompts of 1500-8000 tokens, 32 + 2 * 8
// heads of 128: 101.5 us, launches in a row, 93 % of the measured copy rate (eight blocks an SM, so 32
// registers a thread: left to the compiler, with four tokens a block, 122 instead of 105); 48 single tokens: 4.3
// us, a launch. Calls from Python: 105 and 6.2.
//
// Into 4 bits a block's turned keys go to shared memory first, rounded to 16 bits as a 16-bit
// cache would hold them (pairs that are turned together lie in different groups of 32); then
// four lanes take a group, eight elements each, find its least and greatest by two exchanges
// and write 16 bytes of codes and 4 of step and least value. The step is rounded towards zero,
// so that no code stands for more than the greatest element, which may be the type's last.
// Both quotients are true divisions: elements often lie on a border between two codes, and close
// to one a product with a reciprocal could come out on the other side. 12 prompts of 30-900 tokens,
// 16 + 2 * 8 heads of 64, into 4 bits and gathered again: 30 us for 8.1 us of bytes, launches in a row
// (calls 36); bounded by instructions, some 50 an element of queries, keys and values, in three
// issue slots of four.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/te_attn.h"
#include "api_internal.h"
#include "paged.cuh"
#include "rope.cuh"

namespace teattn {

struct AppendParams {
  PagedCache cache;
  const void* x[3];  // queries, keys, values
  long long stride_t[3], stride_h[3];
  void* q_out;
  int heads[3];
  const double* inv_freq;
  const int* cu;
  const int* cu_pad;
  const int* past;
  int* status;           // may be null
  int batch, total, d, rot;
  float mscale;
  int tokens, heads_per; // tokens and heads (of q, k, then v) of a block
  int units[3];          // of a head: turned; copied beside them; copied of a head of v
  uint32_t units_inv[3], words_inv;
};

constexpr int kAppendThreads = 256, kAppendTokens = 2;
constexpr int kAppendSMs = 152;  // of the GPU that work is cut for

struct Token {
  int pos;   // -1: the row holds no token
  int page;  // -1: its place is outside the cache
};

// Tokens of sequence b; -1: its lengths, or its past, are inconsistent.
__device__ __forceinline__ int tokens_of(const int* cu, const int* cu_pad, const int* past, int total, int b) {
  const int n = cu[b + 1] - cu[b], off = cu_pad[b], end = cu_pad[b + 1];
  // (with no offset below zero the span does not wrap)
  return n < 0 || (off | end | past[b]) < 0 || n > end - off || end > total ? -1 : n;
}

// The status that a call begins with: whether some sequence is inconsistent. (The kernels go by rows,
// and one without rows has none to be found by.)
__global__ void __launch_bounds__(1024) paged_status_kernel(const int* cu, const int* cu_pad, const int* past, int batch, int total, int* status) {
  int bad = 0;
  for (int b = threadIdx.x; b < batch; b += blockDim.x) bad |= tokens_of(cu, cu_pad, past, total, b) < 0 ? 1 : 0;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? kStatusBadSeqlens : 0;
}

// The sequence of packed row r and its token's position; -1 for a row that holds no token. A whole
// warp works on one row.
__device__ __forceinline__ int token_of(const int* cu, const int* cu_pad, const int* past, int batch, int total, int r, int* pos) {
  const int b = sequence_at(cu_pad, batch, r);
  if (b < 0) return -1;
  const int n = tokens_of(cu, cu_pad, past, total, b), i = r - cu_pad[b], first = past[b];
  if (n < 0 || i >= n) return -1;
  const long long at = static_cast<long long>(first) + i;
  *pos = at < INT_MAX ? static_cast<int>(at) : INT_MAX;
  return b;
}

// Codes of one group's eight elements in this lane (the group's others in the lanes beside it:
// four neighbouring lanes hold 32 elements); every lane of the warp takes part.
//
// Steps and codes are those of exact arithmetic, though 32 bits do not hold every difference of
// 16-bit numbers (15 - 1e-7). The step's rounding is towards zero all along: 15 steps of 16 bits are
// an fp32 number, so a difference cut off to fp32 has as many of them as the exact one. Borders
// (c + 1/2) s between codes are fp32 numbers too, with zeros in the fraction's last bits: a difference
// that is not exact takes its odd neighbour, which is no border and lies on the same side of each.
// Dividing keeps that: a difference below a border b is at most b (1 - 2^-24), and its quotient is then
// below c + 1/2 by more than half of the distance to the number before that; likewise above.
template <bool kBF16>
__device__ __forceinline__ uint32_t quantize8(float (&f)[8], uint32_t* meta) {
  float lo = f[0], hi = f[0];
  float sum = 0.f;  // NaN if any element is not finite
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, f[i]);
    hi = fmaxf(hi, f[i]);
    sum += f[i] - f[i];
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float least = lo;
  const bool far = isinf(hi - lo);
  if (far) {  // past fp32's last number: everything halved, which is exact
    lo *= 0.5f;
    hi *= 0.5f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= 0.5f;
  }
  const float fifteenth = __fdiv_rz(__fsub_rz(hi, lo), 15.f);
  *meta = pack_meta<kBF16>(far ? 2.f * fifteenth : fifteenth, least);
  if (sum != 0.f) {
    *meta = 0x7fff7fffu;  // NaN in either type
    return 0;
  }
  const float step = unpack2<kBF16>(*meta).x * (far ? 0.5f : 1.f);
  uint32_t w = 0;
  if (step > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t down = __float_as_uint(__fsub_rz(f[i], lo)), up = __float_as_uint(__fsub_ru(f[i], lo));
      const float d = __uint_as_float(down | ((down ^ up) & 1u));  // (neighbours differ in the last bit)
      w |= static_cast<uint32_t>(min(15, __float2int_rn(d / step))) << (4 * i);
    }
  }
  return w;
}

// V elements per access; kHalf: pairs (c, c + rot/2), otherwise (2c, 2c + 1), as in rope.cu.
template <int V, bool kHalf, bool kBF16, bool k4>
__global__ void __launch_bounds__(kAppendThreads, 8) paged_append_kernel(const __grid_constant__ AppendParams p) {
  // (cos, sin) of pair i of unit u at [token][i][u]; behind them, with 4 bits, turned keys
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Token s_tok[kAppendTokens];
  using T = typename Vec<V>::type;
  constexpr bool kTwo = kHalf || V == 1;
  constexpr int kPair = kHalf ? V : (V == 1 ? 2 : V);
  float2* s_cs = reinterpret_cast<float2*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int r0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.total - r0);
  const int half = p.rot / 2, second = kHalf ? half : 1;
  uint16_t* s_keys = reinterpret_cast<uint16_t*>(smem + static_cast<size_t>(p.tokens) * half * sizeof(float2));
  const int h0 = blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.heads[0] + p.heads[1] + p.heads[2]);
  // heads of the block that are turned (q, k), and those of k and v
  const int turned = max(0, min(h1, p.heads[0] + p.heads[1]) - h0);
  const int k0 = max(h0, p.heads[0]), nk = max(0, min(h1, p.heads[0] + p.heads[1]) - k0);
  const int v0 = max(h0, p.heads[0] + p.heads[1]), nv = max(0, h1 - v0);

  auto source = [&](int t, int head, int e) {
    const int which = head < p.heads[0] ? 0 : head < p.heads[0] + p.heads[1] ? 1 : 2;
    const int h = which == 0 ? head : which == 1 ? head - p.heads[0] : head - p.heads[0] - p.heads[1];
    return static_cast<const uint16_t*>(p.x[which]) + (r0 + t) * p.stride_t[which] + h * p.stride_h[which] + e;
  };
  // where element e of head h of keys (kv = 0) or values goes in a 16-bit cache
  auto cached = [&](int kv, int page, int pos, int h, int e) {
    const int slot = pos & ((1 << p.cache.shift) - 1);
    return reinterpret_cast<uint16_t*>(p.cache.data[kv] + page * p.cache.stride[kv]) + page_row(p.cache, h, slot) * p.d + e;
  };
  struct Unit {
    T a, b;
    int t, head, e, u;
    bool in;
  };
  auto load = [&](int n, int kind, Unit& w) {  // kind 0: turned, 1: copied beside them
    const int th = div_by(n, p.units_inv[kind], p.units[kind]);
    w.u = n - th * p.units[kind];
    w.t = turned > 0 ? th / turned : nt;
    w.in = w.t < nt;
    if (!w.in) return;
    w.head = h0 + th - w.t * turned;
    w.e = kind ? p.rot + w.u * V : w.u * kPair;
    const uint16_t* x = source(w.t, w.head, w.e);
    w.a = *reinterpret_cast<const T*>(x);
    if (kTwo && kind == 0) w.b = *reinterpret_cast<const T*>(x + second);
  };
  const int n_rot = p.units[0] > 0 ? nt * turned * p.units[0] : 0, n_copy = p.units[1] > 0 ? nt * turned * p.units[1] : 0;
  Unit w;
  w.in = false;
  if (n_rot > 0 && tid < n_rot) load(tid, 0, w);

  if (warp < nt) {
    int pos = -1, page = -1;
    const int b = token_of(p.cu, p.cu_pad, p.past, p.batch, p.total, r0 + warp, &pos);
    if (b >= 0) {
      page = page_of(p.cache, b, pos);
      if (page < 0 && p.status && (tid & 31) == 0) atomicOr(p.status, kStatusBadPages);
    } else {
      pos = -1;
    }
    s_tok[warp] = Token{pos, page};
  }
  __syncthreads();
  if (n_rot > 0) {
    const int units = p.units[0], per = half / units;
    for (int c = tid; c < half; c += kAppendThreads) {
      const unsigned long long step = turn_per_position(p.inv_freq[c]);
      const int u = c / per, at = (c - u * per) * units + u;
      for (int t = 0; t < nt; ++t) {
        float sn, cs;
        sincos_at(s_tok[t].pos, step, &sn, &cs);
        s_cs[t * half + at] = make_float2(cs * p.mscale, sn * p.mscale);
      }
    }
    __syncthreads();
  }

  // V elements of a turned or copied unit to their place
  auto put = [&](const Unit& at, int e, T v) {
    const Token tk = s_tok[at.t];
    if (at.head < p.heads[0]) {
      uint16_t* y = static_cast<uint16_t*>(p.q_out) + (static_cast<long long>(r0 + at.t) * p.heads[0] + at.head) * p.d + e;
      *reinterpret_cast<T*>(y) = tk.pos >= 0 ? v : T{};
    } else if constexpr (k4) {
      *reinterpret_cast<T*>(s_keys + (at.t * nk + at.head - k0) * p.d + e) = v;
    } else if (tk.page >= 0) {
      *reinterpret_cast<T*>(cached(0, tk.page, tk.pos, at.head - p.heads[0], e)) = v;
    }
  };
  for (int n = tid; n < n_rot; n += kAppendThreads) {
    if (n != tid) load(n, 0, w);
    if (!w.in) continue;
    const float2* cs = s_cs + w.t * half + w.u;
    float f[V];
    widen<V, kBF16>(w.a, f);
    if constexpr (kTwo) {
      float g[V];
      widen<V, kBF16>(w.b, g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 z = cs[i * p.units[0]];
        const float y1 = f[i] * z.x - g[i] * z.y, y2 = g[i] * z.x + f[i] * z.y;
        f[i] = y1;
        g[i] = y2;
      }
      put(w, w.e + second, narrow<V, kBF16>(g));
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 z = cs[i / 2 * p.units[0]];
        const float y1 = f[i] * z.x - f[i + 1] * z.y, y2 = f[i + 1] * z.x + f[i] * z.y;
        f[i] = y1;
        f[i + 1] = y2;
      }
    }
    put(w, w.e, narrow<V, kBF16>(f));
  }
  for (int n = tid; n < n_copy; n += kAppendThreads) {
    load(n, 1, w);
    if (w.in) put(w, w.e, w.a);
  }
  if constexpr (!k4) {
    // values, two accesses in flight: a place in a token's heads for all of the block's tokens
    const int per = nv * p.units[2];
    for (int n = tid; n < per; n += kAppendThreads) {
      const int hh = div_by(n, p.units_inv[2], p.units[2]), h = v0 + hh, e = (n - hh * p.units[2]) * V;
      for (int t = 0; t < nt; t += 2) {
        T v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (t + k < nt) v[k] = *reinterpret_cast<const T*>(source(t + k, h, e));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (t + k >= nt) continue;
          const Token tk = s_tok[t + k];
          if (tk.page >= 0) *reinterpret_cast<T*>(cached(1, tk.page, tk.pos, h - p.heads[0] - p.heads[1], e)) = v[k];
        }
      }
    }
  } else {
    __syncthreads();
    const int words = p.d / 8, n_w = nt * (nk + nv) * words;  // eight elements a lane
    const uint32_t kv_inv = nk + nv > 0 ? 0xffffffffu / static_cast<uint32_t>(nk + nv) + 1u : 0u;  // ceil(2^32 / n), or 0 for 1
#pragma unroll 1
    for (int base = 0; base < n_w; base += kAppendThreads) {
      const int n = min(base + tid, n_w - 1);  // (every lane takes part in the exchanges)
      const int th = div_by(n, p.words_inv, words), word = n - th * words, t = div_by(th, kv_inv, nk + nv), hh = th - t * (nk + nv);
      const bool key = hh < nk;
      const uint16_t* x = key ? s_keys + (t * nk + hh) * p.d + word * 8 : source(t, v0 + hh - nk, word * 8);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; i += V) {
        float g[V];
        widen<V, kBF16>(*reinterpret_cast<const T*>(x + i), g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[i + j] = g[j];
      }
      uint32_t meta;
      const uint32_t codes = quantize8<kBF16>(f, &meta);
      const Token tk = s_tok[t];
      if (base + tid >= n_w || tk.page < 0) continue;
      const int kv = key ? 0 : 1, h = key ? k0 + hh - p.heads[0] : v0 + hh - nk - p.heads[0] - p.heads[1];
      const long long row = page_row(p.cache, h, tk.pos & ((1 << p.cache.shift) - 1));
      *reinterpret_cast<uint32_t*>(p.cache.data[kv] + tk.page * p.cache.stride[kv] + row * p.cache.row_bytes + word * 4) = codes;
      if (word % 4 == 0)
        *reinterpret_cast<uint32_t*>(p.cache.meta[kv] + tk.page * p.cache.meta_stride[kv] + row * (p.d / 8) + word) = meta;
    }
  }
}

template <int V, bool kHalf, bool k4>
static cudaError_t launch_append_v(AppendParams p, bool bf16, cudaStream_t st) {
  p.units[0] = kHalf ? p.rot / 2 / V : p.rot / (V == 1 ? 2 : V);
  p.units[1] = (p.d - p.rot) / V;
  p.units[2] = p.d / V;
  // Tokens and heads of a block much as in rope.cu: two tokens share the frequencies (four: 6 % slower for
  // the prompts above); with few tokens a block takes a part of a token's heads.
  const int heads = p.heads[0] + p.heads[1] + p.heads[2], all = heads * (p.units[0] + p.units[1]);
  const int share = 5 * kAppendThreads / all;
  p.tokens = p.total < 16 * kAppendSMs || share < 1 ? 1 : share < kAppendTokens ? share : kAppendTokens;
  const int blocks = (p.total + p.tokens - 1) / p.tokens;
  const int want = blocks < 2 * kAppendSMs ? (2 * kAppendSMs + blocks - 1) / blocks : 1;
  const int most = (all + kAppendThreads / 2 - 1) / (kAppendThreads / 2);
  // turned keys of a block stay within 32 KB of shared memory, its units within the divisions
  const int least = max((all + 8191) / 8192, (heads * p.tokens * p.d * 2 + 32767) / 32768);
  int parts = want > most ? most : want;
  parts = parts < least ? least : parts;
  parts = parts < heads ? parts : heads;
  p.heads_per = (heads + parts - 1) / parts;
  for (int i = 0; i < 3; ++i)
    p.units_inv[i] = p.units[i] > 0 ? static_cast<uint32_t>(((1ull << 32) + p.units[i] - 1) / p.units[i]) : 0u;
  p.words_inv = static_cast<uint32_t>(((1ull << 32) + p.d / 8 - 1) / (p.d / 8));
  size_t smem = static_cast<size_t>(p.tokens) * (p.rot / 2) * sizeof(float2);
  if (k4) {
    smem = (smem + 15) / 16 * 16 + static_cast<size_t>(p.tokens) * min(p.heads_per, p.heads[1]) * p.d * 2;
  }
  const dim3 grid(blocks, (heads + p.heads_per - 1) / p.heads_per);
  if (bf16)
    paged_append_kernel<V, kHalf, true, k4><<<grid, kAppendThreads, smem, st>>>(p);
  else
    paged_append_kernel<V, kHalf, false, k4><<<grid, kAppendThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <bool k4>
static cudaError_t launch_append(const AppendParams& p, bool half_layout, bool bf16, cudaStream_t st) {
  // the widest access that the turned part's split, every stride and every pointer allow
  const int split = half_layout ? p.rot / 2 : p.rot;
  auto fits = [&](int n) {
    if (split % n != 0) return false;
    for (int w = 0; w < 3; ++w) {
      if (p.heads[w] == 0) continue;
      if (reinterpret_cast<uintptr_t>(p.x[w]) % (2 * n) != 0 || p.stride_t[w] % n != 0 || p.stride_h[w] % n != 0) return false;
    }
    return p.heads[0] == 0 || reinterpret_cast<uintptr_t>(p.q_out) % (2 * n) == 0;
  };
  int v = 8;
  while (v > 1 && !fits(v)) v /= 2;
  switch (v) {
    case 8: return half_layout ? launch_append_v<8, true, k4>(p, bf16, st) : launch_append_v<8, false, k4>(p, bf16, st);
    case 4: return half_layout ? launch_append_v<4, true, k4>(p, bf16, st) : launch_append_v<4, false, k4>(p, bf16, st);
    case 2: return half_layout ? launch_append_v<2, true, k4>(p, bf16, st) : launch_append_v<2, false, k4>(p, bf16, st);
    default: return half_layout ? launch_append_v<1, true, k4>(p, bf16, st) : launch_append_v<1, false, k4>(p, bf16, st);
  }
}

// ---------------------------------------------------------------------------
// Reading back: eight elements a thread, a warp per row for its place. Prompts as above, 8 heads of 128:
// 40 us in 16 bits for 31.6 us of bytes, 37 in 4 bits for 20.7.
// ---------------------------------------------------------------------------
struct GatherParams {
  PagedCache cache;
  void* y[2];
  const int* cu;
  const int* cu_pad;
  const int* start;
  int* status;
  int batch, total;
  int tokens;  // of a block
  uint32_t words_inv, heads_inv;  // ceil(2^32 / n) of d / 8 and of hkv
};

constexpr int kGatherThreads = 256, kGatherTokens = 8;

template <bool kBF16, bool k4>
__global__ void __launch_bounds__(kGatherThreads) paged_gather_kernel(const __grid_constant__ GatherParams p) {
  __shared__ Token s_tok[kGatherTokens];
  const int tid = threadIdx.x, warp = tid >> 5;
  const int r0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.total - r0);
  if (warp < nt) {
    int pos = -1, page = -1;
    const int b = token_of(p.cu, p.cu_pad, p.start, p.batch, p.total, r0 + warp, &pos);
    if (b >= 0) {
      page = page_of(p.cache, b, pos);
      if (page < 0 && p.status && (tid & 31) == 0) atomicOr(p.status, kStatusBadPages);
    }
    s_tok[warp] = Token{pos, page};
  }
  __syncthreads();
  const int words = p.cache.d / 8, per = p.cache.hkv * words;
  for (int n = tid; n < 2 * nt * per; n += kGatherThreads) {
    const int th = div_by(n, p.words_inv, words), word = n - th * words, tk2 = div_by(th, p.heads_inv, p.cache.hkv);
    const int h = th - tk2 * p.cache.hkv, kv = tk2 >= nt ? 1 : 0, t = tk2 - kv * nt;
    const Token tk = s_tok[t];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (tk.page >= 0) {
      const long long row = page_row(p.cache, h, tk.pos & ((1 << p.cache.shift) - 1));
      const uint8_t* base = p.cache.data[kv] + tk.page * p.cache.stride[kv] + row * p.cache.row_bytes;
      if constexpr (k4) {
        const uint32_t codes = *reinterpret_cast<const uint32_t*>(base + word * 4);
        const uint32_t meta = *reinterpret_cast<const uint32_t*>(p.cache.meta[kv] + tk.page * p.cache.meta_stride[kv] +
                                                                 row * (p.cache.d / 8) + word / 4 * 4);
        v = dequantize8<kBF16>(codes, meta, kCodeMagic<kBF16>);
      } else {
        v = *reinterpret_cast<const uint4*>(base + word * 16);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y[kv]) + (static_cast<long long>(r0 + t) * p.cache.hkv + h) * p.cache.d +
                              word * 8) = v;
  }
}

static bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int api_paged_cache(const te_attn_paged_cache* c, PagedCache* out) {
  if (!c) return api_fail(TE_ERR_INVALID_ARG, "cache must not be NULL");
  if (!c->k || !c->v || !c->page_table) return api_fail(TE_ERR_INVALID_ARG, "k, v and page_table must not be NULL");
  if (!c->k_meta != !c->v_meta) return api_fail(TE_ERR_INVALID_ARG, "k_meta and v_meta go together");
  const bool four = c->k_meta != nullptr;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
    return api_fail(TE_ERR_UNSUPPORTED, "page_size must be a power of two in [16, 4096]");
  if (c->num_pages < 1 || c->max_pages < 1) return api_fail(TE_ERR_INVALID_ARG, "num_pages and max_pages must be >= 1");
  if (static_cast<long long>(c->max_pages) * c->page_size > (1 << 30))
    return api_fail(TE_ERR_UNSUPPORTED, "a sequence's pages hold at most 2^30 tokens");
  if (c->hkv < 1) return api_fail(TE_ERR_INVALID_ARG, "hkv must be >= 1");
  if (c->hkv > 4096) return api_fail(TE_ERR_UNSUPPORTED, "at most 4096 heads");
  if (c->d < 8 || c->d > 256 || c->d % 8 != 0)
    return api_fail(TE_ERR_UNSUPPORTED, "head dim must be a multiple of 8 in [8, 256]");
  if (four && c->d % 32 != 0) return api_fail(TE_ERR_UNSUPPORTED, "a cache of 4 bits needs a head dim that is a multiple of 32");
  if (c->dtype != TE_DTYPE_FP16 && c->dtype != TE_DTYPE_BF16)
    return api_fail(TE_ERR_UNSUPPORTED, "dtype must be TE_DTYPE_FP16 or TE_DTYPE_BF16");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_meta, 16) || !aligned(c->v_meta, 16))
    return api_fail(TE_ERR_INVALID_ARG, "the cache's tensors must be 16-byte aligned");
  if (!aligned(c->page_table, 4)) return api_fail(TE_ERR_INVALID_ARG, "int32 arrays need their natural alignment");
  const int64_t row = four ? c->d / 2 : c->d * 2, page = row * c->page_size * c->hkv;
  const int64_t meta = static_cast<int64_t>(c->d / 8) * c->page_size * c->hkv, most = INT64_MAX / 4 / c->num_pages;
  for (int64_t s : {c->k_stride, c->v_stride})
    if (s < page || s % 16 != 0 || s > most)
      return api_fail(TE_ERR_INVALID_ARG, "page strides must be multiples of 16 bytes, of at least a page");
  if (four)
    for (int64_t s : {c->k_meta_stride, c->v_meta_stride})
      if (s < meta || s % 16 != 0 || s > most)
        return api_fail(TE_ERR_INVALID_ARG, "page strides must be multiples of 16 bytes, of at least a page");
  if (c->table_stride < 0 || c->table_stride > (int64_t(1) << 31))
    return api_fail(TE_ERR_INVALID_ARG, "table_stride must lie in [0, 2^31]");
  int shift = 4;
  while ((1 << shift) < c->page_size) ++shift;
  *out = PagedCache{{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v)},
                    {static_cast<uint8_t*>(c->k_meta), static_cast<uint8_t*>(c->v_meta)},
                    {c->k_stride, c->v_stride},
                    {c->k_meta_stride, c->v_meta_stride},
                    c->page_table,
                    c->table_stride,
                    c->num_pages,
                    c->max_pages,
                    shift,
                    c->hkv,
                    c->d,
                    static_cast<int>(row)};
  return TE_OK;
}

// What append and gather check alike; sets *status to what the lengths say.
static int begin(const int32_t* cu, const int32_t* cu_pad, const int32_t* past, int batch, int total, int32_t* status,
                 cudaStream_t st) {
  if (!cu || !cu_pad || !past) return api_fail(TE_ERR_INVALID_ARG, "cu_seqlens and positions must not be NULL");
  if (batch < 1) return api_fail(TE_ERR_INVALID_ARG, "batch must be >= 1");
  if (total < 0 || total > INT32_MAX - 256) return api_fail(TE_ERR_INVALID_ARG, "rows must lie in [0, 2^31 - 256)");
  for (const void* x : {static_cast<const void*>(cu), static_cast<const void*>(cu_pad), static_cast<const void*>(past),
                        static_cast<const void*>(status)})
    if (!aligned(x, 4)) return api_fail(TE_ERR_INVALID_ARG, "int32 arrays need their natural alignment");
  if (status) {
    paged_status_kernel<<<1, batch < 1024 ? (batch + 31) / 32 * 32 : 1024, 0, st>>>(cu, cu_pad, past, batch, total, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return api_cuda_fail(e, "status");
  }
  return TE_OK;
}

}  // namespace teattn

using namespace teattn;

extern "C" {

int te_attn_paged_append(const te_attn_paged_cache* cache, const void* q, const void* k, const void* v, void* q_out,
                         const double* inv_freq, int n_freq, const int32_t* cu_seqlens,
                         const int32_t* cu_seqlens_padded, const int32_t* past, int batch, int total, int hq,
                         int64_t q_stride_t, int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h,
                         int64_t v_stride_t, int64_t v_stride_h, int interleaved, float mscale, int32_t* status,
                         void* stream) {
  AppendParams p{};
  int rc = api_paged_cache(cache, &p.cache);
  if (rc != TE_OK) return rc;
  if (hq < 0) return api_fail(TE_ERR_INVALID_ARG, "hq must be >= 0");
  if (hq > 4096) return api_fail(TE_ERR_UNSUPPORTED, "at most 4096 heads");
  if (n_freq < 0 || n_freq > cache->d / 2) return api_fail(TE_ERR_INVALID_ARG, "n_freq must lie in [0, d / 2]");
  if (n_freq > 0 && !inv_freq) return api_fail(TE_ERR_INVALID_ARG, "inv_freq must not be NULL");
  if (!std::isfinite(mscale)) return api_fail(TE_ERR_INVALID_ARG, "mscale must be finite");
  if (total > 0 && (!k || !v || (hq > 0 && (!q || !q_out))))
    return api_fail(TE_ERR_INVALID_ARG, "k, v and, with hq > 0, q and q_out must not be NULL");
  for (const void* x : {q, k, v, static_cast<const void*>(q_out)})
    if (!aligned(x, 2)) return api_fail(TE_ERR_INVALID_ARG, "tensors must be 2-byte aligned");
  if (!aligned(inv_freq, 8)) return api_fail(TE_ERR_INVALID_ARG, "inv_freq needs its natural alignment");
  for (int64_t s : {q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h})
    if (s < 0 || s > (int64_t(1) << 31)) return api_fail(TE_ERR_INVALID_ARG, "strides must lie in [0, 2^31]");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = begin(cu_seqlens, cu_seqlens_padded, past, batch, total, status, st);
  if (rc != TE_OK) return rc;
  if (total == 0) return api_ok();
  p.x[0] = q;
  p.x[1] = k;
  p.x[2] = v;
  const int64_t strides[] = {q_stride_t, k_stride_t, v_stride_t, q_stride_h, k_stride_h, v_stride_h};
  for (int i = 0; i < 3; ++i) {
    p.stride_t[i] = strides[i];
    p.stride_h[i] = strides[3 + i];
  }
  p.q_out = q_out;
  p.heads[0] = hq;
  p.heads[1] = p.heads[2] = cache->hkv;
  p.inv_freq = inv_freq;
  p.cu = cu_seqlens;
  p.cu_pad = cu_seqlens_padded;
  p.past = past;
  p.status = status;
  p.batch = batch;
  p.total = total;
  p.d = cache->d;
  p.rot = 2 * n_freq;
  p.mscale = mscale;
  const bool bf16 = cache->dtype == TE_DTYPE_BF16;
  const cudaError_t e = cache->k_meta ? launch_append<true>(p, !interleaved, bf16, st) : launch_append<false>(p, !interleaved, bf16, st);
  return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "paged append");
}

int te_attn_paged_gather(const te_attn_paged_cache* cache, void* k, void* v, const int32_t* cu_seqlens,
                         const int32_t* cu_seqlens_padded, const int32_t* start, int batch, int total,
                         int32_t* status, void* stream) {
  GatherParams p{};
  int rc = api_paged_cache(cache, &p.cache);
  if (rc != TE_OK) return rc;
  if (total > 0 && (!k || !v)) return api_fail(TE_ERR_INVALID_ARG, "k and v must not be NULL");
  if (!aligned(k, 16) || !aligned(v, 16)) return api_fail(TE_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = begin(cu_seqlens, cu_seqlens_padded, start, batch, total, status, st);
  if (rc != TE_OK) return rc;
  if (total == 0) return api_ok();
  p.y[0] = k;
  p.y[1] = v;
  p.cu = cu_seqlens;
  p.cu_pad = cu_seqlens_padded;
  p.start = start;
  p.status = status;
  p.batch = batch;
  p.total = total;
  // enough blocks for the SMs first, then up to eight rows a block
  p.tokens = total >= 8 * 4 * kAppendSMs ? 8 : total >= 4 * kAppendSMs ? 2 : 1;
  auto inverse = [](int n) { return static_cast<uint32_t>(((1ull << 32) + n - 1) / n); };
  p.words_inv = inverse(cache->d / 8);
  p.heads_inv = inverse(cache->hkv);
  const int blocks = (total + p.tokens - 1) / p.tokens;
  const bool bf16 = cache->dtype == TE_DTYPE_BF16;
  if (!cache->k_meta) paged_gather_kernel<true, false><<<blocks, kGatherThreads, 0, st>>>(p);
  else if (bf16) paged_gather_kernel<true, true><<<blocks, kGatherThreads, 0, st>>>(p);
  else paged_gather_kernel<false, true><<<blocks, kGatherThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "paged gather");
}

}  // extern "C"
