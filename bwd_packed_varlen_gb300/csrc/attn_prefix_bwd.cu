// Shared-prefix attention, backward: the lists of row and key tiles, what the tiles need
// of every row (and the rows no tile writes), and the sum of the prefix gradients' parts.
// The dQ and dK/dV kernels between them are the packed problem's, with the prefix as
// further key tiles.
#include <cuda_runtime.h>

#include "attn_prefix.cuh"
#include "pdl.cuh"
#include "sm103_ptx.cuh"

namespace teattn {

// ---------------------------------------------------------------------------
// Lists of (sequence, row tile) and (sequence, key tile) in natural order. With a prefix
// every row tile costs about the same, and the prefix's own dK/dV items, the longest, go
// first by themselves, so the packed problem's sort by cost would only delay the start.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) prefix_bwd_schedule_kernel(const __grid_constant__ PrefixBwd p, int* pref_q) {
  pdl_trigger();
  __shared__ int buf[3][32];
  __shared__ int bad;
  __shared__ unsigned long long tokens[2];  // of queries and of own keys
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    bad = p.prefix_len && (*p.prefix_len < 0 || *p.prefix_len > p.prefix_rows) ? 1 : 0;
    tokens[0] = tokens[1] = 0;
  }
  const bool prefix = prefix_keys(p) > 0;
  __syncthreads();
  int n_q = 0, n_k = 0;
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + threadIdx.x;
    int cq = 0, ck = 0;
    unsigned long long both = 0;  // tokens of this sequence: queries, and keys in the upper half
    if (b < p.batch) {
      const SeqInfo s = load_seq(p, b);
      if (!s.ok) bad = 1;
      both = static_cast<unsigned long long>(s.len_k) << 32 | static_cast<uint32_t>(s.len_q);
      if (s.len_q > 0) {
        if (prefix || s.len_k > 0) cq = ((s.len_q << p.pack_shift) + kBlockM - 1) / kBlockM;
        ck = (seen_keys(s, p.causal != 0) + kBlockN - 1) / kBlockN;
      }
    }
    unsigned long long q = both & 0xffffffffull, k = both >> 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      q += __shfl_xor_sync(0xffffffffu, q, o);
      k += __shfl_xor_sync(0xffffffffu, k, o);
    }
    if (lane == 0) {
      atomicAdd(&tokens[0], q);
      atomicAdd(&tokens[1], k);
    }
    const Scan3 at = block_scan3(cq, ck, 0, buf);
    if (b < p.batch) pref_q[b] = n_q + at.x;
    // a warp writes its 32 sequences' tiles together
#pragma unroll 1
    for (uint32_t some = __ballot_sync(0xffffffffu, cq > 0 || ck > 0); some; some &= some - 1) {
      const int l = __ffs(some) - 1;
      const int seq = __shfl_sync(0xffffffffu, b, l);
      const int q0 = n_q + __shfl_sync(0xffffffffu, at.x, l), nq = __shfl_sync(0xffffffffu, cq, l);
      const int k0 = n_k + __shfl_sync(0xffffffffu, at.y, l), nk = __shfl_sync(0xffffffffu, ck, l);
#pragma unroll 1
      for (int t = lane; t < nq; t += 32)
        if (static_cast<uint32_t>(q0 + t) < static_cast<uint32_t>(p.pair_cap_q)) p.q_pairs[q0 + t] = make_int2(seq, t);
#pragma unroll 1
      for (int t = lane; t < nk; t += 32)
        if (static_cast<uint32_t>(k0 + t) < static_cast<uint32_t>(p.pair_cap_k)) p.k_pairs[k0 + t] = make_int2(seq, t);
    }
    n_q += at.tx;
    n_k += at.ty;
  }
  if (threadIdx.x == 0) {
    // overlapping sequences, which have more tokens than there are rows, can have more tiles
    // than the lists hold: none is computed (the scans' barriers order the sums before this)
    const bool over = tokens[0] > static_cast<unsigned long long>(p.total_q) ||
                      tokens[1] > static_cast<unsigned long long>(p.total_kv) || n_q > p.pair_cap_q || n_k > p.pair_cap_k;
    pref_q[p.batch] = over ? -1 : n_q;
    p.header[kHdrStatus] = bad || over ? kStatusBadSeqlens : 0;
    p.header[kHdrNumQPairs] = over ? 0 : n_q;
    p.header[kHdrNumKPairs] = over ? 0 : n_k;
    p.header[kHdrNextDkdv] = 0;
    p.header[kHdrNextDq] = 0;
  }
}

cudaError_t launch_prefix_bwd_schedule(const PrefixBwd& p, int* pref_q, cudaStream_t st) {
  const int threads = p.batch >= 1024 ? 1024 : (p.batch + 31) / 32 * 32;
  prefix_bwd_schedule_kernel<<<1, threads, 0, st>>>(p, pref_q);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Every query row: -lse log2(e) and -D = -rowsum(dO O) for the tiles that read it, both by
// (sequence, row tile) and by tensor row (rows that are no token: -infinity, which makes
// their P zero); dq of rows no tile writes. Every own key row that no query sees: zeros.
// One warp per row, 16-byte loads. Where d / 8 divides 32 neighbouring lanes read
// neighbouring pieces, four groups in flight, and memory bounds it; at other head dims (48,
// 80, 96, ...) a lane goes through a head by itself, which is slower.
// ---------------------------------------------------------------------------
template <bool kBF16>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<kBF16>(x[i]), v = unpack2<kBF16>(y[i]);
    s = fmaf(u.x, v.x, s);
    s = fmaf(u.y, v.y, s);
  }
  return s;
}

__device__ __forceinline__ void zero_rows(void* base, size_t row, int bytes) {
  uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(base) + row * bytes);
  for (int i = threadIdx.x & 31; i < bytes / 16; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
}

constexpr int kPrepRows = 8, kPrepHeads = 128;  // rows of a block at a time, heads of a pass

template <bool kBF16>
__global__ void __launch_bounds__(256) prefix_prep_kernel(const __grid_constant__ PrefixBwd p) {
  __shared__ int s_q[kCachedOffsets], s_k[kCachedOffsets];
  __shared__ float s_lse[kPrepHeads][kPrepRows + 1], s_delta[kPrepHeads][kPrepRows + 1];
  __shared__ long long s_tile[kPrepRows];  // index of a row's head 0 in the tiles; -1: in none
  const int* q_pad = cache_offsets(p.cu_q_pad, p.batch, s_q);
  const int* k_pad = cache_offsets(p.cu_kv_pad, p.batch, s_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sh = p.pack_shift;
  const bool causal = p.causal != 0, prefix = prefix_keys(p) > 0;
  constexpr float kLog2e = 1.4426950408889634f;
  const int cpr = p.d / 8;  // 16-byte chunks per head
  pdl_trigger();
  // The first rows' sums are formed while the scheduler runs; what comes of them needs its
  // result (small training steps 2 us shorter).
  bool waited = false, none = false;
  // blocks of rows, up to the linear rows past the tensor's last one
  const long long rows_end = p.rows_lin >> sh;
  for (long long r0 = static_cast<long long>(blockIdx.x) * kPrepRows; r0 < rows_end;
       r0 += static_cast<long long>(gridDim.x) * kPrepRows) {
    const long long r = r0 + warp;
    const size_t row = static_cast<size_t>(r);
    int i = 0;
    const int b = r >= p.total_q ? -1 : locate_row(p, q_pad, static_cast<int>(r), &i);
    SeqInfo s{};
    if (b >= 0) s = load_seq(p, b);
    const bool real = b >= 0 && i < s.len_q;
    const bool read = real && (prefix || s.len_k > 0);  // some tile reads this row
    for (int h0 = 0; h0 < p.hq; h0 += kPrepHeads) {
      const int nh = min(kPrepHeads, p.hq - h0);
      for (int h = lane; h < nh; h += 32) {
        s_lse[h][warp] = read ? -(p.lse_in[row * p.hq + h0 + h] * kLog2e) : -INFINITY;
        s_delta[h][warp] = 0.f;
      }
      __syncwarp();
      if (read) {
        const size_t at = (row * p.hq + h0) * p.d;
        const uint4* o = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.out_in) + at);
        const uint4* g = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dout) + at);
        const int chunks = nh * cpr;
        if (32 % cpr == 0) {
          // the lanes of a head are neighbours and add up by shuffles
          for (int c0 = 0; c0 < chunks; c0 += 128) {
            uint4 oa[4], ga[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int c = c0 + 32 * u + lane;
              if (c < chunks) {
                oa[u] = o[c];
                ga[u] = g[c];
              }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int c = c0 + 32 * u + lane;
              float v = c < chunks ? dot8<kBF16>(oa[u], ga[u]) : 0.f;
              for (int w = cpr >> 1; w > 0; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
              if (c < chunks && (c % cpr) == 0) s_delta[c / cpr][warp] = -v;
            }
          }
        } else {
          for (int h = lane; h < nh; h += 32) {
            float v = 0.f;
            for (int c = 0; c < cpr; ++c) v += dot8<kBF16>(o[h * cpr + c], g[h * cpr + c]);
            s_delta[h][warp] = -v;
          }
        }
      }
      if (!waited) {
        pdl_wait();  // pref_q and the header
        waited = true;
        // more tiles than the lists hold (overlapping sequences): no row is a token
        none = p.header[kHdrNumQPairs] != p.pref_q[p.batch];
      }
      if (h0 == 0) {
        // rows that see no key: their tiles leave dq to this kernel
        if (r < p.total_q && (none || !real || (!prefix && row_keys(s, i, causal) == 0)))
          zero_rows(p.dq, row, p.hq * p.d * 2);
        if (lane == 0) s_tile[warp] = read && !none ? static_cast<long long>(packed_index(p, b, i << sh, 0)) : -1;
      }
      __syncthreads();
      // The rows' values leave in runs: of a virtual head, eight rows times its packed heads
      // lie side by side by tensor row, and a row's packed heads by tile.
      for (int z = threadIdx.x; z < nh * kPrepRows; z += 256) {
        const int w = (z >> sh) % kPrepRows, vh = (z >> sh) / kPrepRows, j = z & ((1 << sh) - 1);
        const int h = (vh << sh) + j;
        const float lse = none ? -INFINITY : s_lse[h][w], delta = none ? 0.f : s_delta[h][w];
        const size_t vhead = static_cast<size_t>((h0 >> sh) + vh);
        if (r0 + w < rows_end) {
          const size_t lin = vhead * p.rows_lin + (static_cast<size_t>(r0 + w) << sh) + j;
          p.lse_lin[lin] = lse;
          p.delta_lin[lin] = delta;
        }
        if (s_tile[w] >= 0) {
          const size_t t = static_cast<size_t>(s_tile[w]) + vhead * kBlockM + j;
          if (bounds_ok(t < static_cast<size_t>(p.pair_cap_q) * p.vheads * kBlockM, p.header + kHdrStatus)) {
            p.lse_t[t] = lse;
            p.delta_t[t] = delta;
          }
        }
      }
      __syncthreads();
    }
  }
  if (!waited) {
    pdl_wait();
    none = p.header[kHdrNumQPairs] != p.pref_q[p.batch];
  }
  const long long warps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  for (long long r = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; r < p.total_kv; r += warps) {
    int j = 0;
    const int b = none ? -1 : locate_row(p, k_pad, static_cast<int>(r), &j);
    SeqInfo s{};
    if (b >= 0) s = load_seq(p, b);
    if (b >= 0 && j < seen_keys(s, causal)) continue;  // its tile writes it
    zero_rows(p.dk, static_cast<size_t>(r), p.hkv * p.d * 2);
    zero_rows(p.dv, static_cast<size_t>(r), p.hkv * p.d * 2);
  }
}

cudaError_t launch_prefix_prep(const PrefixBwd& p, bool bf16, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.total_q) > p.total_kv ? p.total_q : p.total_kv;
  const long long want = (rows + 7) / 8;
  if (want == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(want < num_sms * 8 ? want : num_sms * 8);
  return launch_dependent(bf16 ? prefix_prep_kernel<true> : prefix_prep_kernel<false>, grid, 256, 0, st, p);
}

// dK_prefix = scale sum_s part_dk[s], dV_prefix = sum_s part_dv[s] in the order of s, in
// fp32, rounded once; rows that no query sees (behind the real length, or without any
// query) are zeros. With one part the dK/dV kernel wrote the seen rows itself. Memory-
// bound: every fp32 part is read once, 32 bytes per thread and part.
template <bool kBF16>
__global__ void __launch_bounds__(256) prefix_sum_kernel(const __grid_constant__ PrefixBwd p) {
  pdl_wait();
  const int seen = p.total_q > 0 ? prefix_keys(p) : 0;
  const size_t row_elems = static_cast<size_t>(p.hkv) * p.d;
  const size_t n = static_cast<size_t>(p.prefix_rows) * row_elems;
  const size_t first = p.splits > 1 ? 0 : static_cast<size_t>(seen) * row_elems;
  const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x * 8;
  for (size_t i = first + (static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; i < n; i += step) {
    const bool live = i < static_cast<size_t>(seen) * row_elems;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float a[8] = {};
      if (live) {
        const float* src = (w == 0 ? p.part_dk : p.part_dv) + i;
        for (int s = 0; s < p.splits; ++s) {
          const float4 x = *reinterpret_cast<const float4*>(src + s * n), y = *reinterpret_cast<const float4*>(src + s * n + 4);
          a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
          a[4] += y.x; a[5] += y.y; a[6] += y.z; a[7] += y.w;
        }
      }
      const float f = w == 0 ? p.scale : 1.f;
      uint4 v;
      v.x = pack2<kBF16>(a[0] * f, a[1] * f);
      v.y = pack2<kBF16>(a[2] * f, a[3] * f);
      v.z = pack2<kBF16>(a[4] * f, a[5] * f);
      v.w = pack2<kBF16>(a[6] * f, a[7] * f);
      *reinterpret_cast<uint4*>(static_cast<char*>(w == 0 ? p.dkp : p.dvp) + i * 2) = v;
    }
  }
}

cudaError_t launch_prefix_sum(const PrefixBwd& p, bool bf16, int num_sms, cudaStream_t st) {
  const long long blocks = (static_cast<long long>(p.prefix_rows) * p.hkv * p.d / 8 + 255) / 256;
  if (blocks == 0) return cudaSuccess;
  const int grid = static_cast<int>(blocks < num_sms * 8 ? blocks : num_sms * 8);
  return launch_dependent(bf16 ? prefix_sum_kernel<true> : prefix_sum_kernel<false>, static_cast<unsigned>(grid), 256,
                          0, st, p);
}

}  // namespace teattn
