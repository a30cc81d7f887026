// Attention over a paged cache: joins what the slices left of segments that several of them
// share, writes zeros to rows that hold no token, and collects the call's status.
//
// A block of four warps per row of out, per token or, beside long pieces, per head of a sequence (JoinGrid);
// blocks ahead of them look for rows that are no token, or join the other kernel's segments. Of a row's
// pieces O = sum 2^(m_k - M) O_k / L with
// M = max m_k and L = sum 2^(m_k - M) l_k, in fp32, every fourth piece in order by a warp and the
// four warps' sums in order, rounded once. Latency-bound: a decoding step's rows have a few pieces
// (3-5 us of the call). Rows of the other kernel are joined by a thread each, column by column.
#include <cuda_runtime.h>

#include <cmath>

#include "attn_paged.cuh"
#include "pdl.cuh"
#include "sm103_ptx.cuh"
#include "tmap.h"

namespace teattn {

constexpr int kJoinThreads = 128;
constexpr int kJoinBlocks = 16 * kPagedSMs;

__device__ __forceinline__ float ex2j(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Blocks that share the rows of a segment of the kernel of many rows: they lie idle where a slice ends
// with its segment, but split the columns of one with many pieces. One sequence of 512 rows behind 2000
// keys, and four pieces of prompts: 8 blocks 50 and 207.8 us, 16 43 and 209.1, 32 41 and 212.2.
constexpr int kWideJoin = 16;

// A warp adds up the pieces w, w + step, ... <= w1 of row r of the segment that begins at `first`, eight
// columns a lane: maximum, sum and output. Piece w is in slot 1 of the slice that begins the segment,
// in slot 0 of the others.
__device__ __forceinline__ void join_pieces(const PagedParams& p, const PagedParts& parts, int rows, int r, long long first,
                                            long long per, int w, int w1, int step, float& m, float& l, float (&acc)[8]) {
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int x = 0; x < 8; ++x) acc[x] = 0.f;
  for (; w <= w1; w += step) {
    const long long at = (2ll * w + (w * per <= first ? 1 : 0)) * rows + r;
    const float2 ml = parts.ml[at];
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
    if (lane < p.d / 8) {
      a = *reinterpret_cast<const float4*>(parts.o + at * p.d + lane * 8);
      c = *reinterpret_cast<const float4*>(parts.o + at * p.d + lane * 8 + 4);
    }
    const float top = fmaxf(m, ml.x);
    // (a piece without a key has left a sum of 0, or a NaN that it saw)
    const float x = m == -INFINITY ? (l == 0.f ? 0.f : NAN) : ex2j(m - top);
    const float y = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : NAN) : ex2j(ml.x - top);
    const float f[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = acc[e] * x + f[e] * y;
    l = l * x + ml.y * y;
    m = top;
  }
}

// The segment that slice `w` goes on with, if it is the first slice to do so: a thread a row, an
// eighth of the columns a block (its pieces lie column by column).
template <bool kBF16>
__device__ void join_wide(const PagedParams& p, const PagedParts& parts, int w, int part) {
  const long long total = parts.pref[p.batch], per = slice_units(total, parts.slices, parts.least), at = w * per;
  if (at >= total) return;
  constexpr PagedCut cut{kWideRows, kWideKeys, true};
  const Stretch t = stretch_at(p, cut, parts.pref, at, total);
  const long long first = at - t.u0;
  if (t.u0 == 0 || first < at - per) return;  // begins it, or an earlier slice went on with it
  const int w1 = static_cast<int>((first + t.run.n - 1) / per);
  const int row0 = t.tile * kWideRows, rows = min(kWideRows, t.s.n * p.group - row0);
  const int r = (part & 1) * kJoinThreads + threadIdx.x;
  if (r >= rows) return;
  // piece k is in slot 1 of the slice that begins the segment, in slot 0 of the others
  auto slot = [&](int k) { return 2ll * k + (k == w - 1 ? 1 : 0); };
  float M = -INFINITY, L = 0.f;
  for (int k = w - 1; k <= w1; ++k) M = fmaxf(M, parts.ml[slot(k) * kWideRows + r].x);
  // (a piece without a key has left a sum of 0, or a NaN that it saw)
  auto weight = [&](float2 ml) { return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : NAN) : ex2j(ml.x - M); };
  for (int k = w - 1; k <= w1; ++k) {
    const float2 ml = parts.ml[slot(k) * kWideRows + r];
    L += weight(ml) * ml.y;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int i = (row0 + r) / p.group, j = row0 + r - i * p.group;
  const long long row = static_cast<long long>(t.s.off + i) * p.hq + t.head * p.group + j;
  for (int c = part >> 1; c < p.d / 8; c += kWideJoin / 2) {
    float acc[8] = {};
    for (int k = w - 1; k <= w1; ++k) {
      const float f = weight(parts.ml[slot(k) * kWideRows + r]);
      const float* o = parts.o + (slot(k) * p.d + c * 8) * kWideRows + r;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(f, o[e * kWideRows], acc[e]);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.d + c * 8) =
        make_uint4(pack2<kBF16>(acc[0] * inv, acc[1] * inv), pack2<kBF16>(acc[2] * inv, acc[3] * inv),
                   pack2<kBF16>(acc[4] * inv, acc[5] * inv), pack2<kBF16>(acc[6] * inv, acc[7] * inv));
  }
  if (part < 2) p.lse[row] = M * 0.69314718055994531f + logf(L);
}

// How blocks share the rows of the kernel of few rows. Without the other kernel: `heads` heads of a
// token each. With it most tokens may be the other's, and blocks that find nothing to do take a
// nanosecond each: a block `heads` heads of a sequence (parts of its queries), behind `scans` blocks
// that look for rows that are no token. 64 single queries beside four prompts of 512: 19 us, a call 211
// (a block a token with all its heads: a call 271); 19 prompts of 64: 7 us, a block a row 34.
struct JoinGrid {
  int heads, scans, parts;
};
constexpr int kScanTokens = 32;

template <bool kBF16>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ PagedCut few, const __grid_constant__ PagedParts few_parts,
                      const __grid_constant__ PagedParts wide_parts, JoinGrid grid) {
  __shared__ float2 s_ml[4];
  __shared__ float s_o[4][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wide_blocks = wide_parts.slices * kWideJoin;  // ahead of the rows
  const int at_row = blockIdx.x - 1 - wide_blocks;
  PagedSeq s{0, 0, 0, true};
  int b = -1, i0 = 0, i1 = 0, step = 1, hq0 = 0, hq1 = 0;  // queries i0, i0 + step, ... of sequence b; their heads
  auto sequence_of = [&](int tok) {  // by a whole warp
    b = sequence_at(p.cu_q_pad, p.batch, tok);
    if (b >= 0) s = load_paged_seq(p, b);
    return b >= 0 && s.ok && tok - s.off < s.n;
  };
  auto no_token = [&](int tok, int h0, int h1, int at, int threads) {
    const long long row = static_cast<long long>(tok) * p.hq + h0;
    for (int c = at * 8; c < p.d * (h1 - h0); c += threads * 8)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.d + c) = make_uint4(0, 0, 0, 0);
    for (int h = at; h < h1 - h0; h += threads) p.lse[row + h] = 0.f;
  };
  if (at_row < 0) {
  } else if (grid.parts == 0) {  // a token, or a head of it
    const int per_token = p.hq / grid.heads, tok = at_row / per_token;
    hq0 = (at_row - tok * per_token) * grid.heads;
    hq1 = hq0 + grid.heads;
    if (sequence_of(tok)) {
      i0 = tok - s.off;
      i1 = i0 + 1;
    } else {
      pdl_wait();
      no_token(tok, hq0, hq1, threadIdx.x, kJoinThreads);
      return;
    }
  } else if (at_row < grid.scans) {  // rows that are no token, of kScanTokens rows
    pdl_wait();
    for (int k = warp; k < kScanTokens; k += kJoinThreads / 32) {
      const int tok = at_row * kScanTokens + k;
      if (tok < p.total_q && !sequence_of(tok)) no_token(tok, 0, p.hq, lane, 32);
    }
    return;
  } else {  // heads of a sequence, or of every grid.parts-th query
    const int n = at_row - grid.scans, seg = n / grid.parts, per_seq = p.hq / grid.heads;
    b = seg / per_seq;
    hq0 = (seg - b * per_seq) * grid.heads;
    hq1 = hq0 + grid.heads;
    i0 = n - seg * grid.parts;
    step = grid.parts;
    s = load_paged_seq(p, b);
    i1 = s.n;
  }
  pdl_wait();
  if (blockIdx.x == 0) {  // the call's status
    int bits = 0;
    for (int k = threadIdx.x; k < few_parts.slices + wide_parts.slices; k += kJoinThreads) bits |= p.warp_status[k];
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) s_ml[warp].x = __int_as_float(bits);
    __syncthreads();
    if (threadIdx.x == 0)
      p.header[kHdrStatus] = __float_as_int(s_ml[0].x) | __float_as_int(s_ml[1].x) | __float_as_int(s_ml[2].x) | __float_as_int(s_ml[3].x);
    return;
  }
  if (at_row < 0) {
    join_wide<kBF16>(p, wide_parts, (blockIdx.x - 1) / kWideJoin, (blockIdx.x - 1) % kWideJoin);
    return;
  }
  if (!few.takes(p, s)) return;  // the other kernel's
#pragma unroll 1
  for (int n = 0; i0 + n / (hq1 - hq0) * step < i1; ++n) {
    const int i = i0 + n / (hq1 - hq0) * step, hq = hq0 + n % (hq1 - hq0);
    const long long row = static_cast<long long>(s.off + i) * p.hq + hq;
    uint16_t* out = static_cast<uint16_t*>(p.out) + row * p.d;
    const PagedParts& parts = few_parts;
    const int h = hq / p.group;
    const long long rr = static_cast<long long>(i) * p.group + hq - h * p.group;
    const int tile = static_cast<int>(rr / few.rows), r = static_cast<int>(rr - static_cast<long long>(tile) * few.rows);
    const int units = few.run(p, s, tile).n;
    const long long per = slice_units(parts.pref[p.batch], parts.slices, parts.least);
    const long long first = parts.pref[b] + few.before(p, s, tile) + static_cast<long long>(h) * units;
    const int w0 = static_cast<int>(first / per), w1 = static_cast<int>((first + units - 1) / per);
    if (w0 == w1) continue;  // written whole
    float m, l, acc[8];
    const int cols = p.d / 8;  // eight columns a lane
    join_pieces(p, parts, few.rows, r, first, per, w0 + warp, w1, 4, m, l, acc);
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    if (lane < cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s_o[warp][lane * 8 + e] = acc[e];
    }
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, s_ml[w].x);
    float f[4], sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      f[w] = s_ml[w].x == -INFINITY ? (s_ml[w].y == 0.f ? 0.f : NAN) : ex2j(s_ml[w].x - top);
      sum += s_ml[w].y * f[w];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int c = threadIdx.x * 2; c < p.d; c += kJoinThreads * 2) {
      float a = 0.f, d = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        a += s_o[w][c] * f[w];
        d += s_o[w][c + 1] * f[w];
      }
      *reinterpret_cast<uint32_t*>(out + c) = pack2<kBF16>(a * inv, d * inv);
    }
    if (threadIdx.x == 0) p.lse[row] = top * 0.69314718055994531f + logf(sum);
    __syncthreads();  // (the sums in shared memory are read)
  }
}

bool make_tmap_pages(CUtensorMap* map, const PagedCache& c, int kv, bool bf16, int slots) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t page = 1ull << c.shift, row = 2ull * c.d;
  cuuint64_t gdim[4] = {static_cast<cuuint64_t>(c.d), page, static_cast<cuuint64_t>(c.hkv), static_cast<cuuint64_t>(c.num_pages)};
  cuuint64_t gstride[3] = {row, row * page, static_cast<cuuint64_t>(c.stride[kv])};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(slots), 1, 1}, estr[4] = {1, 1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, c.data[kv], gdim, gstride, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_paged_join(const PagedParams& p, const PagedCut& cut, const PagedParts& parts, const PagedParts& wide, bool bf16,
                              cudaStream_t st) {
  // A block a row (a head of a sequence) while that fills the GPU a few times over, then one a token (a sequence).
  JoinGrid g{1, 0, 0};
  long long blocks = static_cast<long long>(wide.slices > 0 ? p.batch : p.total_q) * p.hq;
  if (blocks > 16 * 16 * kPagedSMs) {
    g.heads = p.hq;
    blocks /= p.hq;
  }
  if (wide.slices > 0) {
    const long long most = p.wide_rows / p.group, want = kJoinBlocks / blocks;  // queries that a sequence may have here
    g.parts = static_cast<int>(want < 1 || most < 1 ? 1 : want < most ? want : most);
    g.scans = (p.total_q + kScanTokens - 1) / kScanTokens;
    blocks = g.scans + blocks * g.parts;
  }
  return launch_dependent(bf16 ? paged_join_kernel<true> : paged_join_kernel<false>,
                          dim3(static_cast<unsigned>(blocks + wide.slices * kWideJoin + 1)), dim3(kJoinThreads), 0, st, p, cut, parts, wide, g);
}

}  // namespace teattn
