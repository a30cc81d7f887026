// Shared-prefix attention: launch parameters and work lists of its kernels.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "common.cuh"

namespace teattn {

// A packed problem (AttnParams) whose queries also see every key of a prefix that all
// sequences share: kp, vp [prefix_rows, hkv, d], the first prefix_keys() rows real.
struct PrefixParams : AttnParams {
  const void* kp;
  const void* vp;
  void* dkp;
  void* dvp;
  const int* prefix_len;  // may be null: all prefix_rows
  int prefix_rows;
  // forward work lists (workspace), written by the call's scheduler
  int4* seqs;        // per sequence, x: first compact token (-1: not short), y: first partial
                     // row of its own keys' parts, z: their number (-1: the main kernel wrote
                     // the rows), w: first long row tile
  int* short_tok;    // compact token -> packed row
  int4* longs;       // per long row tile: first partial row (-1: written directly), parts, rows
  int4* entries;     // three int4 per (group, chunk), for every kv head: PrefixEntry
  float2* part_ml;   // partial rows: running maximum (log2 domain) and sum
  float* part_o;     // partial rows: unnormalised output, d columns
  int parts_target;  // chunks that all groups of one kv head together are cut into, about
  int cap_longs, cap_entries, cap_rows;
};

struct Scan3 {
  int x, y, z;     // exclusive sums before this thread
  int tx, ty, tz;  // totals
};

// Exclusive scan of three counters over the block (two barriers). `buf`: 3 x 32 ints.
__device__ __forceinline__ Scan3 block_scan3(int x, int y, int z, int (*buf)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int ix = x, iy = y, iz = z;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    const int uz = __shfl_up_sync(0xffffffffu, iz, o);
    if (lane >= o) {
      ix += ux;
      iy += uy;
      iz += uz;
    }
  }
  if (lane == 31) {
    buf[0][warp] = ix;
    buf[1][warp] = iy;
    buf[2][warp] = iz;
  }
  __syncthreads();
  // every warp sums the warps' totals itself: lane w holds warp w's
  const int wx = lane < nw ? buf[0][lane] : 0, wy = lane < nw ? buf[1][lane] : 0, wz = lane < nw ? buf[2][lane] : 0;
  __syncthreads();
  Scan3 r;
  r.tx = __reduce_add_sync(0xffffffffu, wx);
  r.ty = __reduce_add_sync(0xffffffffu, wy);
  r.tz = __reduce_add_sync(0xffffffffu, wz);
  r.x = __reduce_add_sync(0xffffffffu, lane < warp ? wx : 0) + ix - x;
  r.y = __reduce_add_sync(0xffffffffu, lane < warp ? wy : 0) + iy - y;
  r.z = __reduce_add_sync(0xffffffffu, lane < warp ? wz : 0) + iz - z;
  return r;
}

// locate_row() among offsets copied to shared memory, where they fit: each step of the
// search would otherwise be a trip to L2. Every thread of the block calls cache_offsets().
constexpr int kCachedOffsets = 2048;
__device__ __forceinline__ const int* cache_offsets(const int* cu_pad, int batch, int* shared) {
  if (batch >= kCachedOffsets) return cu_pad;
#pragma unroll 1
  for (int k = threadIdx.x; k <= batch; k += blockDim.x) shared[k] = cu_pad[k];
  __syncthreads();
  return shared;
}

// Real prefix keys; a length outside [0, prefix_rows] counts as 0 (and is reported).
__device__ __forceinline__ int prefix_keys(const PrefixParams& p) {
  if (!p.prefix_len) return p.prefix_rows;
  const int n = *p.prefix_len;
  return n >= 0 && n <= p.prefix_rows ? n : 0;
}

// ---------------------------------------------------------------------------
// Forward work. The rows of a kv head g are its group's queries, token-major: packed row
// r of a token list is (token r / G, head g G + r % G). A sequence of at most kShortRows
// such rows is "short": its rows are packed with those of all other short sequences
// against the prefix (row tiles of the compact token list) and stand alone against its own
// keys. A longer sequence has row tiles of its own, each over the prefix and then its own
// keys. A row tile's key tiles are cut into chunks; rows whose only chunk is the whole are
// written directly, the others leave partial results that the join kernel merges.
// ---------------------------------------------------------------------------
constexpr int kShortRows = 128;
constexpr int kSMs = 152;             // of the GPU that work is cut for
constexpr int kPartsTarget = 2 * kSMs;  // chunks over all kv heads, about: two per SM

__host__ __device__ constexpr int prefix_row_tile(int d) { return d <= 128 ? 256 : 128; }
__host__ __device__ constexpr int prefix_key_tile(int d) { return d <= 128 ? 128 : 64; }

// One chunk of a row tile's keys, complete: nothing else is read to start on it.
struct PrefixEntry {
  int row0, rows;    // packed rows [row0, row0 + rows) of the list
  int seq;           // -1: the compact tokens
  int t0, t1, np;    // key tiles [t0, t1), of which tiles below np are the prefix's
  int slot;          // partial row of (kv head 0, row 0); -1: written directly
  int off_q, off_k, len_k, diag;  // of the sequence (SeqInfo)
};
__device__ __forceinline__ PrefixEntry load_entry(const PrefixParams& p, int e) {
  const int4 a = p.entries[3 * e], b = p.entries[3 * e + 1], c = p.entries[3 * e + 2];
  return PrefixEntry{a.x, a.y, a.z, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
}
__device__ __forceinline__ void store_entry(const PrefixParams& p, int e, const PrefixEntry& v) {
  p.entries[3 * e] = make_int4(v.row0, v.rows, v.seq, 0);
  p.entries[3 * e + 1] = make_int4(v.t0, v.t1, v.np, v.slot);
  p.entries[3 * e + 2] = make_int4(v.off_q, v.off_k, v.len_k, v.diag);
}
// Partial rows before those of chunk c and kv head h, of a row tile's.
__device__ __forceinline__ size_t partial_offset(const PrefixParams& p, int rows, int c, int h) {
  return (static_cast<size_t>(c) * p.hkv + h) * rows;
}

// ---------------------------------------------------------------------------
// Backward: the dQ and dK/dV kernels of the packed problem, with the prefix's keys as
// further key tiles. `pack` = 2^pack_shift heads of a group (the largest power of two that
// divides the group, at most 64) go token by token into one row tile: packed row r of a
// sequence is (token r >> pack_shift, head vh * pack + r % pack) of virtual head vh. A tile
// then covers 128 / pack tokens, so short sequences waste little of it and the heads of a
// group share the key tiles' loads; one TMA box still fetches it.
// The prefix's dK/dV items sweep the rows of the whole tensor, pad rows among them (their
// lse is taken as infinite, so P is 0); with few key tiles the sweep is split, each part
// leaving fp32 partial sums that a reduction adds in order.
// ---------------------------------------------------------------------------
struct PrefixBwd : PrefixParams {
  CUtensorMap tm_kp, tm_vp;
  int pack_shift;
  int vheads;        // hq >> pack_shift
  int vgroup;        // group >> pack_shift
  long long rows_lin;  // total_q << pack_shift, rounded up to a row tile
  float* lse_lin;    // [vheads][rows_lin]: -lse log2(e); -infinity on rows that are no token
  float* delta_lin;  // [vheads][rows_lin]: -rowsum(dO O)
  float* part_dk;    // [splits][prefix_rows][hkv][d] (splits > 1)
  float* part_dv;
  int splits;
};

template <class P>
constexpr bool is_prefix = std::is_same_v<P, PrefixBwd>;

// Compile-time 0 for problems without a prefix: their kernels stay as they are.
template <class P>
__device__ __forceinline__ int pack_shift(const P& p) {
  if constexpr (is_prefix<P>) return p.pack_shift;
  else return 0;
}
template <class P>
__device__ __forceinline__ int virtual_heads(const P& p) {
  if constexpr (is_prefix<P>) return p.vheads;
  else return p.hq;
}
template <class P>
__device__ __forceinline__ int virtual_group(const P& p) {
  if constexpr (is_prefix<P>) return p.vgroup;
  else return p.group;
}
// Prefix keys (0 for problems without a prefix).
template <class P>
__device__ __forceinline__ int prefix_keys_of(const P& p) {
  if constexpr (is_prefix<P>) return prefix_keys(p);
  else return 0;
}
// Own keys that the packed row tile t sees.
template <class P>
__device__ __forceinline__ int tile_keys(const P& p, const SeqInfo& s, int t, bool causal) {
  if constexpr (is_prefix<P>) {
    if (!causal) return s.len_k;
    const int last = min((t + 1) * kBlockM >> p.pack_shift, s.len_q);
    return min(s.len_k, max(0, last + s.diag));
  } else {
    return visible_keys(s, t, causal);
  }
}
// tiled_index() of packed row r and virtual head vh.
template <class P>
__device__ __forceinline__ size_t packed_index(const P& p, int b, int r, int vh) {
  if constexpr (is_prefix<P>) {
    const int pair = p.pref_q[b] + r / kBlockM;
    return (static_cast<size_t>(pair) * p.vheads + vh) * kBlockM + (r % kBlockM);
  } else {
    return tiled_index(p, b, r, vh);
  }
}

cudaError_t launch_prefix_bwd_schedule(const PrefixBwd& p, int* pref_q, cudaStream_t st);
cudaError_t launch_prefix_prep(const PrefixBwd& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_prefix_bwd_dq(const PrefixBwd& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_prefix_bwd_dkdv(const PrefixBwd& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_prefix_sum(const PrefixBwd& p, bool bf16, int num_sms, cudaStream_t st);

cudaError_t launch_prefix_schedule(const PrefixParams& p, cudaStream_t st);
cudaError_t launch_prefix_fwd(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_prefix_join(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace teattn
