// Shared-prefix attention: launch parameters and work lists of its kernels.
#pragma once

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
  int4* seqs;        // per sequence: first compact token, own group, first long group (-1: none)
  int* short_tok;    // compact token -> packed row
  int4* groups;      // two int4 per group
  int2* entries;     // (group, chunk), each for every kv head
  float2* part_ml;   // partial rows: running maximum (log2 domain) and sum
  float* part_o;     // partial rows: unnormalised output, d columns
  int parts_target;  // chunks that all groups of one kv head together are cut into, about
  int cap_groups, cap_entries, cap_rows;
};

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
// against the prefix (prefix groups: row tiles of the compact token list) and alone
// against its own keys (one own group). A longer sequence has row tiles of its own, each
// over the prefix and then its own keys (long groups). A group's key tiles are cut into
// chunks; rows whose only group is one whole chunk are written directly, the others leave
// partial results that the join kernel merges.
// ---------------------------------------------------------------------------
constexpr int kShortRows = 128;
constexpr int kPartsTarget = 2 * 152;  // chunks over all kv heads, about: two per SM

__host__ __device__ constexpr int prefix_row_tile(int d) { return d <= 128 ? 256 : 128; }
__host__ __device__ constexpr int prefix_key_tile(int d) { return d <= 128 ? 128 : 64; }

struct PrefixGroup {
  int seq;    // -1: the compact tokens
  int row0;   // first packed row
  int rows;   // packed rows (at most a row tile)
  int np, no; // key tiles: prefix, own
  int chunks;
  int slot;   // partial row of (chunk 0, kv head 0, row 0); -1: written directly
  int is_long;
};

__device__ __forceinline__ PrefixGroup load_group(const PrefixParams& p, int e) {
  const int4 a = p.groups[2 * e], b = p.groups[2 * e + 1];
  return PrefixGroup{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}
__device__ __forceinline__ void store_group(const PrefixParams& p, int e, const PrefixGroup& g) {
  p.groups[2 * e] = make_int4(g.seq, g.row0, g.rows, g.np);
  p.groups[2 * e + 1] = make_int4(g.no, g.chunks, g.slot, g.is_long);
}
// Key tiles [first, last) of chunk c: the chunks of a group differ by at most one tile.
__device__ __forceinline__ int2 chunk_tiles(const PrefixGroup& g, int c) {
  const int n = g.np + g.no;
  return make_int2(static_cast<int>(static_cast<long long>(n) * c / g.chunks),
                   static_cast<int>(static_cast<long long>(n) * (c + 1) / g.chunks));
}
// Partial row of packed row r (within the group) of chunk c and kv head h.
__device__ __forceinline__ size_t partial_row(const PrefixParams& p, const PrefixGroup& g, int c, int h, int r) {
  return static_cast<size_t>(g.slot) + (static_cast<size_t>(c) * p.hkv + h) * g.rows + r;
}

cudaError_t launch_prefix_schedule(const PrefixParams& p, cudaStream_t st);
cudaError_t launch_prefix_fwd(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_prefix_join(const PrefixParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_prefix_bwd(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace teattn
