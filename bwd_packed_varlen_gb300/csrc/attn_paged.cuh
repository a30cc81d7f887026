// Attention over a paged cache: launch parameters and how the work is cut.
#pragma once

#include "paged.cuh"

namespace teattn {

constexpr int kPagedSMs = 152;        // of the GPU that work is cut for
constexpr int kPagedMaxBatch = 4096;  // prefix sums of the sequences' work fit shared memory

struct PagedParams {
  PagedCache cache;
  const void* q;
  void* out;
  float* lse;
  const int* cu_q;
  const int* cu_q_pad;
  const int* past;
  int batch, total_q, hq, hkv, d, group;
  int window;  // 0: none
  int sinks;
  float scale_log2;
  int* header;
  int* warp_status;  // status bits of each warp of the grid
  long long* pref;   // [batch + 1]: units of work before each sequence
  float2* part_ml;   // partial results, two slots a warp: maximum (log2 domain) and sum per row,
  float* part_o;     // unnormalised output, d columns
};

// Queries and keys of a sequence: token i sees the keys [lo(i), i + past + 1) and the sinks.
struct PagedSeq {
  int off, n, past;  // first row, queries, keys before the first query
  bool ok;
};

__device__ __forceinline__ PagedSeq load_paged_seq(const PagedParams& p, int b) {
  PagedSeq s{p.cu_q_pad[b], p.cu_q[b + 1] - p.cu_q[b], p.past[b], true};
  const int end = p.cu_q_pad[b + 1];
  const long long cap = static_cast<long long>(p.cache.max_pages) << p.cache.shift;
  s.ok = s.n >= 0 && s.off >= 0 && s.n <= end - s.off && end <= p.total_q && s.past >= 0 &&
         (s.n == 0 || s.past + static_cast<long long>(s.n) <= cap);
  if (!s.ok) s.n = 0;
  return s;
}

__device__ __forceinline__ int paged_first(const PagedParams& p, const PagedSeq& s, int i) {
  return p.window > 0 ? max(0, s.past + i + 1 - p.window) : 0;
}

// Blocks of `unit` keys that some query of the sequence sees: the sinks', then from the first
// query's window on.
struct PagedRun {
  int sink_units, first, n;
  __device__ __forceinline__ int unit(int u) const { return u < sink_units ? u : u - sink_units + first; }
};
__device__ __forceinline__ PagedRun paged_run(const PagedParams& p, const PagedSeq& s, int unit) {
  const int keys = s.past + s.n;
  PagedRun r;
  r.first = paged_first(p, s, 0) / unit;
  r.sink_units = p.window > 0 ? min((min(p.sinks, keys) + unit - 1) / unit, r.first) : 0;
  r.n = s.n > 0 ? r.sink_units + (keys + unit - 1) / unit - r.first : 0;
  return r;
}

cudaError_t launch_paged_rows(const PagedParams& p, bool bf16, bool four, int rows, int num_sms, cudaStream_t st);

// Rows that one pass over a sequence's keys takes, for a batch of this shape.
int paged_rows(int batch, int total_q, int group, int d);
// Warps of the whole grid, and with them the slots for partial results.
int paged_warps(int d, bool four);

}  // namespace teattn
