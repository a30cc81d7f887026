// Attention over a paged cache: launch parameters and how the work is cut.
#pragma once

#include <cuda.h>

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
  int wide_rows;     // 0: the kernel of few rows takes every sequence
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
  // (unsigned: with no offset below zero the span does not wrap)
  s.ok = s.n >= 0 && s.off >= 0 && s.n <= end - s.off && static_cast<unsigned>(end) <= static_cast<unsigned>(p.total_q) && s.past >= 0 &&
         (s.n == 0 || s.past + static_cast<long long>(s.n) <= cap);
  if (!s.ok) s.n = 0;
  return s;
}

__device__ __forceinline__ int paged_first(const PagedParams& p, const PagedSeq& s, int i) {
  return p.window > 0 ? max(0, s.past + i + 1 - p.window) : 0;
}

// Blocks of `unit` keys that some query sees: the sinks', then from the first query's window on.
struct PagedRun {
  int sink_units, first, n;
  __device__ __forceinline__ int unit(int u) const { return u < sink_units ? u : u - sink_units + first; }
};
// Run of the queries i0 .. i1.
__device__ __forceinline__ PagedRun paged_run(const PagedParams& p, const PagedSeq& s, int i0, int i1, int unit) {
  const int keys = s.past + i1 + 1;
  PagedRun r;
  r.first = paged_first(p, s, i0) / unit;
  r.sink_units = p.window > 0 ? min((min(p.sinks, keys) + unit - 1) / unit, r.first) : 0;
  r.n = r.sink_units + (keys + unit - 1) / unit - r.first;
  return r;
}

// How a kernel cuts the work: into segments of (sequence, row tile, kv head), each a run of
// blocks of `unit` keys, one behind the other on a line. The rows of a kv head are its group's
// queries, token by token; a row tile holds `rows` of them. Two kernels share the sequences:
// the `wide` one takes those with more than wide_rows rows a kv head, if it is launched at all.
struct PagedCut {
  int rows, unit;
  bool wide;

  __device__ __forceinline__ bool takes(const PagedParams& p, const PagedSeq& s) const {
    const bool many = p.wide_rows > 0 && static_cast<long long>(s.n) * p.group > p.wide_rows;
    return s.n > 0 && many == wide;
  }
  __device__ __forceinline__ int tiles(const PagedParams& p, const PagedSeq& s) const {
    return static_cast<int>((static_cast<long long>(s.n) * p.group + rows - 1) / rows);
  }
  // Run of a row tile. Tiles of few rows take that of the whole sequence, so that a place on the
  // line is found by division; their kernel copies all of it and computes what the tile sees. That is next
  // to nothing for the few tiles of a step or a draft; with many tiles, at d above 128, it is most of the time
  // behind a window (rates beside paged_wide_rows).
  __device__ __forceinline__ PagedRun run(const PagedParams& p, const PagedSeq& s, int tile) const {
    if (!wide) return paged_run(p, s, 0, s.n - 1, unit);
    const int r0 = tile * rows;  // (a call's rows are below 2^31 - 256)
    return paged_run(p, s, r0 / p.group, min((r0 + rows - 1) / p.group, s.n - 1), unit);
  }
  // Units of the first `n` row tiles of a sequence, for tiles of few rows.
  __device__ __forceinline__ long long before(const PagedParams& p, const PagedSeq& s, int n) const {
    return n > 0 ? static_cast<long long>(n) * p.hkv * run(p, s, 0).n : 0;
  }
};

// A stretch of one segment, as a slice of the line goes through it.
struct Stretch {
  int b, head, tile;
  int u0, n;  // units [u0, u0 + n) of the segment's run
  PagedSeq s;
  PagedRun run;
};

// Stretch that begins at place `at` of the line, ending at `end` at the latest.
__device__ __forceinline__ Stretch stretch_at(const PagedParams& p, const PagedCut& cut, const long long* pref, long long at,
                                              long long end) {
  Stretch t;
  int lo = 0, hi = p.batch - 1;  // the last sequence that begins at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pref[mid] <= at) lo = mid; else hi = mid - 1;
  }
  t.b = lo;
  t.s = load_paged_seq(p, lo);
  long long r = at - pref[lo];
  if (cut.wide) {
    // the whole warp looks through the row tiles, 32 at a time
    const int lane = threadIdx.x & 31, tiles = cut.tiles(p, t.s);
    for (t.tile = 0; t.tile < tiles; t.tile += 32) {
      const int mine = t.tile + lane < tiles ? cut.run(p, t.s, t.tile + lane).n : 0;
      long long upto = static_cast<long long>(mine) * p.hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const uint32_t behind = __ballot_sync(0xffffffffu, upto > r);
      const int k = behind ? __ffs(behind) - 1 : 32;  // the tile in which the place lies
      if (k > 0) r -= __shfl_sync(0xffffffffu, upto, k - 1);
      if (k < 32) {
        t.tile += k;
        break;
      }
    }
    t.run = cut.run(p, t.s, t.tile);
    t.head = static_cast<int>(r / t.run.n);
    t.u0 = static_cast<int>(r - static_cast<long long>(t.head) * t.run.n);
  } else {
    t.run = cut.run(p, t.s, 0);
    const int seg = static_cast<int>(r / t.run.n);
    t.u0 = static_cast<int>(r - static_cast<long long>(seg) * t.run.n);
    t.tile = seg / p.hkv;
    t.head = seg - t.tile * p.hkv;
  }
  const long long left = end - at;
  t.n = left < t.run.n - t.u0 ? static_cast<int>(left) : t.run.n - t.u0;
  return t;
}

// The stretch of many rows that follows `t`, which ends at place `at`; with `first` the one there.
__device__ __forceinline__ void next_stretch(const PagedParams& p, const PagedCut& cut, const long long* pref, long long at, long long end,
                                             bool first, Stretch& t) {
  if (!first && ++t.head == p.hkv) {
    t.head = 0;
    if (++t.tile < cut.tiles(p, t.s)) t.run = cut.run(p, t.s, t.tile);
    else first = true;  // the next sequence
  }
  if (first) {
    t = stretch_at(p, cut, pref, at, end);
    return;
  }
  t.u0 = 0;
  t.n = end - at < t.run.n ? static_cast<int>(end - at) : t.run.n;
}

// Row tiles that a thread adds up by itself: a warp of its own for each of 152 short sequences
// took 25 us, a thread alone for one of 1024 tiles a tenth of a millisecond.
constexpr int kTilesOfThread = 8;

// Prefix sums of the sequences' units in `pref` (shared memory, batch + 1 values), by the whole
// block; returns the total. Lengths that do not fit are reported in *status.
__device__ __forceinline__ long long sum_units(const PagedParams& p, const PagedCut& cut, long long* pref, int* status) {
  __shared__ long long warp_sum[32];
  __shared__ long long carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (tid == 0) carry = 0;
  __syncthreads();
#pragma unroll 1
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + tid;
    long long w = 0;
    int tiles = 0;
    PagedSeq s{0, 0, 0, true};
    if (b < p.batch) {
      s = load_paged_seq(p, b);
      if (!s.ok) atomicOr(status, kStatusBadSeqlens);
      if (cut.takes(p, s)) {
        tiles = cut.tiles(p, s);
        if (!cut.wide) w = cut.before(p, s, tiles);
      }
    }
    if (cut.wide) {
      // a thread adds up a sequence of few row tiles, a warp one of many
      const bool many = tiles > kTilesOfThread;
      if (!many) {
        for (int t = 0; t < tiles; ++t) w += cut.run(p, s, t).n;
        w *= p.hkv;
      }
      for (uint32_t some = __ballot_sync(0xffffffffu, many); some; some &= some - 1) {
        const int k = __ffs(some) - 1, n = __shfl_sync(0xffffffffu, tiles, k);
        s = load_paged_seq(p, b - lane + k);
        long long sum = 0;
        for (int t = lane; t < n; t += 32) sum += cut.run(p, s, t).n;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == k) w = sum * p.hkv;
      }
    }
    long long x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long before = carry, all = 0;
    for (int i = 0; i < nw; ++i) {
      if (i < warp) before += warp_sum[i];
      all += warp_sum[i];
    }
    if (b < p.batch) pref[b] = before + x - w;
    __syncthreads();
    if (tid == 0) carry += all;
    __syncthreads();
  }
  const long long total = carry;
  if (tid == 0) pref[p.batch] = total;
  __syncthreads();
  return total;
}

// Units of a slice, equal for all; `least` keeps what is left to join in bounds.
__device__ __forceinline__ long long slice_units(long long total, int slices, int least) {
  const long long per = (total + slices - 1) / slices;
  return per < least ? least : per;
}
// Keys of a warp at least: it needs a microsecond before its first product, and more pieces to join
// cost too. 3 sequences of 20-200 keys, d 64: 9.2 us with 32, 11.3 with 64, 12.5 with 128, 26 with 512;
// 3 of 500 in 16 bits, d 128: 17.8 us with 16, 15.6 with 32, 15.3 with 64.
constexpr int kLeastKeys = 32;
// Key tiles of a block at least (512 rows of one sequence behind 500 keys: 36 us with 1, 37 with 2, 41 with
// 4; behind 2000 keys 51, 50 and 46).
constexpr int kLeastWideUnits = 2;

// Partial results of one kernel: two slots a slice (of the segment that it ends, of the one that
// it begins), each of a row tile's rows; its prefix sums; slices in all.
struct PagedParts {
  long long* pref;
  float2* ml;   // maximum (log2 domain) and sum per row
  float* o;     // unnormalised output, d columns
  int slices, least;
};

// The kernel of few rows, that of many, and the join of both (wide.slices 0: the second was not
// launched). cut: set to how the first one cuts the work.
cudaError_t launch_paged_rows(const PagedParams& p, const PagedParts& parts, bool bf16, bool four, int rows,
                              PagedCut* cut, cudaStream_t st);
cudaError_t launch_paged_tiles(const PagedParams& p, const PagedParts& parts, int first_status, bool bf16, bool four, cudaStream_t st);
cudaError_t launch_paged_join(const PagedParams& p, const PagedCut& cut, const PagedParts& parts, const PagedParts& wide, bool bf16,
                              cudaStream_t st);

// Map of a 16-bit cache: columns, slots of a page, heads, pages; a box of 64 columns and `slots`.
bool make_tmap_pages(CUtensorMap* map, const PagedCache& c, int kv, bool bf16, int slots);

constexpr int kWideRows = 256, kWideKeys = 128;  // of a row tile and a unit of the second kernel

// Rows that one pass over a sequence's keys takes, for a batch of this shape.
int paged_rows(int batch, int total_q, int group, int d, bool four);
// Warps of the first kernel's whole grid.
int paged_warps(int d, bool four, int rows);
// Rows a kv head from which a sequence goes to the second kernel; 0: it is not launched.
int paged_wide_rows(int batch, int total_q, int hq, int hkv, int d, bool four);

}  // namespace teattn
