// Sliding windows with sinks: launch parameters and what the attention kernels need of them.
//
// Query i sits at key position p = i + diag and sees the keys j of [0, row_keys) with
// p - j < window or j < sinks. So a query tile's key tiles are the sinks' and then those from
// its first row's window on, and a key tile's queries end a window behind its last key unless
// it holds a sink: tiles between are not visited, and the work is that of the window, not of
// the sequence (but for the sweeps of sinks behind the 256th, see kSplitSinkTiles).
//
// Measured, bf16, hq 32, hkv 8, d 128, four sequences of 1500-6000 tokens, window 1024, 4 sinks:
// forward 465 us, delta 60, dQ 317, dK/dV 455, lists 29, zero fill 13 (events around each); forward and backward
// in a call 1300 us, 5 products for each visible pair in 429 us at the measured bf16 rate. d 256: 658, 106,
// 1098, 2310, 31, 17. Bounded as the kernels without a window are, by an item's begin and end, and in the
// forward by second readings of scores: a row's offset starts as the maximum over the keys that it sees
// of its first tile, and where those are few (a few sinks, a window's far edge) it lies so low that the
// later tiles' P sum past 2^8, which has their maximum looked for. 1 sink 592 us, 4 465, 16 315, 64 to 128
// 286-289 (instructions 150 million with 4, 110 with 64); none, windows of 1000 and 1024: 501 and 450.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace teattn {

// Rows below this and windows up to it (seen to by the host): positions stay within 32 bits.
constexpr int kWindowLimit = 1 << 30;

struct WindowParams : AttnParams {
  int window;  // >= 1
  int sinks;   // >= 0
  // Backward: a key tile with sinks is seen by every query behind it, while the others' sweeps end
  // with the window. Sweeps of the first kSplitSinkTiles tiles are cut into parts of sweep_tiles query
  // tiles, whose fp32 sums a last kernel adds up in order.
  int sweep_tiles;   // 0: no sweep is cut
  int* pref_s;       // [batch + 1]: slots for parts before each sequence
  int4* slots;       // (sequence, key tile, part): part -1 is the sweep's begin, an ordinary item
  float* part_dk;    // [slots][hkv][128][d]
  float* part_dv;
  int cap_slots;
};

// Sweeps of sinks behind the 256th are not cut: one block takes all queries behind them. dK/dV of the four
// sequences above with 256 sinks 483 us, 300 727, 1024 807; of one of 16384 tokens 533, 1291, 1809.
constexpr int kSplitSinkTiles = 2;
// As long as an ordinary sweep, but so long that few sequences have more than one part. (dK/dV of the
// four sequences above: 694 us with whole sweeps, 452 with cut ones; of 8 tiles
// at least 1303 us for the whole call, of 16 1305, of 32 1399.)
__host__ __device__ constexpr int sweep_tiles_of(int window) {
  return (window + kBlockM - 1) / kBlockM + 1 > 16 ? (window + kBlockM - 1) / kBlockM + 1 : 16;
}

template <class P>
constexpr bool is_window = std::is_base_of_v<WindowParams, P>;

// Key tiles that a query tile visits: step j is tile j of the sinks, then of the window.
struct TileRun {
  int sink_tiles, first, n;
  __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : j - sink_tiles + first; }
};

// First key of query i's window.
__device__ __forceinline__ int window_first(const WindowParams& p, const SeqInfo& s, int i) {
  return max(0, i + s.diag - p.window + 1);
}

// Run of the rows from r0 on, of which the last one sees keys below `hi`; key tiles of bn rows.
template <class P>
__device__ __forceinline__ TileRun tile_run(const P& p, const SeqInfo& s, int r0, int hi, int bn) {
  TileRun r{0, 0, (hi + bn - 1) / bn};
  if constexpr (is_window<P>) {
    r.first = min(window_first(p, s, r0) / bn, r.n);
    r.sink_tiles = min((min(p.sinks, hi) + bn - 1) / bn, r.first);
    r.n += r.sink_tiles - r.first;
  }
  return r;
}

// Which keys a row sees beside its limit: those from `lo` on, and those below `sinks`.
struct RowWindow {
  int lo, sinks;
};
template <class P>
__device__ __forceinline__ RowWindow row_window(const P& p, const SeqInfo& s, int i) {
  if constexpr (is_window<P>) return RowWindow{window_first(p, s, i), p.sinks};
  else return RowWindow{0, 0};
}

// The low n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Bit c: the row, which sees keys below `hi`, sees key `key` + c.
__device__ __forceinline__ uint32_t seen_bits(int hi, RowWindow w, int key) {
  return low_bits(hi - key) & (~low_bits(w.lo - key) | low_bits(w.sinks - key));
}

// Queries at the end of a sequence that see no key: a window or more behind its last one,
// without sinks (upper-left alignment, more queries than keys). First of them.
template <class P>
__device__ __forceinline__ int blind_tail(const P& p, const SeqInfo& s) {
  if constexpr (is_window<P>) {
    if (p.sinks == 0) return min(s.len_q, max(0, s.len_k - s.diag + p.window - 1));
  }
  return s.len_q;
}

// Keys before the first query's window that are no sinks: [from, to) of no query's.
struct KeyGap {
  int from, to;
};
template <class P>
__device__ __forceinline__ KeyGap key_gap(const P& p, const SeqInfo& s) {
  if constexpr (is_window<P>) {
    const int seen = seen_keys(s, true);
    const int to = min(seen, window_first(p, s, 0));
    return KeyGap{min(p.sinks, to), to};
  }
  return KeyGap{0, 0};
}

// Key tiles that some query sees: their number, and tile k of them.
template <class P>
__device__ __forceinline__ TileRun key_tiles(const P& p, const SeqInfo& s) {
  TileRun r{0, 0, (seen_keys(s, p.causal != 0) + kBlockN - 1) / kBlockN};
  if constexpr (is_window<P>) {
    const KeyGap g = key_gap(p, s);
    r.first = g.to / kBlockN;
    r.sink_tiles = min((g.from + kBlockN - 1) / kBlockN, r.first);
    r.n += r.sink_tiles - r.first;
  }
  return r;
}

// One past the last query that sees key j.
template <class P>
__device__ __forceinline__ int last_query(const P& p, const SeqInfo& s, int j) {
  if constexpr (is_window<P>) {
    if (j >= p.sinks) return min(s.len_q, j - s.diag + p.window);
  }
  return s.len_q;
}
// One past the last query that sees a key of tile kt.
template <class P>
__device__ __forceinline__ int tile_last_query(const P& p, const SeqInfo& s, int kt) {
  if constexpr (is_window<P>) {
    if (kt * kBlockN >= p.sinks) return last_query(p, s, min(kt * kBlockN + kBlockN, s.len_k) - 1);
  }
  return s.len_q;
}

// Sweep over key tile kt: query tiles [first, end) of 128 in the ordinary item, and then parts of
// sweep_tiles up to the sequence's last one.
struct Sweep {
  int end, parts;
};
template <class P>
__device__ __forceinline__ Sweep sweep_of(const P& p, const SeqInfo& s, int kt) {
  Sweep w{(tile_last_query(p, s, kt) + kBlockM - 1) / kBlockM, 0};
  if constexpr (is_window<P>) {
    if (p.sweep_tiles > 0 && kt < kSplitSinkTiles && kt * kBlockN < p.sinks) {
      const int last = min(s.len_q, min(kt * kBlockN + kBlockN, s.len_k) - 1 - s.diag + p.window);
      const int first = first_query(s, kt * kBlockN, true) / kBlockM;
      const int end = max((max(last, 0) + kBlockM - 1) / kBlockM, first + p.sweep_tiles);
      if (end < w.end) {
        w.parts = (w.end - end + p.sweep_tiles - 1) / p.sweep_tiles;
        w.end = end;
      }
    }
  }
  return w;
}
// Slots of a sequence's key tiles before kt.
__device__ __forceinline__ int slots_before(const WindowParams& p, const SeqInfo& s, int kt) {
  const int tiles = key_tiles(p, s).n > 0 ? (min(p.sinks, seen_keys(s, true)) + kBlockN - 1) / kBlockN : 0;
  int n = 0;
  for (int k = 0; k < min(min(kt, kSplitSinkTiles), tiles); ++k) {
    const Sweep w = sweep_of(p, s, k);
    n += w.parts > 0 ? w.parts + 1 : 0;
  }
  return n;
}

cudaError_t launch_window_delta(const WindowParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_window_sum(const WindowParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_window_schedule(const WindowParams& p, int* pref_q, int* pref_k, int* pref_f, cudaStream_t st);
cudaError_t launch_window_zero_fill(const WindowParams& p, int mode, int num_sms, cudaStream_t st);
cudaError_t launch_window_fwd(const WindowParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_window_fwd_pair(const WindowParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_window_bwd_dkdv(const WindowParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_window_bwd_dq(const WindowParams& p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace teattn
