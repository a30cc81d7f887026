// Shared-prefix attention, forward.
//
//   S = scale [q Kp^T | q K_b^T + mask],  O = softmax(S) [Vp; V_b],  LSE = log sum exp S
//
// One persistent kernel takes items (rows, chunk of their key tiles, kv head); see
// attn_prefix.cuh. The rows of an item are the queries of one kv head's group packed token
// by token, so a decoding step of many sequences fills the 128-row tiles of the tensor
// cores against the prefix, and K/V tiles are read once for all of them. Roles:
//   warps 0-3   softmax of stream 0 (one thread per row / TMEM lane),
//   warps 4-7   softmax of stream 1 (head_dim <= 128 only),
//   then        an item warp (takes items from the common list and decodes them), a K/V warp
//               and a Q warp (TMA) and an MMA warp.
// An item of at most 128 rows runs on one stream; the streams work on different items and
// their key tiles alternate in the shared K/V ring, so one item's exponentials, first
// scores and stores overlap the other's products (a decoding step's items are a few tiles
// long, and the chain S -> P -> O of a tile is about 2700 cycles against 1000 of tensor
// work). An item of more rows takes both streams, row tile A and B, over the same key tiles.
// Above head_dim 128 O takes half of TMEM and there is one stream; its scores run a tile ahead
// of the products (batch 24, head_dim 256, prefix 20000: 42.2 -> 37.8 us).
// S = Q K^T into TMEM, P = exp2(S scale log2e - m) over it as 16-bit values, O += P V in
// TMEM. The offset m is raised only when a row's maximum exceeds it by more than 2^8.
// P is rounded to 16 bits for the tensor cores (relative to the row's largest value, half a
// step of its type); its sum l, m, O and everything joined later stay in fp32.
//
// Rows that no key tile ends in (a key tile past the sequence's or the prefix's last key)
// hold other sequences' keys or whatever the caller's cache holds: their scores are
// selected away, and their V rows are zeroed in shared memory before the product, so
// that even infinities and NaN there do not reach a result.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "attn_prefix.cuh"
#include "pdl.cuh"
#include "row_store.cuh"
#include "sm103_ptx.cuh"
#include "tmap.h"
#include "work_queue.cuh"

namespace teattn {

// ---------------------------------------------------------------------------
// Scheduler: one block; from the lengths to entries and partial rows, with a thread per
// sequence and block-wide scans. It is on every call's critical path and latency-bound, so
// each phase loads what it needs at once and costs two barriers. The result depends on the
// lengths only.
// ---------------------------------------------------------------------------
constexpr int kPrefixSchedThreads = 1024;

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// Keys that token i of a sequence sees.
__device__ __forceinline__ int keys_seen(int causal, int len_k, int diag, int i) {
  return causal ? min(len_k, max(0, i + 1 + diag)) : len_k;
}
// Own key tiles that the packed rows [row0, row0 + rows) see.
__device__ __forceinline__ int own_tiles(const PrefixParams& p, int len_k, int diag, int row0, int rows, int bn) {
  return div_up(keys_seen(p.causal, len_k, diag, (row0 + rows - 1) / p.group), bn);
}

__global__ void __launch_bounds__(kPrefixSchedThreads) prefix_schedule_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ int buf[3][32];
  __shared__ int bad;
  __shared__ unsigned long long work, tokens;
  // with at most a thread per sequence: their own key tiles, order by those, and spans
  __shared__ __align__(16) int s_tiles[kPrefixSchedThreads];
  __shared__ int s_order[kPrefixSchedThreads], s_first[kPrefixSchedThreads];
  __shared__ int4 s_seq[kPrefixSchedThreads];
  pdl_trigger();
  const int rt = prefix_row_tile(p.d), bn = prefix_key_tile(p.d), tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    bad = p.prefix_len && (*p.prefix_len < 0 || *p.prefix_len > p.prefix_rows) ? 1 : 0;
    work = tokens = 0;
  }
  const int np_keys = prefix_keys(p), np = div_up(np_keys, bn);
  __syncthreads();
  // sequences: compact tokens, long row tiles; an upper bound of the key tiles
  SeqInfo s{};
  int n_tok = 0, n_long = 0, first_tok = 0, first_long = 0;
#pragma unroll 1
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + tid;
    int tok = 0, nl = 0;
    unsigned long long w = 0, q = 0;
    s = SeqInfo{};
    if (b < p.batch) {
      s = load_seq(p, b);
      if (!s.ok) bad = 1;
      const int tiles = div_up(s.len_k, bn);
      const int rows = s.len_q * p.group;  // (total_q * hq is below 2^31)
      q = s.len_q;
      if (rows > kShortRows) {
        nl = ((rows - 1) >> (rt == 256 ? 8 : 7)) + 1;
        w = static_cast<unsigned long long>(nl) * (np + tiles);
      } else if (rows > 0) {
        tok = s.len_q;
        w = tiles;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      w += __shfl_xor_sync(0xffffffffu, w, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    if (lane == 0) {
      atomicAdd(&work, w);
      atomicAdd(&tokens, q);
    }
    const Scan3 at = block_scan3(tok, nl, 0, buf);
    first_tok = tok > 0 ? n_tok + at.x : -1;
    first_long = n_long + at.y;
    if (b < p.batch) {
      p.seqs[b] = make_int4(first_tok, -1, 0, first_long);
#pragma unroll 1
      for (int i = 0; i < tok; ++i)
        if (first_tok + i < p.total_q) p.short_tok[first_tok + i] = s.off_q + i;
    }
    n_tok += at.tx;
    n_long += at.ty;
  }
  // The scans' barriers order the sums before what follows, but not the records: those are
  // written behind the last scan, and the search below reads other threads'. (n_long is the
  // same in every thread; steps of short sequences read only their own thread's record.)
  if (n_long > 0) __syncthreads();
  if (tokens > static_cast<unsigned long long>(p.total_q)) {
    // sequences overlap: more tokens than rows, for which the lists have no room
    if (tid == 0) {
      p.header[kHdrStatus] = kStatusBadSeqlens;
      p.header[kHdrPrefixEntries] = 0;
      p.header[kHdrPrefixChunks] = -1;
      p.header[kHdrNextFwd] = 0;
    }
    return;
  }
  const int short_rows = n_tok * p.group;
  const int n_pre = np > 0 ? div_up(short_rows, rt) : 0;
  const unsigned long long all = work + static_cast<unsigned long long>(n_pre) * np;
  // Chunk length in key tiles: all heads' chunks together about one per SM when there is
  // little to do (an item costs about four tiles before its first), two when there is much.
  const int parts = all >= 8ull * p.parts_target ? p.parts_target : (p.parts_target + 1) / 2;
  // (a 64-bit division would be 500 cycles on the way of every call)
  const int len = all >> 31 ? static_cast<int>((all + parts - 1) / parts)
                            : max(1, static_cast<int>((static_cast<uint32_t>(all) + parts - 1) / parts));
  int n_entries = 0, n_rows = 0;  // running totals
  // Chunk c of a row tile with n key tiles in `chunks` chunks (they differ by one tile at
  // most), as entry `at`; e.slot: the row tile's first partial row.
  auto put_chunk = [&](PrefixEntry e, int n, int chunks, int c, int at) {
    const int q = n / chunks, r = n - q * chunks;
    e.t0 = c * q + min(c, r);
    e.t1 = e.t0 + q + (c < r ? 1 : 0);
    if (e.slot >= 0) e.slot += c * p.hkv * e.rows;
    if (at < p.cap_entries) store_entry(p, at, e);
  };
  // Entries of more than 128 rows, which take both streams of a block, come first: one that
  // came after an entry of fewer would keep a stream idle until the other is through.
  const int pre_chunks = n_pre > 0 ? div_up(np, len) : 0;
  const int last_pre = n_pre > 0 ? short_rows - (n_pre - 1) * rt : 0;
  // compact row tiles that take both streams
  const int wide_pre = n_pre > 0 && rt > 128 ? n_pre - (last_pre > 128 ? 0 : 1) : 0;
  int pre_slot = 0;
#pragma unroll 1
  for (int round = rt > 128 ? 0 : 1; round < 2; ++round) {  // the wide entries, then the others
    const bool wide = round == 0;
    // long row tiles
#pragma unroll 1
    for (int base = 0; base < n_long; base += blockDim.x) {
      const int g = base + tid;
      PrefixEntry e{};
      int n = 0, ch = 0, slots = 0;
      if (g < n_long) {
        int lo = 0, hi = p.batch - 1;  // last sequence whose first row tile is at most g
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.seqs[mid].w <= g) lo = mid; else hi = mid - 1;
        }
        const SeqInfo q = load_seq(p, lo);
        e.seq = lo;
        e.row0 = (g - p.seqs[lo].w) * rt;
        e.rows = min(rt, q.len_q * p.group - e.row0);
        if ((e.rows > 128) == wide) {
          e.np = np;
          e.off_q = q.off_q;
          e.off_k = q.off_k;
          e.len_k = q.len_k;
          e.diag = q.diag;
          n = np + own_tiles(p, q.len_k, q.diag, e.row0, e.rows, bn);
          ch = div_up(n, len);
          slots = ch > 1 ? ch * p.hkv * e.rows : 0;
        } else {
          e.rows = 0;
        }
      }
      const Scan3 at = block_scan3(ch, slots, 0, buf);
      if (e.rows > 0 && g < p.cap_longs) {
        e.slot = slots > 0 ? n_rows + at.y : -1;
        p.longs[g] = make_int4(e.slot, ch, e.rows, 0);
#pragma unroll 1
        for (int c = 0; c < ch; ++c) put_chunk(e, n, ch, c, n_entries + at.x + c);
      }
      n_entries += at.tx;
      n_rows += at.ty;
    }
    // the compact rows against the prefix, chunk-major: row tiles that read the same keys
    // are taken side by side
    if (wide || rt == 128) {
      pre_slot = n_rows;
      n_rows += short_rows * pre_chunks * p.hkv;
    }
    const int u0 = wide || rt == 128 ? 0 : wide_pre, u1 = wide ? wide_pre : n_pre;
#pragma unroll 1
    for (int k = tid; k < (u1 - u0) * pre_chunks; k += blockDim.x) {
      const int c = k / (u1 - u0), u = u0 + k - c * (u1 - u0);
      PrefixEntry e{};
      e.seq = -1;
      e.row0 = u * rt;
      e.rows = min(rt, short_rows - e.row0);
      e.np = np;
      e.slot = pre_slot + u * rt * pre_chunks * p.hkv;
      put_chunk(e, np, pre_chunks, c, n_entries + k);
    }
    n_entries += (u1 - u0) * pre_chunks;
  }
  // Short sequences against their own keys, the longest first (with at most a thread per
  // sequence): the blocks then run out of work together. A sequence's place is the number of
  // sequences that go before it.
  const bool sorted = p.batch <= blockDim.x;
  if (sorted) {
    const int n = first_tok >= 0 ? own_tiles(p, s.len_k, s.diag, 0, s.len_q * p.group, bn) : -1;
    s_tiles[tid] = n;
    s_first[tid] = first_tok;
    s_seq[tid] = make_int4(s.off_q, s.len_q, s.off_k, s.len_k);
    __syncthreads();
    // (threads past the batch hold -1 and come after every sequence)
    int place = 0;
#pragma unroll 4
    for (int j = 0; j < p.batch; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(&s_tiles[j]);
      place += (o.x > n || (o.x == n && j < tid)) + (o.y > n || (o.y == n && j + 1 < tid)) +
               (o.z > n || (o.z == n && j + 2 < tid)) + (o.w > n || (o.w == n && j + 3 < tid));
    }
    s_order[place] = tid;
    __syncthreads();
  }
#pragma unroll 1
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int at_b = base + tid;
    const int b = at_b < p.batch ? (sorted ? s_order[tid] : at_b) : p.batch;
    SeqInfo q{};
    int first = -1;
    if (sorted && b < p.batch) {
      first = s_first[b];
      const int4 v = s_seq[b];
      q.off_q = v.x;
      q.len_q = v.y;
      q.off_k = v.z;
      q.len_k = v.w;
      q.diag = p.causal == 2 ? v.w - v.y : 0;
    } else if (b < p.batch) {
      q = load_seq(p, b);
      first = p.seqs[b].x;
    }
    PrefixEntry e{};
    int n = 0, ch = 0, slots = 0;
    if (first >= 0) {
      e.seq = b;
      e.rows = q.len_q * p.group;
      e.off_q = q.off_q;
      e.off_k = q.off_k;
      e.len_k = q.len_k;
      e.diag = q.diag;
      n = own_tiles(p, q.len_k, q.diag, 0, e.rows, bn);
      ch = div_up(n, len);
      // without a prefix a single chunk is the whole result
      slots = ch > 1 || n_pre > 0 ? ch * p.hkv * e.rows : 0;
    }
    const Scan3 at = block_scan3(ch, slots, 0, buf);
    if (ch > 0) {
      e.slot = slots > 0 ? n_rows + at.y : -1;
      p.seqs[b] = make_int4(first, e.slot, slots > 0 ? ch : -1, 0);
#pragma unroll 1
      for (int c = 0; c < ch; ++c) put_chunk(e, n, ch, c, n_entries + at.x + c);
    }
    n_entries += at.tx;
    n_rows += at.ty;
  }
  if (tid == 0) {
    // the capacities hold for every set of lengths; if they did not, nothing is computed
    const bool over = n_long > p.cap_longs || n_entries > p.cap_entries || n_rows > p.cap_rows;
    p.header[kHdrStatus] = (bad ? kStatusBadSeqlens : 0) | (over ? kStatusInternal : 0);
    p.header[kHdrPrefixEntries] = over ? 0 : n_entries;
    p.header[kHdrPrefixChunks] = over ? -1 : pre_chunks;
    p.header[kHdrPrefixSlot] = pre_slot;
    p.header[kHdrPrefixRows] = short_rows;
    p.header[kHdrNextFwd] = 0;
  }
}

cudaError_t launch_prefix_schedule(const PrefixParams& p, cudaStream_t st) {
  const int threads = p.batch >= kPrefixSchedThreads ? kPrefixSchedThreads : (p.batch + 31) / 32 * 32;
  prefix_schedule_kernel<<<1, threads < 128 ? 128 : threads, 0, st>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Main kernel
// ---------------------------------------------------------------------------
// Tensor maps of one call.
struct PrefixMaps {
  CUtensorMap k, v, kp, vp;
  CUtensorMap q_tile, q_token, q_row;  // boxes of 128 rows (whole tokens), one token's group, one row
  int q_tokens;                        // tokens of q_tile's box; 0: a tile does not hold whole ones
};

template <int kD>
struct PrefixShape {
  static constexpr int kNT = prefix_row_tile(kD) / 128;   // streams
  static constexpr int kBN = prefix_key_tile(kD);          // keys per tile
  static constexpr int kChunks = kD / 64;                  // 64-column chunks of a row
  static constexpr int kQBytes = kChunks * 16384;          // one 128-row Q tile
  static constexpr int kKVBytes = kChunks * kBN * 128;     // one K or V tile
  static constexpr int kStages = kD == 64 ? 4 : 2;
  static constexpr int kStageBytes = kNT * 4 * 2048;       // per softmax warp, for its stores
  static constexpr int kSmemBytes = kNT * kQBytes + 2 * kStages * kKVBytes + kStageBytes + 1024;
  static constexpr int kThreads = kNT * 128 + 128;
  // TMEM columns of O and S of stream x: O_0 O_1 S_0 S_1
  __device__ static constexpr uint32_t col_o(int x) { return static_cast<uint32_t>(x) * 128u; }
  __device__ static constexpr uint32_t col_s(int x) { return 256u + static_cast<uint32_t>(x) * 128u; }
  static_assert(kSmemBytes <= 220 * 1024, "shared memory budget");
};

__device__ __forceinline__ float ex2p(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What the item warp hands to a stream, the K/V warp and the MMA warp (two slots in turn).
struct PrefixItem {
  int n;            // key tiles the stream visits; -1: no more items
  int pair;         // the item takes both streams (n may then be 0 for the first)
  int np;           // the first np key tiles are the prefix's
  int p_key, o_key; // tensor rows of the first prefix key and the first own key
  int p_left;       // prefix keys from the item's first prefix tile on
  int o_left;       // own real keys from the item's first own tile on
  int direct;       // rows are written to out / lse, not to partial rows
  int head;         // kv head
  int part;         // partial row of the stream's first row
  int rows;         // rows of the stream; the arrays hold them rounded up to 32
  int row[128];     // per row: token * hq + head; -1: no row
  int lim[128];     // per row: own keys it sees from the item's first own tile on
};
struct ItemRing {
  PrefixItem item[2];
  // kv: all but the rows is there (the K/V warp starts on that); full: the rows too; empty: the
  // K/V, Q and MMA warps and the stream are through with it
  uint64_t kv[2], full[2], empty[2];
};

// The order of key tiles over the streams, in which the K/V warp loads and the MMA warp
// issues them, one tile a step: before a step one stream without tiles, if there is one,
// takes the next item (the one whose turn it is before the other), then the streams with
// tiles alternate. An item for both streams waits until both have run out. The item warp
// follows the same counts to know which stream takes an item. (One item a step: the first
// item's loads do not wait for the second one to be decoded.)
struct TileOrder {
  int left0 = 0, left1 = 0;  // key tiles that each stream has left (scalars: no local memory)
  int last = 1;
  __device__ __forceinline__ int left(int x) const { return x ? left1 : left0; }
  __device__ __forceinline__ void set(int x, int n) {
    if (x) left1 = n;
    else left0 = n;
  }
  __device__ __forceinline__ void take(int x) {
    set(x, left(x) - 1);
    last = x;
  }
  __device__ __forceinline__ int next() const { return left(1 - last) > 0 ? 1 - last : last; }
  // Stream that takes the next item before this step; -1: none.
  __device__ __forceinline__ int wants(bool able0, bool able1) const {
    const bool w0 = left0 == 0 && able0, w1 = left1 == 0 && able1;
    return last == 1 ? (w0 ? 0 : w1 ? 1 : -1) : (w1 ? 1 : w0 ? 0 : -1);
  }
};

template <int kD, bool kBF16>
__global__ void __launch_bounds__(PrefixShape<kD>::kThreads, 1)
    attn_prefix_fwd_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ PrefixMaps tm) {
  using S = PrefixShape<kD>;
  constexpr int NT = S::kNT, NS = S::kStages, BN = S::kBN;
  constexpr int kWarpItem = NT * 4, kWarpKv = NT * 4 + 1, kWarpMma = NT * 4 + 2, kWarpQ = NT * 4 + 3;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                        // one tile per stream
  uint8_t* sK = sQ + NT * S::kQBytes;
  uint8_t* sV = sK + NS * S::kKVBytes;
  uint8_t* sStage = sV + NS * S::kKVBytes;

  __shared__ uint64_t bar_q_full[NT], bar_q_empty[NT];
  __shared__ uint64_t bar_k_full[NS], bar_k_empty[NS], bar_v_full[NS], bar_v_empty[NS];
  // S and P: of stream x, or with one stream of its two S tiles, which take turns
  __shared__ uint64_t bar_s_full[2], bar_p_ready[2], bar_o_full[NT], bar_o_empty[NT];
  __shared__ uint64_t bar_pv;  // one stream: a product is done
  __shared__ ItemRing rings[NT];
  __shared__ int tiles_loaded;  // by the K/V warp, for the item warp to keep pace with
  __shared__ uint32_t tmem_slot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* status = p.header + kHdrStatus;

  if (tid == 0) {
    tiles_loaded = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_v_empty[i], 1);
    }
    mbar_init(&bar_pv, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_s_full[i], 1);
      mbar_init(&bar_p_ready[i], 128);
    }
    for (int x = 0; x < NT; ++x) {
      mbar_init(&bar_q_full[x], 1);
      mbar_init(&bar_q_empty[x], 1);
      mbar_init(&bar_o_full[x], 1);
      mbar_init(&bar_o_empty[x], 128);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&rings[x].kv[i], 1);
        mbar_init(&rings[x].full[i], 1);
        mbar_init(&rings[x].empty[i], 1 + 32 + 32 + 128);  // K/V warp's lane 0, MMA and Q warps, softmax
      }
    }
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp == kWarpKv && lane == 0) {
    const CUtensorMap* maps[] = {&tm.k, &tm.v, &tm.kp, &tm.vp, &tm.q_tile, &tm.q_token, &tm.q_row};
    for (const CUtensorMap* m : maps) tma_prefetch_desc(m);
  }
  pdl_trigger();
  pdl_wait();  // the scheduler's lists

  if (warp == kWarpItem) {
    // ------------------------------------------------------------- items
    // the first entry is read along with the number of entries (the grid is no larger than
    // the entries' capacity)
    const PrefixEntry first = load_entry(p, blockIdx.x / p.hkv);
    const int n_items = p.header[kHdrPrefixEntries] * p.hkv;
    const int np_keys = prefix_keys(p);
    int nxt = blockIdx.x;
    int puts0 = 0, puts1 = 0;  // hand-overs so far, per stream
    auto puts = [&](int x) { return x ? puts1 : puts0; };
    TileOrder order;
    bool ok = true;
    auto wait_slot = [&](int x) {
      const int n = puts(x);
      return n < 2 || __all_sync(0xffffffffu, mbar_wait(&rings[x].empty[n & 1], ((n >> 1) - 1) & 1, status));
    };
    // An item is taken from the common list only when the tiles before it are loaded but for
    // four: enough to hide its decoding, and no more, since a block that takes items early may
    // sit on them while others have run out (8: usual decoding step 47.5 -> 48.7 us; as many
    // as the slots hold: prompts 695 -> 760 us).
    constexpr int ahead = 4;
    int emitted = 0;  // tiles in the order so far
    auto keep_pace = [&]() -> bool {
      const volatile int* loaded = &tiles_loaded;
      if (emitted - *loaded <= ahead) return true;
      const unsigned long long t0 = global_ns();
      for (uint32_t it = 1;; ++it) {
        __nanosleep(400);
        if (emitted - *loaded <= ahead) return true;
        if ((it & 15u) == 0) {
          if (*reinterpret_cast<volatile int*>(status) & kErrTimeout) return false;
          if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(status, kErrTimeout);
            return false;
          }
        }
      }
    };
#pragma unroll 1
    for (int ii = 0;; ++ii) {
      while (NT == 2 && order.wants(true, true) < 0) {
        order.take(order.next());
        ++emitted;
      }
      if (ii > 0) {
        if (!(ok = __all_sync(0xffffffffu, lane > 0 || keep_pace()))) break;
        if (lane == 0) nxt = next_item(p.header + kHdrNextFwd);
        nxt = __shfl_sync(0xffffffffu, nxt, 0);
      }
      const int item = nxt < n_items ? nxt : -1;
      if (item < 0) break;
      const PrefixEntry e = ii == 0 ? first : load_entry(p, item / p.hkv);
      const int h = item % p.hkv;
      const int np = max(0, min(e.t1, e.np) - e.t0);  // prefix tiles of the chunk
      const int o0 = max(0, e.t0 - e.np);             // first own tile
      const bool pair = e.rows > 128;
      // own tiles end at the last one that a row of the tile sees
      auto tiles = [&](int k) {
        const int rows = min(128, e.rows - k * 128);
        const int no = e.seq >= 0 ? own_tiles(p, e.len_k, e.diag, e.row0 + k * 128, rows, BN) : 0;
        return max(0, min(e.t1, e.np + no) - e.t0);
      };
      const int n0 = tiles(0), n1 = pair ? tiles(1) : 0;
      int x0 = 0;
      if (pair) {
        emitted += order.left0 + order.left1 + max(n0, n1);
        order = TileOrder();
      } else if (NT == 2) {
        x0 = order.wants(true, true);
        order.set(x0, n0);
        order.take(order.next());
        ++emitted;
      } else {
        emitted += n0;
      }
      const int parts = pair ? 2 : 1;  // row tile k of the item goes to stream x0 + k
#pragma unroll 1
      for (int k = 0; k < parts; ++k) {
        const int x = x0 + k, r0 = k * 128, rows = min(128, e.rows - r0);
        // rows: where they lie (all loads in flight at once)
        int tok[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (u * 32 >= rows) break;
          const int r = u * 32 + lane, i = (e.row0 + r0 + r) / p.group;
          tok[u] = r >= rows ? -1 : e.seq < 0 ? p.short_tok[i] : e.off_q + i;
        }
        // the slot's last readers are done with it
        if (!(ok = wait_slot(x))) break;
        const int sl = puts(x) & 1;
        PrefixItem& I = rings[x].item[sl];
        if (lane == 0) {
          I.n = k ? n1 : n0;
          I.pair = pair ? 1 : 0;
          I.np = np;
          I.p_key = e.t0 * BN;
          I.o_key = e.off_k + o0 * BN;
          I.p_left = np_keys - e.t0 * BN;
          I.o_left = e.len_k - o0 * BN;
          I.direct = e.slot < 0 ? 1 : 0;
          I.head = h;
          I.part = e.slot < 0 ? 0 : e.slot + static_cast<int>(partial_offset(p, e.rows, 0, h)) + r0;
          I.rows = rows;
          mbar_arrive(&rings[x].kv[sl]);
        }
        // the rows' places and what they see
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = u * 32 + lane;
          if (u * 32 >= rows) break;
          const int rr = e.row0 + r0 + r, i = rr / p.group, j = rr - i * p.group;
          const bool in = r < rows && bounds_ok(tok[u] >= 0 && tok[u] < p.total_q, status);
          I.row[r] = in ? tok[u] * p.hq + h * p.group + j : -1;
          I.lim[r] = in && e.seq >= 0 ? max(0, keys_seen(p.causal, e.len_k, e.diag, i) - o0 * BN) : 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rings[x].full[sl]);
        if (x) ++puts1;
        else ++puts0;
      }
      if (!ok) break;
    }
    // no more items, on every stream
#pragma unroll 1
    for (int x = 0; x < NT && ok; ++x) {
      if (!(ok = wait_slot(x))) break;
      if (lane == 0) {
        rings[x].item[puts(x) & 1].n = -1;
        mbar_arrive(&rings[x].kv[puts(x) & 1]);
        mbar_arrive(&rings[x].full[puts(x) & 1]);
      }
    }
  } else if (warp == kWarpQ) {
    // ------------------------------------------------------------- Q rows
    // In the order in which the streams take items, so that it never waits for a tile whose
    // last scores wait for rows behind it. Beside the item warp, not in it: one warp needed
    // 5500 cycles for both, and short items came no faster (192 caches of 515 keys: 104 -> 98
    // us; 256 long ones 412 -> 406).
    TileOrder order;
    bool held0 = false, held1 = false, ended0 = false, ended1 = NT == 1;
    int gets0 = 0, gets1 = 0, loads0 = 0, loads1 = 0;
    for (;;) {
      const int x = order.wants(!held0 && !ended0, !held1 && !ended1);
      if (x < 0) {
        if (held0 && held1) {
          held0 = held1 = false;
          order = TileOrder();
        } else if (order.left0 > 0 || order.left1 > 0) {
          order.take(order.next());
        } else {
          break;
        }
        continue;
      }
      const int gets = x ? gets1 : gets0, loads = x ? loads1 : loads0, sl = gets & 1;
      if (!mbar_wait_warp(&rings[x].full[sl], (gets >> 1) & 1, status)) break;
      if (x) ++gets1;
      else ++gets0;
      const PrefixItem& I = rings[x].item[sl];
      const int n = I.n;
      if (n < 0) {
        if (x) ended1 = true;
        else ended0 = true;
        continue;
      }
      if (I.pair != 0) {
        if (x) held1 = true;
        else held0 = true;
      } else {
        order.set(x, n);
      }
      // by TMA: one box of 128 rows where tokens lie side by side and a tile holds whole ones,
      // else token by token (all heads of the group in one box, one lane each), and row by row
      // where a token's heads do not all lie in this tile. A box may start at any 128-byte
      // row of the tile: the swizzle goes by shared-memory address.
      const int rows = I.rows, h0 = I.head * p.group;
      const int row_a = I.row[0], row_z = I.row[rows - 1];
      const int tok_a = row_a / p.hq, tok_z = row_z / p.hq;
      const bool whole = tm.q_tokens > 0 && min(row_a, row_z) >= 0 && row_a - tok_a * p.hq == h0 &&
                         (tok_z - tok_a) * p.group + row_z - tok_z * p.hq - h0 == rows - 1;
      if (loads > 0 && !mbar_wait_warp(&bar_q_empty[x], (loads - 1) & 1, status)) break;
      uint8_t* q_tile = sQ + x * S::kQBytes;
      if (lane == 0) mbar_arrive_expect_tx(&bar_q_full[x], (whole ? 128 : rows) * 128 * S::kChunks);
      __syncwarp();
#pragma unroll 1
      for (int r = lane; r < rows; r += 32) {
        // (a row without a place, after an error: zeros, from behind the last token)
        const int row = I.row[r], t = row < 0 ? p.total_q : row / p.hq, head = row < 0 ? h0 : row - t * p.hq;
        const int j = head - h0;  // the token's rows in the tile: from r - j on
        const bool box = row >= 0 && p.group <= 128 && r >= j && r - j + p.group <= rows;
        if (whole ? r > 0 : box && j > 0) continue;
        const CUtensorMap* map = whole ? &tm.q_tile : box ? &tm.q_token : &tm.q_row;
#pragma unroll 1
        for (int c = 0; c < S::kChunks; ++c)
          tma_load_4d(q_tile + c * 16384 + r * 128, map, &bar_q_full[x], c * 64, head, 0, t);
      }
      __syncwarp();
      mbar_arrive(&rings[x].empty[sl]);
      if (x) ++loads1;
      else ++loads0;
    }
  } else if (warp == kWarpKv) {
    // ------------------------------------------------------------- K and V tiles
    if (lane == 0) {
      struct Tiles {
        int np, p_key, o_key, h, j;
      };
      int it = 0;
      Tiles cur0{}, cur1{};
      int gets0 = 0, gets1 = 0;
      bool held0 = false, held1 = false, ended0 = false, ended1 = NT == 1;
      int pair_left = 0;  // tiles that the item on both streams has left
      int pair_n = 0;
      TileOrder order;
      // K of a tile goes before V of the tile before it: that is the order in which their
      // stages come free, as a stream's next scores do not wait for the other's product (6 %
      // of a step over many long caches; with V beside its K, 1 % less for wide items).
      const CUtensorMap* v_map = nullptr;  // the V tile that is still to be loaded
      int v_key = 0, v_head = 0;
      auto load = [&](uint8_t* base, uint64_t* full, uint64_t* empty, const CUtensorMap* map, int head, int key,
                      int tile) -> bool {
        const int st = tile % NS;
        if (tile >= NS && !mbar_wait(&empty[st], ((tile / NS) - 1) & 1, status)) return false;
        mbar_arrive_expect_tx(&full[st], S::kKVBytes);
#pragma unroll 1
        for (int k = 0; k < S::kChunks; ++k)
          tma_load_4d(base + st * S::kKVBytes + k * BN * 128, map, &full[st], k * 64, head, 0, key);
        return true;
      };
      for (;;) {
        bool flush = false;  // no tile to load before a wait or the end: V of the last one
        const int w = pair_left > 0 ? -1 : order.wants(!held0 && !ended0, !held1 && !ended1);
        if (w >= 0) {
          const int gets = w ? gets1 : gets0, sl = gets & 1;
          uint64_t* bar = &rings[w].kv[sl];
          if (!mbar_try_wait(bar, (gets >> 1) & 1)) {
            flush = v_map != nullptr;
            if (!flush && !mbar_wait(bar, (gets >> 1) & 1, status)) break;
          }
          if (!flush) {
            const PrefixItem& I = rings[w].item[sl];
            const int n = I.n;
            const Tiles c{I.np, I.p_key, I.o_key, I.head, 0};
            const bool pair = I.pair != 0;
            mbar_arrive(&rings[w].empty[sl]);
            if (w) {
              ++gets1;
              cur1 = c;
              if (n < 0) ended1 = true;
              else if (pair) held1 = true;
            } else {
              ++gets0;
              cur0 = c;
              if (n < 0) ended0 = true;
              else if (pair) held0 = true;
            }
            if (n >= 0 && pair) pair_n = max(pair_n, n);
            if (n >= 0 && !pair) order.set(w, n);
          }
        }
        int x = -1;  // stream whose tile is next
        if (pair_left > 0) {
          x = 0;
          --pair_left;
        } else if (!flush && (order.left0 > 0 || order.left1 > 0)) {
          x = order.next();
          order.take(x);
        } else if (!flush && held0 && held1) {
          pair_left = pair_n;
          pair_n = 0;
          held0 = held1 = false;
          order = TileOrder();
          continue;
        } else if (!flush && w < 0) {
          if (!v_map) break;
          flush = true;
        }
        if (x < 0 && !flush) continue;
        const Tiles c = x == 1 ? cur1 : cur0;
        const bool pre = c.j < c.np;
        const int key = pre ? c.p_key + c.j * BN : c.o_key + (c.j - c.np) * BN;
        bool ok = true;
#pragma unroll 1
        for (int kv = 0; kv < 2 && ok; ++kv) {  // K of this tile, V of the one before
          if (kv == 0 ? x < 0 : v_map == nullptr) continue;
          ok = load(kv ? sV : sK, kv ? bar_v_full : bar_k_full, kv ? bar_v_empty : bar_k_empty,
                    kv ? v_map : pre ? &tm.kp : &tm.k, kv ? v_head : c.h, kv ? v_key : key, kv ? it - 1 : it);
        }
        if (!ok) break;
        v_map = nullptr;
        if (x < 0) continue;
        v_map = pre ? &tm.vp : &tm.v;
        v_key = key;
        v_head = c.h;
        if (x) ++cur1.j;
        else ++cur0.j;
        *const_cast<volatile int*>(&tiles_loaded) = ++it;
      }
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------- MMA issuer
    constexpr uint32_t idS = make_idesc_f16(kBF16, false, false, 128, BN);
    constexpr uint32_t idPV = make_idesc_f16(kBF16, false, true, 128, kD);
    const SmemDesc dq = smem_desc(smem_u32(sQ), 16, 1024, kLayoutSW128);
    const SmemDesc dk = smem_desc(smem_u32(sK), 16, 1024, kLayoutSW128);
    const SmemDesc dv = smem_desc(smem_u32(sV), BN * 128, 1024, kLayoutSW128);
    // Items on one stream: one copy of the code serves both streams; a turn of stream x issues
    // the product of its last tile and the scores of its next one. Such items are short, so
    // each passes through all of the code, and its length counts: with a copy per stream and
    // use the kernel was 163 KB long and every role ran at a third of its speed. Items on
    // both streams are long; their loop has a copy per stream (8 % faster).
    struct Stream {
      int n, j;                   // the item's key tiles, and those whose scores are issued
      int n_pre, p_left, o_left;  // as in PrefixItem
      int pend;                   // tile whose scores are issued, product not: its number; -1
      int real;                   // real keys of that tile
      bool first, last;           // it is its item's first or last one
      int np, no;                 // P hand-overs consumed; items whose O is accumulated
      int gets;                   // hand-overs taken (each used its Q tile once)
    };
    Stream s0{}, s1{};
    s0.pend = s1.pend = -1;
    bool held0 = false, held1 = false, ended0 = false, ended1 = NT == 1;
    int it = 0;  // key tiles so far: tile `it` is in stage it % NS
    TileOrder order;
    auto wait_k = [&](int tile) { return mbar_wait_warp(&bar_k_full[tile % NS], (tile / NS) & 1, status); };
    auto wait_v = [&](int tile) { return mbar_wait_warp(&bar_v_full[tile % NS], (tile / NS) & 1, status); };
    // P is there, and for an item's first product the last item's O is read
    auto wait_p = [&](int x, Stream& c, bool first) {
      if (!mbar_wait_warp(&bar_p_ready[x], c.np & 1, status)) return false;
      ++c.np;
      return !first || c.no == 0 || mbar_wait_warp(&bar_o_empty[x], (c.no - 1) & 1, status);
    };
    // The product takes a tile's keys by 16, as far as it has real ones; V rows behind the last
    // one become zeros there (P is 0, but 0 times NaN is not).
    auto zero_v = [&](int tile, int real) {
#pragma unroll 1
      for (int z = real * 8 + lane; z < (real + 15) / 16 * 128; z += 32)
#pragma unroll 1
        for (int k = 0; k < S::kChunks; ++k)
          st_shared_v4(sV + (tile % NS) * S::kKVBytes + k * BN * 128 + z * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
    };
    auto real_keys = [&](const Stream& c, int j) {
      return j < c.n_pre ? c.p_left - j * BN : c.o_left - (j - c.n_pre) * BN;
    };
    // (s: the stream, or with one stream the S tile)
    auto issue_pv = [&](int x, int s, int tile, bool first, int real) {
      const SmemDesc vst{dv.lo + (((tile % NS) * S::kKVBytes) >> 4), dv.hi};
      const uint32_t t_o = tmem + S::col_o(x), t_p = tmem + S::col_s(s), acc0 = first ? 0u : 1u;
      __syncwarp();  // elect.sync in the MMA wrappers needs a converged warp
      if (elect_one())
#pragma unroll
      for (int k = 0; k < BN / 16; ++k)
        if (16 * k < real) mma_ts_one(t_o, t_p + k * 8, vst, k * 2048, idPV, k > 0 ? 1u : acc0);
    };
    auto issue_s = [&](int x, int s, int tile) {
      const SmemDesc qx{dq.lo + ((x * S::kQBytes) >> 4), dq.hi};
      const SmemDesc kst{dk.lo + (((tile % NS) * S::kKVBytes) >> 4), dk.hi};
      const uint32_t t_s = tmem + S::col_s(s);
      __syncwarp();
      if (elect_one())
#pragma unroll
      for (int k = 0; k < kD / 16; ++k)
        mma_ss_one(t_s, qx, (k >> 2) * 16384 + (k & 3) * 32, kst, (k >> 2) * (BN * 128) + (k & 3) * 32, idS, k > 0 ? 1u : 0u);
      mma_commit(&bar_s_full[s]);
    };
    // An item on both streams: in round r both products of tile r - 1 and both scores of tile r.
    auto run_pair = [&]() -> bool {
      const int rounds = max(s0.n, s1.n);
      if (!mbar_wait_warp(&bar_q_full[0], (s0.gets - 1) & 1, status) ||
          !mbar_wait_warp(&bar_q_full[NT - 1], (s1.gets - 1) & 1, status))
        return false;
      if (s0.n == 0) mma_commit(&bar_q_empty[0]);
      if (s1.n == 0) mma_commit(&bar_q_empty[NT - 1]);
#pragma unroll 1
      for (int r = 0; r <= rounds; ++r) {
        bool v_ready = false, k_ready = false;
        auto turn = [&](auto x_tag, Stream& c) -> bool {
          constexpr int x = decltype(x_tag)::value;
          if (r > 0 && r <= c.n) {
            if (!wait_p(x, c, r == 1)) return false;
            const int real = real_keys(c, r - 1);
            if (!v_ready) {
              if (!wait_v(it + r - 1)) return false;
              if (real < BN) zero_v(it + r - 1, real);
              v_ready = true;
            }
            tc_fence_after();
            issue_pv(x, x, it + r - 1, r == 1, real);
          }
          if (r < c.n) {
            if (!k_ready && !wait_k(it + r)) return false;
            k_ready = true;
            tc_fence_after();
            issue_s(x, x, it + r);
            if (r + 1 == c.n) mma_commit(&bar_q_empty[x]);
          } else if (r == c.n && r > 0) {
            mma_commit(&bar_o_full[x]);
            ++c.no;
          }
          return true;
        };
        if (!turn(std::integral_constant<int, 0>{}, s0)) return false;
        if (!turn(std::integral_constant<int, NT - 1>{}, s1)) return false;
        if (r > 0) mma_commit(&bar_v_empty[(it + r - 1) % NS]);
        if (r < rounds) mma_commit(&bar_k_empty[(it + r) % NS]);
      }
      it += rounds;
      return true;
    };
    // One stream (head_dim above 128, O takes half of TMEM): within an item the scores run a
    // tile ahead of the products, into the other S tile.
    auto run_single = [&]() {
      for (int ii = 0;; ++ii) {
        const int sl = ii & 1;
        if (!mbar_wait_warp(&rings[0].full[sl], (ii >> 1) & 1, status)) return;
        const PrefixItem& I = rings[0].item[sl];
        Stream c{};
        c.n = I.n;
        c.n_pre = I.np;
        c.p_left = I.p_left;
        c.o_left = I.o_left;
        __syncwarp();
        mbar_arrive(&rings[0].empty[sl]);
        if (c.n < 0 || !mbar_wait_warp(&bar_q_full[0], ii & 1, status)) return;
        if (c.n == 0) mma_commit(&bar_q_empty[0]);
#pragma unroll 1
        for (int r = 0; r <= c.n; ++r) {
          if (r < c.n) {
            if (!wait_k(it + r)) return;
            tc_fence_after();
            issue_s(0, (it + r) & 1, it + r);
            mma_commit(&bar_k_empty[(it + r) % NS]);
            if (r + 1 == c.n) mma_commit(&bar_q_empty[0]);
          }
          if (r == 0) continue;
          const int t = it + r - 1;
          if (!mbar_wait_warp(&bar_p_ready[t & 1], (t >> 1) & 1, status)) return;
          if (r == 1 && s0.no > 0 && !mbar_wait_warp(&bar_o_empty[0], (s0.no - 1) & 1, status)) return;
          if (!wait_v(t)) return;
          const int real = real_keys(c, r - 1);
          if (real < BN) zero_v(t, real);
          tc_fence_after();
          issue_pv(0, t & 1, t, r == 1, real);
          mma_commit(&bar_v_empty[t % NS]);
          mma_commit(&bar_pv);
          if (r == c.n) {
            mma_commit(&bar_o_full[0]);
            ++s0.no;
          }
        }
        it += c.n;
      }
    };
    if constexpr (NT == 1) run_single();
    else
    for (;;) {
      const int w = order.wants(!held0 && !ended0, !held1 && !ended1);
      if (w >= 0) {
        const int gets = w ? s1.gets : s0.gets, sl = gets & 1;
        if (!mbar_wait_warp(&rings[w].full[sl], (gets >> 1) & 1, status)) break;
        const PrefixItem& I = rings[w].item[sl];
        const int n = I.n, n_pre = I.np, p_left = I.p_left, o_left = I.o_left;
        const bool pair = I.pair != 0;
        __syncwarp();
        mbar_arrive(&rings[w].empty[sl]);
        auto take = [&](Stream& c, bool& held, bool& ended) {
          ++c.gets;
          if (n < 0) {
            ended = true;
          } else {
            c.n = n;
            c.j = 0;
            c.n_pre = n_pre;
            c.p_left = p_left;
            c.o_left = o_left;
            if (pair) held = true;
          }
        };
        if (w) take(s1, held1, ended1);
        else take(s0, held0, ended0);
        if (n >= 0 && !pair) order.set(w, n);
      }
      // a stream acts while it has tiles to score or a product to issue
      const bool act0 = order.left0 > 0 || s0.pend >= 0, act1 = order.left1 > 0 || s1.pend >= 0;
      if (!act0 && !act1) {
        if (NT == 2 && held0 && held1) {
          if (!run_pair()) break;
          held0 = held1 = false;
          order = TileOrder();
        } else if (w < 0) {
          break;
        }
        continue;
      }
      const int x = (order.last == 1 ? act0 : act1) ? 1 - order.last : order.last;
      order.last = x;
      Stream c = NT == 2 && x ? s1 : s0;
      if (c.pend >= 0) {
        if (!wait_p(x, c, c.first) || !wait_v(c.pend)) break;
        if (c.real < BN) zero_v(c.pend, c.real);
        tc_fence_after();
        issue_pv(x, x, c.pend, c.first, c.real);
        mma_commit(&bar_v_empty[c.pend % NS]);
        if (c.last) {
          mma_commit(&bar_o_full[x]);
          ++c.no;
        }
        c.pend = -1;
      }
      if (order.left(x) > 0) {
        order.set(x, order.left(x) - 1);
        if (c.j == 0 && !mbar_wait_warp(&bar_q_full[x], (c.gets - 1) & 1, status)) break;
        if (!wait_k(it)) break;
        tc_fence_after();
        issue_s(x, x, it);
        mma_commit(&bar_k_empty[it % NS]);
        c.first = c.j == 0;
        c.real = real_keys(c, c.j);
        c.last = ++c.j == c.n;
        c.pend = it++;
        if (c.last) mma_commit(&bar_q_empty[x]);
      }
      if (NT == 2 && x) s1 = c;
      else s0 = c;
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int x = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_o = tmem + S::col_o(x) + lane_base;
    using T = typename std::conditional<kBF16, __nv_bfloat16, __half>::type;
    // A scale of 0 becomes the smallest positive one, which gives the same P (2^(S 1e-38) =
    // 1), so that the infinity put on a masked score below stays one.
    const float sl2 = p.scale_log2 == 0.f ? 1.17549435e-38f : p.scale_log2;
    const float masked = sl2 > 0.f ? -INFINITY : INFINITY;
    uint8_t* stage = sStage + warp * 2048;
    int ns = 0, no = 0;  // S hand-overs of this stream, and items with an output, so far
    bool ok = true;
#pragma unroll 1
    for (int ii = 0; ok; ++ii) {
      const int sl = ii & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&rings[x].full[sl], (ii >> 1) & 1, status));
      if (!ok) break;
      const PrefixItem& I = rings[x].item[sl];
      const int n = I.n, n_pre = I.np, p_left = I.p_left;
      const int r = quarter * 32 + lane;
      const bool in = n >= 0 && r < I.rows;
      const int row = in ? I.row[r] : -1, own = in ? I.lim[r] : 0;
      const bool direct = I.direct != 0;
      const size_t part = static_cast<size_t>(I.part) + quarter * 32;  // of the warp's first row
      mbar_arrive(&rings[x].empty[sl]);
      if (n < 0) break;
      const bool live = row >= 0;
      const bool alive = __any_sync(0xffffffffu, live);  // no row of this warp: only hand-overs
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int sb = NT == 1 ? ns & 1 : x;
        const uint32_t t_s = tmem + S::col_s(sb) + lane_base;
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_s_full[sb], (NT == 1 ? ns >> 1 : ns) & 1, status));
        if (!ok) break;
        ++ns;
        if (!alive) {
          mbar_arrive(&bar_p_ready[sb]);
          continue;
        }
        tc_fence_after();
        const int left = j < n_pre ? p_left - j * BN : own - (j - n_pre) * BN;
        // (a lane without a row masks nothing: an offset of infinity keeps its P at zero)
        const int nvalid = live ? min(max(left, 0), BN) : BN;
        // Tiles that some row does not see whole: its masked scores become -infinity (once
        // scaled) in TMEM, 32 columns at a time, and the rest of the code knows no masks.
        // These rare steps are rolled loops: unrolled, with a masked copy of the pass below,
        // the code outgrew the instruction cache and a block's first tile took 5000 cycles.
        if (!__all_sync(0xffffffffu, nvalid >= BN)) {
#pragma unroll 1
          for (int k = 0; k < BN; k += 32) {
            if (__all_sync(0xffffffffu, nvalid >= k + 32)) continue;
            uint32_t sv[32];
            tmem_ld32(t_s + k, sv);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c) sv[c] = k + c < nvalid ? sv[c] : __float_as_uint(masked);
            tmem_st16(t_s + k, *reinterpret_cast<uint32_t(*)[16]>(&sv[0]));
            tmem_st16(t_s + k + 16, *reinterpret_cast<uint32_t(*)[16]>(&sv[16]));
          }
          tmem_st_wait();
        }
        // Row max of the first `cols` columns (log2 domain), from S in TMEM.
        auto max_of = [&](int cols) -> float {
          float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int k = 0; k < cols; k += 32) {
            uint32_t sv[32];
            tmem_ld32(t_s + k, sv);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c)
              mp[c & 3] = max3(mp[c & 3], __uint_as_float(sv[2 * c]) * sl2, __uint_as_float(sv[2 * c + 1]) * sl2);
          }
          return fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]);
        };
        // A row's first tile with a visible key: the max of its first 32 scores starts the
        // offset m; should a later one exceed it by 2^8, the raise below catches it.
        if (__any_sync(0xffffffffu, live && m == -INFINITY && nvalid > 0)) {
          const float mxs = max_of(32);
          if (live && m == -INFINITY && nvalid > 0) m = mxs;
        }
        float alpha = 1.f;
        uint64_t sp[4];
        uint32_t pk[BN / 32][16];
        // a row that has seen no key yet: any finite offset makes its P zeros
        float neg = !live ? -INFINITY : m == -INFINITY ? 0.f : -m;
        bool again;
        do {  // (tested at its end only: the compiler keeps one copy of the pass)
          const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(neg, neg);
#pragma unroll
          for (int k = 0; k < 4; ++k) sp[k] = f2_pack(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < BN / 32; ++k) {
            uint32_t sv[32];
            tmem_ld32(t_s + 32 * k, sv);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 xx = f2_unpack(ffma2(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])),
                                                sl2x2, negm2));
              const float p0 = ex2p(xx.x), p1 = ex2p(xx.y);
              sp[c & 3] = fadd2(sp[c & 3], f2_pack(p0, p1));
              pk[k][c] = pack2<kBF16>(p0, p1);
            }
          }
          // a row whose P sums to at most 2^8 has no entry above 2^8: nothing to raise
          const float2 s01 = f2_unpack(fadd2(fadd2(sp[0], sp[1]), fadd2(sp[2], sp[3])));
          again = __any_sync(0xffffffffu, s01.x + s01.y > 256.0f);
          if (again) {
            const float mxs = max_of(BN);
            const bool raise = live && nvalid > 0 && mxs > m + 8.0f;
            again = __any_sync(0xffffffffu, raise);
            if (raise) {
              // a row without an earlier key has nothing to scale (and l is 0)
              alpha = m == -INFINITY ? 0.f : ex2p(m - mxs);
              m = mxs;
              neg = -mxs;
            }
          }
          // O has to be final for the tiles before this one. With two streams S(j) was issued
          // after P V(j-1), with one it may not be through. At the item's first tile there is
          // nothing to scale: the product will overwrite it.
          if (NT == 1 && again && j > 0) {
            ok = mbar_wait_warp(&bar_pv, ns & 1, status);  // product ns - 2 of all
            if (!ok) break;
            tc_fence_after();
          }
          if (again && j > 0) {
#pragma unroll 1
            for (int c0 = 0; c0 < kD; c0 += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c0, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st16(t_o + c0, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
              tmem_st16(t_o + c0 + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
            }
          }
        } while (again);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < BN / 32; ++k) tmem_st16(t_s + 16 * k, pk[k]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar_p_ready[sb]);
        const float2 s01 = f2_unpack(fadd2(fadd2(sp[0], sp[1]), fadd2(sp[2], sp[3])));
        l = l * alpha + (s01.x + s01.y);
      }
      if (!ok) break;
      if (n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_o_full[x], no & 1, status));
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      if (alive) {
        const uint32_t rows = __ballot_sync(0xffffffffu, live);
        // 64 bytes of every row at a time go through shared memory, so that a store
        // instruction writes eight rows' 64 bytes rather than 32 rows' 16: a 16-byte piece
        // of row r is kept at piece ^ (r / 2 % 4), which spreads both sides over all banks.
        auto store64 = [&](const uint32_t (&w)[16], auto&& put) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            st_shared_v4(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2],
                         w[4 * c + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (((rows >> (8 * k)) & 0xffu) == 0) continue;
            const int rr = 8 * k + (lane >> 2), c = lane & 3;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
            put(rr, c, v);
          }
          __syncwarp();
        };
        if (direct) {
          const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll 1
          for (int c0 = 0; c0 < p.d; c0 += 32) {
            uint32_t o[32], w[16];
            if (n > 0) {
              tmem_ld32(t_o + c0, o);
              tmem_ld_wait();
            }
            // a row without a key: zeros, whatever TMEM holds
#pragma unroll
            for (int c = 0; c < 16; ++c)
              w[c] = n > 0 && l != 0.f
                         ? pack2<kBF16>(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv)
                         : 0u;
            store64(w, [&](int rr, int c, const uint4& v) {
              const int at = __shfl_sync(0xffffffffu, row, rr);
              if (at >= 0 && c0 + 8 * c < p.d)
                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + static_cast<size_t>(at) * p.d + c0 + 8 * c) = v;
            });
          }
          if (live) p.lse[row] = l == 0.f ? -INFINITY : m * 0.69314718055994531f + logf(l);
        } else {
          if (live && bounds_ok(part + lane < static_cast<size_t>(p.cap_rows), status))
            p.part_ml[part + lane] = make_float2(m, l);
          if (n > 0) {
#pragma unroll 1
            for (int c0 = 0; c0 < p.d; c0 += 32) {
              uint32_t o[2][16];
              tmem_ld16(t_o + c0, o[0]);
              tmem_ld16(t_o + c0 + 16, o[1]);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 2; ++u)
                store64(o[u], [&](int rr, int c, const uint4& v) {
                  const int col = c0 + 16 * u + 4 * c;
                  if (((rows >> rr) & 1u) && col < p.d && bounds_ok(part + rr < static_cast<size_t>(p.cap_rows), status))
                    *reinterpret_cast<uint4*>(p.part_o + (part + rr) * p.d + col) = v;
                });
            }
          }
        }
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&bar_o_empty[x]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int kD, bool kBF16>
static cudaError_t launch_fwd_impl(const PrefixParams& p, int num_sms, cudaStream_t st) {
  using S = PrefixShape<kD>;
  PrefixMaps tm;
  // an absent tensor's map is never used: any valid address will do
  const void* any = p.total_kv > 0 ? p.k : p.kp;
  const bool own = p.total_kv > 0, pre = p.prefix_rows > 0;
  tm.q_tokens = 128 % p.group == 0 ? 128 / p.group : 0;
  const int whole = tm.q_tokens > 0 ? p.group : 1, token = p.group <= 128 ? p.group : 1;
  if (!make_tmap_tokens(&tm.k, own ? p.k : any, own ? p.total_kv : 1, 1, p.hkv, p.d, kBF16, S::kBN) ||
      !make_tmap_tokens(&tm.v, own ? p.v : any, own ? p.total_kv : 1, 1, p.hkv, p.d, kBF16, S::kBN) ||
      !make_tmap_tokens(&tm.kp, pre ? p.kp : any, pre ? p.prefix_rows : 1, 1, p.hkv, p.d, kBF16, S::kBN) ||
      !make_tmap_tokens(&tm.vp, pre ? p.vp : any, pre ? p.prefix_rows : 1, 1, p.hkv, p.d, kBF16, S::kBN) ||
      !make_tmap_tokens(&tm.q_tile, p.q, p.total_q, 1, p.hq, p.d, kBF16, 128, whole) ||
      !make_tmap_tokens(&tm.q_token, p.q, p.total_q, 1, p.hq, p.d, kBF16, token, token) ||
      !make_tmap_tokens(&tm.q_row, p.q, p.total_q, 1, p.hq, p.d, kBF16, 1, 1))
    return cudaErrorInvalidValue;
  auto kern = attn_prefix_fwd_kernel<kD, kBF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
  if (e != cudaSuccess) return e;
  const long long most = static_cast<long long>(p.cap_entries) * p.hkv;
  return launch_dependent(kern, static_cast<unsigned>(most < num_sms ? most : num_sms), S::kThreads, S::kSmemBytes, st,
                          p, tm);
}

cudaError_t launch_prefix_fwd(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st) {
  if (bf16) {
    if (p.d <= 64) return launch_fwd_impl<64, true>(p, num_sms, st);
    if (p.d <= 128) return launch_fwd_impl<128, true>(p, num_sms, st);
    return launch_fwd_impl<256, true>(p, num_sms, st);
  }
  if (p.d <= 64) return launch_fwd_impl<64, false>(p, num_sms, st);
  if (p.d <= 128) return launch_fwd_impl<128, false>(p, num_sms, st);
  return launch_fwd_impl<256, false>(p, num_sms, st);
}

// ---------------------------------------------------------------------------
// Join: rows that left partial results, and the rows that hold no token. Of a row's n
// partial rows, O = sum_k 2^(m_k - M) O_k / L with M = max m_k and L = sum_k 2^(m_k - M)
// l_k, in fp32 and in the order of k (per warp), rounded once. Latency-bound with few rows:
// then kWarps warps share a row's parts, four loads in flight each, and add up in shared
// memory; with many, one warp takes a row alone, or several heads of a token.
// ---------------------------------------------------------------------------
template <bool kBF16, int kWarps, int kCols>  // kCols: 128 or 256, at least d
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ PrefixParams p, int slices) {
  using T = typename std::conditional<kBF16, __nv_bfloat16, __half>::type;
  __shared__ float s_acc[kWarps > 1 ? 8 : 1][kWarps > 1 ? kCols : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % kWarps;  // this warp's share of a row's parts
  // (total_q * hq, and with it every count of rows here, is below 2^31)
  const uint32_t w = blockIdx.x * (8 / kWarps) + warp / kWarps;
  const bool any = w < static_cast<uint32_t>(p.total_q) * slices;
  const int t = any ? w / slices : 0, slice = any ? w % slices : 0;
  // several warps per row: one head each
  const int h0 = kWarps > 1 ? slice : static_cast<int>(static_cast<long long>(p.hq) * slice / slices);
  const int h1 = !any ? h0 : kWarps > 1 ? h0 + 1 : static_cast<int>(static_cast<long long>(p.hq) * (slice + 1) / slices);
  __shared__ int s_pad[kCachedOffsets];
  constexpr int kC = kCols / 128;
  constexpr int rt = prefix_row_tile(kCols), tile_shift = rt == 256 ? 8 : 7;
  int i = 0;
  const int b = locate_row(p, cache_offsets(p.cu_q_pad, p.batch, s_pad), t, &i);
  SeqInfo s{};
  if (b >= 0) s = load_seq(p, b);
  pdl_wait();  // the main kernel's results, and the scheduler's
  const int pre_chunks = p.header[kHdrPrefixChunks], pre_slot = p.header[kHdrPrefixSlot];
  const int pre_rows = p.header[kHdrPrefixRows];
  int4 info = make_int4(-1, -1, 0, 0);
  if (b >= 0) info = p.seqs[b];
  // -1 chunks: the lengths allow no result
  const bool real = b >= 0 && i < s.len_q && pre_chunks >= 0;
  if (kWarps == 1 && real && info.x < 0) {
    // a long sequence's token whose row tiles the main kernel wrote whole: nothing to do
    const int4 first = p.longs[info.w + i * p.group / rt], last = p.longs[info.w + (i * p.group + p.group - 1) / rt];
    if (p.group <= rt && first.x < 0 && first.y == 1 && last.x < 0 && last.y == 1) return;
  }
  // several warps per row: slices == hq, one head each, so the loop runs once for all
#pragma unroll 1
  for (int h = h0; h < (kWarps > 1 ? h0 + 1 : h1); ++h) {
    const size_t row = static_cast<size_t>(t) * p.hq + h;
    const int g = h / p.group, j = h - g * p.group;
    // the row's parts: na of row tile a (partial rows a0 + k astep), then nb of its own keys
    bool write = h < h1;
    int na = 0, nb = 0;
    int a0 = 0, astep = 0, b0 = 0, bstep = 0;  // (cap_rows is below 2^31)
    if (real && info.x < 0) {
      const int rr = i * p.group + j;
      const int4 tile = p.longs[info.w + (rr >> tile_shift)];
      write = write && (tile.x >= 0 || tile.y == 0);  // else the main kernel wrote it
      na = tile.y;
      a0 = tile.x + g * tile.z + (rr & (rt - 1));
      astep = p.hkv * tile.z;
    } else if (real) {
      if (pre_chunks > 0) {
        const int rr = (info.x + i) * p.group + j, u = rr >> tile_shift;
        const int rows = min(rt, pre_rows - u * rt);
        na = pre_chunks;
        a0 = pre_slot + u * rt * pre_chunks * p.hkv + g * rows + (rr & (rt - 1));
        astep = p.hkv * rows;
      }
      write = write && info.z >= 0;
      nb = max(info.z, 0);
      const int rows = s.len_q * p.group;
      b0 = info.y + (g * s.len_q + i) * p.group + j;
      bstep = p.hkv * rows;
    }
    const int n = write ? na + nb : 0;
    auto at = [&](int k) { return k < na ? a0 + k * astep : b0 + (k - na) * bstep; };
    // this warp's parts k, k + kWarps, ..., four at a time; the first four are on their way
    // before their weights are known (what a part without a visible key left is not used)
    float4 v[4][kC];
    auto load = [&](int k) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool some = k + u * kWarps < n;
        const float* src = p.part_o + static_cast<size_t>(some ? at(k + u * kWarps) : 0) * p.d;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const int col = 128 * c + 4 * lane;
          v[u][c] = some && col < p.d ? *reinterpret_cast<const float4*>(src + col) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    };
    load(sub);
    const float2 ml0 = lane < n ? p.part_ml[at(lane)] : make_float2(-INFINITY, 0.f);
    float M = ml0.y != 0.f ? ml0.x : -INFINITY;
#pragma unroll 1
    for (int k = lane + 32; k < n; k += 32) {
      const float2 ml = p.part_ml[at(k)];
      if (ml.y != 0.f) M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float acc[4 * kC] = {};
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += 32) {
      const float2 ml = k0 == 0 ? ml0 : k0 + lane < n ? p.part_ml[at(k0 + lane)] : make_float2(-INFINITY, 0.f);
      const float wgt = ml.y != 0.f ? ex2p(ml.x - M) : 0.f;
      L += wgt * ml.y;
#pragma unroll 1
      for (int k = sub; k < min(32, n - k0); k += 4 * kWarps) {
        if (k0 + k > sub) load(k0 + k);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float wk = __shfl_sync(0xffffffffu, wgt, (k + u * kWarps) & 31);
          if (wk == 0.f || k + u * kWarps >= 32) continue;
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            acc[4 * c] = fmaf(wk, v[u][c].x, acc[4 * c]);
            acc[4 * c + 1] = fmaf(wk, v[u][c].y, acc[4 * c + 1]);
            acc[4 * c + 2] = fmaf(wk, v[u][c].z, acc[4 * c + 2]);
            acc[4 * c + 3] = fmaf(wk, v[u][c].w, acc[4 * c + 3]);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if constexpr (kWarps > 1) {
#pragma unroll
      for (int c = 0; c < 4 * kC; ++c) s_acc[warp][(c >> 2) * 128 + 4 * lane + (c & 3)] = acc[c];
      __syncthreads();
      if (sub != 0) return;
#pragma unroll
      for (int o = 1; o < kWarps; ++o)
#pragma unroll
        for (int c = 0; c < 4 * kC; ++c) acc[c] += s_acc[warp + o][(c >> 2) * 128 + 4 * lane + (c & 3)];
    }
    if (!write) continue;
    const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = 128 * c + 4 * lane;
      if (col < p.d) {
        uint2 v;
        v.x = pack2<kBF16>(acc[4 * c] * inv, acc[4 * c + 1] * inv);
        v.y = pack2<kBF16>(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * p.d + col) = v;
      }
    }
    if (lane == 0) p.lse[row] = !real ? 0.f : L == 0.f ? -INFINITY : M * 0.69314718055994531f + logf(L);
  }
}

template <bool kBF16, int kCols>
static cudaError_t launch_join_impl(const PrefixParams& p, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.total_q) * p.hq, few = static_cast<long long>(num_sms) * 16;
  auto blocks = [](long long warps) { return static_cast<unsigned>((warps + 7) / 8); };
  if (rows * 4 <= few) {
    return launch_dependent(prefix_join_kernel<kBF16, 8, kCols>, blocks(rows * 8), 256, 0, st, p, p.hq);
  } else if (rows <= few) {
    return launch_dependent(prefix_join_kernel<kBF16, 4, kCols>, blocks(rows * 4), 256, 0, st, p, p.hq);
  } else {
    // one warp per row while that fills the GPU about twice over, several heads beyond it
    const long long want = (4 * few + p.total_q - 1) / p.total_q;
    const int slices = static_cast<int>(want < p.hq ? want : p.hq);
    return launch_dependent(prefix_join_kernel<kBF16, 1, kCols>, blocks(static_cast<long long>(p.total_q) * slices), 256, 0,
                            st, p, slices);
  }
}

cudaError_t launch_prefix_join(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st) {
  if (p.d <= 128) return bf16 ? launch_join_impl<true, 128>(p, num_sms, st) : launch_join_impl<false, 128>(p, num_sms, st);
  return bf16 ? launch_join_impl<true, 256>(p, num_sms, st) : launch_join_impl<false, 256>(p, num_sms, st);
}

}  // namespace teattn
