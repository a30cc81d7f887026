// Shared-prefix attention, forward.
//
//   S = scale [q Kp^T | q K_b^T + mask],  O = softmax(S) [Vp; V_b],  LSE = log sum exp S
//
// One persistent kernel takes items (group of rows, chunk of its key tiles, kv head); see
// attn_prefix.cuh for the groups. The rows of an item are the queries of one kv head's
// group packed token by token, so a decoding step of many sequences fills the 128-row
// tiles of the tensor cores against the prefix, and K/V tiles are read once for all of
// them. Roles as in the two-tile forward:
//   warps 0-3   softmax of row tile A (one thread per row / TMEM lane),
//   warps 4-7   softmax of row tile B (head_dim <= 128 only),
//   then        an item warp (decodes items and gathers their Q rows, an item ahead), a
//               K/V warp (TMA) and an MMA warp.
// An item of one row tile that leaves partial results is taken in turns: tile j of its keys
// goes to softmax group j % 2, each with its own O, so the chain S -> P -> O of one tile
// overlaps the other's (a decoding step's rows fill a few lanes only; the chain's latency,
// not its work, is what counts). Its Q rows use one half of the Q buffer, and the next
// such item's the other.
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
  pdl_trigger();
  const int rt = prefix_row_tile(p.d), bn = prefix_key_tile(p.d), tid = threadIdx.x, lane = tid & 31;
  const int most_ways = rt / 128;
  if (tid == 0) {
    bad = p.prefix_len && (*p.prefix_len < 0 || *p.prefix_len > p.prefix_rows) ? 1 : 0;
    work = tokens = 0;
  }
  const int np_keys = prefix_keys(p), np = div_up(np_keys, bn);
  __syncthreads();
  // sequences: compact tokens, long row tiles; an upper bound of the key tiles. With at
  // most a thread per sequence, `s` stays for the later phases.
  SeqInfo s{};
  int n_tok = 0, n_long = 0, first_tok = 0, first_long = 0;
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + tid;
    int tok = 0, nl = 0;
    unsigned long long w = 0, q = 0;
    s = SeqInfo{};
    if (b < p.batch) {
      s = load_seq(p, b);
      if (!s.ok) bad = 1;
      const int tiles = div_up(s.len_k, bn);
      const long long rows = static_cast<long long>(s.len_q) * p.group;
      q = s.len_q;
      if (rows > kShortRows) {
        nl = static_cast<int>((rows + rt - 1) / rt);
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
      for (int i = 0; i < tok; ++i)
        if (first_tok + i < p.total_q) p.short_tok[first_tok + i] = s.off_q + i;
    }
    n_tok += at.tx;
    n_long += at.ty;
  }
  // (the scans' barriers order the sums and the records above before what follows)
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
  // chunk length in key tiles: all heads' chunks together about parts_target * hkv
  const int len = static_cast<int>(max(1ull, (all + p.parts_target - 1) / p.parts_target));
  int n_entries = 0, n_rows = 0;  // running totals
  // Chunk c of a row tile with n key tiles in `chunks` chunks (they differ by one tile at
  // most), as entry `at`; e.slot: the row tile's first partial row.
  auto put_chunk = [&](PrefixEntry e, int n, int chunks, int c, int at) {
    const int q = n / chunks, r = n - q * chunks;
    e.t0 = c * q + min(c, r);
    e.t1 = e.t0 + q + (c < r ? 1 : 0);
    if (e.slot >= 0) e.slot += c * e.ways * p.hkv * e.rows;
    if (at < p.cap_entries) store_entry(p, at, e);
  };
  // long row tiles
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
      e.np = np;
      e.off_q = q.off_q;
      e.off_k = q.off_k;
      e.len_k = q.len_k;
      e.diag = q.diag;
      n = np + own_tiles(p, q.len_k, q.diag, e.row0, e.rows, bn);
      ch = div_up(n, len);
      e.ways = ch > 1 && e.rows <= rt / 2 ? most_ways : 1;
      slots = ch > 1 ? ch * e.ways * p.hkv * e.rows : 0;
    }
    const Scan3 at = block_scan3(ch, slots, 0, buf);
    if (g < n_long && g < p.cap_longs) {
      e.slot = slots > 0 ? n_rows + at.y : -1;
      p.longs[g] = make_int4(e.slot, ch * e.ways, e.rows, 0);
      for (int c = 0; c < ch; ++c) put_chunk(e, n, ch, c, n_entries + at.x + c);
    }
    n_entries += at.tx;
    n_rows += at.ty;
  }
  // the compact rows against the prefix, chunk-major: row tiles that read the same keys
  // are taken side by side
  const int pre_chunks = n_pre > 0 ? div_up(np, len) : 0;
  const int pre_slot = n_rows;
  for (int k = tid; k < n_pre * pre_chunks; k += blockDim.x) {
    const int c = k / n_pre, u = k - c * n_pre;
    PrefixEntry e{};
    e.seq = -1;
    e.row0 = u * rt;
    e.rows = min(rt, short_rows - e.row0);
    e.np = np;
    e.ways = e.rows <= rt / 2 ? most_ways : 1;
    e.slot = pre_slot + u * rt * pre_chunks * p.hkv;
    put_chunk(e, np, pre_chunks, c, n_entries + k);
  }
  n_entries += n_pre * pre_chunks;
  if (n_pre > 0) {
    const int last = short_rows - (n_pre - 1) * rt;
    n_rows += ((n_pre - 1) * rt + last * (last <= rt / 2 ? most_ways : 1)) * pre_chunks * p.hkv;
  }
  // short sequences against their own keys
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + tid;
    if (p.batch > blockDim.x) {  // otherwise this thread's sequence is still at hand
      s = SeqInfo{};
      first_tok = -1;
      if (b < p.batch) {
        s = load_seq(p, b);
        first_tok = p.seqs[b].x;
      }
    }
    PrefixEntry e{};
    int n = 0, ch = 0, slots = 0;
    if (b < p.batch && first_tok >= 0) {
      e.seq = b;
      e.rows = s.len_q * p.group;
      e.off_q = s.off_q;
      e.off_k = s.off_k;
      e.len_k = s.len_k;
      e.diag = s.diag;
      n = own_tiles(p, s.len_k, s.diag, 0, e.rows, bn);
      ch = div_up(n, len);
      // without a prefix a single tile is the whole result
      const bool direct = n == 1 && n_pre == 0;
      e.ways = direct ? 1 : most_ways;
      slots = direct ? 0 : ch * e.ways * p.hkv * e.rows;
    }
    const Scan3 at = block_scan3(ch, slots, 0, buf);
    if (ch > 0) {
      e.slot = slots > 0 ? n_rows + at.y : -1;
      p.seqs[b] = make_int4(first_tok, e.slot, slots > 0 ? ch * e.ways : -1, 0);
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
template <int kD>
struct PrefixShape {
  static constexpr int kNT = prefix_row_tile(kD) / 128;   // row tiles of an item
  static constexpr int kBN = prefix_key_tile(kD);          // keys per tile
  static constexpr int kChunks = kD / 64;                  // 64-column chunks of a row
  static constexpr int kQBytes = kChunks * 16384;          // one 128-row Q tile
  static constexpr int kKVBytes = kChunks * kBN * 128;     // one K or V tile
  static constexpr int kStages = kD == 64 ? 4 : 2;
  static constexpr int kSmemBytes = kNT * kQBytes + 2 * kStages * kKVBytes + 1024;
  static constexpr int kThreads = kNT * 128 + 96;
  // TMEM columns of O and S of row tile x: O_0 O_1 S_0 S_1
  __device__ static constexpr uint32_t col_o(int x) { return static_cast<uint32_t>(x) * 128u; }
  __device__ static constexpr uint32_t col_s(int x) { return 256u + static_cast<uint32_t>(x) * 128u; }
  static_assert(kSmemBytes <= 220 * 1024, "shared memory budget");
};

__device__ __forceinline__ float ex2p(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16-byte global -> shared copy; `bytes` 0 fills with zeros without reading.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// What the producer hands over with an item (two of them, in turn).
struct PrefixItem {
  int n[2];         // key tiles that softmax group 0 / 1 visits (0: none)
  int turns;        // 1: group x takes the key tiles x, x + 2, .. of one row tile
                    // 0: group x takes every key tile for row tile x
  int rows;         // rows of the item; the arrays below hold them rounded up to 32
  int half;         // half of the Q buffer that holds the rows; -1: both
  int np;           // the first np key tiles are the prefix's
  int p_key, o_key; // tensor rows of the first prefix key and the first own key
  int p_left;       // prefix keys from the item's first prefix tile on
  int o_left;       // own real keys from the item's first own tile on
  int direct;       // rows are written to out / lse, not to partial rows
  int head;         // kv head
  int part[2];      // partial row of the group's first row
  int row[256];     // per row: token * hq + head; -1: no row
  int lim[256];     // per row: own keys it sees from the item's first own tile on
};

template <int kD, bool kBF16>
__global__ void __launch_bounds__(PrefixShape<kD>::kThreads, 1)
    attn_prefix_fwd_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKp,
                           const __grid_constant__ CUtensorMap tmVp) {
  using S = PrefixShape<kD>;
  constexpr int NT = S::kNT, NS = S::kStages, BN = S::kBN;
  constexpr int kWarpItem = NT * 4, kWarpKv = NT * 4 + 1, kWarpMma = NT * 4 + 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + NT * S::kQBytes;
  uint8_t* sV = sK + NS * S::kKVBytes;

  __shared__ uint64_t bar_q_full[NT], bar_q_empty[NT];  // per 128-row half of the Q buffer
  __shared__ uint64_t bar_k_full[NS], bar_k_empty[NS], bar_v_full[NS], bar_v_empty[NS];
  __shared__ uint64_t bar_s_full[NT], bar_p_ready[NT], bar_o_full[NT], bar_o_empty[NT];
  __shared__ WorkRing ring;
  __shared__ PrefixItem items[2];
  __shared__ uint32_t tmem_slot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* status = p.header + kHdrStatus;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_v_empty[i], 1);
    }
    for (int x = 0; x < NT; ++x) {
      mbar_init(&bar_q_full[x], 32);
      mbar_init(&bar_q_empty[x], 1);
      mbar_init(&bar_s_full[x], 1);
      mbar_init(&bar_p_ready[x], 128);
      mbar_init(&bar_o_full[x], 1);
      mbar_init(&bar_o_empty[x], 128);
    }
    ring_init(ring, 1 + 32 + NT * 128);
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
  pdl_trigger();
  pdl_wait();  // the scheduler's lists

  if (warp == kWarpItem) {
    // ------------------------------------------------------------- items and Q rows
    // the first entry is read along with the number of entries (the grid is no larger than
    // the entries' capacity)
    PrefixEntry first = load_entry(p, blockIdx.x / p.hkv);
    const int n_items = p.header[kHdrPrefixEntries] * p.hkv;
    const int np_keys = prefix_keys(p);
    bool ok = true;
    int nxt = blockIdx.x;
    int uses[2] = {0, 0};  // items so far in each half of the Q buffer
    int half = 0;
    for (int ii = 0; ok; ++ii) {
      const int item = nxt < n_items ? nxt : -1;
      PrefixEntry e{};
      if (item >= 0) {
        if (lane == 0) nxt = next_item(p.header + kHdrNextFwd);
        e = ii == 0 ? first : load_entry(p, item / p.hkv);
        nxt = __shfl_sync(0xffffffffu, nxt, 0);
      }
      // the slot's last readers are done with it
      if (ii >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&ring.empty[ii & 1], ((ii >> 1) - 1) & 1, status));
      if (!ok) break;
      if (item < 0) {
        if (lane == 0) {
          *reinterpret_cast<volatile int*>(&ring.item[ii & 1]) = -1;
          mbar_arrive(&ring.full[ii & 1]);
        }
        break;
      }
      const int h = item % p.hkv;
      const int np = max(0, min(e.t1, e.np) - e.t0);  // prefix tiles of the chunk
      const int o0 = max(0, e.t0 - e.np);             // first own tile
      PrefixItem& I = items[ii & 1];
      // rows: where they lie and what they see (all loads of a batch in flight at once)
      constexpr int kPer = NT * 4;  // rows per lane
      int tok[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int r = u * 32 + lane, i = (e.row0 + r) / p.group;
        tok[u] = r >= e.rows ? -1 : e.seq < 0 ? p.short_tok[i] : e.off_q + i;
      }
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int r = u * 32 + lane;
        if (u * 32 >= e.rows) break;
        const int rr = e.row0 + r, i = rr / p.group, j = rr - i * p.group;
        const bool in = r < e.rows && bounds_ok(tok[u] >= 0 && tok[u] < p.total_q, status);
        I.row[r] = in ? tok[u] * p.hq + h * p.group + j : -1;
        I.lim[r] = in && e.seq >= 0 ? max(0, keys_seen(p.causal, e.len_k, e.diag, i) - o0 * BN) : 0;
      }
      // own tiles end at the last one that a row of the tile sees
      int n[2] = {0, 0};
      const bool turns = e.ways == 2;
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const int rows = min(128, e.rows - x * 128);
        if (rows > 0) {
          const int no = e.seq >= 0 ? own_tiles(p, e.len_k, e.diag, e.row0 + x * 128, rows, BN) : 0;
          n[x] = max(0, min(e.t1, e.np + no) - e.t0);
        }
      }
      if (turns) {
        n[1] = n[0] / 2;
        n[0] -= n[1];
      }
      const bool both = e.rows > 128;
      if (NT == 1) half = 0;
      if (lane == 0) {
        I.n[0] = n[0];
        I.n[1] = n[1];
        I.rows = e.rows;
        I.turns = turns ? 1 : 0;
        I.half = both ? -1 : half;
        I.np = np;
        I.p_key = e.t0 * BN;
        I.o_key = e.off_k + o0 * BN;
        I.p_left = np_keys - e.t0 * BN;
        I.o_left = e.len_k - o0 * BN;
        I.direct = e.slot < 0 ? 1 : 0;
        I.head = h;
        for (int x = 0; x < 2; ++x)
          I.part[x] = e.slot < 0 ? 0
                                 : e.slot + static_cast<int>(partial_offset(p, e.rows, turns ? x : 0, h)) +
                                       (turns ? 0 : x * 128);
        *reinterpret_cast<volatile int*>(&ring.item[ii & 1]) = item;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.full[ii & 1]);
      // Q rows, 16 bytes per lane and step, in the 128-byte swizzle the MMAs read;
      // columns from d on are filled with zeros. Rows past the last stay as they are:
      // they meet no other row.
      const int h0 = both ? 0 : half, h1 = both ? NT - 1 : half;
      for (int x = h0; x <= h1 && ok; ++x)
        if (uses[x] > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bar_q_empty[x], (uses[x] - 1) & 1, status));
      if (!ok) break;
      // (A lane keeps its column; addresses of eight rows are worked out before the copies,
      // which then issue back to back: one by one each took 130 cycles of this warp.)
      constexpr int kPieces = kD / 8, kRowsPer = 32 / (kPieces < 32 ? kPieces : 32);  // rows per step
      const int c = lane % kPieces, r_in = lane / kPieces;
      const bool col = c * 8 < p.d;
      const char* q_col = static_cast<const char*>(p.q) + c * 16;
      uint8_t* s_col = sQ + h0 * S::kQBytes + (c >> 3) * 16384;
      for (int r0 = 0; r0 < e.rows; r0 += 8 * kRowsPer) {
        const char* src[8];
        uint8_t* dst[8];
        int bytes[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = r0 + u * kRowsPer + r_in;
          const int row = r < e.rows ? I.row[r] : -1;
          bytes[u] = row >= 0 && col ? 16 : 0;
          src[u] = bytes[u] ? q_col + static_cast<size_t>(row) * (p.d * 2) : static_cast<const char*>(p.q);
          dst[u] = s_col + (r >> 7) * S::kQBytes + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (r0 + u * kRowsPer + r_in < e.rows) cp_async16(dst[u], src[u], bytes[u]);
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
      for (int x = h0; x <= h1; ++x) {
        mbar_arrive(&bar_q_full[x]);
        ++uses[x];
      }
      if (!both) half ^= 1;
    }
  } else if (warp == kWarpKv) {
    // ------------------------------------------------------------- K and V tiles
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmKp);
      tma_prefetch_desc(&tmVp);
      int it = 0;
      bool ok = true;
      for (int ii = 0; ok; ++ii) {
        const int sl = ii & 1;
        if (!(ok = mbar_wait(&ring.full[sl], (ii >> 1) & 1, status))) break;
        const int item = *reinterpret_cast<volatile int*>(&ring.item[sl]);
        const PrefixItem& I = items[sl];
        const int n = I.turns ? I.n[0] + I.n[1] : max(I.n[0], I.n[1]);
        const int np = I.np, p_key = I.p_key, o_key = I.o_key, h = I.head;
        mbar_arrive(&ring.empty[sl]);
        if (item < 0) break;
        for (int j = 0; j < n; ++j, ++it) {
          const int st = it % NS;
          const bool pre = j < np;
          const CUtensorMap* mk = pre ? &tmKp : &tmK;
          const CUtensorMap* mv = pre ? &tmVp : &tmV;
          const int key = pre ? p_key + j * BN : o_key + (j - np) * BN;
          if (it >= NS && !(ok = mbar_wait(&bar_k_empty[st], ((it / NS) - 1) & 1, status))) break;
          mbar_arrive_expect_tx(&bar_k_full[st], S::kKVBytes);
          for (int c = 0; c < S::kChunks; ++c)
            tma_load_4d(sK + st * S::kKVBytes + c * BN * 128, mk, &bar_k_full[st], c * 64, h, 0, key);
          if (it >= NS && !(ok = mbar_wait(&bar_v_empty[st], ((it / NS) - 1) & 1, status))) break;
          mbar_arrive_expect_tx(&bar_v_full[st], S::kKVBytes);
          for (int c = 0; c < S::kChunks; ++c)
            tma_load_4d(sV + st * S::kKVBytes + c * BN * 128, mv, &bar_v_full[st], c * 64, h, 0, key);
        }
      }
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------- MMA issuer
    constexpr uint32_t idS = make_idesc_f16(kBF16, false, false, 128, BN);
    constexpr uint32_t idPV = make_idesc_f16(kBF16, false, true, 128, kD);
    const SmemDesc dq = smem_desc(smem_u32(sQ), 16, 1024, kLayoutSW128);
    const SmemDesc dk = smem_desc(smem_u32(sK), 16, 1024, kLayoutSW128);
    const SmemDesc dv = smem_desc(smem_u32(sV), BN * 128, 1024, kLayoutSW128);
    int it = 0;
    int np[2] = {0, 0};    // P hand-overs consumed per softmax group
    int no[2] = {0, 0};    // items in which the group was present
    int uses[2] = {0, 0};  // items so far in each half of the Q buffer
    bool ok = true;
    for (int ii = 0; ok; ++ii) {
      const int sl = ii & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[sl], (ii >> 1) & 1, status));
      if (!ok) break;
      const int item = *reinterpret_cast<volatile int*>(&ring.item[sl]);
      const int n[2] = {items[sl].n[0], items[sl].n[1]};
      const bool turns = items[sl].turns != 0;
      const int half = items[sl].half;
      const int n_pre = items[sl].np, p_left = items[sl].p_left, o_left = items[sl].o_left;
      mbar_arrive(&ring.empty[sl]);
      if (item < 0) break;
      const int h0 = half < 0 ? 0 : half, h1 = half < 0 ? NT - 1 : half;
      for (int x = h0; x <= h1 && ok; ++x) ok = mbar_wait_warp(&bar_q_full[x], uses[x]++ & 1, status);
      if (!ok) break;
      auto run_item = [&](auto turns_tag) -> bool {
        constexpr bool kTurns = decltype(turns_tag)::value;
        int s_left = n[0] + n[1];  // scores still to be issued: then the Q rows are free
        // S_x = Q_x K^T for the item's key tile t
        auto issue_s = [&](int x, int t) {
          const int st = (it + t) % NS;
          const SmemDesc qx{dq.lo + (((half < 0 ? x : half) * S::kQBytes) >> 4), dq.hi};
          const SmemDesc kst{dk.lo + ((st * S::kKVBytes) >> 4), dk.hi};
          __syncwarp();  // elect.sync in the MMA wrappers needs a converged warp
#pragma unroll
          for (int s = 0; s < kD / 16; ++s)
            mma_ss(tmem + S::col_s(x), qx, (s >> 2) * 16384 + (s & 3) * 32, kst, (s >> 2) * (BN * 128) + (s & 3) * 32,
                   idS, s > 0 ? 1u : 0u);
          mma_commit(&bar_s_full[x]);
          if (kTurns) mma_commit(&bar_k_empty[st]);
          if (--s_left == 0)
            for (int y = h0; y <= h1; ++y) mma_commit(&bar_q_empty[y]);
        };
        auto wait_k = [&](int t) {
          const int cur = it + t;
          return mbar_wait_warp(&bar_k_full[cur % NS], (cur / NS) & 1, status);
        };
        const int rounds = max(n[0], n[1]);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (n[x] == 0) continue;
          const int t = kTurns ? x : 0;
          if (!wait_k(t)) return false;
          tc_fence_after();
          issue_s(x, t);
        }
        if (!kTurns) mma_commit(&bar_k_empty[it % NS]);
        for (int j = 0; j < rounds; ++j) {
          bool v_ready = false, k_ready = false;
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            if (j >= n[x]) continue;
            const int t = kTurns ? 2 * j + x : j, cur = it + t, st = cur % NS;
            if (!mbar_wait_warp(&bar_p_ready[x], np[x] & 1, status)) return false;
            ++np[x];
            if (j == 0 && no[x] > 0 && !mbar_wait_warp(&bar_o_empty[x], (no[x] - 1) & 1, status)) return false;
            if (kTurns || !v_ready) {
              if (!mbar_wait_warp(&bar_v_full[st], (cur / NS) & 1, status)) return false;
              v_ready = true;
              // V rows that are no real key: zeros (P is 0 there, but 0 times NaN is not)
              const int real = t < n_pre ? p_left - t * BN : o_left - (t - n_pre) * BN;
              if (real < BN) {
                for (int z = real * 8 + lane; z < BN * 8; z += 32)
                  for (int c = 0; c < S::kChunks; ++c)
                    st_shared_v4(sV + st * S::kKVBytes + c * BN * 128 + z * 16, 0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
            tc_fence_after();
            const SmemDesc vst{dv.lo + ((st * S::kKVBytes) >> 4), dv.hi};
            const uint32_t acc0 = j > 0 ? 1u : 0u;
            __syncwarp();
#pragma unroll
            for (int s = 0; s < BN / 16; ++s)
              mma_ts(tmem + S::col_o(x), tmem + S::col_s(x) + s * 8, vst, s * 2048, idPV, s > 0 ? 1u : acc0);
            if (kTurns) mma_commit(&bar_v_empty[st]);
            if (j + 1 < n[x]) {
              const int tn = kTurns ? t + 2 : t + 1;
              if (kTurns || !k_ready) {
                if (!wait_k(tn)) return false;
                k_ready = true;
              }
              tc_fence_after();
              issue_s(x, tn);
            } else {
              mma_commit(&bar_o_full[x]);
            }
          }
          if (!kTurns) {
            mma_commit(&bar_v_empty[(it + j) % NS]);
            if (j + 1 < rounds) mma_commit(&bar_k_empty[(it + j + 1) % NS]);
          }
        }
        it += kTurns ? n[0] + n[1] : rounds;
        return true;
      };
      ok = NT == 2 && turns ? run_item(std::true_type{}) : run_item(std::false_type{});
      if (!ok) break;
      for (int x = 0; x < NT; ++x)
        if (n[x] > 0) ++no[x];
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int x = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + S::col_s(x) + lane_base;
    const uint32_t t_o = tmem + S::col_o(x) + lane_base;
    using T = typename std::conditional<kBF16, __nv_bfloat16, __half>::type;
    // A scale of 0 becomes the smallest positive one, which gives the same P (2^(S 1e-38) =
    // 1), so that the infinity put on a masked score below stays one.
    const float sl2 = p.scale_log2 == 0.f ? 1.17549435e-38f : p.scale_log2;
    const float masked = sl2 > 0.f ? -INFINITY : INFINITY;
    int ns = 0, no = 0;  // S hand-overs and items of this tile so far
    bool ok = true;
    for (int ii = 0; ok; ++ii) {
      const int sl = ii & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[sl], (ii >> 1) & 1, status));
      if (!ok) break;
      const int item = *reinterpret_cast<volatile int*>(&ring.item[sl]);
      const int n = items[sl].n[x], n_pre = items[sl].np, p_left = items[sl].p_left;
      const int turns = items[sl].turns;
      // row of the item: with turns both groups hold the same rows
      const int r = (turns ? 0 : x * 128) + quarter * 32 + lane;
      const bool in = r < items[sl].rows;
      const int row = in ? items[sl].row[r] : -1, own = in ? items[sl].lim[r] : 0;
      const bool direct = items[sl].direct != 0;
      const size_t part = static_cast<size_t>(items[sl].part[x]) + quarter * 32 + lane;
      mbar_arrive(&ring.empty[sl]);
      if (item < 0) break;
      const bool live = row >= 0;
      const bool alive = __any_sync(0xffffffffu, live);  // no row of this warp: only hand-overs
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_s_full[x], ns & 1, status));
        if (!ok) break;
        ++ns;
        if (!alive) {
          mbar_arrive(&bar_p_ready[x]);
          continue;
        }
        tc_fence_after();
        const int t = turns ? 2 * j + x : j;
        const int left = t < n_pre ? p_left - t * BN : own - (t - n_pre) * BN;
        const int nvalid = live ? min(max(left, 0), BN) : 0;
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
        if (__any_sync(0xffffffffu, m == -INFINITY && nvalid > 0)) {
          const float mxs = max_of(32);
          if (m == -INFINITY && nvalid > 0) m = mxs;
        }
        float alpha = 1.f;
        uint64_t sp[4];
        uint32_t pk[BN / 32][16];
        // a row that has seen no key yet: any finite offset makes its P zeros
        const float off = m == -INFINITY ? 0.f : m;
        float neg = -off;
        for (;;) {
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
          if (!__any_sync(0xffffffffu, s01.x + s01.y > 256.0f)) break;
          const float mxs = max_of(BN);
          const bool raise = nvalid > 0 && mxs > m + 8.0f;
          if (!__any_sync(0xffffffffu, raise)) break;
          if (raise) {
            // a row without an earlier key has nothing to scale (and l is 0)
            alpha = m == -INFINITY ? 0.f : ex2p(m - mxs);
            m = mxs;
            neg = -mxs;
          }
          // S(j) was issued after P V(j-1): O is final for the tiles before this one. At the
          // item's first tile there is nothing to scale: the product will overwrite it.
          if (j > 0) {
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
        }
#pragma unroll
        for (int k = 0; k < BN / 32; ++k) tmem_st16(t_s + 16 * k, pk[k]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar_p_ready[x]);
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
      if (alive && direct) {
        const float inv = l > 0.f ? 1.0f / l : 0.f;
        const size_t row_at = static_cast<size_t>(live ? row : 0);
        const auto rows = make_row_pair(static_cast<T*>(p.out) + row_at * p.d, live);
#pragma unroll
        for (int c0 = 0; c0 < kD; c0 += 16) {
          uint32_t o[16];
          if (n > 0) {
            tmem_ld16(t_o + c0, o);
            tmem_ld_wait();
          }
          // a row without a key: zeros, whatever TMEM holds
#pragma unroll
          for (int c = 0; c < 16; ++c) o[c] = n > 0 && l > 0.f ? o[c] : 0u;
          store_pair16<kBF16>(rows, c0, p.d, o, inv);
        }
        if (live) p.lse[row_at] = l > 0.f ? m * 0.69314718055994531f + logf(l) : -INFINITY;
      } else if (alive) {
        if (live && bounds_ok(part < static_cast<size_t>(p.cap_rows), status)) {
          p.part_ml[part] = make_float2(m, l);
        }
        if (n > 0) {
          float* dst = p.part_o + part * p.d;
#pragma unroll
          for (int c0 = 0; c0 < kD; c0 += 16) {
            uint32_t o[16];
            tmem_ld16(t_o + c0, o);
            tmem_ld_wait();
            if (live && bounds_ok(part < static_cast<size_t>(p.cap_rows), status)) {
#pragma unroll
              for (int c = 0; c < 16; c += 4)
                if (c0 + c < p.d)
                  *reinterpret_cast<uint4*>(dst + c0 + c) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
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
  CUtensorMap tk, tv, tkp, tvp;
  // an absent tensor's map is never used: any valid address will do
  const void* any = p.total_kv > 0 ? p.k : p.kp;
  const bool own = p.total_kv > 0, pre = p.prefix_rows > 0;
  if (!make_tmap_tokens(&tk, own ? p.k : any, own ? p.total_kv : 1, 1, p.hkv, p.d, kBF16, S::kBN) ||
      !make_tmap_tokens(&tv, own ? p.v : any, own ? p.total_kv : 1, 1, p.hkv, p.d, kBF16, S::kBN) ||
      !make_tmap_tokens(&tkp, pre ? p.kp : any, pre ? p.prefix_rows : 1, 1, p.hkv, p.d, kBF16, S::kBN) ||
      !make_tmap_tokens(&tvp, pre ? p.vp : any, pre ? p.prefix_rows : 1, 1, p.hkv, p.d, kBF16, S::kBN))
    return cudaErrorInvalidValue;
  auto kern = attn_prefix_fwd_kernel<kD, kBF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
  if (e != cudaSuccess) return e;
  const long long most = static_cast<long long>(p.cap_entries) * p.hkv;
  return launch_dependent(kern, static_cast<unsigned>(most < num_sms ? most : num_sms), S::kThreads, S::kSmemBytes, st,
                          p, tk, tv, tkp, tvp);
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
template <bool kBF16, int kWarps>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ PrefixParams p, int slices) {
  using T = typename std::conditional<kBF16, __nv_bfloat16, __half>::type;
  __shared__ float s_acc[kWarps > 1 ? 8 : 1][kWarps > 1 ? 256 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % kWarps;  // this warp's share of a row's parts
  const long long w = static_cast<long long>(blockIdx.x) * (8 / kWarps) + warp / kWarps;
  const bool any = w < static_cast<long long>(p.total_q) * slices;
  const int t = any ? static_cast<int>(w / slices) : 0, slice = any ? static_cast<int>(w % slices) : 0;
  const int h0 = static_cast<int>(static_cast<long long>(p.hq) * slice / slices);
  const int h1 = any ? static_cast<int>(static_cast<long long>(p.hq) * (slice + 1) / slices) : h0;
  __shared__ int s_pad[kCachedOffsets];
  const int rt = prefix_row_tile(p.d);
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
  for (int h = h0; h < (kWarps > 1 ? h0 + 1 : h1); ++h) {
    const size_t row = static_cast<size_t>(t) * p.hq + h;
    const int g = h / p.group, j = h - g * p.group;
    // the row's parts: na of row tile a (partial rows a0 + k astep), then nb of its own keys
    bool write = h < h1;
    int na = 0, nb = 0;
    size_t a0 = 0, astep = 0, b0 = 0, bstep = 0;
    if (real && info.x < 0) {
      const int rr = i * p.group + j;
      const int4 tile = p.longs[info.w + rr / rt];
      write = write && (tile.x >= 0 || tile.y == 0);  // else the main kernel wrote it
      na = tile.y;
      a0 = static_cast<size_t>(tile.x) + partial_offset(p, tile.z, 0, g) + rr % rt;
      astep = partial_offset(p, tile.z, 1, 0);
    } else if (real) {
      if (pre_chunks > 0) {
        const int rr = (info.x + i) * p.group + j, u = rr / rt;
        const int rows = min(rt, pre_rows - u * rt);
        na = pre_chunks * (rows <= rt / 2 ? rt / 128 : 1);
        a0 = static_cast<size_t>(pre_slot) + static_cast<size_t>(u) * rt * pre_chunks * p.hkv +
             partial_offset(p, rows, 0, g) + rr % rt;
        astep = partial_offset(p, rows, 1, 0);
      }
      write = write && info.z >= 0;
      nb = max(info.z, 0);
      const int rows = s.len_q * p.group;
      b0 = static_cast<size_t>(info.y) + partial_offset(p, rows, 0, g) + i * p.group + j;
      bstep = partial_offset(p, rows, 1, 0);
    }
    const int n = write ? na + nb : 0;
    auto at = [&](int k) { return k < na ? a0 + k * astep : b0 + (k - na) * bstep; };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) {
      const float2 ml = p.part_ml[at(k)];
      if (ml.y > 0.f) M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float acc[8] = {};
    for (int k0 = 0; k0 < n; k0 += 32) {
      float wgt = 0.f;
      if (k0 + lane < n) {
        const float2 ml = p.part_ml[at(k0 + lane)];
        // a part without a visible key left no output
        wgt = ml.y > 0.f ? ex2p(ml.x - M) : 0.f;
        L += wgt * ml.y;
      }
      uint32_t todo = __ballot_sync(0xffffffffu, wgt != 0.f && (k0 + lane) % kWarps == sub);
      while (todo) {
        float wk[4];
        float4 v[4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = todo ? __ffs(todo) - 1 : 0;
          const float ww = __shfl_sync(0xffffffffu, wgt, k);
          wk[u] = todo ? ww : 0.f;
          const float* src = p.part_o + at(k0 + k) * p.d;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = 128 * c + 4 * lane;
            v[u][c] = todo && col < p.d ? *reinterpret_cast<const float4*>(src + col) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          todo &= todo - 1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            acc[4 * c] = fmaf(wk[u], v[u][c].x, acc[4 * c]);
            acc[4 * c + 1] = fmaf(wk[u], v[u][c].y, acc[4 * c + 1]);
            acc[4 * c + 2] = fmaf(wk[u], v[u][c].z, acc[4 * c + 2]);
            acc[4 * c + 3] = fmaf(wk[u], v[u][c].w, acc[4 * c + 3]);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if constexpr (kWarps > 1) {
#pragma unroll
      for (int c = 0; c < 8; ++c) s_acc[warp][(c >> 2) * 128 + 4 * lane + (c & 3)] = acc[c];
      __syncthreads();
      if (sub != 0) return;
#pragma unroll
      for (int o = 1; o < kWarps; ++o)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] += s_acc[warp + o][(c >> 2) * 128 + 4 * lane + (c & 3)];
    }
    if (!write) continue;
    const float inv = L > 0.f ? 1.0f / L : 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = 128 * c + 4 * lane;
      if (col < p.d) {
        uint2 v;
        v.x = pack2<kBF16>(acc[4 * c] * inv, acc[4 * c + 1] * inv);
        v.y = pack2<kBF16>(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * p.d + col) = v;
      }
    }
    if (lane == 0) p.lse[row] = !real ? 0.f : L > 0.f ? M * 0.69314718055994531f + logf(L) : -INFINITY;
  }
}

template <bool kBF16>
static cudaError_t launch_join_impl(const PrefixParams& p, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.total_q) * p.hq, few = static_cast<long long>(num_sms) * 16;
  auto blocks = [](long long warps) { return static_cast<unsigned>((warps + 7) / 8); };
  if (rows * 4 <= few) {
    return launch_dependent(prefix_join_kernel<kBF16, 8>, blocks(rows * 8), 256, 0, st, p, p.hq);
  } else if (rows <= few) {
    return launch_dependent(prefix_join_kernel<kBF16, 4>, blocks(rows * 4), 256, 0, st, p, p.hq);
  } else {
    // one warp per row while that fills the GPU about twice over, several heads beyond it
    const long long want = (4 * few + p.total_q - 1) / p.total_q;
    const int slices = static_cast<int>(want < p.hq ? want : p.hq);
    return launch_dependent(prefix_join_kernel<kBF16, 1>, blocks(static_cast<long long>(p.total_q) * slices), 256, 0,
                            st, p, slices);
  }
}

cudaError_t launch_prefix_join(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? launch_join_impl<true>(p, num_sms, st) : launch_join_impl<false>(p, num_sms, st);
}

}  // namespace teattn
