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
//   then        one producer warp (gathers the Q rows, TMA for K and V) and one MMA warp.
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
#include "row_store.cuh"
#include "sm103_ptx.cuh"
#include "tmap.h"
#include "work_queue.cuh"

namespace teattn {

// ---------------------------------------------------------------------------
// Scheduler: one block; from the lengths to groups, chunks and partial rows. It is a few
// passes over the sequences with block-wide scans; the result depends on lengths only.
// ---------------------------------------------------------------------------
constexpr int kPrefixSchedThreads = 512;

// Exclusive scan of two counters at once over the block; totals in *tx, *ty.
__device__ __forceinline__ int2 block_scan2(int x, int y, unsigned long long* warp_sums, int* tx, int* ty) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const unsigned long long own = static_cast<unsigned long long>(static_cast<unsigned>(x)) |
                                 (static_cast<unsigned long long>(static_cast<unsigned>(y)) << 32);
  unsigned long long v = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  unsigned long long before = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    const unsigned long long s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  __syncthreads();
  v += before - own;
  *tx = static_cast<int>(total & 0xffffffffu);
  *ty = static_cast<int>(total >> 32);
  return make_int2(static_cast<int>(v & 0xffffffffu), static_cast<int>(v >> 32));
}

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// Own key tiles that the rows [row0, row0 + rows) of sequence s see.
__device__ __forceinline__ int own_tiles(const PrefixParams& p, const SeqInfo& s, int row0, int rows, int bn) {
  const int last = (row0 + rows - 1) / p.group;
  return div_up(row_keys(s, last, p.causal != 0), bn);
}

__global__ void __launch_bounds__(kPrefixSchedThreads) prefix_schedule_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ unsigned long long warp_sums[32];
  __shared__ int bad;
  __shared__ unsigned long long work, tokens;
  const int rt = prefix_row_tile(p.d), bn = prefix_key_tile(p.d), tid = threadIdx.x;
  const int np_keys = prefix_keys(p), np = div_up(np_keys, bn);
  if (tid == 0) {
    bad = p.prefix_len && (*p.prefix_len < 0 || *p.prefix_len > p.prefix_rows) ? 1 : 0;
    work = tokens = 0;
  }
  __syncthreads();
  // sequences: compact tokens, own groups, long groups; an upper bound of the key tiles
  int n_tok = 0, n_long = 0;
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + tid;
    int tok = 0, nl = 0;
    if (b < p.batch) {
      const SeqInfo s = load_seq(p, b);
      if (!s.ok) bad = 1;
      const int tiles = div_up(s.len_k, bn);
      const long long rows = static_cast<long long>(s.len_q) * p.group;
      atomicAdd(&tokens, static_cast<unsigned long long>(s.len_q));
      if (rows > kShortRows) {
        nl = static_cast<int>((rows + rt - 1) / rt);
        atomicAdd(&work, static_cast<unsigned long long>(nl) * (np + tiles));
      } else if (rows > 0) {
        tok = s.len_q;
        atomicAdd(&work, static_cast<unsigned long long>(tiles));
      }
    }
    int t0, t1;
    const int2 at = block_scan2(tok, nl, warp_sums, &t0, &t1);
    if (b < p.batch) {
      p.seqs[b] = make_int4(tok > 0 ? n_tok + at.x : -1, -1, nl > 0 ? n_long + at.y : -1, n_long + at.y);
      if (tok > 0) {
        const int row = p.cu_q_pad[b];
        for (int i = 0; i < tok; ++i)
          if (n_tok + at.x + i < p.total_q) p.short_tok[n_tok + at.x + i] = row + i;
      }
    }
    n_tok += t0;
    n_long += t1;
  }
  __syncthreads();
  if (tokens > static_cast<unsigned long long>(p.total_q)) {
    // sequences overlap: more tokens than rows, for which the lists have no room
    if (tid == 0) {
      p.header[kHdrStatus] = kStatusBadSeqlens;
      p.header[kHdrPrefixEntries] = 0;
      p.header[kHdrPrefixFirst] = -2;
      p.header[kHdrNextFwd] = 0;
    }
    return;
  }
  const int short_rows = n_tok * p.group;  // at most 128 per sequence
  const int n_pre = np > 0 ? div_up(short_rows, rt) : 0;
  const unsigned long long all = work + static_cast<unsigned long long>(n_pre) * np;
  // chunk length in key tiles: all heads' chunks together about parts_target * hkv
  const int len = static_cast<int>(max(1ull, (all + p.parts_target - 1) / p.parts_target));
  int n_groups = 0, n_entries = 0, n_rows = 0;  // running totals
  // long groups
  for (int base = 0; base < n_long; base += blockDim.x) {
    const int e = base + tid;
    PrefixGroup g{};
    int ch = 0, slots = 0;
    if (e < n_long) {
      int lo = 0, hi = p.batch - 1;  // last sequence whose first long group is at most e
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.seqs[mid].w <= e) lo = mid; else hi = mid - 1;
      }
      const SeqInfo s = load_seq(p, lo);
      const int u = e - p.seqs[lo].w;
      g.seq = lo;
      g.row0 = u * rt;
      g.rows = min(rt, s.len_q * p.group - g.row0);
      g.np = np;
      g.no = own_tiles(p, s, g.row0, g.rows, bn);
      g.chunks = ch = div_up(g.np + g.no, len);
      g.is_long = 1;
      slots = ch > 1 ? ch * p.hkv * g.rows : 0;
    }
    int t0, t1;
    const int2 at = block_scan2(ch, slots, warp_sums, &t0, &t1);
    if (e < n_long && n_groups + tid < p.cap_groups) {
      g.slot = slots > 0 ? n_rows + at.y : -1;
      store_group(p, e, g);
      for (int c = 0; c < ch; ++c)
        if (n_entries + at.x + c < p.cap_entries) p.entries[n_entries + at.x + c] = make_int2(e, c);
    }
    n_groups += min(static_cast<int>(blockDim.x), n_long - base);
    n_entries += t0;
    n_rows += t1;
  }
  // prefix groups, chunk-major: row tiles that read the same keys are taken side by side
  const int pre_chunks = n_pre > 0 ? div_up(np, len) : 0;
  for (int u = tid; u < n_pre; u += blockDim.x) {
    PrefixGroup g{};
    g.seq = -1;
    g.row0 = u * rt;
    g.rows = min(rt, short_rows - g.row0);
    g.np = np;
    g.chunks = pre_chunks;
    g.slot = n_rows + u * rt * pre_chunks * p.hkv;
    if (n_groups + u < p.cap_groups) store_group(p, n_groups + u, g);
    for (int c = 0; c < pre_chunks; ++c) {
      const int at = n_entries + c * n_pre + u;
      if (at < p.cap_entries) p.entries[at] = make_int2(n_groups + u, c);
    }
  }
  const int first_pre = n_groups;
  n_groups += n_pre;
  n_entries += n_pre * pre_chunks;
  n_rows += short_rows * pre_chunks * p.hkv;
  // own groups of short sequences
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + tid;
    PrefixGroup g{};
    int ch = 0, slots = 0, has = 0;
    if (b < p.batch && p.seqs[b].x >= 0) {
      const SeqInfo s = load_seq(p, b);
      g.seq = b;
      g.rows = s.len_q * p.group;
      g.no = own_tiles(p, s, 0, g.rows, bn);
      g.chunks = ch = div_up(g.no, len);
      has = ch > 0 ? 1 : 0;
      // without a prefix a single chunk is the whole result
      slots = ch > 1 || n_pre > 0 ? ch * p.hkv * g.rows : 0;
    }
    int t0, t1, t2, t3;
    const int2 at = block_scan2(ch, slots, warp_sums, &t0, &t1);
    const int2 ag = block_scan2(has, 0, warp_sums, &t2, &t3);
    if (has && n_groups + ag.x < p.cap_groups) {
      const int e = n_groups + ag.x;
      g.slot = slots > 0 ? n_rows + at.y : -1;
      store_group(p, e, g);
      p.seqs[b].y = e;
      for (int c = 0; c < ch; ++c)
        if (n_entries + at.x + c < p.cap_entries) p.entries[n_entries + at.x + c] = make_int2(e, c);
    }
    n_groups += t2;
    n_entries += t0;
    n_rows += t1;
  }
  __syncthreads();
  if (tid == 0) {
    // the capacities hold for every set of lengths; if they did not, nothing is computed
    const bool over = n_groups > p.cap_groups || n_entries > p.cap_entries || n_rows > p.cap_rows;
    p.header[kHdrStatus] = (bad ? kStatusBadSeqlens : 0) | (over ? kStatusInternal : 0);
    p.header[kHdrPrefixEntries] = over ? 0 : n_entries;
    p.header[kHdrPrefixFirst] = over ? -2 : n_pre > 0 ? first_pre : -1;
    p.header[kHdrNextFwd] = 0;
  }
}

cudaError_t launch_prefix_schedule(const PrefixParams& p, cudaStream_t st) {
  prefix_schedule_kernel<<<1, kPrefixSchedThreads, 0, st>>>(p);
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
  static constexpr int kThreads = kNT * 128 + 64;
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
  int n[2];         // key tiles that row tile A / B visits (0: none)
  int np;           // the first np of them are prefix tiles
  int p_left;       // prefix keys from the item's first prefix tile on
  int o_left;       // own real keys from the item's first own tile on
  int direct;       // rows are written to out / lse, not to partial rows
  int head;         // kv head
  int row[256];     // per row: token * hq + head; -1: no row
  int lim[256];     // per row: own keys it sees from the item's first own tile on
  int part;         // partial row of row 0
};

template <int kD, bool kBF16>
__global__ void __launch_bounds__(PrefixShape<kD>::kThreads, 1)
    attn_prefix_fwd_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKp,
                           const __grid_constant__ CUtensorMap tmVp) {
  using S = PrefixShape<kD>;
  constexpr int NT = S::kNT, NS = S::kStages, BN = S::kBN;
  constexpr int kWarpProducer = NT * 4, kWarpMma = NT * 4 + 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + NT * S::kQBytes;
  uint8_t* sV = sK + NS * S::kKVBytes;

  __shared__ uint64_t bar_q_full, bar_q_empty;
  __shared__ uint64_t bar_k_full[NS], bar_k_empty[NS], bar_v_full[NS], bar_v_empty[NS];
  __shared__ uint64_t bar_s_full[NT], bar_p_ready[NT], bar_o_full[NT], bar_o_empty[NT];
  __shared__ WorkRing ring;
  __shared__ PrefixItem items[2];
  __shared__ uint32_t tmem_slot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* status = p.header + kHdrStatus;

  if (tid == 0) {
    mbar_init(&bar_q_full, 32);
    mbar_init(&bar_q_empty, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_v_empty[i], 1);
    }
    for (int x = 0; x < NT; ++x) {
      mbar_init(&bar_s_full[x], 1);
      mbar_init(&bar_p_ready[x], 128);
      mbar_init(&bar_o_full[x], 1);
      mbar_init(&bar_o_empty[x], 128);
    }
    ring_init(ring, 32 + NT * 128);
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

  if (warp == kWarpProducer) {
    // ------------------------------------------------------------- producer
    const int n_items = p.header[kHdrPrefixEntries] * p.hkv;
    const int np_keys = prefix_keys(p);
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmKp);
      tma_prefetch_desc(&tmVp);
    }
    int it = 0;
    bool ok = true;
    int nxt = blockIdx.x;
    for (int ii = 0; ok; ++ii) {
      const int item = nxt < n_items ? nxt : -1;
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
      if (lane == 0) nxt = next_item(p.header + kHdrNextFwd);
      nxt = __shfl_sync(0xffffffffu, nxt, 0);
      const int2 en = p.entries[item / p.hkv];
      const int h = item % p.hkv;
      const PrefixGroup g = load_group(p, en.x);
      const int2 ct = chunk_tiles(g, en.y);
      SeqInfo s{};
      if (g.seq >= 0) s = load_seq(p, g.seq);
      const int p0 = ct.x, np = max(0, min(ct.y, g.np) - ct.x);  // prefix tiles of the chunk
      const int o0 = max(0, ct.x - g.np);                        // first own tile
      PrefixItem& I = items[ii & 1];
      // rows
      for (int r = lane; r < NT * 128; r += 32) {
        int row = -1, lim = 0;
        if (r < g.rows) {
          const int rr = g.row0 + r, i = rr / p.group, j = rr - i * p.group;
          const int tok = g.seq < 0 ? p.short_tok[i] : s.off_q + i;
          row = tok * p.hq + h * p.group + j;
          if (g.seq >= 0) lim = max(0, row_keys(s, i, p.causal != 0) - o0 * BN);
          if (!bounds_ok(tok >= 0 && tok < p.total_q, status)) row = -1;
        }
        I.row[r] = row;
        I.lim[r] = lim;
      }
      // own tiles end at the last one that a row of the tile sees
      int n[2] = {0, 0};
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const int rows = min(128, g.rows - x * 128);
        if (rows > 0) {
          const int no = g.seq >= 0 ? own_tiles(p, s, g.row0 + x * 128, rows, BN) : 0;
          n[x] = max(0, min(ct.y, g.np + no) - ct.x);
        }
      }
      const int nmax = max(n[0], n[1]);
      if (lane == 0) {
        I.n[0] = n[0];
        I.n[1] = n[1];
        I.np = np;
        I.p_left = np_keys - p0 * BN;
        I.o_left = s.len_k - o0 * BN;
        I.direct = g.slot < 0 ? 1 : 0;
        I.head = h;
        I.part = g.slot < 0 ? 0 : static_cast<int>(partial_row(p, g, en.y, h, 0));
        *reinterpret_cast<volatile int*>(&ring.item[ii & 1]) = item;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.full[ii & 1]);
      if (ii > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bar_q_empty, (ii - 1) & 1, status));
      if (!ok) break;
      // Q rows, 16 bytes per lane and step, in the 128-byte swizzle the MMAs read;
      // columns from d on are filled with zeros. Rows past the last stay as they are:
      // they meet no other row.
      constexpr int kPieces = kD / 8;
      const int pieces = g.rows * kPieces;
      for (int t = lane; t < pieces; t += 32) {
        const int r = t / kPieces, c = t % kPieces;
        const int row = I.row[r];
        const bool in = row >= 0 && c * 8 < p.d;
        const char* src = static_cast<const char*>(p.q) +
                          (in ? (static_cast<size_t>(row) * p.d + c * 8) * 2 : static_cast<size_t>(0));
        uint8_t* dst = sQ + (r >> 7) * S::kQBytes + (c >> 3) * 16384 + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4);
        cp_async16(dst, src, in ? 16 : 0);
      }
      for (int j = 0; j < nmax; ++j, ++it) {
        const int st = it % NS;
        if (lane == 0) {
          const bool pre = j < np;
          const CUtensorMap* mk = pre ? &tmKp : &tmK;
          const CUtensorMap* mv = pre ? &tmVp : &tmV;
          const int key = pre ? (p0 + j) * BN : s.off_k + (o0 + j - np) * BN;
          if (it >= NS) ok = mbar_wait(&bar_k_empty[st], ((it / NS) - 1) & 1, status);
          if (ok) {
            mbar_arrive_expect_tx(&bar_k_full[st], S::kKVBytes);
            for (int c = 0; c < S::kChunks; ++c)
              tma_load_4d(sK + st * S::kKVBytes + c * BN * 128, mk, &bar_k_full[st], c * 64, h, 0, key);
            if (it >= NS) ok = mbar_wait(&bar_v_empty[st], ((it / NS) - 1) & 1, status);
          }
          if (ok) {
            mbar_arrive_expect_tx(&bar_v_full[st], S::kKVBytes);
            for (int c = 0; c < S::kChunks; ++c)
              tma_load_4d(sV + st * S::kKVBytes + c * BN * 128, mv, &bar_v_full[st], c * 64, h, 0, key);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        if (j == 0) {
          // the first K and V tiles are on their way: now the Q rows
          cp_async_wait_all();
          fence_proxy_async_smem();
          mbar_arrive(&bar_q_full);
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
    int np[2] = {0, 0};  // P hand-overs consumed per tile
    int no[2] = {0, 0};  // items in which the tile was present
    bool ok = true;
    auto issue_s = [&](int x, int st) {
      const SmemDesc qx{dq.lo + ((x * S::kQBytes) >> 4), dq.hi};
      const SmemDesc kst{dk.lo + ((st * S::kKVBytes) >> 4), dk.hi};
      __syncwarp();  // elect.sync in the MMA wrappers needs a converged warp
#pragma unroll
      for (int s = 0; s < kD / 16; ++s)
        mma_ss(tmem + S::col_s(x), qx, (s >> 2) * 16384 + (s & 3) * 32, kst, (s >> 2) * (BN * 128) + (s & 3) * 32,
               idS, s > 0 ? 1u : 0u);
      mma_commit(&bar_s_full[x]);
    };
    for (int ii = 0; ok; ++ii) {
      const int sl = ii & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[sl], (ii >> 1) & 1, status));
      if (!ok) break;
      const int item = *reinterpret_cast<volatile int*>(&ring.item[sl]);
      const int n[2] = {items[sl].n[0], items[sl].n[1]};
      const int n_pre = items[sl].np, p_left = items[sl].p_left, o_left = items[sl].o_left;
      mbar_arrive(&ring.empty[sl]);
      if (item < 0) break;
      const int nmax = max(n[0], n[1]);
      if (!(ok = mbar_wait_warp(&bar_q_full, ii & 1, status))) break;
      if (!(ok = mbar_wait_warp(&bar_k_full[it % NS], (it / NS) & 1, status))) break;
      tc_fence_after();
      for (int x = 0; x < NT; ++x)
        if (n[x] > 0) issue_s(x, it % NS);
      mma_commit(&bar_k_empty[it % NS]);
      if (nmax == 1) mma_commit(&bar_q_empty);
      for (int j = 0; j < nmax && ok; ++j) {
        const int cur = it + j, st = cur % NS;
        bool v_ready = false, k_ready = false;
        for (int x = 0; x < NT && ok; ++x) {
          if (j >= n[x]) continue;
          if (!(ok = mbar_wait_warp(&bar_p_ready[x], np[x] & 1, status))) break;
          ++np[x];
          if (j == 0 && no[x] > 0 && !(ok = mbar_wait_warp(&bar_o_empty[x], (no[x] - 1) & 1, status))) break;
          if (!v_ready) {
            if (!(ok = mbar_wait_warp(&bar_v_full[st], (cur / NS) & 1, status))) break;
            v_ready = true;
            // V rows that are no real key: zeros (P is 0 there, but 0 times NaN is not)
            const int real = j < n_pre ? p_left - j * BN : o_left - (j - n_pre) * BN;
            if (real < BN) {
              for (int t = real * 8 + lane; t < BN * 8; t += 32)
                for (int c = 0; c < S::kChunks; ++c)
                  st_shared_v4(sV + st * S::kKVBytes + c * BN * 128 + t * 16, 0, 0, 0, 0);
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
          if (j + 1 < n[x]) {
            const int nx = cur + 1;
            if (!k_ready) {
              if (!(ok = mbar_wait_warp(&bar_k_full[nx % NS], (nx / NS) & 1, status))) break;
              k_ready = true;
            }
            tc_fence_after();
            issue_s(x, nx % NS);
          } else {
            mma_commit(&bar_o_full[x]);
          }
        }
        if (!ok) break;
        mma_commit(&bar_v_empty[st]);
        if (j + 1 < nmax) mma_commit(&bar_k_empty[(cur + 1) % NS]);
        if (j + 2 == nmax) mma_commit(&bar_q_empty);
      }
      if (!ok) break;
      for (int x = 0; x < NT; ++x)
        if (n[x] > 0) ++no[x];
      it += nmax;
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int x = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + S::col_s(x) + lane_base;
    const uint32_t t_o = tmem + S::col_o(x) + lane_base;
    using T = typename std::conditional<kBF16, __nv_bfloat16, __half>::type;
    const int r = x * 128 + quarter * 32 + lane;  // row of the item
    const float sl2 = p.scale_log2;
    int ns = 0, no = 0;  // S hand-overs and items of this tile so far
    bool ok = true;
    for (int ii = 0; ok; ++ii) {
      const int sl = ii & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[sl], (ii >> 1) & 1, status));
      if (!ok) break;
      const int item = *reinterpret_cast<volatile int*>(&ring.item[sl]);
      const int n = items[sl].n[x], n_pre = items[sl].np, p_left = items[sl].p_left;
      const int row = items[sl].row[r], own = items[sl].lim[r];
      const bool direct = items[sl].direct != 0;
      const size_t part = static_cast<size_t>(items[sl].part) + r;
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
        const int left = j < n_pre ? p_left - j * BN : own - (j - n_pre) * BN;
        const int nvalid = live ? min(max(left, 0), BN) : 0;
        const bool full = __all_sync(0xffffffffu, nvalid >= BN);
        // Row max of this tile's visible scores (log2 domain), from S in TMEM.
        auto tile_max = [&]() -> float {
          float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < BN / 32; ++k) {
            uint32_t sv[32];
            tmem_ld32(t_s + 32 * k, sv);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float a = __uint_as_float(sv[2 * c]) * sl2, b = __uint_as_float(sv[2 * c + 1]) * sl2;
              mp[c & 3] = max3(mp[c & 3], 32 * k + 2 * c < nvalid ? a : -INFINITY,
                               32 * k + 2 * c + 1 < nvalid ? b : -INFINITY);
            }
          }
          return fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]);
        };
        // A row's first tile with a visible key: its max, to start the offset m.
        if (__any_sync(0xffffffffu, m == -INFINITY && nvalid > 0)) {
          const float mxs = tile_max();
          if (m == -INFINITY && nvalid > 0) m = mxs;
        }
        float alpha = 1.f;
        uint64_t sp[4];
        uint32_t pk[BN / 32][16];
        auto pass = [&](auto full_tag) {
          constexpr bool kFull = decltype(full_tag)::value;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(-m, -m);
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
              float p0 = ex2p(xx.x), p1 = ex2p(xx.y);
              if constexpr (!kFull) {
                p0 = 32 * k + 2 * c < nvalid ? p0 : 0.f;
                p1 = 32 * k + 2 * c + 1 < nvalid ? p1 : 0.f;
              }
              sp[c & 3] = fadd2(sp[c & 3], f2_pack(p0, p1));
              pk[k][c] = pack2<kBF16>(p0, p1);
            }
          }
        };
        for (;;) {
          if (full)
            pass(std::true_type{});
          else
            pass(std::false_type{});
          // a row whose P sums to at most 2^8 has no entry above 2^8: nothing to raise
          const float2 s01 = f2_unpack(fadd2(fadd2(sp[0], sp[1]), fadd2(sp[2], sp[3])));
          if (!__any_sync(0xffffffffu, s01.x + s01.y > 256.0f)) break;
          const float mxs = tile_max();
          const bool raise = nvalid > 0 && mxs > m + 8.0f;
          if (!__any_sync(0xffffffffu, raise)) break;
          if (raise) {
            alpha = ex2p(m - mxs);
            m = mxs;
          }
          // S(j) was issued after P V(j-1): O is final for the tiles before this one. At the
          // item's first tile there is nothing to scale: the product will overwrite it.
          if (j > 0) {
#pragma unroll
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
  kern<<<static_cast<int>(most < num_sms ? most : num_sms), S::kThreads, S::kSmemBytes, st>>>(p, tk, tv, tkp, tvp);
  return cudaGetLastError();
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
// Join: rows that left partial results, and the rows that hold no token. One warp per
// (token, some heads); of a row's n partial rows, O = sum_c 2^(m_c - M) O_c / L with
// M = max m_c and L = sum_c 2^(m_c - M) l_c, all in fp32, rounded once.
// ---------------------------------------------------------------------------
template <bool kBF16>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ PrefixParams p, int slices) {
  const int lane = threadIdx.x & 31;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= static_cast<long long>(p.total_q) * slices) return;
  const int t = static_cast<int>(w / slices), slice = static_cast<int>(w % slices);
  const int h0 = static_cast<int>(static_cast<long long>(p.hq) * slice / slices);
  const int h1 = static_cast<int>(static_cast<long long>(p.hq) * (slice + 1) / slices);
  using T = typename std::conditional<kBF16, __nv_bfloat16, __half>::type;
  int i = 0;
  const int b = locate_row(p, p.cu_q_pad, t, &i);
  SeqInfo s{};
  if (b >= 0) s = load_seq(p, b);
  const int rt = prefix_row_tile(p.d), first_pre = p.header[kHdrPrefixFirst];
  // -2: the lengths allow no result
  const bool real = b >= 0 && i < s.len_q && first_pre != -2;
  const int4 info = real ? p.seqs[b] : make_int4(-1, -1, -1, 0);
  for (int h = h0; h < h1; ++h) {
    const size_t row = static_cast<size_t>(t) * p.hq + h;
    const int g = h / p.group, j = h - g * p.group;
    // up to two groups hold this row
    PrefixGroup ga{}, gb{};
    int ra = 0, rb = 0, na = 0, nb = 0;
    if (info.z >= 0) {
      const int rr = i * p.group + j;
      ga = load_group(p, info.z + rr / rt);
      if (ga.chunks == 1) continue;  // written by the main kernel
      ra = rr % rt;
      na = ga.chunks;
    } else if (info.x >= 0) {
      if (first_pre >= 0) {
        const int rr = (info.x + i) * p.group + j;
        ga = load_group(p, first_pre + rr / rt);
        ra = rr % rt;
        na = ga.chunks;
      }
      if (info.y >= 0) {
        gb = load_group(p, info.y);
        if (gb.slot < 0) continue;  // written by the main kernel
        rb = i * p.group + j;
        nb = gb.chunks;
      }
    }
    const int n = na + nb;
    auto at = [&](int c) { return c < na ? partial_row(p, ga, c, g, ra) : partial_row(p, gb, c - na, g, rb); };
    float M = -INFINITY;
    for (int c = lane; c < n; c += 32) {
      const float2 ml = p.part_ml[at(c)];
      if (ml.y > 0.f) M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float acc[8] = {};
    for (int c0 = 0; c0 < n; c0 += 32) {
      float wgt = 0.f;
      if (c0 + lane < n) {
        const float2 ml = p.part_ml[at(c0 + lane)];
        // a chunk without a visible key left no output
        wgt = ml.y > 0.f ? ex2p(ml.x - M) : 0.f;
        L += wgt * ml.y;
      }
      const int nc = min(32, n - c0);
      for (int c = 0; c < nc; ++c) {
        const float wc = __shfl_sync(0xffffffffu, wgt, c);
        if (wc == 0.f) continue;
        const float* src = p.part_o + at(c0 + c) * p.d;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = 128 * k + 4 * lane;
          if (col < p.d) {
            const float4 v = *reinterpret_cast<const float4*>(src + col);
            acc[4 * k] = fmaf(wc, v.x, acc[4 * k]);
            acc[4 * k + 1] = fmaf(wc, v.y, acc[4 * k + 1]);
            acc[4 * k + 2] = fmaf(wc, v.z, acc[4 * k + 2]);
            acc[4 * k + 3] = fmaf(wc, v.w, acc[4 * k + 3]);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = L > 0.f ? 1.0f / L : 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int col = 128 * k + 4 * lane;
      if (col < p.d) {
        uint2 v;
        v.x = pack2<kBF16>(acc[4 * k] * inv, acc[4 * k + 1] * inv);
        v.y = pack2<kBF16>(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * p.d + col) = v;
      }
    }
    if (lane == 0) p.lse[row] = !real ? 0.f : L > 0.f ? M * 0.69314718055994531f + logf(L) : -INFINITY;
  }
}

cudaError_t launch_prefix_join(const PrefixParams& p, bool bf16, cudaStream_t st) {
  // enough warps to fill the GPU with few tokens, whole tokens with many
  const int slices = p.total_q >= 4096 ? 1 : (4096 + p.total_q - 1) / p.total_q < p.hq ? (4096 + p.total_q - 1) / p.total_q : p.hq;
  const long long warps = static_cast<long long>(p.total_q) * slices;
  const unsigned blocks = static_cast<unsigned>((warps + 7) / 8);
  if (bf16) prefix_join_kernel<true><<<blocks, 256, 0, st>>>(p, slices);
  else prefix_join_kernel<false><<<blocks, 256, 0, st>>>(p, slices);
  return cudaGetLastError();
}

}  // namespace teattn
