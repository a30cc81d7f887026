// Attention of many queries over a paged cache (pieces of prompts), in 16 or in 4 bits.
//
//   S = scale q K^T over the keys that a query sees,  O = softmax(S) V,  LSE = log sum exp S
//
// The rows of a kv head (its group's queries, token by token) are taken 256 at a time, two tiles
// A and B of 128 over the same key tiles of 128, so that every key tile is fetched once for both.
// Segments (sequence, 256 rows, kv head) lie on a line, key tile by key tile, and every block
// takes an equal slice of it: one short prompt behind a long cache and many side by side both
// fill the GPU. What slices share is joined by attn_paged_join.cu. Roles of a block:
//   warps 0-3, 4-7  softmax of tile A, B (one thread per row / TMEM lane),
//   warp 8          queries, and 16-bit keys and values, by TMA, a box per page or 128 keys,
//   warp 9          the tensor-core products (one elected lane issues),
//   warps 10-13     4 bits: a thread per key turns its codes into 16-bit values in shared memory,
//                   a tile ahead of the products, from registers that hold the next tile's codes.
// TMEM: O_A, O_B, S_A, S_B of 128 columns. The issue order is S_A0, S_B0 | PV_A0, S_A1 | PV_B0,
// S_B1 | ...: while one tile's scores become P, the tensor cores work on the other tile.
// The softmax is attn_fwd_pair.cu's: offset raised only past 2^8, P over S as 16 bits, sums and
// outputs in fp32. Bounded by the chain S, softmax, P V of either tile, 1.7-2.0 us a key tile of
// both at d 128: the tensor cores are 50 % busy, the exponentials' pipe 26 %.
//
// Measured, bf16, hq 32, hkv 8, d 128: four pieces of 100-512 queries behind 2000-12000 keys 208
// us a call (0.93 PFLOP/s), in 4 bits 288; 16384 queries 2380 us, with a window of 1024 601 us. A segment
// costs 6 to 8 us beside its key tiles (first scores, their maximum, the rows' end).
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "attn_paged.cuh"
#include "common.cuh"
#include "pdl.cuh"
#include "row_store.cuh"
#include "sm103_ptx.cuh"
#include "tmap.h"

namespace teattn {

template <int kD, bool k4>
struct TilesShape {
  static_assert(kD == 64 || kD == 128, "O of two tiles fills half of TMEM up to head_dim 128");
  static constexpr int kChunks = kD / 64;
  static constexpr int kTileBytes = kChunks * 16384;  // 128 rows of queries, keys or values
  static constexpr int kStages = kD == 64 ? 4 : 2;
  static constexpr int kSmem = kTileBytes * (2 + 2 * kStages) + 1024;
  static constexpr int kThreads = k4 ? 448 : 320;
  __device__ static constexpr uint32_t col_o(int x) { return static_cast<uint32_t>(x) * 128u; }
  __device__ static constexpr uint32_t col_s(int x) { return 256u + static_cast<uint32_t>(x) * 128u; }
};

struct TilesMaps {
  CUtensorMap k, v;          // boxes of 64 columns and min(page, 128) slots (16 bits only)
  CUtensorMap q;             // boxes of 128 rows (whole tokens of a group), or of one row
  int q_tokens;              // tokens of a box; 0: one row
  int box_slots;
};

__device__ __forceinline__ float ex2t(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t low_bits_of(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// What the rows of a stretch see: keys [lo_some, sees) and the sinks by some row.
struct TileView {
  int row0, rows, sees, lo_some, sinks;
};
__device__ __forceinline__ TileView tile_view(const PagedParams& p, const Stretch& t) {
  const int row0 = t.tile * kWideRows;  // (rows of a sequence are below 2^31)
  const int rows = min(kWideRows, t.s.n * p.group - row0);
  return TileView{row0, rows, t.s.past + (row0 + rows - 1) / p.group + 1, paged_first(p, t.s, row0 / p.group),
                  p.window > 0 ? p.sinks : 0};
}

template <int kD, bool kBF16, bool k4>
__global__ void __launch_bounds__(TilesShape<kD, k4>::kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ PagedParts parts, const __grid_constant__ TilesMaps tm,
                       int first_status) {
  using S = TilesShape<kD, k4>;
  constexpr int NS = S::kStages;
  constexpr PagedCut cut{kWideRows, kWideKeys, true};
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;  // tile A then tile B
  uint8_t* sK = sQ + 2 * S::kTileBytes;
  uint8_t* sV = sK + NS * S::kTileBytes;
  long long* pref = reinterpret_cast<long long*>(sV + NS * S::kTileBytes);

  __shared__ uint64_t bar_q_full, bar_q_empty;
  __shared__ uint64_t bar_k_full[NS], bar_k_empty[NS], bar_v_full[NS], bar_v_empty[NS];
  __shared__ uint64_t bar_s_full[2], bar_p_ready[2], bar_o_full[2], bar_o_empty[2];
  // 16-key blocks of a tile that were loaded: two bits for every 32 keys. A tile's word is read
  // until its product is issued, so five of them are alive at most.
  __shared__ union { uint32_t word; uint8_t part[4]; } s_blocks[8];
  constexpr uint32_t kAllBlocks = 0x03030303u;
  __shared__ uint32_t s_magic;
  __shared__ uint32_t tmem_slot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* status = p.warp_status + first_status + blockIdx.x;
  pdl_trigger();
  if (tid == 0) {
    *status = 0;
    s_magic = kCodeMagic<kBF16>;
    mbar_init(&bar_q_full, 1);
    mbar_init(&bar_q_empty, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar_k_full[i], k4 ? 128 : 1);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_v_full[i], k4 ? 128 : 1);
      mbar_init(&bar_v_empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar_s_full[x], 1);
      mbar_init(&bar_p_ready[x], 128);
      mbar_init(&bar_o_full[x], 1);
      mbar_init(&bar_o_empty[x], 128);
    }
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const long long total = sum_units(p, cut, pref, status);
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.batch; b += blockDim.x) parts.pref[b] = pref[b];
  const long long per = slice_units(total, parts.slices, kLeastWideUnits);
  const long long begin = blockIdx.x * per, end = begin + per < total ? begin + per : total;

  if (warp == 8) {
    // ------------------------------------------------------------- queries, 16-bit keys and values
    int it = 0;
    bool ok = true;
    int ii = 0;
    Stretch t;
#pragma unroll 1
    for (long long at = begin; at < end && ok; ++ii) {
      next_stretch(p, cut, pref, at, end, at == begin, t);
      const TileView w = tile_view(p, t);
      if (ii > 0 && !(ok = mbar_wait_warp(&bar_q_empty, (ii - 1) & 1, status))) break;
      const bool boxes = tm.q_tokens > 0;
      const int q_rows = boxes ? (w.rows > 128 ? 256 : 128) : w.rows;
      if (lane == 0) mbar_arrive_expect_tx(&bar_q_full, q_rows * 128 * S::kChunks);
      __syncwarp();
#pragma unroll 1
      for (int r = boxes ? lane * 128 : lane; r < w.rows; r += boxes ? 32 * 128 : 32) {
        const int rr = w.row0 + r, i = rr / p.group, j = rr - i * p.group;
        for (int c = 0; c < S::kChunks; ++c)
          tma_load_4d(sQ + (r >> 7) * S::kTileBytes + c * 16384 + (r & 127) * 128, &tm.q, &bar_q_full, c * 64,
                      t.head * p.group + j, 0, t.s.off + i);
      }
      if constexpr (!k4) {
        const int nb = 128 / tm.box_slots, mask = (1 << p.cache.shift) - 1;
        // lane: block lane % nb of the tile; pages are looked up a tile ahead
        auto look_up = [&](int u) {
          const int key = t.run.unit(u) * kWideKeys + lane % nb * tm.box_slots;
          if (key >= w.sees || (key + tm.box_slots <= w.lo_some && key >= w.sinks)) return -2;  // not seen
          const int page = page_of(p.cache, t.b, key);
          if (page < 0 && lane < nb) atomicOr(status, kStatusBadPages);
          return page;
        };
        int next = look_up(t.u0);
#pragma unroll 1
        for (int u = t.u0; u < t.u0 + t.n; ++u, ++it) {
          const int page = next, st = it % NS, key0 = t.run.unit(u) * kWideKeys;
          if (u + 1 < t.u0 + t.n) next = look_up(u + 1);
          const uint32_t some = __ballot_sync(0xffffffffu, lane < nb && page >= 0);
          const uint32_t bytes = __popc(some) * tm.box_slots * 128 * S::kChunks;
          uint32_t blocks = 0;
          for (int k = 0; k < 8; ++k) blocks |= ((some >> (16 * k / tm.box_slots)) & 1u) << (8 * (k >> 1) + (k & 1));
#pragma unroll 1
          for (int kv = 0; kv < 2 && ok; ++kv) {
            uint64_t *full = kv ? &bar_v_full[st] : &bar_k_full[st], *empty = kv ? &bar_v_empty[st] : &bar_k_empty[st];
            if (it >= NS && !(ok = mbar_wait_warp(empty, ((it / NS) - 1) & 1, status))) break;
            if (lane == 0) {
              if (kv == 0) *const_cast<volatile uint32_t*>(&s_blocks[it & 7].word) = blocks;
              mbar_arrive_expect_tx(full, bytes);
            }
            __syncwarp();
            // chunk lane / nb of block lane % nb; with 16-slot pages and one box a block 16 lanes have one
            if (lane < nb * S::kChunks && page >= 0)
              tma_load_4d((kv ? sV : sK) + st * S::kTileBytes + lane / nb * 16384 + lane % nb * tm.box_slots * 128, kv ? &tm.v : &tm.k,
                          full, lane / nb * 64, (key0 + lane % nb * tm.box_slots) & mask, t.head, page);
          }
          if (!ok) break;
        }
      }
      at += t.n;
    }
    if (!ok) {  // given up: the copies on their way land before the block ends
      mbar_drain(&bar_q_full, ii & 1);
      if constexpr (!k4) {
        for (int i = it > NS ? it - NS : 0; i <= it; ++i) {
          mbar_drain(&bar_k_full[i % NS], (i / NS) & 1);
          mbar_drain(&bar_v_full[i % NS], (i / NS) & 1);
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------- products
    constexpr uint32_t idS = make_idesc_f16(kBF16, false, false, 128, 128);
    constexpr uint32_t idPV = make_idesc_f16(kBF16, false, true, 128, kD);
    const SmemDesc dq = smem_desc(smem_u32(sQ), 16, 1024, kLayoutSW128);
    const SmemDesc dk = smem_desc(smem_u32(sK), 16, 1024, kLayoutSW128);
    const SmemDesc dv = smem_desc(smem_u32(sV), 16384, 1024, kLayoutSW128);
    int it = 0, np[2] = {0, 0}, no[2] = {0, 0}, ii = 0;
    bool ok = true;
    auto issue_s = [&](int x, int st) {
      const SmemDesc qx{dq.lo + ((x * S::kTileBytes) >> 4), dq.hi};
      const SmemDesc kst{dk.lo + ((st * S::kTileBytes) >> 4), dk.hi};
      __syncwarp();  // elect.sync in the MMA wrappers needs a converged warp
#pragma unroll
      for (int s = 0; s < kD / 16; ++s) {
        const uint32_t off = (s >> 2) * 16384 + (s & 3) * 32;
        mma_ss(tmem + S::col_s(x), qx, off, kst, off, idS, s > 0 ? 1u : 0u);
      }
      mma_commit(&bar_s_full[x]);
    };
    Stretch t, ahead;
    if (begin < end) next_stretch(p, cut, pref, begin, end, true, ahead);
#pragma unroll 1
    for (long long at = begin; at < end && ok; ++ii) {
      t = ahead;
      const TileView w = tile_view(p, t);
      const int nx = w.rows > 128 ? 2 : 1;
      if (!(ok = mbar_wait_warp(&bar_q_full, ii & 1, status))) break;
      if (!(ok = mbar_wait_warp(&bar_k_full[it % NS], (it / NS) & 1, status))) break;
      tc_fence_after();
      for (int x = 0; x < nx; ++x) issue_s(x, it % NS);
      mma_commit(&bar_k_empty[it % NS]);
      if (t.n == 1) mma_commit(&bar_q_empty);
#pragma unroll 1
      for (int j = 0; j < t.n && ok; ++j) {
        const int cur = it + j, st = cur % NS;
        bool v_ready = false, k_ready = false;
        // (worked out while this stretch's last P are awaited)
        if (j + 1 == t.n && at + t.n < end) next_stretch(p, cut, pref, at + t.n, end, false, ahead);
        for (int x = 0; x < nx && ok; ++x) {
          if (!(ok = mbar_wait_warp(&bar_p_ready[x], np[x] & 1, status))) break;
          ++np[x];
          if (j == 0 && no[x] > 0 && !(ok = mbar_wait_warp(&bar_o_empty[x], (no[x] - 1) & 1, status))) break;
          if (!v_ready) {
            if (!(ok = mbar_wait_warp(&bar_v_full[st], (cur / NS) & 1, status))) break;
            v_ready = true;
            if constexpr (!k4) {
              // values of keys that no row sees become zeros: P is 0, but 0 times NaN is not
              const int key0 = t.run.unit(t.u0 + j) * kWideKeys;
              const bool whole = key0 + kWideKeys <= w.sees && (key0 >= w.lo_some || key0 + kWideKeys <= w.sinks);
              // (blocks whose page lies outside the cache were not loaded either)
              const uint32_t blocks = *const_cast<volatile uint32_t*>(&s_blocks[cur & 7].word);
              if (!whole || blocks != kAllBlocks) {
#pragma unroll 1
                for (int z = lane; z < 128 * 8; z += 32) {
                  const int r = z >> 3, key = key0 + r;
                  if (key < w.sees && (key >= w.lo_some || key < w.sinks) && ((blocks >> (8 * (r >> 5) + ((r >> 4) & 1))) & 1u)) continue;
#pragma unroll
                  for (int c = 0; c < S::kChunks; ++c) st_shared_v4(sV + st * S::kTileBytes + c * 16384 + z * 16, 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
          }
          tc_fence_after();
          const SmemDesc vst{dv.lo + ((st * S::kTileBytes) >> 4), dv.hi};
          __syncwarp();
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma_ts(tmem + S::col_o(x), tmem + S::col_s(x) + s * 8, vst, s * 2048, idPV, s > 0 || j > 0 ? 1u : 0u);
          if (j + 1 < t.n) {
            if (!k_ready) {
              if (!(ok = mbar_wait_warp(&bar_k_full[(cur + 1) % NS], ((cur + 1) / NS) & 1, status))) break;
              k_ready = true;
            }
            tc_fence_after();
            issue_s(x, (cur + 1) % NS);
          } else {
            mma_commit(&bar_o_full[x]);
          }
        }
        if (!ok) break;
        mma_commit(&bar_v_empty[st]);
        if (j + 1 < t.n) mma_commit(&bar_k_empty[(cur + 1) % NS]);
        if (j + 2 == t.n) mma_commit(&bar_q_empty);
      }
      for (int x = 0; x < nx; ++x) ++no[x];
      it += t.n;
      at += t.n;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------- softmax A / B
    const int x = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + S::col_s(x) + lane_base, t_o = tmem + S::col_o(x) + lane_base;
    using T = typename std::conditional<kBF16, __nv_bfloat16, __half>::type;
    const float sl2 = p.scale_log2;
    int ns = 0, no = 0;  // tiles and stretches of this side so far
    int skipped = 0;     // tiles that the other side had alone
    bool ok = true;
    Stretch t;
    if (begin < end) next_stretch(p, cut, pref, begin, end, true, t);
#pragma unroll 1
    for (long long at = begin; at < end && ok;) {
      const TileView w = tile_view(p, t);
      at += t.n;
      if (x == 1 && w.rows <= 128) {
        skipped += t.n;
        if (at < end) next_stretch(p, cut, pref, at, end, false, t);
        continue;
      }
      const int r = x * 128 + quarter * 32 + lane, rr = w.row0 + min(r, w.rows - 1), i = rr / p.group;
      const bool live = r < w.rows;
      // (rows behind the last one see everything: their warp then takes the way without masks)
      const int hi = live ? t.s.past + i + 1 : INT_MAX, lo = live ? paged_first(p, t.s, i) : 0;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int u = t.u0; u < t.u0 + t.n; ++u) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_s_full[x], ns & 1, status));
        if (!ok) break;
        tc_fence_after();
        const int key0 = t.run.unit(u) * kWideKeys;
        // bit c % 32 of word c / 32: the row sees the key of column c
        const uint32_t blocks = *const_cast<volatile uint32_t*>(&s_blocks[(ns + skipped) & 7].word);
        ++ns;
        uint32_t seen[4];
        const bool full = __all_sync(0xffffffffu, key0 + kWideKeys <= hi && (key0 >= lo || key0 + kWideKeys <= w.sinks) &&
                                                      blocks == kAllBlocks);
        bool some = true;
        if (full) {
#pragma unroll
          for (int k = 0; k < 4; ++k) seen[k] = ~0u;
        } else {
          uint32_t any = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = key0 + 32 * k;
            seen[k] = low_bits_of(hi - key) & (~low_bits_of(lo - key) | low_bits_of(w.sinks - key));
            if (!((blocks >> (8 * k)) & 1u)) seen[k] &= 0xffff0000u;
            if (!((blocks >> (8 * k)) & 2u)) seen[k] &= 0x0000ffffu;
            any |= seen[k];
          }
          some = any != 0;
        }
        auto valid = [&](int c) { return ((seen[c / 32] >> (c % 32)) & 1u) != 0; };
        auto tile_max = [&]() -> float {
          float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t sv[32];
            tmem_ld32(t_s + 32 * k, sv);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c)
              mp[c & 3] = max3(mp[c & 3], valid(32 * k + 2 * c) ? __uint_as_float(sv[2 * c]) * sl2 : -INFINITY,
                               valid(32 * k + 2 * c + 1) ? __uint_as_float(sv[2 * c + 1]) * sl2 : -INFINITY);
          }
          return fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]);
        };
        // a row's first tile with a visible key: its max, to start the offset m
        if (__any_sync(0xffffffffu, m == -INFINITY && some)) {
          const float mxs = tile_max();
          if (m == -INFINITY && some) m = mxs;
        }
        float alpha = 1.f;
        uint64_t sp[4];
        uint32_t pk[4][16];
        auto pass = [&](auto full_tag) {
          constexpr bool kFull = decltype(full_tag)::value;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(-m, -m);
#pragma unroll
          for (int k = 0; k < 4; ++k) sp[k] = f2_pack(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t sv[32];
            tmem_ld32(t_s + 32 * k, sv);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 xx = f2_unpack(ffma2(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sl2x2, negm2));
              float p0 = ex2t(xx.x), p1 = ex2t(xx.y);
              if constexpr (!kFull) {
                p0 = valid(32 * k + 2 * c) ? p0 : 0.f;
                p1 = valid(32 * k + 2 * c + 1) ? p1 : 0.f;
              }
              sp[c & 3] = fadd2(sp[c & 3], f2_pack(p0, p1));
              pk[k][c] = pack2<kBF16>(p0, p1);
            }
          }
        };
        for (;;) {
          if (full) pass(std::true_type{});
          else pass(std::false_type{});
          const float2 s01 = f2_unpack(fadd2(fadd2(sp[0], sp[1]), fadd2(sp[2], sp[3])));
          // a row whose P sums to at most 2^8 has no entry above 2^8: nothing to raise
          if (!__any_sync(0xffffffffu, s01.x + s01.y > 256.0f)) break;
          const float mxs = tile_max();
          const bool raise = some && mxs > m + 8.0f;
          if (!__any_sync(0xffffffffu, raise)) break;
          if (raise) {
            alpha = ex2t(m - mxs);
            m = mxs;
          }
          // (O is final for the tiles before: S of this one was issued behind their products)
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
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_st16(t_s + 16 * k, pk[k]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar_p_ready[x]);
        const float2 s01 = f2_unpack(fadd2(fadd2(sp[0], sp[1]), fadd2(sp[2], sp[3])));
        l = l * alpha + (s01.x + s01.y);
      }
      if (!ok) break;
      const int j = rr - i * p.group;
      const long long row = static_cast<long long>(t.s.off + i) * p.hq + t.head * p.group + j;
      const bool store = live && bounds_ok(row < static_cast<long long>(p.total_q) * p.hq, status);
      const bool whole = t.n == t.run.n, begins = t.u0 == 0;
      if (at < end) next_stretch(p, cut, pref, at, end, false, t);  // (while the last products run)
      ok = __all_sync(0xffffffffu, mbar_wait(&bar_o_full[x], no & 1, status));
      if (!ok) break;
      ++no;
      tc_fence_after();
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        const auto rows = make_row_pair(static_cast<T*>(p.out) + row * p.d, store);
#pragma unroll
        for (int c0 = 0; c0 < kD; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(t_o + c0, o);
          tmem_ld_wait();
          store_pair16<kBF16>(rows, c0, p.d, o, inv);
        }
        if (store) p.lse[row] = m * 0.69314718055994531f + logf(l);
      } else {
        // column by column, so that a warp's 32 rows lie side by side
        const long long slot = 2ll * blockIdx.x + (begins ? 1 : 0);
        parts.ml[slot * kWideRows + r] = make_float2(m, l);
        float* part = parts.o + slot * p.d * kWideRows + r;
#pragma unroll
        for (int c0 = 0; c0 < kD; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(t_o + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (c0 + c < p.d) part[(c0 + c) * kWideRows] = __uint_as_float(o[c]);
        }
      }
      tc_fence_before();
      mbar_arrive(&bar_o_empty[x]);
    }
  } else if constexpr (k4) {
    // ------------------------------------------------------------- 4 bits to 16
    const int r = tid - 320;  // key of the tile
    int it = 0;
    bool ok = true;
    constexpr int kG = kD / 32;
    const uint32_t magic = *const_cast<volatile uint32_t*>(&s_magic);
    struct Raw {
      uint4 code[kG];
      uint32_t meta[kG];
      bool there;
    };
    Stretch t;
#pragma unroll 1
    for (long long at = begin; at < end && ok;) {
      next_stretch(p, cut, pref, at, end, at == begin, t);
      const TileView w = tile_view(p, t);
      // keys or values of a unit, into registers; a key that no row sees stands for zeros
      auto fetch = [&](int u, int kv, Raw& raw) {
        const int key = t.run.unit(u) * kWideKeys + r;
        int page = -1;
        if (key < w.sees && (key >= w.lo_some || key < w.sinks)) {
          page = page_of(p.cache, t.b, key);
          if (page < 0) atomicOr(status, kStatusBadPages);
        }
        raw.there = page >= 0;
        const long long row = page_row(p.cache, t.head, key & ((1 << p.cache.shift) - 1));
        const uint8_t* code = p.cache.data[kv] + page * p.cache.stride[kv] + row * p.cache.row_bytes;
        const uint8_t* meta = p.cache.meta[kv] + page * p.cache.meta_stride[kv] + row * (p.d / 8);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const bool in = page >= 0 && g * 32 < p.d;
          raw.code[g] = in ? *reinterpret_cast<const uint4*>(code + g * 16) : make_uint4(0, 0, 0, 0);
          raw.meta[g] = in ? *reinterpret_cast<const uint32_t*>(meta + g * 4) : 0u;
        }
      };
      auto put = [&](uint8_t* tile, const Raw& raw) {
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const uint32_t words[4] = {raw.code[g].x, raw.code[g].y, raw.code[g].z, raw.code[g].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = dequantize8<kBF16>(words[k], raw.meta[g], magic);
            const int piece = (g & 1) * 4 + k;
            st_shared_v4(tile + (g >> 1) * 16384 + r * 128 + ((piece ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
          }
        }
        fence_proxy_async_smem();
      };
      Raw k, v;
      fetch(t.u0, 0, k);
      fetch(t.u0, 1, v);
#pragma unroll 1
      for (int u = t.u0; u < t.u0 + t.n && ok; ++u, ++it) {
        const int st = it % NS;
        const bool more = u + 1 < t.u0 + t.n;
        if (it >= NS && !(ok = mbar_wait_warp(&bar_k_empty[st], ((it / NS) - 1) & 1, status))) break;
        // (a page holds 16 keys at least; a block of which some row sees a key counts as there)
        const uint32_t there = __ballot_sync(0xffffffffu, k.there);
        if (lane == 0)
          *const_cast<volatile uint8_t*>(&s_blocks[it & 7].part[warp - 10]) = ((there & 0xffffu) != 0 ? 1 : 0) | (there >> 16 != 0 ? 2 : 0);
        put(sK + st * S::kTileBytes, k);
        mbar_arrive(&bar_k_full[st]);
        if (more) fetch(u + 1, 0, k);
        if (it >= NS && !(ok = mbar_wait_warp(&bar_v_empty[st], ((it / NS) - 1) & 1, status))) break;
        put(sV + st * S::kTileBytes, v);
        mbar_arrive(&bar_v_full[st]);
        if (more) fetch(u + 1, 1, v);
      }
      at += t.n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  pdl_wait();  // complete only after the kernel ahead, for the join behind both
}

template <int kD, bool kBF16, bool k4>
static cudaError_t launch_tiles_impl(const PagedParams& p, const PagedParts& parts, int first_status, cudaStream_t st) {
  using S = TilesShape<kD, k4>;
  TilesMaps tm{};
  tm.box_slots = 1 << (p.cache.shift < 7 ? p.cache.shift : 7);
  tm.q_tokens = 128 % p.group == 0 ? 128 / p.group : 0;
  const bool boxes = tm.q_tokens > 0;
  if (!make_tmap_tokens(&tm.q, p.q, p.total_q, 1, p.hq, p.d, kBF16, boxes ? 128 : 1, boxes ? p.group : 1)) return cudaErrorInvalidValue;
  if (!k4 && (!make_tmap_pages(&tm.k, p.cache, 0, kBF16, tm.box_slots) || !make_tmap_pages(&tm.v, p.cache, 1, kBF16, tm.box_slots)))
    return cudaErrorInvalidValue;
  auto kern = paged_tiles_kernel<kD, kBF16, k4>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem + (kPagedMaxBatch + 1) * 8);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(parts.slices), dim3(S::kThreads), S::kSmem + (p.batch + 1) * sizeof(long long), st, p, parts, tm,
                          first_status);
}

template <bool kBF16, bool k4>
static cudaError_t launch_tiles_d(const PagedParams& p, const PagedParts& parts, int first_status, cudaStream_t st) {
  return p.d <= 64 ? launch_tiles_impl<64, kBF16, k4>(p, parts, first_status, st)
                   : launch_tiles_impl<128, kBF16, k4>(p, parts, first_status, st);
}

cudaError_t launch_paged_tiles(const PagedParams& p, const PagedParts& parts, int first_status, bool bf16, bool four, cudaStream_t st) {
  if (four) return bf16 ? launch_tiles_d<true, true>(p, parts, first_status, st) : launch_tiles_d<false, true>(p, parts, first_status, st);
  return bf16 ? launch_tiles_d<true, false>(p, parts, first_status, st) : launch_tiles_d<false, false>(p, parts, first_status, st);
}

int paged_wide_rows(int batch, int total_q, int hq, int hkv, int d, bool four) {
  // Above head_dim 128 the kernel of few rows takes all, 8 rows a pass: four pieces of 100-512 queries behind
  // 2000-12000 keys 4524 us (4 bits 4090), through a window of 1024 798 (844); 8192 queries from the first on
  // 24283, through that window 15623. At d 128 these take 214 (288), 106 (109), 828 and 356 us here.
  if (d > 128) return 0;
  // Rows a kv head from which a sequence is faster here. With a segment for every SM, at d 128, 64
  // sequences of 2000 keys: 20 rows 160 us here, 202 there, which reads keys once for every 16 rows; in 4
  // bits 20 rows 197 and 189, 48 rows 199 and 317; at d 64 20 rows 138 and 120, 32 rows 138 and 137. With
  // fewer segments blocks wait for one another's key tiles: 8 sequences, 32 rows 50 and 32 us.
  const int least = static_cast<long long>(batch) * hkv < kPagedSMs ? 64 : four || d <= 64 ? 32 : 16;
  // Launched where sequences must have many rows on average, or some sequence may have many enough
  // to outweigh a launch for nothing (4 us): 512 rows of one sequence take 34 us here and 36 there behind
  // 500 keys, 43 and 50 behind 2000, 86 and 210 behind 20000 (in 4 bits 88 and 379).
  const int group = hq / hkv;
  const long long rows = static_cast<long long>(total_q) * group, over = rows - static_cast<long long>(batch) * group;
  return rows > static_cast<long long>(least) * batch || over >= 512 ? least : 0;
}

}  // namespace teattn
