// Attention of few queries over a paged cache, in 16 or in 4 bits.
//
//   S = scale q K^T over the keys that a query sees,  O = softmax(S) V,  LSE = log sum exp S
//
// A decoding step reads every cached key and value once and does next to nothing with it, so
// what counts is to keep loads in flight everywhere and all the time. The work is a line of
// units (16 or 32 keys of one sequence, kv head and row tile), cut into equal slices, one for
// each warp of the grid: no warp waits for another, and a long cache is spread over the GPU as
// evenly as many short ones. A warp copies its units into a ring of its own in shared memory
// (TMA; no role but its own, no barrier across warps) and multiplies them with the warp-wide
// tensor instructions, keys as the rows of the tile:
//   S^T = K Q^T  (16 keys x 8 rows a product), P^T = exp2(S^T scale log2e - m), O^T += V^T P^T,
// since a kv head's group has 8 rows or a few more in one step: with queries as the 128 rows of
// a tcgen05 tile 120 would be empty, with 16-row query tiles half. P^T comes out of the scores'
// registers in the place where the second product wants it but transposed (movmatrix).
// The offset m is raised only when a score exceeds it by more than 2^8; sums of P stay in each
// lane until the end. P is rounded to 16 bits for the product, everything else is fp32.
//
// 4 bits: a lane takes a word of eight codes of a key, spreads it into pairs, takes the magic
// number off and applies step and least value with one fused multiply-add a pair: exactly the
// 16-bit values that the codes stand for, in registers, so that shared memory sees the 4 bits only.
// Which element of a head goes to which place of a product is free as long as Q and K, or V and
// O, agree; the places are chosen so that a lane's word feeds its own registers.
//
// Slices cut sequences anywhere. A warp that has a whole segment (sequence, row tile, head)
// writes its rows; the others leave maximum, sum and unnormalised output in fp32, which a second
// kernel joins in the order of the keys, and which also writes zeros to rows that hold no token.
//
// Measured, bf16, hq 32, hkv 8, d 128, one query a sequence. 16 bits: 64 sequences of 200-4000 keys
// 102 us a call (94 of them here, at 6.04 TB/s; the copy rate is 6.7), 32 with a window of 4096
// 92 us: bounded by HBM. 4 bits: 128 sequences of 1000-16000 keys 328 us for 210 us of bytes:
// bounded by instructions, 450 a 16-key block, most of them unpacking (the ALU pipe is 60 % busy).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "attn_paged.cuh"
#include "common.cuh"
#include "pdl.cuh"
#include "sm103_ptx.cuh"
#include "tmap.h"

namespace teattn {

template <int kD, int kNT, bool k4>
struct RowsShape {
  static constexpr int kRows = 8 * kNT;
  static constexpr int kBlocks = k4 || kD == 64 ? 2 : 1;  // 16-key blocks of a unit
  static constexpr int kUnit = 16 * kBlocks;
  // As many warps as registers (168 a thread of 12 warps) and rings leave: at d 128 in 4 bits 8, 10,
  // 14 and 16 were slower; at d 64 16 warps of two stages faster than 12 of three.
  static constexpr int kWarps = k4 ? (kD == 256 ? 6 : kD == 64 ? 16 : 12) : (kD == 256 ? 4 : 8);
  // (a 4-bit ring is laid out for kD elements a row, whatever d is)
  static constexpr int kDataBytes = kUnit * (k4 ? kD / 2 : 2 * kD);  // keys or values of a unit
  static constexpr int kMetaBytes = k4 ? kUnit * kD / 8 : 0;
  static constexpr int kStageBytes = 2 * (kDataBytes + kMetaBytes);
  static constexpr int kStages = k4 && kD == 64 ? 2 : 3;
  static constexpr int kLeast = kLeastKeys / kUnit;
  static constexpr int kSmem = kWarps * kStages * kStageBytes + 1024;
  static_assert(kSmem <= 208 * 1024, "shared memory budget");
};

struct RowsMaps {
  CUtensorMap k, v;  // boxes of 64 columns and a 16-key block's rows (16 bits only)
};

__device__ __forceinline__ float ex2r(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool kBF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kBF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool kTrans>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// kExact: 4 bits, d is kD (offsets into a row are then constants).
template <int kD, int kNT, bool kBF16, bool k4, bool kExact>
__global__ void __launch_bounds__(RowsShape<kD, kNT, k4>::kWarps * 32, 1)
    paged_rows_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ PagedParts parts,
                      const __grid_constant__ RowsMaps tm) {
  using S = RowsShape<kD, kNT, k4>;
  constexpr int kRows = S::kRows, kUnit = S::kUnit, kBlocks = S::kBlocks, NS = S::kStages, kSteps = kD / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  long long* pref = reinterpret_cast<long long*>(smem + S::kWarps * NS * S::kStageBytes);  // [batch + 1]
  __shared__ uint64_t bar[S::kWarps][NS];
  __shared__ uint32_t s_magic;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int warps = gridDim.x * S::kWarps;
  // neighbouring slices on different SMs, so that few of them still use all
  const int mine = warp * gridDim.x + blockIdx.x;
  // a word of its own for each warp's status, which the join collects: no launch ahead of this
  // one has to clear a common one
  int* status = p.warp_status + mine;
  pdl_trigger();
  if (tid == 0) s_magic = kCodeMagic<kBF16>;
  if (lane == 0) {
    *status = 0;
    for (int i = 0; i < NS; ++i) mbar_init(&bar[warp][i], 1);
    fence_barrier_init();
  }
  constexpr PagedCut cut{kRows, kUnit, false};
  const long long total = sum_units(p, cut, pref, status);
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.batch; b += blockDim.x) parts.pref[b] = pref[b];
  const long long per = slice_units(total, warps, S::kLeast);
  const long long begin = mine * per, end = begin + per < total ? begin + per : total;
  if (begin >= end) return;

  uint8_t* ring = smem + warp * NS * S::kStageBytes;
  const int row_bytes = kExact ? kD / 2 : p.cache.row_bytes, meta_bytes = kExact ? kD / 8 : p.d / 8;
  // ------------------------------------------------------------- loads
  // Pages are looked up 32 blocks of 16 keys at a time, a batch ahead of its use. A lane works out
  // where its block lies once, and issues its copies when the block's unit comes: a unit then
  // costs the warp a few instructions.
  constexpr int kBatch = 32 / kBlocks;  // units of a batch
  Stretch lt = stretch_at(p, cut, pref, begin, end);
  int lu = lt.u0;      // first unit of the batch that is looked up next
  int ahead_n = 0;     // its units,
  int ahead_page = -1, ahead_head = 0, ahead_slot = 0;  // and this lane's block of them
  long long looked = begin;  // places looked up so far
  auto look_up = [&]() {
    ahead_n = 0;
    if (looked >= end) return;
    if (lu == lt.u0 + lt.n) {
      lt = stretch_at(p, cut, pref, looked, end);
      lu = lt.u0;
    }
    ahead_n = min(kBatch, lt.u0 + lt.n - lu);
    ahead_page = -1;
    ahead_head = lt.head;
    if (lane / kBlocks < ahead_n) {
      const int key = lt.run.unit(lu + lane / kBlocks) * kUnit + lane % kBlocks * 16;
      // (blocks of a unit that no query sees are not looked at)
      if (key < lt.s.past + lt.s.n && (key + 16 > paged_first(p, lt.s, 0) || key < p.sinks)) {
        ahead_page = page_of(p.cache, lt.b, key);
        if (ahead_page < 0) atomicOr(status, kStatusBadPages);
      }
      ahead_slot = key & ((1 << p.cache.shift) - 1);
    }
    lu += ahead_n;
    looked += ahead_n;
  };
  int batch_n = 0, at = 0;        // units of the current batch, and those of them that are on their way
  uint32_t batch_seen = 0;        // bit l: block l is loaded
  const uint8_t* src[4];          // 4 bits: of this lane's block, codes and steps of keys and values
  int page = -1, head = 0, slot = 0;  // 16 bits: its coordinates
  auto next_batch = [&]() {
    batch_n = ahead_n;
    at = 0;
    batch_seen = __ballot_sync(0xffffffffu, ahead_page >= 0);
    page = ahead_page;
    head = ahead_head;
    slot = ahead_slot;
    if constexpr (k4) {
      const long long row = page_row(p.cache, head, slot);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        src[kv] = p.cache.data[kv] + page * p.cache.stride[kv] + row * row_bytes;
        src[2 + kv] = p.cache.meta[kv] + page * p.cache.meta_stride[kv] + row * meta_bytes;
      }
    }
    look_up();
  };
  look_up();
  const int units = static_cast<int>(end - begin);
  int loaded = 0, load_stage = 0;
  uint32_t seen_fifo = 0;  // blocks of the units on their way, the oldest lowest
  auto load_next = [&](int pending) {  // pending: units on their way before this one
    if (at == batch_n) next_batch();
    const uint32_t seen = (batch_seen >> (at * kBlocks)) & ((1u << kBlocks) - 1u);
    seen_fifo |= seen << (pending * kBlocks);
    uint8_t* dst = ring + load_stage * S::kStageBytes;
    uint64_t* full = &bar[warp][load_stage];
    const uint32_t block_bytes = k4 ? 2 * 16 * (row_bytes + meta_bytes) : 2 * 16 * 2 * kD;
    if (lane == 0) mbar_arrive_expect_tx(full, __popc(seen) * block_bytes);
    __syncwarp();
    if (lane / kBlocks == at && page >= 0) {
      const int k = lane % kBlocks;
      if constexpr (k4) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          bulk_load(dst + kv * S::kDataBytes + k * 16 * row_bytes, src[kv], 16 * row_bytes, full);
          bulk_load(dst + 2 * S::kDataBytes + kv * S::kMetaBytes + k * 16 * meta_bytes, src[2 + kv], 16 * meta_bytes, full);
        }
      } else {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int c = 0; c < kD / 64; ++c)
            tma_load_4d(dst + kv * S::kDataBytes + c * kUnit * 128 + k * 16 * 128, kv ? &tm.v : &tm.k, full, c * 64, slot, head, page);
      }
    }
    ++at;
    ++loaded;
    load_stage = load_stage + 1 == NS ? 0 : load_stage + 1;
  };
  while (loaded < NS && loaded < units) load_next(loaded);

  // ------------------------------------------------------------- products
  const float sl2 = p.scale_log2;
  const uint32_t magic = lds32(smem_u32(&s_magic));
  int done = 0, stage_at = 0, phase = 0;
  while (done < units) {
    const Stretch t = stretch_at(p, cut, pref, begin + done, end);
    const int row0 = t.tile * kRows, rows = min(kRows, t.s.n * p.group - row0);
    const int i0 = row0 / p.group, i1 = (row0 + rows - 1) / p.group;  // first and last query
    const int sees_all = t.s.past + i0 + 1, sees = t.s.past + i1 + 1;  // keys below: of every row, of some
    const int lo_some = paged_first(p, t.s, i0), lo_all = paged_first(p, t.s, i1);
    const int sinks = p.window > 0 ? p.sinks : 0;
    // this lane's rows of the scores: 8 nt + 2 t4, + 1
    int hi[kNT][2], lo[kNT][2];
    float m[kNT][2], l[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t4 + e, i = (row0 + r) / p.group;
        hi[nt][e] = r < rows ? t.s.past + i + 1 : 0;
        lo[nt][e] = paged_first(p, t.s, i);
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
    // Q^T as the second operand: column g of n-tile nt is row 8 nt + g
    uint32_t qf[kNT][kSteps][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int r = 8 * nt + g, rr = row0 + min(r, rows - 1), i = rr / p.group, j = rr - i * p.group;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) +
                          (static_cast<long long>(t.s.off + i) * p.hq + t.head * p.group + j) * p.d;
      if constexpr (k4) {
        // pairs (c, c + 4) of the eight elements that this lane's word of K holds
#pragma unroll
        for (int w = 0; w < kD / 32; ++w) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (w * 32 < p.d) v = *reinterpret_cast<const uint4*>(q + w * 32 + t4 * 8);
          qf[nt][2 * w][0] = __byte_perm(v.x, v.z, 0x5410);
          qf[nt][2 * w][1] = __byte_perm(v.x, v.z, 0x7632);
          qf[nt][2 * w + 1][0] = __byte_perm(v.y, v.w, 0x5410);
          qf[nt][2 * w + 1][1] = __byte_perm(v.y, v.w, 0x7632);
        }
      } else {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = 16 * s + 8 * e + 2 * t4;
            qf[nt][s][e] = c < p.d ? *reinterpret_cast<const uint32_t*>(q + c) : 0u;
          }
      }
    }
    float o[kNT][kSteps][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][s][e] = 0.f;

#pragma unroll 1
    for (int u = t.u0; u < t.u0 + t.n; ++u) {
      if (!mbar_wait_warp(&bar[warp][stage_at], phase, status)) {
        for (int i = done; i < loaded; ++i) {
          mbar_drain(&bar[warp][stage_at], phase);
          stage_at = stage_at + 1 == NS ? 0 : stage_at + 1;
          phase ^= stage_at == 0 ? 1 : 0;
        }
        return;
      }
      const uint32_t stage = smem_u32(ring + stage_at * S::kStageBytes);
      const uint32_t loaded_blocks = seen_fifo & ((1u << kBlocks) - 1u);
      const int key0 = t.run.unit(u) * kUnit;
      const bool full = loaded_blocks == (1u << kBlocks) - 1u && key0 + kUnit <= sees_all && (key0 >= lo_all || key0 + kUnit <= sinks);
      if (full || (loaded_blocks != 0 && key0 < sees && (key0 + kUnit > lo_some || key0 < sinks))) {
        // the unit, as code without masks for those that every row sees whole
        auto unit = [&](auto full_tag) {
          constexpr bool kFull = decltype(full_tag)::value;
          // ---- S^T, every other product into a second sum: each waits for the one before it
          float sc[kBlocks][kNT][4], odd[kBlocks][kNT][4];
#pragma unroll
          for (int k = 0; k < kBlocks; ++k)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[k][nt][e] = odd[k][nt][e] = 0.f;
          if constexpr (k4) {
            const uint32_t words = stage + g * row_bytes + t4 * 4;
            const uint32_t metas = stage + 2 * S::kDataBytes + g * meta_bytes;
#pragma unroll
            for (int w = 0; w < kD / 32; ++w) {
              if (!kExact && w * 32 >= p.d) break;
#pragma unroll
              for (int k = 0; k < kBlocks; ++k) {
                uint32_t a[2][4];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const int row = 16 * k + 8 * half;
                  const uint32_t mt = lds32(metas + row * meta_bytes + w * 4);
                  value_pairs<kBF16>(lds32(words + row * row_bytes + w * 16), __byte_perm(mt, mt, 0x1010),
                                     __byte_perm(mt, mt, 0x3232), magic, a[half]);
                }
                const uint32_t a0[4] = {a[0][0], a[1][0], a[0][1], a[1][1]}, a1[4] = {a[0][2], a[1][2], a[0][3], a[1][3]};
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                  mma16816<kBF16>(sc[k][nt], a0, qf[nt][2 * w][0], qf[nt][2 * w][1]);
                  mma16816<kBF16>(odd[k][nt], a1, qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
                }
              }
            }
          } else {
            // lanes 0-7: keys 0-7, columns 0-7; 8-15: keys 8-15; 16-31: columns 8-15
            const int row = lane & 15, piece = lane >> 4;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
              for (int k = 0; k < kBlocks; ++k) {
                uint32_t a[4];
                ldmatrix4<false>(a, stage + (s >> 2) * (kUnit * 128) + (k * 16 + row) * 128 + ((((s & 3) * 2 + piece) ^ (row & 7)) << 4));
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) mma16816<kBF16>(s & 1 ? odd[k][nt] : sc[k][nt], a, qf[nt][s][0], qf[nt][s][1]);
              }
          }
#pragma unroll
          for (int k = 0; k < kBlocks; ++k)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[k][nt][e] += odd[k][nt][e];
          // ---- which of them are seen; bit 4 k + e of the lane's scores
          [[maybe_unused]] uint32_t seen[kNT];
          if constexpr (!kFull) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              seen[nt] = 0;
#pragma unroll
              for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int key = key0 + 16 * k + g + (e >> 1) * 8;
                  if (((loaded_blocks >> k) & 1u) && key < hi[nt][e & 1] && (key >= lo[nt][e & 1] || key < sinks))
                    seen[nt] |= 1u << (4 * k + e);
                }
            }
          }
          auto is_seen = [&](int nt, int k, int e) {
            if constexpr (kFull) return true;
            else return ((seen[nt] >> (4 * k + e)) & 1u) != 0;
          };
          // ---- relative to the offset (log2 domain); raised where a score lies 8 above it
          float x[kBlocks][kNT][4];
          auto relative = [&]() {
            float top = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int k = 0; k < kBlocks; ++k) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  x[k][nt][e] = fmaf(sc[k][nt][e], sl2, -m[nt][e & 1]);
                  if constexpr (!kFull) x[k][nt][e] = is_seen(nt, k, e) ? x[k][nt][e] : -INFINITY;
                }
                top = max3(top, x[k][nt][0], x[k][nt][1]);
                top = max3(top, x[k][nt][2], x[k][nt][3]);
              }
            return top;
          };
          if (__any_sync(0xffffffffu, relative() > 8.f)) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float y = -INFINITY;
#pragma unroll
                for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if (is_seen(nt, k, e + 2 * h)) y = fmaxf(y, sc[k][nt][e + 2 * h] * sl2);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
                if (y > m[nt][e] + 8.f || (m[nt][e] == -INFINITY && y > -INFINITY)) {
                  const float alpha = ex2r(m[nt][e] - y);
                  m[nt][e] = y;
                  l[nt][e] *= alpha;
#pragma unroll
                  for (int s = 0; s < kSteps; ++s) {
                    o[nt][s][e] *= alpha;
                    o[nt][s][e + 2] *= alpha;
                  }
                }
              }
            relative();
          }
          // ---- P^T and O^T
#pragma unroll
          for (int k = 0; k < kBlocks; ++k) {
            uint32_t pf[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              float e4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // (a row that has seen no key yet has an infinite offset)
                e4[e] = ex2r(x[k][nt][e]);
                if constexpr (!kFull) e4[e] = is_seen(nt, k, e) ? e4[e] : 0.f;
                l[nt][e & 1] += e4[e];
              }
              pf[nt][0] = transpose8x8(pack2<kBF16>(e4[0], e4[1]));
              pf[nt][1] = transpose8x8(pack2<kBF16>(e4[2], e4[3]));
            }
            // values of keys that no row sees count as zeros, whatever they hold
            uint32_t keep[2] = {~0u, ~0u};
            if constexpr (!kFull) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                keep[h] = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int key = key0 + 16 * k + 8 * h + 2 * t4 + e;
                  if (((loaded_blocks >> k) & 1u) && key < sees && (key >= lo_some || key < sinks)) keep[h] |= 0xffffu << (16 * e);
                }
              }
            }
            if constexpr (k4) {
              const uint32_t words = stage + S::kDataBytes + (k * 16 + 2 * t4) * row_bytes + g * 4;
              const uint32_t metas = stage + 2 * S::kDataBytes + S::kMetaBytes + (k * 16 + 2 * t4) * meta_bytes + (g >> 2) * 4;
#pragma unroll
              for (int c = 0; c < kD / 64; ++c) {
                if (!kExact && c * 64 >= p.d) break;
                const bool in = kExact || c * 64 + g * 8 < p.d;  // (a last half of 32 elements is of half the lanes)
                uint32_t lo4[2][4], hi4[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t wa = 0, wb = 0, ma = 0, mb = 0;
                  if (in) {
                    wa = lds32(words + 8 * h * row_bytes + c * 32);
                    wb = lds32(words + (8 * h + 1) * row_bytes + c * 32);
                    ma = lds32(metas + 8 * h * meta_bytes + c * 8);
                    mb = lds32(metas + (8 * h + 1) * meta_bytes + c * 8);
                  }
                  const uint32_t step2 = __byte_perm(ma, mb, 0x5410) & keep[h], least2 = __byte_perm(ma, mb, 0x7632) & keep[h];
                  const uint32_t w0 = __byte_perm(wa, wb, 0x5410), w1 = __byte_perm(wa, wb, 0x7632);
                  value_pairs<kBF16>(w0, step2, least2, magic, lo4[h]);
                  value_pairs<kBF16>(w1, step2, least2, magic, hi4[h]);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const uint32_t af[4] = {lo4[0][y], hi4[0][y], lo4[1][y], hi4[1][y]};
#pragma unroll
                  for (int nt = 0; nt < kNT; ++nt) mma16816<kBF16>(o[nt][4 * c + y], af, pf[nt][0], pf[nt][1]);
                }
              }
            } else {
              // lanes 0-7: keys 0-7, columns 0-7; 8-15: columns 8-15; 16-31: keys 8-15
              const int row = k * 16 + (lane & 7) + ((lane >> 4) << 3), piece = (lane >> 3) & 1;
#pragma unroll
              for (int s = 0; s < kSteps; ++s) {
                uint32_t a[4];
                ldmatrix4<true>(a, stage + S::kDataBytes + (s >> 2) * (kUnit * 128) + row * 128 +
                                       ((((s & 3) * 2 + piece) ^ (row & 7)) << 4));
                if constexpr (!kFull) {
                  a[0] &= keep[0];
                  a[1] &= keep[0];
                  a[2] &= keep[1];
                  a[3] &= keep[1];
                }
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) mma16816<kBF16>(o[nt][s], a, pf[nt][0], pf[nt][1]);
              }
            }
          }
        };
        if (full) unit(std::true_type{});
        else unit(std::false_type{});
      }
      __syncwarp();  // every lane has read the stage
      ++done;
      seen_fifo >>= kBlocks;
      stage_at = stage_at + 1 == NS ? 0 : stage_at + 1;
      phase ^= stage_at == 0 ? 1 : 0;
      if (loaded < units) load_next(loaded - done);
    }

    // ---- the rows: sums over the lanes that hold other keys, then out or to a partial slot
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
    const bool whole = t.n == t.run.n;
    const int slot = 2 * mine + (t.u0 == 0 ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t4 + e;
        if (r >= rows) continue;
        const int rr = row0 + r, i = rr / p.group, j = rr - i * p.group;
        const long long at_row = static_cast<long long>(t.s.off + i) * p.hq + t.head * p.group + j;
        if (!bounds_ok(at_row < static_cast<long long>(p.total_q) * p.hq, status)) continue;
        const float inv = whole ? (l[nt][e] > 0.f ? 1.f / l[nt][e] : l[nt][e] == 0.f ? 0.f : NAN) : 1.f;
        if (g == 0) {
          if (whole) p.lse[at_row] = m[nt][e] * 0.69314718055994531f + logf(l[nt][e]);
          else parts.ml[static_cast<long long>(slot) * kRows + r] = make_float2(m[nt][e], l[nt][e]);
        }
        uint16_t* out = static_cast<uint16_t*>(p.out) + at_row * p.d;
        float* part = parts.o + (static_cast<long long>(slot) * kRows + r) * p.d;
        if constexpr (k4) {
          // elements 64 c + 8 g + 0..7 are this lane's
#pragma unroll
          for (int c = 0; c < kD / 64; ++c) {
            const int col = c * 64 + g * 8;
            if (col >= p.d) break;
            float f[8];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              f[x] = o[nt][4 * c + x][e] * inv;
              f[x + 4] = o[nt][4 * c + x][e + 2] * inv;
            }
            if (whole) {
              *reinterpret_cast<uint4*>(out + col) = make_uint4(pack2<kBF16>(f[0], f[1]), pack2<kBF16>(f[2], f[3]),
                                                               pack2<kBF16>(f[4], f[5]), pack2<kBF16>(f[6], f[7]));
            } else {
              *reinterpret_cast<float4*>(part + col) = make_float4(f[0], f[1], f[2], f[3]);
              *reinterpret_cast<float4*>(part + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int col = 16 * s + 8 * h + g;
              if (col >= p.d) continue;
              const float f = o[nt][s][e + 2 * h] * inv;
              if (whole) out[col] = static_cast<uint16_t>(pack2<kBF16>(f, 0.f));
              else part[col] = f;
            }
        }
      }
  }
}

template <int kD, int kNT, bool kBF16, bool k4>
static cudaError_t launch_rows_impl(const PagedParams& p, const PagedParts& parts, PagedCut* cut, cudaStream_t st) {
  using S = RowsShape<kD, kNT, k4>;
  *cut = PagedCut{S::kRows, S::kUnit, false};
  RowsMaps tm{};
  if (!k4 && (!make_tmap_pages(&tm.k, p.cache, 0, kBF16, 16) || !make_tmap_pages(&tm.v, p.cache, 1, kBF16, 16)))
    return cudaErrorInvalidValue;
  const int smem = S::kSmem + (p.batch + 1) * static_cast<int>(sizeof(long long));
  auto kern = k4 && p.d == kD ? paged_rows_kernel<kD, kNT, kBF16, k4, k4> : paged_rows_kernel<kD, kNT, kBF16, k4, false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem + (kPagedMaxBatch + 1) * 8);
  if (e != cudaSuccess) return e;
  kern<<<parts.slices / S::kWarps, S::kWarps * 32, smem, st>>>(p, parts, tm);
  return cudaGetLastError();
}

template <int kD, bool kBF16, bool k4>
static cudaError_t launch_rows_nt(const PagedParams& p, const PagedParts& parts, int rows, PagedCut* cut, cudaStream_t st) {
  if constexpr (!k4 && kD <= 128) {
    if (rows == 16) return launch_rows_impl<kD, 2, kBF16, k4>(p, parts, cut, st);
  }
  return launch_rows_impl<kD, 1, kBF16, k4>(p, parts, cut, st);
}

template <bool kBF16, bool k4>
static cudaError_t launch_rows_d(const PagedParams& p, const PagedParts& parts, int rows, PagedCut* cut, cudaStream_t st) {
  return p.d <= 64    ? launch_rows_nt<64, kBF16, k4>(p, parts, rows, cut, st)
         : p.d <= 128 ? launch_rows_nt<128, kBF16, k4>(p, parts, rows, cut, st)
                      : launch_rows_nt<256, kBF16, k4>(p, parts, rows, cut, st);
}

cudaError_t launch_paged_rows(const PagedParams& p, const PagedParts& parts, bool bf16, bool four, int rows,
                              PagedCut* cut, cudaStream_t st) {
  if (four)
    return bf16 ? launch_rows_d<true, true>(p, parts, rows, cut, st) : launch_rows_d<false, true>(p, parts, rows, cut, st);
  return bf16 ? launch_rows_d<true, false>(p, parts, rows, cut, st) : launch_rows_d<false, false>(p, parts, rows, cut, st);
}

int paged_rows(int batch, int total_q, int group, int d, bool four) {
  // In 16 bits a pass of 16 rows takes hardly longer than one of 8: 64 sequences of 2000 keys with 12 rows
  // 113 us in one pass, 187 in two; with 8 rows 104 and 105. In 4 bits it takes twice as long, for the products and
  // scores of a second n-tile: with 12 rows 115 us in one pass and 106 in two, so eight are taken always.
  // (Above head_dim 128 16 rows' output and queries would not fit the registers.)
  if (four || d > 128) return 8;
  const long long each = (static_cast<long long>(total_q) + batch - 1) / batch * group;
  return each <= 8 ? 8 : 16;
}

int paged_warps(int d, bool four, int rows) {
  auto pick = [&](auto shape_d) {
    constexpr int kD = decltype(shape_d)::value;
    if (four) return RowsShape<kD, 1, true>::kWarps;
    return rows == 16 ? RowsShape<kD, kD <= 128 ? 2 : 1, false>::kWarps : RowsShape<kD, 1, false>::kWarps;
  };
  const int warps = d <= 64 ? pick(std::integral_constant<int, 64>{})
                    : d <= 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 256>{});
  return warps * kPagedSMs;
}

}  // namespace teattn
