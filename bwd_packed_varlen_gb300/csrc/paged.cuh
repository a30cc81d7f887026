// Paged key/value caches: where a position's keys and values lie, and the 4-bit form.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/te_attn.h"
#include "common.cuh"
#include "sm103_ptx.cuh"

namespace teattn {

struct PagedCache {
  uint8_t* data[2];  // keys, values
  uint8_t* meta[2];  // 4 bits: step and least value of every 32 elements
  long long stride[2], meta_stride[2];  // bytes from page to page
  const int* table;
  long long table_stride;
  int num_pages, max_pages;
  int shift;      // page_size = 1 << shift
  int hkv, d;
  int row_bytes;  // of one token and head in data; in meta: d / 8
};

// Page of position pos of sequence b; -1 if it is behind the table or outside the cache.
__device__ __forceinline__ int page_of(const PagedCache& c, int b, int pos) {
  const int n = pos >> c.shift;
  if (n >= c.max_pages) return -1;
  const int page = c.table[b * c.table_stride + n];
  return page >= 0 && page < c.num_pages ? page : -1;
}

// Sequence whose rows [cu_pad[b], cu_pad[b + 1]) hold row r; -1: none. A whole warp works on one row:
// one trip to memory for up to 32 sequences, of which the last that begins at or before the row is
// it. Only where that one does not hold the row are all spans looked at: none does, or offsets that fall
// back have their own order (and may give the row several sequences: one of them then).
__device__ __forceinline__ int sequence_at(const int* cu_pad, int batch, int r) {
  int before = 0;
  for (int k = threadIdx.x & 31; k < batch; k += 32) before += cu_pad[k] <= r ? 1 : 0;
  int b = __reduce_add_sync(0xffffffffu, before) - 1;
  if (b >= 0 && cu_pad[b] <= r && r < cu_pad[b + 1]) return b;
  b = -1;
#pragma unroll 1
  for (int k = threadIdx.x & 31; k < batch; k += 32)
    if (cu_pad[k] <= r && r < cu_pad[k + 1]) b = k;
  return __reduce_max_sync(0xffffffffu, b);
}

// Token row of (page, head, slot) within a page, in units of rows.
__device__ __forceinline__ long long page_row(const PagedCache& c, int head, int slot) {
  return (static_cast<long long>(head) << c.shift) + slot;
}

// The two 16-bit numbers of a group: step in the low half, least value in the high one.
template <bool kBF16>
__device__ __forceinline__ uint32_t pack_meta(float step, float least) {
  if constexpr (kBF16)
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rz(step))) |
           static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(least))) << 16;
  else
    return static_cast<uint32_t>(__half_as_ushort(__float2half_rz(step))) |
           static_cast<uint32_t>(__half_as_ushort(__float2half_rn(least))) << 16;
}

// Codes become numbers by a magic one, the usual way for small integers: put into the fraction of 128
// (bf16) or 1024 (fp16), which is then taken off; both steps are exact.
template <bool kBF16>
constexpr uint32_t kCodeMagic = kBF16 ? 0x43004300u : 0x64006400u;

// The two codes in bits 0-3 and 16-19 of w (kHigh, fp16 alone, whose fraction has room for them:
// bits 4-7 and 20-23). `magic` is kCodeMagic from a place that the compiler cannot see into: with
// mask and magic both constants it spends two instructions on the one that does both.
template <bool kBF16, bool kHigh = false>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "r"(kHigh ? 0x00f000f0u : 0x000f000fu), "r"(magic));  // (w & mask) | magic
  if constexpr (kBF16) {
    static_assert(!kHigh, "bf16 keeps seven bits of a fraction");
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), __float2bfloat162_rn(128.f));
    return *reinterpret_cast<const uint32_t*>(&y);
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&x);
    const __half2 y = kHigh ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-64.f)) : __hsub2(h, __float2half2_rn(1024.f));
    return *reinterpret_cast<const uint32_t*>(&y);
  }
}

// step * code + least for a pair, rounded once to 16 bits: the value that the codes stand for.
template <bool kBF16>
__device__ __forceinline__ uint32_t value_pair(uint32_t codes, uint32_t step2, uint32_t least2) {
  uint32_t r;
  if constexpr (kBF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(codes), "r"(step2), "r"(least2));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(codes), "r"(step2), "r"(least2));
  return r;
}

// The four pairs (i, i + 4) of a word's codes as values.
template <bool kBF16>
__device__ __forceinline__ void value_pairs(uint32_t w, uint32_t step2, uint32_t least2, uint32_t magic, uint32_t (&r)[4]) {
  if constexpr (kBF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = value_pair<true>(code_pair<true>(w >> (4 * i), magic), step2, least2);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      r[i] = value_pair<false>(code_pair<false>(w >> (4 * i), magic), step2, least2);
      r[i + 1] = value_pair<false>(code_pair<false, true>(w >> (4 * i), magic), step2, least2);
    }
  }
}

// The eight elements of a word of codes, in order.
template <bool kBF16>
__device__ __forceinline__ uint4 dequantize8(uint32_t codes, uint32_t meta, uint32_t magic) {
  uint32_t r[4];
  value_pairs<kBF16>(codes, __byte_perm(meta, meta, 0x1010), __byte_perm(meta, meta, 0x3232), magic, r);
  return make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410), __byte_perm(r[0], r[1], 0x7632),
                    __byte_perm(r[2], r[3], 0x7632));
}

// Host: the device form of a cache after its checks: TE_OK or an error code.
int api_paged_cache(const te_attn_paged_cache* c, PagedCache* out);

}  // namespace teattn
