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

// Two neighbouring codes c0, c1 < 16, given as bits 0-3 and 16-19, as numbers: put into the
// fraction of 128 (bf16) or 1024 (fp16), which is then taken off; both steps are exact.
template <bool kBF16>
__device__ __forceinline__ uint32_t code_pair(uint32_t bits) {
  if constexpr (kBF16) {
    const uint32_t w = bits | 0x43004300u;
    const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(128.f));
    return *reinterpret_cast<const uint32_t*>(&x);
  } else {
    const uint32_t w = bits | 0x64006400u;
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1024.f));
    return *reinterpret_cast<const uint32_t*>(&x);
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

// The eight elements of a word of codes, in order.
template <bool kBF16>
__device__ __forceinline__ uint4 dequantize8(uint32_t codes, uint32_t meta) {
  const uint32_t step2 = __byte_perm(meta, meta, 0x1010), least2 = __byte_perm(meta, meta, 0x3232);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = codes >> (8 * i), bits = (c & 15u) | (c & 0xf0u) << 12;
    r[i] = value_pair<kBF16>(code_pair<kBF16>(bits), step2, least2);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Host: the device form of a cache after its checks: TE_OK or an error code.
int api_paged_cache(const te_attn_paged_cache* c, PagedCache* out);

}  // namespace teattn
