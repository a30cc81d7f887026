// Shared-prefix attention, backward: the sum of the prefix gradients' parts. The dQ and
// dK/dV kernels are the packed problem's, with the prefix as further key tiles.
#include <cuda_runtime.h>

#include "attn_prefix.cuh"
#include "sm103_ptx.cuh"

namespace teattn {

// dK_prefix = scale sum_s part_dk[s], dV_prefix = sum_s part_dv[s] in the order of s, in
// fp32, rounded once; rows that no query sees (behind the real length, or without any
// query) are zeros. With one part the dK/dV kernel wrote the seen rows itself. Memory-
// bound: every fp32 part is read once, 32 bytes per thread and part.
template <bool kBF16>
__global__ void __launch_bounds__(256) prefix_sum_kernel(const __grid_constant__ PrefixBwd p) {
  const int seen = p.total_q > 0 ? prefix_keys(p) : 0;
  const size_t row_elems = static_cast<size_t>(p.hkv) * p.d;
  const size_t n = static_cast<size_t>(p.prefix_rows) * row_elems;
  const size_t first = p.splits > 1 ? 0 : static_cast<size_t>(seen) * row_elems;
  const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x * 8;
  for (size_t i = first + (static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; i < n; i += step) {
    const bool live = i < static_cast<size_t>(seen) * row_elems;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float a[8] = {};
      if (live) {
        const float* src = (w == 0 ? p.part_dk : p.part_dv) + i;
        for (int s = 0; s < p.splits; ++s) {
          const float4 x = *reinterpret_cast<const float4*>(src + s * n), y = *reinterpret_cast<const float4*>(src + s * n + 4);
          a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
          a[4] += y.x; a[5] += y.y; a[6] += y.z; a[7] += y.w;
        }
      }
      const float f = w == 0 ? p.scale : 1.f;
      uint4 v;
      v.x = pack2<kBF16>(a[0] * f, a[1] * f);
      v.y = pack2<kBF16>(a[2] * f, a[3] * f);
      v.z = pack2<kBF16>(a[4] * f, a[5] * f);
      v.w = pack2<kBF16>(a[6] * f, a[7] * f);
      *reinterpret_cast<uint4*>(static_cast<char*>(w == 0 ? p.dkp : p.dvp) + i * 2) = v;
    }
  }
}

cudaError_t launch_prefix_sum(const PrefixBwd& p, bool bf16, int num_sms, cudaStream_t st) {
  const long long blocks = (static_cast<long long>(p.prefix_rows) * p.hkv * p.d / 8 + 255) / 256;
  if (blocks == 0) return cudaSuccess;
  const int grid = static_cast<int>(blocks < num_sms * 8 ? blocks : num_sms * 8);
  if (bf16) prefix_sum_kernel<true><<<grid, 256, 0, st>>>(p);
  else prefix_sum_kernel<false><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace teattn
