// Shared-prefix attention: launch parameters of its kernels.
#pragma once

#include "common.cuh"

namespace teattn {

// A packed problem (AttnParams) whose queries also see every key of a prefix that all
// sequences share: kp, vp [prefix_rows, hkv, d], the first prefix_keys() rows real.
struct PrefixParams : AttnParams {
  const void* kp;
  const void* vp;
  void* dkp;
  void* dvp;
  const int* prefix_len;  // may be null: all prefix_rows
  int prefix_rows;
};

// Real prefix keys; a length outside [0, prefix_rows] counts as 0 (and is reported).
__device__ __forceinline__ int prefix_keys(const PrefixParams& p) {
  if (!p.prefix_len) return p.prefix_rows;
  const int n = *p.prefix_len;
  return n >= 0 && n <= p.prefix_rows ? n : 0;
}

cudaError_t launch_prefix_fwd(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_prefix_bwd(const PrefixParams& p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace teattn
