// What the library's entry points share on the host (internal; defined in
// te_attn_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/te_attn.h"

namespace teattn {

// Set the thread's last error and return the code / clear it and return TE_OK.
int api_fail(int code, const char* msg) noexcept;
int api_ok() noexcept;
int api_cuda_fail(cudaError_t e, const char* where) noexcept;

// SM count of the current device (0: no device).
int api_num_sms();

// The argument checks that every attention entry point shares: TE_OK or an error code.
int api_check_common(int batch, int total_q, int total_kv, int hq, int hkv, int d, float attn_scale,
                     int mask_type, int dtype, const int32_t* cu_q, const int32_t* cu_kv,
                     const int32_t* cu_q_pad, const int32_t* cu_kv_pad);

// Runs launch(ctx) between two events on `st` when kernel timing is enabled.
cudaError_t api_timed(int kernel, cudaStream_t st, cudaError_t (*launch)(void*), void* ctx);

template <typename F>
cudaError_t api_timed(int kernel, cudaStream_t st, F&& f) {
  using T = std::remove_reference_t<F>;
  struct Call {
    static cudaError_t go(void* c) { return (*static_cast<T*>(c))(); }
  };
  return api_timed(kernel, st, &Call::go, &f);
}

}  // namespace teattn
