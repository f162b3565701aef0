// Device helpers of the state space and token score kernels: element types and row lengths.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ssm_internal.h"

namespace rnngb {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Row n's length, clamped to [0, S]; one outside is reported in *status.
__device__ __forceinline__ int64_t row_length(const int32_t* lens, int64_t n, int64_t S, int* status)
{
    if (!lens) return S;
    const int64_t len = lens[n];
    if (len < 0 || len > S) {
        *status = 2;   // RNN_ERR_INVALID_INPUT
        return len < 0 ? 0 : S;
    }
    return len;
}

}  // namespace rnngb
