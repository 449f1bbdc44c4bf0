// op_elem.cuh -- element access and reductions shared by the model
// operators' kernels.  Values are widened to binary32 when read and rounded
// once when written.
#pragma once

#include <cuda_fp8.h>

#include "elem_ops.cuh"

namespace rar {

template <int DT>
__device__ __forceinline__ float widen(uint32_t bits) {
    if constexpr (DT == DT_F32) return __uint_as_float(bits);
    else if constexpr (DT == DT_BF16) return bf16_bits_to_float(bits & 0xFFFFu);
    else return f16_bits_to_float(bits & 0xFFFFu);
}
template <int DT>
__device__ __forceinline__ uint32_t narrow(float f) {
    if constexpr (DT == DT_F32) return __float_as_uint(f);
    else if constexpr (DT == DT_BF16) return float_to_bf16_bits(f);
    else return float_to_f16_bits(f);
}
template <int DT>
__device__ __forceinline__ float load_f(const void *base, long long i) {
    return widen<DT>(load_elem<DT>(static_cast<const char *>(base), i));
}
template <int DT>
__device__ __forceinline__ void store_f(void *base, long long i, float f) {
    store_elem<DT>(static_cast<char *>(base), i, narrow<DT>(f));
}

// An index array of 32- or 64-bit signed integers.
__device__ __forceinline__ long long load_index(const void *base, int bytes, long long i) {
    return bytes == 8 ? __ldg(static_cast<const long long *>(base) + i) : (long long)__ldg(static_cast<const int *>(base) + i);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {  // NaN is passed over
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
// Sum over the block in a fixed order; `red` holds a float per warp.  Every
// thread gets the result, and may reuse `red` after its next barrier.
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = warp_sum(v);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < (int)blockDim.x / 32; w++) t += red[w];
    return t;
}

// The scale of a group whose largest magnitude is amax: the e4m3 range
// [-448, 448] spans the group; never 0, infinite or NaN.
__device__ __forceinline__ float scale_of(float amax) {
    return fmaxf(__fdiv_rn(fminf(amax, 3.402823466e38f), 448.0f), 1.175494351e-38f);
}
__device__ __forceinline__ uint8_t to_e4m3(float v) {
    return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// Calls f(IntC<dtype>{}) for a floating dtype.
template <typename F>
cudaError_t dispatch_float(int dtype, F &&f) {
    switch (dtype) {
    case DT_F32: return f(IntC<DT_F32>{});
    case DT_BF16: return f(IntC<DT_BF16>{});
    case DT_F16: return f(IntC<DT_F16>{});
    }
    return cudaErrorInvalidValue;
}

}  // namespace rar
