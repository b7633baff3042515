// The two 16-bit element types of the attention-side operators, as bit
// patterns: conversion to and from fp32 (round to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

inline bool known_dtype(int d) { return d == MOE_DT_BF16 || d == MOE_DT_F16; }

// BF: bf16, else fp16
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    if (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (BF) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool BF>
__device__ __forceinline__ float to_f32(uint16_t u) {
    return BF ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}
template <bool BF>
__device__ __forceinline__ uint16_t from_f32(float v) {
    return BF ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

}  // namespace moe
