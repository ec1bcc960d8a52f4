// Device helpers shared by the operators around the layer: eight elements of a
// row as floats, and sums and maxima over lanes and workgroups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mega_moe.h"

namespace mega_moe {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Two floats as packed BF16, rounded to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ void unpack8(const u32x4_t& d, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(d[i] << 16);
        v[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
    }
}

// Elements i .. i + 7 as they lie in memory: one 16-byte word or two.
template <bool F32>
__device__ __forceinline__ const u32x4_t* raw8(const void* p, size_t i) {
    if constexpr (F32) return reinterpret_cast<const u32x4_t*>(static_cast<const float*>(p) + i);
    else return reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i);
}

template <bool F32, int N>
__device__ __forceinline__ void values8(const u32x4_t (&d)[N], float (&v)[8]) {
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(d[0][j]);
            v[4 + j] = __uint_as_float(d[N - 1][j]);
        }
    } else {
        unpack8(d[0], v);
    }
}

// Elements i .. i+7 (i a multiple of 8, p 16-byte aligned).
template <bool F32>
__device__ __forceinline__ void load8(const void* p, size_t i, float (&v)[8]) {
    if constexpr (F32) {
        const u32x4_t* q = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(p) + i);
        const u32x4_t a = q[0], b = q[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(a[j]);
            v[4 + j] = __uint_as_float(b[j]);
        }
    } else {
        unpack8(*reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i), v);
    }
}

// The same with the type as a uniform run-time value.
__device__ __forceinline__ void load8(const void* p, int type, size_t i, float (&v)[8]) {
    if (type == MEGA_MOE_F32) load8<true>(p, i, v);
    else load8<false>(p, i, v);
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, size_t i, const float (&v)[8]) {
    if constexpr (F32) {
        u32x4_t a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = __float_as_uint(v[j]);
            b[j] = __float_as_uint(v[4 + j]);
        }
        u32x4_t* q = reinterpret_cast<u32x4_t*>(static_cast<float*>(p) + i);
        q[0] = a;
        q[1] = b;
    } else {
        u32x4_t d;
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i) = d;
    }
}

__device__ __forceinline__ void store8(void* p, int type, size_t i, const float (&v)[8]) {
    if (type == MEGA_MOE_F32) store8<true>(p, i, v);
    else store8<false>(p, i, v);
}

// Every lane gets the wave's sum; the order is fixed.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

// Sums of N values over the workgroup (up to 16 waves), the waves' sums added
// in order.  `part` is an LDS array that no earlier sum of the same phase
// uses; a barrier must lie between two uses of one.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (&part)[16][N]) {
    const int wave = threadIdx.x >> 6, waves = (blockDim.x + 63) >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) part[wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = part[0][i];
    for (int w = 1; w < waves; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += part[w][i];
    }
}

// The same over groups of nt threads (whole waves), each for itself; every
// group of the workgroup calls it.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (&part)[16][N], int group, int nt) {
    const int wave = threadIdx.x >> 6, waves = nt >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) part[wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = part[group * waves][i];
    for (int w = 1; w < waves; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += part[group * waves + w][i];
    }
}

}  // namespace mega_moe
