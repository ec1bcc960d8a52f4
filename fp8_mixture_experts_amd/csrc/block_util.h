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

template <bool F32>
__device__ __forceinline__ void values8(const u32x4_t& d0, const u32x4_t& d1, float (&v)[8]) {
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(d0[j]);
            v[4 + j] = __uint_as_float(d1[j]);
        }
    } else {
        unpack8(d0, v);
    }
}

template <bool F32, int N>
__device__ __forceinline__ void values8(const u32x4_t (&d)[N], float (&v)[8]) {
    values8<F32>(d[0], d[N - 1], v);
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

__device__ __forceinline__ u32x4_t pack8(const float (&v)[8]) {
    u32x4_t d;
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    return d;
}

// Elements i .. i+7 (i a multiple of 8, p 16-byte aligned).  STREAM: what is read
// again only after a whole layer; it leaves the caches to what is read next.
template <bool F32, bool STREAM = false>
__device__ __forceinline__ void store8(void* p, size_t i, const float (&v)[8]) {
    const auto put = [](u32x4_t* q, const u32x4_t& d) {
        if constexpr (STREAM) __builtin_nontemporal_store(d, q);
        else *q = d;
    };
    if constexpr (F32) {
        u32x4_t a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = __float_as_uint(v[j]);
            b[j] = __float_as_uint(v[4 + j]);
        }
        u32x4_t* q = reinterpret_cast<u32x4_t*>(static_cast<float*>(p) + i);
        put(q, a);
        put(q + 1, b);
    } else {
        put(reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i), pack8(v));
    }
}

template <bool F32>
__device__ __forceinline__ void stream8(void* p, size_t i, const float (&v)[8]) {
    store8<F32, true>(p, i, v);
}

// The same with the type as a uniform run-time value.
__device__ __forceinline__ void stream8(void* p, int type, size_t i, const float (&v)[8]) {
    if (type == MEGA_MOE_F32) stream8<true>(p, i, v);
    else stream8<false>(p, i, v);
}

// Another lane's value by a data-parallel move: 1 and 2 are xor within a quad,
// 4 and 8 (mirrors of 8 and of 16 lanes) pair groups whose lanes agree.
template <int D>
__device__ __forceinline__ uint32_t lane_pair(uint32_t v) {
    constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, ctrl, 0xf, 0xf, true);
}

// op over LANES neighbouring lanes (8, 16, 32 or 64); every lane gets the result, and
// the order is fixed.  All steps are vector moves, none goes through LDS.
template <int LANES, typename F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, F op) {
    v = op(v, lane_pair<1>(v));
    v = op(v, lane_pair<2>(v));
    v = op(v, lane_pair<4>(v));
    if constexpr (LANES >= 16) v = op(v, lane_pair<8>(v));
    if constexpr (LANES >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    if constexpr (LANES == 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    return __uint_as_float(over_lanes<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
    return __uint_as_float(over_lanes<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}

template <int LANES>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
    return over_lanes<LANES>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// The same for a wave of float64 values, moved in halves.
template <typename F>
__device__ __forceinline__ double over_wave(double v, F op) {
    const auto step = [&](auto move) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        uint32_t lo[2], hi[2];
        move((uint32_t)b, lo);
        move((uint32_t)(b >> 32), hi);
        v = op(__builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]),
               __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]));
    };
    step([](uint32_t x, uint32_t (&o)[2]) { o[0] = x, o[1] = lane_pair<1>(x); });
    step([](uint32_t x, uint32_t (&o)[2]) { o[0] = x, o[1] = lane_pair<2>(x); });
    step([](uint32_t x, uint32_t (&o)[2]) { o[0] = x, o[1] = lane_pair<4>(x); });
    step([](uint32_t x, uint32_t (&o)[2]) { o[0] = x, o[1] = lane_pair<8>(x); });
    step([](uint32_t x, uint32_t (&o)[2]) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        o[0] = r[0], o[1] = r[1];
    });
    step([](uint32_t x, uint32_t (&o)[2]) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        o[0] = r[0], o[1] = r[1];
    });
    return v;
}

__device__ __forceinline__ float wave_sum(float v) { return lanes_sum<64>(v); }
__device__ __forceinline__ float wave_max(float v) { return lanes_max<64>(v); }

__device__ __forceinline__ double wave_sum(double v) {
    return over_wave(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ double wave_max(double v) {
    return over_wave(v, [](double a, double b) { return fmax(a, b); });
}

// Sums of N values over groups of nt threads (whole waves, up to 16), each for
// itself; every group of the workgroup calls it.  The waves' sums meet in
// `part`, an LDS array that no earlier sum of the same phase uses; a barrier
// must lie between two uses of one.  Sixteen lanes then take a wave's sum each:
// one read and four moves, not a chain of reads.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (&part)[16][N], int group, int nt) {
    const int wave = threadIdx.x >> 6, waves = nt >> 6, lane = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) part[wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<16>(lane < waves ? part[group * waves + lane][i] : 0.0f);
}

// The same over the workgroup.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (&part)[16][N]) {
    group_sum(v, part, 0, (int)blockDim.x);
}

}  // namespace mega_moe
