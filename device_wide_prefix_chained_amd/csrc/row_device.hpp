// row_device.hpp -- parts shared by the norms' kernels: a row in the registers
// of a workgroup, eight neighbouring channels a thread, and sums over it.
#pragma once

#include "block_device.hpp"

namespace dwps {

constexpr int kVec = 8;  // neighbouring channels of a thread
constexpr int kMostWaves = 16;

// The workgroup's sums of n values, in every thread: wave sums meet in
// shared memory, and every row of lanes adds the up to 16 of them.
template <int n>
__device__ __forceinline__ void group_totals(float (&v)[n], float (*shared)[kMostWaves]) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = wave_total(v[i]);
    const uint32_t waves = blockDim.x >> 6;
    if (waves == 1u) return;
    if ((threadIdx.x & 63u) == 0u) {
#pragma unroll
        for (int i = 0; i < n; ++i) shared[i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
    const uint32_t l = threadIdx.x & 15u;
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = row_total(l < waves ? shared[i][l] : 0.0f);
}

// n neighbouring values from p, or `none` without p; `have` of them exist.
template <class T, int n>
__device__ __forceinline__ void load_n(float (&v)[n], const T *p, uint32_t have, float none) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = (uint32_t)i < have ? none : 0.0f;
    } else if (have >= (uint32_t)n) {
        const Pack<T, n> r = *reinterpret_cast<const Pack<T, n> *>(p);
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = (float)r.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = (uint32_t)i < have ? (float)p[i] : 0.0f;
    }
}
template <class T, int n>
__device__ __forceinline__ void store_n(T *p, const float (&v)[n], uint32_t have) {
    if (have >= (uint32_t)n) {
        Pack<T, n> r;
#pragma unroll
        for (int i = 0; i < n; ++i) r.v[i] = (T)v[i];
        *reinterpret_cast<Pack<T, n> *>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if ((uint32_t)i < have) p[i] = (T)v[i];
    }
}
template <class T>
__device__ __forceinline__ const T *at_row(const void *p, int64_t t, int64_t stride, uint32_t c) {
    return p ? static_cast<const T *>(p) + t * stride + c : nullptr;
}
__device__ __forceinline__ const float *at_col(const float *p, uint32_t c) { return p ? p + c : nullptr; }

// Eight activations as they were loaded: 16-bit types stay packed until they
// are used, so that nothing waits for them before.
template <class T>
struct Raw8 {
    float v[8];
    __device__ __forceinline__ void load(const T *p) {
        const Pack<T, 8> r = *reinterpret_cast<const Pack<T, 8> *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)r.v[i];
    }
    __device__ __forceinline__ void values(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[i];
    }
};
template <class T>
struct Raw8Packed {
    typedef uint32_t words __attribute__((ext_vector_type(4)));
    typedef words words_at_2 __attribute__((aligned(2), may_alias));
    words w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const words_at_2 *>(p); }
    __device__ __forceinline__ void values(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t b = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            o[i] = (float)__builtin_bit_cast(T, b);
        }
    }
};
template <>
struct Raw8<bf16_t> : Raw8Packed<bf16_t> {};
template <>
struct Raw8<f16_t> : Raw8Packed<f16_t> {};

}  // namespace dwps
