// lm_device.h -- device helpers shared by the selective state-space and loss
// kernels: rows of 16- or 32-bit activations at any element alignment, and
// the gate functions in 32 bits.
#pragma once

#include "../h3conv_device.h"
#include "lm_internal.h"

namespace h3c {

// This block's number in a grid that grid_of() made.
__device__ __forceinline__ int64_t block_id() { return blockIdx.x + (int64_t)blockIdx.z * kGridX; }

// Valid steps of batch row b.
__device__ __forceinline__ int64_t row_len(const int32_t *lengths, int64_t b, int64_t N) {
    if (!lengths) return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n > N ? N : n);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One element to and from fp32; bf16 rounds to nearest even in hardware.
template <int IO>
__device__ __forceinline__ float to_f(typename io_elem<IO>::T v) {
    if constexpr (IO == IO_BF16) return __uint_as_float((uint32_t)v << 16);
    else return (float)v;
}
template <int IO>
__device__ __forceinline__ typename io_elem<IO>::T from_f(float v) {
    if constexpr (IO == IO_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    else return (typename io_elem<IO>::T)v;
}

// n consecutive elements at any element alignment (rows of an odd length
// start anywhere): the target reads and writes unaligned vectors.
template <class T, int n>
struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[n]; };

template <int IO, int n>
__device__ __forceinline__ void ld_row(const typename io_elem<IO>::T *p, float (&o)[n]) {
    using T = typename io_elem<IO>::T;
    const Pack<T, n> r = *reinterpret_cast<const Pack<T, n> *>(p);
#pragma unroll
    for (int i = 0; i < n; ++i) o[i] = to_f<IO>(r.v[i]);
}
// p[i] for i < valid, else zero
template <int IO, int n>
__device__ __forceinline__ void ld_row(const typename io_elem<IO>::T *p, float (&o)[n], int64_t valid) {
    if (valid >= n) {
        ld_row<IO, n>(p, o);
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) o[i] = i < valid ? to_f<IO>(p[i]) : 0.f;
    }
}
template <int IO, int n>
__device__ __forceinline__ void st_row(typename io_elem<IO>::T *p, const float (&o)[n], int64_t valid) {
    using T = typename io_elem<IO>::T;
    if (valid >= n) {
        Pack<T, n> r;
#pragma unroll
        for (int i = 0; i < n; ++i) r.v[i] = from_f<IO>(o[i]);
        *reinterpret_cast<Pack<T, n> *>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i < valid) p[i] = from_f<IO>(o[i]);
    }
}

// 1 / (1 + e^-x); e^-x = inf gives 0.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// log(1 + e^x).  For small e = e^x, 1 + e rounds; log(w) e / (w - 1) with
// w = fl(1 + e) undoes that rounding, so the relative error stays near one
// ulp down to the smallest step sizes.
__device__ __forceinline__ float softplus(float x) {
    const float e = __builtin_amdgcn_exp2f(kLog2e * fminf(x, 20.f));
    const float w = 1.f + e, d = w - 1.f;
    const float l = kLn2 * __builtin_amdgcn_logf(w);
    const float r = d > 0.f ? l * e * __builtin_amdgcn_rcpf(d) : e;
    return x > 20.f ? x : (x != x ? x : r);
}

}  // namespace h3c
