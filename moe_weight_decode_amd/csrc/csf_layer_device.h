// Device helpers of the layer operators: wave reductions and 8-element runs of
// bfloat16, half or float rows at any element alignment.  Internal linkage.
#pragma once

#include "csf_device.h"
#include "csf_layer.h"

namespace csf {
namespace {

// A launch holds fewer than 2^32 threads, and a larger one runs in part without an
// error: more workgroups than kGridMost (of up to 1024 threads) take several
// launches, the first workgroup of each in a.first.
constexpr uint32_t kGridMost = 1u << 21;

template <typename Args, typename Launch>
void launch_groups(Args a, uint32_t groups, Launch &&launch) {
    for (a.first = 0; a.first < groups; a.first += kGridMost) {
        const uint32_t left = groups - a.first;
        launch(a, dim3(left < kGridMost ? left : kGridMost));
    }
}

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
// 16 and 8 bytes at any 2-byte alignment: gfx950 loads and stores them whole
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_byte __attribute__((ext_vector_type(2), aligned(1)));

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_or_zero(float v) {
    return __uint_as_float(dpp_or_zero<CTRL, ROWS>(__float_as_uint(v)));
}

// Sum over the wave, the same in every lane: shifts by 1, 2, 4, 8 within rows
// of 16 lanes, then the rows' last lanes broadcast onward; lane 63 holds it.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_or_zero<0x111>(v);
    v += dpp_or_zero<0x112>(v);
    v += dpp_or_zero<0x114>(v);
    v += dpp_or_zero<0x118>(v);
    v += dpp_or_zero<0x142, 0xA>(v);
    v += dpp_or_zero<0x143, 0xC>(v);
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Largest unsigned value over the wave, the same in every lane (0 is the identity).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp_or_zero<0x111, 0xF>(v));
    v = max(v, dpp_or_zero<0x112, 0xF>(v));
    v = max(v, dpp_or_zero<0x114, 0xF>(v));
    v = max(v, dpp_or_zero<0x118, 0xF>(v));
    v = max(v, dpp_or_zero<0x142, 0xA>(v));
    v = max(v, dpp_or_zero<0x143, 0xC>(v));
    return __builtin_amdgcn_readlane(v, 63);
}

// Two floats rounded to the type (to nearest, ties to even), packed.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__bf16>(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2bf));
}
template <>
__device__ __forceinline__ uint32_t pack2<_Float16>(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2h));
}

template <typename T>
__device__ __forceinline__ v2f unpack2(uint32_t v);
template <>
__device__ __forceinline__ v2f unpack2<__bf16>(uint32_t v) {
    return (v2f){__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)};
}
template <>
__device__ __forceinline__ v2f unpack2<_Float16>(uint32_t v) {
    return __builtin_convertvector(__builtin_bit_cast(v2h, v), v2f);
}

// Elements p[0 .. 7] (n of them, the rest 0) as floats.
template <typename T>
__device__ __forceinline__ void load8(const T *p, uint32_t n, float (&v)[8]) {
    if (n >= 8u) {
        if constexpr (sizeof(T) == 4) {
            const f32x4_any a = *reinterpret_cast<const f32x4_any *>(p), b = *reinterpret_cast<const f32x4_any *>(p + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const u32x4_any a = *reinterpret_cast<const u32x4_any *>(p);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const v2f f = unpack2<T>(w[i]);
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] = i < n ? (float)p[i] : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, uint32_t n, const float (&v)[8]) {
    if (n >= 8u) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4_any *>(p) = (f32x4_any){v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4_any *>(p + 4) = (f32x4_any){v[4], v[5], v[6], v[7]};
        } else {
            *reinterpret_cast<u32x4_any *>(p) = (u32x4_any){pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                           pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])};
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            if (i < n) p[i] = (T)v[i];
    }
}

}  // namespace
}  // namespace csf
