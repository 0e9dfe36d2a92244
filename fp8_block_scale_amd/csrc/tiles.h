// Helpers that the grouped and dense products and the row-wise operators share.
#pragma once
#include "common.h"
#include "linear.h"

namespace moe {

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Two FP32 values to FP16 (else BF16) at once (one packed conversion, round to nearest even).
template <bool F16>
__device__ __forceinline__ uint32_t to16x2(float lo, float hi) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2f v = {lo, hi};
    if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2h));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));
}

// 16-bit values (FP16, else BF16) and FP32, one and eight at once.
template <bool F16>
__device__ __forceinline__ float widen(uint32_t v) {
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
    else return bf16_bits_to_f32(v & 0xffffu);
}
template <bool F16>
__device__ __forceinline__ void widen8(const u32x4 &r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = widen<F16>(r[i]);
        f[2 * i + 1] = widen<F16>(r[i] >> 16);
    }
}
template <bool F16>
__device__ __forceinline__ u32x4 narrow8(const float (&f)[8]) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = to16x2<F16>(f[2 * i], f[2 * i + 1]);
    return o;
}

// Activations of the products' epilogues (FP32; the reciprocal and exp2
// instructions are within one unit in the last place).
__device__ __forceinline__ float silu(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}
// tanh form: 0.5 z (1 + tanh(u)) = z / (1 + e^-2u), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu(float z) {
    const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u2 * -1.44269504088896340736f));
}
__device__ __forceinline__ float act1(float z, int act) {
    return act == kActSilu ? silu(z) : act == kActGelu ? gelu(z) : z;
}

// Order of the output tiles of a product: panels of PANEL row tiles, column
// tiles outer and the panel's row tiles inner, so that the tiles that run at
// the same time on an XCD (neighbours in this order) share both operands in
// its L2.  Item i of rows x cols -> its row and column tile.
template <int PANEL>
__device__ __forceinline__ void panel_tile(int i, int rows, int cols, int &row, int &col) {
    const int panel = i / (PANEL * cols);
    const int first = panel * PANEL;
    const int height = rows - first < PANEL ? rows - first : PANEL;
    const int rem = i - first * cols;
    col = rem / height;
    row = first + rem - col * height;
}

}  // namespace moe
