// packed.cuh -- arithmetic on pairs: two fp32 values in one register pair (an instruction of half
// the issue slots of two), and 16-bit pairs taken into fp32 sums as they are.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "encoder.h"

namespace sdtw {

// Two neighbouring 16-bit elements as one word, and a word's two elements. By copies: a compiler takes an element and a word
// for different objects, and may drop the store of one that is read as the other.
template <typename T> __device__ __forceinline__ uint32_t word_of(const T* e) {
    uint32_t w;
    memcpy(&w, e, 4);
    return w;
}
template <typename T> struct Halves {
    T e[2];
    __device__ __forceinline__ explicit Halves(uint32_t w) { memcpy(e, &w, 4); }
};

// two fp32 values rounded to 16 bits each, lo in the low half
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The two values that pack2 made, added to x and y. The instruction takes a 16-bit operand as it
// is: 1.1 cycles a value and warp, where unpacking them for packed fp32 adds took 4 (shifts and
// masks run at half rate).
template <typename T> __device__ __forceinline__ void add_pair(float& x, float& y, uint32_t v);
template <> __device__ __forceinline__ void add_pair<__nv_bfloat16>(float& x, float& y, uint32_t v) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(x), "+f"(y) : "r"(v));
}
template <> __device__ __forceinline__ void add_pair<__half>(float& x, float& y, uint32_t v) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.f16 %0, lo, %0;\n\tadd.rn.f32.f16 %1, hi, %1;\n\t}"
        : "+f"(x), "+f"(y) : "r"(v));
}
// The same, from other values: x = v's low half + a, y = its high half + b.
template <typename T> __device__ __forceinline__ void sum_pair(float& x, float& y, uint32_t v, float a, float b);
template <> __device__ __forceinline__ void sum_pair<__nv_bfloat16>(float& x, float& y, uint32_t v, float a, float b) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %3;\n\tadd.rn.f32.bf16 %1, hi, %4;\n\t}"
        : "=f"(x), "=f"(y) : "r"(v), "f"(a), "f"(b));
}
template <> __device__ __forceinline__ void sum_pair<__half>(float& x, float& y, uint32_t v, float a, float b) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.f16 %0, lo, %3;\n\tadd.rn.f32.f16 %1, hi, %4;\n\t}"
        : "=f"(x), "=f"(y) : "r"(v), "f"(a), "f"(b));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// VEC elements as fp32 pairs; a lone one has a zero beside it.
template <int VEC> constexpr int kPairs = (VEC + 1) / 2;
using Pair = unsigned long long;
template <int VEC> __device__ __forceinline__ void pairs_of(const float (&v)[VEC], Pair (&out)[kPairs<VEC>]) {
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) out[q] = pk2(v[2 * q], VEC == 1 ? 0.f : v[2 * q + 1]);
}
// v + c
template <typename T, int VEC> __device__ __forceinline__ void plus(const Pack<T, VEC>& v, float c, Pair (&out)[kPairs<VEC>]) {
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) {
        if constexpr (VEC == 1) {
            out[q] = pk2(to_f32(v.e[0]) + c, 0.f);
        } else if constexpr (sizeof(T) == 4) {
            out[q] = add2(pk2(v.e[2 * q], v.e[2 * q + 1]), pk2(c, c));
        } else {
            float x, y;
            sum_pair<T>(x, y, word_of(&v.e[2 * q]), c, c);
            out[q] = pk2(x, y);
        }
    }
}
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> rounded(const Pair (&v)[kPairs<VEC>]) {
    Pack<T, VEC> o;
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) {
        float x, y;
        upk2(v[q], x, y);
        if constexpr (VEC == 1) o.e[0] = from_f32<T>(x);
        else if constexpr (sizeof(T) == 4) o.e[2 * q] = x, o.e[2 * q + 1] = y;
        else {
            const Halves<T> h(pack2<T>(x, y));
            o.e[2 * q] = h.e[0], o.e[2 * q + 1] = h.e[1];
        }
    }
    return o;
}
// s + v, the even elements in one half and the odd ones in the other
template <typename T, int VEC> __device__ __forceinline__ Pair sum_onto(Pair s, const Pack<T, VEC>& v) {
    float x, y;
    upk2(s, x, y);
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) {
        if constexpr (VEC == 1) x += to_f32(v.e[0]);
        else if constexpr (sizeof(T) == 4) x += v.e[2 * q], y += v.e[2 * q + 1];
        else add_pair<T>(x, y, word_of(&v.e[2 * q]));
    }
    return pk2(x, y);
}
__device__ __forceinline__ float both(Pair v) {
    float x, y;
    upk2(v, x, y);
    return x + y;
}
// v - m, element by element
template <typename T, int VEC> __device__ __forceinline__ void minus(const Pack<T, VEC>& v, const Pair (&m)[kPairs<VEC>], Pair (&out)[kPairs<VEC>]) {
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) {
        float x, y;
        upk2(m[q], x, y);
        if constexpr (VEC == 1) {
            out[q] = pk2(to_f32(v.e[0]) - x, 0.f);
        } else if constexpr (sizeof(T) == 4) {
            out[q] = sub2(pk2(v.e[2 * q], v.e[2 * q + 1]), m[q]);
        } else {
            float a, b;
            sum_pair<T>(a, b, word_of(&v.e[2 * q]), -x, -y);
            out[q] = pk2(a, b);
        }
    }
}

}  // namespace sdtw
