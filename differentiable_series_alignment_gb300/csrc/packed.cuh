// packed.cuh -- arithmetic on pairs: two fp32 values in one register pair (an instruction of half
// the issue slots of two), and 16-bit pairs taken into fp32 sums as they are.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"

namespace sdtw {

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

}  // namespace sdtw
