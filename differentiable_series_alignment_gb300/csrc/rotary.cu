// rotary.cu -- rotation of feature pairs by the angles of their positions.
//
//   a' = a cos - b sin,  b' = b cos + a sin   (inverse: sin -> -sin, the gradient)
//
// for the pairs (a, b) of a head's first R features: neighbours (interleaved) or the
// two halves; features from R on are copied. Cosines and sines come from a table that
// the program makes once, rounded once from 64 bits: an angle formed in fp32 would be
// off by position * 2^-24 radians. One read and one write of q and k bound it; both
// tensors are turned by one launch, and a thread turns the same features of several
// heads with the cosines it holds in registers.
#include "encoder.h"

namespace sdtw {
namespace {

constexpr int kRotThreads = 256;

// A unit is 16 bytes of one feature row (VEC features): for halves it is VEC pairs, that
// is VEC features of each half; the units after them copy the features from R on.
template <typename T, int VEC, int HEADS>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p)
{
    using P = Pack<T, VEC>;
    const int half = p.R / 2;
    const int turns = p.interleaved ? p.R / VEC : half / VEC;
    const int units = turns + (p.D - p.R) / VEC;
    const int heads = p.H[0] + (p.in[1] ? p.H[1] : 0);
    const long long items = (long long)p.B * p.N * units;
    for (long long it = (long long)blockIdx.x * kRotThreads + threadIdx.x; it < items;
         it += (long long)gridDim.x * kRotThreads)
      for (int g = blockIdx.y; g * HEADS < heads; g += gridDim.y) {
        // 32-bit division wherever the sizes allow it: two of 64 bits cost more than the turns
        long long token;
        int u;
        if (items <= 0x7fffffff) {
            token = (unsigned)it / (unsigned)units;
            u = (int)((unsigned)it - (unsigned)token * (unsigned)units);
        } else {
            token = it / units;
            u = (int)(it - token * units);
        }
        const int b = token <= 0x7fffffff ? (int)((unsigned)token / (unsigned)p.N) : (int)(token / p.N);
        const int n = (int)(token - (long long)b * p.N);
        const bool turn = u < turns;
        const int c0 = turn ? u * VEC : p.R + (u - turns) * VEC;   // first feature of the unit
        const bool two = turn && !p.interleaved;                    // its partners are half further on
        const T* src[HEADS];
        T* dst[HEADS];
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const int head = g * HEADS + h;
            const int w = head >= p.H[0];
            const int hh = head - (w ? p.H[0] : 0);
            const bool live = head < heads;
            src[h] = live ? static_cast<const T*>(p.in[w]) + (b * p.stride[w][0] + n * p.stride[w][1] + hh * p.stride[w][2]) + c0
                          : nullptr;
            dst[h] = live ? static_cast<T*>(p.out[w]) + (((long long)b * p.N + n) * p.H[w] + hh) * p.D + c0 : nullptr;
        }
        P va[HEADS], vb[HEADS];
#pragma unroll
        for (int h = 0; h < HEADS; ++h)
            if (src[h]) {
                va[h] = *reinterpret_cast<const P*>(src[h]);
                if (two) vb[h] = *reinterpret_cast<const P*>(src[h] + half);
            }
        if (turn) {
            const int pos = p.positions ? p.positions[b * p.pos_stride_b + n] : n;
            // a position outside the table has no angle: its features become NaN
            const bool known = pos >= 0 && pos < p.length;
            const float2* row = reinterpret_cast<const float2*>(p.table) + (long long)(known ? pos : 0) * half;
            const float nan = __int_as_float(0x7fffffff);
            if (p.interleaved) {
                if (VEC >= 2) {
                    constexpr int PAIRS = VEC >= 2 ? VEC / 2 : 1;
                    float2 cs[PAIRS];
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) {
                        cs[e] = row[c0 / 2 + e];
                        if (p.inverse) cs[e].y = -cs[e].y;
                        if (!known) cs[e] = make_float2(nan, nan);
                    }
#pragma unroll
                    for (int h = 0; h < HEADS; ++h)
                        if (src[h]) {
#pragma unroll
                            for (int e = 0; e < PAIRS; ++e) {
                                const float a = to_f32(va[h].e[(2 * e) % VEC]), c = to_f32(va[h].e[(2 * e + 1) % VEC]);
                                va[h].e[(2 * e) % VEC] = from_f32<T>(a * cs[e].x - c * cs[e].y);
                                va[h].e[(2 * e + 1) % VEC] = from_f32<T>(c * cs[e].x + a * cs[e].y);
                            }
                            *reinterpret_cast<P*>(dst[h]) = va[h];
                        }
                } else {
                    // one feature: its partner is its neighbour
                    float2 cs = row[c0 / 2];
                    if (p.inverse) cs.y = -cs.y;
                    if (!known) cs = make_float2(nan, nan);
                    const int mate = (c0 & 1) ? -1 : 1;
#pragma unroll
                    for (int h = 0; h < HEADS; ++h)
                        if (src[h]) {
                            const float a = to_f32(va[h].e[0]), c = to_f32(src[h][mate]);
                            dst[h][0] = from_f32<T>(a * cs.x - (float)mate * c * cs.y);
                        }
                }
            } else {
                float2 cs[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    cs[e] = row[c0 + e];
                    if (p.inverse) cs[e].y = -cs[e].y;
                    if (!known) cs[e] = make_float2(nan, nan);
                }
#pragma unroll
                for (int h = 0; h < HEADS; ++h)
                    if (src[h]) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float a = to_f32(va[h].e[e]), c = to_f32(vb[h].e[e]);
                            va[h].e[e] = from_f32<T>(a * cs[e].x - c * cs[e].y);
                            vb[h].e[e] = from_f32<T>(c * cs[e].x + a * cs[e].y);
                        }
                        *reinterpret_cast<P*>(dst[h]) = va[h];
                        *reinterpret_cast<P*>(dst[h] + half) = vb[h];
                    }
            }
        } else {
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (src[h]) *reinterpret_cast<P*>(dst[h]) = va[h];
        }
    }
}

template <typename T, int VEC> cudaError_t run_rotary(const RotaryParams& p, cudaStream_t s)
{
    const int heads = p.H[0] + (p.in[1] ? p.H[1] : 0);
    const int units = (p.interleaved ? p.R : p.R / 2) / VEC + (p.D - p.R) / VEC;
    const long long one = (long long)p.B * p.N * units;
    // four heads a thread reuse its cosines; one a thread where that would leave SMs idle
    const bool many = one * ((heads + 3) / 4) >= 152ll * 4 * kRotThreads;
    long long x = (one + kRotThreads - 1) / kRotThreads;
    if (x > 1 << 24) x = 1 << 24;
    const int groups = many ? (heads + 3) / 4 : heads;
    const dim3 grid((unsigned)x, (unsigned)(groups < 65535 ? groups : 65535));
    if (many) rotary_kernel<T, VEC, 4><<<grid, kRotThreads, 0, s>>>(p);
    else rotary_kernel<T, VEC, 1><<<grid, kRotThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t rotary_typed(const RotaryParams& p, cudaStream_t s)
{
    constexpr int VEC = 16 / sizeof(T);
    bool packed = p.D % VEC == 0 && (p.interleaved ? p.R : p.R / 2) % VEC == 0 && (p.D - p.R) % VEC == 0 &&
                  (reinterpret_cast<uintptr_t>(p.table) & 7) == 0;
    for (int w = 0; w < 2; ++w)
        if (p.in[w]) {
            packed = packed && aligned16(p.in[w]) && aligned16(p.out[w]);
            for (int k = 0; k < 3; ++k) packed = packed && p.stride[w][k] % VEC == 0;
        }
    return packed ? run_rotary<T, VEC>(p, s) : run_rotary<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t s)
{
    if (p.dtype == SDTW_F32) return rotary_typed<float>(p, s);
    if (p.dtype == SDTW_BF16) return rotary_typed<__nv_bfloat16>(p, s);
    return rotary_typed<__half>(p, s);
}

}  // namespace sdtw
