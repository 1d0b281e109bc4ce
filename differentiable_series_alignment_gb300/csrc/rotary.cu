// rotary.cu -- rotation of feature pairs by the angles of their positions.
//
//   a' = a cos - b sin,  b' = b cos + a sin   (inverse: sin -> -sin, the gradient)
//
// for the pairs (a, b) of a head's first R features: neighbours (interleaved) or the
// two halves; features from R on are copied. Cosines and sines come from a table that
// the program makes once, rounded once from 64 bits: an angle formed in fp32 would be
// off by position * 2^-24 radians. One read and one write of q and k bound it; both
// tensors are turned by one launch, and a thread turns the same features of several
// heads with the cosines it holds in registers. 4 x 4096 samples, 16 + 4 heads of 128, bf16: 34 us a
// direction, 4.9 TB/s of the 5.6 of a plain copy of as many bytes (43 with the caches flushed before, 55 for neighbouring
// pairs). Halves of R / 2 features that are no multiple of a pack go feature by feature: D = 80 with R = 40 72 us,
// with R = 80 33.
#include "encoder.h"

namespace sdtw {
namespace {

constexpr int kRotThreads = 256;

// n pairs' cosines and sines, two pairs a load where they come in pairs
template <int N> __device__ __forceinline__ void turns_of(const float2* row, float2 (&cs)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float4 t = *reinterpret_cast<const float4*>(row + e);
            cs[e] = make_float2(t.x, t.y), cs[e + 1] = make_float2(t.z, t.w);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) cs[e] = row[e];
    }
}

// The turned pair (a, b), the first product of each sum unrounded. Written out, so that packs and single
// elements, whichever the alignment allows, give the same bits.
__device__ __forceinline__ float turned_a(float a, float b, float2 t) { return fmaf(a, t.x, -(b * t.y)); }
__device__ __forceinline__ float turned_b(float a, float b, float2 t) { return fmaf(b, t.x, a * t.y); }

// A unit is 16 bytes of one feature row (VEC features): for halves it is VEC pairs, that
// is VEC features of each half; the units after them copy the features from R on. A thread
// has one unit of one token and goes through heads HEADS at a time, its cosines in registers.
template <typename T, int VEC, int HEADS>
__global__ void __launch_bounds__(kRotThreads, 3) rotary_kernel(const RotaryParams p)
{
    using P = Pack<T, VEC>;
    const int half = p.R / 2;
    const int turns = p.interleaved ? p.R / VEC : half / VEC;
    const int units = turns + (p.D - p.R) / VEC;
    const int heads = p.H[0] + (p.in[1] ? p.H[1] : 0);
    const long long items = (long long)p.B * p.N * units;
    for (long long it = (long long)blockIdx.x * kRotThreads + threadIdx.x; it < items;
         it += (long long)gridDim.x * kRotThreads) {
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
        // cosines and sines of the unit's pairs; a lone feature (VEC 1) has its neighbour's
        float2 cs[VEC];
        int mate = 0;   // VEC 1, interleaved: where the partner is
        if (turn) {
            const int pos = p.positions ? p.positions[b * p.pos_stride_b + n] : n;
            // a position outside the table has no angle: its features become NaN
            const bool known = pos >= 0 && pos < p.length;
            const float2* row = reinterpret_cast<const float2*>(p.table) + (long long)(known ? pos : 0) * half;
            constexpr int PAIRS = VEC >= 2 ? VEC / 2 : 1;
            if (p.interleaved) {
                float2 few[PAIRS];
                turns_of<PAIRS>(row + c0 / 2, few);
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) cs[e] = few[e];
                if (VEC == 1) mate = (c0 & 1) ? -1 : 1;
            } else {
                turns_of<VEC>(row + c0, cs);
            }
            const float nan = __int_as_float(0x7fffffff);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (p.inverse) cs[e].y = -cs[e].y;
                if (!known) cs[e] = make_float2(nan, nan);
            }
        }
        const long long in0 = b * p.stride[0][0] + n * p.stride[0][1] + c0, in1 = b * p.stride[1][0] + n * p.stride[1][1] + c0;
        const long long out0 = token * p.H[0] * p.D + c0, out1 = token * p.H[1] * p.D + c0;
        for (int h0 = blockIdx.y * HEADS; h0 < heads; h0 += gridDim.y * HEADS) {
            const T* src[HEADS];
            T* dst[HEADS];
            P va[HEADS], vb[HEADS];
#pragma unroll
            for (int q = 0; q < HEADS; ++q) {
                const int h = h0 + q, w = h >= p.H[0], hh = w ? h - p.H[0] : h;
                if (h >= heads) continue;
                src[q] = w ? static_cast<const T*>(p.in[1]) + in1 + hh * p.stride[1][2]
                           : static_cast<const T*>(p.in[0]) + in0 + hh * p.stride[0][2];
                dst[q] = w ? static_cast<T*>(p.out[1]) + out1 + (long long)hh * p.D : static_cast<T*>(p.out[0]) + out0 + (long long)hh * p.D;
                va[q] = *reinterpret_cast<const P*>(src[q]);
                if (two) vb[q] = *reinterpret_cast<const P*>(src[q] + half);
                else if (VEC == 1 && turn) vb[q].e[0] = src[q][mate];
            }
#pragma unroll
            for (int q = 0; q < HEADS; ++q) {
                if (h0 + q >= heads) continue;
                if (two) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float x = to_f32(va[q].e[e]), y = to_f32(vb[q].e[e]);
                        va[q].e[e] = from_f32<T>(turned_a(x, y, cs[e]));
                        vb[q].e[e] = from_f32<T>(turned_b(x, y, cs[e]));
                    }
                    *reinterpret_cast<P*>(dst[q] + half) = vb[q];
                } else if (turn && VEC == 1) {
                    const float x = to_f32(va[q].e[0]), y = to_f32(vb[q].e[0]);
                    va[q].e[0] = from_f32<T>(mate > 0 ? turned_a(x, y, cs[0]) : turned_b(y, x, cs[0]));
                } else if (turn) {
#pragma unroll
                    for (int e = 0; e + 1 < VEC; e += 2) {
                        const float x = to_f32(va[q].e[e]), y = to_f32(va[q].e[e + 1]);
                        va[q].e[e] = from_f32<T>(turned_a(x, y, cs[e / 2]));
                        va[q].e[e + 1] = from_f32<T>(turned_b(x, y, cs[e / 2]));
                    }
                }
                *reinterpret_cast<P*>(dst[q]) = va[q];
            }
        }
    }
}

template <typename T, int VEC> cudaError_t run_rotary(const RotaryParams& p, cudaStream_t s)
{
    const int heads = p.H[0] + (p.in[1] ? p.H[1] : 0);
    const int units = (p.interleaved ? p.R : p.R / 2) / VEC + (p.D - p.R) / VEC;
    const long long one = (long long)p.B * p.N * units;
    long long x = (one + kRotThreads - 1) / kRotThreads;
    if (x > 1 << 24) x = 1 << 24;
    // the heads are shared out over as many CTAs as fill the SMs three times over (three are resident):
    // 8 x 4096 samples, 16 heads of 64, fp32 49 us, 51 with two times, where the last ones are fewer;
    // a thread takes two heads at a time, one where there is too little work for that
    const long long full = 152ll * 9;
    const bool pairs = x * ((heads + 1) / 2) >= full;
    const long long steps = pairs ? (heads + 1) / 2 : heads;
    long long y = (full + x - 1) / x;
    y = y > steps ? steps : y;
    y = y > 65535 ? 65535 : y;
    const dim3 grid((unsigned)x, (unsigned)y);
    if (pairs) rotary_kernel<T, VEC, 2><<<grid, kRotThreads, 0, s>>>(p);
    else rotary_kernel<T, VEC, 1><<<grid, kRotThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t rotary_typed(const RotaryParams& p, cudaStream_t s)
{
    constexpr int VEC = 16 / sizeof(T);
    bool packed = p.D % VEC == 0 && (p.interleaved ? p.R : p.R / 2) % VEC == 0 && (p.D - p.R) % VEC == 0 &&
                  aligned16(p.table) && p.R % 4 == 0;
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
