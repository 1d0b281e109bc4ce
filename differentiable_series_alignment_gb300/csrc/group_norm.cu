// group_norm.cu -- group norm with an activation, channels last, forward and backward.
//
//   over a batch element's n = n_b cg values of a group: mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps),
//   xh = (x - mu) r, z = xh w + b, y = act(z)
//   dz = dy act'(z), g = dz w, dx = r (g - mean g - xh mean(g xh)), dw = sum dz xh, db = sum dz
//
// A CTA a group of a batch element. The weights' gradients are summed over the positions by the CTA, over the batch by a
// second launch in a fixed order.
#include <type_traits>

#include "activation.cuh"
#include "block.h"

namespace sdtw {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) v += red[w];
    return v;
}
__device__ __forceinline__ float wval(const void* p, int c, int wdtype, float none) {
    if (p == nullptr) return none;
    if (wdtype == SDTW_F32) return static_cast<const float*>(p)[c];
    if (wdtype == SDTW_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[c]);
    return to_f32(static_cast<const __half*>(p)[c]);
}
__device__ __forceinline__ void wstore(void* p, int c, int wdtype, float v) {
    if (wdtype == SDTW_F32) static_cast<float*>(p)[c] = v;
    else if (wdtype == SDTW_BF16) static_cast<__nv_bfloat16*>(p)[c] = from_f32<__nv_bfloat16>(v);
    else static_cast<__half*>(p)[c] = from_f32<__half>(v);
}

template <typename T, int ACT> __global__ void __launch_bounds__(kThreads) group_fwd_kernel(const GroupNormParams p)
{
    __shared__ float red[kThreads / 32];
    const int b = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
    const long long base = (long long)b * p.S * p.C + g * p.cg;
    const T* x = static_cast<const T*>(p.x) + base;
    T* y = static_cast<T*>(p.y) + base;
    const long long n = (long long)len * p.cg, all = (long long)p.S * p.cg;
    auto at = [&](long long i) { return i / p.cg * p.C + i % p.cg; };
    float s = 0.f;
    for (long long i = threadIdx.x; i < n; i += kThreads) s += to_f32(x[at(i)]);
    const float mu = n ? block_sum(s, red) / (float)n : 0.f;
    float q = 0.f;
    for (long long i = threadIdx.x; i < n; i += kThreads) {
        const float d = to_f32(x[at(i)]) - mu;
        q = fmaf(d, d, q);
    }
    const float r = n ? 1.f / sqrtf(block_sum(q, red) / (float)n + p.eps) : 0.f;
    for (long long i = threadIdx.x; i < all; i += kThreads) {
        float none, v = 0.f;
        const int c = g * p.cg + (int)(i % p.cg);
        if (i < n)
            v = activate<ACT, sizeof(T) == 4, false>(fmaf((to_f32(x[at(i)]) - mu) * r, wval(p.weight, c, p.wdtype, 1.f),
                                                          wval(p.bias, c, p.wdtype, 0.f)), none);
        y[at(i)] = from_f32<T>(v);
    }
    if (threadIdx.x == 0 && p.mean) p.mean[blockIdx.x] = mu, p.rstd[blockIdx.x] = r;
}

template <typename T, int ACT> __global__ void __launch_bounds__(kThreads) group_bwd_kernel(const GroupNormParams p)
{
    __shared__ float red[kThreads / 32];
    const int b = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
    const long long base = (long long)b * p.S * p.C + g * p.cg;
    const T* x = static_cast<const T*>(p.x) + base;
    const T* dy = static_cast<const T*>(p.dy) + base;
    const float mu = p.mean[blockIdx.x], r = p.rstd[blockIdx.x];
    const float n = (float)len * p.cg;
    float s1 = 0.f, s2 = 0.f;
    auto value = [&](int i, int c, float& xh, float w) {
        float slope;
        xh = (to_f32(x[(long long)i * p.C + c]) - mu) * r;
        activate<ACT, sizeof(T) == 4, true>(fmaf(xh, w, wval(p.bias, g * p.cg + c, p.wdtype, 0.f)), slope);
        return to_f32(dy[(long long)i * p.C + c]) * slope;
    };
    for (int c = 0; c < p.cg; ++c) {
        const float w = wval(p.weight, g * p.cg + c, p.wdtype, 1.f);
        float dw = 0.f, db = 0.f, xh;
        for (int i = threadIdx.x; i < len; i += kThreads) {
            const float dz = value(i, c, xh, w);
            db += dz;
            dw = fmaf(dz, xh, dw);
        }
        dw = block_sum(dw, red);
        db = block_sum(db, red);
        s1 = fmaf(db, w, s1);
        s2 = fmaf(dw, w, s2);
        if (threadIdx.x == 0 && p.partial) {
            p.partial[(long long)b * p.C + g * p.cg + c] = dw;
            p.partial[((long long)p.B + b) * p.C + g * p.cg + c] = db;
        }
    }
    if (!p.dx) return;
    T* dx = static_cast<T*>(p.dx) + base;
    s1 /= n;
    s2 /= n;
    for (int c = 0; c < p.cg; ++c) {
        const float w = wval(p.weight, g * p.cg + c, p.wdtype, 1.f);
        for (int i = threadIdx.x; i < p.S; i += kThreads) {
            float xh, v = 0.f;
            if (i < len) {
                const float dz = value(i, c, xh, w);
                v = r * (dz * w - s1 - xh * s2);
            }
            dx[(long long)i * p.C + c] = from_f32<T>(v);
        }
    }
}

__global__ void group_fold_kernel(const GroupNormParams p)
{
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    void* dst = blockIdx.y ? p.dbias : p.dweight;
    if (c >= p.C || !dst) return;
    float s = 0.f;
    for (int b = 0; b < p.B; ++b) s += p.partial[((long long)blockIdx.y * p.B + b) * p.C + c];
    wstore(dst, c, p.wdtype, s);
}

template <typename F> cudaError_t with_type(int dtype, F f) {
    if (dtype == SDTW_F32) return f(float());
    if (dtype == SDTW_BF16) return f(__nv_bfloat16());
    return f(__half());
}

}  // namespace

size_t group_norm_workspace(const GroupNormParams& p, bool backward, int) { return backward ? sizeof(float) * 2 * p.B * p.C : 0; }

cudaError_t launch_group_norm_forward(const GroupNormParams& p, int, cudaStream_t s)
{
    return with_type(p.dtype, [&](auto t) {
        return with_activation(p.activation, [&](auto act) {
            group_fwd_kernel<decltype(t), act()><<<p.B * p.G, kThreads, 0, s>>>(p);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_group_norm_backward(const GroupNormParams& p, int, cudaStream_t s)
{
    const cudaError_t e = with_type(p.dtype, [&](auto t) {
        return with_activation(p.activation, [&](auto act) {
            group_bwd_kernel<decltype(t), act()><<<p.B * p.G, kThreads, 0, s>>>(p);
            return cudaGetLastError();
        });
    });
    if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
    group_fold_kernel<<<dim3((p.C + 127) / 128, 2), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sdtw
