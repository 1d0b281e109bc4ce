// gated.cu -- gated linear units, forward and backward.
//
//   g = x Wg^T + bg, u = x Wu^T + bu, h = act(g) u
//   dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dbg, dbu = column sums
//
// Products of any strides by tiles of 64 x 64 on the FP32 pipe.
#include <type_traits>

#include "activation.cuh"
#include "block.h"

namespace sdtw {
namespace {

constexpr int kTile = 64, kDepth = 16;

template <typename T> struct Matrix {   // element (i, k)
    const T* p;
    long long si, sk, rows;
    __device__ __forceinline__ float at(long long i, long long k, long long depth) const {
        return i < rows && k < depth ? to_f32(p[i * si + k * sk]) : 0.f;
    }
};

// acc += A(i0 .. i0 + 63, :) B(j0 .. j0 + 63, :)^T; a thread of 256 has 4 x 4 of it
template <typename A, typename B>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], const Matrix<A>& a, const Matrix<B>& b, long long i0, long long j0, long long depth)
{
    __shared__ float as[kDepth][kTile + 1], bs[kDepth][kTile + 1];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (long long k0 = 0; k0 < depth; k0 += kDepth) {
        __syncthreads();
        for (int q = threadIdx.x; q < kTile * kDepth; q += 256) {
            as[q % kDepth][q / kDepth] = a.at(i0 + q / kDepth, k0 + q % kDepth, depth);
            bs[q % kDepth][q / kDepth] = b.at(j0 + q / kDepth, k0 + q % kDepth, depth);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(as[k][ty * 4 + r], bs[k][tx * 4 + c], acc[r][c]);
    }
}

// h, or with GRADS the gradients of both products
template <typename T, int ACT, bool GRADS> __global__ void __launch_bounds__(256) gated_kernel(const GatedParams p)
{
    const sdtw_gated& a = p.a;
    const long long i0 = (long long)blockIdx.x * kTile, j0 = (long long)blockIdx.y * kTile;
    const Matrix<T> x{static_cast<const T*>(a.x), a.x_stride, 1, a.R}, wg{static_cast<const T*>(a.gate_weight), a.gate_stride, 1, a.F},
        wu{static_cast<const T*>(a.up_weight), a.up_stride, 1, a.F};
    float g[4][4] = {}, u[4][4] = {};
    tile_product(g, x, wg, i0, j0, a.K);
    tile_product(u, x, wu, i0, j0, a.K);
    for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) {
            const long long i = i0 + threadIdx.x / 16 * 4 + r, j = j0 + threadIdx.x % 16 * 4 + c;
            if (i >= a.R || j >= a.F) continue;
            const float gv = g[r][c] + (a.gate_bias ? to_f32(static_cast<const T*>(a.gate_bias)[j]) : 0.f);
            const float uv = u[r][c] + (a.up_bias ? to_f32(static_cast<const T*>(a.up_bias)[j]) : 0.f);
            float slope;
            const float v = activate<ACT, sizeof(T) == 4, GRADS>(gv, slope);
            if (GRADS) {
                const float d = to_f32(static_cast<const T*>(p.dh)[i * a.F + j]);
                p.grads[i * 2 * a.F + j] = d * uv * slope;
                p.grads[i * 2 * a.F + a.F + j] = d * v;
            } else {
                static_cast<T*>(p.h)[i * a.F + j] = from_f32<T>(v * uv);
            }
        }
}

template <typename T> __global__ void __launch_bounds__(256) gated_dx_kernel(const GatedParams p)
{
    const sdtw_gated& a = p.a;
    const long long i0 = (long long)blockIdx.x * kTile, j0 = (long long)blockIdx.y * kTile;
    const Matrix<float> dg{p.grads, 2ll * a.F, 1, a.R}, du{p.grads + a.F, 2ll * a.F, 1, a.R};
    const Matrix<T> wg{static_cast<const T*>(a.gate_weight), 1, a.gate_stride, a.K}, wu{static_cast<const T*>(a.up_weight), 1, a.up_stride, a.K};
    float acc[4][4] = {};
    tile_product(acc, dg, wg, i0, j0, a.F);
    tile_product(acc, du, wu, i0, j0, a.F);
    for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) {
            const long long i = i0 + threadIdx.x / 16 * 4 + r, j = j0 + threadIdx.x % 16 * 4 + c;
            if (i < a.R && j < a.K) static_cast<T*>(p.dx)[i * a.K + j] = from_f32<T>(acc[r][c]);
        }
}

template <typename T> __global__ void __launch_bounds__(256) gated_dw_kernel(const GatedParams p)
{
    const sdtw_gated& a = p.a;
    void* out = blockIdx.z ? p.dup_weight : p.dgate_weight;
    if (!out) return;
    const long long i0 = (long long)blockIdx.x * kTile, j0 = (long long)blockIdx.y * kTile;
    const Matrix<float> d{p.grads + blockIdx.z * a.F, 1, 2ll * a.F, a.F};
    const Matrix<T> x{static_cast<const T*>(a.x), 1, a.x_stride, a.K};
    float acc[4][4] = {};
    tile_product(acc, d, x, i0, j0, a.R);
    for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) {
            const long long i = i0 + threadIdx.x / 16 * 4 + r, j = j0 + threadIdx.x % 16 * 4 + c;
            if (i < a.F && j < a.K) static_cast<T*>(out)[i * a.K + j] = from_f32<T>(acc[r][c]);
        }
}

template <typename T> __global__ void __launch_bounds__(256) gated_db_kernel(const GatedParams p)
{
    __shared__ float part[8][32];
    const sdtw_gated& a = p.a;
    void* out = blockIdx.y ? p.dup_bias : p.dgate_bias;
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x % 32, lane = threadIdx.x / 32;
    float s = 0.f;
    if (c < a.F)
        for (long long i = lane; i < a.R; i += 8) s += p.grads[i * 2 * a.F + blockIdx.y * a.F + c];
    part[lane][threadIdx.x % 32] = s;
    __syncthreads();
    if (lane == 0 && c < a.F) {
        s = 0.f;
        for (int w = 0; w < 8; ++w) s += part[w][threadIdx.x];
        static_cast<T*>(out)[c] = from_f32<T>(s);
    }
}

template <typename F> cudaError_t with_type(int dtype, F f) {
    if (dtype == SDTW_F32) return f(float());
    if (dtype == SDTW_BF16) return f(__nv_bfloat16());
    return f(__half());
}
unsigned tiles(long long n) { return (unsigned)((n + kTile - 1) / kTile); }

}  // namespace

size_t gated_workspace(const GatedParams& p, bool backward, int) { return backward ? sizeof(float) * 2 * p.a.R * p.a.F : 0; }

cudaError_t launch_gated_forward(const GatedParams& p, void*, int, cudaStream_t s)
{
    return with_type(p.a.dtype, [&](auto t) {
        return with_activation(p.a.activation, [&](auto act) {
            gated_kernel<decltype(t), act(), false><<<dim3(tiles(p.a.R), tiles(p.a.F)), 256, 0, s>>>(p);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_gated_backward(const GatedParams& p0, void* ws, int, cudaStream_t s)
{
    GatedParams p = p0;
    p.grads = static_cast<float*>(ws);
    return with_type(p.a.dtype, [&](auto t) {
        using T = decltype(t);
        with_activation(p.a.activation, [&](auto act) {
            gated_kernel<T, act(), true><<<dim3(tiles(p.a.R), tiles(p.a.F)), 256, 0, s>>>(p);
            return cudaSuccess;
        });
        if (p.dx) gated_dx_kernel<T><<<dim3(tiles(p.a.R), tiles(p.a.K)), 256, 0, s>>>(p);
        if (p.dgate_weight || p.dup_weight) gated_dw_kernel<T><<<dim3(tiles(p.a.F), tiles(p.a.K), 2), 256, 0, s>>>(p);
        if (p.dgate_bias || p.dup_bias) gated_db_kernel<T><<<dim3((p.a.F + 31) / 32, 2), 256, 0, s>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace sdtw
