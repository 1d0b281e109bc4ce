// norm.cu -- layer norm over the last dimension, forward and backward.
//
//   mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps), xh = (x - mu) r, y = xh w + b
//   g = dy w, dx = r (g - mean g - xh mean(g xh)), dw = sum_rows dy xh, db = sum_rows dy
//
// A row is read once: L lanes of a warp (short rows) or a whole CTA (long rows) keep it
// in registers, so that the variance is the mean square of centred values (no
// cancellation of E[x^2] - mu^2) at no further traffic. Rows too long for that are read
// again from the cache. The weights' gradients are summed in registers over the rows
// that a CTA takes (a column stays with its thread), then over the CTAs by a second
// launch in a fixed order: no atomics, the same bits every time.
#include "encoder.h"

namespace sdtw {
namespace {

constexpr int kThreads = 256;

template <int W> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, W);
    return v;
}

// Sums over the row's threads: L lanes of a warp, or whole warps (L >= 64), which meet at a
// barrier of their own. red: a float2 per warp of the CTA, two sets that take turns, so that one
// barrier does: who writes a set again has met everyone who read it last.
template <int L> __device__ __forceinline__ float2 row_sums(float x, float y, float2* red, int& turn) {
    constexpr int W = L < 32 ? L : 32;
    x = group_sum<W>(x);
    y = group_sum<W>(y);
    if constexpr (L > 32) {
        const int warp = threadIdx.x >> 5, first = warp / (L / 32) * (L / 32);
        red += (turn ^= 1) * (kThreads / 32);
        if ((threadIdx.x & 31) == 0) red[warp] = make_float2(x, y);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / (L / 32)), "n"(L) : "memory");
        x = y = 0.f;
#pragma unroll
        for (int w = 0; w < L / 32; ++w) {
            const float2 v = red[first + w];
            x += v.x;
            y += v.y;
        }
    }
    return make_float2(x, y);
}
template <int L> __device__ __forceinline__ float row_sum(float v, float2* red, int& turn) {
    return row_sums<L>(v, 0.f, red, turn).x;
}

// The sums of one row, or of two at a time.
template <int L, int R> __device__ __forceinline__ void all_sums(float (&v)[R], float2* red, int& turn) {
    const float2 s = row_sums<L>(v[0], R > 1 ? v[R - 1] : 0.f, red, turn);
    v[0] = s.x;
    if (R > 1) v[R - 1] = s.y;
}

__device__ __forceinline__ float wval(const void* p, int c, int wdtype, float none) {
    if (p == nullptr) return none;
    if (wdtype == SDTW_F32) return static_cast<const float*>(p)[c];
    if (wdtype == SDTW_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[c]);
    return to_f32(static_cast<const __half*>(p)[c]);
}
template <typename W, int VEC> __device__ __forceinline__ void wload(const void* p, int c0, float (&out)[VEC]) {
    constexpr int N = VEC * sizeof(W) > 16 ? 16 / sizeof(W) : VEC;   // elements of one load
#pragma unroll
    for (int k = 0; k < VEC; k += N) {
        const Pack<W, N> v = *reinterpret_cast<const Pack<W, N>*>(static_cast<const W*>(p) + c0 + k);
#pragma unroll
        for (int e = 0; e < N; ++e) out[k + e] = to_f32(v.e[e]);
    }
}
// VEC weights from c0; with VEC > 1 the array is 16-byte aligned. Read from the cache for every
// row: held in registers they would take the place of rows in flight.
template <int VEC> __device__ __forceinline__ void weights(const void* p, int c0, int wdtype, float none, float (&out)[VEC]) {
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = none;
    } else if (wdtype == SDTW_F32) {
        wload<float, VEC>(p, c0, out);
    } else if (wdtype == SDTW_BF16) {
        wload<__nv_bfloat16, VEC>(p, c0, out);
    } else {
        wload<__half, VEC>(p, c0, out);
    }
}
__device__ __forceinline__ void wstore(void* p, int c, int wdtype, float v) {
    if (wdtype == SDTW_F32) static_cast<float*>(p)[c] = v;
    else if (wdtype == SDTW_BF16) static_cast<__nv_bfloat16*>(p)[c] = from_f32<__nv_bfloat16>(v);
    else static_cast<__half*>(p)[c] = from_f32<__half>(v);
}

// L threads per row, K packs of VEC elements per thread, R rows at a time (their sums run side by
// side, and weights that are not kept in registers are read once for all); C is a multiple of VEC.
template <typename T, int VEC, int K, int L, int R>
__global__ void __launch_bounds__(kThreads, 4) norm_fwd_kernel(const NormParams p)
{
    __shared__ float2 red[2 * kThreads / 32];
    int turn = 0;
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x % L;
    const long long step = (long long)gridDim.x * (kThreads / L) * R;
    const int packs = p.C / VEC;
    const float inv_c = 1.f / (float)p.C;
    float w1[VEC], b1[VEC];   // one pack a thread: its weights stay in registers
    if (K == 1 && lane < packs) {
        weights<VEC>(p.weight, lane * VEC, p.wdtype, 1.f, w1);
        weights<VEC>(p.bias, lane * VEC, p.wdtype, 0.f, b1);
    }
    // every thread of a warp (of the CTA, for long rows) makes the same number of rounds: the sums
    // are collective
    for (long long r0 = (long long)blockIdx.x * (kThreads / L) * R; r0 < p.rows; r0 += step) {
        const long long r = r0 + threadIdx.x / L * R;
        P v[R][K];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const P* src = reinterpret_cast<const P*>(static_cast<const T*>(p.x) + (r + i < p.rows ? r + i : 0) * p.C);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs) v[i][k] = src[lane + k * L];
        }
        float mu[R], rs[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            mu[i] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) mu[i] += to_f32(v[i][k].e[e]);
        }
        all_sums<L, R>(mu, red, turn);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            mu[i] *= inv_c;
            rs[i] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float d = to_f32(v[i][k].e[e]) - mu[i];
                        rs[i] = fmaf(d, d, rs[i]);
                    }
        }
        all_sums<L, R>(rs, red, turn);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rs[i] = 1.f / sqrtf(rs[i] * inv_c + p.eps);
            if (lane == 0 && p.mean && r + i < p.rows) {
                p.mean[r + i] = mu[i];
                p.rstd[r + i] = rs[i];
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * L < packs) {
                float w[VEC], b[VEC];
                if (K > 1) {
                    weights<VEC>(p.weight, (lane + k * L) * VEC, p.wdtype, 1.f, w);
                    weights<VEC>(p.bias, (lane + k * L) * VEC, p.wdtype, 0.f, b);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) w[e] = w1[e], b[e] = b1[e];
                }
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (r + i < p.rows) {
                        P o;
#pragma unroll
                        for (int e = 0; e < VEC; ++e) o.e[e] = from_f32<T>(fmaf((to_f32(v[i][k].e[e]) - mu[i]) * rs[i], w[e], b[e]));
                        reinterpret_cast<P*>(static_cast<T*>(p.y) + (r + i) * p.C)[lane + k * L] = o;
                    }
            }
    }
}

// Rows of any length, element by element: the row is read again from the cache.
template <typename T> __global__ void __launch_bounds__(kThreads) norm_fwd_long_kernel(const NormParams p)
{
    __shared__ float2 red[2 * kThreads / 32];
    int turn = 0;
    const float inv_c = 1.f / (float)p.C;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* src = static_cast<const T*>(p.x) + r * p.C;
        T* dst = static_cast<T*>(p.y) + r * p.C;
        float s = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) s += to_f32(src[c]);
        const float mu = row_sum<kThreads>(s, red, turn) * inv_c;
        float q = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float d = to_f32(src[c]) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = 1.f / sqrtf(row_sum<kThreads>(q, red, turn) * inv_c + p.eps);
        for (int c = threadIdx.x; c < p.C; c += kThreads)
            dst[c] = from_f32<T>(fmaf((to_f32(src[c]) - mu) * rs, wval(p.weight, c, p.wdtype, 1.f),
                                      wval(p.bias, c, p.wdtype, 0.f)));
        if (threadIdx.x == 0 && p.mean) {
            p.mean[r] = mu;
            p.rstd[r] = rs;
        }
    }
}

template <typename T, int VEC, int K, int L>
__global__ void __launch_bounds__(kThreads, K == 1 ? 4 : K == 2 ? 2 : 1) norm_bwd_kernel(const NormParams p)
{
    __shared__ float2 red[2 * kThreads / 32];
    int turn = 0;
    extern __shared__ float fold[];   // L < kThreads: [kThreads / L][C] sums of one gradient at a time
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    const long long step = (long long)gridDim.x * (kThreads / L);
    const int packs = p.C / VEC;
    const float inv_c = 1.f / (float)p.C;
    float dw[K][VEC], db[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[k][e] = db[k][e] = 0.f;
    auto fetch = [&](long long r, P (&xv)[K], P (&gv)[K], float& mu, float& rs) {
        const long long row = r < p.rows ? r : 0;
        const P* xs = reinterpret_cast<const P*>(static_cast<const T*>(p.x) + row * p.C);
        const P* gs = reinterpret_cast<const P*>(static_cast<const T*>(p.dy) + row * p.C);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * L < packs) {
                xv[k] = xs[lane + k * L];
                gv[k] = gs[lane + k * L];
            }
        mu = p.mean[row];
        rs = p.rstd[row];
    };
    float w1[VEC];   // one pack a thread: its weights stay in registers
    if (K == 1 && lane < packs) weights<VEC>(p.weight, lane * VEC, p.wdtype, 1.f, w1);
    auto row_weights = [&](int k, float (&w)[VEC]) {
        if (K > 1) {
            weights<VEC>(p.weight, (lane + k * L) * VEC, p.wdtype, 1.f, w);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = w1[e];
        }
    };
    for (long long r0 = (long long)blockIdx.x * (kThreads / L); r0 < p.rows; r0 += step) {
        const long long r = r0 + group;
        const bool live = r < p.rows;
        P xv[K], gv[K];
        float mu, rs;
        fetch(r, xv, gv, mu, rs);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * L < packs) {
                float w[VEC];
                row_weights(k, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (to_f32(xv[k].e[e]) - mu) * rs, dy = to_f32(gv[k].e[e]);
                    const float g = dy * w[e];
                    s1 += g;
                    s2 = fmaf(g, xh, s2);
                    if (live) {
                        dw[k][e] = fmaf(dy, xh, dw[k][e]);
                        db[k][e] += dy;
                    }
                }
            }
        const float2 sums = row_sums<L>(s1, s2, red, turn);
        s1 = sums.x * inv_c;
        s2 = sums.y * inv_c;
        if (live && p.dx) {
            P* dst = reinterpret_cast<P*>(static_cast<T*>(p.dx) + r * p.C);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs) {
                    P o;
                    float w[VEC];
                    row_weights(k, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xh = (to_f32(xv[k].e[e]) - mu) * rs;
                        o.e[e] = from_f32<T>(rs * (to_f32(gv[k].e[e]) * w[e] - s1 - xh * s2));
                    }
                    dst[lane + k * L] = o;
                }
        }
    }
    if (!p.partial) return;
    for (int which = 0; which < 2; ++which) {
        float* out = p.partial + ((long long)which * gridDim.x + blockIdx.x) * p.C;
        if (L == kThreads) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) out[(lane + k * L) * VEC + e] = which ? db[k][e] : dw[k][e];
        } else {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        fold[group * p.C + (lane + k * L) * VEC + e] = which ? db[k][e] : dw[k][e];
            __syncthreads();
            for (int c = threadIdx.x; c < p.C; c += kThreads) {
                float s = 0.f;
                for (int g = 0; g < kThreads / L; ++g) s += fold[g * p.C + c];
                out[c] = s;
            }
        }
    }
}

// Rows of any length: dx by rows, reading the row twice; the columns' sums go straight
// to this CTA's partial row, which it alone touches.
template <typename T> __global__ void __launch_bounds__(kThreads) norm_bwd_long_kernel(const NormParams p)
{
    __shared__ float2 red[2 * kThreads / 32];
    int turn = 0;
    const float inv_c = 1.f / (float)p.C;
    float* pw = p.partial ? p.partial + (long long)blockIdx.x * p.C : nullptr;
    float* pb = p.partial ? p.partial + ((long long)gridDim.x + blockIdx.x) * p.C : nullptr;
    if (pw)
        for (int c = threadIdx.x; c < p.C; c += kThreads) pw[c] = pb[c] = 0.f;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* xs = static_cast<const T*>(p.x) + r * p.C;
        const T* gs = static_cast<const T*>(p.dy) + r * p.C;
        const float mu = p.mean[r], rs = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float xh = (to_f32(xs[c]) - mu) * rs, dy = to_f32(gs[c]);
            const float g = dy * wval(p.weight, c, p.wdtype, 1.f);
            s1 += g;
            s2 = fmaf(g, xh, s2);
            if (pw) {
                pw[c] = fmaf(dy, xh, pw[c]);
                pb[c] += dy;
            }
        }
        const float2 sums = row_sums<kThreads>(s1, s2, red, turn);
        s1 = sums.x * inv_c;
        s2 = sums.y * inv_c;
        if (p.dx) {
            T* dst = static_cast<T*>(p.dx) + r * p.C;
            for (int c = threadIdx.x; c < p.C; c += kThreads) {
                const float xh = (to_f32(xs[c]) - mu) * rs;
                const float g = to_f32(gs[c]) * wval(p.weight, c, p.wdtype, 1.f);
                dst[c] = from_f32<T>(rs * (g - s1 - xh * s2));
            }
        }
    }
}

// dw, db: the CTAs' partial rows added in a fixed order. 32 columns by 32 row lanes, four
// rows in flight each.
__global__ void __launch_bounds__(1024) norm_fold_kernel(const NormParams p, int ctas)
{
    __shared__ float part[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    const float* src = p.partial + (long long)blockIdx.y * ctas * p.C;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < p.C)
        for (int t = lane; t < ctas; t += 128) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (t + 32 * q < ctas) s[q] += src[(long long)(t + 32 * q) * p.C + c];
        }
    part[lane][threadIdx.x & 31] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    // transposed: a warp adds one column's 32 lanes
    const float v = group_sum<32>(part[threadIdx.x & 31][lane]);
    const int col = blockIdx.x * 32 + lane;
    void* dst = blockIdx.y ? p.dbias : p.dweight;
    if ((threadIdx.x & 31) == 0 && col < p.C && dst) wstore(dst, col, p.wdtype, v);
}

template <typename T, int VEC, int K, int L, int R = 1> cudaError_t run_fwd(const NormParams& p, cudaStream_t s)
{
    constexpr int rows = kThreads / L * R;
    const long long need = (p.rows + rows - 1) / rows, most = K == 1 ? 152 * 16 : 1ll << 30;
    norm_fwd_kernel<T, VEC, K, L, R><<<(unsigned)(need < most ? need : most), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int VEC, int K, int L> cudaError_t run_bwd(const NormParams& p, int ctas, cudaStream_t s)
{
    const size_t smem = L == kThreads ? 0 : (size_t)(kThreads / L) * p.C * sizeof(float);
    norm_bwd_kernel<T, VEC, K, L><<<ctas, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

// Threads per row. Forward: up to 32 lanes hold a row in up to 4 packs each, so that its sums
// need no barrier. Backward: a pack a thread as far as the CTA goes, since two sums are kept per
// element besides the two rows: 65535 rows of 1024 bf16 took 132 us with 4 packs a lane (224
// registers, one CTA per SM).
template <typename T, int VEC> cudaError_t pick_fwd(const NormParams& p, cudaStream_t s)
{
    const int packs = p.C / VEC;
    if (packs <= 4) return run_fwd<T, VEC, 1, 4>(p, s);
    if (packs <= 8) return run_fwd<T, VEC, 1, 8>(p, s);
    if (packs <= 16) return run_fwd<T, VEC, 1, 16>(p, s);
    if (packs <= 32) return run_fwd<T, VEC, 1, 32>(p, s);
    if (packs <= 64) return p.rows >= 152 * 64 ? run_fwd<T, VEC, 1, 64, 2>(p, s) : run_fwd<T, VEC, 1, 64>(p, s);
    if (packs <= 128) return p.rows >= 152 * 64 ? run_fwd<T, VEC, 4, 32>(p, s) : run_fwd<T, VEC, 1, 128>(p, s);
    if (packs <= kThreads) return run_fwd<T, VEC, 1, kThreads>(p, s);
    if (packs <= 2 * kThreads) return run_fwd<T, VEC, 2, kThreads>(p, s);
    if (packs <= 4 * kThreads) return run_fwd<T, VEC, 4, kThreads>(p, s);
    norm_fwd_long_kernel<T><<<(unsigned)(p.rows < (1 << 30) ? p.rows : 1 << 30), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int VEC> cudaError_t pick_bwd(const NormParams& p, int ctas, cudaStream_t s)
{
    const int packs = p.C / VEC;
    if (packs <= 4) return run_bwd<T, VEC, 1, 4>(p, ctas, s);
    if (packs <= 8) return run_bwd<T, VEC, 1, 8>(p, ctas, s);
    if (packs <= 16) return run_bwd<T, VEC, 1, 16>(p, ctas, s);
    if (packs <= 32) return run_bwd<T, VEC, 1, 32>(p, ctas, s);
    if (packs <= 64) return run_bwd<T, VEC, 1, 64>(p, ctas, s);
    if (packs <= 128) return run_bwd<T, VEC, 1, 128>(p, ctas, s);
    if (packs <= kThreads) return run_bwd<T, VEC, 1, kThreads>(p, ctas, s);
    if (packs <= 2 * kThreads) return run_bwd<T, VEC, 2, kThreads>(p, ctas, s);
    if (packs <= 4 * kThreads) return run_bwd<T, VEC, 4, kThreads>(p, ctas, s);
    norm_bwd_long_kernel<T><<<ctas, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t norm_typed(const NormParams& p, bool backward, int ctas, cudaStream_t s)
{
    constexpr int VEC = 16 / sizeof(T);
    const bool packed = p.C % VEC == 0 && aligned16(p.x) && aligned16(p.weight) && aligned16(p.bias) &&
                        (backward ? aligned16(p.dy) && aligned16(p.dx) : aligned16(p.y));
    if (backward) return packed ? pick_bwd<T, VEC>(p, ctas, s) : pick_bwd<T, 1>(p, ctas, s);
    return packed ? pick_fwd<T, VEC>(p, s) : pick_fwd<T, 1>(p, s);
}

cudaError_t norm_any(const NormParams& p, bool backward, int ctas, cudaStream_t s)
{
    if (p.dtype == SDTW_F32) return norm_typed<float>(p, backward, ctas, s);
    if (p.dtype == SDTW_BF16) return norm_typed<__nv_bfloat16>(p, backward, ctas, s);
    return norm_typed<__half>(p, backward, ctas, s);
}

}  // namespace

// Four CTAs per SM (as many as are resident where a thread has one pack); fewer where there
// are few rows, which are then not worth another partial row.
int norm_partial_ctas(long long rows, int C, int sms)
{
    (void)C;
    const long long most = 4ll * sms, need = (rows + 7) / 8;
    return (int)(need < most ? (need < 1 ? 1 : need) : most);
}

cudaError_t launch_norm_forward(const NormParams& p, cudaStream_t s) { return norm_any(p, false, 0, s); }

cudaError_t launch_norm_backward(const NormParams& p, int ctas, cudaStream_t s)
{
    cudaError_t e = norm_any(p, true, ctas, s);
    if (e != cudaSuccess || !p.partial) return e;
    norm_fold_kernel<<<dim3((p.C + 31) / 32, 2), 1024, 0, s>>>(p, ctas);
    return cudaGetLastError();
}

}  // namespace sdtw
