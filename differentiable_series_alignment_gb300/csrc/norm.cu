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
//
// Memory bounds it, and next to it the instructions of 16-bit rows: elements are taken into fp32 by
// mixed-precision adds and worked on in pairs, which halved the instructions of both directions
// (the backward issued 69 % of the time before), and coming rows are on their way to shared memory
// meanwhile. 65535 rows of 1024 with fp32 weights: bf16 forward 51 us (5.2 TB/s), backward 80 us
// (5.1 TB/s) and 6 for the fold, caches flushed before; fp32 forward 108 us (5.0), backward
// 138 (5.9). A plain copy of as many bytes runs at 5.6 TB/s. Without the rows ahead fp32 took 149 and 164.
// Rows of 4096 and 8192 bf16 have two and four packs a thread and fewer CTAs per SM: as many elements take 70 and 64 us
// forward, 117 and 135 backward. A row length that is no multiple of a pack is taken element by element, and so is one of
// more than 1024 packs: 1003 bf16 217 and 500 us, 8200 166 and 668, where the backward sums its columns in memory.
#include <algorithm>

#include "encoder.h"
#include "packed.cuh"

namespace sdtw {
namespace {

constexpr int kThreads = 256;
// Backward CTAs per SM, by packs a thread. With four of one pack (64 registers) the sums of the weights'
// gradients spilled: 65535 rows of 1024 bf16 took 99 us where three take 83.
template <int K> constexpr int kBwdCtas = K == 1 ? 3 : K == 2 ? 2 : 1;

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

// VEC elements as fp32 pairs; a lone one has a zero beside it.
template <int VEC> constexpr int kPairs = (VEC + 1) / 2;
using Pair = unsigned long long;
template <int VEC> __device__ __forceinline__ void pairs_of(const float (&v)[VEC], Pair (&out)[kPairs<VEC>]) {
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) out[q] = pk2(v[2 * q], VEC == 1 ? 0.f : v[2 * q + 1]);
}
template <int VEC> __device__ __forceinline__ void weight_pairs(const void* p, int c0, int wdtype, float none, Pair (&out)[kPairs<VEC>]) {
    float w[VEC];
    weights<VEC>(p, c0, wdtype, none, w);
    pairs_of<VEC>(w, out);
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
            float x = c, y = c;
            add_pair<T>(x, y, *reinterpret_cast<const uint32_t*>(&v.e[2 * q]));
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
        else *reinterpret_cast<uint32_t*>(&o.e[2 * q]) = pack2<T>(x, y);
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
        else add_pair<T>(x, y, *reinterpret_cast<const uint32_t*>(&v.e[2 * q]));
    }
    return pk2(x, y);
}
__device__ __forceinline__ float both(Pair v) {
    float x, y;
    upk2(v, x, y);
    return x + y;
}

// Packs on their way from memory: a thread copies its own packs of coming rounds to shared memory
// and reads back only those, so that nobody waits for anybody. An SM then has some 100 KB in flight
// whatever its threads are busy with, where loads to registers leave it idle from a round's sums
// to its stores.
__device__ __forceinline__ void fetch16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch_mark() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// L threads per row, K packs of VEC elements per thread, R rows at a time (their sums run side by
// side, and weights that are not kept in registers are read once for all); C is a multiple of VEC.
// AHEAD rounds of rows are on their way while one is worked on (0: a round loads its own).
template <typename T, int VEC, int K, int L, int R, int AHEAD>
__global__ void __launch_bounds__(kThreads, 4) norm_fwd_kernel(const NormParams p)
{
    __shared__ float2 red[2 * kThreads / 32];
    extern __shared__ __align__(16) unsigned char ring[];   // [AHEAD + 1][R][K][kThreads] packs
    int turn = 0;
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x % L;
    const long long step = (long long)gridDim.x * (kThreads / L) * R;
    const int packs = p.C / VEC;
    const float inv_c = 1.f / (float)p.C;
    constexpr int Q = kPairs<VEC>;
    Pair w1[Q], b1[Q];   // one pack a thread: its weights stay in registers
    if (K == 1 && lane < packs) {
        weight_pairs<VEC>(p.weight, lane * VEC, p.wdtype, 1.f, w1);
        weight_pairs<VEC>(p.bias, lane * VEC, p.wdtype, 0.f, b1);
    }
    // A warp with a whole row has them in shared memory, in pieces of 16 bytes that neighbouring lanes
    // find side by side. Read from the cache for every row, at strides of 32 bytes, they kept it
    // busier than x and y did (65535 rows of 1024 bf16: 65 us, L1 at 86 %; 53 us so).
    constexpr bool HELD = K > 1 && L == 32 && VEC > 1;
    constexpr int FOURS = HELD ? VEC / 4 : 1;
    __shared__ float4 held[2 * FOURS][HELD ? K * L : 1];
    if constexpr (HELD) {
        for (int c = threadIdx.x; c < packs; c += kThreads)
#pragma unroll
            for (int h = 0; h < FOURS; ++h) {
                float w[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = wval(p.weight, c * VEC + 4 * h + e, p.wdtype, 1.f);
                    b[e] = wval(p.bias, c * VEC + 4 * h + e, p.wdtype, 0.f);
                }
                held[h][c] = make_float4(w[0], w[1], w[2], w[3]);
                held[FOURS + h][c] = make_float4(b[0], b[1], b[2], b[3]);
            }
        __syncthreads();
    }
    auto row_weights = [&](int k, Pair (&w)[Q], Pair (&b)[Q]) {
        if constexpr (K == 1) {
#pragma unroll
            for (int q = 0; q < Q; ++q) w[q] = w1[q], b[q] = b1[q];
        } else if constexpr (HELD) {
#pragma unroll
            for (int h = 0; h < FOURS; ++h) {
                const float4 x = held[h][lane + k * L], y = held[FOURS + h][lane + k * L];
                w[2 * h] = pk2(x.x, x.y), w[2 * h + 1] = pk2(x.z, x.w);
                b[2 * h] = pk2(y.x, y.y), b[2 * h + 1] = pk2(y.z, y.w);
            }
        } else {
            weight_pairs<VEC>(p.weight, (lane + k * L) * VEC, p.wdtype, 1.f, w);
            weight_pairs<VEC>(p.bias, (lane + k * L) * VEC, p.wdtype, 0.f, b);
        }
    };
    // every thread of a warp (of the CTA, for long rows) makes the same number of rounds: the sums
    // are collective
    auto row = [&](long long r) { return reinterpret_cast<const P*>(static_cast<const T*>(p.x) + (r < p.rows ? r : 0) * p.C); };
    auto slot = [&](int stage, int i, int k) { return reinterpret_cast<P*>(ring) + ((stage * R + i) * K + k) * kThreads + threadIdx.x; };
    auto send = [&](long long r, int stage) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (r + i < p.rows && lane + k * L < packs) fetch16(slot(stage, i, k), row(r + i) + lane + k * L);
        fetch_mark();
    };
    const long long own = (long long)blockIdx.x * (kThreads / L) * R + threadIdx.x / L * R;
    int stage = 0;
    if constexpr (AHEAD > 0)
        for (int s = 0; s < AHEAD; ++s) send(own + s * step, s);
    for (long long r0 = (long long)blockIdx.x * (kThreads / L) * R; r0 < p.rows; r0 += step) {
        const long long r = r0 + threadIdx.x / L * R;
        P v[R][K];
        if constexpr (AHEAD > 0) {
            send(r + AHEAD * step, stage == 0 ? AHEAD : stage - 1);   // where the last round's were: they are in use no more
            fetch_wait<AHEAD>();
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs) v[i][k] = AHEAD > 0 ? *slot(stage, i, k) : row(r + i)[lane + k * L];
        stage = stage == AHEAD ? 0 : stage + 1;
        float mu[R], rs[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            Pair s = pk2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs) s = sum_onto(s, v[i][k]);
            mu[i] = both(s);
        }
        all_sums<L, R>(mu, red, turn);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            mu[i] *= inv_c;
            Pair s = pk2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs) {
                    Pair d[Q];
                    plus<T, VEC>(v[i][k], -mu[i], d);
#pragma unroll
                    for (int q = 0; q < Q; ++q) s = fma2(d[q], d[q], s);
                }
            rs[i] = both(s);
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
                Pair w[Q], b[Q];
                row_weights(k, w, b);
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (r + i < p.rows) {
                        Pair d[Q];
                        plus<T, VEC>(v[i][k], -mu[i], d);
#pragma unroll
                        for (int q = 0; q < Q; ++q) d[q] = fma2(mul2(d[q], pk2(rs[i], rs[i])), w[q], b[q]);
                        reinterpret_cast<P*>(static_cast<T*>(p.y) + (r + i) * p.C)[lane + k * L] = rounded<T, VEC>(d);
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

template <typename T, int VEC, int K, int L, int AHEAD>
__global__ void __launch_bounds__(kThreads, kBwdCtas<K>) norm_bwd_kernel(const NormParams p)
{
    __shared__ float2 red[2 * kThreads / 32];
    int turn = 0;
    extern __shared__ __align__(16) unsigned char ring[];   // [AHEAD + 1][K][x, dy][kThreads] packs
    float* fold = reinterpret_cast<float*>(ring);           // at the end, L < kThreads: [kThreads / L][C] sums of one gradient at a time
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    const long long step = (long long)gridDim.x * (kThreads / L);
    const int packs = p.C / VEC;
    const float inv_c = 1.f / (float)p.C;
    constexpr int Q = kPairs<VEC>;
    Pair dw[K][Q], db[K][Q];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int q = 0; q < Q; ++q) dw[k][q] = db[k][q] = pk2(0.f, 0.f);
    auto row = [&](const void* base, long long r) { return reinterpret_cast<const P*>(static_cast<const T*>(base) + (r < p.rows ? r : 0) * p.C); };
    auto slot = [&](int stage, int k, int which) { return reinterpret_cast<P*>(ring) + ((stage * K + k) * 2 + which) * kThreads + threadIdx.x; };
    auto send = [&](long long r, int stage) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (r < p.rows && lane + k * L < packs) {
                fetch16(slot(stage, k, 0), row(p.x, r) + lane + k * L);
                fetch16(slot(stage, k, 1), row(p.dy, r) + lane + k * L);
            }
        fetch_mark();
    };
    Pair w1[Q];   // one pack a thread: its weights stay in registers
    if (K == 1 && lane < packs) weight_pairs<VEC>(p.weight, lane * VEC, p.wdtype, 1.f, w1);
    const long long own = (long long)blockIdx.x * (kThreads / L) + group;
    int stage = 0;
    if constexpr (AHEAD > 0)
        for (int s = 0; s < AHEAD; ++s) send(own + s * step, s);
    float mu_next = p.mean[own < p.rows ? own : 0], rs_next = p.rstd[own < p.rows ? own : 0];
    for (long long r0 = (long long)blockIdx.x * (kThreads / L); r0 < p.rows; r0 += step) {
        const long long r = r0 + group;
        const bool live = r < p.rows;
        P xv[K], gv[K];
        const float mu = mu_next, rs = rs_next;
        const long long next = r + step < p.rows ? r + step : 0;
        mu_next = p.mean[next], rs_next = p.rstd[next];
        if constexpr (AHEAD > 0) {
            send(r + AHEAD * step, stage == 0 ? AHEAD : stage - 1);   // where the last round's were: they are in use no more
            fetch_wait<AHEAD>();
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * L < packs) {
                xv[k] = AHEAD > 0 ? *slot(stage, k, 0) : row(p.x, r)[lane + k * L];
                gv[k] = AHEAD > 0 ? *slot(stage, k, 1) : row(p.dy, r)[lane + k * L];
            }
        stage = stage == AHEAD ? 0 : stage + 1;
        Pair xh[K][Q], g[K][Q], s1 = pk2(0.f, 0.f), s2 = pk2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (live && lane + k * L < packs) {
                Pair w[Q];
                if (K > 1) weight_pairs<VEC>(p.weight, (lane + k * L) * VEC, p.wdtype, 1.f, w);
                plus<T, VEC>(xv[k], -mu, xh[k]);
                plus<T, VEC>(gv[k], 0.f, g[k]);
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    xh[k][q] = mul2(xh[k][q], pk2(rs, rs));
                    dw[k][q] = fma2(g[k][q], xh[k][q], dw[k][q]);
                    db[k][q] = add2(db[k][q], g[k][q]);
                    g[k][q] = mul2(g[k][q], K == 1 ? w1[q] : w[q]);
                    s1 = add2(s1, g[k][q]);
                    s2 = fma2(g[k][q], xh[k][q], s2);
                }
            }
        const float2 sums = row_sums<L>(both(s1), both(s2), red, turn);
        const float m1 = -sums.x * inv_c, m2 = -sums.y * inv_c;
        if (live && p.dx) {
            P* dst = reinterpret_cast<P*>(static_cast<T*>(p.dx) + r * p.C);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs) {
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        g[k][q] = mul2(fma2(xh[k][q], pk2(m2, m2), add2(g[k][q], pk2(m1, m1))), pk2(rs, rs));
                    dst[lane + k * L] = rounded<T, VEC>(g[k]);
                }
        }
    }
    if (!p.partial) return;
    auto put = [](float* dst, const Pair (&v)[Q]) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float x, y;
            upk2(v[q], x, y);
            dst[2 * q] = x;
            if (VEC > 1) dst[2 * q + 1] = y;
        }
    };
    for (int which = 0; which < 2; ++which) {
        float* out = p.partial + ((long long)which * gridDim.x + blockIdx.x) * p.C;
        if (L == kThreads) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs)
                    put(out + (lane + k * L) * VEC, which ? db[k] : dw[k]);
        } else {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (lane + k * L < packs)
                    put(fold + group * p.C + (lane + k * L) * VEC, which ? db[k] : dw[k]);
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

// dw, db: the CTAs' partial rows added in a fixed order. 32 columns by 32 row lanes, eight
// rows in flight each: two waits for the cache at the most partial rows there are.
__global__ void __launch_bounds__(1024) norm_fold_kernel(const NormParams p, int ctas)
{
    __shared__ float part[32][33];
    after_previous();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    const float* src = p.partial + (long long)blockIdx.y * ctas * p.C;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < p.C)
        for (int t = lane; t < ctas; t += 256) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (t + 32 * q < ctas) s[q] += src[(long long)(t + 32 * q) * p.C + c];
        }
    part[lane][threadIdx.x & 31] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
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
    constexpr int AHEAD = VEC == 1 ? 0 : R * K == 4 ? 1 : 2;
    constexpr size_t smem = AHEAD ? (AHEAD + 1) * R * K * kThreads * 16 : 0;
    const long long need = (p.rows + rows - 1) / rows, most = AHEAD ? 152 * 4 : K == 1 ? 152 * 16 : 1ll << 30;
    if constexpr (AHEAD > 0)
        if (const cudaError_t e = allow_smem<norm_fwd_kernel<T, VEC, K, L, R, AHEAD>>(smem); e != cudaSuccess) return e;
    norm_fwd_kernel<T, VEC, K, L, R, AHEAD><<<(unsigned)(need < most ? need : most), kThreads, smem, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int VEC, int K, int L> cudaError_t run_bwd(const NormParams& p, int& ctas, cudaStream_t s)
{
    ctas = std::min(ctas, 152 * kBwdCtas<K>);
    constexpr int AHEAD = VEC == 1 ? 0 : K == 1 ? 2 : 1;
    constexpr size_t ring = AHEAD ? (AHEAD + 1) * K * 2 * kThreads * 16 : 0;
    const size_t fold = L == kThreads ? 0 : (size_t)(kThreads / L) * p.C * sizeof(float), smem = ring > fold ? ring : fold;
    if constexpr (AHEAD > 0)
        if (const cudaError_t e = allow_smem<norm_bwd_kernel<T, VEC, K, L, AHEAD>>(ring); e != cudaSuccess) return e;
    norm_bwd_kernel<T, VEC, K, L, AHEAD><<<ctas, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

// Threads per row. Forward: up to 32 lanes hold a row in up to 4 packs each, so that its sums
// need no barrier (65535 rows of 1024 bf16: 51 us, 75 with 128 threads a row), where there are rows
// for all the warps. Backward: a pack a thread as far as the CTA goes, since two sums are kept per
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
template <typename T, int VEC> cudaError_t pick_bwd(const NormParams& p, int& ctas, cudaStream_t s)
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

template <typename T> cudaError_t norm_typed(const NormParams& p, bool backward, int& ctas, cudaStream_t s)
{
    constexpr int VEC = 16 / sizeof(T);
    const bool packed = p.C % VEC == 0 && aligned16(p.x) && aligned16(p.weight) && aligned16(p.bias) &&
                        (backward ? aligned16(p.dy) && aligned16(p.dx) : aligned16(p.y));
    if (backward) return packed ? pick_bwd<T, VEC>(p, ctas, s) : pick_bwd<T, 1>(p, ctas, s);
    return packed ? pick_fwd<T, VEC>(p, s) : pick_fwd<T, 1>(p, s);
}

cudaError_t norm_any(const NormParams& p, bool backward, int& ctas, cudaStream_t s)
{
    if (p.dtype == SDTW_F32) return norm_typed<float>(p, backward, ctas, s);
    if (p.dtype == SDTW_BF16) return norm_typed<__nv_bfloat16>(p, backward, ctas, s);
    return norm_typed<__half>(p, backward, ctas, s);
}

}  // namespace

// At most as many CTAs as are resident, and their partial rows; fewer where there are few rows, which
// are then not worth another partial row.
int norm_partial_ctas(long long rows, int sms)
{
    const long long most = (long long)kBwdCtas<1> * sms, need = (rows + 7) / 8;
    return (int)(need < most ? (need < 1 ? 1 : need) : most);
}

cudaError_t launch_norm_forward(const NormParams& p, cudaStream_t s) {
    int none = 0;
    return norm_any(p, false, none, s);
}

cudaError_t launch_norm_backward(const NormParams& p, int ctas, cudaStream_t s)
{
    cudaError_t e = norm_any(p, true, ctas, s);
    if (e != cudaSuccess || !p.partial) return e;
    return launch_behind(norm_fold_kernel, dim3((p.C + 31) / 32, 2), 1024, s, p, ctas);
}

}  // namespace sdtw
