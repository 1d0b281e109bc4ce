// attn.cu -- attention on the FP32 pipe: fp32 tensors, and 16-bit ones whose head size
// or alignment the tensor-core kernels cannot take.
//
//   S = scale q k^T on the visible keys, lse = log sum exp S, P = exp(S - lse), o = P v
//   delta = sum_d do o, dP = do v^T, dS = P (dP - delta)
//   dq = scale dS k, dk = scale dS^T q, dv = P^T do
//
// Forward: one CTA per 64 packed rows (rows of the heads that share a key head, see
// encoder.h; 16 where there are no more, and another kernel below for up to 12) walks the keys in tiles of 64 with the running maximum and sum of the
// softmax; S never leaves the SM. Backward: P is computed again from lse. One kernel
// walks the keys for a tile of rows and gives dq, another walks the rows for a tile of
// keys and gives dk and dv, summed over the heads that share them: no atomics, the same
// bits every time, at the price of computing S and dP twice.
// 256 threads hold 4 x 4 of every 64 x 64 product (rows ty + 16 i, columns tx + 16 j), so
// that a step of four features costs 8 16-byte shared loads for 64 FMAs; row pitches of
// D + 4 floats keep those loads free of bank conflicts.
// 8 x 512 samples, 4 heads of 64, fp32: forward 75 us (29 TFLOP/s), backward 229 (33 TFLOP/s) of the pipe's
// 74. The 16-byte loads of a product's operands return four times what they read (each value goes to 16
// threads), which keeps the load unit busy 82 % of the time, and 256 CTAs fill 304 places unevenly.
// With 8 x 4 products a thread, half the threads and a third fewer loads, the latency of each warp's chain
// took its place: 78 and 221 us.
#include <cfloat>

#include "common.cuh"
#include "encoder.h"

namespace sdtw {
namespace {

constexpr int kT = 64;            // rows and keys per tile
constexpr int kThr = 256;
constexpr int kPitchP = kT + 4;   // pitch of a 64 x 64 tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Rows [0, ROWS) of a tile: row_ptr(i) is the row's first element or null (zeros). packed: rows
// begin at boundaries of four elements and D is a multiple of four. All loads of a thread
// go out before its stores.
template <typename T, int DP, int ROWS = kT, typename F>
__device__ __forceinline__ void load_tile(float* dst, int D, bool packed, F row_ptr)
{
    constexpr int LD = DP + 4, ALL = ROWS * (DP / 4), N = (ALL + kThr - 1) / kThr;
    float4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int e = threadIdx.x + k * kThr, r = e / (DP / 4), c = (e % (DP / 4)) * 4;
        const T* src = e < ALL ? row_ptr(r) : nullptr;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src == nullptr || c >= D) continue;
        if (packed) {
            const Pack<T, 4> x = *reinterpret_cast<const Pack<T, 4>*>(src + c);
            v[k] = make_float4(to_f32(x.e[0]), to_f32(x.e[1]), to_f32(x.e[2]), to_f32(x.e[3]));
        } else {
            v[k].x = to_f32(src[c]);
            if (c + 1 < D) v[k].y = to_f32(src[c + 1]);
            if (c + 2 < D) v[k].z = to_f32(src[c + 2]);
            if (c + 3 < D) v[k].w = to_f32(src[c + 3]);
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int e = threadIdx.x + k * kThr;
        if (e < ALL) *reinterpret_cast<float4*>(dst + e / (DP / 4) * LD + (e % (DP / 4)) * 4) = v[k];
    }
}

// acc[i][j] = sum_d a[ty + 16 i][d] * b[tx + 16 j][d], even and odd d apart in packed pairs
// (one instruction for two products).
template <int DP, int R>
__device__ __forceinline__ void dot_tile(float (&acc)[R][4], const float* a, const float* b, int ty, int tx)
{
    constexpr int LD = DP + 4;
    unsigned long long s[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = pk2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        ulonglong2 x[R], y[4];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(a + (ty + 16 * i) * LD + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(b + (tx + 16 * j) * LD + d);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = fma2(x[i].y, y[j].y, fma2(x[i].x, y[j].x, s[i][j]));
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            upk2(s[i][j], lo, hi);
            acc[i][j] = lo + hi;
        }
}

// out[i][c] += sum_k p[ty + 16 i][k] * v[k][column c of this thread]; columns tx * 4 + 64 cc
// (DP >= 64), tx * 2 (DP = 32).
template <int DP> struct Cols {
    static constexpr int W = DP >= 64 ? 4 : 2;     // consecutive columns
    static constexpr int N = DP >= 64 ? DP / 64 : 1;
    static __device__ __forceinline__ int at(int tx, int cc, int w) { return tx * W + 64 * cc + w; }
};
template <int DP, int R>
__device__ __forceinline__ void mul_tile(unsigned long long (&out)[R][Cols<DP>::N * Cols<DP>::W / 2], const float* p, const float* v,
                                         int ty, int tx)
{
    constexpr int LD = DP + 4, W = Cols<DP>::W, NC = Cols<DP>::N;
#pragma unroll 2
    for (int k = 0; k < kT; k += 4) {
        float4 x[R];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4*>(p + (ty + 16 * i) * kPitchP + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            unsigned long long a[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float e = q == 0 ? x[i].x : q == 1 ? x[i].y : q == 2 ? x[i].z : x[i].w;
                a[i] = pk2(e, e);
            }
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                const float* src = v + (k + q) * LD + Cols<DP>::at(tx, cc, 0);
                unsigned long long y[W / 2];
                if constexpr (W == 4) {
                    const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(src);
                    y[0] = t.x, y[1] = t.y;
                } else {
                    y[0] = *reinterpret_cast<const unsigned long long*>(src);
                }
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int w = 0; w < W / 2; ++w) out[i][cc * (W / 2) + w] = fma2(a[i], y[w], out[i][cc * (W / 2) + w]);
            }
        }
    }
}
// the two halves of a packed accumulator, scaled
template <int NP> __device__ __forceinline__ void unpack(const unsigned long long (&acc)[NP], float mul, float (&out)[2 * NP]) {
#pragma unroll
    for (int c = 0; c < NP; ++c) {
        upk2(acc[c], out[2 * c], out[2 * c + 1]);
        out[2 * c] *= mul;
        out[2 * c + 1] *= mul;
    }
}

// max / sum over the 16 lanes (tx) that share a row
__device__ __forceinline__ float max16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o, 16));
    return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, 16);
    return v;
}

// R rows a thread: tiles of 64 rows, or of 16 where there are no more, which have a quarter of the
// products: 8 rows, B = 16, 4 key heads of 128, 8000 keys 326 us, 537 with tiles of 64.
template <typename T, int DP, int R> __global__ void __launch_bounds__(kThr, DP == 128 && R > 1 ? 1 : 2) attn_fwd_simt(const AttnParams p)
{
    extern __shared__ float sm[];
    if (p.splits > 1) let_next_come();
    constexpr int TR = 16 * R, LD = DP + 4, NC = Cols<DP>::N * Cols<DP>::W;
    float* Q = sm;
    float* K = Q + TR * LD;
    float* V = K + kT * LD;
    float* P = V + kT * LD;
    const sdtw_attention& a = p.a;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int heads = a.B * a.Hkv, bh = blockIdx.x % heads;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    // the last rows see the most keys under a causal mask: they start first
    const int r0 = (((p.rows + TR - 1) / TR) - 1 - (int)(blockIdx.x / heads)) * TR;
    const int last = min(r0 + TR, p.rows) - 1;
    const RowRange rr(a, b);
    const int n_first = r0 / p.G, n_last = min(last / p.G, rr.n_b - 1);
    int lo = 0, hi = 0;
    if (n_first <= n_last) {
        lo = rr.lo(n_first);
        hi = rr.hi(n_last);
    }
    // this CTA's share of the key tiles
    int t_lo = lo / kT, t_hi = hi > lo ? (hi + kT - 1) / kT : t_lo;
    if (p.splits > 1) {
        const int per = (t_hi - t_lo + p.splits - 1) / p.splits;
        t_lo = min(t_lo + per * (int)blockIdx.y, t_hi);
        t_hi = min(t_lo + per, t_hi);
    }
    const T* q = static_cast<const T*>(a.q) + b * a.q_stride[0];
    const T* kk = static_cast<const T*>(a.k) + b * a.k_stride[0] + hk * a.k_stride[2];
    const T* vv = static_cast<const T*>(a.v) + b * a.v_stride[0] + hk * a.v_stride[2];
    load_tile<T, DP, TR>(Q, a.D, p.packed, [&](int i) -> const T* {
        const int r = r0 + i;
        if (r >= p.rows) return nullptr;
        const int n = r / p.G;
        if (n >= rr.n_b) return nullptr;
        return q + n * a.q_stride[1] + (hk * p.G + r % p.G) * a.q_stride[2];
    });
    int klo[R], khi[R];   // visible keys of this thread's rows
    float m[R], l[R];
    unsigned long long o[R][NC / 2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + ty + 16 * i;
        const int n = r / p.G;
        const bool live = r < p.rows && n < rr.n_b;
        klo[i] = live ? rr.lo(n) : 0;
        khi[i] = live ? rr.hi(n) : 0;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) o[i][c] = pk2(0.f, 0.f);
    }
    const float s2 = a.scale * kLog2e;
    for (int t = t_lo; t < t_hi; ++t) {
        const int j0 = t * kT;
        __syncthreads();
        load_tile<T, DP>(K, a.D, p.packed, [&](int j) -> const T* { return j0 + j < rr.m_b ? kk + (j0 + j) * a.k_stride[1] : nullptr; });
        load_tile<T, DP>(V, a.D, p.packed, [&](int j) -> const T* { return j0 + j < rr.m_b ? vv + (j0 + j) * a.v_stride[1] : nullptr; });
        __syncthreads();
        float s[R][4];
        dot_tile<DP, R>(s, Q, K, ty, tx);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + tx + 16 * j;
                s[i][j] = (key >= klo[i] && key < khi[i]) ? s[i][j] * s2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            mx = max16(mx);
            const float base = mx == -INFINITY ? 0.f : mx;   // nothing seen yet: every term is 0
            const float keep = ex2(m[i] - base);
            m[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = ex2(s[i][j] - base);
                sum += e;
                P[(ty + 16 * i) * kPitchP + tx + 16 * j] = e;
            }
            l[i] = l[i] * keep + sum;
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) o[i][c] = fma2(o[i][c], pk2(keep, keep), pk2(0.f, 0.f));
        }
        __syncthreads();
        mul_tile<DP, R>(o, P, V, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + ty + 16 * i;
        const float total = sum16(l[i]);
        if (r >= p.rows) continue;
        const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
        const float lse = total == 0.f ? -INFINITY : (m[i] + log2f(total)) * kLn2;
        float res[NC];
        unpack(o[i], inv, res);
        if (total == 0.f)   // 0 whatever the keys hold that other rows of the tile see
#pragma unroll
            for (int c = 0; c < NC; ++c) res[c] = 0.f;
        const int n = r / p.G, h = hk * p.G + r % p.G;
        if (p.splits > 1) {
            const long long row = (((long long)blockIdx.y * a.B + b) * a.Hkv + hk) * p.rows + r;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = Cols<DP>::at(tx, c / Cols<DP>::W, c % Cols<DP>::W);
                if (d < a.D) p.part_o[row * a.D + d] = res[c];
            }
            if (tx == 0) p.part_lse[row] = lse;
        } else {
            const long long at = (((long long)b * a.N + n) * a.Hq + h) * a.D;
            T* out = static_cast<T*>(p.out) + at;
            T* rest = p.out_rest ? static_cast<T*>(p.out_rest) + at : nullptr;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = Cols<DP>::at(tx, c / Cols<DP>::W, c % Cols<DP>::W);
                if (d < a.D) store_rounded(out + d, rest ? rest + d : nullptr, res[c]);
            }
            if (tx == 0 && p.lse) p.lse[((long long)b * a.Hq + h) * a.N + n] = lse;
        }
    }
}

// R packed rows a CTA over a long key axis (new samples over a cache): K and V go straight into
// registers, once for every R rows, and that bounds it. Eight lanes have a key, DP / 8 of its features each, and a
// running maximum, sum and output of their own for every row, so that nothing is exchanged but the three
// shuffles of a score; 16 packs of 4 features a lane are on their way at a time. The 32 groups of
// eight lanes are joined at the end. Measured against tiles of 16 rows in shared memory, fp32: one row,
// B = 8, 4 heads of 64, 4000 keys 23 us (2.9 TB/s) and 55; 8 rows, B = 16, 4 key heads of 128, 8000 keys 225 us
// and 326; 12 rows, B = 8, 2 key heads of 64, 3000 keys 29 us and 31; 16 rows, 4 key heads of 64, 6000 keys
// 104 us and 82: it takes up to 12 rows.
template <typename T, int DP, int R> __global__ void __launch_bounds__(kThr, R == 1 ? 2 : 1) attn_fwd_few(const AttnParams p)
{
    constexpr int F = DP / 32, U = 8 / F, kGroups = kThr / 8, kWarps = kThr / 32;
    __shared__ __align__(16) float s_o[kWarps][R][DP];
    __shared__ float s_m[kWarps][R], s_l[kWarps][R];
    if (p.splits > 1) let_next_come();
    const sdtw_attention& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7, group = threadIdx.x >> 3;
    const int b = blockIdx.x / a.Hkv, hk = blockIdx.x % a.Hkv;
    const RowRange rr(a, b);
    const int r0 = blockIdx.z * R, n_first = r0 / p.G, n_last = min((min(r0 + R, p.rows) - 1) / p.G, rr.n_b - 1);
    const int lo = n_first <= n_last ? rr.lo(n_first) : 0, hi = n_first <= n_last ? rr.hi(n_last) : 0;
    // this CTA's share, in the key tiles that the shares are counted in
    int t_lo = lo / kT, t_hi = hi > lo ? (hi + kT - 1) / kT : t_lo;
    if (p.splits > 1) {
        const int per = (t_hi - t_lo + p.splits - 1) / p.splits;
        t_lo = min(t_lo + per * (int)blockIdx.y, t_hi);
        t_hi = min(t_lo + per, t_hi);
    }
    const int first = max(lo, t_lo * kT), end = min(hi, t_hi * kT);
    using P4 = Pack<T, 4>;
    auto pairs = [](const P4& v, unsigned long long (&out)[2]) {
        out[0] = pk2(to_f32(v.e[0]), to_f32(v.e[1]));
        out[1] = pk2(to_f32(v.e[2]), to_f32(v.e[3]));
    };
    int klo[R], khi[R];
    float m[R], l[R];
    unsigned long long q[R][F][2], o[R][F][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i, n = r / p.G;
        const bool live = r < p.rows && n < rr.n_b;
        klo[i] = live ? rr.lo(n) : 0;
        khi[i] = live ? rr.hi(n) : 0;
        m[i] = -INFINITY;
        l[i] = 0.f;
        const T* src = static_cast<const T*>(a.q) + b * a.q_stride[0] + n * a.q_stride[1] + (hk * p.G + r % p.G) * a.q_stride[2];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int c = (sub + 8 * f) * 4;
            q[i][f][0] = q[i][f][1] = o[i][f][0] = o[i][f][1] = pk2(0.f, 0.f);
            if (live && c < a.D) pairs(*reinterpret_cast<const P4*>(src + c), q[i][f]);
        }
    }
    const T* kk = static_cast<const T*>(a.k) + b * a.k_stride[0] + hk * a.k_stride[2];
    const T* vv = static_cast<const T*>(a.v) + b * a.v_stride[0] + hk * a.v_stride[2];
    const float s2 = a.scale * kLog2e;
    for (int j0 = first; j0 < end; j0 += kGroups * U) {
        P4 kx[U][F], vx[U][F];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kGroups + group;
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int c = (sub + 8 * f) * 4;
                kx[u][f] = vx[u][f] = P4{};
                if (j < end && c < a.D) {
                    kx[u][f] = *reinterpret_cast<const P4*>(kk + j * a.k_stride[1] + c);
                    vx[u][f] = *reinterpret_cast<const P4*>(vv + j * a.v_stride[1] + c);
                }
            }
        }
        float e[R][U];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                unsigned long long s = pk2(0.f, 0.f);
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    unsigned long long x[2];
                    pairs(kx[u][f], x);
                    s = fma2(q[i][f][1], x[1], fma2(q[i][f][0], x[0], s));
                }
                float x, y;
                upk2(s, x, y);
                x += y;
#pragma unroll
                for (int w = 4; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
                const int j = j0 + u * kGroups + group;
                e[i][u] = j < end && j >= klo[i] && j < khi[i] ? x * s2 : -INFINITY;
            }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float mx = m[i];
#pragma unroll
            for (int u = 0; u < U; ++u) mx = fmaxf(mx, e[i][u]);
            const float base = mx == -INFINITY ? 0.f : mx;   // nothing seen yet: every term is 0
            const float keep = ex2(m[i] - base);
            m[i] = mx;
            l[i] *= keep;
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int h = 0; h < 2; ++h) o[i][f][h] = fma2(o[i][f][h], pk2(keep, keep), pk2(0.f, 0.f));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * kGroups + group;
                if (j >= end || j < klo[i] || j >= khi[i]) continue;   // what is hidden is not touched, NaN or not
                const float x = ex2(e[i][u] - base);
                l[i] += x;
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    unsigned long long y[2];
                    pairs(vx[u][f], y);
                    o[i][f][0] = fma2(pk2(x, x), y[0], o[i][f][0]);
                    o[i][f][1] = fma2(pk2(x, x), y[1], o[i][f][1]);
                }
            }
        }
    }
    // the warp's four groups, then the warps
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int w = 8; w < 32; w <<= 1) {
            const float m1 = __shfl_xor_sync(0xffffffffu, m[i], w), l1 = __shfl_xor_sync(0xffffffffu, l[i], w);
            const float mx = fmaxf(m[i], m1), base = mx == -INFINITY ? 0.f : mx;
            const float k0 = ex2(m[i] - base), k1 = ex2(m1 - base);
            m[i] = mx;
            l[i] = l[i] * k0 + l1 * k1;
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    o[i][f][h] = fma2(__shfl_xor_sync(0xffffffffu, o[i][f][h], w), pk2(k1, k1),
                                      fma2(o[i][f][h], pk2(k0, k0), pk2(0.f, 0.f)));
        }
        if (lane < 8) {
#pragma unroll
            for (int f = 0; f < F; ++f) {
                ulonglong2 x;
                x.x = o[i][f][0], x.y = o[i][f][1];
                *reinterpret_cast<ulonglong2*>(&s_o[warp][i][(sub + 8 * f) * 4]) = x;
            }
            if (lane == 0) s_m[warp][i] = m[i], s_l[warp][i] = l[i];
        }
    }
    __syncthreads();
    for (int at = threadIdx.x; at < R * DP; at += kThr) {
        const int i = at / DP, d = at % DP, r = r0 + i;
        if (r >= p.rows || d >= a.D) continue;
        float mx = -INFINITY, total = 0.f, res = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][i]);
        const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float x = ex2(s_m[w][i] - base);
            total = fmaf(s_l[w][i], x, total);
            res = fmaf(s_o[w][i][d], x, res);
        }
        res *= total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
        const float lse = total == 0.f ? -INFINITY : (mx + log2f(total)) * kLn2;
        const int n = r / p.G, h = hk * p.G + r % p.G;
        if (p.splits > 1) {
            const long long row = (((long long)blockIdx.y * a.B + b) * a.Hkv + hk) * p.rows + r;
            p.part_o[row * a.D + d] = res;
            if (d == 0) p.part_lse[row] = lse;
        } else {
            const long long o_at = (((long long)b * a.N + n) * a.Hq + h) * a.D + d;
            store_rounded(static_cast<T*>(p.out) + o_at, p.out_rest ? static_cast<T*>(p.out_rest) + o_at : nullptr, res);
            if (d == 0 && p.lse) p.lse[((long long)b * a.Hq + h) * a.N + n] = lse;
        }
    }
}

// o = sum_s exp(lse_s - lse) o_s, lse = log sum_s exp lse_s: the shares of the key axis
// joined, one warp per packed row. There are at most 128 shares; eight shares' rows
// are in flight at a time. V: consecutive features per lane and load.
template <typename T, int V> __global__ void __launch_bounds__(128) attn_combine_kernel(const AttnParams p)
{
    __shared__ float weight[4][128];
    after_previous();
    const sdtw_attention& a = p.a;
    const long long all = (long long)a.B * a.Hkv * p.rows;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= all) return;
    const int r = (int)(row % p.rows);
    const int hk = (int)(row / p.rows % a.Hkv), b = (int)(row / p.rows / a.Hkv);
    const int n = r / p.G, h = hk * p.G + r % p.G;
    float w[4], m = -INFINITY;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        w[q] = lane + 32 * q < p.splits ? p.part_lse[(lane + 32 * q) * all + row] : -INFINITY;
        m = w[q] > m || isnan(w[q]) ? w[q] : m;   // NaN, from a row of NaN, stays
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, m, o);
        m = x > m || isnan(x) ? x : m;
    }
    const float base = m == -INFINITY ? 0.f : m;
    float total = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) total += w[q] = ex2((w[q] - base) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = total == 0.f ? 0.f : 1.f / total;
    float* ws = weight[threadIdx.x >> 5];
#pragma unroll
    for (int q = 0; q < 4; ++q) ws[lane + 32 * q] = w[q] * inv;
    __syncwarp();
    const long long at = (((long long)b * a.N + n) * a.Hq + h) * a.D;
    using P = Pack<float, V>;
    for (int d = lane * V; d < a.D; d += 32 * V) {
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
        const float* src = p.part_o + row * a.D + d;
        for (int s0 = 0; s0 < p.splits; s0 += 8) {
            P v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (s0 + q < p.splits) v[q] = *reinterpret_cast<const P*>(src + (s0 + q) * all * a.D);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (s0 + q < p.splits)
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(ws[s0 + q], v[q].e[e], acc[e]);
        }
        Pack<T, V> o, rest;
#pragma unroll
        for (int e = 0; e < V; ++e) store_rounded(&o.e[e], &rest.e[e], acc[e]);
        *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(p.out) + at + d) = o;
        if (p.out_rest) *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(p.out_rest) + at + d) = rest;
    }
    if (lane == 0 && p.lse)
        p.lse[((long long)b * a.Hq + h) * a.N + n] = total == 0.f ? -INFINITY : m + logf(total);
}

// What the backward kernels need of a row: lse in base-2 units (+inf where the row sees
// nothing or does not exist, which makes its probabilities 0) and delta = sum_d do o. The
// difference dP - delta cancels where one key has most of a row, so o is taken with what
// its rounding to 16 bits left; with the rounded o alone dq and dk were up to 5 times
// further from their 64-bit values than a plain fp32 pass on short fp16 sequences.
// One read of o, its rest and do bounds it: 2 x 4096 samples, 16 heads of 128, bf16 20 us, 5.0 TB/s.
// Eight lanes per packed row, 32 rows per CTA, in packed order and padded to whole tiles;
// VEC elements per load. For fp16 on the tensor cores also the largest squared norm of do
// of the CTA's rows, and in further CTAs of v of 32 keys; rows that see no key and keys that no row
// sees have none.
template <typename T, int VEC> __global__ void __launch_bounds__(256) attn_rowinfo_kernel(const AttnParams p)
{
    __shared__ float most[8];
    const sdtw_attention& a = p.a;
    const int sub = threadIdx.x & 7;
    const long long row_ctas = (long long)a.B * a.Hkv * (p.rows_pad / 32);
    float norm = 0.f;
    using P = Pack<T, VEC>;
    if (blockIdx.x < row_ctas) {
        const long long at = (long long)blockIdx.x * 32 + (threadIdx.x >> 3);
        const unsigned per = (unsigned)p.rows_pad / 32, bh = blockIdx.x / per;
        const int r = (int)(blockIdx.x - bh * per) * 32 + (threadIdx.x >> 3);
        const int b = (int)(bh / (unsigned)a.Hkv), hk = (int)(bh - (unsigned)b * a.Hkv);
        const int n_b = a.q_lengths ? min(max(a.q_lengths[b], 0), a.N) : a.N;
        const int n = r / p.G, h = hk * p.G + r % p.G;
        float lse = -INFINITY, delta = 0.f;
        if (r < p.rows && n < n_b) {
            lse = p.lse_in[((long long)b * a.Hq + h) * a.N + n];
            const long long o = (((long long)b * a.N + n) * a.Hq + h) * a.D;
            const T* x = static_cast<const T*>(p.out) + o;
            const T* rest = p.out_rest ? static_cast<const T*>(p.out_rest) + o : nullptr;
            const T* g = static_cast<const T*>(p.dout) + o;
            for (int d = sub * VEC; d < a.D && lse != -INFINITY; d += 8 * VEC) {
                const P xv = *reinterpret_cast<const P*>(x + d), gv = *reinterpret_cast<const P*>(g + d);
                P rv;
                if (rest) rv = *reinterpret_cast<const P*>(rest + d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float gf = to_f32(gv.e[e]);
                    delta = fmaf(to_f32(xv.e[e]) + (rest ? to_f32(rv.e[e]) : 0.f), gf, delta);
                    norm = fmaf(gf, gf, norm);
                }
            }
        }
#pragma unroll
        for (int q = 4; q > 0; q >>= 1) delta += __shfl_xor_sync(0xffffffffu, delta, q);
        if (sub == 0) {
            const bool none = lse == -INFINITY;
            p.row_lse[at] = none ? INFINITY : lse * kLog2e - (float)p.grad_shift;
            p.row_delta[at] = none ? 0.f : delta;
        }
    } else {
        const int per = (a.M + 31) / 32;
        const int c = (int)(blockIdx.x - row_ctas), bh = c / per, b = bh / a.Hkv;
        const RowRange rr(a, b);
        const int j = c % per * 32 + (threadIdx.x >> 3);
        if (j < rr.m_b && rr.row_lo(j) < rr.row_hi(j)) {
            const T* v = static_cast<const T*>(a.v) + b * a.v_stride[0] + j * a.v_stride[1] + bh % a.Hkv * a.v_stride[2];
            for (int d = sub * VEC; d < a.D; d += 8 * VEC) {
                const P vv = *reinterpret_cast<const P*>(v + d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) norm = fmaf(to_f32(vv.e[e]), to_f32(vv.e[e]), norm);
            }
        }
    }
    if (!p.norm_rows) return;
#pragma unroll
    for (int q = 4; q > 0; q >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, q);
#pragma unroll
    for (int q = 16; q > 4; q >>= 1) norm = fmaxf(norm, __shfl_xor_sync(0xffffffffu, norm, q));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = norm;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) norm = fmaxf(norm, most[w]);
        if (blockIdx.x < row_ctas) p.norm_rows[blockIdx.x] = norm;
        else p.norm_keys[blockIdx.x - row_ctas] = norm;
    }
}

// dq of 64 packed rows: S and dP = do v^T per key tile, dq += dS k.
template <typename T, int DP> __device__ __forceinline__ void dq_cta(const AttnParams& p, const int block, float* sm)
{
    constexpr int LD = DP + 4, NC = Cols<DP>::N * Cols<DP>::W;
    float* Q = sm;
    float* G = Q + kT * LD;
    float* K = G + kT * LD;
    float* V = K + kT * LD;
    float* S = V + kT * LD;
    const sdtw_attention& a = p.a;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int heads = a.B * a.Hkv, bh = block % heads;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int r0 = (((p.rows + kT - 1) / kT) - 1 - block / heads) * kT;
    const int last = min(r0 + kT, p.rows) - 1;
    const RowRange rr(a, b);
    const int n_first = r0 / p.G, n_last = min(last / p.G, rr.n_b - 1);
    int lo = 0, hi = 0;
    if (n_first <= n_last) {
        lo = rr.lo(n_first);
        hi = rr.hi(n_last);
    }
    const T* q = static_cast<const T*>(a.q) + b * a.q_stride[0];
    const T* dout = static_cast<const T*>(p.dout);
    const T* kk = static_cast<const T*>(a.k) + b * a.k_stride[0] + hk * a.k_stride[2];
    const T* vv = static_cast<const T*>(a.v) + b * a.v_stride[0] + hk * a.v_stride[2];
    load_tile<T, DP>(Q, a.D, p.packed, [&](int i) -> const T* {
        const int r = r0 + i;
        const int n = r / p.G;
        return r < p.rows && n < rr.n_b ? q + n * a.q_stride[1] + (hk * p.G + r % p.G) * a.q_stride[2] : nullptr;
    });
    load_tile<T, DP>(G, a.D, p.packed, [&](int i) -> const T* {
        const int r = r0 + i;
        const int n = r / p.G;
        return r < p.rows && n < rr.n_b ? dout + (((long long)b * a.N + n) * a.Hq + hk * p.G + r % p.G) * a.D : nullptr;
    });
    int klo[4], khi[4];
    float lse[4], delta[4];
    unsigned long long dq[4][NC / 2];
    const long long info = ((long long)b * a.Hkv + hk) * p.rows_pad;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty + 16 * i;
        const int n = r / p.G;
        const bool live = r < p.rows && n < rr.n_b;
        klo[i] = live ? rr.lo(n) : 0;
        khi[i] = live ? rr.hi(n) : 0;
        lse[i] = p.row_lse[info + r];
        delta[i] = p.row_delta[info + r];
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) dq[i][c] = pk2(0.f, 0.f);
    }
    const float s2 = a.scale * kLog2e, back = ex2(-(float)p.grad_shift);
    for (int j0 = lo / kT * kT; j0 < hi; j0 += kT) {
        __syncthreads();
        load_tile<T, DP>(K, a.D, p.packed, [&](int j) -> const T* { return j0 + j < rr.m_b ? kk + (j0 + j) * a.k_stride[1] : nullptr; });
        load_tile<T, DP>(V, a.D, p.packed, [&](int j) -> const T* { return j0 + j < rr.m_b ? vv + (j0 + j) * a.v_stride[1] : nullptr; });
        __syncthreads();
        float s[4][4], dp[4][4];
        dot_tile<DP, 4>(s, Q, K, ty, tx);
        dot_tile<DP, 4>(dp, G, V, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + tx + 16 * j;
                const bool see = key >= klo[i] && key < khi[i];
                S[(ty + 16 * i) * kPitchP + tx + 16 * j] =
                    see ? ex2(fmaf(s[i][j], s2, -lse[i])) * (dp[i][j] - delta[i]) : 0.f;
            }
        __syncthreads();
        mul_tile<DP, 4>(dq, S, K, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty + 16 * i;
        if (r >= p.rows) continue;
        float res[NC];
        unpack(dq[i], back, res);
        if (klo[i] >= khi[i])   // 0 whatever the keys hold that other rows of the tile see
#pragma unroll
            for (int c = 0; c < NC; ++c) res[c] = 0.f;
        T* out = static_cast<T*>(p.dq) + (((long long)b * a.N + r / p.G) * a.Hq + hk * p.G + r % p.G) * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = Cols<DP>::at(tx, c / Cols<DP>::W, c % Cols<DP>::W);
            if (d < a.D) out[d] = from_f32<T>(res[c] * a.scale);
        }
    }
}

// dk and dv of 64 keys: S^T and dP^T per tile of packed rows, dv += P^T do, dk += dS^T q.
template <typename T, int DP> __device__ __forceinline__ void dkv_cta(const AttnParams& p, const int block, float* sm)
{
    constexpr int LD = DP + 4, NC = Cols<DP>::N * Cols<DP>::W;
    float* K = sm;
    float* V = K + kT * LD;
    float* Q = V + kT * LD;
    float* G = Q + kT * LD;
    float* P = G + kT * LD;
    float* S = P + kT * kPitchP;
    const sdtw_attention& a = p.a;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int heads = a.B * a.Hkv, bh = block % heads;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int j0 = block / heads * kT;   // the first keys are seen by the most rows
    const RowRange rr(a, b);
    const RowRange::Rows rows = rr.seeing(j0, j0 + kT, p.G);
    const T* q = static_cast<const T*>(a.q) + b * a.q_stride[0];
    const T* dout = static_cast<const T*>(p.dout);
    const T* kk = static_cast<const T*>(a.k) + b * a.k_stride[0] + hk * a.k_stride[2];
    const T* vv = static_cast<const T*>(a.v) + b * a.v_stride[0] + hk * a.v_stride[2];
    load_tile<T, DP>(K, a.D, p.packed, [&](int j) -> const T* { return j0 + j < rr.m_b ? kk + (j0 + j) * a.k_stride[1] : nullptr; });
    load_tile<T, DP>(V, a.D, p.packed, [&](int j) -> const T* { return j0 + j < rr.m_b ? vv + (j0 + j) * a.v_stride[1] : nullptr; });
    unsigned long long dk[4][NC / 2], dv[4][NC / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) dk[i][c] = dv[i][c] = pk2(0.f, 0.f);
    const float s2 = a.scale * kLog2e, back = ex2(-(float)p.grad_shift);
    const long long info = ((long long)b * a.Hkv + hk) * p.rows_pad;
    for (int r0 = rows.lo / kT * kT; r0 < rows.hi; r0 += kT) {
        __syncthreads();
        load_tile<T, DP>(Q, a.D, p.packed, [&](int i) -> const T* {
            const int r = r0 + i;
            const int n = r / p.G;
            return r < p.rows && n < rr.n_b ? q + n * a.q_stride[1] + (hk * p.G + r % p.G) * a.q_stride[2] : nullptr;
        });
        load_tile<T, DP>(G, a.D, p.packed, [&](int i) -> const T* {
            const int r = r0 + i;
            const int n = r / p.G;
            return r < p.rows && n < rr.n_b ? dout + (((long long)b * a.N + n) * a.Hq + hk * p.G + r % p.G) * a.D : nullptr;
        });
        __syncthreads();
        // rows that see no key, which stand before the first, are cleared: 0 * NaN is not 0
        if (const int blind = min(rr.first_row() * p.G - r0, kT) * LD; blind > 0) {
            for (int e = threadIdx.x; e < blind; e += kThr) Q[e] = G[e] = 0.f;
            __syncthreads();
        }
        float s[4][4], dp[4][4];
        dot_tile<DP, 4>(s, K, Q, ty, tx);
        dot_tile<DP, 4>(dp, V, G, ty, tx);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + tx + 16 * j;
            const int n = r / p.G;
            const bool live = n < rr.n_b;
            const int klo = live ? rr.lo(n) : 0, khi = live ? rr.hi(n) : 0;
            const float lse = p.row_lse[info + r], delta = p.row_delta[info + r];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = j0 + ty + 16 * i;
                const bool see = key >= klo && key < khi;
                const float e = see ? ex2(fmaf(s[i][j], s2, -lse)) : 0.f;
                P[(ty + 16 * i) * kPitchP + tx + 16 * j] = e;
                S[(ty + 16 * i) * kPitchP + tx + 16 * j] = see ? e * (dp[i][j] - delta) : 0.f;
            }
        }
        __syncthreads();
        mul_tile<DP, 4>(dv, P, G, ty, tx);
        mul_tile<DP, 4>(dk, S, Q, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + ty + 16 * i;
        if (j >= a.M) continue;
        const long long o = (((long long)b * a.M + j) * a.Hkv + hk) * a.D;
        float rk[NC], rv[NC];
        unpack(dk[i], back, rk);
        unpack(dv[i], back, rv);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = Cols<DP>::at(tx, c / Cols<DP>::W, c % Cols<DP>::W);
            if (d < a.D) {
                if (p.dk) static_cast<T*>(p.dk)[o + d] = from_f32<T>(rk[c] * a.scale);
                if (p.dv) static_cast<T*>(p.dv)[o + d] = from_f32<T>(rv[c]);
            }
        }
    }
}

// Both kinds of CTAs in one launch, the ones that take longer first.
template <typename T, int DP> __global__ void __launch_bounds__(kThr, DP == 128 ? 1 : 2) attn_bwd_simt(const AttnParams p, const int dkv)
{
    extern __shared__ float sm[];
    if ((int)blockIdx.x < dkv) dkv_cta<T, DP>(p, (int)blockIdx.x, sm);
    else dq_cta<T, DP>(p, (int)blockIdx.x - dkv, sm);
}

template <typename T, int DP, int R> cudaError_t fwd_simt(const AttnParams& p, cudaStream_t s)
{
    constexpr size_t smem = sizeof(float) * ((16 * R + 2 * kT) * (DP + 4) + 16 * R * kPitchP);
    const cudaError_t e = allow_smem<attn_fwd_simt<T, DP, R>>(smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)((p.rows + 16 * R - 1) / (16 * R));
    attn_fwd_simt<T, DP, R><<<dim3(tiles * p.a.B * p.a.Hkv, p.splits), kThr, smem, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int DP> cudaError_t fwd_simt(const AttnParams& p, cudaStream_t s)
{
    if (p.few) {
        const dim3 grid((unsigned)(p.a.B * p.a.Hkv), p.splits, (p.rows + 3) / 4);
        if (p.rows == 1) attn_fwd_few<T, DP, 1><<<grid, kThr, 0, s>>>(p);
        else if (p.rows == 2) attn_fwd_few<T, DP, 2><<<grid, kThr, 0, s>>>(p);
        else attn_fwd_few<T, DP, 4><<<grid, kThr, 0, s>>>(p);
        return cudaGetLastError();
    }
    return p.rows <= 16 ? fwd_simt<T, DP, 1>(p, s) : fwd_simt<T, DP, 4>(p, s);
}

template <typename T, int DP> cudaError_t bwd_simt(const AttnParams& p, cudaStream_t s)
{
    constexpr size_t smem = sizeof(float) * (4 * kT * (DP + 4) + 2 * kT * kPitchP);
    const cudaError_t e = allow_smem<attn_bwd_simt<T, DP>>(smem);
    if (e != cudaSuccess) return e;
    const int heads = p.a.B * p.a.Hkv;
    const int dkv = p.dk ? (p.a.M + kT - 1) / kT * heads : 0, dq = p.dq ? (p.rows + kT - 1) / kT * heads : 0;
    attn_bwd_simt<T, DP><<<(unsigned)(dkv + dq), kThr, smem, s>>>(p, dkv);
    return cudaGetLastError();
}

template <typename T> cudaError_t fwd_typed(const AttnParams& p, cudaStream_t s)
{
    return p.a.D <= 32 ? fwd_simt<T, 32>(p, s) : p.a.D <= 64 ? fwd_simt<T, 64>(p, s) : fwd_simt<T, 128>(p, s);
}
template <typename T> cudaError_t bwd_typed(const AttnParams& p, cudaStream_t s)
{
    return p.a.D <= 32 ? bwd_simt<T, 32>(p, s) : p.a.D <= 64 ? bwd_simt<T, 64>(p, s) : bwd_simt<T, 128>(p, s);
}

}  // namespace

cudaError_t launch_attn_forward_simt(const AttnParams& p, cudaStream_t s)
{
    if (p.a.dtype == SDTW_F32) return fwd_typed<float>(p, s);
    if (p.a.dtype == SDTW_BF16) return fwd_typed<__nv_bfloat16>(p, s);
    return fwd_typed<__half>(p, s);
}

cudaError_t launch_attn_backward_simt(const AttnParams& p, cudaStream_t s)
{
    if (p.a.dtype == SDTW_F32) return bwd_typed<float>(p, s);
    if (p.a.dtype == SDTW_BF16) return bwd_typed<__nv_bfloat16>(p, s);
    return bwd_typed<__half>(p, s);
}

template <typename T> static cudaError_t combine_typed(const AttnParams& p, cudaStream_t s)
{
    const unsigned grid = (unsigned)(((long long)p.a.B * p.a.Hkv * p.rows + 3) / 4);
    if (p.a.D % 4 == 0 && aligned16(p.out) && aligned16(p.out_rest)) return launch_behind(attn_combine_kernel<T, 4>, grid, 128, s, p);
    return launch_behind(attn_combine_kernel<T, 1>, grid, 128, s, p);
}

cudaError_t launch_attn_combine(const AttnParams& p, cudaStream_t s)
{
    if (p.a.dtype == SDTW_F32) return combine_typed<float>(p, s);
    if (p.a.dtype == SDTW_BF16) return combine_typed<__nv_bfloat16>(p, s);
    return combine_typed<__half>(p, s);
}

template <typename T> static cudaError_t rowinfo_typed(const AttnParams& p, cudaStream_t s)
{
    long long grid = (long long)p.a.B * p.a.Hkv * (p.rows_pad / 32);
    if (p.norm_rows) grid += (long long)p.a.B * p.a.Hkv * ((p.a.M + 31) / 32);
    constexpr int VEC = 16 / sizeof(T);
    bool packed = p.a.D % VEC == 0 && aligned16(p.out) && aligned16(p.out_rest) && aligned16(p.dout);
    if (p.norm_rows) packed = packed && p.tc;   // whose v has 16-byte rows
    if (packed) attn_rowinfo_kernel<T, VEC><<<(unsigned)grid, 256, 0, s>>>(p);
    else attn_rowinfo_kernel<T, 1><<<(unsigned)grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn_rowinfo(const AttnParams& p, cudaStream_t s)
{
    if (p.a.dtype == SDTW_F32) return rowinfo_typed<float>(p, s);
    if (p.a.dtype == SDTW_BF16) return rowinfo_typed<__nv_bfloat16>(p, s);
    return rowinfo_typed<__half>(p, s);
}

}  // namespace sdtw
