// group_norm.cu -- group norm with an activation, channels last, forward and backward.
//
//   over a batch element's n = n_b cg values of a group: mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps),
//   xh = (x - mu) r, z = xh w + b, y = act(z)
//   dz = dy act'(z), g = dz w, dx = r (g - mean g - xh mean(g xh)), dw = sum dz xh, db = sum dz
//
// Memory bounds it: x is read once and y written once, x and dy once for dx. A slab, whole groups of a batch element's
// channels at least 128 bytes wide, stays in the shared memory of a cluster of up to 16 CTAs that share its positions, from
// its one load to its results; sums of its groups go between the CTAs through shared memory. The variance is the mean
// square of centred values. A thread has the same channels throughout, and sums the weights' gradients in registers over
// all that its CTA takes; the CTAs' sums are added by a second launch in a fixed order: the same bits every time. Slabs
// that a cluster cannot hold are read again, from the cache where it has them.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "activation.cuh"
#include "block.h"
#include "packed.cuh"

namespace sdtw {
namespace {

constexpr int kThreads = 256, kWarpsG = kThreads / 32, kMostCtas = 16;

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
template <bool EXACT, bool SLOPE> __device__ __forceinline__ float activate_as(int activation, float z, float& slope) {
    switch (activation) {
        case SDTW_ACT_SILU: return activate<SDTW_ACT_SILU, EXACT, SLOPE>(z, slope);
        case SDTW_ACT_GELU: return activate<SDTW_ACT_GELU, EXACT, SLOPE>(z, slope);
        case SDTW_ACT_RELU: return activate<SDTW_ACT_RELU, EXACT, SLOPE>(z, slope);
        default: return activate<SDTW_ACT_NONE, EXACT, SLOPE>(z, slope);
    }
}
// v[e] = activation of v[e], or its derivative
template <bool EXACT, bool SLOPE, int VEC> __device__ __forceinline__ void activate_all(int activation, float (&v)[VEC]) {
    auto each = [&](auto act) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float slope;
            const float y = activate<act(), EXACT, SLOPE>(v[e], slope);
            v[e] = SLOPE ? slope : y;
        }
    };
    switch (activation) {
        case SDTW_ACT_SILU: each(std::integral_constant<int, SDTW_ACT_SILU>()); break;
        case SDTW_ACT_GELU: each(std::integral_constant<int, SDTW_ACT_GELU>()); break;
        case SDTW_ACT_RELU: each(std::integral_constant<int, SDTW_ACT_RELU>()); break;
        default: each(std::integral_constant<int, SDTW_ACT_NONE>());
    }
}

// How a call is laid over the GPU. A CTA has `items` batch elements at a time, `lanes` rows of each in flight, `packs` packs
// to a row of its slab; thread = (item * lanes + row) * packs + pack. With several items of a few positions there are no
// clusters.
struct Layout {
    bool fits;               // else the kernels of any size take it
    bool held;               // in shared memory
    int vec, width, packs;   // elements of a pack; channels and packs of a slab
    int slabs, items, lanes, rounds;   // rounds: rows of a thread
    int ctas, part;          // CTAs of a cluster, positions of each
    int columns;             // CTAs or clusters side by side that share the items of a slab
    size_t smem;
};

__device__ __forceinline__ void cluster_sync_g() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(const float* mine, int cta, float v) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(mine);
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
}

// Sums of the CTA's (and the cluster's) groups. `v` are a thread's sums of its channels, red holds those of all threads, one
// row of threads after the other; a warp adds up a group, then the CTAs' sums of it are exchanged. Every thread finds the sum of
// group `g` of its item in sums[item * groups + g]. `parts`: [ctas][items * groups], of this call alone.
template <int VEC>
__device__ __forceinline__ void group_sums(const float (&v)[VEC], float* red, float* parts, float* sums, const Layout& L, int cg, int rank)
{
    const int groups = L.width / cg, all = L.items * groups, rows = L.lanes, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)threadIdx.x < L.items * rows * L.packs) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) red[threadIdx.x * VEC + e] = v[e];
    }
    __syncthreads();
    const int n = rows * cg;
    for (int k = warp; k < all; k += kWarpsG) {
        const float* first = red + k / groups * rows * L.width + k % groups * cg;
        float s = 0.f;
        for (int i = lane; i < n; i += 32) s += first[i / cg * L.width + i % cg];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (L.ctas == 1) {
            if (lane == 0) sums[k] = s;
        } else if (lane < L.ctas) {
            store_remote(parts + rank * all + k, lane, s);
        }
    }
    if (L.ctas > 1) {
        cluster_sync_g();
        for (int k = threadIdx.x; k < all; k += kThreads) {
            float s = 0.f;
            for (int c = 0; c < L.ctas; ++c) s += parts[c * all + k];
            sums[k] = s;
        }
    }
    __syncthreads();
}

template <typename T, int VEC> __device__ __forceinline__ void unpack(const Pack<T, VEC>& p, float (&v)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = to_f32(p.e[e]);
}
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> packed_of(const float (&v)[VEC]) {
    Pack<T, VEC> p;
    if constexpr (VEC > 1 && sizeof(T) == 2) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) *reinterpret_cast<uint32_t*>(&p.e[e]) = pack2<T>(v[e], v[e + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p.e[e] = from_f32<T>(v[e]);
    }
    return p;
}
__device__ __forceinline__ void fetch16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// What a thread has of a round of items: rows [first, first + rounds * lanes) of its batch element, every lanes-th.
struct Place {
    int item, row, pack, b, len, first, last;   // its rows are first + k lanes < last
    long long at;                               // of the first, in elements
    bool on;
    __device__ __forceinline__ Place(const GroupNormParams& p, const Layout& L, int slab, int b0, int rank) {
        pack = threadIdx.x % L.packs;
        row = threadIdx.x / L.packs % L.lanes;
        item = threadIdx.x / (L.packs * L.lanes);
        b = b0 + item;
        on = item < L.items && b < p.B;
        len = !on ? 0 : p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
        first = rank * L.part + row;
        last = on ? min(p.S, (rank + 1) * L.part) : 0;
        at = ((long long)b * p.S + first) * p.C + slab * L.width + pack * L.vec;
    }
};

template <typename T, int VEC, bool HELD> __global__ void __launch_bounds__(kThreads, 2) group_fwd_kernel(const GroupNormParams p, const Layout L)
{
    extern __shared__ __align__(16) unsigned char held[];   // [rounds][kThreads] packs, then the sums
    using P = Pack<T, VEC>;
    const int slab = blockIdx.x / L.ctas % L.slabs, rank = blockIdx.x % L.ctas, groups = L.width / p.cg, all = L.items * groups;
    float* red = reinterpret_cast<float*>(held + (HELD ? (size_t)L.rounds * kThreads * 16 : 0));
    float* sums = red + kThreads * VEC;                     // of values, of squares
    float* parts = sums + 2 * all;                          // likewise
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.y);
    float w[VEC], bias[VEC];
    int group[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = threadIdx.x % L.packs * VEC + e;
        group[e] = c / p.cg;
        w[e] = wval(p.weight, slab * L.width + c, p.wdtype, 1.f);
        bias[e] = wval(p.bias, slab * L.width + c, p.wdtype, 0.f);
    }
    if (L.ctas > 1) cluster_sync_g();                       // the others have begun
    const long long step = (long long)L.lanes * p.C;
    for (int b0 = blockIdx.x / (L.ctas * L.slabs) * L.items; b0 < p.B; b0 += L.columns * L.items) {
        const Place at(p, L, slab, b0, rank);
        const int there = min(at.last, at.len);             // rows that take part
        P* mine = reinterpret_cast<P*>(held) + threadIdx.x;
        auto value = [&](int k) { return HELD ? mine[k * kThreads] : *reinterpret_cast<const P*>(x + at.at + k * step); };
        if constexpr (HELD) {
            for (int k = 0, s = at.first; s < there; ++k, s += L.lanes) fetch16(mine + k * kThreads, x + at.at + k * step);
            fetched();
        }
        float s[VEC] = {};
        for (int k = 0, i = at.first; i < there; ++k, i += L.lanes) {
            float v[VEC];
            unpack<T, VEC>(value(k), v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] += v[e];
        }
        group_sums<VEC>(s, red, parts, sums, L, p.cg, rank);
        const float n = (float)at.len * (float)p.cg, inv = at.len ? 1.f / n : 0.f;
        float mu[VEC], rw[VEC];
        const int g0 = at.item < L.items ? at.item * groups : 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) mu[e] = sums[g0 + group[e]] * inv, s[e] = 0.f;
        for (int k = 0, i = at.first; i < there; ++k, i += L.lanes) {
            float v[VEC];
            unpack<T, VEC>(value(k), v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] = fmaf(v[e] - mu[e], v[e] - mu[e], s[e]);
        }
        group_sums<VEC>(s, red, parts + L.ctas * all, sums + all, L, p.cg, rank);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float r = at.len ? 1.f / sqrtf(sums[all + g0 + group[e]] * inv + p.eps) : 0.f;
            if (p.mean && rank == 0 && at.on && at.row == 0 && (at.pack * VEC + e) % p.cg == 0) {
                const long long to = (long long)at.b * p.G + slab * groups + group[e];
                p.mean[to] = mu[e], p.rstd[to] = r;
            }
            rw[e] = r * w[e];
        }
        for (int k = 0, i = at.first; i < at.last; ++k, i += L.lanes) {
            float v[VEC] = {};
            if (i < there) {
                unpack<T, VEC>(value(k), v);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = fmaf(v[e] - mu[e], rw[e], bias[e]);
                activate_all<sizeof(T) == 4, false, VEC>(p.activation, v);
            }
            *reinterpret_cast<P*>(y + at.at + k * step) = packed_of<T, VEC>(v);
        }
    }
}

template <typename T, int VEC, bool HELD> __global__ void __launch_bounds__(kThreads, 2) group_bwd_kernel(const GroupNormParams p, const Layout L)
{
    extern __shared__ __align__(16) unsigned char held[];   // [rounds][x, dy][kThreads] packs, then the sums
    using P = Pack<T, VEC>;
    const int slab = blockIdx.x / L.ctas % L.slabs, rank = blockIdx.x % L.ctas, groups = L.width / p.cg, all = L.items * groups;
    const int column = blockIdx.x / (L.ctas * L.slabs);
    float* red = reinterpret_cast<float*>(held + (HELD ? (size_t)L.rounds * 2 * kThreads * 16 : 0));
    float* sums = red + kThreads * VEC;
    float* parts = sums + 2 * all;
    const T *x = static_cast<const T*>(p.x), *dy = static_cast<const T*>(p.dy);
    T* dx = static_cast<T*>(p.dx);
    float w[VEC], bias[VEC], dw[VEC] = {}, db[VEC] = {};
    int group[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = threadIdx.x % L.packs * VEC + e;
        group[e] = c / p.cg;
        w[e] = wval(p.weight, slab * L.width + c, p.wdtype, 1.f);
        bias[e] = wval(p.bias, slab * L.width + c, p.wdtype, 0.f);
    }
    if (L.ctas > 1) cluster_sync_g();
    const long long step = (long long)L.lanes * p.C;
    int turn = 0;
    for (int b0 = column * L.items; b0 < p.B; b0 += L.columns * L.items, turn ^= 1) {
        const Place at(p, L, slab, b0, rank);
        const int there = min(at.last, at.len);
        P* mine = reinterpret_cast<P*>(held) + threadIdx.x;
        auto value = [&](int k, int which) {
            return HELD ? mine[(2 * k + which) * kThreads] : *reinterpret_cast<const P*>((which ? dy : x) + at.at + k * step);
        };
        if constexpr (HELD)
            for (int k = 0, s = at.first; s < there; ++k, s += L.lanes) {
                fetch16(mine + 2 * k * kThreads, x + at.at + k * step);
                fetch16(mine + (2 * k + 1) * kThreads, dy + at.at + k * step);
            }
        float mu[VEC], r[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const long long from = (long long)(at.on ? at.b : 0) * p.G + slab * groups + group[e];
            mu[e] = p.mean[from], r[e] = p.rstd[from];
        }
        if constexpr (HELD) fetched();
        // xh and dz of a pack
        auto both = [&](int k, float (&xh)[VEC], float (&dz)[VEC]) {
            float z[VEC];
            unpack<T, VEC>(value(k, 0), xh);
            unpack<T, VEC>(value(k, 1), dz);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                xh[e] = (xh[e] - mu[e]) * r[e];
                z[e] = fmaf(xh[e], w[e], bias[e]);
            }
            activate_all<sizeof(T) == 4, true, VEC>(p.activation, z);
#pragma unroll
            for (int e = 0; e < VEC; ++e) dz[e] *= z[e];
        };
        float s1[VEC] = {}, s2[VEC] = {};
        for (int k = 0, i = at.first; i < there; ++k, i += L.lanes) {
            float xh[VEC], dz[VEC];
            both(k, xh, dz);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s1[e] += dz[e];
                s2[e] = fmaf(dz[e], xh[e], s2[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            db[e] += s1[e], dw[e] += s2[e];
            s1[e] *= w[e], s2[e] *= w[e];
        }
        if (!dx) continue;
        group_sums<VEC>(s1, red, parts + 2 * turn * L.ctas * all, sums, L, p.cg, rank);
        group_sums<VEC>(s2, red, parts + (2 * turn + 1) * L.ctas * all, sums + all, L, p.cg, rank);
        const float inv = at.len ? 1.f / ((float)at.len * (float)p.cg) : 0.f;
        const int g0 = at.item < L.items ? at.item * groups : 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s1[e] = sums[g0 + group[e]] * inv, s2[e] = sums[all + g0 + group[e]] * inv;
        for (int k = 0, i = at.first; i < at.last; ++k, i += L.lanes) {
            float xh[VEC], dz[VEC] = {};
            if (i < there) {
                both(k, xh, dz);
#pragma unroll
                for (int e = 0; e < VEC; ++e) dz[e] = r[e] * (fmaf(dz[e], w[e], -s1[e]) - xh[e] * s2[e]);
            }
            *reinterpret_cast<P*>(dx + at.at + k * step) = packed_of<T, VEC>(dz);
        }
    }
    if (!p.partial) return;
    // the threads of a pack, one after the other
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) red[threadIdx.x * VEC + e] = which ? db[e] : dw[e];
        __syncthreads();
        float* out = p.partial + (((long long)column * L.ctas + rank) * 2 + which) * p.C + slab * L.width;
        for (int c = threadIdx.x; c < L.width; c += kThreads) {
            float s = 0.f;
            for (int k = 0; k < L.items * L.lanes; ++k) s += red[k * L.width + c];
            out[c] = s;
        }
    }
}

// ---- groups too wide for the above: a CTA a group of a batch element
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
template <typename T> __global__ void __launch_bounds__(kThreads) group_fwd_any_kernel(const GroupNormParams p)
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
            v = activate_as<sizeof(T) == 4, false>(p.activation, fmaf((to_f32(x[at(i)]) - mu) * r, wval(p.weight, c, p.wdtype, 1.f),
                                                                      wval(p.bias, c, p.wdtype, 0.f)), none);
        y[at(i)] = from_f32<T>(v);
    }
    if (threadIdx.x == 0 && p.mean) p.mean[blockIdx.x] = mu, p.rstd[blockIdx.x] = r;
}

template <typename T> __global__ void __launch_bounds__(kThreads) group_bwd_any_kernel(const GroupNormParams p)
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
        activate_as<sizeof(T) == 4, true>(p.activation, fmaf(xh, w, wval(p.bias, g * p.cg + c, p.wdtype, 0.f)), slope);
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
            p.partial[2ll * b * p.C + g * p.cg + c] = dw;
            p.partial[(2ll * b + 1) * p.C + g * p.cg + c] = db;
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

// dw, db: the partial rows added in a fixed order, 32 columns by 32 row lanes
__global__ void __launch_bounds__(1024) group_fold_kernel(const GroupNormParams p, int rows)
{
    __shared__ float part[32][33];
    after_previous();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    float s[4] = {};
    if (c < p.C)
        for (int t = lane; t < rows; t += 128) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (t + 32 * q < rows) s[q] += p.partial[(2ll * (t + 32 * q) + blockIdx.y) * p.C + c];
        }
    part[lane][threadIdx.x & 31] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    float v = part[threadIdx.x & 31][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int col = blockIdx.x * 32 + lane;
    void* dst = blockIdx.y ? p.dbias : p.dweight;
    if ((threadIdx.x & 31) == 0 && col < p.C && dst) wstore(dst, col, p.wdtype, v);
}

template <typename F> cudaError_t with_type(int dtype, F f) {
    if (dtype == SDTW_F32) return f(float());
    if (dtype == SDTW_BF16) return f(__nv_bfloat16());
    return f(__half());
}

long long gcd(long long a, long long b) { return b ? gcd(b, a % b) : a; }

// Both alignments' layouts are asked for by the size of the workspace, which so does not depend on addresses.
Layout layout(const GroupNormParams& p, bool backward, bool packs, int sms)
{
    Layout L{};
    const int size = dtype_size(p.dtype);
    L.vec = packs && p.C % (16 / size) == 0 ? 16 / size : 1;
    const long long whole = p.cg / gcd(p.cg, L.vec) * L.vec;    // channels of whole groups and whole packs
    L.width = (int)whole;
    // at least 128 bytes a row, or all channels
    for (long long j = 1; whole * j <= p.C; ++j)
        if (p.C % (whole * j) == 0) {
            if (j > 1 && whole * j > kThreads * L.vec) break;
            L.width = (int)(whole * j);
            if (L.width * size >= 128) break;
        }
    L.packs = L.width / L.vec;
    if (L.packs > kThreads) return L;
    L.fits = true;
    L.slabs = p.C / L.width;
    const int most = kThreads / L.packs;
    L.lanes = std::min(most, p.S);
    L.items = std::min(most / L.lanes, p.B);
    // few items are spread over the SMs
    while (L.items > 1 && (long long)((p.B + L.items - 1) / L.items) * L.slabs < sms) L.items = (L.items + 1) / 2;
    const int arrays = backward ? 2 : 1;
    const size_t sums = ((size_t)kThreads * L.vec + 2 * L.items * (L.width / p.cg)) * sizeof(float);
    auto bytes = [&](int ctas) {
        const size_t exchange = ctas > 1 ? (size_t)4 * ctas * (L.width / p.cg) * sizeof(float) : 0;
        const long long rounds = ((p.S + ctas - 1) / ctas + L.lanes - 1) / L.lanes;
        return std::pair<size_t, long long>(sums + exchange, rounds * kThreads * 16 * arrays);
    };
    // CTAs of a cluster: until three fit on an SM side by side, and there are two an SM
    L.ctas = 1;
    const long long clusters = (long long)((p.B + L.items - 1) / L.items) * L.slabs;
    while (L.ctas < kMostCtas && L.items == 1 && (p.S + 2 * L.ctas - 1) / (2 * L.ctas) >= 2 * L.lanes &&
           ((long long)bytes(L.ctas).first + bytes(L.ctas).second > 72 * 1024 || clusters * L.ctas < 2 * sms))
        L.ctas *= 2;
    const auto need = bytes(L.ctas);
    L.part = (p.S + L.ctas - 1) / L.ctas;
    L.rounds = (L.part + L.lanes - 1) / L.lanes;
    L.held = L.vec > 1 && (long long)need.first + need.second <= 220 * 1024;
    L.smem = need.first + (L.held ? (size_t)need.second : 0);
    // persistent where there are many small items
    const long long wanted = (p.B + L.items - 1) / L.items, per_sm = std::max<long long>(1, std::min<long long>(8, 220 * 1024 / (long long)L.smem));
    L.columns = (int)std::min(wanted, std::max(1ll, L.ctas > 1 ? wanted : (sms * per_sm + L.slabs - 1) / L.slabs));
    return L;
}

template <auto Kernel> cudaError_t launch(const GroupNormParams& p, const Layout& L, cudaStream_t s)
{
    if (const cudaError_t e = allow_smem<Kernel>(226 * 1024); e != cudaSuccess) return e;
    if (L.ctas > 8)
        if (const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)L.ctas, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.gridDim = dim3((unsigned)((long long)L.columns * L.slabs * L.ctas)), c.blockDim = dim3(kThreads), c.stream = s, c.attrs = &at;
    c.numAttrs = L.ctas > 1 ? 1 : 0, c.dynamicSmemBytes = L.smem;
    return cudaLaunchKernelEx(&c, Kernel, p, L);
}

bool packs(const GroupNormParams& p) { return aligned16(p.x) && aligned16(p.y) && aligned16(p.dy) && aligned16(p.dx); }
int partial_rows(const GroupNormParams& p, const Layout& L) { return L.fits ? L.columns * L.ctas : p.B; }

}  // namespace

size_t group_norm_workspace(const GroupNormParams& p, bool backward, int sms)
{
    if (!backward) return 0;
    const size_t rows = std::max(partial_rows(p, layout(p, true, true, sms)), partial_rows(p, layout(p, true, false, sms)));
    return sizeof(float) * 2 * rows * p.C;
}

cudaError_t launch_group_norm_forward(const GroupNormParams& p, int sms, cudaStream_t s)
{
    const Layout L = layout(p, false, packs(p), sms);
    return with_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int VEC = 16 / sizeof(T);
        if (L.fits) return L.vec == 1 ? launch<group_fwd_kernel<T, 1, false>>(p, L, s) : L.held ? launch<group_fwd_kernel<T, VEC, true>>(p, L, s)
                                                                                              : launch<group_fwd_kernel<T, VEC, false>>(p, L, s);
        group_fwd_any_kernel<T><<<p.B * p.G, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_group_norm_backward(const GroupNormParams& p0, int sms, cudaStream_t s)
{
    GroupNormParams p = p0;
    if (!p.dweight && !p.dbias) p.partial = nullptr;
    const Layout L = layout(p, true, packs(p), sms);
    const cudaError_t e = with_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int VEC = 16 / sizeof(T);
        if (L.fits) return L.vec == 1 ? launch<group_bwd_kernel<T, 1, false>>(p, L, s) : L.held ? launch<group_bwd_kernel<T, VEC, true>>(p, L, s)
                                                                                              : launch<group_bwd_kernel<T, VEC, false>>(p, L, s);
        group_bwd_any_kernel<T><<<p.B * p.G, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !p.partial) return e;
    return launch_behind(group_fold_kernel, dim3((p.C + 31) / 32, 2), 1024, s, p, partial_rows(p, L));
}

}  // namespace sdtw
