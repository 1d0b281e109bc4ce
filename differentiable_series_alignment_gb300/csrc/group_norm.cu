// group_norm.cu -- group norm with an activation, channels last, forward and backward.
//
//   over a batch element's n = n_b cg values of a group: mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps),
//   xh = (x - mu) r, z = xh w + b, y = act(z)
//   dz = dy act'(z), g = dz w, dx = r (g - mean g - xh mean(g xh)), dw = sum dz xh, db = sum dz
//
// Memory bounds it: x is read once and y written once, x and dy once for dx. A slab, whole groups of a batch element's
// channels at least 64 bytes wide, stays in the shared memory of a cluster of up to 16 CTAs that share its positions, from
// its one load to its results; sums of its groups go between the CTAs through shared memory. The variance is the mean
// square of centred values. A thread has the same channels throughout, and sums the weights' gradients in registers over
// all that its CTA takes; the CTAs' sums are added by a second launch in a fixed order: the same bits every time. Slabs
// that a cluster cannot hold are read again, from the cache where it has them.
//
// Measured: 16 x 4096 x 512 bf16 by 32 groups with SiLU 41 us forward (3.3 TB/s), 85 backward (2.4); 64 such 147 and 306; 65535 rows of
// 1024 by groups of 128 70 and 97 (3.8 and 4.1 TB/s). Not memory bounds these but instructions (three passes over a
// pack, an exponential and a reciprocal an element in each that needs the activation) and the barriers between passes. Reading slabs again
// in place of keeping them takes 47 and 100 us, 64 such 176 and 405.
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
// z = activation of z, or its derivative
template <bool EXACT, bool SLOPE, int Q> __device__ __forceinline__ void activate_all(int activation, Pair (&z)[Q]) {
    auto each = [&](auto act) {
#pragma unroll
        for (int q = 0; q < Q; ++q) z[q] = activate2<act(), EXACT, SLOPE>(z[q]);
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
struct Div {                 // by multiplication, of numbers below 2^16
    unsigned mul;
    int by;
};
__device__ __forceinline__ int operator/(int n, const Div& d) { return d.by == 1 ? n : (int)__umulhi((unsigned)n, d.mul); }
struct Layout {
    bool fits;               // else the kernels of any size take it
    bool small;              // groups within a warp: lanes of a group, packs of a lane (items)
    bool held;               // in shared memory
    int vec, width, packs;   // elements of a pack; channels and packs of a slab
    int slabs, items, lanes, rounds;   // rounds: rows of a thread
    int ctas, part;          // CTAs of a cluster, positions of each
    int columns;             // CTAs or clusters side by side that share the items of a slab
    int groups;              // of a slab
    int entries, side;       // sums of a group in a row of threads; rows of them that a warp adds up side by side
    Div by_packs, by_lanes, by_cg, by_entries;
    size_t smem;
    // rows of a thread among n positions from its first on
    __device__ __forceinline__ int count(int n) const { return n > 0 ? lanes == 1 ? n : ((n - 1) >> 16) ? (n - 1) / lanes + 1 : (n - 1) / by_lanes + 1 : 0; }
};

// The cluster's CTAs have begun: told at a kernel's start, waited for before the first store to another's shared memory, when the
// loads are on their way
__device__ __forceinline__ void cluster_begin() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_begun() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync_g() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cta_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_id() {
    int r;
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void store_remote(const float* mine, int cta, float v) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(mine);
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
}

// Sums of the CTA's (and the cluster's) groups, NV of them side by side. `v` are a thread's sums of its channels; where a pack lies
// within a group they are one. red holds those of all threads, one row of threads after the other; a warp adds up a
// group, then the CTAs' sums of it are exchanged. parts: [ctas][NV][items * groups], of this call alone. What becomes of a group's
// sum is done once, by the thread that calls finish(which, item * groups + group, sum).
template <int VEC, bool WITHIN, int NV, typename F>
__device__ __forceinline__ void group_sums(const Pair (&v)[NV][kPairs<VEC>], float* red, float* parts, const Layout& L, int rank, F finish)
{
    const int groups = L.groups, all = L.items * groups, rows = L.lanes, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int across = WITHIN ? L.packs : L.width, n = L.entries;   // entries of a row, of a group's row
    const bool mine = (int)threadIdx.x < L.items * rows * L.packs;
#pragma unroll
    for (int w = 0; w < NV; ++w) {
        float* to = red + w * (WITHIN ? kThreads : kThreads * VEC);
        if (mine && WITHIN) {
            Pair t = v[w][0];
#pragma unroll
            for (int q = 1; q < kPairs<VEC>; ++q) t = add2(t, v[w][q]);
            to[threadIdx.x] = both(t);
        } else if (mine) {
#pragma unroll
            for (int q = 0; q < kPairs<VEC>; ++q) {
                float x, y;
                upk2(v[w][q], x, y);
                to[threadIdx.x * VEC + 2 * q] = x;
                if (VEC > 1) to[threadIdx.x * VEC + 2 * q + 1] = y;
            }
        }
    }
    __syncthreads();
    const int side = L.side;                                // rows of a group that a warp has side by side
    const int r0 = n < 32 ? lane / L.by_entries : 0, c0 = lane - r0 * n;
    for (int k = warp; k < NV * all; k += kWarpsG) {
        const int w = NV > 1 && k >= all ? 1 : 0, j = k - w * all, item = L.items > 1 ? j / groups : 0;
        const float* first = red + w * (WITHIN ? kThreads : kThreads * VEC) + item * rows * across + (j - item * groups) * n;
        float s = 0.f;
        if (r0 < side)
            for (int r = r0; r < rows; r += side)
                for (int c = c0; c < n; c += 32) s += first[r * across + c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (L.ctas == 1) {
            if (lane == 0) finish(w, j, s);
        } else if (lane < L.ctas) {
            store_remote(parts + rank * NV * all + k, lane, s);
        }
    }
    if (L.ctas > 1) {
        cluster_sync_g();
        for (int k = threadIdx.x; k < NV * all; k += kThreads) {
            float s = 0.f;
            for (int c = 0; c < L.ctas; ++c) s += parts[c * NV * all + k];
            finish(NV > 1 && k >= all ? 1 : 0, NV > 1 && k >= all ? k - all : k, s);
        }
    }
    __syncthreads();
}
// A thread's channels' entries of a group's [groups]: one for all of them where a pack lies within a group
template <int VEC, bool WITHIN> constexpr int kOf = WITHIN ? 1 : kPairs<VEC>;
template <int VEC, bool WITHIN> __device__ __forceinline__ void of_channels(const float* from, int c0, const Div& cg, Pair (&v)[kOf<VEC, WITHIN>]) {
    if constexpr (WITHIN) {
        const float x = from[c0 / cg];
        v[0] = pk2(x, x);
    } else {
#pragma unroll
        for (int q = 0; q < kPairs<VEC>; ++q) v[q] = pk2(from[(c0 + 2 * q) / cg], VEC > 1 ? from[(c0 + 2 * q + 1) / cg] : 0.f);
    }
}
template <typename T, int VEC, bool WITHIN>
__device__ __forceinline__ void less(const Pack<T, VEC>& v, const Pair (&m)[kOf<VEC, WITHIN>], Pair (&out)[kPairs<VEC>]) {
    if constexpr (WITHIN) {
        float x, y;
        upk2(m[0], x, y);
        plus<T, VEC>(v, -x, out);
    } else {
        minus<T, VEC>(v, m, out);
    }
}

// s + v, channel by channel
template <typename T, int VEC> __device__ __forceinline__ void add_onto(Pair (&s)[kPairs<VEC>], const Pack<T, VEC>& v) {
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) {
        float x, y;
        upk2(s[q], x, y);
        if constexpr (VEC == 1) x += to_f32(v.e[0]);
        else if constexpr (sizeof(T) == 4) x += v.e[2 * q], y += v.e[2 * q + 1];
        else add_pair<T>(x, y, word_of(&v.e[2 * q]));
        s[q] = pk2(x, y);
    }
}
__device__ __forceinline__ void fetch16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
// A thread's rows come in four groups, so that it has begun with the first when the last are still on their way.
constexpr int kBatches = 4;
__device__ __forceinline__ void mark_batch() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <typename F> __device__ __forceinline__ void by_batches(int rounds, F f) {
    const int n = (rounds + kBatches - 1) / kBatches;
    asm volatile("cp.async.wait_group 3;" ::: "memory");
    f(0, n);
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    f(n, 2 * n);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    f(2 * n, 3 * n);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    f(3 * n, rounds);
}

// What a thread has of a round of items: rows [first, first + rounds * lanes) of its batch element, every lanes-th.
struct Place {
    int item, row, pack, b, len, first, last;   // its rows are first + k lanes < last
    long long at;                               // of the first, in elements
    bool on;
    __device__ __forceinline__ Place(const GroupNormParams& p, const Layout& L, int slab, int b0, int rank) {
        const int line = (int)threadIdx.x / L.by_packs;
        pack = threadIdx.x - line * L.packs;
        item = line / L.by_lanes;
        row = line - item * L.lanes;
        b = b0 + item;
        on = item < L.items && b < p.B;
        len = !on ? 0 : p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
        first = rank * L.part + row;
        last = on ? (int)min((long long)p.S, (rank + 1ll) * L.part) : 0;
        at = ((long long)b * p.S + first) * p.C + slab * L.width + pack * L.vec;
    }
};

// The slab's weights in shared memory, as fp32: [width] of either
__device__ __forceinline__ void take_weights(float* to, const GroupNormParams& p, const Layout& L, int slab) {
    for (int c = threadIdx.x; c < L.width; c += kThreads) {
        to[c] = wval(p.weight, slab * L.width + c, p.wdtype, 1.f);
        to[L.width + c] = wval(p.bias, slab * L.width + c, p.wdtype, 0.f);
    }
}
// VEC weights, all on their way at once
template <int VEC> __device__ __forceinline__ void read_weights(const void* p, int c, int wdtype, float none, float (&v)[VEC]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = none;
    } else if (wdtype == SDTW_F32) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = static_cast<const float*>(p)[c + e];
    } else if (wdtype == SDTW_BF16) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = to_f32(static_cast<const __nv_bfloat16*>(p)[c + e]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = to_f32(static_cast<const __half*>(p)[c + e]);
    }
}
__device__ __forceinline__ float length_of(const GroupNormParams& p, int b) {
    return (float)(b >= p.B ? 0 : p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S);
}
template <int VEC> __device__ __forceinline__ void read_floats(const float* from, Pair (&v)[kPairs<VEC>]) {
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) v[q] = VEC > 1 ? *reinterpret_cast<const Pair*>(from + 2 * q) : pk2(from[0], 0.f);
}

template <typename T, int VEC, bool HELD, bool WITHIN> __global__ void __launch_bounds__(kThreads, 3) group_fwd_kernel(const GroupNormParams p, const Layout L)
{
    extern __shared__ __align__(16) unsigned char held[];   // [rounds][kThreads] packs, then the weights and the sums
    using P = Pack<T, VEC>;
    constexpr int Q = kPairs<VEC>, AHEAD = HELD ? 4 : 8;
    const int slab = blockIdx.y, rank = L.ctas > 1 ? cta_rank() : 0, column = L.ctas > 1 ? cluster_id() : blockIdx.x;
    const int groups = L.groups, all = L.items * groups;
    float* weights = reinterpret_cast<float*>(held + (HELD ? (size_t)L.rounds * kThreads * 16 : 0));
    float* red = weights + 2 * L.width;
    float* stats = red + kThreads * VEC;                    // mean, 1 / deviation
    float* parts = stats + 2 * all;
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.y);
    if (L.ctas > 1) cluster_begin();
    take_weights(weights, p, L, slab);
    const long long step = (long long)L.lanes * p.C;
    const int c0 = ((int)threadIdx.x - (int)threadIdx.x / L.by_packs * L.packs) * VEC;
    for (int b0 = column * L.items; b0 < p.B; b0 += L.columns * L.items) {
        const Place at(p, L, slab, b0, rank);
        const int there = min(at.last, at.len);             // rows that take part
        P* mine = reinterpret_cast<P*>(held) + threadIdx.x;
        const T* src = x + at.at;
        auto value = [&](int k) { return HELD ? mine[k * kThreads] : *reinterpret_cast<const P*>(src + k * step); };
        const int rounds = L.count(there - at.first), last = L.count(at.last - at.first);   // of this thread
        if constexpr (HELD) {
            const int n = (rounds + kBatches - 1) / kBatches;
            for (int g = 0, k = 0; g < kBatches; ++g) {
#pragma unroll 4
                for (; k < min(rounds, (g + 1) * n); ++k) fetch16(mine + k * kThreads, src + k * step);
                mark_batch();
            }
        }
        Pair s[1][Q], mu[kOf<VEC, WITHIN>], rw[Q], bias[Q], d[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) s[0][q] = pk2(0.f, 0.f);
        mu[0] = pk2(0.f, 0.f);
        auto add = [&](int from, int to) {
            to = min(to, rounds);
#pragma unroll AHEAD
            for (int k = from; k < to; ++k) add_onto<T, VEC>(s[0], value(k));
        };
        if constexpr (HELD) by_batches(rounds, add);
        else add(0, rounds);
        if (L.ctas > 1) cluster_begun();                    // a cluster has one batch element
        auto count = [&](int k) { return length_of(p, L.items > 1 ? b0 + k / groups : b0) * (float)p.cg; };
        group_sums<VEC, WITHIN, 1>(s, red, parts, L, rank, [&](int, int k, float sum) { stats[k] = count(k) > 0.f ? sum / count(k) : 0.f; });
        const float* mine_stats = stats + (at.item < L.items ? at.item * groups : 0);
        of_channels<VEC, WITHIN>(mine_stats, c0, L.by_cg, mu);
#pragma unroll
        for (int q = 0; q < Q; ++q) s[0][q] = pk2(0.f, 0.f);
#pragma unroll AHEAD
        for (int k = 0; k < rounds; ++k) {
            less<T, VEC, WITHIN>(value(k), mu, d);
#pragma unroll
            for (int q = 0; q < Q; ++q) s[0][q] = fma2(d[q], d[q], s[0][q]);
        }
        group_sums<VEC, WITHIN, 1>(s, red, parts + L.ctas * all, L, rank, [&](int, int k, float sum) {
            const float r = count(k) > 0.f ? 1.f / sqrtf(sum / count(k) + p.eps) : 0.f;
            stats[all + k] = r;
            if (p.mean && rank == 0 && b0 + k / groups < p.B) {
                const long long to = (long long)(b0 + k / groups) * p.G + slab * groups + k % groups;
                p.mean[to] = stats[k], p.rstd[to] = r;
            }
        });
        read_floats<VEC>(weights + c0, rw);
        read_floats<VEC>(weights + L.width + c0, bias);
        Pair r[kOf<VEC, WITHIN>];
        of_channels<VEC, WITHIN>(mine_stats + all, c0, L.by_cg, r);
#pragma unroll
        for (int q = 0; q < Q; ++q) rw[q] = mul2(rw[q], r[WITHIN ? 0 : q]);
        T* dst = y + at.at;
        auto put = [&](int k, const P& v) {
            Pair z[Q];
            less<T, VEC, WITHIN>(v, mu, z);
#pragma unroll
            for (int q = 0; q < Q; ++q) z[q] = fma2(z[q], rw[q], bias[q]);
            activate_all<sizeof(T) == 4, false, Q>(p.activation, z);
            *reinterpret_cast<P*>(dst + k * step) = rounded<T, VEC>(z);
        };
        int first = 0;
        if constexpr (!HELD) {   // rows that are read again come four at a time (2 x 8192 x 512 fp32: 28 us, one by one 38)
            for (; first + 4 <= rounds; first += 4) {
                P v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = value(first + i);
#pragma unroll
                for (int i = 0; i < 4; ++i) put(first + i, v[i]);
            }
        }
#pragma unroll 4
        for (int k = first; k < rounds; ++k) put(k, value(k));
#pragma unroll
        for (int q = 0; q < Q; ++q) d[q] = pk2(0.f, 0.f);
        for (int k = rounds; k < last; ++k) *reinterpret_cast<P*>(dst + k * step) = rounded<T, VEC>(d);
    }
}

template <typename T, int VEC, bool HELD, bool WITHIN> __global__ void __launch_bounds__(kThreads, WITHIN ? 3 : 2) group_bwd_kernel(const GroupNormParams p, const Layout L)
{
    extern __shared__ __align__(16) unsigned char held[];   // [rounds][x, dy][kThreads] packs, then the weights and the sums
    using P = Pack<T, VEC>;
    constexpr int Q = kPairs<VEC>, AHEAD = HELD ? 1 : 4;     // rows that come from memory at a time
    const int slab = blockIdx.y, rank = L.ctas > 1 ? cta_rank() : 0, column = L.ctas > 1 ? cluster_id() : blockIdx.x;
    const int groups = L.groups, all = L.items * groups;
    float* weights = reinterpret_cast<float*>(held + (HELD ? (size_t)L.rounds * 2 * kThreads * 16 : 0));
    float* red = weights + 2 * L.width;
    float* stats = red + (WITHIN && VEC > 1 ? 1 : 2) * kThreads * VEC;   // mean g, mean g xh
    float* parts = stats + 2 * all;
    const T *x = static_cast<const T*>(p.x), *dy = static_cast<const T*>(p.dy);
    T* dx = static_cast<T*>(p.dx);
    if (L.ctas > 1) cluster_begin();
    take_weights(weights, p, L, slab);
    __syncthreads();
    const long long step = (long long)L.lanes * p.C;
    const int c0 = ((int)threadIdx.x - (int)threadIdx.x / L.by_packs * L.packs) * VEC;
    Pair w[Q], bias[Q], sum[2][Q];                          // of the weights' gradients
    read_floats<VEC>(weights + c0, w);
    read_floats<VEC>(weights + L.width + c0, bias);
#pragma unroll
    for (int q = 0; q < Q; ++q) sum[0][q] = sum[1][q] = pk2(0.f, 0.f);
    int turn = 0;
    for (int b0 = column * L.items; b0 < p.B; b0 += L.columns * L.items, turn ^= 1) {
        const Place at(p, L, slab, b0, rank);
        const int there = min(at.last, at.len);
        P* mine = reinterpret_cast<P*>(held) + threadIdx.x;
        const T *sx = x + at.at, *sd = dy + at.at;
        auto value = [&](int k, int which) {
            return HELD ? mine[(2 * k + which) * kThreads] : *reinterpret_cast<const P*>((which ? sd : sx) + k * step);
        };
        const int rounds = L.count(there - at.first), last = L.count(at.last - at.first);
        if constexpr (HELD) {
            const int n = (rounds + kBatches - 1) / kBatches;
            for (int g = 0, k = 0; g < kBatches; ++g) {
#pragma unroll 2
                for (; k < min(rounds, (g + 1) * n); ++k) {
                    fetch16(mine + 2 * k * kThreads, sx + k * step);
                    fetch16(mine + (2 * k + 1) * kThreads, sd + k * step);
                }
                mark_batch();
            }
        }
        Pair mu[kOf<VEC, WITHIN>], r[kOf<VEC, WITHIN>], s[2][Q];
        const long long from = (long long)(at.on ? at.b : 0) * p.G + slab * groups;
        of_channels<VEC, WITHIN>(p.mean + from, c0, L.by_cg, mu);
        of_channels<VEC, WITHIN>(p.rstd + from, c0, L.by_cg, r);
        // xh and dz of a pack
        auto values = [&](const P& vx, const P& vd, Pair (&xh)[Q], Pair (&dz)[Q]) {
            Pair z[Q];
            less<T, VEC, WITHIN>(vx, mu, xh);
            plus<T, VEC>(vd, 0.f, dz);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                xh[q] = mul2(xh[q], r[WITHIN ? 0 : q]);
                z[q] = fma2(xh[q], w[q], bias[q]);
            }
            activate_all<sizeof(T) == 4, true, Q>(p.activation, z);
#pragma unroll
            for (int q = 0; q < Q; ++q) dz[q] = mul2(dz[q], z[q]);
        };
#pragma unroll
        for (int q = 0; q < Q; ++q) s[0][q] = s[1][q] = pk2(0.f, 0.f);
        auto add = [&](int from, int to) {
            to = min(to, rounds);
            auto take = [&](const P& vx, const P& vd) {
                Pair xh[Q], dz[Q];
                values(vx, vd, xh, dz);
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    s[0][q] = add2(s[0][q], dz[q]);
                    s[1][q] = fma2(dz[q], xh[q], s[1][q]);
                }
            };
            if constexpr (AHEAD > 1) {
                for (; from + AHEAD <= to; from += AHEAD) {
                    P vx[AHEAD], vd[AHEAD];
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) vx[i] = value(from + i, 0), vd[i] = value(from + i, 1);
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) take(vx[i], vd[i]);
                }
            }
#pragma unroll 2
            for (int k = from; k < to; ++k) take(value(k, 0), value(k, 1));
        };
        if constexpr (HELD) by_batches(rounds, add);
        else add(0, rounds);
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int k = 0; k < 2; ++k) sum[k][q] = add2(sum[k][q], s[k][q]), s[k][q] = mul2(s[k][q], w[q]);
        if (L.ctas > 1) cluster_begun();                    // a cluster has one batch element
        if (!dx) continue;
        group_sums<VEC, WITHIN, 2>(s, red, parts + 2 * turn * L.ctas * all, L, rank, [&](int which, int k, float t) {
            const float n = length_of(p, L.items > 1 ? b0 + k / groups : b0) * (float)p.cg;
            stats[which * all + k] = n > 0.f ? t / n : 0.f;
        });
        const float* mine_stats = stats + (at.item < L.items ? at.item * groups : 0);
        Pair m1[kOf<VEC, WITHIN>], m2[kOf<VEC, WITHIN>];
        of_channels<VEC, WITHIN>(mine_stats, c0, L.by_cg, m1);
        of_channels<VEC, WITHIN>(mine_stats + all, c0, L.by_cg, m2);
        T* dst = dx + at.at;
        auto put = [&](int k, const P& vx, const P& vd) {
            Pair xh[Q], dz[Q];
            values(vx, vd, xh, dz);
#pragma unroll
            for (int q = 0; q < Q; ++q) dz[q] = mul2(r[WITHIN ? 0 : q], sub2(sub2(mul2(dz[q], w[q]), m1[WITHIN ? 0 : q]), mul2(xh[q], m2[WITHIN ? 0 : q])));
            *reinterpret_cast<P*>(dst + k * step) = rounded<T, VEC>(dz);
        };
        int first = 0;
        if constexpr (AHEAD > 1) {
            for (; first + AHEAD <= rounds; first += AHEAD) {
                P vx[AHEAD], vd[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) vx[i] = value(first + i, 0), vd[i] = value(first + i, 1);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) put(first + i, vx[i], vd[i]);
            }
        }
#pragma unroll 2
        for (int k = first; k < rounds; ++k) put(k, value(k, 0), value(k, 1));
        Pair none[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) none[q] = pk2(0.f, 0.f);
        for (int k = rounds; k < last; ++k) *reinterpret_cast<P*>(dst + k * step) = rounded<T, VEC>(none);
    }
    if (!p.partial) return;
    // the threads of a pack, one after the other
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float u, v;
            upk2(sum[1 - which][q], u, v);
            red[threadIdx.x * VEC + 2 * q] = u;
            if (VEC > 1) red[threadIdx.x * VEC + 2 * q + 1] = v;
        }
        __syncthreads();
        float* out = p.partial + (((long long)column * L.ctas + rank) * 2 + which) * p.C + slab * L.width;
        for (int c = threadIdx.x; c < L.width; c += kThreads) {
            float s = 0.f;
            for (int k = 0; k < L.items * L.lanes; ++k) s += red[k * L.width + c];
            out[c] = s;
        }
    }
}

// ---- groups of a few positions (normalising row by row): a group is `lanes` lanes of a warp, at most two packs each, whose
// sums need no barrier (65535 rows of 1024 by groups of 128 bf16: 70 us forward and 97 backward, as slabs 486 and 458; 16 rows of
// 512 forward: 3.1 and 4.2). A thread's group and channels stay the same over the batch elements that it takes, every
// columns-th; the coming ones' packs are on their way to shared memory meanwhile, a thread's to places of its own.
__device__ __forceinline__ float lane_sum(float v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// 1 / sqrt(v); for results of 16 bits by the approximation, within 2^-22
template <bool EXACT> __device__ __forceinline__ float rsqrt_of(float v) { return EXACT ? 1.f / sqrtf(v) : rsqrtf(v); }
constexpr int kSmallPacks = 2, kAhead = 3;

template <typename T, int VEC, int K, bool BWD> __global__ void __launch_bounds__(kThreads, (BWD ? 2 : 4) / K) group_small_kernel(const GroupNormParams p, const Layout L)
{
    using P = Pack<T, VEC>;
    constexpr int Q = kPairs<VEC>;
    const long long id = ((long long)blockIdx.x * kThreads + threadIdx.x) / L.lanes;
    const int lane = threadIdx.x % L.lanes, g = (int)(id % p.G), per = p.cg / VEC, packs = p.S * per;
    const int column = (int)(id / p.G), end = column < L.columns ? p.B : 0;   // the last CTA's threads may be too many
    const T *x = static_cast<const T*>(p.x), *dy = static_cast<const T*>(p.dy);
    T* out = static_cast<T*>(BWD ? p.dx : p.y);
    int row[K], c[K];
    Pair w[K][Q], bias[K][Q], dw[K][Q] = {}, db[K][Q] = {};
    bool has[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int q = lane + k * L.lanes;
        has[k] = q < packs;
        row[k] = has[k] ? q / per : 0;
        c[k] = g * p.cg + (has[k] ? q % per * VEC : 0);
        float t[VEC];
        read_weights<VEC>(p.weight, c[k], p.wdtype, 1.f, t);
        pairs_of<VEC>(t, w[k]);
        read_weights<VEC>(p.bias, c[k], p.wdtype, 0.f, t);
        pairs_of<VEC>(t, bias[k]);
    }
    auto length = [&](int b) { return b < end ? p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S : 0; };
    // [kAhead + 1][K][x, dy][kThreads] packs, and after them [kAhead + 1][mean, rstd][kThreads]
    extern __shared__ __align__(16) unsigned char held[];
    constexpr int N = BWD ? 2 : 1;
    float* stat = reinterpret_cast<float*>(held + (kAhead + 1) * K * N * kThreads * 16);
    auto slot = [&](int stage, int k, int which) { return reinterpret_cast<P*>(held) + ((stage * K + k) * N + which) * kThreads + threadIdx.x; };
    // places of the batch element to send for, and of the one in work
    const long long step = (long long)L.columns * p.S * p.C, element = (long long)p.S * p.C;
    long long ahead = column * element, here = ahead, stats = column * p.G + g;
    int place[K];
#pragma unroll
    for (int k = 0; k < K; ++k) place[k] = row[k] * p.C + c[k];
    int sent = column;
    auto send = [&](int stage) {
        const int len = length(sent);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (has[k] && row[k] < len) {
                fetch16(slot(stage, k, 0), x + ahead + place[k]);
                if (BWD) fetch16(slot(stage, k, N - 1), dy + ahead + place[k]);
            }
        if (BWD && len > 0) {
            fetch4(stat + 2 * stage * kThreads + threadIdx.x, p.mean + (long long)sent * p.G + g);
            fetch4(stat + (2 * stage + 1) * kThreads + threadIdx.x, p.rstd + (long long)sent * p.G + g);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ahead += step, sent += L.columns;
    };
    for (int k = 0; k < kAhead; ++k) send(k);
    int stage = 0;
    const float full = 1.f / ((float)p.S * (float)p.cg);
    // every lane of a warp makes the same number of rounds: the sums are collective
    const int most = (p.B + L.columns - 1) / L.columns;
    for (int b = column, turn = 0; turn < most; ++turn, b += L.columns, here += step, stats += (long long)L.columns * p.G) {
        const int len = length(b);
        Pair v[K][Q], d[K][Q], s1 = pk2(0.f, 0.f), s2 = s1;
        bool in[K];
        const float inv = len == p.S ? full : len ? 1.f / ((float)len * (float)p.cg) : 0.f;
        send(stage == 0 ? kAhead : stage - 1);   // where the last round's were
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
#pragma unroll
        for (int k = 0; k < K; ++k) {
            in[k] = has[k] && row[k] < len;
            if (in[k]) {
                plus<T, VEC>(*slot(stage, k, 0), 0.f, v[k]);
                if (BWD) plus<T, VEC>(*slot(stage, k, N - 1), 0.f, d[k]);
            }
        }
        float mu = 0.f, r = 0.f;
        if (BWD && len > 0) mu = stat[2 * stage * kThreads + threadIdx.x], r = stat[(2 * stage + 1) * kThreads + threadIdx.x];
        stage = stage == kAhead ? 0 : stage + 1;
        if constexpr (!BWD) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in[k]) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) s1 = add2(s1, v[k][q]);
                }
            mu = lane_sum(both(s1), L.lanes) * inv;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in[k]) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        v[k][q] = sub2(v[k][q], pk2(mu, mu));
                        s2 = fma2(v[k][q], v[k][q], s2);
                    }
                }
            r = len ? rsqrt_of<sizeof(T) == 4>(lane_sum(both(s2), L.lanes) * inv + p.eps) : 0.f;
            if (p.mean && lane == 0 && b < end) p.mean[stats] = mu, p.rstd[stats] = r;
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in[k]) {
                    Pair z[Q];
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        v[k][q] = mul2(sub2(v[k][q], pk2(mu, mu)), pk2(r, r));
                        z[q] = fma2(v[k][q], w[k][q], bias[k][q]);
                    }
                    activate_all<sizeof(T) == 4, true, Q>(p.activation, z);
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        d[k][q] = mul2(d[k][q], z[q]);
                        db[k][q] = add2(db[k][q], d[k][q]);
                        dw[k][q] = fma2(d[k][q], v[k][q], dw[k][q]);
                        d[k][q] = mul2(d[k][q], w[k][q]);
                        s1 = add2(s1, d[k][q]);
                        s2 = fma2(d[k][q], v[k][q], s2);
                    }
                }
            const float m1 = lane_sum(both(s1), L.lanes) * inv, m2 = lane_sum(both(s2), L.lanes) * inv;
            s1 = pk2(m1, m1), s2 = pk2(m2, m2);
        }
        if (out && b < end) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (has[k]) {
                    if (!in[k]) {
#pragma unroll
                        for (int q = 0; q < Q; ++q) v[k][q] = pk2(0.f, 0.f);
                    } else if constexpr (BWD) {
#pragma unroll
                        for (int q = 0; q < Q; ++q) v[k][q] = mul2(pk2(r, r), sub2(sub2(d[k][q], s1), mul2(v[k][q], s2)));
                    } else {
#pragma unroll
                        for (int q = 0; q < Q; ++q) v[k][q] = fma2(mul2(v[k][q], pk2(r, r)), w[k][q], bias[k][q]);
                        activate_all<sizeof(T) == 4, false, Q>(p.activation, v[k]);
                    }
                    *reinterpret_cast<P*>(out + here + place[k]) = rounded<T, VEC>(v[k]);
                }
        }
    }
    if (BWD && p.partial && column < L.columns) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (has[k]) {
                float* to = p.partial + 2 * ((long long)column * p.S + row[k]) * p.C + c[k];
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    float u, v;
                    upk2(dw[k][q], u, v);
                    to[2 * q] = u, to[2 * q + 1] = v;
                    upk2(db[k][q], u, v);
                    to[p.C + 2 * q] = u, to[p.C + 2 * q + 1] = v;
                }
            }
    }
}

// ---- groups too wide for the above: a CTA a group of a batch element, a thread a channel
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
// A thread's sums are long here, and carry what their additions leave (Kahan).
struct Sum {
    float s = 0.f, left = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float y = v - left, t = s + y;
        left = (t - s) - y;
        s = t;
    }
};
template <typename T> __global__ void __launch_bounds__(kThreads) group_fwd_any_kernel(const GroupNormParams p)
{
    __shared__ float red[kThreads / 32];
    const int b = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
    const long long base = (long long)b * p.S * p.C + (long long)g * p.cg;
    const T* x = static_cast<const T*>(p.x) + base;
    T* y = static_cast<T*>(p.y) + base;
    const float n = (float)len * (float)p.cg;
    Sum s, q;
    for (int i = 0; i < len; ++i)
        for (int c = threadIdx.x; c < p.cg; c += kThreads) s.add(to_f32(x[(long long)i * p.C + c]));
    const float mu = len ? block_sum(s.s, red) / n : 0.f;
    for (int i = 0; i < len; ++i)
        for (int c = threadIdx.x; c < p.cg; c += kThreads) {
            const float d = to_f32(x[(long long)i * p.C + c]) - mu;
            q.add(d * d);
        }
    const float r = len ? 1.f / sqrtf(block_sum(q.s, red) / n + p.eps) : 0.f;
    for (int c = threadIdx.x; c < p.cg; c += kThreads) {
        const float w = r * wval(p.weight, g * p.cg + c, p.wdtype, 1.f), bias = wval(p.bias, g * p.cg + c, p.wdtype, 0.f);
        for (int i = 0; i < p.S; ++i) {
            float none;
            const long long at = (long long)i * p.C + c;
            y[at] = from_f32<T>(i < len ? activate_as<sizeof(T) == 4, false>(p.activation, fmaf(to_f32(x[at]) - mu, w, bias), none) : 0.f);
        }
    }
    if (threadIdx.x == 0 && p.mean) p.mean[blockIdx.x] = mu, p.rstd[blockIdx.x] = r;
}

template <typename T> __global__ void __launch_bounds__(kThreads) group_bwd_any_kernel(const GroupNormParams p)
{
    __shared__ float red[kThreads / 32];
    const int b = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
    const long long base = (long long)b * p.S * p.C + (long long)g * p.cg;
    const T* x = static_cast<const T*>(p.x) + base;
    const T* dy = static_cast<const T*>(p.dy) + base;
    const float mu = p.mean[blockIdx.x], r = p.rstd[blockIdx.x], n = (float)len * (float)p.cg;
    auto value = [&](long long at, float w, float bias, float& xh) {
        float slope;
        xh = (to_f32(x[at]) - mu) * r;
        activate_as<sizeof(T) == 4, true>(p.activation, fmaf(xh, w, bias), slope);
        return to_f32(dy[at]) * slope;
    };
    Sum t1, t2;
    float xh;
    for (int c = threadIdx.x; c < p.cg; c += kThreads) {
        const int channel = g * p.cg + c;
        const float w = wval(p.weight, channel, p.wdtype, 1.f), bias = wval(p.bias, channel, p.wdtype, 0.f);
        Sum dw, db;
        for (int i = 0; i < len; ++i) {
            const float dz = value((long long)i * p.C + c, w, bias, xh);
            db.add(dz);
            dw.add(dz * xh);
        }
        t1.add(db.s * w);
        t2.add(dw.s * w);
        if (p.partial) p.partial[2ll * b * p.C + channel] = dw.s, p.partial[(2ll * b + 1) * p.C + channel] = db.s;
    }
    if (!p.dx) return;
    const float s1 = block_sum(t1.s, red) / n, s2 = block_sum(t2.s, red) / n;
    T* dx = static_cast<T*>(p.dx) + base;
    for (int c = threadIdx.x; c < p.cg; c += kThreads) {
        const float w = wval(p.weight, g * p.cg + c, p.wdtype, 1.f), bias = wval(p.bias, g * p.cg + c, p.wdtype, 0.f);
        for (int i = 0; i < p.S; ++i) {
            const long long at = (long long)i * p.C + c;
            dx[at] = from_f32<T>(0.f);
            if (i < len) {
                const float dz = value(at, w, bias, xh);
                dx[at] = from_f32<T>(r * (dz * w - s1 - xh * s2));
            }
        }
    }
}

// dw, db: the partial rows added in a fixed order, 32 columns by 32 row lanes
__global__ void __launch_bounds__(1024) group_fold_kernel(const GroupNormParams p, long long rows)
{
    __shared__ float part[32][33];
    after_previous();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    float s[4] = {};
    if (c < p.C)
        for (long long t = lane; t < rows; t += 128) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (t + 32 * q < rows) s[q] += p.partial[(2 * (t + 32 * q) + blockIdx.y) * p.C + c];
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

constexpr size_t kSlabBytes = 220 * 1024;   // of a CTA's shared memory

Div div_by(int d) { return Div{(unsigned)((0x100000000ull + d - 1) / d), d}; }   // of 1: not multiplied by

long long gcd(long long a, long long b) { return b ? gcd(b, a % b) : a; }

// Both alignments' layouts are asked for by the size of the workspace, which so does not depend on addresses.
Layout layout(const GroupNormParams& p, bool backward, bool packs, int sms)
{
    Layout L{};
    const int size = dtype_size(p.dtype);
    L.vec = packs && p.C % (16 / size) == 0 ? 16 / size : 1;
    if (L.vec > 1 && p.cg % L.vec == 0 && (long long)p.S * (p.cg / L.vec) <= 32 * kSmallPacks) {
        const int packs = p.S * (p.cg / L.vec);
        L.small = L.fits = true;
        L.lanes = 1;
        while (L.lanes < 32 && L.lanes < packs) L.lanes *= 2;
        L.items = packs > 32 ? 2 : 1;
        // as many columns as fill the SMs
        const long long most = std::max(1ll, (long long)sms * (backward ? 2 : 4) / L.items * kThreads / L.lanes / p.G);
        L.columns = (int)std::min<long long>(most, p.B);
        return L;
    }
    const long long whole = p.cg / gcd(p.cg, L.vec) * L.vec;    // channels of whole groups and whole packs
    L.width = (int)whole;
    // at least 64 bytes a row, or all channels: wider slabs take larger clusters (128 bytes: backward of 16 x 4096 x 512 bf16
    // 98 us for 88), rows of 32 bytes 96
    for (long long j = 1; whole * j <= std::min(p.C, kThreads * L.vec) && L.width * size < 64; ++j)
        if (p.C % (whole * j) == 0) L.width = (int)(whole * j);
    L.packs = L.width / L.vec;
    if (L.packs > kThreads) return L;
    L.slabs = p.C / L.width;
    if (L.slabs > 65535) return L;
    L.fits = true;
    const int most = kThreads / L.packs;
    L.lanes = std::min(most, p.S);
    L.items = std::min(most / L.lanes, p.B);
    // few items are spread over the SMs
    while (L.items > 1 && (long long)((p.B + L.items - 1) / L.items) * L.slabs < sms) L.items = (L.items + 1) / 2;
    const int arrays = backward ? 2 : 1;
    const bool one = p.cg % L.vec == 0 && L.vec > 1;             // sum of a thread for each of a group's
    const size_t sums = (2 * (size_t)L.width + (size_t)(one ? 1 : arrays) * kThreads * L.vec + 2 * L.items * (L.width / p.cg)) * sizeof(float);
    auto bytes = [&](int ctas) {
        const size_t exchange = ctas > 1 ? (size_t)4 * ctas * (L.width / p.cg) * sizeof(float) : 0;
        const long long rounds = ((p.S - 1ll + ctas) / ctas + L.lanes - 1) / L.lanes;
        return std::pair<size_t, long long>(sums + exchange, rounds * kThreads * 16 * arrays);
    };
    // CTAs of a cluster: until three fit on an SM side by side, or, where there are fewer than two an SM, until a thread has
    // eight rows: a cluster's exchanges take some 2 us (16 x 4096 x 512 bf16 with 1, 2, 4, 8 and 16 CTAs: forward 69, 61,
    // 43, 59 and 107 us, of which this takes 4; backward 118, 112, 123, 85 and 140, of which it takes 8). Two an SM are enough for eight
    // CTAs, as sixteen cost more (16 x 5000 x 512: backward 113 us, with sixteen 156; 16 x 12000: forward 121 and 149).
    // What the CTAs exchange has to fit: up to 64 KB for 16 CTAs and 256 groups, but a slab that is all of 2008 channels, each its own group,
    // takes 32 KB for every CTA.
    L.ctas = 1;
    const long long clusters = (long long)((p.B + L.items - 1) / L.items) * L.slabs;
    while (L.ctas < kMostCtas && L.items == 1 && (p.S + 2ll * L.ctas - 1) / (2 * L.ctas) >= 2 * L.lanes && bytes(2 * L.ctas).first <= kSlabBytes &&
           ((long long)bytes(L.ctas).first + bytes(L.ctas).second > (L.ctas == 8 ? 112 : 75) * 1024 ||
            (clusters * L.ctas < 2 * sms && p.S >= 16ll * L.ctas * L.lanes)))
        L.ctas *= 2;
    const auto need = bytes(L.ctas);
    L.part = (int)((p.S - 1ll + L.ctas) / L.ctas);
    L.rounds = (int)((L.part + L.lanes - 1ll) / L.lanes);
    L.held = L.vec > 1 && (long long)need.first + need.second <= (long long)kSlabBytes;
    L.smem = need.first + (L.held ? (size_t)need.second : 0);
    L.groups = L.width / p.cg;
    L.entries = p.cg % L.vec == 0 ? p.cg / L.vec : p.cg;
    L.side = L.entries < 32 ? 32 / L.entries : 1;
    L.by_packs = div_by(L.packs), L.by_lanes = div_by(L.lanes), L.by_cg = div_by(p.cg), L.by_entries = div_by(L.entries);
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
    c.gridDim = dim3((unsigned)(L.columns * L.ctas), (unsigned)L.slabs), c.blockDim = dim3(kThreads), c.stream = s, c.attrs = &at;
    c.numAttrs = L.ctas > 1 ? 1 : 0, c.dynamicSmemBytes = L.smem;
    return cudaLaunchKernelEx(&c, Kernel, p, L);
}

bool packs(const GroupNormParams& p) { return aligned16(p.x) && aligned16(p.y) && aligned16(p.dy) && aligned16(p.dx); }
long long partial_rows(const GroupNormParams& p, const Layout& L) { return L.small ? (long long)L.columns * p.S : L.fits ? L.columns * L.ctas : p.B; }
template <typename T, int VEC, bool BWD> cudaError_t run_small(const GroupNormParams& p, const Layout& L, cudaStream_t s)
{
    const unsigned grid = (unsigned)(((long long)L.columns * p.G * L.lanes + kThreads - 1) / kThreads);
    auto go = [&](auto k) {
        constexpr size_t smem = (kAhead + 1) * kThreads * (k() * 16 + 4) * (BWD ? 2 : 1);
        const cudaError_t e = allow_smem<group_small_kernel<T, VEC, k(), BWD>>(smem);
        if (e != cudaSuccess) return e;
        group_small_kernel<T, VEC, k(), BWD><<<grid, kThreads, smem, s>>>(p, L);
        return cudaGetLastError();
    };
    return L.items == 1 ? go(std::integral_constant<int, 1>()) : go(std::integral_constant<int, 2>());
}

}  // namespace

size_t group_norm_workspace(const GroupNormParams& p, bool backward, int sms)
{
    if (!backward) return 0;
    const long long rows = std::max(partial_rows(p, layout(p, true, true, sms)), partial_rows(p, layout(p, true, false, sms)));
    return sizeof(float) * 2 * (size_t)rows * p.C;
}

cudaError_t launch_group_norm_forward(const GroupNormParams& p, int sms, cudaStream_t s)
{
    const Layout L = layout(p, false, packs(p), sms);
    return with_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int VEC = 16 / sizeof(T);
        if (L.small) return run_small<T, VEC, false>(p, L, s);
        const bool within = p.cg % L.vec == 0;
        if (L.fits && L.vec == 1) return launch<group_fwd_kernel<T, 1, false, true>>(p, L, s);
        if (L.fits && L.held) return within ? launch<group_fwd_kernel<T, VEC, true, true>>(p, L, s) : launch<group_fwd_kernel<T, VEC, true, false>>(p, L, s);
        if (L.fits) return within ? launch<group_fwd_kernel<T, VEC, false, true>>(p, L, s) : launch<group_fwd_kernel<T, VEC, false, false>>(p, L, s);
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
        if (L.small) return run_small<T, VEC, true>(p, L, s);
        const bool within = p.cg % L.vec == 0;
        if (L.fits && L.vec == 1) return launch<group_bwd_kernel<T, 1, false, true>>(p, L, s);
        if (L.fits && L.held) return within ? launch<group_bwd_kernel<T, VEC, true, true>>(p, L, s) : launch<group_bwd_kernel<T, VEC, true, false>>(p, L, s);
        if (L.fits) return within ? launch<group_bwd_kernel<T, VEC, false, true>>(p, L, s) : launch<group_bwd_kernel<T, VEC, false, false>>(p, L, s);
        group_bwd_any_kernel<T><<<p.B * p.G, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !p.partial) return e;
    return launch_behind(group_fold_kernel, dim3((p.C + 31) / 32, 2), 1024, s, p, partial_rows(p, L));
}

}  // namespace sdtw
