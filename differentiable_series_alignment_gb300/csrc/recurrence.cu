// recurrence.cu -- a gated linear recurrence along a series, forward and backward.
//
//   a_t = sigmoid(gate_t), h_t = a_t h_{t-1} + (1 - a_t) x_t (tied) or a_t h_{t-1} + x_t
//   e_t = dh_t + r_{t+1}, r_t = a_t e_t, dx_t = (1 - a_t) e_t or e_t, dgate_t = e_t (h_{t-1} - x_t or h_{t-1}) a_t (1 - a_t)
//
// Steps h -> a h + u compose: the steps of a run of positions are one pair (A, H), h -> A h + H, and those of the
// gradient one pair (A, R) with the same A. A warp has a run of ROWS positions of 32 lanes' channels, a lane two of
// them (one where sizes are odd): it loads its run into registers and composes it, the CTA's warps and then the CTAs of a cluster
// exchange their pairs through shared memory, and each goes over its run again from the state before it. A cluster so takes
// CTAs x warps x ROWS positions at a time, and carries the state to the next. The order of all sums is fixed by the sizes:
// the same bits every time. The backward pass computes the states again from those that the forward pass kept, one in
// SDTW_RECURRENCE_STEP positions: 3 reads and 2 writes where stored states would be another read.
#include "activation.cuh"
#include "block.h"
#include "packed.cuh"

#include <type_traits>

namespace sdtw {
namespace {

constexpr int kStep = SDTW_RECURRENCE_STEP;
constexpr int kWarps = 8, kMostCtas = 8;   // of a CTA; of a cluster
using Pair = unsigned long long;           // two channels' fp32 values

__device__ __forceinline__ Pair pair(float v) { return pk2(v, v); }

// VEC elements as they lie in memory, in a register that nothing looks into before all of a run's loads are on their way
template <typename T, int VEC> struct Raw {
    using type = uint32_t;
};
template <> struct Raw<float, 2> {
    using type = Pair;
};
// what gives a = 1 and b = 0, and 0
template <typename T> __device__ __forceinline__ uint32_t open_bits() {
    return sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
}
__device__ __forceinline__ void set_raw(uint32_t& r, uint32_t v) { r = v; }
__device__ __forceinline__ void set_raw(Pair& r, uint32_t v) { r = (Pair)v << 32 | v; }
template <typename T, int VEC> __device__ __forceinline__ void load(typename Raw<T, VEC>::type& r, const T* p) {
    if constexpr (sizeof(T) * VEC == 8) asm volatile("ld.global.b64 %0, [%1];" : "=l"(r) : "l"(p));
    else if constexpr (sizeof(T) * VEC == 4) asm volatile("ld.global.b32 %0, [%1];" : "=r"(r) : "l"(p));
    else asm volatile("ld.global.u16 %0, [%1];" : "=r"(r) : "l"(p));
}
template <typename T, int VEC> __device__ __forceinline__ void load_if(typename Raw<T, VEC>::type& r, const T* p, bool there) {
    if constexpr (sizeof(T) * VEC == 8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.b64 %0, [%1];\n\t}" : "+l"(r) : "l"(p), "r"((int)there));
    else if constexpr (sizeof(T) * VEC == 4)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.b32 %0, [%1];\n\t}" : "+r"(r) : "l"(p), "r"((int)there));
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.u16 %0, [%1];\n\t}" : "+r"(r) : "l"(p), "r"((int)there));
}
template <typename T, int VEC> __device__ __forceinline__ Pair value(typename Raw<T, VEC>::type r) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC == 2) return r;
        else return pk2(__uint_as_float(r), 0.f);
    } else {
        const T* e = reinterpret_cast<const T*>(&r);
        return pk2(to_f32(e[0]), VEC > 1 ? to_f32(e[1]) : 0.f);
    }
}
template <typename T, int VEC> __device__ __forceinline__ void store(T* p, Pair v) {
    if constexpr (sizeof(T) * VEC == 8) {
        *reinterpret_cast<Pair*>(p) = v;
    } else {
        float x, y;
        upk2(v, x, y);
        if constexpr (VEC == 1) *p = from_f32<T>(x);
        else *reinterpret_cast<uint32_t*>(p) = pack2<T>(x, y);
    }
}
template <int VEC> __device__ __forceinline__ Pair load_f32(const float* p) { return VEC == 1 ? pk2(p[0], 0.f) : *reinterpret_cast<const Pair*>(p); }
template <int VEC> __device__ __forceinline__ void store_f32(float* p, Pair v) {
    float x, y;
    upk2(v, x, y);
    if (VEC == 1) p[0] = x;
    else *reinterpret_cast<Pair*>(p) = v;
}

// a = 1 / (1 + e), b = 1 - a = e a with e = exp(-gate): neither loses digits where the other is near 1. EXACT, for
// results of 32 bits: a is 0 and b 1 from e = 2^120 on; otherwise e ends at 2^126, which 16 bits of either do not show. A
// NaN stays.
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float min_nan(float v, float most) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(most));
    return r;
}
template <bool EXACT, int VEC> __device__ __forceinline__ void gates(Pair z, Pair& a, Pair& b) {
    if constexpr (EXACT) {
        float g[2], f[2] = {0.f, 0.f}, o[2] = {0.f, 0.f};
        upk2(z, g[0], g[1]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float e = expf(-g[k]);
            const bool closed = g[k] < -83.f;
            f[k] = closed ? 0.f : reciprocal(1.f + e);
            o[k] = closed ? 1.f : e * f[k];
        }
        a = pk2(f[0], f[1]), b = pk2(o[0], o[1]);
    } else {
        float t0, t1;
        upk2(mul2(z, pair(-1.4426950408889634f)), t0, t1);
        const Pair e = pk2(ex2(min_nan(t0, 126.f)), VEC > 1 ? ex2(min_nan(t1, 126.f)) : 0.f);
        upk2(add2(e, pair(1.f)), t0, t1);
        a = pk2(reciprocal(t0), VEC > 1 ? reciprocal(t1) : 1.f);
        b = mul2(e, a);
    }
}

// A batch element's positions, in the order of the recurrence
struct Element {
    int len, reverse;
    __device__ __forceinline__ Element(const sdtw_recurrence& a, int b)
        : len(a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N), reverse(a.reverse) {}
    __device__ __forceinline__ int row(int t) const { return reverse && t < len ? len - 1 - t : t; }
};

// ---- clusters
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(const void* mine, int cta, Pair x, Pair y) {
    uint32_t at = (uint32_t)__cvta_generic_to_shared(mine), there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(there), "l"(x), "l"(y) : "memory");
}

struct alignas(16) Run {   // h -> a h + h0
    Pair a, h;
};

// Rows [t, t + ROWS) of a run, in the recurrence's order: `there` of them are within the element's length, `none` stands
// for the others. A row's offset is within 32 bits.
template <typename T, int VEC, int ROWS>
__device__ __forceinline__ void fetch(typename Raw<T, VEC>::type (&out)[ROWS], const T* first, int step, int there, uint32_t none) {
    if (there >= ROWS) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) load<T, VEC>(out[i], first + i * step);
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            set_raw(out[i], none);
            load_if<T, VEC>(out[i], first + i * step, i < there);
        }
    }
}

// Zeros behind the runs, from position t on.
template <typename T, int VEC> __device__ __forceinline__ void clear(T* base, long long C, int t, int N, int warp, int warps) {
    for (t += warp; t < N; t += warps) store<T, VEC>(base + t * C, pair(0.f));
}

template <typename T, int VEC, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 2) recurrence_fwd_kernel(const RecurrenceParams p, int ctas)
{
    __shared__ Run run[2][kWarps][32], total[2][kMostCtas][32];
    const sdtw_recurrence& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x % ctas;
    const int columns = (a.C + 32 * VEC - 1) / (32 * VEC), id = blockIdx.x / ctas, b = id / columns;
    const int c = (id % columns * 32 + lane) * VEC;
    const bool on = c < a.C;
    const Element el(a, b);
    const long long bc = (long long)b * a.C + c;
    const int per = ctas * kWarps * ROWS;                 // positions that the cluster takes at a time
    const int steps = (a.N + kStep - 1) / kStep, rounds = (el.len + per - 1) / per;
    const int sign = el.reverse ? -1 : 1, xs = sign * (int)a.x_stride[1], gs = sign * (int)a.gate_stride[1], step = sign * a.C;
    const T* x = static_cast<const T*>(a.x) + b * a.x_stride[0] + c;
    const T* gate = static_cast<const T*>(a.gate) + b * a.gate_stride[0] + c;
    T* out = static_cast<T*>(p.h) + (long long)b * a.N * a.C + c;
    if (ctas > 1) cluster_arrive();
    Pair carry = a.state && on ? load_f32<VEC>(a.state + bc) : pair(0.f);
    typename Raw<T, VEC>::type xr[ROWS], gr[ROWS];
    int t = (rank * kWarps + warp) * ROWS;
    auto get = [&](int at) {
        const int there = on ? el.len - at : 0;
        const long long r = el.row(at);
        fetch<T, VEC, ROWS>(xr, x + r * a.x_stride[1], xs, there, 0);
        fetch<T, VEC, ROWS>(gr, gate + r * a.gate_stride[1], gs, there, open_bits<T>());
    };
    get(t);
    if (ctas > 1) cluster_wait();                         // the others have begun
    for (int round = 0; round < rounds; ++round, t += per) {
        const int there = el.len - t, turn = round & 1;
        Pair f[ROWS], u[ROWS];
        Run own{pair(1.f), pair(0.f)};
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            Pair o;
            gates<sizeof(T) == 4, VEC>(value<T, VEC>(gr[i]), f[i], o);
            u[i] = a.tied ? mul2(o, value<T, VEC>(xr[i])) : value<T, VEC>(xr[i]);
            own.a = mul2(own.a, f[i]);
            own.h = fma2(f[i], own.h, u[i]);
        }
        if (round + 1 < rounds) get(t + per);
        run[turn][warp][lane] = own;
        __syncthreads();
        Run all{pair(1.f), pair(0.f)}, before = all;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) before = all;
            const Run r = run[turn][w][lane];
            all.h = fma2(r.a, all.h, r.h);
            all.a = mul2(all.a, r.a);
        }
        Pair h = carry;
        if (ctas > 1) {
            for (int k = warp; k < ctas; k += kWarps) store_remote(&total[turn][rank][lane], k, all.a, all.h);
            cluster_arrive();
            cluster_wait();
            for (int k = 0; k < ctas; ++k) {
                if (k == rank) h = carry;
                const Run r = total[turn][k][lane];
                carry = fma2(r.a, carry, r.h);
            }
        } else {
            carry = fma2(all.a, carry, all.h);
        }
        h = fma2(before.a, h, before.h);
        if (!on) continue;
        if (p.kept && t % kStep == 0 && t < a.N) store_f32<VEC>(p.kept + ((long long)b * steps + t / kStep) * a.C + c, h);
        const long long r = el.row(t);
        T* dst = out + r * a.C;
        if (there >= ROWS) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                h = fma2(f[i], h, u[i]);
                store<T, VEC>(dst + i * step, h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                h = fma2(f[i], h, u[i]);
                if (i < there) store<T, VEC>(dst + i * step, h);
            }
            clear<T, VEC>(out, a.C, max(t, el.len), min(t + ROWS, a.N), 0, 1);
        }
    }
    if (!on) return;
    clear<T, VEC>(out, a.C, rounds * per, a.N, rank * kWarps + warp, ctas * kWarps);
    if (p.last && rank == 0 && warp == 0) store_f32<VEC>(p.last + bc, carry);
}

template <typename T, int VEC, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 2) recurrence_bwd_kernel(const RecurrenceParams p, int ctas)
{
    __shared__ Run run[2][kWarps][32], total[2][kMostCtas][32];
    __shared__ Pair back[2][kWarps][32];
    static_assert(kWarps * ROWS == kStep, "a CTA's run begins with a kept state");
    const sdtw_recurrence& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x % ctas;
    const int columns = (a.C + 32 * VEC - 1) / (32 * VEC), id = blockIdx.x / ctas, b = id / columns;
    const int c = (id % columns * 32 + lane) * VEC;
    const bool on = c < a.C;
    const Element el(a, b);
    const long long bc = (long long)b * a.C + c, base = (long long)b * a.N * a.C + c;
    const int per = ctas * kStep;
    const int steps = (a.N + kStep - 1) / kStep, rounds = (el.len + per - 1) / per;
    const int sign = el.reverse ? -1 : 1, xs = sign * (int)a.x_stride[1], gs = sign * (int)a.gate_stride[1], step = sign * a.C;
    const T* x = static_cast<const T*>(a.x) + b * a.x_stride[0] + c;
    const T* gate = static_cast<const T*>(a.gate) + b * a.gate_stride[0] + c;
    const T* dh = p.dh ? static_cast<const T*>(p.dh) + base : nullptr;
    T *dx = static_cast<T*>(p.dx) + base, *dgate = static_cast<T*>(p.dgate) + base;
    if (ctas > 1) cluster_arrive();
    Pair carry = p.dlast && on ? load_f32<VEC>(p.dlast + bc) : pair(0.f);
    typename Raw<T, VEC>::type xr[ROWS], gr[ROWS], dr[ROWS];
    Pair state = pair(0.f);
    int t = (rounds - 1) * per + (rank * kWarps + warp) * ROWS;
    auto get = [&](int at) {
        const int there = on ? el.len - at : 0;
        const long long r = el.row(at);
        fetch<T, VEC, ROWS>(xr, x + r * a.x_stride[1], xs, there, 0);
        fetch<T, VEC, ROWS>(gr, gate + r * a.gate_stride[1], gs, there, open_bits<T>());
        fetch<T, VEC, ROWS>(dr, dh + r * a.C, step, dh ? there : 0, 0);
        state = there > 0 ? load_f32<VEC>(p.kept_in + ((long long)b * steps + at / kStep) * a.C + c) : pair(0.f);
    };
    if (rounds > 0) get(t);
    if (ctas > 1) cluster_wait();
    for (int round = rounds - 1; round >= 0; --round, t -= per) {
        const int there = on ? el.len - t : 0, turn = round & 1;
        Pair f[ROWS], o[ROWS], v[ROWS], d[ROWS], h = state;
        Run own{pair(1.f), pair(0.f)};
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            gates<sizeof(T) == 4, VEC>(value<T, VEC>(gr[i]), f[i], o[i]);
            v[i] = value<T, VEC>(xr[i]);
            d[i] = value<T, VEC>(dr[i]);
            own.a = mul2(own.a, f[i]);
            own.h = fma2(f[i], own.h, a.tied ? mul2(o[i], v[i]) : v[i]);
        }
        Pair r = pair(0.f);
#pragma unroll
        for (int i = ROWS - 1; i >= 0; --i) r = mul2(f[i], add2(d[i], r));
        if (round > 0) get(t - per);
        run[turn][warp][lane] = own;
        back[turn][warp][lane] = r;
        __syncthreads();
        // states before the run, and what the later runs of the CTA hand back
        Run behind{pair(1.f), pair(0.f)};
        Pair all_a = pair(1.f), all_r = pair(0.f);
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            if (w == warp) behind = Run{all_a, all_r};
            const Pair wa = run[turn][w][lane].a;
            all_r = fma2(wa, all_r, back[turn][w][lane]);
            all_a = mul2(all_a, wa);
        }
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) {
                const Run q = run[turn][w][lane];
                h = fma2(q.a, h, q.h);
            }
        r = carry;
        if (ctas > 1) {
            for (int k = warp; k < ctas; k += kWarps) store_remote(&total[turn][rank][lane], k, all_a, all_r);
            cluster_arrive();
            cluster_wait();
            for (int k = ctas - 1; k >= 0; --k) {
                if (k == rank) r = carry;
                const Run q = total[turn][k][lane];
                carry = fma2(q.a, carry, q.h);
            }
        } else {
            carry = fma2(all_a, carry, all_r);
        }
        r = fma2(behind.a, r, behind.h);
        if (!on) continue;
        const long long row = (long long)el.row(t) * a.C;
        Pair before[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            before[i] = a.tied ? fma2(v[i], pair(-1.f), h) : h;
            h = fma2(f[i], h, a.tied ? mul2(o[i], v[i]) : v[i]);
        }
        auto go = [&](bool every) {
#pragma unroll
            for (int i = ROWS - 1; i >= 0; --i) {
                const Pair e = add2(d[i], r), g = mul2(o[i], e);
                r = mul2(f[i], e);
                if (every || i < there) {
                    store<T, VEC>(dx + row + i * step, a.tied ? g : e);
                    store<T, VEC>(dgate + row + i * step, mul2(mul2(g, f[i]), before[i]));
                }
            }
        };
        if (there >= ROWS) go(true);
        else go(false);
        if (there < ROWS) {
            clear<T, VEC>(dx, a.C, max(t, el.len), min(t + ROWS, a.N), 0, 1);
            clear<T, VEC>(dgate, a.C, max(t, el.len), min(t + ROWS, a.N), 0, 1);
        }
    }
    if (!on) return;
    clear<T, VEC>(dx, a.C, rounds * per, a.N, rank * kWarps + warp, ctas * kWarps);
    clear<T, VEC>(dgate, a.C, rounds * per, a.N, rank * kWarps + warp, ctas * kWarps);
    if (p.dstate && rank == 0 && warp == 0) store_f32<VEC>(p.dstate + bc, carry);
}

// A few new samples: a thread has its channels' positions from first to last, all of them on their way at once.
template <typename T, int VEC, int ROWS> __global__ void __launch_bounds__(128) recurrence_few_kernel(const RecurrenceParams p)
{
    const sdtw_recurrence& a = p.a;
    const int columns = (a.C + VEC - 1) / VEC;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int b = (int)(i / columns), c = (int)(i % columns) * VEC;
    if (b >= a.B) return;
    const Element el(a, b);
    const long long bc = (long long)b * a.C + c, r = el.row(0), base = (long long)b * a.N * a.C + c;
    typename Raw<T, VEC>::type xr[ROWS], gr[ROWS];
    const int sign = el.reverse ? -1 : 1;
    fetch<T, VEC, ROWS>(xr, static_cast<const T*>(a.x) + b * a.x_stride[0] + c + r * a.x_stride[1], sign * (int)a.x_stride[1], el.len, 0);
    fetch<T, VEC, ROWS>(gr, static_cast<const T*>(a.gate) + b * a.gate_stride[0] + c + r * a.gate_stride[1], sign * (int)a.gate_stride[1], el.len, open_bits<T>());
    Pair h = a.state ? load_f32<VEC>(a.state + bc) : pair(0.f);
    if (p.kept) store_f32<VEC>(p.kept + bc, h);
    T* out = static_cast<T*>(p.h) + base;
#pragma unroll
    for (int t = 0; t < ROWS; ++t)
        if (t < el.len) {
            Pair f, o;
            gates<sizeof(T) == 4, VEC>(value<T, VEC>(gr[t]), f, o);
            const Pair v = value<T, VEC>(xr[t]);
            h = fma2(f, h, a.tied ? mul2(o, v) : v);
            store<T, VEC>(out + el.row(t) * (long long)a.C, h);
        } else if (t < a.N) {
            store<T, VEC>(out + (long long)t * a.C, pair(0.f));
        }
    if (p.last) store_f32<VEC>(p.last + bc, h);
}

template <typename... P> cudaError_t launch_clusters(void (*kernel)(P...), long long clusters, int ctas, cudaStream_t s, const RecurrenceParams& p)
{
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ctas, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.gridDim = dim3((unsigned)(clusters * ctas)), c.blockDim = dim3(kWarps * 32), c.stream = s, c.attrs = &at, c.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, p, ctas);
}

// CTAs of a cluster: as many as it takes to have two a SM, no more than there are runs.
int cluster_size(long long clusters, int N, int positions, int sms)
{
    int k = 1;
    while (k < kMostCtas && clusters * k < 2ll * sms && (long long)k * positions < N) k *= 2;
    return k;
}

constexpr int kFewRows = 8;

template <typename T, int VEC> cudaError_t run_vec(const RecurrenceParams& p, bool backward, int sms, cudaStream_t s)
{
    constexpr int ROWS = sizeof(T) == 4 ? 8 : 16;   // forward: two arrays' rows in flight, and their gates
    const sdtw_recurrence& a = p.a;
    const long long clusters = (long long)a.B * ((a.C + 32 * VEC - 1) / (32 * VEC));
    if (backward) return launch_clusters(recurrence_bwd_kernel<T, VEC, kStep / kWarps>, clusters, cluster_size(clusters, a.N, kStep, sms), s, p);
    if (a.N <= kFewRows) {
        const long long threads = (long long)a.B * ((a.C + VEC - 1) / VEC);
        if (a.N == 1) recurrence_few_kernel<T, VEC, 1><<<(unsigned)((threads + 127) / 128), 128, 0, s>>>(p);
        else recurrence_few_kernel<T, VEC, kFewRows><<<(unsigned)((threads + 127) / 128), 128, 0, s>>>(p);
        return cudaGetLastError();
    }
    return launch_clusters(recurrence_fwd_kernel<T, VEC, ROWS>, clusters, cluster_size(clusters, a.N, kWarps * ROWS, sms), s, p);
}

template <typename T> cudaError_t run(const RecurrenceParams& p, bool backward, int sms, cudaStream_t s)
{
    const sdtw_recurrence& a = p.a;
    constexpr uintptr_t mask = 2 * sizeof(T) - 1;
    auto even = [](const void* q, uintptr_t m) { return (reinterpret_cast<uintptr_t>(q) & m) == 0; };
    bool pairs = a.C % 2 == 0 && even(a.x, mask) && even(a.gate, mask) && even(a.state, 7);
    for (int i = 0; i < 2; ++i) pairs = pairs && a.x_stride[i] % 2 == 0 && a.gate_stride[i] % 2 == 0;
    pairs = pairs && (backward ? even(p.dh, mask) && even(p.dx, mask) && even(p.dgate, mask) && even(p.dlast, 7) && even(p.dstate, 7) && even(p.kept_in, 7)
                               : even(p.h, mask) && even(p.last, 7) && even(p.kept, 7));
    return pairs ? run_vec<T, 2>(p, backward, sms, s) : run_vec<T, 1>(p, backward, sms, s);
}
cudaError_t any(const RecurrenceParams& p, bool backward, int sms, cudaStream_t s)
{
    if (p.a.dtype == SDTW_F32) return run<float>(p, backward, sms, s);
    if (p.a.dtype == SDTW_BF16) return run<__nv_bfloat16>(p, backward, sms, s);
    return run<__half>(p, backward, sms, s);
}

}  // namespace

cudaError_t launch_recurrence_forward(const RecurrenceParams& p, int sms, cudaStream_t s) { return any(p, false, sms, s); }
cudaError_t launch_recurrence_backward(const RecurrenceParams& p, int sms, cudaStream_t s) { return any(p, true, sms, s); }

}  // namespace sdtw
