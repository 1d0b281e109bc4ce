// recurrence.cu -- a gated linear recurrence along a series, forward and backward.
//
//   a_t = sigmoid(gate_t), h_t = a_t h_{t-1} + (1 - a_t) x_t (tied) or a_t h_{t-1} + x_t
//   e_t = dh_t + r_{t+1}, r_t = a_t e_t, dx_t = (1 - a_t) e_t or e_t, dgate_t = e_t (h_{t-1} - x_t or h_{t-1}) a_t (1 - a_t)
//
// Steps h -> a h + u compose: the steps of a run of positions are one pair (A, H), h -> A h + H, and those of the
// gradient one pair (A, R) with the same A, R = sum_i a_1 .. a_i dh_i. A warp has a run of ROWS positions of 32 lanes' channels,
// a lane two of them (one where sizes are odd): it composes its run, the CTA's warps and then the CTAs of a cluster
// exchange their pairs through shared memory, and each goes over its run again from the state before it. A cluster so takes
// CTAs x warps x ROWS positions at a time, and carries the state to the next. The order of all sums is fixed by the sizes:
// the same bits every time. The backward pass computes the states again from those that the forward pass kept, one in
// SDTW_RECURRENCE_STEP positions: 3 reads and 2 writes where stored states would be another read.
//
// Coming positions are on their way to shared memory meanwhile (TMA; sizes and addresses that do not allow it are loaded by
// the lanes that use them). Pairs go between CTAs by stores that report to the receiver's mbarrier: a
// cluster's own barrier also waits for the results that are on their way to memory. One warp folds the CTAs' pairs and hands the
// state on: read by every warp, they took 900 cycles of shared memory a round.
//
// Measured: 16 x 8192 x 1024 bf16 132 us forward (6.1 TB/s) and 242 backward (5.6); 4 such 41 and 71; 4 in fp32 68 and 112 (5.9 and 6.0 TB/s of
// a copy's 6.8); 2 x 16383 x 264 fp16 24 and 40. Memory bounds the many; the few by their rounds, which pass the
// state on one after the other. Loaded by the lanes that use them, 4 x 8192 x 1023 takes 123 and 187 us.
#include "activation.cuh"
#include "attn_tc.cuh"
#include "block.h"
#include "packed.cuh"

#include <atomic>
#include <initializer_list>
#include <type_traits>

namespace sdtw {
namespace {

constexpr int kStep = SDTW_RECURRENCE_STEP;
constexpr int kMostCtas = 16;   // of a cluster
constexpr int kStages = 3;      // of the forward pass's ring: coming, in work, and results on their way out

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
        const Halves<T> h(r);
        return pk2(to_f32(h.e[0]), VEC > 1 ? to_f32(h.e[1]) : 0.f);
    }
}
template <typename T, int VEC> __device__ __forceinline__ void store(T* p, Pair v) {
    if constexpr (sizeof(T) * VEC == 8) {
        *reinterpret_cast<Pair*>(p) = v;
    } else {
        float x, y;
        upk2(v, x, y);
        if constexpr (VEC == 1) *p = from_f32<T>(x);
        else *reinterpret_cast<Pack<T, 2>*>(p) = rounded<T, 2>({v});
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
// results of 32 bits, takes expf. Beyond e = 2^126 a is 0, a closed gate: smaller ones than that are no normal numbers. b is
// 1 there, where e may be infinite.
// A NaN stays, and in its channel, by a reciprocal for each: two channels that share one, 1 / s = t / (s t), share its rounding and a
// NaN too. It cost 2 x 16383 x 264 fp16 25.6 us for 24.7 forward, and 16 x 8192 x 1024 bf16 nothing.
template <bool EXACT, int VEC> __device__ __forceinline__ void gates(Pair z, Pair& a, Pair& b) {
    float t[2], e[2] = {}, f[2] = {}, o[2] = {};
    upk2(EXACT ? z : mul2(z, pair(-1.4426950408889634f)), t[0], t[1]);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        e[k] = EXACT ? expf(-t[k]) : ex2(t[k]);
        f[k] = reciprocal(1.f + e[k]);
        o[k] = e[k] > 0x1p125f ? 1.f : e[k] * f[k];
    }
    a = pk2(f[0], f[1]), b = pk2(o[0], o[1]);
}

// A batch element's positions, in the order of the recurrence
struct Element {
    int len, reverse;
    __device__ __forceinline__ Element(const sdtw_recurrence& a, int b)
        : len(a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N), reverse(a.reverse) {}
    __device__ __forceinline__ int row(int t) const { return reverse && t < len ? len - 1 - t : t; }
};

// ---- clusters
__device__ int g_status;

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t mine, int cta) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(cta));
    return there;
}
// 16 bytes to another CTA's shared memory, reported to its barrier
__device__ __forceinline__ void send_pairs(uint32_t there, uint32_t bar, Pair x, Pair y) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(there), "l"(x), "l"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Bounded: false, the status word set and the CTA's `late` too, when it ran out. Who gave up a wait may have read what was not there, and
// others go on from it: at its end the cluster makes NaN of all its results.
__device__ __forceinline__ bool wait_arrived(uint32_t bar, uint32_t parity, unsigned long long limit_ns, int& late) {
    if (arrived(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!arrived(bar, parity))
        if (global_ns() - t0 > limit_ns) {
            atomicOr(&g_status, kStatusTimeout);
            *static_cast<volatile int*>(&late) = 1;
            return false;
        }
    return true;
}
// All threads of the cluster, at its end: no store may come to a CTA that has ended. Whether one of them was late.
__device__ __forceinline__ bool any_late(int& late, int ctas) {
    __syncthreads();
    if (ctas > 1) {
        if (*static_cast<volatile int*>(&late) && (int)threadIdx.x < ctas)
            asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(in_cta((uint32_t)__cvta_generic_to_shared(&late), (int)threadIdx.x)) : "memory");
        cluster_sync();
    }
    return *static_cast<volatile int*>(&late) != 0;
}
__device__ __forceinline__ Pair not_a_number() { return pk2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff)); }

struct alignas(16) Run {   // h -> a h + h0
    Pair a, h;
};

// Rows [t, t + ROWS) of a run, in the recurrence's order: `there` of them are within the element's length, `none` stands
// for the others.
template <typename T, int VEC, int ROWS>
__device__ __forceinline__ void fetch(typename Raw<T, VEC>::type (&out)[ROWS], const T* first, int step, int there, uint32_t none) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        set_raw(out[i], none);
        load_if<T, VEC>(out[i], first + i * step, i < there);
    }
}

// Zeros behind the runs, from position t on.
template <typename T, int VEC> __device__ __forceinline__ void clear(T* base, long long C, int t, int N, int warp, int warps) {
    for (t += warp; t < N; t += warps) store<T, VEC>(base + t * C, pair(0.f));
}

// The CTA's positions of one array, as they lie in memory: in a ring of stages in shared memory, or in the lanes' registers.
template <typename T, int VEC, int ROWS, bool RING> struct Rows {
    typename Raw<T, VEC>::type raw[ROWS];
    __device__ __forceinline__ Pair at(int i, const unsigned char*) const { return value<T, VEC>(raw[i]); }
};
template <typename T, int VEC, int ROWS> struct Rows<T, VEC, ROWS, true> {
    __device__ __forceinline__ Pair at(int, const unsigned char* mine) const { return value<T, VEC>(*reinterpret_cast<const typename Raw<T, VEC>::type*>(mine)); }
};
// What TMA loads from: (B, N, C) arrays in boxes of a CTA's positions by 32 lanes' channels.
struct RecurrenceMaps {
    CUtensorMap x, gate, dh, h;
    int x_batch, gate_batch;   // 0: every batch element is the same one
};
__device__ __forceinline__ void load_box(unsigned char* to, const CUtensorMap* m, int c, int row, int b, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(m), "r"(bar), "r"(c), "r"(row), "r"(b)
                 : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* m, const unsigned char* from, int c, int row, int b) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(m),
                 "r"((uint32_t)__cvta_generic_to_shared(from)), "r"(c), "r"(row), "r"(b)
                 : "memory");
}
__device__ __forceinline__ void stored() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }   // shared memory is read no more
// Rows of a stage that stand for no position, as this lane will read them. Boxes that come there later come after it.
template <typename T, int VEC, int ROWS> __device__ __forceinline__ void blank(unsigned char* mine, int step, int there, uint32_t none) {
    for (int i = max(there, 0); i < ROWS; ++i) set_raw(*reinterpret_cast<typename Raw<T, VEC>::type*>(mine + i * step), none);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// TIED: 1, 0, or -1: as the call says.
template <typename T, int VEC, int ROWS, int WARPS, bool RING, int TIED>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) recurrence_fwd_kernel(const RecurrenceParams p, const __grid_constant__ RecurrenceMaps maps, int ctas)
{
    constexpr int bytes = 32 * VEC * sizeof(T), image = RING ? WARPS * ROWS * bytes : 0;
    __shared__ Run run[WARPS][32];
    __shared__ Pair s_in[32];                             // states before the CTA's positions
    __shared__ uint64_t s_bar[2 + kStages + 1];           // of the exchange, by turns; of the stages; one that nothing arrives at
    __shared__ int s_late;
    extern __shared__ __align__(128) unsigned char ring[];   // [kStages][x, gate][WARPS ROWS][32 VEC], then [2][ctas][32] Runs
    Run* total = reinterpret_cast<Run*>(ring + kStages * 2 * image);
    const sdtw_recurrence& a = p.a;
    const bool tied = TIED < 0 ? a.tied != 0 : TIED != 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x % ctas;
    const int columns = (a.C + 32 * VEC - 1) / (32 * VEC), id = blockIdx.x / ctas, b = id / columns;
    const int c0 = id % columns * 32 * VEC, c = c0 + lane * VEC;
    const bool on = c < a.C;
    const Element el(a, b);
    const long long bc = (long long)b * a.C + c;
    const int per = ctas * WARPS * ROWS;                 // positions that the cluster takes at a time
    const int steps = (a.N + kStep - 1) / kStep, rounds = (el.len + per - 1) / per;
    const int sign = el.reverse ? -1 : 1, xs = sign * (int)a.x_stride[1], gs = sign * (int)a.gate_stride[1], step = sign * a.C;
    const T* x = static_cast<const T*>(a.x) + b * a.x_stride[0];
    const T* gate = static_cast<const T*>(a.gate) + b * a.gate_stride[0];
    T* out = static_cast<T*>(p.h) + (long long)b * a.N * a.C + c;
    const uint32_t bars = (uint32_t)__cvta_generic_to_shared(s_bar);
    if (threadIdx.x == 0) s_late = 0;
    if (threadIdx.x < 2 + kStages + 1) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * threadIdx.x) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    Pair carry = a.state && on ? load_f32<VEC>(a.state + bc) : pair(0.f);
    const int t0 = rank * WARPS * ROWS;                  // the CTA's first position
    int t = t0 + warp * ROWS;
    // A box has its rows as they lie in memory: backwards in time, the other way round.
    const int line = el.reverse ? -bytes : bytes;
    auto send = [&](int round) {
        if (round >= rounds || threadIdx.x != 0) return;
        const int at = t0 + round * per, row = el.reverse ? el.len - at - WARPS * ROWS : at;
        unsigned char* stage = ring + round % kStages * 2 * image;
        const uint32_t bar = bars + 8 * (2 + round % kStages);
        expect(bar, at < el.len ? 2 * image : 0);
        if (at >= el.len) return;
        load_box(stage, &maps.x, c0, row, b * maps.x_batch, bar);
        load_box(stage + image, &maps.gate, c0, row, b * maps.gate_batch, bar);
    };
    // results of whole tiles go out from x's place in their stage
    auto whole = [&](int round) { return RING && round >= 0 && el.len - (t0 + round * per) >= WARPS * ROWS; };
    auto put_out = [&](int round) {
        if (!whole(round) || threadIdx.x != 0) return;
        const int at = t0 + round * per;
        store_box(&maps.h, ring + round % kStages * 2 * image, c0, el.reverse ? el.len - at - WARPS * ROWS : at, b);
    };
    if constexpr (RING) {
        __syncthreads();                                  // the barriers are there
        send(0);
    }
    if (ctas > 1) cluster_sync();                         // the others have begun, with barriers
    if (RING && p.skip == 2 && rank == 0 && warp == 1) wait_arrived(bars + 8 * (2 + kStages), 0, p.wait_ns, s_late);
    bool ok = true;
    for (int round = 0; round < rounds; ++round, t += per) {
        const int there = el.len - t, turn = round & 1;
        Rows<T, VEC, ROWS, RING> xr, gr;
        unsigned char* mine = ring + round % kStages * 2 * image + (el.reverse ? WARPS * ROWS - 1 - warp * ROWS : warp * ROWS) * bytes + lane * VEC * sizeof(T);
        if constexpr (RING) {
            __syncthreads();                              // the last round's results are in their stage
            if (threadIdx.x == 0) stored();               // those of the round before it have left theirs, the next to be filled
            put_out(round - 1);
            send(round + 1);
            wait_arrived(bars + 8 * (2 + round % kStages), (uint32_t)(round / kStages) & 1, p.wait_ns, s_late);
            if (there < ROWS) {
                blank<T, VEC, ROWS>(mine, line, there, 0);
                blank<T, VEC, ROWS>(mine + image, line, there, open_bits<T>());
            }
        } else {
            const long long r = el.row(t);
            fetch<T, VEC, ROWS>(xr.raw, x + r * a.x_stride[1] + c, xs, on ? there : 0, 0);
            fetch<T, VEC, ROWS>(gr.raw, gate + r * a.gate_stride[1] + c, gs, on ? there : 0, open_bits<T>());
        }
        Pair f[ROWS], u[ROWS];
        Run own{pair(1.f), pair(0.f)};
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            Pair o;
            gates<sizeof(T) == 4, VEC>(gr.at(i, mine + image + i * line), f[i], o);
            u[i] = tied ? mul2(o, xr.at(i, mine + i * line)) : xr.at(i, mine + i * line);
            own.a = mul2(own.a, f[i]);
            own.h = fma2(f[i], own.h, u[i]);
        }
        run[warp][lane] = own;
        __syncthreads();
        // the runs before this warp's; the last warp goes on to the CTA's
        Run before{pair(1.f), pair(0.f)};
#pragma unroll
        for (int w0 = 0; w0 < WARPS; w0 += 4)
            if (w0 < warp) {
                Run r[4];   // all on their way before the first is used
#pragma unroll
                for (int w = 0; w < 4; ++w) r[w] = run[w0 + w][lane];
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w0 + w < warp) {
                        before.h = fma2(r[w].a, before.h, r[w].h);
                        before.a = mul2(before.a, r[w].a);
                    }
            }
        if (warp == WARPS - 1) {
            const Pair all_a = mul2(before.a, own.a), all_h = fma2(own.a, before.h, own.h);
            Pair in = carry;
            if (ctas > 1) {
                const uint32_t bar = bars + 8 * turn, slot = (uint32_t)__cvta_generic_to_shared(&total[(turn * ctas + rank) * 32 + lane]);
                if (lane == 0) expect(bar, ctas * 512);
                if (!(p.skip == 1 && rank == 0))
                    for (int k = 0; k < ctas; ++k) send_pairs(in_cta(slot, k), in_cta(bar, k), all_a, all_h);
                if (!wait_arrived(bar, (uint32_t)(round >> 1) & 1, ok ? p.wait_ns : 0, s_late)) ok = false;
                for (int k0 = 0; k0 < ctas; k0 += 4) {
                    Run r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[k] = total[(turn * ctas + min(k0 + k, ctas - 1)) * 32 + lane];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        in = k0 + k == rank ? carry : in;
                        carry = k0 + k < ctas ? fma2(r[k].a, carry, r[k].h) : carry;
                    }
                }
            } else {
                carry = fma2(all_a, in, all_h);
            }
            s_in[lane] = in;
        }
        __syncthreads();
        Pair h = fma2(before.a, s_in[lane], before.h);
        if (whole(round)) {
            if (on && p.kept && t % kStep == 0) store_f32<VEC>(p.kept + ((long long)b * steps + t / kStep) * a.C + c, h);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                h = fma2(f[i], h, u[i]);
                store<T, VEC>(reinterpret_cast<T*>(mine + i * line), h);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            continue;
        }
        if (!on) continue;
        if (p.kept && t % kStep == 0 && t < a.N) store_f32<VEC>(p.kept + ((long long)b * steps + t / kStep) * a.C + c, h);
        T* dst = out + (long long)el.row(t) * a.C;
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
    if constexpr (RING) {
        __syncthreads();
        put_out(rounds - 1);
        if (threadIdx.x == 0) stored();
    }
    if (any_late(s_late, ctas)) {
        if (RING && threadIdx.x == 0) {   // loads on their way come before the CTA ends, and results are written, not only read
            for (int k = max(0, rounds - kStages); k < rounds; ++k) wait_arrived(bars + 8 * (2 + k % kStages), (uint32_t)(k / kStages) & 1, p.wait_ns, s_late);
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        carry = not_a_number();
        for (t = t0 + warp * ROWS; on && t < el.len; t += per) {
            if (p.kept && t % kStep == 0) store_f32<VEC>(p.kept + ((long long)b * steps + t / kStep) * a.C + c, carry);
            for (int i = 0; i < min(ROWS, el.len - t); ++i) store<T, VEC>(out + (long long)el.row(t + i) * a.C, carry);
        }
    }
    if (!on) return;
    clear<T, VEC>(out, a.C, rounds * per, a.N, rank * WARPS + warp, ctas * WARPS);
    if (p.last && rank == 0 && warp == WARPS - 1) store_f32<VEC>(p.last + bc, carry);
}

template <typename T, int VEC, int ROWS, int WARPS, bool RING, int TIED>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) recurrence_bwd_kernel(const RecurrenceParams p, const __grid_constant__ RecurrenceMaps maps, int ctas)
{
    constexpr int bytes = 32 * VEC * sizeof(T), image = RING ? WARPS * ROWS * bytes : 0;
    __shared__ Run run[WARPS][32];
    __shared__ Pair back[WARPS][32], s_in[32];            // s_in: what the positions after the CTA's hand back
    __shared__ uint64_t s_bar[2 + 2 + 1];                 // as in the forward pass
    __shared__ int s_late;
    extern __shared__ __align__(128) unsigned char ring[];   // [2][x, gate, dh][WARPS ROWS][32 VEC], then [2][ctas][32] Runs
    Run* total = reinterpret_cast<Run*>(ring + 2 * 3 * image);
    static_assert(WARPS * ROWS % kStep == 0 || kStep % (WARPS * ROWS) == 0, "kept states at CTAs' first positions");
    const sdtw_recurrence& a = p.a;
    const bool tied = TIED < 0 ? a.tied != 0 : TIED != 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x % ctas;
    const int columns = (a.C + 32 * VEC - 1) / (32 * VEC), id = blockIdx.x / ctas, b = id / columns;
    const int c0 = id % columns * 32 * VEC, c = c0 + lane * VEC;
    const bool on = c < a.C;
    const Element el(a, b);
    const long long bc = (long long)b * a.C + c, base = (long long)b * a.N * a.C;
    const int per = ctas * WARPS * ROWS;
    const int steps = (a.N + kStep - 1) / kStep, rounds = (el.len + per - 1) / per;
    const int sign = el.reverse ? -1 : 1, xs = sign * (int)a.x_stride[1], gs = sign * (int)a.gate_stride[1], step = sign * a.C;
    const T* x = static_cast<const T*>(a.x) + b * a.x_stride[0];
    const T* gate = static_cast<const T*>(a.gate) + b * a.gate_stride[0];
    const T* dh = static_cast<const T*>(p.dh) + base;
    T *dx = static_cast<T*>(p.dx) + base + c, *dgate = static_cast<T*>(p.dgate) + base + c;
    const uint32_t bars = (uint32_t)__cvta_generic_to_shared(s_bar);
    if (threadIdx.x == 0) s_late = 0;
    if (threadIdx.x < 5) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * threadIdx.x) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    Pair carry = p.dlast && on ? load_f32<VEC>(p.dlast + bc) : pair(0.f);
    const int t0 = rank * WARPS * ROWS;
    const int line = el.reverse ? -bytes : bytes;
    auto send = [&](int round) {
        if (round < 0 || threadIdx.x != 0) return;
        const int at = t0 + round * per, row = el.reverse ? el.len - at - WARPS * ROWS : at;
        unsigned char* stage = ring + (round & 1) * 3 * image;
        const uint32_t bar = bars + 8 * (2 + (round & 1));
        expect(bar, at < el.len ? (p.dh ? 3 : 2) * image : 0);
        if (at >= el.len) return;
        load_box(stage, &maps.x, c0, row, b * maps.x_batch, bar);
        load_box(stage + image, &maps.gate, c0, row, b * maps.gate_batch, bar);
        if (p.dh) load_box(stage + 2 * image, &maps.dh, c0, row, b, bar);
    };
    auto kept = [&](int round) {   // the state before the CTA's first position
        const int at = t0 + round * per;
        return on && round >= 0 && at < el.len ? load_f32<VEC>(p.kept_in + ((long long)b * steps + at / kStep) * a.C + c) : pair(0.f);
    };
    if constexpr (RING) {
        __syncthreads();
        send(rounds - 1);
    }
    Pair state = kept(rounds - 1);
    if (ctas > 1) cluster_sync();
    if (RING && p.skip == 2 && rank == 0 && warp == 1) wait_arrived(bars + 8 * 4, 0, p.wait_ns, s_late);
    bool ok = true;
    int turn = 0, phase = 0;
    for (int round = rounds - 1; round >= 0; --round) {
        const int t = t0 + round * per + warp * ROWS, there = on ? el.len - t : 0;
        Rows<T, VEC, ROWS, RING> xr, gr, dr;
        unsigned char* mine = ring + (round & 1) * 3 * image + (el.reverse ? WARPS * ROWS - 1 - warp * ROWS : warp * ROWS) * bytes + lane * VEC * sizeof(T);
        if constexpr (RING) {
            __syncthreads();
            send(round - 1);
            wait_arrived(bars + 8 * (2 + (round & 1)), (uint32_t)((rounds - 1 - round) >> 1) & 1, p.wait_ns, s_late);
            if (el.len - t < ROWS) {
                blank<T, VEC, ROWS>(mine, line, el.len - t, 0);
                blank<T, VEC, ROWS>(mine + image, line, el.len - t, open_bits<T>());
            }
            if (el.len - t < ROWS || !p.dh) blank<T, VEC, ROWS>(mine + 2 * image, line, p.dh ? el.len - t : 0, 0);
        } else {
            const long long r = el.row(t);
            fetch<T, VEC, ROWS>(xr.raw, x + r * a.x_stride[1] + c, xs, there, 0);
            fetch<T, VEC, ROWS>(gr.raw, gate + r * a.gate_stride[1] + c, gs, there, open_bits<T>());
            fetch<T, VEC, ROWS>(dr.raw, dh + r * a.C + c, step, p.dh ? there : 0, 0);
        }
        Pair f[ROWS], o[ROWS], h = state, r = pair(0.f);
        Run own{pair(1.f), pair(0.f)};
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            gates<sizeof(T) == 4, VEC>(gr.at(i, mine + image + i * line), f[i], o[i]);
            const Pair v = xr.at(i, mine + i * line);
            own.a = mul2(own.a, f[i]);
            own.h = fma2(f[i], own.h, tied ? mul2(o[i], v) : v);
            r = fma2(own.a, dr.at(i, mine + 2 * image + i * line), r);
        }
        run[warp][lane] = own;
        back[warp][lane] = r;
        state = kept(round - 1);
        __syncthreads();
        // what the later runs of the CTA hand back; the first warp goes on to the CTA's
        Run behind{pair(1.f), pair(0.f)};
#pragma unroll
        for (int w0 = WARPS - 4; w0 >= 0; w0 -= 4)
            if (w0 + 3 > warp) {
                Pair wa[4], wr[4];   // all on their way before the first is used
#pragma unroll
                for (int w = 0; w < 4; ++w) wa[w] = run[w0 + w][lane].a, wr[w] = back[w0 + w][lane];
#pragma unroll
                for (int w = 3; w >= 0; --w)
                    if (w0 + w > warp) {
                        behind.h = fma2(wa[w], behind.h, wr[w]);
                        behind.a = mul2(behind.a, wa[w]);
                    }
            }
        if (warp == 0) {
            const Pair all_a = mul2(behind.a, own.a), all_r = fma2(own.a, behind.h, r);
            Pair in = carry;
            if (ctas > 1) {
                const uint32_t bar = bars + 8 * turn, slot = (uint32_t)__cvta_generic_to_shared(&total[(turn * ctas + rank) * 32 + lane]);
                if (lane == 0) expect(bar, ctas * 512);
                if (!(p.skip == 1 && rank == 0))
                    for (int k = 0; k < ctas; ++k) send_pairs(in_cta(slot, k), in_cta(bar, k), all_a, all_r);
                if (!wait_arrived(bar, (uint32_t)phase, ok ? p.wait_ns : 0, s_late)) ok = false;
                for (int k0 = ctas - 1; k0 >= 0; k0 -= 4) {
                    Run q[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = total[(turn * ctas + max(k0 - k, 0)) * 32 + lane];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        in = k0 - k == rank ? carry : in;
                        carry = k0 - k >= 0 ? fma2(q[k].a, carry, q[k].h) : carry;
                    }
                }
            } else {
                carry = fma2(all_a, in, all_r);
            }
            s_in[lane] = in;
        }
        // the state before the run
#pragma unroll
        for (int w0 = 0; w0 < WARPS; w0 += 4)
            if (w0 < warp) {
                Run q[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) q[w] = run[w0 + w][lane];
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w0 + w < warp) h = fma2(q[w].a, h, q[w].h);
            }
        __syncthreads();
        r = s_in[lane];
        phase ^= turn;   // every second round
        turn ^= 1;
        r = fma2(behind.a, r, behind.h);
        if (!on) continue;
        const long long row = (long long)el.row(t) * a.C;
        Pair w[ROWS];   // dgate_t / e_t
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const Pair v = xr.at(i, mine + i * line);
            w[i] = mul2(mul2(f[i], o[i]), tied ? fma2(v, pair(-1.f), h) : h);
            h = fma2(f[i], h, tied ? mul2(o[i], v) : v);
        }
        auto go = [&](bool every) {
#pragma unroll
            for (int i = ROWS - 1; i >= 0; --i) {
                const Pair e = add2(dr.at(i, mine + 2 * image + i * line), r);
                r = mul2(f[i], e);
                if (every || i < there) {
                    store<T, VEC>(dx + row + i * step, tied ? mul2(o[i], e) : e);
                    store<T, VEC>(dgate + row + i * step, mul2(w[i], e));
                }
            }
        };
        if (there >= ROWS) {
            go(true);
        } else {
            go(false);
            clear<T, VEC>(dx, a.C, max(t, el.len), min(t + ROWS, a.N), 0, 1);
            clear<T, VEC>(dgate, a.C, max(t, el.len), min(t + ROWS, a.N), 0, 1);
        }
    }
    if (any_late(s_late, ctas)) {
        if (RING && threadIdx.x == 0)
            for (int k = min(rounds, 2) - 1; k >= 0; --k) wait_arrived(bars + 8 * (2 + (k & 1)), (uint32_t)((rounds - 1 - k) >> 1) & 1, p.wait_ns, s_late);
        carry = not_a_number();
        for (int t = t0 + warp * ROWS; on && t < el.len; t += per)
            for (int i = 0; i < min(ROWS, el.len - t); ++i) {
                const long long at = (long long)el.row(t + i) * a.C;
                store<T, VEC>(dx + at, carry);
                store<T, VEC>(dgate + at, carry);
            }
    }
    if (!on) return;
    clear<T, VEC>(dx, a.C, rounds * per, a.N, rank * WARPS + warp, ctas * WARPS);
    clear<T, VEC>(dgate, a.C, rounds * per, a.N, rank * WARPS + warp, ctas * WARPS);
    if (p.dstate && rank == 0 && warp == 0) store_f32<VEC>(p.dstate + bc, carry);
}

// A few new samples: a thread has its channels' positions from first to last, all of them on their way at once (64 x 1 x 1024 bf16:
// 1.7 us, by the scan 12.4; 4096 x 8 x 1024: 39 us, 681). Their backward pass is the scan's: 19 and 1070 us.
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

template <auto Kernel> cudaError_t launch_clusters(long long clusters, int ctas, int warps, size_t images, size_t totals, cudaStream_t s, const RecurrenceParams& p,
                                                  const RecurrenceMaps& maps)
{
    if (const cudaError_t e = allow_smem<Kernel>(images + kMostCtas * totals); e != cudaSuccess) return e;
    if (ctas > 8)
        if (const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ctas, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.gridDim = dim3((unsigned)(clusters * ctas)), c.blockDim = dim3(warps * 32), c.stream = s, c.attrs = &at, c.numAttrs = ctas > 1 ? 1 : 0;
    c.dynamicSmemBytes = images + (ctas > 1 ? ctas * totals : 0);
    return cudaLaunchKernelEx(&c, Kernel, p, maps, ctas);
}

bool map_positions(CUtensorMap* m, const RecurrenceParams& p, const void* base, long long batch, long long row, int channels, int positions)
{
    const sdtw_recurrence& a = p.a;
    const int size = dtype_size(a.dtype);
    const cuuint64_t dims[3] = {(cuuint64_t)a.C, (cuuint64_t)a.N, (cuuint64_t)(batch ? a.B : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)(a.N > 1 ? row * size : 16), (cuuint64_t)(a.B > 1 && batch ? batch * size : 16)};
    const cuuint32_t box[3] = {(cuuint32_t)channels, (cuuint32_t)positions, 1};
    return atc::encode(m, a.dtype, 3, base, dims, strides, box, false);
}

constexpr int kFewRows = 8;

template <typename T, int VEC, int ROWS, int WARPS, bool RING, int TIED> cudaError_t run_warps(const RecurrenceParams& p, bool backward, int ctas, cudaStream_t s)
{
    const sdtw_recurrence& a = p.a;
    const long long clusters = (long long)a.B * ((a.C + 32 * VEC - 1) / (32 * VEC));
    constexpr size_t image = RING ? WARPS * ROWS * 32 * VEC * sizeof(T) : 0;
    const size_t images = (backward ? 2 * 3 : kStages * 2) * image, totals = sizeof(Run) * 2 * 32;   // of a CTA of the cluster
    RecurrenceMaps maps{};
    if (RING) {
        maps.x_batch = a.x_stride[0] != 0, maps.gate_batch = a.gate_stride[0] != 0;
        if (!map_positions(&maps.x, p, a.x, a.x_stride[0], a.x_stride[1], 32 * VEC, WARPS * ROWS) ||
            !map_positions(&maps.gate, p, a.gate, a.gate_stride[0], a.gate_stride[1], 32 * VEC, WARPS * ROWS) ||
            (p.dh && !map_positions(&maps.dh, p, p.dh, (long long)a.N * a.C, a.C, 32 * VEC, WARPS * ROWS)) ||
            (!backward && !map_positions(&maps.h, p, p.h, (long long)a.N * a.C, a.C, 32 * VEC, WARPS * ROWS)))
            return cudaErrorInvalidValue;
    }
    if (backward) return launch_clusters<recurrence_bwd_kernel<T, VEC, ROWS, WARPS, RING, TIED>>(clusters, ctas, WARPS, images, totals, s, p, maps);
    return launch_clusters<recurrence_fwd_kernel<T, VEC, ROWS, WARPS, RING, TIED>>(clusters, ctas, WARPS, images, totals, s, p, maps);
}
// How many clusters of 2^i CTAs can be resident at once; asked once per device.
template <auto Kernel> int resident(int i, int threads, size_t smem)
{
    static std::atomic<int> known[8][5];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::atomic<int>* place = dev < 8 ? &known[dev][i] : nullptr;
    if (place && (n = place->load(std::memory_order_relaxed)) > 0) return n - 1;
    if (allow_smem<Kernel>(smem) != cudaSuccess || (i > 3 && cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess))
        return 0;
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 1u << i, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.gridDim = dim3(1u << i), c.blockDim = dim3((unsigned)threads), c.dynamicSmemBytes = smem, c.attrs = &at, c.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, Kernel, &c) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (place) place->store(n + 1, std::memory_order_relaxed);
    return n;
}

// Few clusters of long series are of CTAs of sixteen warps, one an SM, sixteen CTAs to a cluster or eight, where all are resident at
// once: what a round costs, some 2 us whatever its size, then comes least often (2 x 16383 x 264 fp16, ten clusters of eight:
// 24.0 and 39.7 us, with eight warps 29.0 and 43.3; 1 x 8192 x 768 fp32 20.3 and 32.7, 25.8 and 34.3). Four such CTAs lose to eight of
// eight warps, with as many positions (2 x 8192 x 640 bf16: 22.8 and 40.6 us for 21.1 and 36.5), and so do they all where one round is
// enough (1 x 1024 x 64 bf16: 6.4 us for 5.0). Many clusters take two CTAs of eight warps an SM, as many to a cluster as all find such
// places: those of a second turn would run by themselves (bf16 forward with 1, 2, 4 and 8 CTAs: 4 x 8192 x 1024 82, 54, 40 and 46 us, 16 x
// 8192 x 1024 130, 144, 141 and 162; the former with sixteen warps in fp32, backward, 121 for 97).
template <typename T, int VEC, int ROWS, bool RING, int TIED> cudaError_t run_rows(const RecurrenceParams& p, bool backward, int sms, cudaStream_t s)
{
    const sdtw_recurrence& a = p.a;
    const long long clusters = (long long)a.B * ((a.C + 32 * VEC - 1) / (32 * VEC));
    if constexpr (RING) {
        constexpr size_t image = 16 * ROWS * 32 * VEC * sizeof(T), totals = sizeof(Run) * 2 * 32;
        for (int i = 4; i >= 3 && 8 * clusters <= sms && a.N > 64 * ROWS; --i) {
            if (8ll * ROWS << i >= a.N) continue;              // half as many would do
            const int n = backward ? resident<recurrence_bwd_kernel<T, VEC, ROWS, 16, RING, TIED>>(i, 512, 6 * image + kMostCtas * totals)
                                   : resident<recurrence_fwd_kernel<T, VEC, ROWS, 16, RING, TIED>>(i, 512, 2 * kStages * image + kMostCtas * totals);
            if (clusters <= n) return run_warps<T, VEC, ROWS, 16, RING, TIED>(p, backward, 1 << i, s);
        }
    }
    int k = 1;
    while (k < 8 && clusters * 2 * k <= 2ll * sms && 8ll * ROWS * k < a.N) k *= 2;
    return run_warps<T, VEC, ROWS, 8, RING, TIED>(p, backward, k, s);
}
template <typename T, int VEC> cudaError_t run_few(const RecurrenceParams& p, cudaStream_t s)
{
    const long long threads = (long long)p.a.B * ((p.a.C + VEC - 1) / VEC);
    if (p.a.N == 1) recurrence_few_kernel<T, VEC, 1><<<(unsigned)((threads + 127) / 128), 128, 0, s>>>(p);
    else recurrence_few_kernel<T, VEC, kFewRows><<<(unsigned)((threads + 127) / 128), 128, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t run(const RecurrenceParams& p, bool backward, int sms, cudaStream_t s)
{
    const sdtw_recurrence& a = p.a;
    auto on = [](const void* q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) == 0; };
    auto strides = [&](int n) {
        return a.C % n == 0 && a.x_stride[0] % n == 0 && a.x_stride[1] % n == 0 && a.gate_stride[0] % n == 0 && a.gate_stride[1] % n == 0;
    };
    constexpr int pack = 16 / sizeof(T);
    bool pairs = strides(2) && on(a.x, 2 * sizeof(T)) && on(a.gate, 2 * sizeof(T)) && on(a.state, 8);
    pairs = pairs && (backward ? on(p.dh, 2 * sizeof(T)) && on(p.dx, 2 * sizeof(T)) && on(p.dgate, 2 * sizeof(T)) && on(p.dlast, 8) && on(p.dstate, 8) && on(p.kept_in, 8)
                               : on(p.h, 2 * sizeof(T)) && on(p.last, 8) && on(p.kept, 8));
    if (!backward && a.N <= kFewRows) return pairs ? run_few<T, 2>(p, s) : run_few<T, 1>(p, s);
    bool ring = pairs && strides(pack) && on(a.x, 16) && on(a.gate, 16) && on(p.dh, 16) && on(p.h, 16);
    for (const long long* st : {a.x_stride, a.gate_stride})
        ring = ring && (a.N == 1 || st[1] > 0) && (a.B == 1 || (st[0] >= 0 && st[0] < (1ll << 36)));   // as tensor maps have them
    if (!ring) return run_rows<T, 1, 8, false, -1>(p, backward, sms, s);
    constexpr int ROWS = sizeof(T) == 4 ? 8 : 16;
    return a.tied ? run_rows<T, 2, ROWS, true, 1>(p, backward, sms, s) : run_rows<T, 2, ROWS, true, 0>(p, backward, sms, s);
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

cudaError_t recurrence_take_status(int* out, cudaStream_t s)
{
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e;
}

}  // namespace sdtw
