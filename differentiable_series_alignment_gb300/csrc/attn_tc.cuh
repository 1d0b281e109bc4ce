// attn_tc.cuh -- what the tensor-core attention kernels share: tensor maps of packed
// rows and of keys, operand descriptors, bounded waits, and packed 16-bit conversions.
//
// Operands sit in shared memory as TMA writes them: boxes of 64 features (128 bytes,
// 128-byte swizzle) by up to 128 rows, 16 KB apart. One image serves both ways round: as a
// K-major operand of a product over the features, and as an MN-major operand (features
// along N) of a product over the rows. Probabilities are A operands from tensor memory.
#pragma once

#include <cuda.h>

#include "encoder.h"
#include "packed.cuh"
#include "tc.cuh"

namespace sdtw {
namespace atc {

using namespace tc;

constexpr int kKeys = 128;            // keys per tile
constexpr uint32_t kBox = 128 * 128;  // bytes of a 128-row box of 64 16-bit features
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---- instruction and operand descriptors (kind::f16, fp32 accumulation)
template <typename T> struct Fmt;
template <> struct Fmt<__half> { static constexpr uint32_t v = 0; };
template <> struct Fmt<__nv_bfloat16> { static constexpr uint32_t v = 1; };

template <typename T> __device__ __forceinline__ uint32_t idesc(int M, int N, bool b_mn) {
    return (1u << 4) | (Fmt<T>::v << 7) | (Fmt<T>::v << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// MN-major, 128-byte swizzle: 64-element groups along N a box apart, 8-row groups along
// K 1 KiB apart. sdesc (tc.cuh) is the K-major form of the same image.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(kBox >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    mma_bf16(d, a, b, id, acc);   // kind::f16: the types are in the instruction descriptor
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(id), "r"(acc));
}

// One thread of a converged warp. The compiler knows that elect.sync leaves one thread, and
// keeps the operands of the products that it issues in uniform registers; behind a
// comparison of lane numbers every product cost about 150 cycles to issue, more than the 64
// that it takes to run.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

// A value that every lane of the warp holds alike, made known as such to the compiler: what
// the issuing warp computes with then stays in uniform registers, as its products' operands
// have to be.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// D[128 x N] = A[128 x features] B[N x features]^T over `steps` <= MAX steps of 16 features, both
// K-major images; N of id.
template <int MAX>
__device__ __forceinline__ void mma_features(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t id) {
    const uint64_t ad = sdesc(a), bd = sdesc(b);
#pragma unroll
    for (int s = 0; s < MAX; ++s) {
        const uint32_t o = ((uint32_t)(s >> 2) * kBox + (uint32_t)(s & 3) * 32) >> 4;   // the address field counts 16 bytes
        if (s < steps) mma_ss(d, ad + o, bd + o, id, s > 0 ? 1u : 0u);
    }
}

// ---- TMA
__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tma5(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, int c4,
                                     uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}
template <int DP>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* m, int n0, int hk, int b, uint32_t bar) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) tma5(dst + c * kBox, m, c * 64, 0, hk, n0, b, bar);
}
template <int DP>
__device__ __forceinline__ void load_keys(uint32_t dst, const CUtensorMap* m, int j0, int hk, int b, uint32_t bar) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) tma4(dst + c * kBox, m, c * 64, j0, hk, b, bar);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// One warp clears rows [from, to) of an image that a product over its rows is about to read: what lies
// beyond a sequence's length, or in rows that see no key, may be NaN, and 0 * NaN is not 0.
template <int DP> __device__ __forceinline__ void clear_rows(uint32_t img, int from, int lane, int to = 128) {
    for (int c = 0; c < DP / 64; ++c)
        for (uint32_t o = (uint32_t)from * 128 + lane * 16; o < (uint32_t)to * 128; o += 512)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(img + c * kBox + o), "r"(0) : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// ---- waits: bounded. After one that ran out the caller waits no more, and since it may then give others what is not
// there, or not yet, the whole CTA's results become NaN: whoever writes them asks `cta` when its own last
// wait is over. The status word is set too.
struct Late {
    int* status;   // of the device
    int* cta;      // shared memory, 0 at first
    __device__ __forceinline__ void set() const {
        atomicOr(status, kStatusTimeout);
        *static_cast<volatile int*>(cta) = 1;
        __threadfence_block();
    }
    // by a whole warp
    __device__ __forceinline__ bool any() const { return __any_sync(0xffffffffu, *static_cast<volatile int*>(cta) != 0); }
};

__device__ __forceinline__ void wait_for(bool& ok, uint32_t bar, uint32_t parity, unsigned long long limit_ns, const Late& late) {
    if (!ok || mbar_test(bar, parity)) return;
    const unsigned long long t0 = global_ns();
    while (!mbar_test(bar, parity)) {
        if (global_ns() - t0 > limit_ns) {
            late.set();
            ok = false;
            return;
        }
    }
}

// The same by a whole warp, which learns one answer.
__device__ __forceinline__ void wait_warp(bool& ok, uint32_t bar, uint32_t parity, unsigned long long limit_ns, const Late& late) {
    wait_for(ok, bar, parity, limit_ns, late);
    ok = __all_sync(0xffffffffu, ok);
}

// ---- tensor memory
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 32 rows of F features (a lane a row) through shared memory to their places in global
// memory, a whole row's 16-byte pieces by neighbouring lanes: stored straight from the lanes
// that hold them, 32 rows at a time, results took 7000 cycles of a CTA's end. `area` is
// 32 * F * 2 bytes of the warp's own; `at` is the row's place in elements, or < 0.
template <int F> __device__ __forceinline__ uint32_t stage_at(uint32_t area, int row, int piece) {
    return area + row * (F * 2) + ((piece ^ (F == 64 ? row & 7 : (row >> 1) & 3)) << 4);
}
template <int F> __device__ __forceinline__ void stage_out(uint32_t area, void* out, long long at, int pieces, int lane) {
    constexpr int PER = F / 8;
    __syncwarp();
    const int c = lane % PER;
#pragma unroll 2
    for (int i = 0; i < PER; ++i) {
        const int row = i * (32 / PER) + lane / PER;
        const long long o = __shfl_sync(0xffffffffu, at, row);
        if (o < 0 || c >= pieces) continue;
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(stage_at<F>(area, row, c)));
        reinterpret_cast<uint4*>(static_cast<unsigned char*>(out) + o * 2)[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t* w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
// 16 columns of an accumulator in tensor memory from `col`, times mul, and (other) of the one 128
// columns on, times mul1.
__device__ __forceinline__ void read_acc(uint32_t col, bool read, bool other, float mul, float mul1, float (&o)[16]) {
    if (read) {
        tmem_ld16(col, o);
    } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) o[q] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) o[q] *= mul;
    if (other) {
        float x[16];
        tmem_ld16(col + 128, x);
#pragma unroll
        for (int q = 0; q < 16; ++q) o[q] = fmaf(x[q], mul1, o[q]);
    }
}
// F features of an accumulator (this lane's row, from column col) times mul, and more (apart, so
// that neither overflows), rounded into out and, where it is wanted, what the rounding left into
// rest; `zero`: the row is 0 whatever the accumulator holds. area: 32 * F * 2 bytes, twice that
// with rest.
template <typename T, int F>
__device__ __forceinline__ void write_rows(uint32_t area, uint32_t col, bool read, bool other, bool zero, float mul, float mul1,
                                           float more, void* out, void* rest, long long at, int pieces, int lane) {
#pragma unroll 1   // run once a CTA: what counts is how much code there is to fetch
    for (int f = 0; f < F; f += 16) {
        float o[16];
        read_acc(col + f, read, other, mul, mul1, o);
#pragma unroll
        for (int q = 0; q < 16; q += 8) {
            uint32_t w[4], z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x = zero ? 0.f : o[q + 2 * k] * more, y = zero ? 0.f : o[q + 2 * k + 1] * more;
                w[k] = pack2<T>(x, y);
                if (rest) {
                    const Halves<T> h(w[k]);
                    z[k] = pack2<T>(x - to_f32(h.e[0]), y - to_f32(h.e[1]));
                }
            }
            st_shared16(stage_at<F>(area, lane, (f + q) / 8), w);
            if (rest) st_shared16(stage_at<F>(area + 32 * F * 2, lane, (f + q) / 8), z);
        }
    }
    stage_out<F>(area, out, at, pieces, lane);
    if (rest) stage_out<F>(area + 32 * F * 2, rest, at, pieces, lane);
}
// The same in fp32, F features of 4 bytes in an area of 32 * F * 4 bytes: F / 2 16-bit places.
template <int F>
__device__ __forceinline__ void write_rows_f32(uint32_t area, uint32_t col, bool read, bool other, bool zero, float mul, float mul1, float* out,
                                               long long at, int pieces, int lane) {
#pragma unroll 1
    for (int f = 0; f < F; f += 16) {
        float o[16];
        read_acc(col + f, read, other, mul, mul1, o);
#pragma unroll
        for (int q = 0; q < 16; q += 4) {
            uint32_t w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) w[z] = __float_as_uint(zero ? 0.f : o[q + z]);
            st_shared16(stage_at<2 * F>(area, lane, (f + q) / 4), w);
        }
    }
    stage_out<2 * F>(area, out, at < 0 ? at : 2 * at, pieces, lane);
}

// Key tiles [lo, hi) that the packed rows [r0, r1) see.
struct Tiles {
    int lo, hi;
    __device__ __forceinline__ Tiles(const RowRange& rr, int r0, int r1, int G) : lo(0), hi(0) {
        const int n0 = r0 / G, n1 = min((r1 - 1) / G, rr.n_b - 1);
        if (r0 >= r1 || n0 > n1) return;
        const int a = rr.lo(n0), b = rr.hi(n1);
        if (a >= b) return;
        lo = a / kKeys;
        hi = (b + kKeys - 1) / kKeys;
    }
};

// ---- host: tensor maps
// A map with the 128-byte swizzle, or with rows as they are; strides in bytes, of all dimensions but the first.
bool encode(CUtensorMap* m, int dtype, int rank, const void* p, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, bool swizzled = true);
struct Maps {
    CUtensorMap q, k, v, dout;
};

// Packed rows of a (B, N, Hq, D) tensor: (features, head in group, key head, position, batch).
// RT rows per load.
bool map_rows(CUtensorMap* m, const void* p, const long long* stride, const sdtw_attention& a, int G, int RT);
// Keys of a (B, M, Hkv, D) tensor: (features, position, key head, batch).
bool map_keys(CUtensorMap* m, const void* p, const long long* stride, const sdtw_attention& a);

}  // namespace atc
}  // namespace sdtw
