// gated_tc.cuh -- the products of gated linear units on the tensor cores (tcgen05), one kernel for all of them:
//
//   FWD   h = act(x Wg^T + bg) * (x Wu^T + bu)       rows of x by features f, both products side by side in one tile
//   GRAD  the same two products again, and from them and dh: dg and du, rounded to the operands' type
//   DX    dx = dg Wg + du Wu                          one sum over the features f of both
//   DW    dWg = dg^T x, dWu = du^T x                  sums over the rows
//
// Operands are 16 bits. They come by TMA in blocks of 64 along the sum, 128 bytes a row with the 128-byte swizzle; what
// a tensor map leaves out (rows, features, the tail of the sum) arrives as zeros. x, dg and W lie along their rows, so
// that a sum over features has K-major operands and a sum over rows MN-major ones: no operand is transposed in memory.
// fp32 operands are split into three bf16 parts, v = v0 + v1 + v2 to 24 bits, and a product is the sum of the six part products
// above 2^-24 of it, (0,2) (2,0) (1,1) (0,1) (1,0) (0,0), smallest first. A block of either operand comes with all its parts. The
// tensor cores cut off what an addition leaves below the accumulator's last bit, always towards 0: over a sum of 6000 terms
// that came to 250 times the result's own rounding. Sums of fp32 so leave the accumulator after every block of 64 terms and
// are added up in registers, rounded to nearest.
//
// A persistent CTA: a loading warp, an issuing warp, and eight warps that turn a finished accumulator into results while
// the next one is summed (two accumulators in tensor memory). Large calls take pairs of CTAs (cta_group::2) with 256 rows and 256
// columns of accumulator to a tile: each CTA has 128 of the rows and loads half of the other operand, which both use. The
// first of a pair issues for both.
//
// Measured, 16384 x 1024 to 4096 bf16: FWD 140 us (1960 TFLOP/s; a library's product of x with both weights alone 143),
// GRAD 150, DX 178, DW 182 in a backward pass of 514. The tensor pipe bounds them, and the power that it takes: one at a time, 2048 to
// 2048 features, FWD, GRAD and DX run in 147, 152 and 148 us with the pipe 85 % busy. fp32, 16384 x 64 to 256: 18 us forward, 65 backward, bound by the
// epilogue of two blocks of sum (three parts of dg and du are written) and the launches around it.
#pragma once
#include <algorithm>
#include <type_traits>

#include "activation.cuh"
#include "attn_tc.cuh"
#include "block.h"

namespace sdtw {
namespace gtc {

using namespace atc;

enum Kind { FWD, GRAD, DX, DW };

constexpr int kRows = 128, kBlock = 64;               // rows of a tile; length of a block of the sum
constexpr uint32_t kABytes = kRows * kBlock * 2;

// One piece of the sum: the first part of A. The first piece takes the first map of B, the second the other.
struct Seg {
    unsigned char a;
};

struct Params {
    CUtensorMap a, b[2];
    Seg seg[2];
    int segs, blocks;                                  // the sum: segs pieces of `blocks` blocks
    bool grouped_a, grouped_b;                         // maps of MN-major operands have groups of 64 columns as a dimension
    int tiles_m, tiles_n, group, set0, sets, tiles;    // sets: DW's weights, from set0 on
    int whole, cuts;                                   // tiles summed whole; pieces of the others' sums, or 0 (below)
    long long M;                                       // rows and columns of the result
    int N, F, activation;
    void* out[2];                                      // FWD h; DX dx; DW both weights' gradients
    const void *bias[2], *dh;
    // GRAD: dg and du, rounded, as parts 0 .. parts - 1 and parts .. 2 parts - 1 of (2 parts, M, ld)
    uint16_t* grads;
    long long ld;
    float* sums;                                       // GRAD, with biases: [M / 32][2 F] column sums of 32 rows
    float* shares;                                     // DX, DW: [cuts][tiles not summed whole][rows of a tile][its columns]
    const unsigned* top;                               // fp16: what dg and du are scaled by (grads_scale)
    unsigned long long wait_ns;
    int skip;                                          // test hook: nothing is loaded
};

// the operands' type
template <typename T> struct Operand { using type = T; };
template <> struct Operand<float> { using type = __nv_bfloat16; };
template <typename T> constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
template <typename T> constexpr int kRun = sizeof(T) == 4 ? 1 : 1 << 30;   // blocks that one accumulator takes

template <int NB, int PARTS> struct Shape {
    static constexpr int ctas = NB == 256 ? 2 : 1;     // that share a tile
    static constexpr uint32_t b_bytes = NB / ctas * kBlock * 2, stage = PARTS * (kABytes + b_bytes);   // of a CTA
    static constexpr uint32_t area = 4096;             // of shared memory, a warp's own
    static constexpr int stages = PARTS > 1 ? 2 : NB == 64 ? 7 : 6;
    static constexpr uint32_t smem = stages * stage + 8 * area;
    static constexpr int columns = 2 * NB;             // of tensor memory
    static constexpr int rows = ctas * kRows;          // of a tile
};

constexpr int kLoad = 8, kIssue = 9, kThreadsG = 320;

static __device__ int g_status;   // of this file's kernels

__device__ __forceinline__ bool aligned16_dev(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// The same by a CTA of a pair, reported to the first one's barrier
__device__ __forceinline__ void tma3_pair(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma4_pair(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
// Rows [row, row + 64) of `groups` groups of 64 columns from col on, a group after the other: one copy where the columns are whole
// groups, which the map then has as a dimension of their own.
template <int CTAS, int GROUPS> __device__ __forceinline__ void load_groups(uint32_t dst, const CUtensorMap* m, bool grouped, int col, int row, int part, uint32_t bar) {
    if (grouped) {
        if constexpr (CTAS == 2) tma4_pair(dst, m, 0, row, col / 64, part, bar);
        else tma4(dst, m, 0, row, col / 64, part, bar);
    } else {
#pragma unroll
        for (int c = 0; c < GROUPS; ++c) {
            if constexpr (CTAS == 2) tma3_pair(dst + c * kBlock * 128, m, col + c * 64, row, part, bar);
            else tma3(dst + c * kBlock * 128, m, col + c * 64, row, part, bar);
        }
    }
}
template <int CTAS> __device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar) {
    if constexpr (CTAS == 2) tma3_pair(dst, m, c0, c1, c2, bar);
    else tma3(dst, m, c0, c1, c2, bar);
}
template <int CTAS> __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(acc));
    else mma_ss(d, a, b, id, acc);
}
// of a pair: reported to both
template <int CTAS> __device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"((uint16_t)3)
                     : "memory");
    else mma_commit(bar);
}
template <int CTAS> __device__ __forceinline__ void alloc(uint32_t* to, int columns) {
    if constexpr (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(to, columns);
    }
}
template <int CTAS> __device__ __forceinline__ void dealloc(uint32_t tmem, int columns) {
    if constexpr (CTAS == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
    else tmem_dealloc(tmem, columns);
}
// All threads of the CTA, or of the pair, have come here.
template <int CTAS> __device__ __forceinline__ void meet() {
    if constexpr (CTAS == 2) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
}
__device__ __forceinline__ uint32_t in_cta(uint32_t mine, int cta) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(cta));
    return there;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {   // of this cluster
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ int cta_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// MN-major blocks of 64 rows: groups of 64 elements 8 KB apart
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((kBlock * 128) >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
template <typename T> __device__ __forceinline__ uint32_t idesc2(int M, int N, bool a_mn, bool b_mn) {
    return idesc<T>(M, N, b_mn) | ((a_mn ? 1u : 0u) << 15);
}

// A tile's place. Tiles of a column follow one another in groups of some rows of tiles, so that those in work at a time are
// a block of about nine columns, or all of fewer, and share their operands in the cache: 8192 x 2048 from 2 x 4096 features read
// 397 MB from memory in groups of 16 rows, three times what there is.
struct Tile {
    int m, n, set, first, last;   // blocks [first, last) of the sum
    int share;                    // where a part of a sum goes, or -1
    __device__ __forceinline__ void place(const Params& p, int t) {
        const int per = p.tiles_m * p.tiles_n;
        set = t / per;
        t -= set * per;
        set += p.set0;
        const int G = p.group, group = t / (G * p.tiles_n), rows = min(G, p.tiles_m - group * G), in = t - group * G * p.tiles_n;
        n = in / rows;
        m = group * G + in - n * rows;
    }
};
// What a worker (a CTA, or a pair) does: every workers-th of the whole tiles, as many as all have alike, and of the pieces of the
// sums of those that are left. A piece's tiles follow one another, so that workers read the same rows of an operand at the same
// time: where each worker had a range of its own of one tile's sum, DW of 16384 x 1024 to 4096 read dg twice and a half and took 218 us
// for 182. Pieces go to memory in fp32 and are added up, in their order, by a launch of their own.
struct Work {
    const Params& p;
    int t, stride, left;
    __device__ __forceinline__ Work(const Params& p_, int worker, int workers) : p(p_), t(worker), stride(workers), left(p_.tiles - p_.whole) {}
    __device__ __forceinline__ bool next(Tile& tile) {
        const int total = p.segs * p.blocks;
        if (t < p.whole) {
            tile.place(p, t);
            tile.first = 0, tile.last = total, tile.share = -1;
        } else {
            const int q = t - p.whole, cut = p.cuts ? q / left : 1;
            if (cut >= p.cuts) return false;
            tile.place(p, p.whole + q - cut * left);
            tile.first = (int)((long long)total * cut / p.cuts), tile.last = (int)((long long)total * (cut + 1) / p.cuts);
            tile.share = q;
        }
        t += stride;
        return true;
    }
};

// ---- 32 rows by 32 columns between a warp's registers (a lane a row) and memory, through its own shared memory, so that
// neighbouring lanes read and write neighbouring addresses
template <typename O> __device__ __forceinline__ uint32_t chunk_at(uint32_t area, int row, int piece) {
    if constexpr (sizeof(O) == 4) return area + row * 128 + ((piece ^ (row & 7)) << 4);
    else return area + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}
template <typename O> __device__ __forceinline__ uint32_t element_at(uint32_t area, int row, int c) {
    constexpr int E = 16 / sizeof(O);
    return chunk_at<O>(area, row, c / E) + (c % E) * sizeof(O);
}
template <typename O> __device__ __forceinline__ void words_of(const float* v, uint32_t (&w)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(O) == 4) w[k] = __float_as_uint(v[k]);
        else w[k] = pack2<O>(v[2 * k], v[2 * k + 1]);
    }
}
// rows and cols: how many of either there are; vec: 16-byte accesses are aligned
template <typename O>
__device__ __forceinline__ void put_chunk(uint32_t area, const float (&v)[32], O* out, long long ld, int rows, int cols, bool vec, int lane)
{
    constexpr int E = 16 / sizeof(O), P = 32 / E;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < P; ++q) {
        uint32_t w[4];
        words_of<O>(v + q * E, w);
        st_shared16(chunk_at<O>(area, lane, q), w);
    }
    __syncwarp();
    if (vec && cols % E == 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int row = i * (32 / P) + lane / P, q = lane % P;
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(chunk_at<O>(area, row, q)));
            if (row < rows && q * E < cols) *reinterpret_cast<uint4*>(out + row * ld + q * E) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll 4
        for (int row = 0; row < rows; ++row)
            if (lane < cols) {
                if constexpr (sizeof(O) == 4) {
                    uint32_t w;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(element_at<O>(area, row, lane)));
                    out[row * ld + lane] = __uint_as_float(w);
                } else {
                    uint16_t w;
                    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(element_at<O>(area, row, lane)));
                    reinterpret_cast<uint16_t*>(out)[row * ld + lane] = w;
                }
            }
    }
}
// A lane's row
template <typename O> __device__ __forceinline__ void read_chunk(uint32_t area, float (&v)[32], int lane) {
    constexpr int E = 16 / sizeof(O), P = 32 / E;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        uint32_t u[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                     : "r"(chunk_at<O>(area, lane, q)));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(O) == 4) {
                v[q * E + k] = __uint_as_float(u[k]);
            } else {
                const Halves<O> h(u[k]);
                v[q * E + 2 * k] = to_f32(h.e[0]);
                v[q * E + 2 * k + 1] = to_f32(h.e[1]);
            }
        }
    }
}
// Element by element; what is not there is 0.
template <typename O>
__device__ __forceinline__ void get_chunk(uint32_t area, float (&v)[32], const O* in, long long ld, int rows, int cols, int lane)
{
    using Bits = typename std::conditional<sizeof(O) == 4, uint32_t, uint16_t>::type;
    __syncwarp();
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 8) {   // eight rows on their way at a time
        Bits w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = r0 + i < rows && lane < cols ? reinterpret_cast<const Bits*>(in)[(r0 + i) * ld + lane] : Bits(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(O) == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(element_at<O>(area, r0 + i, lane)), "r"(w[i]) : "memory");
            else asm volatile("st.shared.b16 [%0], %1;" ::"r"(element_at<O>(area, r0 + i, lane)), "h"(w[i]) : "memory");
        }
    }
    __syncwarp();
    read_chunk<O>(area, v, lane);
}
// The same of aligned 16 bytes, in two steps: on their way to the area, and taken from there.
template <typename O> __device__ __forceinline__ void ask_chunk(uint32_t area, const O* in, long long ld, int rows, int cols, int lane) {
    constexpr int E = 16 / sizeof(O), P = 32 / E;
    __syncwarp();   // everyone has taken what was there
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int row = i * (32 / P) + lane / P, q = lane % P;
        const bool there = row < rows && q * E < cols;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(chunk_at<O>(area, row, q)), "l"(there ? in + row * ld + q * E : in),
                     "r"(there ? 16 : 0)
                     : "memory");
    }
}
template <typename O> __device__ __forceinline__ void take_chunk(uint32_t area, float (&v)[32], int lane) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    read_chunk<O>(area, v, lane);
}
// Sums over the 32 lanes of each of v's entries; lane l receives that of entry l. 31 shuffles in a fixed order.
__device__ __forceinline__ float column_sums(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const bool up = lane & o;
            const float other = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + o], o);
            v[j] = (up ? v[j + o] : v[j]) + other;
        }
    return v[0];
}

// Lane l has the bias of column l.
__device__ __forceinline__ void add_bias(float (&v)[32], float bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, bias, j);
}

// h in place of g, or with dh the gradients of g and u in their places
template <int ACT, bool EXACT, bool GRADS> __device__ __forceinline__ void gate32(float (&g)[32], float (&u)[32], const float (&d)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        float slope;
        const float v = activate<ACT, EXACT, GRADS>(g[j], slope);
        if (GRADS) {
            g[j] = d[j] * u[j] * slope;
            u[j] = d[j] * v;
        } else {
            g[j] = v * u[j];
        }
    }
}
template <bool EXACT, bool GRADS> __device__ __forceinline__ void gate_by(int activation, float (&g)[32], float (&u)[32], const float (&d)[32]) {
    switch (activation) {
        case SDTW_ACT_SILU: gate32<SDTW_ACT_SILU, EXACT, GRADS>(g, u, d); break;
        case SDTW_ACT_GELU: gate32<SDTW_ACT_GELU, EXACT, GRADS>(g, u, d); break;
        case SDTW_ACT_RELU: gate32<SDTW_ACT_RELU, EXACT, GRADS>(g, u, d); break;
        default: gate32<SDTW_ACT_SIGMOID, EXACT, GRADS>(g, u, d); break;
    }
}

// fp16 keeps dg and du times a power of two, so that as much of what they are ends neither beyond 65504 nor among the subnormal
// numbers as its range allows. |u| <= |x| |Wu| + |bu| by the rows' norms, |g| alike, |act(g)| <= |g| (a sigmoid's: 1) and the slopes are
// at most 1.13: |dg| and |du| are below |dh| (1.13 |u| + |act(g)|), which comes to [2^14, 2^15). Values 2^-28 of that still have all their
// bits. The bound is some sqrt(K) / 4 above what there is. By the largest |dh| alone, brought to [1/4, 1/2), one entry
// of 2000 among 1e-2 left the other rows' dx 30 times as far off as their rounding.
// top: bits of the largest |dh|, of the largest squared norm of a row of x, Wg and Wu, of the largest |bg| and |bu|.
constexpr int kTops = 6;
__device__ __forceinline__ float grads_scale(const unsigned* top, int activation) {
    auto at = [&](int i) { return __uint_as_float(top[i]); };
    const float dh = at(0), g = sqrtf(at(1) * at(2)) + at(4), u = sqrtf(at(1) * at(3)) + at(5);
    const float most = dh * (1.13f * u + (activation == SDTW_ACT_SIGMOID ? fmaxf(g, 1.f) : g));
    int exponent = 0;
    if (most > 0.f && most < INFINITY) {
        frexpf(most, &exponent);
        return ldexpf(1.f, 15 - exponent);
    }
    if (!(dh > 0.f && dh < INFINITY)) return 1.f;
    frexpf(dh, &exponent);   // infinities and NaN among the operands: the others' results may still be finite
    return ldexpf(1.f, -1 - exponent);
}

// T: the call's type. NB: columns of the accumulator; FWD and GRAD have NB / 2 features of either product in them.
template <int KIND, typename T, int NB>
__global__ void __launch_bounds__(kThreadsG, 1) gated_tc_kernel(const __grid_constant__ Params p)
{
    constexpr int PARTS = kParts<T>;
    using Sh = Shape<NB, PARTS>;
    using O = typename Operand<T>::type;
    constexpr bool PAIR = KIND == FWD || KIND == GRAD, A_MN = KIND == DW, B_MN = KIND == DX || KIND == DW;
    constexpr int WIDTH = PAIR ? NB / 2 : NB;             // columns of a tile's result
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ uint64_t s_full[Sh::stages], s_empty[Sh::stages], s_done[2], s_free[2], s_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_late;
    const Late late{&g_status, &s_late};
    constexpr int CTAS = Sh::ctas;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, rank = CTAS == 2 ? uniform(cta_rank()) : 0;
    const int worker = blockIdx.x / CTAS, workers = gridDim.x / CTAS;
    if (warp == kLoad && lane == 0) {
        prefetch_map(&p.a), prefetch_map(&p.b[0]), prefetch_map(&p.b[1]);
        s_late = 0;
        for (int e = 0; e < Sh::stages; ++e) mbar_init(smem_u32(&s_full[e]), 1), mbar_init(smem_u32(&s_empty[e]), 1);
        for (int e = 0; e < 2; ++e) mbar_init(smem_u32(&s_done[e]), 1), mbar_init(smem_u32(&s_free[e]), 8 * CTAS);
        mbar_init(smem_u32(&s_end), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssue) alloc<CTAS>(&s_tmem, Sh::columns);
    fence_before_sync();
    meet<CTAS>();
    fence_after_sync();
    const uint32_t tmem = (uint32_t)uniform((int)s_tmem), ring = smem_u32(dyn);
    bool ok = true;

    if (warp == kLoad) {
        // The whole warp goes through the blocks and one elected thread sends: behind a comparison of lane numbers a block's
        // copies took longer to issue than its products to run.
        int sent = 0, e = 0;   // blocks, and the place of the next
        uint32_t parity = 1;   // of the place's last release; of the first round there is none
        Work work(p, worker, workers);
        for (Tile tile; ok && !p.skip && work.next(tile);) {
            const int row = uniform(tile.m * Sh::rows + rank * kRows), col = uniform(tile.n * (PAIR ? WIDTH : NB)), set = uniform(tile.set);
            const int last = uniform(tile.last), first = uniform(tile.first);
            int seg = first / p.blocks, block = first - seg * p.blocks;
            for (int k = first; k < last; ++k) {
                if (sent >= Sh::stages) wait_warp(ok, smem_u32(&s_empty[e]), parity, p.wait_ns, late);
                if (!ok) break;
                if (elect_one()) {
                    const int at = block * kBlock, first_a = seg ? p.seg[1].a : p.seg[0].a;
                    const CUtensorMap* map_b = seg ? &p.b[1] : &p.b[0];   // a sum of two pieces has a map for either
                    const uint32_t mine = smem_u32(&s_full[e]), bar = CTAS == 2 ? in_cta(mine, 0) : mine;
                    if (rank == 0) mbar_expect_tx(mine, CTAS * Sh::stage);
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t a = ring + e * Sh::stage + part * kABytes;
                        const uint32_t b = ring + e * Sh::stage + PARTS * kABytes + part * Sh::b_bytes;
                        if constexpr (A_MN) load_groups<CTAS, kRows / 64>(a, &p.a, p.grouped_a, row, at, first_a + set * PARTS + part, bar);
                        else load3<CTAS>(a, &p.a, at, row, first_a + part, bar);
                        if constexpr (PAIR && CTAS == 2) {   // the first CTA has the gate's weights, the second the others
                            load3<CTAS>(b, rank ? &p.b[1] : &p.b[0], at, col, part, bar);
                        } else if constexpr (PAIR) {
                            load3<CTAS>(b, &p.b[0], at, col, part, bar);
                            load3<CTAS>(b + Sh::b_bytes / 2, &p.b[1], at, col, part, bar);
                        } else {
                            load_groups<CTAS, NB / CTAS / 64>(b, map_b, p.grouped_b, col + rank * (NB / CTAS), at, part, bar);
                        }
                    }
                }
                __syncwarp();
                if (++block == p.blocks) block = 0, ++seg;
                if (++e == Sh::stages) e = 0, parity ^= 1;
                ++sent;
            }
        }
        // no copy may be writing shared memory when the CTA ends
        bool drained = true;   // a pair's are all reported to the first CTA, for which the second waits at the end
        for (int k = max(0, sent - Sh::stages); k < sent && rank == 0; ++k)
            wait_warp(drained, smem_u32(&s_full[k % Sh::stages]), (uint32_t)((k / Sh::stages) & 1), p.wait_ns, late);
    } else if (warp == kIssue) {
        const uint32_t id = idesc2<O>(Sh::rows, NB, A_MN, B_MN);
        int n = 0, e = 0;      // accumulators filled; the place of the next block
        uint32_t parity = 0;   // of its arrival
        Work work(p, worker, workers);
        for (Tile tile; ok && rank == 0 && work.next(tile);) {
            const int first = uniform(tile.first), last = uniform(tile.last);
            for (int k = first, in = 0; k < last; ++k) {   // in: of the run
                if (in == 0) {
                    if (n >= 2) wait_warp(ok, smem_u32(&s_free[n & 1]), (uint32_t)((n / 2 - 1) & 1), p.wait_ns, late);
                    fence_after_sync();
                }
                const uint32_t d = tmem + (n & 1) * NB;
                const bool ends = k == last - 1 || in == kRun<T> - 1;
                wait_warp(ok, smem_u32(&s_full[e]), parity, p.wait_ns, late);
                fence_after_sync();
                if (ok && elect_one()) {
                    // pairs of parts, the smallest products first
                    constexpr int PAIRS = PARTS == 3 ? 6 : 1, PA[6] = {0, 2, 1, 0, 1, 0}, PB[6] = {2, 0, 1, 1, 0, 0};
#pragma unroll
                    for (int q = 0; q < PAIRS; ++q) {
                        const uint32_t a = ring + e * Sh::stage + (PARTS == 3 ? PA[q] : 0) * kABytes;
                        const uint32_t b = ring + e * Sh::stage + PARTS * kABytes + (PARTS == 3 ? PB[q] : 0) * Sh::b_bytes;
                        const uint64_t ad = A_MN ? desc_mn(a) : sdesc(a), bd = B_MN ? desc_mn(b) : sdesc(b);
#pragma unroll
                        for (int s = 0; s < kBlock / 16; ++s)   // 16 of the sum: 32 bytes along a row, or 16 rows
                            mma<CTAS>(d, ad + s * (A_MN ? 128 : 2), bd + s * (B_MN ? 128 : 2), id, in > 0 || q > 0 || s > 0 ? 1u : 0u);
                    }
                    commit<CTAS>(smem_u32(&s_empty[e]));
                    if (ends) commit<CTAS>(smem_u32(&s_done[n & 1]));
                }
                __syncwarp();
                in = ends ? 0 : in + 1;
                n += ends;
                if (++e == Sh::stages) e = 0, parity ^= 1;
            }
        }
        // every MMA has read its operands and written its result before the CTA ends
        if (rank == 0) {
            if (elect_one()) commit<CTAS>(smem_u32(&s_end));   // by the thread that issued them
            __syncwarp();
            bool fin = true;
            wait_warp(fin, smem_u32(&s_end), 0, p.wait_ns, late);
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t area = ring + Sh::stages * Sh::stage + warp * Sh::area;
        const float up = std::is_same<T, __half>::value && p.top ? grads_scale(p.top, p.activation) : 1.f;
        const float down = 1.f / up;
        // 16-bit pieces of dh have half of the area to themselves; fp32's are taken before results are put there
        const uint32_t dh_area = sizeof(T) == 2 ? area + 2048 : area;
        const bool dh_packs = p.F % (16 / (int)sizeof(T)) == 0 && aligned16_dev(p.dh);
        // the accumulator has been read by this warp
        auto release = [&](int which) {
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (CTAS == 2) arrive_at(in_cta(smem_u32(&s_free[which]), 0));
                else mbar_arrive(smem_u32(&s_free[which]));
            }
        };
        int n = 0;
        Work work(p, worker, workers);
        for (Tile tile; work.next(tile);) {
            const long long row0 = (long long)tile.m * Sh::rows + rank * kRows + quarter * 32;
            const int rows = (int)min(32ll, p.M - row0);
            const int limit = PAIR ? p.F : p.N;
            // what 32 columns take from memory, on its way before the accumulator is there
            float bias[2] = {0.f, 0.f};
            auto ask = [&](int c) {
                const int col = tile.n * WIDTH + c * 32, cols = min(32, limit - col);
                if (c >= WIDTH / 32 || rows <= 0 || cols <= 0) return;
                if constexpr (PAIR)
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        if (p.bias[w] && lane < cols) bias[w] = to_f32(static_cast<const T*>(p.bias[w])[col + lane]);
                if constexpr (KIND == GRAD)
                    if (dh_packs) ask_chunk<T>(dh_area, static_cast<const T*>(p.dh) + row0 * p.F + col, p.F, rows, cols, lane);
            };
            // 32 columns of the result from the accumulators
            auto finish = [&](int c, float (&g)[32], float (&u)[32]) {
                const int col = tile.n * WIDTH + c * 32, cols = min(32, limit - col);
                if (rows <= 0 || cols <= 0) return;
                float dh[32];
                if constexpr (KIND == GRAD) {
                    if (dh_packs) take_chunk<T>(dh_area, dh, lane);
                    else get_chunk<T>(area, dh, static_cast<const T*>(p.dh) + row0 * p.F + col, p.F, rows, cols, lane);
                }
                if constexpr (PAIR) {
                    if (p.bias[0]) add_bias(g, bias[0]);
                    if (p.bias[1]) add_bias(u, bias[1]);
                    ask(c + 2);
                }
                const bool bad = !ok || late.any();
                if constexpr (KIND == FWD) {
                    gate_by<sizeof(T) == 4, false>(p.activation, g, u, g);
                } else if constexpr (KIND == GRAD) {
                    gate_by<sizeof(T) == 4, true>(p.activation, g, u, dh);
                    if (lane >= rows) {   // rows that are not there: 0 by a NaN bias is not 0
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = u[j] = 0.f;
                    }
                } else if constexpr (KIND == DX || KIND == DW) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) g[j] *= down;
                }
                if (bad) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        g[j] = __int_as_float(0x7fffffff);
                        if (PAIR) u[j] = g[j];
                    }
                }
                if constexpr (KIND == GRAD) {
#pragma unroll 1
                    for (int which = 0; which < 2; ++which) {
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = std::is_same<T, __half>::value ? (which ? u[j] : g[j]) * up : which ? u[j] : g[j];
#pragma unroll 1
                        for (int part = 0; part < PARTS; ++part) {
                            put_chunk<O>(area, v, reinterpret_cast<O*>(p.grads) + ((which * PARTS + part) * p.M + row0) * p.ld + col, p.ld, rows, cols, true, lane);
                            if (part + 1 < PARTS)   // what the parts so far leave, exact
#pragma unroll
                                for (int j = 0; j < 32; j += 2) {
                                    const Halves<O> h(pack2<O>(v[j], v[j + 1]));
                                    v[j] -= to_f32(h.e[0]), v[j + 1] -= to_f32(h.e[1]);
                                }
                        }
                        if (p.sums) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = which ? u[j] : g[j];
                            const float s = column_sums(v, lane);
                            if (lane < cols) p.sums[row0 / 32 * 2 * p.F + which * p.F + col + lane] = s;
                        }
                    }
                } else if ((KIND == DX || KIND == DW) && tile.share >= 0) {
                    float* out = p.shares + ((long long)tile.share * Sh::rows + rank * kRows + quarter * 32) * NB + c * 32;
                    put_chunk<float>(area, g, out, NB, rows, cols, true, lane);
                } else {
                    T* base = static_cast<T*>(p.out[KIND == DW ? tile.set : 0]);
                    if (base) put_chunk<T>(area, g, base + row0 * limit + col, limit, rows, cols, limit % (16 / (int)sizeof(T)) == 0 && aligned16_dev(base), lane);
                }
            };
            auto await = [&] {
                wait_warp(ok, smem_u32(&s_done[n & 1]), (uint32_t)((n / 2) & 1), p.wait_ns, late);
                fence_after_sync();
                return tmem + ((uint32_t)(quarter * 32) << 16) + (n & 1) * NB;
            };
            if constexpr (sizeof(T) == 4) {
                constexpr int C = (WIDTH / 32 + 1) / 2;   // times 32 columns of this warp, added up over the runs
                float g[C][32], u[PAIR ? C : 1][32];
                ask(half);
                for (int k = tile.first; k < tile.last; k += kRun<T>, ++n) {
                    const uint32_t acc = await();
                    if (half < WIDTH / 32) {
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            float v[32];
#pragma unroll
                            for (int w = 0; w < (PAIR ? 2 : 1); ++w) {
                                float (&to)[32] = w ? u[c] : g[c];
                                tmem_ld32_nowait(acc + w * WIDTH + (half + 2 * c) * 32, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j) to[j] = k == tile.first ? v[j] : to[j] + v[j];
                            }
                        }
                    }
                    release(n & 1);
                }
                if (half < WIDTH / 32) {
#pragma unroll
                    for (int c = 0; c < C; ++c) finish(half + 2 * c, g[c], PAIR ? u[c] : g[c]);
                }
            } else {
                ask(half);
                const uint32_t acc = await();
#pragma unroll 1
                for (int c = half; c < WIDTH / 32; c += 2) {
                    float g[32], u[32];
                    tmem_ld32_nowait(acc + c * 32, g);
                    if constexpr (PAIR) tmem_ld32_nowait(acc + WIDTH + c * 32, u);
                    tmem_wait_ld();
                    if (c + 2 >= WIDTH / 32) release(n & 1);
                    finish(c, g, u);
                }
                if (half >= WIDTH / 32) release(n & 1);   // narrow tiles leave nothing for the other warps
                ++n;
            }
        }
    }
    fence_before_sync();
    meet<CTAS>();
    if (warp == kIssue) {
        fence_after_sync();
        dealloc<CTAS>(tmem, Sh::columns);
    }
}

// dx, or a weight's gradient, of the tiles whose sums were shared
template <typename T, int NB> __global__ void __launch_bounds__(256) gated_join_kernel(const __grid_constant__ Params p)
{
    after_previous();
    constexpr int ROWS = Shape<NB, 1>::rows, PIECES = ROWS * NB / 4 / 64;   // of four columns, 64 at a time by four groups of threads
    __shared__ float4 part[3][64];
    const int group = threadIdx.x / 64, lane = threadIdx.x % 64;
    Tile tile;
    tile.place(p, p.whole + blockIdx.x);
    T* out = static_cast<T*>(p.out[tile.set]);
    if (!out) return;
    const int left = p.tiles - p.whole, per = (p.cuts + 3) / 4, from = min(group * per, p.cuts), to = min(from + per, p.cuts);
    const float* parts = p.shares + (long long)blockIdx.x * ROWS * NB;
    const bool vec = p.N % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(T) - 1)) == 0;
    for (int k = blockIdx.y; k < PIECES; k += gridDim.y) {
        const int e = (k * 64 + lane) * 4, r = e / NB, c = e % NB;
        const long long row = (long long)tile.m * ROWS + r;
        const int col = tile.n * NB + c;
        const bool in = row < p.M && col < p.N;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) {
#pragma unroll 8
            for (int w = from; w < to; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(parts + (long long)w * left * ROWS * NB + e);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
        }
        __syncthreads();
        if (group > 0) part[group - 1][lane] = s;
        __syncthreads();
        if (group > 0 || !in) continue;
#pragma unroll
        for (int g = 0; g < 3; ++g) s.x += part[g][lane].x, s.y += part[g][lane].y, s.z += part[g][lane].z, s.w += part[g][lane].w;
        T* dst = out + row * p.N + col;
        if (vec) {
            Pack<T, 4> v;
            v.e[0] = from_f32<T>(s.x), v.e[1] = from_f32<T>(s.y), v.e[2] = from_f32<T>(s.z), v.e[3] = from_f32<T>(s.w);
            *reinterpret_cast<Pack<T, 4>*>(dst) = v;
        } else {
            const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < p.N) dst[j] = from_f32<T>(v[j]);
        }
    }
}

// How many tiles there are and how they are shared out. Cutting sums pays where the blocks that it saves the last round take longer
// than the pieces' way through memory and another launch (GRAD and DX of 256 x 1024 to 4096 bf16: 31 us, uncut 46). Returns about
// how long it all takes, in us: a block takes 0.34 at 256 columns, 0.22 and 0.15 at 128 and 64 (loads bound these), in
// three parts 1 and 0.7, a tile 1.5 besides.
inline double share_out(Params& p, int rows, int width, int nb, int parts, int workers, bool share)
{
    p.tiles_m = (int)((p.M + rows - 1) / rows), p.tiles_n = (p.N + width - 1) / width;
    const int side = std::min(p.tiles_n, 9);
    p.group = (workers + side - 1) / side;
    p.tiles = p.tiles_m * p.tiles_n * p.sets;
    p.whole = p.tiles, p.cuts = 0;
    const int left = p.tiles % workers, rounds = p.tiles / workers, total = p.segs * p.blocks;
    const double block = parts > 1 ? (nb == 128 ? 1. : 0.7) : nb == 256 ? 0.34 : nb == 128 ? 0.22 : 0.15, whole = rounds * (1.5 + block * total);
    double last = left ? 1.5 + block * total : 0.;
    if (!share || left == 0) return whole + last;
    for (int r = 1; r <= 6; ++r) {                         // as many pieces as take r rounds, of four blocks at the least
        const int cuts = std::min(r * workers / left, total / (parts > 1 ? 1 : 4));
        if (cuts < 2) continue;
        const double t = r * (1.5 + block * ((total + cuts - 1) / cuts)) + 4. + 3e-7 * cuts * left * rows * width * sizeof(float);
        if (t < last) last = t, p.cuts = cuts, p.whole = p.tiles - left;
    }
    return whole + last;
}
inline size_t share_bytes(const Params& p, int rows, int width) { return (size_t)p.cuts * (p.tiles - p.whole) * rows * width * sizeof(float); }

template <int KIND, typename T, int NB> cudaError_t run(Params& p, int sms, cudaStream_t s)
{
    using Sh = Shape<NB, kParts<T>>;
    if (const cudaError_t e = allow_smem<gated_tc_kernel<KIND, T, NB>>(Sh::smem); e != cudaSuccess) return e;
    const int workers = sms / Sh::ctas;
    share_out(p, Sh::rows, KIND == FWD || KIND == GRAD ? NB / 2 : NB, NB, kParts<T>, workers, KIND == DX || KIND == DW);
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = Sh::ctas, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    const int busy = (int)std::min<long long>(workers, std::max((long long)p.whole, (long long)p.cuts * (p.tiles - p.whole)));
    c.gridDim = dim3((unsigned)(busy * Sh::ctas)), c.blockDim = dim3(kThreadsG), c.dynamicSmemBytes = Sh::smem;
    c.stream = s, c.attrs = &at, c.numAttrs = Sh::ctas > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&c, gated_tc_kernel<KIND, T, NB>, (const Params&)p);
    if constexpr (KIND == DX || KIND == DW)
        if (e == cudaSuccess && p.cuts) {
            const int tiles = p.tiles - p.whole, pieces = Sh::rows * NB / 4 / 64;
            return launch_behind(gated_join_kernel<T, NB>, dim3((unsigned)tiles, (unsigned)std::min(pieces, std::max(1, 8 * sms / tiles))), 256, s, p);
        }
    return e;
}
template <int KIND, typename T> cudaError_t run_nb(Params& p, int NB, int sms, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2)   // fp32's sums are in registers: half as many columns
        if (NB == 256) return run<KIND, T, 256>(p, sms, s);
    return NB == 128 ? run<KIND, T, 128>(p, sms, s) : run<KIND, T, 64>(p, sms, s);
}
template <int KIND> cudaError_t run_kind(Params& p, int dtype, int NB, int sms, cudaStream_t s)
{
    if (dtype == SDTW_F32) return run_nb<KIND, float>(p, NB, sms, s);
    if (dtype == SDTW_BF16) return run_nb<KIND, __nv_bfloat16>(p, NB, sms, s);
    return run_nb<KIND, __half>(p, NB, sms, s);
}
static cudaError_t take_status_of_file(int* out, cudaStream_t s)
{
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e;
}

// one file each, compiled side by side; NB is 256, 128 or 64
cudaError_t run_fwd(Params& p, int dtype, int NB, int sms, cudaStream_t s);
cudaError_t run_grad(Params& p, int dtype, int NB, int sms, cudaStream_t s);
cudaError_t run_dx(Params& p, int dtype, int NB, int sms, cudaStream_t s);
cudaError_t run_dw(Params& p, int dtype, int NB, int sms, cudaStream_t s);

}  // namespace gtc
}  // namespace sdtw
