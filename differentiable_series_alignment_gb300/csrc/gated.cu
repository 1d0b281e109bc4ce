// gated.cu -- gated linear units, forward and backward.
//
//   g = x Wg^T + bg, u = x Wu^T + bu, h = act(g) u
//   dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dbg, dbu = column sums
//
// The products run on the tensor cores (gated_tc.cuh). Here are the kernels around them: operands brought into the form that
// TMA loads, few rows, sums over row tiles and over shares of a sum, and the order of it all.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gated_tc.cuh"

namespace sdtw {
namespace {

using gtc::kParts;

// ---- few rows: the weights are read once, straight into the registers of m16n8k16 products. A CTA has 16 features of both
// weights; its eight warps share the sum, 32 of it at a time. In those a lane holds 8 neighbours of its row for both
// operands, and takes them as the fragments of two products: which of the sum's terms a position stands for does not
// matter as long as both operands agree. Tiles of 128 rows on the tensor cores would be empty but for these (bf16, 1024 to 4096: 8, 16
// and 32 rows 3.3, 4.3 and 5.5 us with the weights in the cache; by tiles 10.4, 10.4 and 9.5; by the dots below 7.8
// and 13.3 for 8 and 16). From memory its 16.8 MB of weights bound it, whose loads all leave at once and only once.
template <typename T> __device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kFew = 32;   // rows at the most

__device__ __forceinline__ float activate_by(int activation, bool exact, float z) {
    float none;
    switch (activation) {
        case SDTW_ACT_SILU: return exact ? activate<SDTW_ACT_SILU, true, false>(z, none) : activate<SDTW_ACT_SILU, false, false>(z, none);
        case SDTW_ACT_GELU: return activate<SDTW_ACT_GELU, true, false>(z, none);
        case SDTW_ACT_RELU: return activate<SDTW_ACT_RELU, true, false>(z, none);
        default: return exact ? activate<SDTW_ACT_SIGMOID, true, false>(z, none) : activate<SDTW_ACT_SIGMOID, false, false>(z, none);
    }
}

template <typename T, int NT> __global__ void __launch_bounds__(256) gated_few_kernel(const GatedParams p)
{
    constexpr int N = 8 * NT;
    __shared__ float part[8][2][16][N + 1];
    after_previous();
    const sdtw_gated& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, at = (lane & 3) * 8, f0 = blockIdx.x * 16;
    const int R = (int)a.R;
    // volatile: in this order, before the products. Not by the read-only path (ld.global.nc): this kernel begins before the one in front of
    // it has ended, which may be writing these operands.
    auto load = [&](const void* base, long long stride, int r, int rows, int k) {
        uint4 v = make_uint4(0, 0, 0, 0);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                     : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                     : "l"(static_cast<const T*>(base) + r * stride + k), "r"((int)(r < rows && k < a.K)));
        return v;
    };
    float acc[2][NT][4] = {};
    constexpr int AHEAD = NT == 4 ? 2 : 4;   // pieces whose loads are all on their way before the first product
    for (int k0 = warp * 32 * AHEAD; k0 < a.K; k0 += 256 * AHEAD) {   // a warp's pieces are neighbours: 256 bytes of a row
        uint4 w[AHEAD][2][2], x[AHEAD][NT];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int k = k0 + i * 32 + at;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[i][0][h] = load(a.gate_weight, a.gate_stride, f0 + row + 8 * h, a.F, k);
                w[i][1][h] = load(a.up_weight, a.up_stride, f0 + row + 8 * h, a.F, k);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) x[i][t] = load(a.x, a.x_stride, t * 8 + row, R, k);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma16816<T>(acc[m][t], w[i][m][0].x, w[i][m][1].x, w[i][m][0].y, w[i][m][1].y, x[i][t].x, x[i][t].y);
                    mma16816<T>(acc[m][t], w[i][m][0].z, w[i][m][1].z, w[i][m][0].w, w[i][m][1].w, x[i][t].z, x[i][t].w);
                }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) part[warp][m][row + 8 * (q >> 1)][t * 8 + (lane & 3) * 2 + (q & 1)] = acc[m][t][q];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * N; i += 256) {
        const int f = f0 + i % 16, r = i / 16;
        if (f >= a.F || r >= R) continue;
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) g += part[w][0][i % 16][r], u += part[w][1][i % 16][r];
        if (a.gate_bias) g += to_f32(static_cast<const T*>(a.gate_bias)[f]);
        if (a.up_bias) u += to_f32(static_cast<const T*>(a.up_bias)[f]);
        static_cast<T*>(p.h)[(long long)r * a.F + f] = from_f32<T>(activate_by(a.activation, false, g) * u);
    }
}

// Few rows of fp32, or of any stride and address: a warp two features, eight rows at a time, so that what it reads of x serves
// four rows of weights; VEC neighbours of a row at a time where they are one aligned load. (1024 to 4096 fp32: 8 rows 10 us, 32 rows 40;
// by tiles 42 and 42. 16 rows of 1022 bf16: 15, by tiles 24. Its loads bound
// it, 12 of 16 bytes to 128 multiply-adds of a lane: 32 rows are 14 TFLOP/s of the FP32 pipe's 74.)
template <typename T, int VEC> __global__ void __launch_bounds__(256) gated_dot_kernel(const GatedParams p)
{
    using P = Pack<T, VEC>;
    const sdtw_gated& a = p.a;
    const int lane = threadIdx.x & 31, f0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 2;
    after_previous();
    if (f0 >= a.F) return;
    const T* w[4];   // gate and up of either feature
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long f = min(f0 + i / 2, a.F - 1);
        w[i] = i % 2 ? static_cast<const T*>(a.up_weight) + f * a.up_stride : static_cast<const T*>(a.gate_weight) + f * a.gate_stride;
    }
    for (int r0 = 0; r0 < a.R; r0 += 8) {
        const T* x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) x[r] = static_cast<const T*>(a.x) + min((long long)r0 + r, a.R - 1) * a.x_stride;
        float acc[4][8] = {};
#pragma unroll 2
        for (int k = lane * VEC; k < a.K; k += 32 * VEC) {
            P wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) wv[i] = *reinterpret_cast<const P*>(w[i] + k);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const P xv = *reinterpret_cast<const P*>(x[r] + k);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[i][r] = fmaf(to_f32(wv[i].e[e]), to_f32(xv.e[e]), acc[i][r]);
            }
        }
        // the 32 sums over the lanes: lane 8 i + r receives that of acc[i][r]
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = acc[j / 8][j % 8];
        float s = gtc::column_sums(v, lane);
        const int f = f0 + lane / 16, r = lane % 8;
        const void* bias = lane / 8 % 2 ? a.up_bias : a.gate_bias;
        if (bias && f < a.F) s += to_f32(static_cast<const T*>(bias)[f]);
        const float u = __shfl_down_sync(0xffffffffu, s, 8);
        if (lane / 8 % 2 == 0 && f < a.F && r0 + r < a.R)
            static_cast<T*>(p.h)[(r0 + r) * (long long)a.F + f] = from_f32<T>(activate_by(a.activation, sizeof(T) == 4, s) * u);
    }
}

// ---- operands that TMA cannot load as they are: rows copied to a pitch of whole 16 bytes, fp32 as its three bf16 parts
struct PackJob {
    const void* from[3];
    uint16_t* to[3];
    long long stride[3], rows[3];
    int first[4];    // CTAs of a job; a CTA has kPackQuads times four columns, one row after the other
    bool quads[3];   // four columns are one aligned load
    int cols, pitch;
};
constexpr int kPackQuads = 1024;
template <typename T> __global__ void __launch_bounds__(256) gated_pack_kernel(const PackJob j)
{
    using O = typename gtc::Operand<T>::type;
    int w = 0;
    while (w < 2 && (int)blockIdx.x >= j.first[w + 1]) ++w;
    const int across = (j.cols + 3) / 4;
    const long long part = j.rows[w] * j.pitch, quads = j.rows[w] * across;
#pragma unroll
    for (int i = 0; i < kPackQuads / 256; ++i) {
        const long long q = (long long)(blockIdx.x - j.first[w]) * kPackQuads + i * 256 + threadIdx.x;
        if (q >= quads) return;
        const long long r = q / across;
        const int c = (int)(q - r * across) * 4;
        const T* from = static_cast<const T*>(j.from[w]) + r * j.stride[w] + c;
        O* to = reinterpret_cast<O*>(j.to[w]) + r * j.pitch + c;   // the pitch is a multiple of eight: four are always there
        float v[4];
        if (j.quads[w]) {
            const Pack<T, 4> p = *reinterpret_cast<const Pack<T, 4>*>(from);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = to_f32(p.e[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = c + e < j.cols ? to_f32(from[e]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kParts<T>; ++k) {
            const uint2 u = make_uint2(pack2<O>(v[0], v[1]), pack2<O>(v[2], v[3]));
            *reinterpret_cast<uint2*>(to + k * part) = u;
            const Halves<O> lo(u.x), hi(u.y);
#pragma unroll
            for (int z = 0; z < 2; ++z) v[z] -= to_f32(lo.e[z]), v[2 + z] -= to_f32(hi.e[z]);
        }
    }
}

// ---- fp16: what bounds dg and du (gtc::grads_scale): the largest |dh|, |bias| and squared norms of rows. The maximum of bit patterns
// does not depend on their order. A backward pass of 1021 x 250 to 683, launched call by call, takes 46 us with it, 43 with |dh| alone; of 128 x
// 1024 to 4096 47 and 43, of 16384 rows 574 and 573.
struct Ranges {
    const __half *dh, *rows[3], *bias[2];   // rows of x and of both weights
    long long n, stride[3], count[3];
    int K, F;
    unsigned* top;
};
// f of each of n values, by all lanes of the calling threads; eight at a time where they are aligned
template <typename F> __device__ __forceinline__ void each_half(const __half* v, long long n, long long thread, long long threads, F f)
{
    long long done = 0;
    if ((reinterpret_cast<uintptr_t>(v) & 15) == 0) {
        done = n / 8 * 8;
        for (long long i = thread * 8; i < done; i += threads * 8) {
            const Pack<__half, 8> p = *reinterpret_cast<const Pack<__half, 8>*>(v + i);
#pragma unroll
            for (int e = 0; e < 8; ++e) f(to_f32(p.e[e]));
        }
    }
    for (long long i = done + thread; i < n; i += threads) f(to_f32(v[i]));
}
__global__ void __launch_bounds__(256) gated_range_kernel(const Ranges r)
{
    const long long thread = (long long)blockIdx.x * 256 + threadIdx.x, threads = (long long)gridDim.x * 256;
    const int lane = threadIdx.x & 31;
    auto bits = [](float v) { return __float_as_uint(v) & 0x7fffffffu; };   // NaN is the largest
    __shared__ unsigned tops[gtc::kTops];
    if (threadIdx.x < gtc::kTops) tops[threadIdx.x] = 0;
    __syncthreads();
    auto tell = [&](int which, unsigned m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) atomicMax(tops + which, m);
    };
    unsigned m = 0;
    each_half(r.dh, r.n, thread, threads, [&](float v) { m = max(m, bits(v)); });
    tell(0, m);
    for (int w = 0; w < 3; ++w) {
        m = 0;
        for (long long row = thread / 32; row < r.count[w]; row += threads / 32) {
            float s = 0.f;
            each_half(r.rows[w] + row * r.stride[w], r.K, lane, 32, [&](float v) { s = fmaf(v, v, s); });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            m = max(m, bits(s));
        }
        tell(1 + w, m);
    }
    for (int w = 0; w < 2; ++w) {
        m = 0;
        if (r.bias[w]) each_half(r.bias[w], r.F, thread, threads, [&](float v) { m = max(m, bits(v)); });
        tell(4 + w, m);
    }
    __syncthreads();
    if (threadIdx.x < gtc::kTops && tops[threadIdx.x]) atomicMax(r.top + threadIdx.x, tops[threadIdx.x]);
}
// ---- column sums of row tiles, added in a fixed order
template <typename T> __global__ void __launch_bounds__(1024) gated_bias_kernel(const float* sums, long long n, int F, T* dgate, T* dup)
{
    __shared__ float part[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    float s[4] = {};
    if (c < 2 * F)
        for (long long t = lane; t < n; t += 128) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (t + 32 * q < n) s[q] += sums[(t + 32 * q) * 2 * F + c];
        }
    part[lane][threadIdx.x & 31] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    float v = part[threadIdx.x & 31][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int col = blockIdx.x * 32 + lane;
    T* dst = col < F ? dgate : dup;
    if ((threadIdx.x & 31) == 0 && col < 2 * F && dst) dst[col < F ? col : col - F] = from_f32<T>(v);
}
template <typename F> cudaError_t with_type(int dtype, F f) {
    if (dtype == SDTW_F32) return f(float());
    if (dtype == SDTW_BF16) return f(__nv_bfloat16());
    return f(__half());
}

size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
bool loadable(const void* p, long long stride, long long rows, int dtype) {
    return dtype != SDTW_F32 && aligned16(p) && (rows == 1 || (stride > 0 && stride % 8 == 0 && stride < (1ll << 38)));
}

// A 16-bit operand: (parts, rows, cols) of a pitch.
struct Image {
    const void* p;
    long long pitch, rows;
    int cols, parts;
    bool map(CUtensorMap* m, int dtype, int box_cols, int box_rows) const {
        const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
        const long long row = rows > 1 ? pitch * 2 : 16;
        const cuuint64_t strides[2] = {(cuuint64_t)row, (cuuint64_t)(parts > 1 ? pitch * 2 * rows : 16)};
        const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
        return atc::encode(m, dtype == SDTW_F32 ? SDTW_BF16 : dtype, 3, p, dims, strides, box);
    }
};

// Groups of 64 columns as a dimension, `groups` of them to a box of 64 rows; for columns that are whole groups.
bool map_groups(const Image& m, CUtensorMap* to, int dtype, int groups)
{
    const cuuint64_t dims[4] = {64, (cuuint64_t)m.rows, (cuuint64_t)(m.cols / 64), (cuuint64_t)m.parts};
    const cuuint64_t strides[3] = {(cuuint64_t)(m.rows > 1 ? m.pitch * 2 : 16), 128, (cuuint64_t)(m.parts > 1 ? m.pitch * 2 * m.rows : 16)};
    const cuuint32_t box[4] = {64, 64, (cuuint32_t)groups, 1};
    return atc::encode(to, dtype == SDTW_F32 ? SDTW_BF16 : dtype, 4, m.p, dims, strides, box);
}
// An MN-major operand of which a CTA takes `columns` columns
bool map_mn(const Image& m, CUtensorMap* to, int dtype, int columns)
{
    return m.cols % 64 == 0 ? map_groups(m, to, dtype, columns / 64) : m.map(to, dtype, 64, 64);
}

struct Plan {
    Image x, w[2], grads;
    PackJob pack;
    int pack_ctas = 0;
    float *sums = nullptr, *shares = nullptr;
    unsigned* top = nullptr;
    int dx_nb = 256, dw_nb = 256;
    size_t bytes = 0;
};

int tiles_of(long long n, int tile) { return (int)((n + tile - 1) / tile); }

// Columns of an accumulator, by the least time that `time(columns)` expects: wide tiles need the fewest loads, narrow ones
// reach more SMs (bf16 forward with 256, 128 and 64 columns: 16384 x 1024 to 4096 143, 236 and 434 us, 1024 x 512 to 1024 8.8, 6.3
// and 7.8, 256 x 1024 to 4096 11.1, 8.3 and 11.5).
template <typename F> int pick_nb(int dtype, F time)
{
    int best = 0;
    double least = 1e30;
    for (int nb = dtype == SDTW_F32 ? 128 : 256; nb >= 64; nb /= 2)
        if (const double t = time(nb); t < least) least = t, best = nb;
    return best;
}

Plan make_plan(const GatedParams& p, void* ws, bool backward, int sms)
{
    const sdtw_gated& a = p.a;
    Plan plan;
    char* base = static_cast<char*>(ws);
    auto carve = [&](size_t n) {
        char* at = base + plan.bytes;
        plan.bytes += align_up(n);
        return at;
    };
    const int parts = a.dtype == SDTW_F32 ? 3 : 1;
    PackJob& j = plan.pack;
    j = PackJob{};
    j.cols = a.K, j.pitch = (a.K + 7) / 8 * 8;
    int jobs = 0;
    auto operand = [&](const void* from, long long stride, long long rows) {
        if (loadable(from, stride, rows, a.dtype)) return Image{from, stride, rows, a.K, 1};
        uint16_t* to = reinterpret_cast<uint16_t*>(carve((size_t)parts * rows * j.pitch * 2));
        j.from[jobs] = from, j.to[jobs] = to, j.stride[jobs] = stride, j.rows[jobs] = rows;
        j.first[jobs] = plan.pack_ctas;
        j.quads[jobs] = a.K % 4 == 0 && stride % 4 == 0 && reinterpret_cast<uintptr_t>(from) % (4 * dtype_size(a.dtype)) == 0;
        plan.pack_ctas += (int)((rows * ((a.K + 3) / 4) + kPackQuads - 1) / kPackQuads);
        for (int k = ++jobs; k < 4; ++k) j.first[k] = plan.pack_ctas;
        return Image{to, j.pitch, rows, a.K, parts};
    };
    plan.x = operand(a.x, a.x_stride, a.R);
    plan.w[0] = operand(a.gate_weight, a.gate_stride, a.F);
    plan.w[1] = operand(a.up_weight, a.up_stride, a.F);
    if (!backward) return plan;
    const long long pitch = (a.F + 7) / 8 * 8;
    plan.grads = Image{carve((size_t)2 * parts * a.R * pitch * 2), pitch, a.R, a.F, 2 * parts};
    plan.sums = reinterpret_cast<float*>(carve((size_t)tiles_of(a.R, 32) * 2 * a.F * sizeof(float)));
    plan.top = reinterpret_cast<unsigned*>(carve(gtc::kTops * sizeof(unsigned)));
    // Columns of dx's and the weights' accumulators, by the least time, and room for their shares; one of the weights'
    // gradients alone may share its sums otherwise than both.
    size_t shares = 0;
    auto time = [&](int sets, int nb, size_t& bytes) {   // sets 0: dx
        const int ctas = nb == 256 ? 2 : 1;   // 256 columns are a pair's tile, of 256 rows
        gtc::Params g{};
        g.segs = sets ? 1 : 2, g.blocks = sets ? tiles_of(a.R, 64) : tiles_of(a.F, 64);
        g.sets = sets ? sets : 1, g.M = sets ? a.F : a.R, g.N = a.K;
        const double t = gtc::share_out(g, 128 * ctas, nb, nb, parts, sms / ctas, true);
        bytes = gtc::share_bytes(g, 128 * ctas, nb);
        return t;
    };
    size_t bytes;
    plan.dx_nb = pick_nb(a.dtype, [&](int nb) { return time(0, nb, bytes); });
    plan.dw_nb = pick_nb(a.dtype, [&](int nb) { return time(2, nb, bytes); });
    for (int sets : {0, 1, 2}) {
        time(sets, sets ? plan.dw_nb : plan.dx_nb, bytes);
        shares = std::max(shares, bytes);
    }
    plan.shares = reinterpret_cast<float*>(carve(shares));
    return plan;
}

cudaError_t pack_operands(const GatedParams& p, const Plan& plan, cudaStream_t s)
{
    if (!plan.pack_ctas) return cudaSuccess;
    return with_type(p.a.dtype, [&](auto t) {
        gated_pack_kernel<decltype(t)><<<plan.pack_ctas, 256, 0, s>>>(plan.pack);
        return cudaGetLastError();
    });
}

// Both products, side by side.
cudaError_t products(const GatedParams& p, const Plan& plan, bool grads, bool want_sums, int sms, cudaStream_t s)
{
    const sdtw_gated& a = p.a;
    gtc::Params g{};
    g.segs = 1, g.blocks = tiles_of(a.K, 64);
    g.sets = 1;
    g.M = a.R, g.N = g.F = a.F, g.activation = a.activation;
    const int nb = pick_nb(a.dtype, [&](int n) {
        gtc::Params t = g;
        const int ctas = n == 256 ? 2 : 1;
        return gtc::share_out(t, 128 * ctas, n / 2, n, plan.x.parts, sms / ctas, false);
    });
    const int width = nb / 2;
    if (!plan.x.map(&g.a, a.dtype, 64, 128) || !plan.w[0].map(&g.b[0], a.dtype, 64, width) || !plan.w[1].map(&g.b[1], a.dtype, 64, width))
        return cudaErrorInvalidValue;
    g.out[0] = p.h, g.bias[0] = a.gate_bias, g.bias[1] = a.up_bias, g.dh = p.dh;
    g.grads = static_cast<uint16_t*>(const_cast<void*>(plan.grads.p)), g.ld = plan.grads.pitch;
    g.sums = want_sums ? plan.sums : nullptr;
    g.top = grads && a.dtype == SDTW_F16 ? plan.top : nullptr;
    g.wait_ns = p.wait_ns, g.skip = p.skip;
    return grads ? gtc::run_grad(g, a.dtype, nb, sms, s) : gtc::run_fwd(g, a.dtype, nb, sms, s);
}

}  // namespace

bool gated_is_few(const GatedParams& p) { return p.a.R <= kFew; }

size_t gated_workspace(const GatedParams& p, bool backward, int sms)
{
    return !backward && gated_is_few(p) ? 0 : make_plan(p, nullptr, backward, sms).bytes;
}

cudaError_t launch_gated_forward(const GatedParams& p, void* ws, int sms, cudaStream_t s)
{
    const sdtw_gated& a = p.a;
    // launched behind the kernels before them: one call of 16 rows, 1024 to 4096 bf16, after the other takes 4.3 us then, 4.6 without;
    // launched one by one, from memory, 6.4 and 8.2
    if (gated_is_few(p))
        return with_type(a.dtype, [&](auto t) {
            using T = decltype(t);
            if constexpr (sizeof(T) == 2)
                if (a.K % 8 == 0 && loadable(a.x, a.x_stride, a.R, a.dtype) && loadable(a.gate_weight, a.gate_stride, a.F, a.dtype) &&
                    loadable(a.up_weight, a.up_stride, a.F, a.dtype)) {
                    const unsigned grid = (unsigned)tiles_of(a.F, 16);
                    if (a.R <= 8) return launch_behind(gated_few_kernel<T, 1>, grid, 256, s, p);
                    if (a.R <= 16) return launch_behind(gated_few_kernel<T, 2>, grid, 256, s, p);
                    return launch_behind(gated_few_kernel<T, 4>, grid, 256, s, p);
                }
            auto quad = [&](const void* q, long long stride) { return reinterpret_cast<uintptr_t>(q) % (4 * sizeof(T)) == 0 && stride % 4 == 0; };
            if (a.K % 4 == 0 && quad(a.x, a.x_stride) && quad(a.gate_weight, a.gate_stride) && quad(a.up_weight, a.up_stride))
                return launch_behind(gated_dot_kernel<T, 4>, tiles_of(a.F, 16), 256, s, p);
            return launch_behind(gated_dot_kernel<T, 1>, tiles_of(a.F, 16), 256, s, p);
        });
    const Plan plan = make_plan(p, ws, false, sms);
    if (const cudaError_t e = pack_operands(p, plan, s); e != cudaSuccess) return e;
    return products(p, plan, false, false, sms, s);
}

cudaError_t launch_gated_backward(const GatedParams& p, void* ws, int sms, cudaStream_t s)
{
    const sdtw_gated& a = p.a;
    const Plan plan = make_plan(p, ws, true, sms);
    const int parts = plan.x.parts;
    cudaError_t e = pack_operands(p, plan, s);
    if (e != cudaSuccess) return e;
    if (a.dtype == SDTW_F16) {
        if ((e = cudaMemsetAsync(plan.top, 0, gtc::kTops * sizeof(unsigned), s)) != cudaSuccess) return e;
        auto half = [](const void* q) { return static_cast<const __half*>(q); };
        const Ranges r{half(p.dh), {half(a.x), half(a.gate_weight), half(a.up_weight)}, {half(a.gate_bias), half(a.up_bias)},
                       a.R * a.F, {a.x_stride, a.gate_stride, a.up_stride}, {a.R, a.F, a.F}, a.K, a.F, plan.top};
        const long long values = a.R * a.F + (a.R + 2ll * a.F) * a.K;
        gated_range_kernel<<<(unsigned)std::min(values / 8192 + 1, (long long)sms * 8), 256, 0, s>>>(r);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const bool biases = p.dgate_bias || p.dup_bias;
    if ((e = products(p, plan, true, biases, sms, s)) != cudaSuccess) return e;
    gtc::Params g{};
    g.top = a.dtype == SDTW_F16 ? plan.top : nullptr;
    g.activation = a.activation;
    g.wait_ns = p.wait_ns;
    if (p.dx) {
        const int columns = plan.dx_nb == 256 ? 128 : plan.dx_nb;   // of a CTA
        if (!plan.grads.map(&g.a, a.dtype, 64, 128) || !map_mn(plan.w[0], &g.b[0], a.dtype, columns) || !map_mn(plan.w[1], &g.b[1], a.dtype, columns))
            return cudaErrorInvalidValue;
        g.grouped_b = a.K % 64 == 0;
        g.segs = 2, g.seg[1].a = (unsigned char)parts, g.blocks = tiles_of(a.F, 64);
        g.sets = 1, g.set0 = 0;
        g.M = a.R, g.N = a.K, g.out[0] = p.dx, g.shares = plan.shares;
        if ((e = gtc::run_dx(g, a.dtype, plan.dx_nb, sms, s)) != cudaSuccess) return e;
    }
    if (p.dgate_weight || p.dup_weight) {
        if (!map_mn(plan.grads, &g.a, a.dtype, 128) || !map_mn(plan.x, &g.b[0], a.dtype, plan.dw_nb == 256 ? 128 : plan.dw_nb)) return cudaErrorInvalidValue;
        g.grouped_a = a.F % 64 == 0, g.grouped_b = a.K % 64 == 0;
        g.b[1] = g.b[0];
        g.segs = 1, g.blocks = tiles_of(a.R, 64);
        g.set0 = p.dgate_weight ? 0 : 1, g.sets = p.dgate_weight && p.dup_weight ? 2 : 1;
        g.M = a.F, g.N = a.K, g.out[0] = p.dgate_weight, g.out[1] = p.dup_weight, g.shares = plan.shares;
        if ((e = gtc::run_dw(g, a.dtype, plan.dw_nb, sms, s)) != cudaSuccess) return e;
    }
    if (biases)
        e = with_type(a.dtype, [&](auto t) {
            using T = decltype(t);
            gated_bias_kernel<T><<<(2 * a.F + 31) / 32, 1024, 0, s>>>(plan.sums, tiles_of(a.R, 32), a.F, static_cast<T*>(p.dgate_bias),
                                                                     static_cast<T*>(p.dup_bias));
            return cudaGetLastError();
        });
    return e;
}

}  // namespace sdtw
