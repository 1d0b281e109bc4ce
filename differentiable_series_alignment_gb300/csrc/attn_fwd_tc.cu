// attn_fwd_tc.cu -- attention's forward pass on the tensor cores (bf16 and fp16).
//
// One CTA takes NT = 2 tiles of up to 128 packed rows and walks the visible keys in tiles of
// 128. Two warps issue S_w = Q_w K^T and O_w += P_w V, a warp a row tile w, so that the tensor
// cores work on one tile while the other's softmax runs and its issuing warp waits. Four
// warps are a tile's softmax, a thread a row; one more warp feeds a ring of K and V tiles by
// TMA. Tensor memory holds S_0, S_1 (P_w over S_w, as a 16-bit A operand) and O_0, O_1: all
// 512 columns. O_w takes the first 64 keys of a tile while the softmax is still at the others.
//
// A single tile of rows (new samples over a cache) takes both halves of the machine: its key
// tiles alternate between them, each with a maximum, a sum and an O of its own, which are
// joined at the end. Every tile's way through scores, softmax and product is a chain of some
// 2700 cycles, longer than its K and V take to arrive.
//
// NT = 1 is the same with one tile of rows, half of the tensor memory and less than half of the
// shared memory: for heads of up to 64 two such CTAs share an SM and one's start and end go
// under the other's products (32 x 512 samples, 8 heads of 64: 47 us with NT = 2), and wider
// heads take it where there are too few tiles for every SM.
//
// The running maximum is renewed only when a row's scores rise by more than 2^8 over it, so
// that the accumulator in tensor memory is rarely read back for rescaling: probabilities are
// then at most 2^8, which fp32 sums and 16-bit operands take as well as 1.
//
// Probabilities are rounded to 16 bits for their product with V, and O is divided by the sum of
// the rounded ones: in the backward pass their errors then enter delta = do . o only by how they
// differ from key to key, as those of dS itself do. Divided by the exact sum, which lse keeps,
// dq was up to 1.9 times as far from its 64-bit value as a plain fp32 pass.
//
// 4 x 4096 samples, causal, 16 heads of 128 over 4 key heads: 224 us, 1230 TFLOP/s. A tile's chain of
// scores, maximum, exponentials and product takes some 3600 cycles, the products of two tiles 2048 of
// them: latency bounds it, next to the power limit (1365 of 1400 W). Clusters of two CTAs that share
// the loads of K and V, and 16 softmax warps, made it no faster. A softmax thread holds 128 scores and spills 88
// bytes at 168 registers. One new sample of 16 streams over 8192 keys, 32 heads of 128 over 8: 76 us, 5.0 TB/s of K and V.
#include "attn_tc.cuh"

namespace sdtw {
namespace atc {
namespace {

__device__ int g_status;

constexpr float kLazy = 8.f;   // log2 of how far scores may rise over the maximum in use

template <int DP, int NT> struct FwdShape {
    static constexpr int loader = 4 * NT, issuer = loader + 1;   // warps: 4 a tile for its softmax, then these
    static constexpr int threads = 32 * (issuer + NT);
    static constexpr uint32_t tile = (DP / 64) * kBox;   // bytes of a row or key tile
    static constexpr int slots = DP == 128 || NT == 1 ? 5 : 10;   // K and V tiles in flight: 160 KB, 80 of two CTAs
    // two tiles of 128 features: with the static arrays, rounded up to 1 KB, all of the 227 KB
    // that a CTA can have
    static constexpr uint32_t smem = NT * tile + slots * tile;
    static constexpr int columns = 256 * NT;             // of tensor memory: S, then O
};

// fp16 cannot hold small probabilities in full: 2^7 more of them, up to 2^15 in all.
template <typename T> struct Lift { static constexpr float v = 0.f; };
template <> struct Lift<__half> { static constexpr float v = 7.f; };

template <typename T, int DP, int NT>
__global__ void __launch_bounds__(FwdShape<DP, NT>::threads, NT == 1 ? 2 : 1) attn_fwd_tc_kernel(const AttnParams p, const __grid_constant__ Maps maps)
{
    using Sh = FwdShape<DP, NT>;
    constexpr int kLoader = Sh::loader, kIssuer = Sh::issuer;
    extern __shared__ __align__(1024) unsigned char dyn[];   // as the swizzle of the images asks
    __shared__ uint64_t s_q[NT], s_full[Sh::slots], s_empty[Sh::slots], s_s[NT], s_p[NT][2], s_o[NT], s_end[NT], s_turn[NT];
    __shared__ float s_join[3][128];
    __shared__ uint32_t s_tmem;
    __shared__ int s_late;
    const Late late{&g_status, &s_late};
    const sdtw_attention& a = p.a;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (p.splits > 1) let_next_come();
    if (warp == kLoader && lane == 0) prefetch_map(&maps.q), prefetch_map(&maps.k), prefetch_map(&maps.v);
    const int heads = a.B * a.Hkv, bh = blockIdx.x % heads;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int RT = p.tile_rows;
    // the last rows see the most keys under a causal mask: they start first
    const int groups = (p.rows + NT * RT - 1) / (NT * RT);
    const int r00 = (groups - 1 - (int)(blockIdx.x / heads)) * NT * RT;
    const RowRange rr(a, b);
    Tiles t0(rr, r00, min(r00 + RT, p.rows), p.G), t1(rr, r00 + RT, min(r00 + NT * RT, p.rows), p.G);   // NT 1: t1 is empty
    int T0 = t0.hi == 0 ? t1.lo : t1.hi == 0 ? t0.lo : min(t0.lo, t1.lo), T1 = max(t0.hi, t1.hi);
    if (p.splits > 1) {   // this CTA's share of the key tiles
        const int per = (T1 - T0 + p.splits - 1) / p.splits;
        T0 = min(T0 + per * (int)blockIdx.y, T1);
        T1 = min(T0 + per, T1);
        t0.lo = max(t0.lo, T0), t0.hi = min(t0.hi, T1);
        t1.lo = max(t1.lo, T0), t1.hi = min(t1.hi, T1);
    }
    const bool any0 = t0.lo < t0.hi, any1 = t1.lo < t1.hi;
    const bool alternate = NT == 2 && p.rows <= RT;   // one tile of rows: key tiles T0, T0 + 2, .. and T0 + 1, T0 + 3, ..
    const bool solo = NT == 1 || alternate;           // no entry of the ring is read by two warps
    // Ring entries in use. K and V of a tile are neighbours, so with a multiple of four of them an
    // entry always serves the same half: a warp that saw only every other phase of an entry's
    // barrier would take the phase before last for the one it waits for.
    const int slots = alternate ? Sh::slots / 4 * 4 : Sh::slots;
    if (!any0 && !any1) T1 = T0;
    T0 = uniform(T0), T1 = uniform(T1);
    t0.lo = uniform(t0.lo), t0.hi = uniform(t0.hi), t1.lo = uniform(t1.lo), t1.hi = uniform(t1.hi);

    const uint32_t q_img = smem_u32(dyn), ring = q_img + NT * Sh::tile;
    // the loader makes the barriers and sends for the first tiles before the CTA has met
    const uint32_t row_bytes = (uint32_t)RT * 128 * (DP / 64);
    if (warp == kLoader && lane == 0) {
        s_late = 0;
        for (int w = 0; w < NT; ++w) {
            mbar_init(smem_u32(&s_q[w]), 1);
            mbar_init(smem_u32(&s_s[w]), 1);
            mbar_init(smem_u32(&s_p[w][0]), 4);
            mbar_init(smem_u32(&s_p[w][1]), 4);
            mbar_init(smem_u32(&s_o[w]), 1);
            mbar_init(smem_u32(&s_end[w]), 1);
            mbar_init(smem_u32(&s_turn[w]), 1);
        }
        for (int e = 0; e < Sh::slots; ++e) {
            mbar_init(smem_u32(&s_full[e]), 1);
            mbar_init(smem_u32(&s_empty[e]), solo ? 1 : 2);   // issuing warps that read it
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (p.skip != 1 && any0) {
            mbar_expect_tx(smem_u32(&s_q[0]), row_bytes);
            load_rows<DP>(q_img, &maps.q, r00 / p.G, hk, b, smem_u32(&s_q[0]));
        }
    }
    if (warp == kIssuer) tmem_alloc(&s_tmem, Sh::columns);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
    bool ok = true;

    if (warp == kLoader) {
        if (lane == 0 && p.skip != 1) {
            const int n0 = r00 / p.G;
            const int total = 2 * (T1 - T0);
            int issued = 0;
            auto left_out = [&](int i) { return p.skip == 2 && ((T0 + (i >> 1)) & 1); };   // test hook: every second key tile
            for (int i = 0; i < total && ok; ++i) {
                if (left_out(i)) continue;
                const int e = i % slots;
                if (i >= slots) wait_for(ok, smem_u32(&s_empty[e]), (uint32_t)((i / slots - 1) & 1), p.wait_ns, late);
                if (!ok) break;
                const uint32_t bar = smem_u32(&s_full[e]);
                mbar_expect_tx(bar, Sh::tile);
                load_keys<DP>(ring + e * Sh::tile, (i & 1) ? &maps.v : &maps.k, (T0 + (i >> 1)) * kKeys, hk, b, bar);
                issued = i + 1;
                if (NT == 2 && i == 0 && any1) {
                    mbar_expect_tx(smem_u32(&s_q[NT - 1]), row_bytes);
                    load_rows<DP>(q_img + Sh::tile, &maps.q, n0 + RT / p.G, hk, b, smem_u32(&s_q[NT - 1]));
                }
            }
            // no copy may be writing shared memory when the CTA ends
            bool drained = true;
            for (int i = max(0, issued - slots); i < issued; ++i)
                if (!left_out(i)) wait_for(drained, smem_u32(&s_full[i % slots]), (uint32_t)((i / slots) & 1), p.wait_ns, late);
            if (any0) wait_for(drained, smem_u32(&s_q[0]), 0, p.wait_ns, late);
            if (NT == 2 && any1 && issued > 0) wait_for(drained, smem_u32(&s_q[NT - 1]), 0, p.wait_ns, late);
        }
        __syncwarp();
    } else if (warp >= kIssuer) {
        const int w = warp - kIssuer;
        const int lo = w ? t1.lo : t0.lo, hi = w ? t1.hi : t0.hi;
        const int steps = (a.D + 15) / 16;
        const uint32_t id_s = idesc<T>(128, kKeys, false), id_o = idesc<T>(128, steps * 16, true);
        const uint32_t s_col = tmem + w * 128, o_col = tmem + NT * 128 + w * 128, q = q_img + (alternate ? 0 : w) * Sh::tile;
        // The two warps take turns, O_w of a tile and S_w of the next at a time. Left to themselves
        // their products interleave, both tiles' scores come late and together, and so do both
        // softmaxes, with the tensor cores idle meanwhile.
        auto take_turn = [&](int j) {
            const int k = j - (T0 - 1) - (w == 0);   // the other's k-th pass; the first turn is tile 0's
            if (k >= 0) wait_warp(ok, smem_u32(&s_turn[w]), (uint32_t)(k & 1), p.wait_ns, late);
        };
        // a warp's own tiles in turn: O of one, then the scores of the next
        auto products = [&](uint32_t vimg, int j, int i, bool last) {
            const int tail = rr.m_b - j * kKeys;
            if (ok && tail < kKeys && rr.m_b < a.M) clear_rows<DP>(vimg, tail, lane);   // both warps: the same zeros
            const uint64_t vd = sdesc_mn(vimg);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                wait_warp(ok, smem_u32(&s_p[w][part]), (uint32_t)(i & 1), p.wait_ns, late);
                if (part == 0 && !solo) take_turn(j);
                fence_after_sync();
                if (ok && elect_one()) {
#pragma unroll
                    for (int s = 4 * part; s < 4 * part + 4; ++s)
                        mma_ts(o_col, s_col + s * 8, vd + s * 128, id_o, (i > 0 || s > 0) ? 1u : 0u);
                    if (part == 1 && last) mma_commit(smem_u32(&s_o[w]));
                }
                __syncwarp();
            }
        };
        auto scores = [&](uint32_t kimg) {
            fence_after_sync();
            if (ok && elect_one()) {
                mma_features<DP / 16>(s_col, q, kimg, steps, id_s);
                mma_commit(smem_u32(&s_s[w]));
            }
            __syncwarp();
        };
        if (solo) {
            const int step = NT == 1 ? 1 : 2, own = (T1 - T0 - w + step - 1) / step;
            for (int i = -1; i < own; ++i) {
                const int iv = 2 * (step * i + w) + 1, ik = 2 * (step * (i + 1) + w);   // ring entries
                if (i >= 0) {
                    const int e = iv % slots;
                    wait_warp(ok, smem_u32(&s_full[e]), (uint32_t)((iv / slots) & 1), p.wait_ns, late);
                    products(ring + (uint32_t)e * Sh::tile, T0 + step * i + w, i, i == own - 1);
                    if (ok && elect_one()) mma_commit(smem_u32(&s_empty[e]));
                    __syncwarp();
                }
                if (i + 1 < own) {
                    const int e = ik % slots;
                    if (i < 0) wait_warp(ok, smem_u32(&s_q[0]), 0, p.wait_ns, late);
                    wait_warp(ok, smem_u32(&s_full[e]), (uint32_t)((ik / slots) & 1), p.wait_ns, late);
                    scores(ring + (uint32_t)e * Sh::tile);
                    if (ok && elect_one()) mma_commit(smem_u32(&s_empty[e]));
                    __syncwarp();
                }
            }
        }
        int e_v = slots - 1, e_k = 0;   // ring entries of V(j) and K(j + 1)
        uint32_t ph_v = 1, ph_k = 0;        // and the parities of their arrivals
        for (int j = T0 - 1; j < T1 && !solo; ++j) {
            // a warp gives every entry back once it is there, also those that its tile does not see:
            // one that ran ahead would give back an entry's next use for its last
            if (j >= T0) wait_warp(ok, smem_u32(&s_full[e_v]), ph_v, p.wait_ns, late);
            if (j >= lo && j < hi) products(ring + (uint32_t)e_v * Sh::tile, j, j - lo, j == hi - 1);
            if (j + 1 < T1) wait_warp(ok, smem_u32(&s_full[e_k]), ph_k, p.wait_ns, late);
            if (j + 1 >= lo && j + 1 < hi) {
                if (!(j >= lo && j < hi)) take_turn(j);
                if (j + 1 == lo) wait_warp(ok, smem_u32(&s_q[w]), 0, p.wait_ns, late);
                scores(ring + (uint32_t)e_k * Sh::tile);
            }
            if (!(j >= lo && j < hi) && !(j + 1 >= lo && j + 1 < hi)) take_turn(j);
            if (ok && elect_one()) {
                mbar_arrive(smem_u32(&s_turn[(w + 1) % NT]));
                if (j >= T0) mma_commit(smem_u32(&s_empty[e_v]));
                if (j + 1 < T1) mma_commit(smem_u32(&s_empty[e_k]));
            }
            __syncwarp();
            // entries alternate: V(j + 1) follows K(j + 1), K(j + 2) follows it
            if ((e_v += 2) >= slots) e_v -= slots, ph_v ^= 1;
            if ((e_k += 2) >= slots) e_k -= slots, ph_k ^= 1;
        }
        // every MMA has read its operands and written its result before the CTA ends
        if (lane == 0) {
            mma_commit(smem_u32(&s_end[w]));
            bool fin = true;
            wait_for(fin, smem_u32(&s_end[w]), 0, p.wait_ns, late);
        }
        __syncwarp();
    } else if (warp < kLoader) {
        const int w = warp >> 2, quarter = warp & 3;
        const int step = alternate ? 2 : 1, lo = alternate ? T0 + w : w ? t1.lo : t0.lo, hi = alternate ? T1 : w ? t1.hi : t0.hi;
        const int r = r00 + (alternate ? 0 : w) * RT + quarter * 32 + lane;
        const bool mine = quarter * 32 + lane < RT && r < p.rows;
        const int n = mine ? r / p.G : 0, h = hk * p.G + (mine ? r % p.G : 0);
        const bool live = mine && n < rr.n_b;
        const int klo = live ? rr.lo(n) : 0, khi = live ? max(klo, rr.hi(n)) : 0;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_col = tmem + lanes + w * 128, o_col = tmem + lanes + NT * 128 + w * 128;
        const float s2 = a.scale * kLog2e;
        const int o_cols = (a.D + 15) / 16 * 16;
        float m = -INFINITY, top = -INFINITY, off = 0.f;   // maximum in use, its trigger, its base
        float l = 0.f, lr = 0.f;                           // sums of the probabilities, exact and rounded
        for (int j = lo, i = 0; j < hi; j += step, ++i) {
            wait_warp(ok, smem_u32(&s_s[w]), (uint32_t)(i & 1), p.wait_ns, late);
            fence_after_sync();
            float s[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_nowait(s_col + c * 32, s + c * 32);
            tmem_wait_ld();
            const int j0 = j * kKeys;
            if (__any_sync(0xffffffffu, live && (j0 < klo || j0 + kKeys > khi))) {
                const int first = klo - j0, count = khi - klo;
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if ((unsigned)(c - first) >= (unsigned)count) s[c] = -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 124; c += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], s[c + q], s[c + 4 + q]);
            const float now = max3(max3(mx[0], s[124], s[125]), max3(mx[1], s[126], s[127]), fmaxf(mx[2], mx[3]));
            if (__any_sync(0xffffffffu, live && now > top)) {
                const float old = m;
                m = fmaxf(m, now);
                const float keep = m == old ? 1.f : ex2((old - m) * s2);
                l *= keep;
                lr *= keep;
                off = (m == -INFINITY ? 0.f : m * s2) - Lift<T>::v;
                top = m + kLazy / s2;
                if (i > 0) {
                    for (int c = 0; c < o_cols; c += 16) {
                        float o[16];
                        tmem_ld16(o_col + c, o);
                        uint32_t u[16];
#pragma unroll
                        for (int q = 0; q < 16; ++q) u[q] = __float_as_uint(o[q] * keep);
                        tmem_st16(o_col + c, u);
                    }
                }
            }
            const unsigned long long mul = pk2(s2, s2), sub = pk2(-off, -off);
            unsigned long long sum0 = pk2(0.f, 0.f), sum1 = pk2(0.f, 0.f);
            float seen[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                uint32_t u[16];
#pragma unroll
                for (int q = 0; q < 32; q += 4) {
                    float e[4];
                    upk2(fma2(pk2(s[c + q], s[c + q + 1]), mul, sub), e[0], e[1]);
                    upk2(fma2(pk2(s[c + q + 2], s[c + q + 3]), mul, sub), e[2], e[3]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) e[z] = ex2(e[z]);
                    sum0 = add2(sum0, pk2(e[0], e[1]));
                    sum1 = add2(sum1, pk2(e[2], e[3]));
                    u[q / 2] = pack2<T>(e[0], e[1]);
                    u[q / 2 + 1] = pack2<T>(e[2], e[3]);
                    add_pair<T>(seen[0], seen[1], u[q / 2]);
                    add_pair<T>(seen[2], seen[3], u[q / 2 + 1]);
                }
                tmem_st16(s_col + c / 2, u);
                if (c == 32) {   // the first 64 keys are there
                    tmem_wait_st();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_p[w][0]));
                }
            }
            lr += (seen[0] + seen[1]) + (seen[2] + seen[3]);
            float x, y;
            upk2(add2(sum0, sum1), x, y);
            l += x + y;
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_p[w][1]));
        }
        bool read = lo < hi, other = false;
        if (read) {
            wait_warp(ok, smem_u32(&s_o[w]), 0, p.wait_ns, late);
            fence_after_sync();
        }
        float mul = 0.f, mul1 = 0.f, total = l, by = lr;
        if (NT == 2 && alternate) {   // warps 0-3 join the two; a lane's row lies in the same lane of O_0 and O_1
            const int row = quarter * 32 + lane;
            if (w == 1) s_join[0][row] = l == 0.f ? -INFINITY : off, s_join[1][row] = l, s_join[2][row] = lr;
            fence_before_sync();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            fence_after_sync();
            other = T1 - T0 > 1;
            const float off1 = s_join[0][row], l1 = s_join[1][row];
            const float both = fmaxf(l == 0.f ? -INFINITY : off, off1);
            mul = l == 0.f ? 0.f : ex2(off - both);
            mul1 = off1 == -INFINITY ? 0.f : ex2(off1 - both);
            total = l * mul + l1 * mul1;
            by = lr * mul + s_join[2][row] * mul1;
            off = both;
        } else {
            mul = 1.f;
        }
        ok = ok && !late.any();
        if (!(alternate && w == 1)) {
            const bool seen = live && read && total != 0.f;
            const float inv = !ok ? NAN : seen ? 1.f / by : 0.f;
            const float lse2 = !ok ? NAN : seen ? off + log2f(total) : -INFINITY;
            read = read && ok;
            other = other && ok;
            mul = ok ? mul * inv : NAN;
            mul1 *= inv;
            // through the rows' part of Q's image
            const uint32_t area = q_img + w * Sh::tile + (uint32_t)(quarter * 32 * DP * 2);
            if (p.splits > 1) {
                const long long place = mine ? ((((long long)blockIdx.y * a.B + b) * a.Hkv + hk) * p.rows + r) : -1;
#pragma unroll 1
                for (int f = 0; f < DP; f += 32)
                    write_rows_f32<32>(area, o_col + f, read, other, ok && !seen, mul, mul1, p.part_o,
                                       mine ? place * a.D + f : -1, min(32, a.D - f) / 4, lane);
                if (mine) p.part_lse[place] = lse2 * kLn2;
            } else {
                const long long at = mine ? (((long long)b * a.N + n) * a.Hq + h) * a.D : -1;
                constexpr int F = DP / 2;   // at a time: the area holds them and what their rounding leaves
#pragma unroll 1
                for (int f = 0; f < DP; f += F)
                    write_rows<T, F>(area, o_col + f, read, other, ok && !seen, mul, mul1, 1.f, p.out, p.out_rest,
                                     mine ? at + f : -1, min(F, a.D - f) / 8, lane);
                if (mine && p.lse) p.lse[((long long)b * a.Hq + h) * a.N + n] = lse2 * kLn2;
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kIssuer) {
        fence_after_sync();
        tmem_dealloc(tmem, Sh::columns);
    }
}

template <typename T, int DP, int NT> cudaError_t run_fwd(const AttnParams& p, const Maps& m, cudaStream_t s)
{
    using Sh = FwdShape<DP, NT>;
    const cudaError_t e = allow_smem<attn_fwd_tc_kernel<T, DP, NT>>(Sh::smem);
    if (e != cudaSuccess) return e;
    const unsigned groups = (unsigned)((p.rows + NT * p.tile_rows - 1) / (NT * p.tile_rows));
    attn_fwd_tc_kernel<T, DP, NT><<<dim3(groups * p.a.B * p.a.Hkv, p.splits), Sh::threads, Sh::smem, s>>>(p, m);
    return cudaGetLastError();
}
template <typename T> cudaError_t pick_fwd(const AttnParams& p, const Maps& m, cudaStream_t s)
{
    if (p.row_tiles == 1) return p.a.D <= 64 ? run_fwd<T, 64, 1>(p, m, s) : run_fwd<T, 128, 1>(p, m, s);
    return p.a.D <= 64 ? run_fwd<T, 64, 2>(p, m, s) : run_fwd<T, 128, 2>(p, m, s);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

}  // namespace

bool encode(CUtensorMap* m, int dtype, int rank, const void* p, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, bool swizzled)
{
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    const EncodeFn fn = encode_fn();
    auto go = [&] {
        const CUtensorMapDataType type = dtype == SDTW_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : dtype == SDTW_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        return fn(m, type, (cuuint32_t)rank, const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    if (!fn) return false;
    if (go() == CUDA_SUCCESS) return true;
    // a thread whose first CUDA call this is (autograd's own, for one) has no context before it names its device
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && go() == CUDA_SUCCESS;
}

namespace {

// A dimension of one element is never stepped along: its stride need only be valid.
cuuint64_t step(long long stride, int size) { return size > 1 ? (cuuint64_t)stride * 2 : 16; }

}  // namespace

bool map_rows(CUtensorMap* m, const void* p, const long long* stride, const sdtw_attention& a, int G, int RT)
{
    const cuuint64_t dims[5] = {(cuuint64_t)a.D, (cuuint64_t)G, (cuuint64_t)a.Hkv, (cuuint64_t)a.N, (cuuint64_t)a.B};
    const cuuint64_t st[4] = {step(stride[2], G), step(stride[2] * G, a.Hkv), step(stride[1], a.N), step(stride[0], a.B)};
    const cuuint32_t box[5] = {64, (cuuint32_t)G, 1, (cuuint32_t)(RT / G), 1};
    return encode(m, a.dtype, 5, p, dims, st, box);
}

bool map_keys(CUtensorMap* m, const void* p, const long long* stride, const sdtw_attention& a)
{
    const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.M, (cuuint64_t)a.Hkv, (cuuint64_t)a.B};
    const cuuint64_t st[3] = {step(stride[1], a.M), step(stride[2], a.Hkv), step(stride[0], a.B)};
    const cuuint32_t box[4] = {64, kKeys, 1, 1};
    return encode(m, a.dtype, 4, p, dims, st, box);
}

}  // namespace atc

cudaError_t launch_attn_forward_tc(const AttnParams& p, cudaStream_t s)
{
    atc::Maps m{};
    const sdtw_attention& a = p.a;
    if (!atc::map_rows(&m.q, a.q, a.q_stride, a, p.G, p.tile_rows) || !atc::map_keys(&m.k, a.k, a.k_stride, a) ||
        !atc::map_keys(&m.v, a.v, a.v_stride, a))
        return cudaErrorInvalidValue;
    return a.dtype == SDTW_BF16 ? atc::pick_fwd<__nv_bfloat16>(p, m, s) : atc::pick_fwd<__half>(p, m, s);
}

cudaError_t attn_forward_take_status(int* out, cudaStream_t s)
{
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, atc::g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbolAsync(atc::g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e;
}

}  // namespace sdtw
