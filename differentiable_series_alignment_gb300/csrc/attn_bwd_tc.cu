// attn_bwd_tc.cu -- attention's backward pass on the tensor cores (bf16 and fp16).
//
// CTAs of two kinds, each computing P = exp(S - lse) and dS = P (dP - delta) again from q, k, v,
// do and the row's lse and delta:
//   dkv: a CTA holds 128 keys and walks the packed rows that see them;
//     S^T = K Q^T and dP^T = V dO^T go to tensor memory, P^T and dS^T come back there as
//     16-bit A operands, dV += P^T dO and dK += dS^T Q;
//   dq: a CTA holds a tile of packed rows and walks their keys;
//     S = Q K^T, dP = dO V^T, dQ += dS K.
// That is 7 products where one kernel would need 5, but no result is summed across CTAs:
// no atomics, no partial dQ in memory, the same bits every time. The gradients of heads
// that share keys are summed in the accumulator, as rows of one problem. Both kinds are one
// launch: the dkv CTAs, few and long, start first and the dq CTAs fill the SMs that they leave.
// Sixteen warps turn scores into probabilities (four warpgroups, 32 of the 128 columns each; eight
// warps of 64 columns were as fast: the products set the pace, not the warps), one more loads by
// TMA, two issue the products: one S and what P enters, the other dP and what dS enters.
// The 16-bit operands have tensor memory of their own where it is large enough (dq; dkv of heads of
// up to 64): the next scores are then made as soon as the last ones have been read. The dkv CTAs
// of wider heads have P^T over S^T and dS^T over dP^T: while the tensor cores run dV and the next S^T, the
// warps compute dS^T; while they run dK and the next dP^T, the next P^T.
// P and dS are rounded to the operands' 16 bits. Next to a result's own rounding that of dS is as large again, in squares, for dq
// and dk, that of P for dv, and what the forward pass's rounded P leaves in delta comes on top for dq and dk: up to 1.5
// times the error of a plain fp32 pass. dS as two 16-bit parts, each with a product of its own, would bring dq and dk to 1.02 to
// 1.14 (a model in 64 bits) and took the case below from 379 to 475 us with flushed caches: not kept.
// 2 x 4096 samples, causal, 16 heads of 128 over 4 key heads: 353 us for the 7 products of the visible
// tiles, 1370 TFLOP/s, with the card near its power limit (a plain bf16 product sustains 1717).
// 32 x 512 samples, 8 heads of 64, padded: 104 us: the products are
// half as long as for 128 features, the exponentials, loads and hand-overs of a tile as many.
#include "attn_tc.cuh"

namespace sdtw {
namespace atc {
namespace {

__device__ int g_status;

constexpr int kWorkers = 16;             // warps
constexpr int kWork = 32 * kWorkers;     // threads
constexpr int kLoader = kWorkers, kIssuer = kWorkers + 1;
constexpr int kThreadsB = kWork + 96;
constexpr int kCols = 32;                // of a tile's 128 columns, per warp

template <int DP> struct BwdShape {
    static constexpr uint32_t tile = (DP / 64) * kBox;
    static constexpr int stages = DP == 128 ? 2 : 4;   // dkv: (Q, dO) pairs in flight, 128 KB
    static constexpr int slots = DP == 128 ? 5 : 10;   // dq: K and V tiles in flight, 160 KB
    // with the static arrays, rounded up to 1 KB, all of the 227 KB that a CTA can have
    static constexpr uint32_t smem_dkv = 2 * tile + 2 * stages * tile, smem_dq = 2 * tile + slots * tile;
};

// A warp's tensor-memory accesses are done: one of the barrier's arrivals.
__device__ __forceinline__ void done(uint64_t& bar) {
    fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
}
__device__ __forceinline__ void work_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

// fp16 operands: dS is scaled by the power of two that keeps |dP - delta| <= 2 |do| |v| below 1
// for the largest row of do and of v, so that neither small upstream gradients nor large ones
// leave the format's range. bf16 has the range of fp32: 1.
template <typename T> __device__ __forceinline__ float grad_scale(const AttnParams&, int, int) { return 1.f; }
template <> __device__ __forceinline__ float grad_scale<__half>(const AttnParams& p, int bh, int lane) {
    const int nr = p.rows_pad / 32, nk = (p.a.M + 31) / 32;
    float g = 0.f, v = 0.f;
    for (int i = lane; i < nr; i += 32) g = fmaxf(g, p.norm_rows[(long long)bh * nr + i]);
    for (int i = lane; i < nk; i += 32) v = fmaxf(v, p.norm_keys[(long long)bh * nk + i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    const float most = 2.f * sqrtf(g) * sqrtf(v);
    if (!(most > 0.f) || isinf(most)) return 1.f;
    int e;
    frexpf(most, &e);
    return ldexpf(1.f, -min(max(e, -100), 100));
}

// dV/dK/dQ += A[128 x 128 from tensor memory] B, B an image read over its rows. A is in 64 columns of
// its own (APART), or its pairs of 16 lie over the first half of the 32 scores that they came from.
template <bool APART> __device__ __forceinline__ uint32_t a_col(int part) { return part * (APART ? kCols / 2 : kCols); }
template <bool APART>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t img, uint32_t id, bool first) {
    const uint64_t bd = sdesc_mn(img);
#pragma unroll
    for (int s = 0; s < 8; ++s)
        mma_ts(d, a + a_col<APART>(s >> 1) + (s & 1) * 8, bd + s * 128, id, (!first || s > 0) ? 1u : 0u);
}

template <typename T, int DP>
__device__ __forceinline__ void dkv_cta(const AttnParams& p, const Maps& maps, const int block, unsigned char* dyn)
{
    using Sh = BwdShape<DP>;
    __shared__ uint64_t s_kv, s_full[Sh::stages], s_empty[Sh::stages], s_s, s_p, s_dp, s_ds, s_end;
    __shared__ uint64_t s_read[2], s_free[2];   // APART: S^T and dP^T read, P^T and dS^T used
    __shared__ volatile int s_issued;           // else: S^T tiles issued after the first
    constexpr bool APART = DP == 64;
    __shared__ uint32_t s_tmem;
    __shared__ int s_late;
    const Late late{&g_status, &s_late};
    __shared__ __align__(16) float s_row[2][2][128];   // -lse and -delta of the tile's rows, two tiles
    const sdtw_attention& a = p.a;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int heads = a.B * a.Hkv, bh = block % heads;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int RT = p.tile_rows, G = p.G;
    const int j0 = block / heads * kKeys;   // the first keys are seen by the most rows
    const RowRange rr(a, b);
    // tiles of packed rows that see a key of this CTA
    const RowRange::Rows rows = rr.seeing(j0, j0 + kKeys, G);
    int t_lo = rows.lo / RT, t_hi = (rows.hi + RT - 1) / RT;
    t_lo = uniform(t_lo), t_hi = uniform(t_hi);
    const int tiles = t_hi - t_lo;

    const uint32_t base = smem_u32(dyn);
    const uint32_t k_img = base, v_img = base + Sh::tile, ring = base + 2 * Sh::tile;
    if (threadIdx.x == 0) {
        s_late = 0;
        mbar_init(smem_u32(&s_kv), 1);
        for (int e = 0; e < Sh::stages; ++e) {
            mbar_init(smem_u32(&s_full[e]), 1);
            mbar_init(smem_u32(&s_empty[e]), 2);   // both issuing warps
        }
        mbar_init(smem_u32(&s_s), 1);
        mbar_init(smem_u32(&s_p), kWorkers);
        mbar_init(smem_u32(&s_dp), 1);
        mbar_init(smem_u32(&s_ds), kWorkers);
        mbar_init(smem_u32(&s_end), 2);
        s_issued = 0;
        for (int k = 0; k < 2; ++k) {
            mbar_init(smem_u32(&s_read[k]), kWorkers);
            mbar_init(smem_u32(&s_free[k]), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (RT < 128 && warp < kWorkers)   // rows that no load writes, but the products over the rows read
        for (int i = warp; i < 2 * Sh::stages; i += kWorkers) clear_rows<DP>(ring + i * Sh::tile, RT, lane);
    if (warp == kIssuer) tmem_alloc(&s_tmem, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
    const uint32_t c_s = tmem, c_dp = tmem + 128, c_dv = tmem + 256, c_dk = c_dv + DP;
    const uint32_t c_p = APART ? tmem + 384 : c_s, c_ds = APART ? tmem + 448 : c_dp;   // 16-bit operands
    bool ok = true;

    if (warp == kLoader) {
        if (lane == 0 && tiles > 0 && p.skip != 1) {
            mbar_expect_tx(smem_u32(&s_kv), 2 * Sh::tile);
            load_keys<DP>(k_img, &maps.k, j0, hk, b, smem_u32(&s_kv));
            load_keys<DP>(v_img, &maps.v, j0, hk, b, smem_u32(&s_kv));
            const uint32_t bytes = 2u * RT * 128 * (DP / 64);
            int issued = 0;
            for (int i = 0; i < tiles && ok; ++i) {
                const int e = i % Sh::stages;
                if (i >= Sh::stages) wait_for(ok, smem_u32(&s_empty[e]), (uint32_t)((i / Sh::stages - 1) & 1), p.wait_ns, late);
                if (!ok) break;
                const uint32_t bar = smem_u32(&s_full[e]), dst = ring + e * 2 * Sh::tile;
                const int n0 = (t_lo + i) * (RT / G);
                mbar_expect_tx(bar, bytes);
                load_rows<DP>(dst, &maps.q, n0, hk, b, bar);
                load_rows<DP>(dst + Sh::tile, &maps.dout, n0, hk, b, bar);
                issued = i + 1;
            }
            bool drained = true;   // no copy may be writing shared memory when the CTA ends
            for (int i = max(0, issued - Sh::stages); i < issued; ++i)
                wait_for(drained, smem_u32(&s_full[i % Sh::stages]), (uint32_t)((i / Sh::stages) & 1), p.wait_ns, late);
            wait_for(drained, smem_u32(&s_kv), 0, p.wait_ns, late);
        }
        __syncwarp();
    } else if (warp >= kIssuer) {
        // one warp: S^T, then dV += P^T dO; the other: dP^T, then dK += dS^T Q
        const bool grad = warp == kIssuer + 1;
        const int steps = (a.D + 15) / 16;
        const uint32_t id_s = idesc<T>(128, 128, false), id_o = idesc<T>(128, steps * 16, true);
        const uint32_t col = grad ? c_dp : c_s, acc = grad ? c_dk : c_dv, key_img = grad ? v_img : k_img;
        const uint32_t made = smem_u32(grad ? &s_dp : &s_s), ready = smem_u32(grad ? &s_ds : &s_p);
        // rows of the first tile before `head`, which see no key, and rows from `rows_b` on hold anything
        const int head = rr.first_row() * G - t_lo * RT, rows_b = rr.n_b * G;
        if (tiles > 0) wait_warp(ok, smem_u32(&s_kv), 0, p.wait_ns, late);
        const uint32_t operand = grad ? c_ds : c_p;
        int e = 0, pe = 0;   // ring entries of the next scores and of the next product with rows
        uint32_t ph = 0;
        auto scores = [&](int i) {
            const uint32_t img = ring + (uint32_t)e * 2 * Sh::tile;
            wait_warp(ok, smem_u32(&s_full[e]), ph, p.wait_ns, late);
            const int tail = rows_b - (t_lo + i) * RT;
            if (ok && tail < RT && rr.n_b < a.N) {   // both warps: the same zeros
                clear_rows<DP>(img, tail, lane);
                clear_rows<DP>(img + Sh::tile, tail, lane);
            }
            if (ok && i == 0 && head > 0) {
                clear_rows<DP>(img, 0, lane, head);
                clear_rows<DP>(img + Sh::tile, 0, lane, head);
            }
            fence_after_sync();
            if (ok && elect_one()) {
                mma_features<DP / 16>(col, key_img, img + (grad ? Sh::tile : 0), steps, id_s);
                mma_commit(made);
            }
            __syncwarp();
            if (++e == Sh::stages) e = 0, ph ^= 1;
        };
        if (tiles > 0) scores(0);
        for (int i = 0; i < tiles; ++i) {
            if (APART && i + 1 < tiles) {
                wait_warp(ok, smem_u32(&s_read[grad]), (uint32_t)(i & 1), p.wait_ns, late);
                scores(i + 1);
            }
            // dV takes dO, dK takes Q
            const uint32_t rows_img = ring + (uint32_t)pe * 2 * Sh::tile + (grad ? 0 : Sh::tile);
            if (p.skip == 2 && i + 1 == tiles) late.set(), ok = false;   // test hook: gives up
            wait_warp(ok, ready, (uint32_t)(i & 1), p.wait_ns, late);
            // dK and the next dP^T would interleave with the next S^T, which the warps wait for first. Only
            // the order in the queue hangs on this, so it waits a while and no longer.
            if (!APART && grad && i + 1 < tiles)
                for (int k = 0; k < 1000 && s_issued <= i; ++k) __nanosleep(20);
            fence_after_sync();
            if (ok && elect_one()) {
                mma_rows<APART>(acc, operand, rows_img, id_o, i == 0);
                mma_commit(smem_u32(&s_empty[pe]));
                if (APART) mma_commit(smem_u32(&s_free[grad]));
            }
            __syncwarp();
            if (++pe == Sh::stages) pe = 0;
            if (!APART && i + 1 < tiles) scores(i + 1);
            if (!APART && !grad && lane == 0) s_issued = i + 1;
        }
        if (lane == 0) {
            mma_commit(smem_u32(&s_end));
            bool fin = true;
            wait_for(fin, smem_u32(&s_end), 0, p.wait_ns, late);
        }
        __syncwarp();
    } else {
        const int part = warp >> 2, quarter = warp & 3;   // columns and rows of a tile
        const int key = j0 + quarter * 32 + lane;
        const bool live = key < rr.m_b;
        // packed rows that see this key
        const int rlo = live ? rr.row_lo(key) * G : 0, rhi = live ? max(rlo, rr.row_hi(key) * G) : 0;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const float s2 = a.scale * kLog2e;
        const float gs = grad_scale<T>(p, bh, lane);
        const unsigned long long mul = pk2(s2, s2), gmul = pk2(gs, gs);
        const long long info = (long long)bh * p.rows_pad;
        const int mine = threadIdx.x & 127, which = (threadIdx.x >> 7) & 1;
        // this thread's entry of a tile's row values, fetched two tiles ahead by 256 threads. The value
        // is only touched when it is put: an iteration waited 450 cycles for a negation of it
        const float* values = (which ? p.row_delta : p.row_lse) + info;
        auto valid = [&](int i) { return i < tiles && mine < RT && (t_lo + i) * RT + mine < p.rows; };
        auto fetch = [&](int i) { return valid(i) ? values[(t_lo + i) * RT + mine] : 0.f; };
        auto put = [&](int i, float v) { s_row[i & 1][which][mine] = which ? -gs * v : valid(i) ? -v : -INFINITY; };
        float next = 0.f;
        if (part < 2) {
            const float first = fetch(0);
            next = fetch(1);
            put(0, first);
        }
        // a wait that ran out does not end the loop: the other warps would wait at the barrier
        for (int i = 0; i < tiles; ++i) {
            work_sync();
            if (part < 2) {
                put(i + 1, next);
                next = fetch(i + 2);
            }
            const float4* lse4 = reinterpret_cast<const float4*>(s_row[i & 1][0] + part * kCols);
            const float4* del4 = reinterpret_cast<const float4*>(s_row[i & 1][1] + part * kCols);
            const int r0 = (t_lo + i) * RT + part * kCols;
            wait_warp(ok, smem_u32(&s_s), (uint32_t)(i & 1), p.wait_ns, late);
            fence_after_sync();
            float s[kCols];
            tmem_ld32_nowait(c_s + lanes + part * kCols, s);
            tmem_wait_ld();
            if (APART) done(s_read[0]);
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
                const float4 l = lse4[c / 4];
                upk2(fma2(pk2(s[c], s[c + 1]), mul, pk2(l.x, l.y)), s[c], s[c + 1]);
                upk2(fma2(pk2(s[c + 2], s[c + 3]), mul, pk2(l.z, l.w)), s[c + 2], s[c + 3]);
            }
            if (__any_sync(0xffffffffu, live && (r0 < rlo || r0 + kCols > rhi))) {
                const int first = rlo - r0, count = rhi - rlo;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if ((unsigned)(c - first) >= (unsigned)count) s[c] = -INFINITY;
            }
            uint32_t u[kCols / 2];
#pragma unroll
            for (int c = 0; c < kCols; c += 2) {
                s[c] = ex2(s[c]);
                s[c + 1] = ex2(s[c + 1]);
                u[c / 2] = pack2<T>(s[c], s[c + 1]);
            }
            if (APART && i > 0) {   // dV has taken the last probabilities
                wait_warp(ok, smem_u32(&s_free[0]), (uint32_t)((i - 1) & 1), p.wait_ns, late);
                fence_after_sync();
            }
            tmem_st16(c_p + lanes + a_col<APART>(part), u);
            tmem_wait_st();
            done(s_p);

            wait_warp(ok, smem_u32(&s_dp), (uint32_t)(i & 1), p.wait_ns, late);
            fence_after_sync();
            float d[kCols];
            tmem_ld32_nowait(c_dp + lanes + part * kCols, d);
            tmem_wait_ld();
            if (APART) done(s_read[1]);
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
                const float4 e = del4[c / 4];
                float x, y;
                upk2(mul2(pk2(s[c], s[c + 1]), fma2(pk2(d[c], d[c + 1]), gmul, pk2(e.x, e.y))), x, y);
                u[c / 2] = pack2<T>(x, y);
                upk2(mul2(pk2(s[c + 2], s[c + 3]), fma2(pk2(d[c + 2], d[c + 3]), gmul, pk2(e.z, e.w))), x, y);
                u[c / 2 + 1] = pack2<T>(x, y);
            }
            if (APART && i > 0) {   // dK has taken the last gradients
                wait_warp(ok, smem_u32(&s_free[1]), (uint32_t)((i - 1) & 1), p.wait_ns, late);
                fence_after_sync();
            }
            tmem_st16(c_ds + lanes + a_col<APART>(part), u);
            tmem_wait_st();
            done(s_ds);
        }
        if (tiles > 0) {
            wait_warp(ok, smem_u32(&s_end), 0, p.wait_ns, late);
            fence_after_sync();
        }
        ok = ok && !late.any();
        // half of the warpgroups write dV, half dK, each half of the features, through the images of K
        // and V
        constexpr int F = DP / 2;
        const bool is_k = part & 1;
        const int f0 = (part >> 1) * F;
        const float unlift = ex2(-(float)p.grad_shift), more = is_k ? a.scale / gs : 1.f;
        const bool some = tiles > 0 && live;
        const long long at = key < a.M ? (((long long)b * a.M + key) * a.Hkv + hk) * a.D + f0 : -1;
        write_rows<T, F>(base + (uint32_t)warp * 32 * F * 2, (is_k ? c_dk : c_dv) + lanes + f0, tiles > 0 && ok, false, ok && !some,
                         ok ? unlift : NAN, 0.f, more, is_k ? p.dk : p.dv, nullptr, at, min(F, a.D - f0) / 8, lane);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kIssuer) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int DP>
__device__ __forceinline__ void dq_cta(const AttnParams& p, const Maps& maps, const int block, unsigned char* dyn)
{
    using Sh = BwdShape<DP>;
    __shared__ uint64_t s_q, s_full[Sh::slots], s_empty[Sh::slots], s_s, s_sread, s_dp, s_dpread, s_ds[2], s_dsfree[2], s_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_late;
    const Late late{&g_status, &s_late};
    const sdtw_attention& a = p.a;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int heads = a.B * a.Hkv, bh = block % heads;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int RT = p.tile_rows, G = p.G;
    const int row_tiles = (p.rows + RT - 1) / RT;
    const int r0 = (row_tiles - 1 - block / heads) * RT;
    const RowRange rr(a, b);
    Tiles t(rr, r0, min(r0 + RT, p.rows), G);
    t.lo = uniform(t.lo), t.hi = uniform(t.hi);
    const int tiles = t.hi - t.lo;

    const uint32_t base = smem_u32(dyn);
    const uint32_t q_img = base, g_img = base + Sh::tile, ring = base + 2 * Sh::tile;
    if (threadIdx.x == 0) {
        s_late = 0;
        mbar_init(smem_u32(&s_q), 1);
        for (int e = 0; e < Sh::slots; ++e) {
            mbar_init(smem_u32(&s_full[e]), 1);
            mbar_init(smem_u32(&s_empty[e]), 1);
        }
        mbar_init(smem_u32(&s_s), 1);
        mbar_init(smem_u32(&s_sread), kWorkers);
        mbar_init(smem_u32(&s_dp), 1);
        mbar_init(smem_u32(&s_dpread), kWorkers);
        for (int k = 0; k < 2; ++k) {
            mbar_init(smem_u32(&s_ds[k]), kWorkers);
            mbar_init(smem_u32(&s_dsfree[k]), 1);
        }
        mbar_init(smem_u32(&s_end), 2);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuer) tmem_alloc(&s_tmem, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
    // scores are read at once and dS has columns of its own, twice: the next S and dP are made
    // meanwhile, and the next dS need not wait for the product with the last one
    const uint32_t c_s = tmem, c_dp = tmem + 128, c_ds = tmem + 256, c_dq = tmem + 384;
    bool ok = true;

    if (warp == kLoader) {
        if (lane == 0 && tiles > 0 && p.skip != 1) {
            mbar_expect_tx(smem_u32(&s_q), 2u * RT * 128 * (DP / 64));
            load_rows<DP>(q_img, &maps.q, r0 / G, hk, b, smem_u32(&s_q));
            load_rows<DP>(g_img, &maps.dout, r0 / G, hk, b, smem_u32(&s_q));
            int issued = 0;
            for (int i = 0; i < 2 * tiles && ok; ++i) {
                const int e = i % Sh::slots;
                if (i >= Sh::slots) wait_for(ok, smem_u32(&s_empty[e]), (uint32_t)((i / Sh::slots - 1) & 1), p.wait_ns, late);
                if (!ok) break;
                const uint32_t bar = smem_u32(&s_full[e]);
                mbar_expect_tx(bar, Sh::tile);
                load_keys<DP>(ring + e * Sh::tile, (i & 1) ? &maps.v : &maps.k, (t.lo + (i >> 1)) * kKeys, hk, b, bar);
                issued = i + 1;
            }
            bool drained = true;
            for (int i = max(0, issued - Sh::slots); i < issued; ++i)
                wait_for(drained, smem_u32(&s_full[i % Sh::slots]), (uint32_t)((i / Sh::slots) & 1), p.wait_ns, late);
            wait_for(drained, smem_u32(&s_q), 0, p.wait_ns, late);
        }
        __syncwarp();
    } else if (warp >= kIssuer) {
        // one warp: S(j); the other: dP(j), then dQ += dS K
        const bool grad = warp == kIssuer + 1;
        const int steps = (a.D + 15) / 16;
        const uint32_t id_s = idesc<T>(128, kKeys, false), id_o = idesc<T>(128, steps * 16, true);
        if (tiles > 0) wait_warp(ok, smem_u32(&s_q), 0, p.wait_ns, late);
        auto clear_tail = [&](int j, uint32_t kimg) {   // both warps: the same zeros
            const int tail = rr.m_b - (t.lo + j) * kKeys;
            if (ok && tail < kKeys && rr.m_b < a.M) clear_rows<DP>(kimg, tail, lane);
        };
        int e_k = 0, e_v = 1;   // ring entries of K(j) and V(j), and the parities of their arrivals
        uint32_t ph_k = 0, ph_v = 0;
        if (!grad) {
            for (int j = 0; j < tiles; ++j) {
                if (j > 0) wait_warp(ok, smem_u32(&s_sread), (uint32_t)((j - 1) & 1), p.wait_ns, late);
                wait_warp(ok, smem_u32(&s_full[e_k]), ph_k, p.wait_ns, late);
                const uint32_t kimg = ring + (uint32_t)e_k * Sh::tile;
                clear_tail(j, kimg);
                fence_after_sync();
                if (ok && elect_one()) {
                    mma_features<DP / 16>(c_s, q_img, kimg, steps, id_s);
                    mma_commit(smem_u32(&s_s));
                }
                __syncwarp();
                if ((e_k += 2) >= Sh::slots) e_k -= Sh::slots, ph_k ^= 1;
            }
        } else {
            auto upstream = [&]() {
                wait_warp(ok, smem_u32(&s_full[e_v]), ph_v, p.wait_ns, late);
                fence_after_sync();
                if (ok && elect_one()) {
                    mma_features<DP / 16>(c_dp, g_img, ring + (uint32_t)e_v * Sh::tile, steps, id_s);
                    mma_commit(smem_u32(&s_dp));
                    mma_commit(smem_u32(&s_empty[e_v]));
                }
                __syncwarp();
                if ((e_v += 2) >= Sh::slots) e_v -= Sh::slots, ph_v ^= 1;
            };
            if (tiles > 0) upstream();
            for (int j = 0; j < tiles; ++j) {
                if (j + 1 < tiles) {
                    wait_warp(ok, smem_u32(&s_dpread), (uint32_t)(j & 1), p.wait_ns, late);
                    upstream();
                }
                const uint32_t kimg = ring + (uint32_t)e_k * Sh::tile;
                if (p.skip == 2 && j + 1 == tiles) late.set(), ok = false;
                wait_warp(ok, smem_u32(&s_ds[j & 1]), (uint32_t)((j >> 1) & 1), p.wait_ns, late);
                clear_tail(j, kimg);
                fence_after_sync();
                if (ok && elect_one()) {
                    mma_rows<true>(c_dq, c_ds + (j & 1) * 64, kimg, id_o, j == 0);
                    mma_commit(smem_u32(&s_empty[e_k]));   // S(j) was done before dS(j)
                    mma_commit(smem_u32(&s_dsfree[j & 1]));
                }
                __syncwarp();
                if ((e_k += 2) >= Sh::slots) e_k -= Sh::slots;
            }
        }
        if (lane == 0) {
            mma_commit(smem_u32(&s_end));
            bool fin = true;
            wait_for(fin, smem_u32(&s_end), 0, p.wait_ns, late);
        }
        __syncwarp();
    } else {
        const int part = warp >> 2, quarter = warp & 3;   // columns and rows of a tile
        const int r = r0 + quarter * 32 + lane;
        const bool mine = quarter * 32 + lane < RT && r < p.rows;
        const int n = mine ? r / G : 0, h = hk * G + (mine ? r % G : 0);
        const bool live = mine && n < rr.n_b;
        const int klo = live ? rr.lo(n) : 0, khi = live ? max(klo, rr.hi(n)) : 0;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const float s2 = a.scale * kLog2e;
        const float gs = grad_scale<T>(p, bh, lane);
        const long long info = (long long)bh * p.rows_pad + r;
        const float nlse = live ? -p.row_lse[info] : -INFINITY, ndel = live ? -gs * p.row_delta[info] : 0.f;
        const unsigned long long mul = pk2(s2, s2), sub = pk2(nlse, nlse), gmul = pk2(gs, gs), gsub = pk2(ndel, ndel);
        for (int j = 0; j < tiles; ++j) {
            const int j0 = (t.lo + j) * kKeys + part * kCols;
            wait_warp(ok, smem_u32(&s_s), (uint32_t)(j & 1), p.wait_ns, late);
            fence_after_sync();
            float s[kCols];
            tmem_ld32_nowait(c_s + lanes + part * kCols, s);
            tmem_wait_ld();
            done(s_sread);
#pragma unroll
            for (int c = 0; c < kCols; c += 2) upk2(fma2(pk2(s[c], s[c + 1]), mul, sub), s[c], s[c + 1]);
            const bool edge = __any_sync(0xffffffffu, live && (j0 < klo || j0 + kCols > khi));
            const int first = klo - j0, count = khi - klo;
            if (edge) {
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if ((unsigned)(c - first) >= (unsigned)count) s[c] = -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < kCols; ++c) s[c] = ex2(s[c]);
            wait_warp(ok, smem_u32(&s_dp), (uint32_t)(j & 1), p.wait_ns, late);
            fence_after_sync();
            float d[kCols];
            tmem_ld32_nowait(c_dp + lanes + part * kCols, d);
            tmem_wait_ld();
            done(s_dpread);
            if (edge) {   // dP of a key beyond the length may be NaN
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if ((unsigned)(c - first) >= (unsigned)count) d[c] = 0.f;
            }
            uint32_t u[kCols / 2];
#pragma unroll
            for (int c = 0; c < kCols; c += 2) {
                float x, y;
                upk2(mul2(pk2(s[c], s[c + 1]), fma2(pk2(d[c], d[c + 1]), gmul, gsub)), x, y);
                u[c / 2] = pack2<T>(x, y);
            }
            if (j > 1) {   // dQ has taken the gradients before the last
                wait_warp(ok, smem_u32(&s_dsfree[j & 1]), (uint32_t)(((j >> 1) - 1) & 1), p.wait_ns, late);
                fence_after_sync();
            }
            tmem_st16(c_ds + (j & 1) * 64 + lanes + a_col<true>(part), u);
            tmem_wait_st();
            done(s_ds[j & 1]);
        }
        if (tiles > 0) {
            wait_warp(ok, smem_u32(&s_end), 0, p.wait_ns, late);
            fence_after_sync();
        }
        ok = ok && !late.any();
        // a warpgroup writes 32 features, through the images of Q and dO
        const float unlift = ex2(-(float)p.grad_shift), more = a.scale / gs;
        const int f0 = part * 32;
        if (f0 < DP) {
            const long long at = mine ? (((long long)b * a.N + n) * a.Hq + h) * a.D + f0 : -1;
            write_rows<T, 32>(base + (uint32_t)warp * 32 * 64, c_dq + lanes + f0, tiles > 0 && ok, false,
                              ok && !(live && klo < khi && tiles > 0), ok ? unlift : NAN, 0.f, more, p.dq, nullptr, at, min(32, a.D - f0) / 8, lane);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kIssuer) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreadsB, 1) attn_bwd_tc_kernel(const AttnParams p, const __grid_constant__ Maps maps, const int dkv)
{
    extern __shared__ __align__(1024) unsigned char dyn[];   // as the swizzle of the images asks
    if (threadIdx.x == kWork) prefetch_map(&maps.q), prefetch_map(&maps.k), prefetch_map(&maps.v), prefetch_map(&maps.dout);
    if ((int)blockIdx.x < dkv) dkv_cta<T, DP>(p, maps, (int)blockIdx.x, dyn);
    else dq_cta<T, DP>(p, maps, (int)blockIdx.x - dkv, dyn);
}

template <typename T, int DP> cudaError_t run_bwd(const AttnParams& p, const Maps& m, cudaStream_t s)
{
    using Sh = BwdShape<DP>;
    constexpr uint32_t smem = Sh::smem_dkv > Sh::smem_dq ? Sh::smem_dkv : Sh::smem_dq;
    const cudaError_t e = allow_smem<attn_bwd_tc_kernel<T, DP>>(smem);
    if (e != cudaSuccess) return e;
    const int heads = p.a.B * p.a.Hkv;
    const int dkv = p.dk ? (p.a.M + kKeys - 1) / kKeys * heads : 0;
    const int dq = p.dq ? (p.rows + p.tile_rows - 1) / p.tile_rows * heads : 0;
    attn_bwd_tc_kernel<T, DP><<<(unsigned)(dkv + dq), kThreadsB, smem, s>>>(p, m, dkv);
    return cudaGetLastError();
}

}  // namespace
}  // namespace atc

cudaError_t launch_attn_backward_tc(const AttnParams& p, cudaStream_t s)
{
    atc::Maps m{};
    const sdtw_attention& a = p.a;
    const long long flat[3] = {(long long)a.N * a.Hq * a.D, (long long)a.Hq * a.D, a.D};
    if (!atc::map_rows(&m.q, a.q, a.q_stride, a, p.G, p.tile_rows) || !atc::map_rows(&m.dout, p.dout, flat, a, p.G, p.tile_rows) ||
        !atc::map_keys(&m.k, a.k, a.k_stride, a) || !atc::map_keys(&m.v, a.v, a.v_stride, a))
        return cudaErrorInvalidValue;
    if (a.dtype == SDTW_BF16)
        return a.D <= 64 ? atc::run_bwd<__nv_bfloat16, 64>(p, m, s) : atc::run_bwd<__nv_bfloat16, 128>(p, m, s);
    return a.D <= 64 ? atc::run_bwd<__half, 64>(p, m, s) : atc::run_bwd<__half, 128>(p, m, s);
}

cudaError_t attn_backward_take_status(int* out, cudaStream_t s)
{
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, atc::g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbolAsync(atc::g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e;
}

}  // namespace sdtw
