// encoder_api.cu -- the C ABI of the sequence-encoder operators: validation on the host
// before any launch, workspace carving and launches on the caller's stream.
#include <cmath>

#include "encoder.h"
#include "kernels.h"

using namespace sdtw;

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

bool good_dtype(int d) { return d == SDTW_F32 || d == SDTW_BF16 || d == SDTW_F16; }

int device_sms()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 152;
    return n;
}

sdtw_status check_ws(const void* ws, size_t have, size_t need)
{
    if (need == 0) return SDTW_OK;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) || have < need) return SDTW_ERR_WORKSPACE;
    return SDTW_OK;
}

sdtw_status check_norm(long long rows, int C, int dtype, int wdtype)
{
    if (rows < 1 || C < 1) return SDTW_ERR_EMPTY;
    if (!good_dtype(dtype) || !good_dtype(wdtype)) return SDTW_ERR_ARG;
    if (rows > (1ll << 40) || C > (1 << 24)) return SDTW_ERR_TOO_LARGE;
    return SDTW_OK;
}

sdtw_status check_attention(const sdtw_attention* a)
{
    if (!a) return SDTW_ERR_ARG;
    if (a->B < 1 || a->N < 1 || a->M < 1 || a->Hq < 1 || a->Hkv < 1 || a->D < 1) return SDTW_ERR_EMPTY;
    if (a->Hq % a->Hkv) return SDTW_ERR_SHAPE;
    if (!a->q || !a->k || !a->v || !good_dtype(a->dtype)) return SDTW_ERR_ARG;
    if (a->window_left < -1 || a->window_right < -1) return SDTW_ERR_ARG;
    if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return SDTW_ERR_ARG;
    // 32-bit positions, packed rows and grids (of at least 64-row tiles)
    const long long G = a->Hq / a->Hkv, heads = (long long)a->B * a->Hkv, most = 1ll << 27;
    if (a->D > 128 || a->N * G > most || a->M > most || heads > most || ((a->N * G + 63) / 64) * heads > most || ((a->M + 63ll) / 64) * heads > most ||
        (a->N * G + 127) / 8 * heads > most)
        return SDTW_ERR_TOO_LARGE;
    return SDTW_OK;
}

// Shares of the key axis. Row tiles that alone would leave SMs idle are split along their
// keys, and the shares joined by a second launch. A CTA takes `fixed` us and `tile` us a key
// tile, `waves` of them follow one another on an SM; joining takes a launch and the shares'
// fp32 rows twice through memory. The least sum of these is taken.
int key_splits(const AttnParams& p, int tile_rows, int tile_keys, int resident, double fixed, double tile)
{
    const sdtw_attention& a = p.a;
    const long long ctas = (long long)((p.rows + tile_rows - 1) / tile_rows) * a.B * a.Hkv;
    const long long slots = (long long)device_sms() * resident;
    if (ctas >= slots) return 1;
    long long keys = a.M;   // that a tile of rows sees at the most
    if (p.a.window_left >= 0 && p.a.window_right >= 0) {
        const long long span = (long long)p.a.window_left + p.a.window_right + (tile_rows - 1) / p.G + 1 + tile_keys;
        if (span < keys) keys = span;
    }
    const int tiles = (int)((keys + tile_keys - 1) / tile_keys);
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= tiles && s <= 128; ++s) {
        const double rounds = (double)((ctas * s + slots - 1) / slots);
        const double join = s == 1 ? 0. : 5. + 1e-6 * 2. * s * (double)(a.B * (long long)a.Hkv * p.rows) * a.D * 4. / 5.;
        const double cost = rounds * (fixed + tile * ((tiles + s - 1) / s)) + join;
        if (cost < least) least = cost, best = s;
    }
    return best;
}

AttnParams attn_params(const sdtw_attention* a)
{
    AttnParams p{};
    p.a = *a;
    // a window that reaches past every key is none (and its sums stay within 32 bits)
    if (p.a.window_left >= a->N + a->M) p.a.window_left = -1;
    if (p.a.window_right >= a->N + a->M) p.a.window_right = -1;
    p.G = a->Hq / a->Hkv;
    p.rows = a->N * p.G;
    p.rows_pad = (p.rows + 127) / 128 * 128;
    p.tc = attn_tc_fits(*a);
    p.packed = a->D % 4 == 0 && aligned16(a->q) && aligned16(a->k) && aligned16(a->v);
    for (int i = 0; i < 3; ++i) p.packed = p.packed && a->q_stride[i] % 4 == 0 && a->k_stride[i] % 4 == 0 && a->v_stride[i] % 4 == 0;
    p.tile_rows = p.tc ? 128 / p.G * p.G : 64;
    // Row tiles of a tensor-core CTA: see attn_fwd_tc.cu. A single row tile (new samples over a
    // cache) has its key tiles done two at a time.
    const bool single = p.rows <= p.tile_rows;
    const long long tiles = (long long)((p.rows + p.tile_rows - 1) / p.tile_rows) * a->B * a->Hkv;
    p.row_tiles = single ? (a->M > 128 ? 2 : 1) : a->D <= 64 || tiles < 2ll * device_sms() ? 1 : 2;
    p.few = !p.tc && p.packed && p.rows <= 12;   // see attn.cu
    if (!p.tc) p.splits = p.few ? key_splits(p, 4, 64, p.rows == 1 ? 2 : 1, 3., 0.5) : key_splits(p, 64, 64, 2, 3., 2.);
    else if (single && p.row_tiles == 2) p.splits = key_splits(p, p.tile_rows, 256, 1, 5., 1.5);
    else p.splits = key_splits(p, p.row_tiles * p.tile_rows, 128, p.row_tiles == 1 && a->D <= 64 ? 2 : 1, 5., 1.5);
    p.grad_shift = 32;
    p.wait_ns = debug_wait_ns();
    return p;
}

size_t carve_forward(AttnParams& p, void* ws)
{
    if (p.splits <= 1) return 0;
    const size_t rows = (size_t)p.splits * p.a.B * p.a.Hkv * p.rows;
    char* base = static_cast<char*>(ws);
    p.part_o = reinterpret_cast<float*>(base);
    const size_t o = align_up(rows * p.a.D * sizeof(float));
    p.part_lse = reinterpret_cast<float*>(base + o);
    return o + align_up(rows * sizeof(float));
}

size_t carve_backward(AttnParams& p, void* ws)
{
    const size_t rows = align_up((size_t)p.a.B * p.a.Hkv * p.rows_pad * sizeof(float));
    char* base = static_cast<char*>(ws);
    p.row_lse = reinterpret_cast<float*>(base);
    p.row_delta = reinterpret_cast<float*>(base + rows);
    size_t o = 2 * rows;
    if (p.tc && p.a.dtype == SDTW_F16) {
        const size_t heads = (size_t)p.a.B * p.a.Hkv;
        p.norm_rows = reinterpret_cast<float*>(base + o);
        o += align_up(heads * (p.rows_pad / 32) * sizeof(float));
        p.norm_keys = reinterpret_cast<float*>(base + o);
        o += align_up(heads * ((p.a.M + 31) / 32) * sizeof(float));
        p.grad_shift = 15;
    }
    return o;
}

}  // namespace

namespace sdtw {

// The tensor-core kernels take 16-bit elements whose rows TMA can load: 16-byte
// addresses and strides, none of them 0 (broadcast), and a group of heads within one tile.
bool attn_tc_fits(const sdtw_attention& a)
{
    if (a.dtype == SDTW_F32 || a.D % 8 || a.Hq / a.Hkv > 128) return false;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v)) return false;
    const int qs[3] = {a.B, a.N, a.Hq}, ks[3] = {a.B, a.M, a.Hkv};
    for (int i = 0; i < 3; ++i) {
        if (qs[i] > 1 && (a.q_stride[i] <= 0 || a.q_stride[i] % 8)) return false;
        if (ks[i] > 1 && (a.k_stride[i] <= 0 || a.k_stride[i] % 8 || a.v_stride[i] <= 0 || a.v_stride[i] % 8)) return false;
    }
    return true;
}

}  // namespace sdtw

namespace {

#define ENC_CUDA(call)                                 \
    do {                                               \
        if ((call) != cudaSuccess) return SDTW_ERR_CUDA; \
    } while (0)

}  // namespace

extern "C" {

sdtw_status sdtw_layernorm_forward(const void* x, const void* weight, const void* bias, long long rows, int C,
                                   float eps, int dtype, int wdtype, void* y, float* mean, float* rstd, void* stream)
{
    if (sdtw_status s = check_norm(rows, C, dtype, wdtype)) return s;
    if (!x || !y || (!mean != !rstd) || !(eps >= 0.f) || !std::isfinite(eps)) return SDTW_ERR_ARG;
    NormParams p{};
    p.x = x, p.weight = weight, p.bias = bias, p.y = y, p.mean = mean, p.rstd = rstd;
    p.rows = rows, p.C = C, p.dtype = dtype, p.wdtype = wdtype, p.eps = eps;
    ENC_CUDA(launch_norm_forward(p, static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

size_t sdtw_layernorm_workspace_bytes(long long rows, int C)
{
    if (check_norm(rows, C, SDTW_F32, SDTW_F32) != SDTW_OK) return 0;
    return align_up(2 * sizeof(float) * (size_t)norm_partial_ctas(rows, device_sms()) * C);
}

sdtw_status sdtw_layernorm_backward(const void* dy, const void* x, const void* weight, const float* mean,
                                    const float* rstd, long long rows, int C, int dtype, int wdtype, void* dx,
                                    void* dweight, void* dbias, void* ws, size_t ws_bytes, void* stream)
{
    if (sdtw_status s = check_norm(rows, C, dtype, wdtype)) return s;
    if (!dy || !x || !mean || !rstd) return SDTW_ERR_ARG;
    if (!dx && !dweight && !dbias) return SDTW_OK;
    NormParams p{};
    if (dweight || dbias) {
        if (sdtw_status s = check_ws(ws, ws_bytes, sdtw_layernorm_workspace_bytes(rows, C))) return s;
        p.partial = static_cast<float*>(ws);
    }
    p.dy = dy, p.x = x, p.weight = weight, p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd);
    p.dx = dx, p.dweight = dweight, p.dbias = dbias;
    p.rows = rows, p.C = C, p.dtype = dtype, p.wdtype = wdtype;
    ENC_CUDA(launch_norm_backward(p, norm_partial_ctas(rows, device_sms()), static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

sdtw_status sdtw_rotary(const void* q, const long long* q_stride, const void* k, const long long* k_stride, int B,
                        int N, int Hq, int Hkv, int D, int R, const float* table, int length, const int* positions,
                        long long pos_stride_b, int interleaved, int inverse, int dtype, void* q_out, void* k_out,
                        void* stream)
{
    if (B < 1 || N < 1 || Hq < 1 || D < 1 || length < 1 || (k && Hkv < 1)) return SDTW_ERR_EMPTY;
    if (!q || !q_stride || !q_out || !table || !good_dtype(dtype) || (!k != !k_out) || (k && !k_stride))
        return SDTW_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(table) & 7) return SDTW_ERR_ARG;   // a pair's cosine and sine are one load
    if (R < 2 || R % 2 || R > D) return SDTW_ERR_SHAPE;
    if (positions ? (pos_stride_b != 0 && pos_stride_b < N) : N > length) return SDTW_ERR_SHAPE;
    if (D > (1 << 20) || Hq > (1 << 20) || (k && Hkv > (1 << 20))) return SDTW_ERR_TOO_LARGE;
    RotaryParams p{};
    p.in[0] = q, p.in[1] = k, p.out[0] = q_out, p.out[1] = k_out;
    for (int i = 0; i < 3; ++i) {
        p.stride[0][i] = q_stride[i];
        p.stride[1][i] = k ? k_stride[i] : 0;
    }
    p.H[0] = Hq, p.H[1] = k ? Hkv : 0;
    p.table = table, p.positions = positions, p.pos_stride_b = pos_stride_b;
    p.B = B, p.N = N, p.D = D, p.R = R, p.length = length;
    p.dtype = dtype, p.interleaved = interleaved != 0, p.inverse = inverse != 0;
    ENC_CUDA(launch_rotary(p, static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

size_t sdtw_attention_workspace_bytes(const sdtw_attention* a, int backward)
{
    if (check_attention(a) != SDTW_OK) return 0;
    AttnParams p = attn_params(a);
    return backward ? carve_backward(p, nullptr) : carve_forward(p, nullptr);
}

sdtw_status sdtw_attention_forward(const sdtw_attention* a, void* out, void* out_rest, float* lse, void* ws,
                                   size_t ws_bytes, void* stream)
{
    if (sdtw_status s = check_attention(a)) return s;
    if (!out) return SDTW_ERR_ARG;
    AttnParams p = attn_params(a);
    if (sdtw_status s = check_ws(ws, ws_bytes, carve_forward(p, ws))) return s;
    p.out = out, p.out_rest = out_rest, p.lse = lse;
    if (p.tc && !(aligned16(out) && aligned16(out_rest))) p.tc = false;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.tc) p.skip = debug_take_skip_publish();
    ENC_CUDA(p.tc ? launch_attn_forward_tc(p, st) : launch_attn_forward_simt(p, st));
    if (p.splits > 1) ENC_CUDA(launch_attn_combine(p, st));
    return SDTW_OK;
}

sdtw_status sdtw_attention_backward(const sdtw_attention* a, const void* out, const void* out_rest,
                                    const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws,
                                    size_t ws_bytes, void* stream)
{
    if (sdtw_status s = check_attention(a)) return s;
    if (!out || !lse || !dout || (!dk != !dv)) return SDTW_ERR_ARG;
    if (!dq && !dk) return SDTW_OK;
    AttnParams p = attn_params(a);
    if (sdtw_status s = check_ws(ws, ws_bytes, carve_backward(p, ws))) return s;
    p.out = const_cast<void*>(out), p.out_rest = const_cast<void*>(out_rest), p.lse_in = lse, p.dout = dout, p.dq = dq, p.dk = dk, p.dv = dv;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // results of another alignment than torch's go the general way
    if (p.tc && !(aligned16(out) && aligned16(dout) && aligned16(dq) && aligned16(dk) && aligned16(dv))) {
        p.tc = false;
        p.norm_rows = p.norm_keys = nullptr;
        p.grad_shift = 32;
    }
    p.packed = p.packed && aligned16(dout);
    if (p.tc) p.skip = debug_take_skip_publish();
    ENC_CUDA(launch_attn_rowinfo(p, st));
    ENC_CUDA(p.tc ? launch_attn_backward_tc(p, st) : launch_attn_backward_simt(p, st));
    return SDTW_OK;
}

sdtw_status sdtw_encoder_status(void* stream)
{
    int forward = 0, backward = 0;
    ENC_CUDA(attn_forward_take_status(&forward, static_cast<cudaStream_t>(stream)));
    ENC_CUDA(attn_backward_take_status(&backward, static_cast<cudaStream_t>(stream)));
    return forward || backward ? SDTW_ERR_TIMEOUT : SDTW_OK;
}

}  // extern "C"
