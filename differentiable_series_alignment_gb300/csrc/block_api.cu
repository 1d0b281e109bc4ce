// block_api.cu -- the C ABI of group norm, gated recurrence and gated linear units: validation on the host before any
// launch, and launches on the caller's stream.
#include <cmath>

#include "block.h"
#include "kernels.h"

using namespace sdtw;

namespace {

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
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || have < need) return SDTW_ERR_WORKSPACE;
    return SDTW_OK;
}

sdtw_status check_group_norm(int B, int S, int G, int C, int dtype, int wdtype)
{
    if (B < 1 || S < 1 || G < 1 || C < 1) return SDTW_ERR_EMPTY;
    if (C % G) return SDTW_ERR_SHAPE;
    if (!good_dtype(dtype) || !good_dtype(wdtype)) return SDTW_ERR_ARG;
    // 32-bit grids and counts of a group's values in fp32's and the workspace's reach
    if (B > (1 << 30) || C > (1 << 24) || (long long)B * G > 0x7fffffffll || (long long)S * C > (1ll << 40) || (long long)B * C > (1ll << 40)) return SDTW_ERR_TOO_LARGE;
    return SDTW_OK;
}

sdtw_status check_recurrence(const sdtw_recurrence* a)
{
    if (!a) return SDTW_ERR_ARG;
    if (a->B < 1 || a->N < 1 || a->C < 1) return SDTW_ERR_EMPTY;
    if (!a->x || !a->gate || !good_dtype(a->dtype)) return SDTW_ERR_ARG;
    // 32-bit positions and grids, and offsets of 128 positions
    const auto far = [](long long stride) { return stride > (1 << 23) || stride < -(1 << 23); };
    if (a->N >= (1 << 30) || a->C > (1 << 23) || far(a->x_stride[1]) || far(a->gate_stride[1]) || (long long)a->B * ((a->C + 31ll) / 32) > 0x7fffffffll)
        return SDTW_ERR_TOO_LARGE;
    return SDTW_OK;
}

sdtw_status check_gated(const sdtw_gated* a)
{
    if (!a) return SDTW_ERR_ARG;
    if (a->R < 1 || a->K < 1 || a->F < 1) return SDTW_ERR_EMPTY;
    if (!a->x || !a->gate_weight || !a->up_weight || !good_dtype(a->dtype)) return SDTW_ERR_ARG;
    if (a->activation < SDTW_ACT_SILU || a->activation > SDTW_ACT_SIGMOID) return SDTW_ERR_ARG;
    // 32-bit coordinates, tiles and grids
    if (a->R > (1ll << 30) || a->K > (1 << 20) || a->F > (1 << 20) || a->R * a->K > (1ll << 40) || a->R * a->F > (1ll << 38)) return SDTW_ERR_TOO_LARGE;
    return SDTW_OK;
}

#define BLOCK_CUDA(call)                                 \
    do {                                                 \
        if ((call) != cudaSuccess) return SDTW_ERR_CUDA; \
    } while (0)

}  // namespace

extern "C" {

size_t sdtw_groupnorm_workspace_bytes(int B, int S, int G, int C, int dtype, int backward)
{
    if (check_group_norm(B, S, G, C, dtype, SDTW_F32) != SDTW_OK) return 0;
    GroupNormParams p{};
    p.B = B, p.S = S, p.G = G, p.C = C, p.cg = C / G, p.dtype = dtype;
    return group_norm_workspace(p, backward != 0, device_sms());
}

sdtw_status sdtw_groupnorm_forward(const void* x, const void* weight, const void* bias, const int* lengths, int B, int S,
                                   int G, int C, float eps, int activation, int dtype, int wdtype, void* y, float* mean,
                                   float* rstd, void* ws, size_t ws_bytes, void* stream)
{
    if (sdtw_status s = check_group_norm(B, S, G, C, dtype, wdtype)) return s;
    if (!x || !y || (!mean != !rstd) || !(eps >= 0.f) || !std::isfinite(eps)) return SDTW_ERR_ARG;
    if (activation < SDTW_ACT_NONE || activation > SDTW_ACT_RELU) return SDTW_ERR_ARG;
    if (sdtw_status s = check_ws(ws, ws_bytes, sdtw_groupnorm_workspace_bytes(B, S, G, C, dtype, 0))) return s;
    GroupNormParams p{};
    p.x = x, p.weight = weight, p.bias = bias, p.lengths = lengths, p.y = y, p.mean = mean, p.rstd = rstd;
    p.B = B, p.S = S, p.G = G, p.C = C, p.cg = C / G;
    p.eps = eps, p.activation = activation, p.dtype = dtype, p.wdtype = wdtype;
    p.partial = static_cast<float*>(ws);
    BLOCK_CUDA(launch_group_norm_forward(p, device_sms(), static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

sdtw_status sdtw_groupnorm_backward(const void* dy, const void* x, const void* weight, const void* bias, const int* lengths,
                                    const float* mean, const float* rstd, int B, int S, int G, int C, int activation,
                                    int dtype, int wdtype, void* dx, void* dweight, void* dbias, void* ws, size_t ws_bytes,
                                    void* stream)
{
    if (sdtw_status s = check_group_norm(B, S, G, C, dtype, wdtype)) return s;
    if (!dy || !x || !mean || !rstd) return SDTW_ERR_ARG;
    if (activation < SDTW_ACT_NONE || activation > SDTW_ACT_RELU) return SDTW_ERR_ARG;
    if (!dx && !dweight && !dbias) return SDTW_OK;
    if (sdtw_status s = check_ws(ws, ws_bytes, sdtw_groupnorm_workspace_bytes(B, S, G, C, dtype, 1))) return s;
    GroupNormParams p{};
    p.dy = dy, p.x = x, p.weight = weight, p.bias = bias, p.lengths = lengths;
    p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd);
    p.dx = dx, p.dweight = dweight, p.dbias = dbias;
    p.B = B, p.S = S, p.G = G, p.C = C, p.cg = C / G;
    p.activation = activation, p.dtype = dtype, p.wdtype = wdtype;
    p.partial = static_cast<float*>(ws);
    BLOCK_CUDA(launch_group_norm_backward(p, device_sms(), static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

sdtw_status sdtw_recurrence_forward(const sdtw_recurrence* a, void* h, float* last, float* kept, void* stream)
{
    if (sdtw_status s = check_recurrence(a)) return s;
    if (!h) return SDTW_ERR_ARG;
    RecurrenceParams p{};
    p.a = *a, p.h = h, p.last = last, p.kept = kept;
    p.wait_ns = debug_wait_ns(), p.skip = debug_take_skip_publish();
    BLOCK_CUDA(launch_recurrence_forward(p, device_sms(), static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

sdtw_status sdtw_recurrence_backward(const sdtw_recurrence* a, const float* kept, const void* dh, const float* dlast, void* dx,
                                     void* dgate, float* dstate, void* stream)
{
    if (sdtw_status s = check_recurrence(a)) return s;
    if (!kept || !dx || !dgate) return SDTW_ERR_ARG;
    RecurrenceParams p{};
    p.a = *a, p.kept_in = kept, p.dh = dh, p.dlast = dlast, p.dx = dx, p.dgate = dgate, p.dstate = dstate;
    p.wait_ns = debug_wait_ns(), p.skip = debug_take_skip_publish();
    BLOCK_CUDA(launch_recurrence_backward(p, device_sms(), static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

size_t sdtw_gated_workspace_bytes(const sdtw_gated* a, int backward)
{
    if (check_gated(a) != SDTW_OK) return 0;
    GatedParams p{};
    p.a = *a;
    return gated_workspace(p, backward != 0, device_sms());
}

sdtw_status sdtw_gated_forward(const sdtw_gated* a, void* h, void* ws, size_t ws_bytes, void* stream)
{
    if (sdtw_status s = check_gated(a)) return s;
    if (!h) return SDTW_ERR_ARG;
    if (sdtw_status s = check_ws(ws, ws_bytes, sdtw_gated_workspace_bytes(a, 0))) return s;
    GatedParams p{};
    p.a = *a, p.h = h, p.wait_ns = debug_wait_ns();
    if (!gated_is_few(p)) p.skip = debug_take_skip_publish();
    BLOCK_CUDA(launch_gated_forward(p, ws, device_sms(), static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

sdtw_status sdtw_gated_backward(const sdtw_gated* a, const void* dh, void* dx, void* dgate_weight, void* dup_weight,
                                void* dgate_bias, void* dup_bias, void* ws, size_t ws_bytes, void* stream)
{
    if (sdtw_status s = check_gated(a)) return s;
    if (!dh) return SDTW_ERR_ARG;
    if (!dx && !dgate_weight && !dup_weight && !dgate_bias && !dup_bias) return SDTW_OK;
    if (sdtw_status s = check_ws(ws, ws_bytes, sdtw_gated_workspace_bytes(a, 1))) return s;
    GatedParams p{};
    p.a = *a, p.dh = dh, p.dx = dx, p.dgate_weight = dgate_weight, p.dup_weight = dup_weight;
    p.dgate_bias = dgate_bias, p.dup_bias = dup_bias;
    p.wait_ns = debug_wait_ns(), p.skip = debug_take_skip_publish();
    BLOCK_CUDA(launch_gated_backward(p, ws, device_sms(), static_cast<cudaStream_t>(stream)));
    return SDTW_OK;
}

}  // extern "C"
