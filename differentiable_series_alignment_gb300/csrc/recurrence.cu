// recurrence.cu -- a gated linear recurrence along a series, forward and backward.
//
//   a_t = sigmoid(gate_t), h_t = a_t h_{t-1} + (1 - a_t) x_t (tied) or a_t h_{t-1} + x_t
//   e_t = dh_t + a_{t+1} e_{t+1}, dx_t = (1 - a_t) e_t or e_t, dgate_t = e_t (h_{t-1} - x_t or h_{t-1}) a_t (1 - a_t)
//
// A thread a channel of a batch element, from the first position to the last. The backward pass computes the states again
// from those that the forward pass kept.
#include "activation.cuh"
#include "block.h"

namespace sdtw {
namespace {

constexpr int kStep = SDTW_RECURRENCE_STEP;

struct Element {   // a batch element's positions, in the order of the recurrence
    int len, reverse;
    __device__ __forceinline__ Element(const sdtw_recurrence& a, int b)
        : len(a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N), reverse(a.reverse) {}
    __device__ __forceinline__ int row(int t) const { return reverse && t < len ? len - 1 - t : t; }
};

template <typename T> __global__ void recurrence_fwd_kernel(const RecurrenceParams p)
{
    const sdtw_recurrence& a = p.a;
    const int per = (a.C + 63) / 64, c = blockIdx.x % per * 64 + threadIdx.x, b = blockIdx.x / per;
    if (c >= a.C) return;
    const Element el(a, b);
    const long long bc = (long long)b * a.C + c;
    const T* x = static_cast<const T*>(a.x) + b * a.x_stride[0] + c;
    const T* g = static_cast<const T*>(a.gate) + b * a.gate_stride[0] + c;
    T* out = static_cast<T*>(p.h) + (long long)b * a.N * a.C + c;
    const int steps = (a.N + kStep - 1) / kStep;
    float h = a.state ? a.state[bc] : 0.f;
    for (int t = 0; t < a.N; ++t) {
        if (p.kept && t % kStep == 0) p.kept[((long long)b * steps + t / kStep) * a.C + c] = h;
        const long long r = el.row(t);
        if (t < el.len) {
            const float z = to_f32(g[r * a.gate_stride[1]]), v = to_f32(x[r * a.x_stride[1]]);
            h = fmaf(sigmoid<true>(z), h, a.tied ? sigmoid<true>(-z) * v : v);
        }
        out[r * a.C] = from_f32<T>(t < el.len ? h : 0.f);
    }
    if (p.last) p.last[bc] = h;
}

template <typename T> __global__ void recurrence_bwd_kernel(const RecurrenceParams p)
{
    const sdtw_recurrence& a = p.a;
    const int per = (a.C + 63) / 64, c = blockIdx.x % per * 64 + threadIdx.x, b = blockIdx.x / per;
    if (c >= a.C) return;
    const Element el(a, b);
    const long long bc = (long long)b * a.C + c, base = (long long)b * a.N * a.C + c;
    const T* x = static_cast<const T*>(a.x) + b * a.x_stride[0] + c;
    const T* g = static_cast<const T*>(a.gate) + b * a.gate_stride[0] + c;
    const int steps = (a.N + kStep - 1) / kStep;
    float e = p.dlast ? p.dlast[bc] : 0.f;
    for (int t = a.N - 1; t >= el.len; --t) {
        static_cast<T*>(p.dx)[base + (long long)t * a.C] = from_f32<T>(0.f);
        static_cast<T*>(p.dgate)[base + (long long)t * a.C] = from_f32<T>(0.f);
    }
    for (int k = (el.len + kStep - 1) / kStep - 1; k >= 0; --k) {
        float before[kStep];
        float h = p.kept_in[((long long)b * steps + k) * a.C + c];
        const int n = min(kStep, el.len - k * kStep);
        for (int i = 0; i < n; ++i) {
            const long long r = el.row(k * kStep + i);
            const float z = to_f32(g[r * a.gate_stride[1]]), v = to_f32(x[r * a.x_stride[1]]);
            before[i] = h;
            h = fmaf(sigmoid<true>(z), h, a.tied ? sigmoid<true>(-z) * v : v);
        }
        for (int i = n - 1; i >= 0; --i) {
            const long long r = el.row(k * kStep + i);
            const float z = to_f32(g[r * a.gate_stride[1]]), v = to_f32(x[r * a.x_stride[1]]);
            const float f = sigmoid<true>(z), o = sigmoid<true>(-z);
            if (p.dh) e += to_f32(static_cast<const T*>(p.dh)[base + r * a.C]);
            static_cast<T*>(p.dx)[base + r * a.C] = from_f32<T>(a.tied ? o * e : e);
            static_cast<T*>(p.dgate)[base + r * a.C] = from_f32<T>(e * (a.tied ? before[i] - v : before[i]) * (f * o));
            e *= f;
        }
    }
    if (p.dstate) p.dstate[bc] = e;
}

template <typename T> cudaError_t run(const RecurrenceParams& p, bool backward, cudaStream_t s)
{
    const unsigned grid = (unsigned)((p.a.C + 63) / 64 * p.a.B);
    if (backward) recurrence_bwd_kernel<T><<<grid, 64, 0, s>>>(p);
    else recurrence_fwd_kernel<T><<<grid, 64, 0, s>>>(p);
    return cudaGetLastError();
}
cudaError_t any(const RecurrenceParams& p, bool backward, cudaStream_t s)
{
    if (p.a.dtype == SDTW_F32) return run<float>(p, backward, s);
    if (p.a.dtype == SDTW_BF16) return run<__nv_bfloat16>(p, backward, s);
    return run<__half>(p, backward, s);
}

}  // namespace

cudaError_t launch_recurrence_forward(const RecurrenceParams& p, int, cudaStream_t s) { return any(p, false, s); }
cudaError_t launch_recurrence_backward(const RecurrenceParams& p, int, cudaStream_t s) { return any(p, true, s); }

}  // namespace sdtw
