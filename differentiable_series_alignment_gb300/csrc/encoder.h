// encoder.h -- host-side declarations of the sequence-encoder operators' launchers
// (layer norm, rotary positions, attention) and the element types they share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/sdtw.h"
#include "attn_range.h"

namespace sdtw {

// Elements of 32 or 16 bits; all arithmetic is in fp32, each result rounded once.
template <typename T> __device__ __forceinline__ float to_f32(T v) { return static_cast<float>(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v) { return static_cast<T>(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// v rounded into *out and, where rest is wanted, what that rounding left, rounded too.
template <typename T> __device__ __forceinline__ void store_rounded(T* out, T* rest, float v) {
    const T r = from_f32<T>(v);
    *out = r;
    if (rest) *rest = from_f32<T>(v - to_f32(r));
}

// VEC consecutive elements, loaded and stored as one access of VEC * sizeof(T) bytes.
template <typename T, int VEC> struct alignas(VEC * sizeof(T)) Pack {
    T e[VEC];
};

inline int dtype_size(int dtype) { return dtype == SDTW_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Allows a kernel its dynamic shared memory, once per device.
template <auto Kernel> cudaError_t allow_smem(size_t bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launches a kernel that reads what the one before it in the stream writes, and begins with
// after_previous(): its CTAs come while the other's last ones run, which hides what a launch takes
// (2 us of the 16 of a small call that joins the shares of a key axis).
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = grid, c.blockDim = dim3(threads), c.stream = s, c.attrs = &at, c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}
// Returns when the kernels before this one are complete and their results visible.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the kernel behind this one come as soon as all CTAs have said so; it waits for them in after_previous().
__device__ __forceinline__ void let_next_come() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct NormParams {
    const void *x, *weight, *bias, *dy;
    void *y, *dx, *dweight, *dbias;
    float *mean, *rstd;
    float* partial;   // backward: [2][ctas][C] sums of the weight's and the bias's gradient
    long long rows;
    int C, dtype, wdtype;
    float eps;
};
int norm_partial_ctas(long long rows, int sms);   // CTAs of the backward = partial rows, at most
cudaError_t launch_norm_forward(const NormParams& p, cudaStream_t s);
cudaError_t launch_norm_backward(const NormParams& p, int ctas, cudaStream_t s);

struct RotaryParams {
    const void* in[2];        // q, k (k may be null)
    void* out[2];             // contiguous (B, N, H, D)
    long long stride[2][3];   // batch, position, head strides of the inputs, in elements
    int H[2];
    const float* table;       // (length, R / 2, 2): cos, sin
    const int* positions;     // (B, N), (N) or null: 0 .. N-1
    long long pos_stride_b;   // N or 0
    int B, N, D, R, length, dtype, interleaved, inverse;
};
cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t s);

// Attention over "packed rows": the G = Hq / Hkv query heads that share a key head are
// rows of one problem, row r = n G + (head in group), so that a tile of keys is read
// once for all of them, and a single new token of G heads is a problem of G rows.
struct AttnParams {
    sdtw_attention a;
    int G;                    // Hq / Hkv
    int rows;                 // N * G
    void* out;                // (B, N, Hq, D)
    void* out_rest;           // like out, or null: what the rounding of out left
    float* lse;               // (B, Hq, N) or null (forward)
    // keys split over CTAs: each writes its normalised rows and their lse here
    int splits;
    float* part_o;            // [splits][B][Hkv][rows][D]
    float* part_lse;          // [splits][B][Hkv][rows]
    // backward
    const void* dout;
    void *dq, *dk, *dv;
    const float* lse_in;      // (B, Hq, N)
    // [B][Hkv][rows_pad]: lse in base-2 units less grad_shift, +inf where a row sees nothing. The backward
    // kernels so hold 2^grad_shift P and dS and scale their results back: probabilities near the
    // bottom of the format's range reach the products instead of being flushed to 0.
    float* row_lse;
    int grad_shift;
    bool few;        // at most 12 rows, read in packs: the kernel for new samples over a cache
    // fp16 on the tensor cores: the largest squared norm of do in every 32 packed rows
    // ([B][Hkv][rows_pad / 32]) and of v in every 32 keys ([B][Hkv][ceil(M / 32)])
    float *norm_rows, *norm_keys;
    float* row_delta;         // [B][Hkv][rows_pad]: sum_d do * o
    int rows_pad;             // rows rounded up to 128
    bool packed;              // rows of four-element packs: D, strides and addresses allow them
    // tensor-core kernels
    bool tc;                  // taken by them (attn_tc_fits)
    int tile_rows;            // packed rows of a tile: whole positions, up to 128
    int row_tiles;            // forward: row tiles of a CTA, 1 or 2
    unsigned long long wait_ns;
    // test hook. 1: nothing is loaded, so that every wait runs out; 2: one chain of waits alone does, in the forward
    // pass for want of every second key tile, in the backward pass before the last product of a sum
    int skip;
};
bool attn_tc_fits(const sdtw_attention& a);
cudaError_t launch_attn_forward_tc(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_backward_tc(const AttnParams& p, cudaStream_t s);
cudaError_t attn_backward_take_status(int* out, cudaStream_t s);
cudaError_t attn_forward_take_status(int* out, cudaStream_t s);
cudaError_t launch_attn_forward_simt(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_combine(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_rowinfo(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_backward_simt(const AttnParams& p, cudaStream_t s);

}  // namespace sdtw
