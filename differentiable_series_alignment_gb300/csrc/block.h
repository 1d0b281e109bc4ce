// block.h -- host-side declarations of the launchers of the encoder block without attention: group norm, gated
// recurrence and gated linear units.
#pragma once
#include "encoder.h"

namespace sdtw {

struct GroupNormParams {
    const void *x, *weight, *bias, *dy;
    void *y, *dx, *dweight, *dbias;
    const int* lengths;
    float *mean, *rstd;     // (B, G)
    float* partial;         // backward: sums of the weight's and the bias's gradient
    int B, S, G, C, cg;     // cg = C / G
    float eps;
    int activation, dtype, wdtype;
};
size_t group_norm_workspace(const GroupNormParams& p, bool backward, int sms);
cudaError_t launch_group_norm_forward(const GroupNormParams& p, int sms, cudaStream_t s);
cudaError_t launch_group_norm_backward(const GroupNormParams& p, int sms, cudaStream_t s);

struct RecurrenceParams {
    sdtw_recurrence a;
    void* h;
    float *last, *kept;
    const float* kept_in;
    const void* dh;
    const float* dlast;
    void *dx, *dgate;
    float* dstate;
    unsigned long long wait_ns;   // of a wait within a cluster
    int skip;                     // test hook, of a cluster's first CTA. 1: it sends nothing; 2: one of its warps alone gives up a wait
};
cudaError_t launch_recurrence_forward(const RecurrenceParams& p, int sms, cudaStream_t s);
cudaError_t launch_recurrence_backward(const RecurrenceParams& p, int sms, cudaStream_t s);
cudaError_t recurrence_take_status(int* out, cudaStream_t s);

struct GatedParams {
    sdtw_gated a;
    void* h;
    const void* dh;
    void *dx, *dgate_weight, *dup_weight, *dgate_bias, *dup_bias;
    unsigned long long wait_ns;   // of a wait on the tensor cores
    int skip;                     // test hook: the next kernel on the tensor cores loads nothing
};
size_t gated_workspace(const GatedParams& p, bool backward, int sms);
bool gated_is_few(const GatedParams& p);   // a forward pass that stays off the tensor cores
cudaError_t launch_gated_forward(const GatedParams& p, void* ws, int sms, cudaStream_t s);
cudaError_t launch_gated_backward(const GatedParams& p, void* ws, int sms, cudaStream_t s);
cudaError_t gated_fwd_take_status(int* out, cudaStream_t s);
cudaError_t gated_grad_take_status(int* out, cudaStream_t s);
cudaError_t gated_dx_take_status(int* out, cudaStream_t s);
cudaError_t gated_dw_take_status(int* out, cudaStream_t s);

}  // namespace sdtw
