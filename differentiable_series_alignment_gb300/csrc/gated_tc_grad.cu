// gated_tc_grad.cu -- gated linear units on the tensor cores: the gradients of the two products (gated_tc.cuh).
#include "gated_tc.cuh"

namespace sdtw {
namespace gtc {

cudaError_t run_grad(Params& p, int dtype, int NB, int sms, cudaStream_t s) { return run_kind<GRAD>(p, dtype, NB, sms, s); }

}  // namespace gtc

cudaError_t gated_grad_take_status(int* out, cudaStream_t s) { return gtc::take_status_of_file(out, s); }

}  // namespace sdtw
