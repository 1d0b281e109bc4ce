// gated_tc_dx.cu -- gated linear units on the tensor cores: the gradient of x (gated_tc.cuh).
#include "gated_tc.cuh"

namespace sdtw {
namespace gtc {

cudaError_t run_dx(Params& p, int dtype, int NB, int sms, cudaStream_t s) { return run_kind<DX>(p, dtype, NB, sms, s); }

}  // namespace gtc

cudaError_t gated_dx_take_status(int* out, cudaStream_t s) { return gtc::take_status_of_file(out, s); }

}  // namespace sdtw
