// gated_tc_fwd.cu -- gated linear units on the tensor cores: the forward pass (gated_tc.cuh).
#include "gated_tc.cuh"

namespace sdtw {
namespace gtc {

cudaError_t run_fwd(Params& p, int dtype, int NB, int sms, cudaStream_t s) { return run_kind<FWD>(p, dtype, NB, sms, s); }

}  // namespace gtc

cudaError_t gated_fwd_take_status(int* out, cudaStream_t s) { return gtc::take_status_of_file(out, s); }

}  // namespace sdtw
