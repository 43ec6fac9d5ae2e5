// The tensor-core decode under a sliding window with sinks (pkv_decode_tc.cuh).
#include "pkv_decode_tc.cuh"

namespace pkv {

cudaError_t launch_decode_tc_window(DecodeParams& p, pkv_dtype q_dt, pkv_dtype c_dt, int num_sms, cudaStream_t st) {
    return launch_tc<DecodeMode::kWindow>(p, q_dt, c_dt, num_sms, st);
}

}  // namespace pkv
