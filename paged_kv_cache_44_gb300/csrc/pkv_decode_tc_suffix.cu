// The tensor-core decode of each sequence's own tokens, behind the ones it
// shares with its group (pkv_decode_tc.cuh).
#include "pkv_decode_tc.cuh"

namespace pkv {

cudaError_t launch_decode_tc_suffix(DecodeParams& p, pkv_dtype q_dt, pkv_dtype c_dt, int num_sms, cudaStream_t st) {
    if (c_dt != PKV_BF16 || q_dt != PKV_BF16) return cudaErrorInvalidValue;
    return p.d == 64 ? launch_bs<64, false, BF16, DecodeMode::kSuffix>(p, num_sms, st)
                     : launch_bs<128, false, BF16, DecodeMode::kSuffix>(p, num_sms, st);
}

}  // namespace pkv
