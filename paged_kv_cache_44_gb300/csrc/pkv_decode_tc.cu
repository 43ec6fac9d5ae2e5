// The tensor-core decode through block tables (pkv_decode_tc.cuh), and the
// choice of its modes; each mode's kernels are compiled on their own.
#include "pkv_decode_tc.cuh"

namespace pkv {

bool decode_tc_supports(pkv_dtype q_dt, pkv_dtype c_dt, int d, int bs, int NB) {
    if (!(d == 64 || d == 128) || !(bs == 16 || bs == 32)) return false;
    if ((long long)NB * bs >= (1LL << 31)) return false;      // TMA row coordinates are 32-bit
    if (c_dt == PKV_BF16) return q_dt == PKV_BF16;
    return c_dt == PKV_FP8_E4M3 && (q_dt == PKV_BF16 || q_dt == PKV_F32);
}

cudaError_t launch_decode_tc(DecodeParams& p, pkv_dtype q_dt, pkv_dtype c_dt, int num_sms, cudaStream_t st,
                             DecodeMode mode) {
    if (p.S == 0) return cudaSuccess;
    switch (mode) {
        case DecodeMode::kBlockTable: return launch_tc<DecodeMode::kBlockTable>(p, q_dt, c_dt, num_sms, st);
        case DecodeMode::kTokenTable: return launch_decode_tc_token(p, q_dt, c_dt, num_sms, st);
        case DecodeMode::kWindow: return launch_decode_tc_window(p, q_dt, c_dt, num_sms, st);
        case DecodeMode::kScored: return launch_decode_tc_scored(p, q_dt, c_dt, num_sms, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pkv
