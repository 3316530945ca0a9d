// delta_tc.h -- the gated delta rule in chunks on the tensor cores (delta_tc.cu).
#pragma once
#include <cuda_runtime.h>

#include "kdn_internal.h"

namespace kdn {
namespace delta {

// Whether a call may take this form (a backward call then does, whatever its
// length), and whether a forward call does.
bool tc_takes(int B, int H, int dk, int dv, int nseq, kdn_dtype in_dtype);
bool tc_takes_fwd(int B, int H, int T, int dk, int dv, int nseq, kdn_dtype in_dtype);
// Scratch of a forward call.
long long tc_fwd_bytes(int B, int H, int T, int nseq);
kdn_status tc_fwd(const DeltaArgs& a, char* ws, cudaStream_t stream, long long wait_ns);
// The same of a backward call, whose grad_out is bf16 too.
long long tc_bwd_bytes(int B, int H, int T, int nseq);
kdn_status tc_bwd(const DeltaArgs& a, char* ws, cudaStream_t stream, long long wait_ns);

}  // namespace delta
}  // namespace kdn
