// Internal interface of the draft verification kernel (qg_verify.cu) for the C ABI.
#pragma once

#include "qg_internal.h"

namespace qg {

struct VerifyArgs {
    const void* target;       // [B, G + 1, V] of type
    int64_t t_seq, t_row;     // strides in elements
    const void* draft;        // [B, G, V] of type, or null: the drafts are certain
    int64_t d_seq, d_row;
    int type;
    const int64_t* tokens;    // [B, G]
    int64_t ldt;
    const float* uniform;     // [B, G]; null: greedy
    int64_t ldu;
    const float* noise;       // [B, V]
    int64_t ldn;
    const int32_t* lengths;   // [B] or null (G)
    int32_t* accepted;        // [B]
    int64_t* out;             // [B, G + 1]
    int B, G, V;
    void* ws;
};

size_t verify_workspace_bytes(int B, int G, int V, int sms);

cudaError_t launch_verify(const VerifyArgs& a, const LaunchCtl& c, cudaStream_t st);

}  // namespace qg
