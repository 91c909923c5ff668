// Internal interface of the log-probability kernel (qg_logprobs.cu) for the C ABI.
#pragma once

#include "qg_internal.h"

namespace qg {

constexpr int kMaxTopK = QG_MAX_TOP_K;

struct LogprobArgs {
    const void* logits;        // [M, ld] of type
    int type;                  // QG_BF16, QG_FP16 or QG_FP32
    int64_t ld;
    const int64_t* tokens;     // [M, ldt], T asked in each row
    int64_t ldt;
    int T;
    float* token_lp;           // [M, T]
    float* entropy;            // [M] or null
    int top_k;
    int64_t* top_ids;          // [M, top_k]
    float* top_lp;             // [M, top_k]
    int M, V;
};

cudaError_t launch_logprobs(const LogprobArgs& a, const LaunchCtl& c, cudaStream_t st);

}  // namespace qg
