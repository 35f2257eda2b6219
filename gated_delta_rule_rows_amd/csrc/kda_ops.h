// Internal interface between kda_ops_abi.cpp and the kernels of the prompt,
// single-token and log-probability operators (kda_prompt.hip,
// kda_logprobs.hip).  Not installed; callers use include/kda.h.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace kda {

// Rows of B sequences packed one after another: sequence b's rows are
// offsets[b] .. offsets[b+1]-1 of [R][heads][128], its state s_ptrs[b]
// ([H][128][128] f32, updated in place; a null entry leaves the sequence out).
struct PromptArgs {
    float* const* s_ptrs;
    const int32_t* offsets;   // device, B + 1 entries
    const void* q;            // [R][Hk][128]
    const void* k;            // [R][Hk][128]
    const void* v;            // [R][H][128]
    const void* g;            // KDA: [R][H][128] in the row dtype; linear: [R][H] f32
    const void* beta;         // KDA: [R][H] in the row dtype; linear: null
    float* o;                 // [R][H][128] or null
    void* work;
    int R;
    int B;
    int Hk;                   // key heads; value head h reads key head h / (H / Hk)
    int H;
};

long long prompt_work_bytes(int R, int B, int H);
long long linear_work_bytes(int R, int B, int H);
hipError_t launch_prompt(const PromptArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_linear_prompt(const PromptArgs& a, bool bf16, hipStream_t stream);

// One token of each of n = L * B (layer, session) states.
struct StepArgs {
    float* const* s_ptrs;     // n entries; a null entry leaves the session out
    const void* q;            // [n][Hk][128]
    const void* k;
    const void* v;            // [n][H][128]
    const float* g;           // [n][H]
    float* o;                 // [n][H][128] or null
    long long n;
    int Hk;
    int H;
};

hipError_t launch_linear_step(const StepArgs& a, bool bf16, hipStream_t stream);

struct LogprobArgs {
    const void* logits;       // row r at element r * ld
    long long ld;
    int t;
    int V;
    int n_top;                // 0..KDA_TOP_MAX
    const uint32_t* tokens;   // t, or null
    float* lp;                // t, or null
    float* entropy;           // t, or null
    uint32_t* top_ids;        // [t][n_top], or null
    float* top_lp;            // [t][n_top], or null
    void* work;
};

long long logprob_work_bytes(int t, int V, int n_top);
hipError_t launch_logprobs(const LogprobArgs& a, bool bf16, hipStream_t stream);

}  // namespace kda
