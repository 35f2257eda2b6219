// C ABI of the prompt, single-token and log-probability operators: host-side
// argument validation, then one enqueue, as in kda_abi.cpp.

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "kda.h"
#include "kda_check.h"
#include "kda_launch.h"
#include "kda_ops.h"

using namespace kda;

namespace {

constexpr unsigned long long kRow = kD;         // elements of a row of one head
constexpr int kLogprobRows = (1 << 26) - 1;     // a wave each, 2^32 threads

int check_heads(const char* fn, int Hk, int H) {
    if (H < 1 || H > 65535) return refuse(KDA_ERR_RANGE, "%s: H=%d outside 1..65535", fn, H);
    if (Hk < 1 || H % Hk != 0)
        return refuse(KDA_ERR_RANGE, "%s: Hk=%d must be >= 1 and divide H=%d", fn, Hk, H);
    return KDA_OK;
}

// The products keep every launch below the 2^32 threads of a grid.
int check_packed(const char* fn, int R, int B, int H) {
    if (R < 0 || R > KDA_PROMPT_ROWS_MAX)
        return refuse(KDA_ERR_RANGE, "%s: R=%d outside 0..%d", fn, R, KDA_PROMPT_ROWS_MAX);
    if (B < 1 || B > KDA_PROMPT_SEQS_MAX)
        return refuse(KDA_ERR_RANGE, "%s: B=%d outside 1..%d", fn, B, KDA_PROMPT_SEQS_MAX);
    if (static_cast<long long>(R) * H > 1ll << 34)
        return refuse(KDA_ERR_RANGE, "%s: R*H=%lld too large", fn, static_cast<long long>(R) * H);
    if (static_cast<long long>(B) * H > 1ll << 20)
        return refuse(KDA_ERR_RANGE, "%s: B*H=%lld too large", fn, static_cast<long long>(B) * H);
    return KDA_OK;
}

int check_work(const char* fn, long long have, long long need) {
    if (have < need)
        return refuse(KDA_ERR_RANGE, "%s: work_bytes=%lld, need %lld", fn, have, need);
    return KDA_OK;
}

// kda_prompt (linear = false) and kda_linear_prompt.
int prompt(const char* fn, bool linear, const PromptArgs& a, int in_dtype, long long work_bytes,
           void* stream) {
    int rc;
    if ((rc = check_dtype(fn, in_dtype)) || (rc = check_heads(fn, a.Hk, a.H)) ||
        (rc = check_packed(fn, a.R, a.B, a.H)))
        return rc;
    const long long need = linear ? linear_work_bytes(a.R, a.B, a.H) : prompt_work_bytes(a.R, a.B, a.H);
    if ((rc = check_work(fn, work_bytes, need))) return rc;
    const unsigned es = in_dtype == KDA_IN_BF16 ? 2 : 4;
    const bool none = a.R == 0;   // empty tensors have no address
    const unsigned long long kr = static_cast<unsigned long long>(a.R) * a.Hk;
    const unsigned long long vr = static_cast<unsigned long long>(a.R) * a.H;
    const Span in[] = {
        {"s_ptrs", a.s_ptrs, a.B * 8ull, 8, false},
        {"offsets", a.offsets, (a.B + 1) * 4ull, 4, false},
        {"q", a.q, kr * kRow * es, 16, none},
        {"k", a.k, kr * kRow * es, 16, none},
        {"v", a.v, vr * kRow * es, 16, none},
        {"g", a.g, linear ? vr * 4 : vr * kRow * es, linear ? 4u : 16u, none},
        {"beta", a.beta, linear ? 0 : vr * es, es, linear || none},
    };
    const Span out[] = {
        {"o", a.o, vr * kRow * 4, 16, true},
        {"work", a.work, static_cast<unsigned long long>(need), 16, need == 0},
    };
    if ((rc = check_spans(fn, in, 7)) || (rc = check_spans(fn, out, 2)) ||
        (rc = check_alias(fn, out, 2, in, 7)))
        return rc;
    if (none) return launched(fn, hipSuccess);
    const auto st = static_cast<hipStream_t>(stream);
    return launched(fn, linear ? launch_linear_prompt(a, in_dtype == KDA_IN_BF16, st)
                               : launch_prompt(a, in_dtype == KDA_IN_BF16, st));
}

}  // namespace

extern "C" {

long long kda_prompt_work_bytes(int R, int B, int H) {
    if (check_heads("kda_prompt_work_bytes", 1, H) || check_packed("kda_prompt_work_bytes", R, B, H))
        return -1;
    return prompt_work_bytes(R, B, H);
}

int kda_prompt(float* const* s_ptrs, const int32_t* offsets, const void* q, const void* k,
               const void* v, const void* g, const void* beta, float* o, int R, int B, int H,
               int in_dtype, void* work, long long work_bytes, void* stream) {
    PromptArgs a{};
    a.s_ptrs = s_ptrs; a.offsets = offsets;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.o = o; a.work = work;
    a.R = R; a.B = B; a.Hk = H; a.H = H;
    return prompt("kda_prompt", false, a, in_dtype, work_bytes, stream);
}

long long kda_linear_prompt_work_bytes(int R, int B, int H) {
    if (check_heads("kda_linear_prompt_work_bytes", 1, H) ||
        check_packed("kda_linear_prompt_work_bytes", R, B, H))
        return -1;
    return linear_work_bytes(R, B, H);
}

int kda_linear_prompt(float* const* s_ptrs, const int32_t* offsets, const void* q, const void* k,
                      const void* v, const float* g, float* o, int R, int B, int Hk, int H,
                      int in_dtype, void* work, long long work_bytes, void* stream) {
    PromptArgs a{};
    a.s_ptrs = s_ptrs; a.offsets = offsets;
    a.q = q; a.k = k; a.v = v; a.g = g; a.o = o; a.work = work;
    a.R = R; a.B = B; a.Hk = Hk; a.H = H;
    return prompt("kda_linear_prompt", true, a, in_dtype, work_bytes, stream);
}

int kda_linear_step(float* const* s_ptrs, const void* q, const void* k, const void* v,
                    const float* g, float* o, int L, int B, int Hk, int H, int in_dtype,
                    void* stream) {
    const char* fn = "kda_linear_step";
    int rc;
    if ((rc = check_dtype(fn, in_dtype)) || (rc = check_counts(fn, L, H)) ||
        (rc = check_heads(fn, Hk, H)))
        return rc;
    if (B < 1) return refuse(KDA_ERR_RANGE, "%s: B=%d, need B >= 1", fn, B);
    const unsigned long long n = static_cast<unsigned long long>(L) * B;
    if (n > INT_MAX || n * H >= 1u << 24)   // 2^32 threads
        return refuse(KDA_ERR_RANGE, "%s: L*B*H=%llu too large", fn, n * H);
    const unsigned es = in_dtype == KDA_IN_BF16 ? 2 : 4;
    const Span in[] = {
        {"s_ptrs", s_ptrs, n * 8, 8, false},
        {"q", q, n * Hk * kRow * es, 16, false},
        {"k", k, n * Hk * kRow * es, 16, false},
        {"v", v, n * H * kRow * es, 16, false},
        {"g", g, n * H * 4, 4, false},
    };
    const Span out[] = {{"o", o, n * H * kRow * 4, 16, true}};
    if ((rc = check_spans(fn, in, 5)) || (rc = check_spans(fn, out, 1)) ||
        (rc = check_alias(fn, out, 1, in, 5)))
        return rc;
    StepArgs a{};
    a.s_ptrs = s_ptrs;
    a.q = q; a.k = k; a.v = v; a.g = g; a.o = o;
    a.n = static_cast<long long>(n); a.Hk = Hk; a.H = H;
    return launched(fn, launch_linear_step(a, in_dtype == KDA_IN_BF16,
                                           static_cast<hipStream_t>(stream)));
}

long long kda_logprobs_work_bytes(int t, int V, int n_top) {
    const char* fn = "kda_logprobs_work_bytes";
    if (t < 1 || t > kLogprobRows || V < 1 || V > 1 << 30 || n_top < 0 || n_top > KDA_TOP_MAX) {
        refuse(KDA_ERR_RANGE, "%s: t=%d, V=%d, n_top=%d: need t in 1..2^26-1, V in 1..2^30, n_top in 0..%d", fn,
               t, V, n_top, KDA_TOP_MAX);
        return -1;
    }
    return logprob_work_bytes(t, V, n_top);
}

int kda_logprobs(const void* logits, int t, int V, long long ld, int in_dtype,
                 const uint32_t* tokens, int n_top, float* lp, float* entropy, uint32_t* top_ids,
                 float* top_lp, void* work, long long work_bytes, void* stream) {
    const char* fn = "kda_logprobs";
    int rc;
    if ((rc = check_dtype(fn, in_dtype))) return rc;
    if (t < 1 || t > kLogprobRows)
        return refuse(KDA_ERR_RANGE, "%s: t=%d outside 1..%d", fn, t, kLogprobRows);
    if (V < 1 || V > 1 << 30) return refuse(KDA_ERR_RANGE, "%s: V=%d outside 1..2^30", fn, V);
    if (n_top < 0 || n_top > KDA_TOP_MAX)
        return refuse(KDA_ERR_RANGE, "%s: n_top=%d outside 0..%d", fn, n_top, KDA_TOP_MAX);
    if (t == 1) ld = V;
    if (ld < V) return refuse(KDA_ERR_RANGE, "%s: ld=%lld < V=%d (rows would overlap)", fn, ld, V);
    if (ld > (1ll << 40) / t)
        return refuse(KDA_ERR_RANGE, "%s: ld=%lld too large for t=%d", fn, ld, t);
    if ((tokens == nullptr) != (lp == nullptr))
        return refuse(KDA_ERR_ARG, "%s: tokens and lp go together", fn);
    const bool top = n_top > 0;
    if (!lp && !entropy && !top) return refuse(KDA_ERR_ARG, "%s: nothing is asked for", fn);
    const long long need = logprob_work_bytes(t, V, n_top);
    if ((rc = check_work(fn, work_bytes, need))) return rc;
    const unsigned es = in_dtype == KDA_IN_BF16 ? 2 : 4;
    const unsigned long long rows = static_cast<unsigned long long>(t);
    const Span in[] = {
        {"logits", logits, ((rows - 1) * ld + V) * es, es, false},
        {"tokens", tokens, rows * 4, 4, true},
    };
    const Span out[] = {
        {"lp", lp, rows * 4, 4, true},
        {"entropy", entropy, rows * 4, 4, true},
        {"top_ids", top ? top_ids : nullptr, rows * n_top * 4, 4, !top},
        {"top_lp", top ? top_lp : nullptr, rows * n_top * 4, 4, !top},
        {"work", work, static_cast<unsigned long long>(need), 16, need == 0},
    };
    if ((rc = check_spans(fn, in, 2)) || (rc = check_spans(fn, out, 5)) ||
        (rc = check_alias(fn, out, 5, in, 2)))
        return rc;
    LogprobArgs a{};
    a.logits = logits; a.ld = ld; a.t = t; a.V = V; a.n_top = n_top;
    a.tokens = tokens; a.lp = lp; a.entropy = entropy; a.top_ids = top_ids; a.top_lp = top_lp;
    a.work = work;
    return launched(fn, launch_logprobs(a, in_dtype == KDA_IN_BF16,
                                        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
