// Drives kda_ops_abi.cpp's validation on the host: every entry point accepted
// and refused, with the launchers replaced by stubs that record the call, and
// two threads refusing at once (each keeps its own message).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <string>
#include <thread>
#include <vector>

#include "kda.h"
#include "kda_check.h"
#include "kda_ops.h"

static int launches = 0;

namespace kda {
long long prompt_work_bytes(int R, int B, int H) { return 64ll * (R + B) * H; }
long long linear_work_bytes(int R, int, int) { return R > 512 ? 4096 : 0; }
long long logprob_work_bytes(int t, int, int n) { return t < 4 ? 16ll * (n + 1) : 0; }
hipError_t launch_prompt(const PromptArgs& a, bool, hipStream_t) { ++launches; return a.H == 7 ? hipErrorInvalidValue : hipSuccess; }
hipError_t launch_linear_prompt(const PromptArgs&, bool, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_linear_step(const StepArgs&, bool, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_logprobs(const LogprobArgs&, bool, hipStream_t) { ++launches; return hipSuccess; }
}  // namespace kda

extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

static int bad = 0;

static void expect(int got, int want, const char* what) {
    if (got != want) {
        std::printf("FAIL %s: %d, want %d (%s)\n", what, got, want, kda::g_err);
        ++bad;
    }
}

static void* at(uintptr_t i) { return reinterpret_cast<void*>(uintptr_t{0x10000000} + i * (uintptr_t{1} << 40)); }

int main() {
    auto* s = static_cast<float* const*>(at(0));
    auto* off = static_cast<const int32_t*>(at(1));
    auto *q = at(2), *k = at(3), *v = at(4), *beta = at(6), *work = at(8);
    auto *g = static_cast<float*>(at(5)), *o = static_cast<float*>(at(7));
    const long long big = 1ll << 39;
    expect(kda_prompt(s, off, q, k, v, g, beta, o, 100, 3, 4, KDA_IN_BF16, work, big, nullptr), KDA_OK, "prompt");
    expect(kda_prompt(s, off, q, k, v, g, beta, nullptr, 100, 3, 4, KDA_IN_F32, work, big, nullptr), KDA_OK, "prompt state");
    expect(kda_prompt(s, off, q, k, v, g, beta, o, 100, 3, 7, KDA_IN_F32, work, big, nullptr), KDA_ERR_HIP, "failed launch");
    expect(kda_prompt(s, off, q, k, v, g, beta, o, 100, 3, 4, KDA_IN_F32, work, 100, nullptr), KDA_ERR_RANGE, "small work");
    expect(kda_prompt(s, off, q, k, v, g, beta, static_cast<float*>(q), 100, 3, 4, KDA_IN_F32, work, big, nullptr), KDA_ERR_ALIAS, "alias");
    expect(kda_prompt(s, off, q, k, v, g, nullptr, o, 100, 3, 4, KDA_IN_F32, work, big, nullptr), KDA_ERR_ARG, "null");
    expect(kda_prompt(s, off, q, k, v, g, beta, o, KDA_PROMPT_ROWS_MAX, KDA_PROMPT_SEQS_MAX, 65535, KDA_IN_F32, work, big, nullptr), KDA_ERR_RANGE, "too many");
    expect(kda_linear_prompt(s, off, q, k, v, g, o, 100, 3, 2, 4, KDA_IN_BF16, nullptr, 0, nullptr), KDA_OK, "linear");
    expect(kda_linear_prompt(s, off, q, k, v, g, o, 1000, 3, 2, 4, KDA_IN_BF16, nullptr, 0, nullptr), KDA_ERR_RANGE, "linear work");
    expect(kda_linear_prompt(s, off, q, k, v, g, o, 1000, 3, 3, 4, KDA_IN_BF16, work, big, nullptr), KDA_ERR_RANGE, "linear heads");
    expect(kda_linear_prompt(s, off, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 3, 2, 4, KDA_IN_BF16, nullptr, 0, nullptr), KDA_OK, "linear no rows");
    expect(kda_linear_step(s, q, k, v, g, o, 2, 3, 2, 4, KDA_IN_F32, nullptr), KDA_OK, "step");
    expect(kda_linear_step(s, q, k, v, g, o, 2, 0, 2, 4, KDA_IN_F32, nullptr), KDA_ERR_RANGE, "step B");
    expect(kda_linear_step(s, q, k, v, g, o, 1 << 20, 1 << 20, 1, 1, KDA_IN_F32, nullptr), KDA_ERR_RANGE, "step size");
    auto* tok = static_cast<uint32_t*>(at(9));
    auto *lp = static_cast<float*>(at(10)), *ent = static_cast<float*>(at(11)), *top = static_cast<float*>(at(12));
    auto* ids = static_cast<uint32_t*>(at(13));
    expect(kda_logprobs(q, 3, 100, 100, KDA_IN_F32, tok, 5, lp, ent, ids, top, work, big, nullptr), KDA_OK, "logprobs");
    expect(kda_logprobs(q, 9, 100, 200, KDA_IN_BF16, nullptr, 0, nullptr, ent, nullptr, nullptr, nullptr, 0, nullptr), KDA_OK, "entropy");
    expect(kda_logprobs(q, 3, 100, 100, KDA_IN_F32, tok, 5, lp, ent, ids, top, work, 95, nullptr), KDA_ERR_RANGE, "logprobs work");
    expect(kda_logprobs(q, 3, 100, 100, KDA_IN_F32, nullptr, 0, nullptr, nullptr, nullptr, nullptr, work, big, nullptr), KDA_ERR_ARG, "nothing");
    expect(kda_logprobs(q, 3, 100, 100, KDA_IN_F32, tok, 5, lp, lp, ids, top, work, big, nullptr), KDA_ERR_ALIAS, "logprobs alias");
    expect(launches, 7, "launches");   // the accepted calls with rows
    if (kda_prompt_work_bytes(1, 0, 1) != -1 || kda_linear_prompt_work_bytes(-1, 1, 1) != -1 || kda_logprobs_work_bytes(0, 1, 1) != -1 ||
        kda_prompt_work_bytes(10, 2, 3) != 64 * 12 * 3) {
        std::printf("FAIL work bytes\n");
        ++bad;
    }
    std::vector<std::thread> threads;
    bool mine[2] = {false, false};
    for (int i = 0; i < 2; ++i)
        threads.emplace_back([&, i] {
            bool ok = true;
            for (int n = 0; n < 2000; ++n) {
                if (i == 0) kda_linear_step(s, q, k, v, g, o, 0, 1, 1, 1, KDA_IN_F32, nullptr);
                else kda_logprobs(q, 0, 1, 1, KDA_IN_F32, tok, 0, lp, nullptr, nullptr, nullptr, nullptr, 0, nullptr);
                ok = ok && std::strstr(kda::g_err, i == 0 ? "kda_linear_step: L=0" : "kda_logprobs: t=0");
            }
            mine[i] = ok;
        });
    for (auto& t : threads) t.join();
    if (!mine[0] || !mine[1]) {
        std::printf("FAIL messages of two threads\n");
        ++bad;
    }
    if (!bad) std::printf("OK\n");
    return bad != 0;
}
