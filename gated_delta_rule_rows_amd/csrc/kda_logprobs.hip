// gfx950 kernels of kda_logprobs: log probabilities of given tokens, entropy
// and the top alternatives of logits rows.
//
// With m = max x, z = sum exp(x - m), y = x - m:
//   lp = y[token] - log z,   entropy = log z - (sum exp(y) y) / z
// and the top n by (value, lowest index first).  One workgroup a row: a pass
// for m, one for the sums, one pass for each alternative.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_launch.h"
#include "kda_ops.h"

namespace kda {
namespace {

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, int i) {
    if constexpr (BF16) {
        const uint32_t b = static_cast<const uint16_t*>(row)[i];
        return __builtin_bit_cast(float, b << 16);
    } else {
        return static_cast<const float*>(row)[i];
    }
}

// Keys order as (value, then lowest index): greater is better, -0 equals +0.
__device__ __forceinline__ uint64_t key_of(float x, int i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);
    const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return static_cast<uint64_t>(o) << 32 | ~static_cast<uint32_t>(i);
}

constexpr int kThreads = 1024;

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T x, T* part, F f) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x = f(x, static_cast<T>(__shfl_xor(x, m)));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) x = f(x, part[w]);
    return x;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprob_row_kernel(LogprobArgs a) {
    __shared__ float pf[kThreads / 64];
    __shared__ unsigned long long pk[kThreads / 64];
    const int tid = threadIdx.x;
    const long long r = blockIdx.x;
    const void* row = static_cast<const char*>(a.logits) + r * a.ld * (BF16 ? 2 : 4);
    const float inf = __builtin_inff(), nan = __builtin_nanf("");

    float m = -inf;
    bool bad = false;   // a NaN or +inf: no distribution
    for (int i = tid; i < a.V; i += kThreads) {
        const float x = logit<BF16>(row, i);
        bad |= !(x < inf);
        m = fmaxf(m, x);
    }
    bad = __syncthreads_or(bad);
    m = block_reduce(m, pf, [](float x, float y) { return fmaxf(x, y); });
    const bool empty = m == -inf;
    float z = 0.f, w = 0.f;
    if (!bad && !empty) {
        for (int i = tid; i < a.V; i += kThreads) {
            const float y = logit<BF16>(row, i) - m;
            const float p = expf(y);
            z += p;
            if (p > 0.f) w = fmaf(p, y, w);
        }
    }
    const auto add = [](float x, float y) { return x + y; };
    z = block_reduce(z, pf, add);
    w = block_reduce(w, pf, add);
    const float log_z = logf(z);
    if (tid == 0) {
        if (a.lp) {
            const uint32_t tok = a.tokens[r];
            float lp = nan;
            if (!bad && tok < static_cast<uint32_t>(a.V))
                lp = empty ? -inf : logit<BF16>(row, static_cast<int>(tok)) - m - log_z;
            a.lp[r] = lp;
        }
        if (a.entropy) a.entropy[r] = bad ? nan : empty ? 0.f : log_z - w / z;
    }
    unsigned long long last = ~0ull;
    for (int n = 0; n < a.n_top; ++n) {
        unsigned long long best = 0;
        if (!bad && !empty) {
            for (int i = tid; i < a.V; i += kThreads) {
                const float x = logit<BF16>(row, i);
                const unsigned long long key = key_of(x, i);
                if (x > -inf && key < last && key > best) best = key;
            }
        }
        best = block_reduce(best, pk, [](unsigned long long x, unsigned long long y) { return x > y ? x : y; });
        if (tid == 0) {
            const uint32_t id = ~static_cast<uint32_t>(best);
            const bool none = best == 0;
            a.top_ids[r * a.n_top + n] = none ? kNoToken : id;
            a.top_lp[r * a.n_top + n] =
                bad ? nan : none ? -inf : logit<BF16>(row, static_cast<int>(id)) - m - log_z;
        }
        last = best;
    }
}

}  // namespace

long long logprob_work_bytes(int, int, int) { return 0; }

hipError_t launch_logprobs(const LogprobArgs& a, bool bf16, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.t));
    if (bf16)
        logprob_row_kernel<true><<<grid, dim3(kThreads), 0, stream>>>(a);
    else
        logprob_row_kernel<false><<<grid, dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kda
