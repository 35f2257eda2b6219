// gfx950 kernels of the prompt and single-token operators: the KDA delta rule
// and linear attention with one decay for each head, over the same
// [H][128][128] f32 states as the verify scan.
//
// One row of one head (i = key channel, j = value channel):
//   KDA     S' = diag(exp(clamp(g, -5, 0))) S,  e = beta (v - S'^T k)
//   linear  S' = exp(min(g, 0)) S,              e = v
//   both    S  = S' + k e^T,  o = S^T q / sqrt(128)
//
// Row kernel: a workgroup owns 32 value columns of one (sequence, head) and
// walks its rows; 8 neighbouring lanes share a column, 16 keys each, and
// reduce with three lane exchanges.  Rows are staged 16 at a time in LDS.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_launch.h"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr float kScale = 0.0883883476483184405501055452631f;   // 1/sqrt(128)
constexpr float kGateLow = -5.0f;

template <bool BF16>
__device__ __forceinline__ float load(const void* p, long long i) {
    if constexpr (BF16) {
        const uint32_t b = static_cast<const uint16_t*>(p)[i];
        return __builtin_bit_cast(float, b << 16);
    } else {
        return static_cast<const float*>(p)[i];
    }
}

// Rows [first, last) of sequence b, held inside [0, R] whatever the table says.
__device__ __forceinline__ void sequence(const PromptArgs& a, int b, int& first, int& last) {
    first = min(max(a.offsets[b], 0), a.R);
    last = min(max(a.offsets[b + 1], first), a.R);
}

constexpr int kTileRows = 16;
constexpr int kRowCols = 32;   // value columns of a workgroup

template <bool LINEAR, bool BF16>
__global__ void __launch_bounds__(256) row_kernel(PromptArgs a) {
    __shared__ float qs[kTileRows][kD], ks[kTileRows][kD], ds[LINEAR ? 1 : kTileRows][kD];
    __shared__ float vs[kTileRows][kRowCols], bs[kTileRows];
    const int tid = threadIdx.x;
    const int slices = kD / kRowCols;
    const int slice = blockIdx.x % slices;
    const int h = blockIdx.x / slices % a.H;
    const int b = blockIdx.x / slices / a.H;
    const int hk = h / (a.H / a.Hk);
    int first, last;
    sequence(a, b, first, last);
    float* s = a.s_ptrs[b];
    if (s == nullptr || first >= last) return;
    s += static_cast<long long>(h) * kD * kD;

    const int ki = tid & 7;              // keys 4*ki + 32*m + 0..3
    const int cl = tid >> 3;             // column within the slice
    const int col = slice * kRowCols + cl;
    float S[16];
#pragma unroll
    for (int m = 0; m < 16; ++m) S[m] = s[(4 * ki + 32 * (m >> 2) + (m & 3)) * kD + col];

    for (int t0 = first; t0 < last; t0 += kTileRows) {
        const int n = min(kTileRows, last - t0);
        __syncthreads();
        for (int x = tid; x < n * kD; x += 256) {
            const int t = x / kD, c = x % kD;
            const long long kr = (static_cast<long long>(t0 + t) * a.Hk + hk) * kD + c;
            qs[t][c] = load<BF16>(a.q, kr);
            ks[t][c] = load<BF16>(a.k, kr);
            if constexpr (!LINEAR) {
                const long long r = (static_cast<long long>(t0 + t) * a.H + h) * kD + c;
                ds[t][c] = expf(fminf(fmaxf(load<BF16>(a.g, r), kGateLow), 0.f));
            }
        }
        for (int x = tid; x < n * kRowCols; x += 256) {
            const int t = x / kRowCols, c = x % kRowCols;
            vs[t][c] = load<BF16>(a.v, (static_cast<long long>(t0 + t) * a.H + h) * kD +
                                           slice * kRowCols + c);
        }
        if (tid < n) {
            const long long r = static_cast<long long>(t0 + tid) * a.H + h;
            if constexpr (LINEAR)
                bs[tid] = expf(fminf(static_cast<const float*>(a.g)[r], 0.f));
            else
                bs[tid] = load<BF16>(a.beta, r);
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            float e = vs[t][cl];
            if constexpr (LINEAR) {
                const float d = bs[t];
#pragma unroll
                for (int m = 0; m < 16; ++m) S[m] *= d;
            } else {
                float u = 0.f;
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                    const int i = 4 * ki + 32 * (m >> 2) + (m & 3);
                    S[m] *= ds[t][i];
                    u = fmaf(ks[t][i], S[m], u);
                }
                u += __shfl_xor(u, 1);
                u += __shfl_xor(u, 2);
                u += __shfl_xor(u, 4);
                e = bs[t] * (e - u);
            }
            float w = 0.f;
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                const int i = 4 * ki + 32 * (m >> 2) + (m & 3);
                S[m] = fmaf(ks[t][i], e, S[m]);
                w = fmaf(qs[t][i], S[m], w);
            }
            w += __shfl_xor(w, 1);
            w += __shfl_xor(w, 2);
            w += __shfl_xor(w, 4);
            if (a.o != nullptr && ki == 0)
                a.o[(static_cast<long long>(t0 + t) * a.H + h) * kD + col] = w * kScale;
        }
    }
#pragma unroll
    for (int m = 0; m < 16; ++m) s[(4 * ki + 32 * (m >> 2) + (m & 3)) * kD + col] = S[m];
}

template <bool LINEAR>
hipError_t launch_rows(const PromptArgs& a, bool bf16, hipStream_t stream) {
    const long long blocks = static_cast<long long>(a.B) * a.H * (kD / kRowCols);
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (bf16)
        row_kernel<LINEAR, true><<<grid, dim3(256), 0, stream>>>(a);
    else
        row_kernel<LINEAR, false><<<grid, dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

// ------------------------------------------------------------------ single token
//
// A workgroup owns one (layer, session, head): the head's 64 KiB state is read
// once and written once, 16 bytes a lane, all 16 loads of a lane in flight
// before the first use.  HBM-bound.
template <bool BF16>
__global__ void __launch_bounds__(256) linear_step_kernel(StepArgs a) {
    __shared__ float qs[kD], ks[kD];
    __shared__ float4 part[4][32];
    const int tid = threadIdx.x;
    const int h = blockIdx.x % a.H;
    const long long n = blockIdx.x / a.H;
    const int hk = h / (a.H / a.Hk);
    float* s = a.s_ptrs[n];
    if (s == nullptr) return;
    s += static_cast<long long>(h) * kD * kD;
    const int c4 = tid & 31;
    const int r0 = tid >> 5;
    float4* s4 = reinterpret_cast<float4*>(s);
    float4 S[16];
#pragma unroll
    for (int m = 0; m < 16; ++m) S[m] = s4[(r0 + 8 * m) * 32 + c4];
    const long long kr = (n * a.Hk + hk) * kD;
    if (tid < kD)
        qs[tid] = load<BF16>(a.q, kr + tid);
    else
        ks[tid - kD] = load<BF16>(a.k, kr + tid - kD);
    const long long r = n * a.H + h;
    const float d = expf(fminf(a.g[r], 0.f));
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = load<BF16>(a.v, r * kD + 4 * c4 + c);
    __syncthreads();
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < 16; ++m) {
        const float kk = ks[r0 + 8 * m], qq = qs[r0 + 8 * m];
        S[m].x = fmaf(kk, v[0], S[m].x * d);
        S[m].y = fmaf(kk, v[1], S[m].y * d);
        S[m].z = fmaf(kk, v[2], S[m].z * d);
        S[m].w = fmaf(kk, v[3], S[m].w * d);
        w.x = fmaf(qq, S[m].x, w.x);
        w.y = fmaf(qq, S[m].y, w.y);
        w.z = fmaf(qq, S[m].z, w.z);
        w.w = fmaf(qq, S[m].w, w.w);
        s4[(r0 + 8 * m) * 32 + c4] = S[m];
    }
    if (a.o == nullptr) return;
    w.x += __shfl_xor(w.x, 32);
    w.y += __shfl_xor(w.y, 32);
    w.z += __shfl_xor(w.z, 32);
    w.w += __shfl_xor(w.w, 32);
    if ((tid & 63) < 32) part[tid >> 6][c4] = w;
    __syncthreads();
    if (tid < 32) {
        float4 x = part[0][tid];
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            x.x += part[i][tid].x;
            x.y += part[i][tid].y;
            x.z += part[i][tid].z;
            x.w += part[i][tid].w;
        }
        x.x *= kScale;
        x.y *= kScale;
        x.z *= kScale;
        x.w *= kScale;
        reinterpret_cast<float4*>(a.o + r * kD)[tid] = x;
    }
}

}  // namespace

long long prompt_work_bytes(int, int, int) { return 0; }
long long linear_work_bytes(int, int, int) { return 0; }

hipError_t launch_prompt(const PromptArgs& a, bool bf16, hipStream_t stream) {
    return launch_rows<false>(a, bf16, stream);
}

hipError_t launch_linear_prompt(const PromptArgs& a, bool bf16, hipStream_t stream) {
    return launch_rows<true>(a, bf16, stream);
}

hipError_t launch_linear_step(const StepArgs& a, bool bf16, hipStream_t stream) {
    const long long blocks = a.n * a.H;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (bf16)
        linear_step_kernel<true><<<grid, dim3(256), 0, stream>>>(a);
    else
        linear_step_kernel<false><<<grid, dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kda
