// gfx950 kernels of kda_accept_sampled: drafted tokens verified against the
// target's probabilities from given random numbers.
//
// Row r of a session, p = softmax(x / T): the draft d is accepted while
// u q(d) < p(d).  At the first row j that does not accept (or the last row),
// the token is drawn from weights w = max(p - q, 0) (the last row: p): the
// lowest v whose running sum passes u_last times the whole sum.
//
// Three launches.  The first reads the logits once: of every part of a row the
// maximum m and z = sum e^{(x - m) / T}, the exponentials in f32, their sums in
// f64.  The second joins a session's rows, finds j and sums the weights of row j
// by parts; the third finds the part that holds the place, and the token in it.
// The weights are computed in f64: p - q cancels, and a running sum decides
// which of two tokens a random number near their border gives.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_cache.h"
#include "kda_launch.h"
#include "kda_seq.h"

namespace kda {
namespace {

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.44269504088896340736;
constexpr float kSlack = 4.0f;       // the carried maximum may lag by this much
constexpr int kThreads = 256;
constexpr int kMostParts = 64;       // of a row: a lane joins a part

// m, and z relative to it; z is NaN where a value is NaN or +inf.
struct Stat {
    double z;
    float m;
    int pad;
};

// A session's row j, as the second launch leaves it for the third.
struct Found {
    double z;
    double scale;  // 1 / T; 0: no token
    float m;
    int row;       // -1: the session has no rows
    int j;
    int drafted;   // weights max(p - q, 0) unless these are all 0; else p
    int last;      // the session's last row
};

// Sums of a part's weights and probabilities (times z).
struct Mass {
    double w, p;
};

struct Split {
    Stat* stats;     // [R][parts]
    Found* found;    // [B]
    Mass* mass;      // [B][pieces]
    int parts;       // of a row in the first launch
    int pieces;      // of row j in the second
};

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, long long i) {
    if constexpr (BF16)
        return __builtin_bit_cast(float, static_cast<uint32_t>(static_cast<const uint16_t*>(row)[i]) << 16);
    else
        return static_cast<const float*>(row)[i];
}

template <bool BF16>
__device__ __forceinline__ const void* row_at(const SampledArgs& a, long long r) {
    return static_cast<const char*>(a.logits) + r * a.ld * (BF16 ? 2 : 4);
}

// 1 / T of a session; 0 where T is no positive finite number.
__device__ __forceinline__ double scale_of(const SampledArgs& a, int b) {
    if (!a.temp) return 1.0;
    const float t = a.temp[b];
    return t > 0.f && t < kInf ? 1.0 / t : 0.0;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

// s moved to a maximum m >= s.m.
__device__ __forceinline__ double moved(Stat s, float m, double scale) {
    return s.m == -kInf ? s.z : s.z * exp((static_cast<double>(s.m) - m) * scale);
}

// Adds E values of a lane.
template <int E>
__device__ __forceinline__ void take(Stat& s, const float (&x)[E], double scale) {
    float top = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, x[e]);
    const float rate = static_cast<float>(scale), by = static_cast<float>(scale * kLog2e);
    if (__ballot((top - s.m) * rate > kSlack || s.m == -kInf)) {
        const float m = fmaxf(s.m, top);
        s.z = moved(s, m, scale);
        s.m = m;
    }
    const float base = s.m == -kInf ? 0.f : s.m;
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z += __builtin_amdgcn_exp2f((x[e] - base) * by);
    s.z += z;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_stats_kernel(SampledArgs a, Split w) {
    constexpr int E = BF16 ? 8 : 4;
    const int part = blockIdx.x % w.parts;
    const Part f = find_part(a, 1, blockIdx.x / w.parts);
    if (f.b < 0) return;
    const double scale = scale_of(a, f.b);
    if (scale == 0.0) return;
    const long long r = f.first + f.index;
    const void* row = row_at<BF16>(a, r);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // from the first 16-byte boundary on in whole loads
    const int head = min(a.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (BF16 ? 2 : 4));
    const int loads = (a.V - head) / E, tail = a.V - head - loads * E;
    const int each = (loads + w.parts - 1) / w.parts;
    const int begin = min(part * each, loads), end = min(begin + each, loads);
    const uint4* body = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + head * (BF16 ? 2 : 4));
    Stat s{0.0, -kInf, 0};
    for (int i = begin + tid; i < end; i += kThreads) {
        const uint4 u = body[i];
        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (BF16)
                x[e] = __builtin_bit_cast(float, e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
            else
                x[e] = __builtin_bit_cast(float, v[e]);
        }
        take<E>(s, x, scale);
    }
    if (wave == 0) {
        const bool first = part == 0 && lane < head, last = part == w.parts - 1 && lane < tail;
        const float x[2] = {first ? logit<BF16>(row, lane) : -kInf, last ? logit<BF16>(row, a.V - tail + lane) : -kInf};
        take<2>(s, x, scale);
    }
    __shared__ Stat waves[kThreads / 64];
    const float m = wave_max(s.m);
    const double z = wave_sum(moved(s, m, scale));
    if (lane == 0) waves[wave] = Stat{z, m, 0};
    __syncthreads();
    if (tid == 0) {
        float top = waves[0].m;
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) top = fmaxf(top, waves[i].m);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) sum += moved(waves[i], top, scale);
        w.stats[r * w.parts + part] = Stat{sum, top, 0};
    }
}

// m and z of row r, in every lane.
__device__ __forceinline__ Stat row_stat(const Split& w, long long r, double scale) {
    const int lane = threadIdx.x & 63;
    Stat s{0.0, -kInf, 0};
    if (lane < w.parts) s = w.stats[r * w.parts + lane];
    const float m = wave_max(s.m);
    return Stat{wave_sum(moved(s, m, scale)), m, 0};
}

// Weight of token v in row j, times z, and e = p z.
template <bool BF16>
__device__ __forceinline__ double weight(const SampledArgs& a, const Found& f, const void* row, int v, uint32_t draft, double& e) {
    e = exp((static_cast<double>(logit<BF16>(row, v)) - f.m) * f.scale);
    if (!f.drafted) return e;
    if (!a.probs) return static_cast<uint32_t>(v) == draft ? 0.0 : e;
    return fmax(e - f.z * a.probs[f.row * a.probs_ld + v], 0.0);
}

// The tokens of a thread: contiguous, so that running sums go by thread.
__device__ __forceinline__ void range_of(const SampledArgs& a, const Split& w, int piece, int& from, int& to) {
    const int each = (a.V + w.pieces - 1) / w.pieces, begin = min(piece * each, a.V), end = min(begin + each, a.V);
    const int mine = (each + kThreads - 1) / kThreads;
    from = min(begin + static_cast<int>(threadIdx.x) * mine, end);
    to = min(from + mine, end);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_accept_kernel(SampledArgs a, Split w) {
    __shared__ int stop;
    __shared__ Found shared;
    __shared__ Mass waves[kThreads / 64];
    const int piece = blockIdx.x % w.pieces, b = blockIdx.x / w.pieces;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int first, last;
    sequence(a, b, first, last);
    const int n = last - first;
    if (n == 0) {
        if (piece == 0 && tid == 0) w.found[b].row = -1;
        return;
    }
    const double scale = scale_of(a, b);
    if (tid == 0) stop = scale == 0.0 ? 0 : n - 1;
    __syncthreads();
    for (int i = wave; i < n - 1; i += kThreads / 64) {
        const long long r = first + i;
        double p = __builtin_nan("");
        if (scale != 0.0) {
            const Stat s = row_stat(w, r, scale);
            const uint32_t d = a.drafts[r];
            p = s.m == -kInf ? __builtin_nan("") : 0.0;
            if (d < static_cast<uint32_t>(a.V) && s.m != -kInf)
                p = exp((static_cast<double>(logit<BF16>(row_at<BF16>(a, r), d)) - s.m) * scale) / s.z;
            else if (s.z != s.z)
                p = s.z;
            if (lane == 0) {
                const double q = !a.probs ? 1.0 : d < static_cast<uint32_t>(a.V) ? a.probs[r * a.probs_ld + d] : 1.0;
                if (!(static_cast<double>(a.u[r]) * q < p)) atomicMin(&stop, i);
            }
        }
        if (lane == 0 && piece == 0 && a.p_draft) a.p_draft[r] = static_cast<float>(p);
    }
    __syncthreads();
    if (wave == 0) {
        const int j = stop;
        const long long r = first + j;
        Stat s{0.0, -kInf, 0};
        if (scale != 0.0) s = row_stat(w, r, scale);
        if (lane == 0) {
            const bool bad = s.m == -kInf || !(s.z < __builtin_inf());
            shared = Found{s.z, bad ? 0.0 : scale, s.m, static_cast<int>(r), j, j < n - 1, last - 1};
            if (piece == 0) w.found[b] = shared;
        }
    }
    __syncthreads();
    const Found f = shared;
    if (f.scale == 0.0) return;
    const void* row = row_at<BF16>(a, f.row);
    const uint32_t draft = f.drafted && !a.probs ? a.drafts[f.row] : KDA_NO_TOKEN;
    int from, to;
    range_of(a, w, piece, from, to);
    Mass sum{0.0, 0.0};
    for (int v = from; v < to; ++v) {
        double e;
        sum.w += weight<BF16>(a, f, row, v, draft, e);
        sum.p += e;
    }
    sum.w = wave_sum(sum.w);
    sum.p = wave_sum(sum.p);
    if (lane == 0) waves[wave] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = waves[0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) {
            sum.w += waves[i].w;
            sum.p += waves[i].p;
        }
        w.mass[b * w.pieces + piece] = sum;
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_token_kernel(SampledArgs a, Split w) {
    __shared__ double waves[kThreads / 64];
    __shared__ int token, behind;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Found f = w.found[b];
    if (f.row < 0) return;
    if (f.scale == 0.0) {
        if (tid == 0) {
            a.out[2 * b] = f.j;
            a.out[2 * b + 1] = KDA_NO_TOKEN;
        }
        return;
    }
    // the piece: the first whose running sum passes the place (every wave finds it)
    Mass mass{0.0, 0.0};
    if (lane < w.pieces) mass = w.mass[b * w.pieces + lane];
    if (f.drafted && !(wave_sum(mass.w) > 0.0)) f.drafted = 0;
    const double mine = f.drafted ? mass.w : mass.p;
    double upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(upto, d);
        if (lane >= d) upto += y;
    }
    const double place = static_cast<double>(a.u[f.last]) * __shfl(upto, 63);
    uint64_t mask = __ballot(mine > 0.0 && upto > place);
    if (mask == 0) {   // a place at or behind the end: the last piece with weight
        mask = __ballot(mine > 0.0);
        mask = mask ? 1ull << (63 - __builtin_clzll(mask)) : 1ull;
    }
    const int piece = __builtin_ctzll(mask);
    const double before = __shfl(upto - mine, piece);
    // the token in it
    const void* row = row_at<BF16>(a, f.row);
    const uint32_t draft = f.drafted && !a.probs ? a.drafts[f.row] : KDA_NO_TOKEN;
    int from, to;
    range_of(a, w, piece, from, to);
    double sum = 0.0, e;
    for (int v = from; v < to; ++v) sum += weight<BF16>(a, f, row, v, draft, e);
    double run = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(run, d);
        if (lane >= d) run += y;
    }
    if (lane == 63) waves[wave] = run;
    if (tid == 0) {
        token = a.V;
        behind = -1;
    }
    __syncthreads();
    double at = before + run - sum;
    for (int i = 0; i < wave; ++i) at += waves[i];
    if (sum > 0.0) {
        int lowest = a.V, highest = -1;
        for (int v = from; v < to; ++v) {
            const double x = weight<BF16>(a, f, row, v, draft, e);
            at += x;
            if (x > 0.0) {
                highest = v;
                if (at > place && lowest == a.V) lowest = v;
            }
        }
        if (lowest < a.V) atomicMin(&token, lowest);
        if (highest >= 0) atomicMax(&behind, highest);
    }
    __syncthreads();
    if (tid == 0) {
        a.out[2 * b] = f.j;
        a.out[2 * b + 1] = static_cast<uint32_t>(token < a.V ? token : behind);
    }
}

// Enough workgroups to fill the chip, each with four loads a lane at least.
int parts_of(int R, int V, int es) {
    const long long loads = (static_cast<long long>(V) * es + 15) / 16;
    long long p = (loads + 4 * kThreads - 1) / (4 * kThreads);
    const long long fill = (1024 + R - 1) / R;
    p = p < fill ? p : fill;
    return static_cast<int>(p > kMostParts ? kMostParts : p);
}

int pieces_of(int B, int V) {
    long long p = (static_cast<long long>(V) + 4 * kThreads - 1) / (4 * kThreads);
    const long long fill = (1024 + B - 1) / B;
    p = p < fill ? p : fill;
    return static_cast<int>(p > kMostParts ? kMostParts : p);
}

template <bool BF16>
hipError_t launch(const SampledArgs& a, hipStream_t stream) {
    Split w{};
    w.parts = parts_of(a.R, a.V, BF16 ? 2 : 4);
    w.pieces = pieces_of(a.B, a.V);
    w.stats = static_cast<Stat*>(a.work);
    w.mass = reinterpret_cast<Mass*>(w.stats + static_cast<long long>(a.R) * w.parts);
    w.found = reinterpret_cast<Found*>(w.mass + static_cast<long long>(a.B) * w.pieces);
    sample_stats_kernel<BF16><<<dim3(static_cast<unsigned>(a.R + a.B) * w.parts), dim3(kThreads), 0, stream>>>(a, w);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sample_accept_kernel<BF16><<<dim3(static_cast<unsigned>(a.B) * w.pieces), dim3(kThreads), 0, stream>>>(a, w);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    sample_token_kernel<BF16><<<dim3(static_cast<unsigned>(a.B)), dim3(kThreads), 0, stream>>>(a, w);
    return hipGetLastError();
}

}  // namespace

long long sampled_work_bytes(int R, int B, int V) {
    // f32 rows are the longer ones: never fewer parts than bf16 rows
    return static_cast<long long>(R) * parts_of(R, V, 4) * static_cast<long long>(sizeof(Stat)) +
           static_cast<long long>(B) * (pieces_of(B, V) * static_cast<long long>(sizeof(Mass)) + static_cast<long long>(sizeof(Found)));
}

long long sampled_workgroups(int R, int B, int V) {
    if (R < 1) return 0;
    const long long rows = (static_cast<long long>(R) + B) * parts_of(R, V, 4), pieces = static_cast<long long>(B) * pieces_of(B, V);
    return rows > pieces ? rows : pieces;
}

hipError_t launch_sampled(const SampledArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace kda
