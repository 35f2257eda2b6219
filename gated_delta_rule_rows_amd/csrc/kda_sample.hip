// gfx950 kernels of kda_accept_sampled: drafted tokens verified against the
// target's probabilities from given random numbers.
//
// Row r of a session, p = softmax(x / T): the draft d is accepted while
// u q(d) < p(d).  At the first row j that does not accept (or the last row),
// the token is drawn from weights w = max(p - q, 0) (the last row: p): the
// lowest v whose running sum passes u_last times the whole sum.
//
// Three launches.  The first reads the logits once: of every part of a row the
// maximum m and z = sum e^{(x - m) / T}.  In the second each workgroup joins its
// session's rows, finds j and sums the weights of a piece of row j; the third
// finds the piece that holds the place, and the token in it.  (As the work of the
// second's last workgroup the third's cost more than a launch: release and acquire
// over the chip's eight L2 caches, 28 us for 15 rows of 50,001 against 18.)
// The exponentials of whole rows are f32; their sums, a draft's p, p - q (which
// cancels) and the running sums (which decide between two tokens near their border)
// are f64.  An f32 exponential is off by three roundings of its argument (log2(e) / T,
// x - m and their product), 3 (m - x) / T half steps, and its own; the sum of a row by
// the mean of that, and the mean of (m - x) / T under p is ln V at most: it is the row's
// entropy less the logarithm of a sum of 1 at least.
//
// On an MI355X, calls in a loop: 64 sessions x 8 rows of 150,000 bf16 58 us (38 at
// the 5.1 TB/s of a large copy): the logits 36 us, 4.3 TB/s, bound by VALU (0.8-0.9),
// the sums of row j 19 us, the token 5.  One round of 15 rows of 150,000 f32 17 us, a
// token for each of 15 sessions 14 us: three launches of 4 to 8 us, latency.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kda.h"
#include "kda_cache.h"
#include "kda_launch.h"
#include "kda_seq.h"

namespace kda {
namespace {

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.44269504088896340736;
constexpr float kSlack = 6.0f;       // the carried reference may lag by this much (base 2)
constexpr int kThreads = 256;
constexpr int kMostParts = 64;       // of a row: a lane joins a part
constexpr int kChunk = 4096;         // tokens of a piece, if that makes no more than 64 pieces
constexpr int kAcceptThreads = 512;
constexpr int kTokenThreads = 512;

// m, about the largest x, and z = sum 2^{(x - m) by}, by = log2(e) / T; z is NaN where a value is NaN
// or +inf.  (Taken as x by - c in one operation a power would be cheaper, but where x / T is large the rounding
// of c alone would pass f32's range.)
struct Stat {
    double z;
    float m;
    int pad;
};

// A session's row j.
struct Found {
    double z;
    double u;      // of the session's last row
    double by;     // 0: no token
    float m;
    int row;       // -1: the session has no rows
    int j;
    int drafted;   // weights max(p - q, 0) unless these are all 0; else p
};

// Sums of a part's weights and probabilities (times z).
struct Mass {
    double w, p;
};

struct Split {
    Stat* stats;     // [R][parts]
    Mass* mass;      // [B][pieces]
    Found* found;    // [B]
    int parts;       // of a row in the first launch
    int pieces;      // of row j, each with a sum
    int groups;      // workgroups of a session in the second launch
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

// log2(e) / T of a session; 0 where T is no finite number of 1e-30 at least (it has to be one in f32).
__device__ __forceinline__ double by_of(const SampledArgs& a, int b) {
    const float t = a.temp ? a.temp[b] : 1.f;
    return t >= 1e-30f && t < kInf ? kLog2e / t : 0.0;
}

__device__ __forceinline__ double wave_sum(double x) { return of_lane(running_sum(x), 63); }

__device__ __forceinline__ float wave_max(float x) {
    return of_lane(running(x, -kInf, [](float a, float b) { return fmaxf(a, b); }), 63);
}

// s's z at a reference m >= s.m.
__device__ __forceinline__ double moved(Stat s, float m, double by) {
    return s.m == -kInf ? s.z : s.z * exp2((static_cast<double>(s.m) - m) * by);
}

// Adds E values of a lane.
template <int E>
__device__ __forceinline__ void take(Stat& s, const float (&x)[E], double by) {
    const float by32 = static_cast<float>(by);
    float top = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, x[e]);
    if (__ballot(((top - s.m) * by32 > kSlack) | (s.m == -kInf))) {
        const float m = fmaxf(s.m, top);
        s.z = moved(s, m, by);
        s.m = m;
    }
    const float base = s.m == -kInf ? 0.f : s.m;
    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) z[e & 3] += __builtin_amdgcn_exp2f((x[e] - base) * by32);
    s.z += (z[0] + z[1]) + (z[2] + z[3]);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_stats_kernel(SampledArgs a, Split w) {
    constexpr int E = BF16 ? 8 : 4;
    const int part = blockIdx.x % w.parts;
    const Part f = find_part(a, 1, blockIdx.x / w.parts);
    if (f.b < 0) return;
    const double by = by_of(a, f.b);
    if (by == 0.0) return;
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
    constexpr int U = 4;   // loads ahead
    const uint32_t low = BF16 ? 0xFF80FF80u : 0xFF800000u;   // -inf
    const auto fetch = [&](int i0, uint4 (&u)[U]) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k * kThreads + tid;
            u[k] = i < end ? body[i] : make_uint4(low, low, low, low);
        }
    };
    uint4 u[U], next[U];
    fetch(begin, next);
    for (int i0 = begin; i0 < end; i0 += U * kThreads) {
#pragma unroll
        for (int k = 0; k < U; ++k) u[k] = next[k];
        if (i0 + U * kThreads < end) fetch(i0 + U * kThreads, next);
        float x[U * E];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const uint32_t v[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if constexpr (BF16)
                    x[k * E + e] = __builtin_bit_cast(float, e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
                else
                    x[k * E + e] = __builtin_bit_cast(float, v[e]);
            }
        }
        take<U * E>(s, x, by);
    }
    if (wave == 0) {
        const bool first = part == 0 && lane < head, last = part == w.parts - 1 && lane < tail;
        const float x[2] = {first ? logit<BF16>(row, lane) : -kInf, last ? logit<BF16>(row, a.V - tail + lane) : -kInf};
        take<2>(s, x, by);
    }
    __shared__ Stat waves[kThreads / 64];
    const float m = wave_max(s.m);
    const double z = wave_sum(moved(s, m, by));
    if (lane == 0) waves[wave] = Stat{z, m, 0};
    __syncthreads();
    if (tid == 0) {
        float top = waves[0].m;
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) top = fmaxf(top, waves[i].m);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) sum += moved(waves[i], top, by);
        w.stats[r * w.parts + part] = Stat{sum, top, 0};
    }
}

// m and z of row r, in every lane.
__device__ __forceinline__ Stat row_stat(const Split& w, long long r, double by) {
    const int lane = threadIdx.x & 63;
    Stat s{0.0, -kInf, 0};
    if (lane < w.parts) s = w.stats[r * w.parts + lane];
    const float m = wave_max(s.m);
    return Stat{wave_sum(moved(s, m, by)), m, 0};
}

// Weights of a row, times z.
struct Weights {
    const void* row;
    const float* probs;
    double z;
    float m, by;             // e = 2^{(x - m) by}
    uint32_t draft;
};

// What they are: p, p without the draft, or max(p - q, 0).
enum { kWhole, kOthers, kLeft };

__device__ __forceinline__ int kind_of(const SampledArgs& a, const Found& f) { return !f.drafted ? kWhole : a.probs ? kLeft : kOthers; }

template <bool BF16>
__device__ __forceinline__ Weights weights_of(const SampledArgs& a, const Found& f) {
    return Weights{row_at<BF16>(a, f.row), a.probs ? a.probs + f.row * a.probs_ld : nullptr, f.z, f.m, static_cast<float>(f.by),
                   a.probs ? KDA_NO_TOKEN : a.drafts[f.row]};
}

// Weights w and e = p z of tokens v0, v0 + step, ... below end (> v0 - step N); 0 behind it.
template <bool BF16, int KIND, int N>
__device__ __forceinline__ void weigh(const Weights& of, int v0, int step, int end, double (&w)[N], double (&e)[N]) {
    float x[N], q[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int v = min(v0 + i * step, end - 1);
        x[i] = logit<BF16>(of.row, v);
        if constexpr (KIND == kLeft) q[i] = of.probs[v];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int v = v0 + i * step;
        e[i] = v < end ? __builtin_amdgcn_exp2f((x[i] - of.m) * of.by) : 0.f;
        w[i] = e[i];
        if constexpr (KIND == kOthers) w[i] = static_cast<uint32_t>(v) == of.draft ? 0.0 : e[i];
        if constexpr (KIND == kLeft) w[i] = v < end ? fmax(fma(-of.z, static_cast<double>(q[i]), e[i]), 0.0) : 0.0;
    }
}

// f(KIND) for a kind known on the device, the same for all lanes.
template <typename F>
__device__ __forceinline__ void by_kind(int kind, F&& f) {
    if (kind == kWhole)
        f(std::integral_constant<int, kWhole>{});
    else if (kind == kOthers)
        f(std::integral_constant<int, kOthers>{});
    else
        f(std::integral_constant<int, kLeft>{});
}

__device__ __forceinline__ int piece_tokens(const SampledArgs& a, const Split& w) { return (a.V + w.pieces - 1) / w.pieces; }

// The token of a session.
template <bool BF16>
__global__ void __launch_bounds__(kTokenThreads) sample_token_kernel(SampledArgs a, Split w) {
    constexpr int WAVES = kTokenThreads / 64, N = kChunk / kTokenThreads;
    static_assert(WAVES * N == 64, "a lane for each 64 tokens of a chunk");
    __shared__ double sums[64];
    __shared__ int token, behind;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Found f = w.found[b];
    Mass mass{0.0, 0.0};
    if (lane < w.pieces) mass = w.mass[b * w.pieces + lane];
    if (f.row < 0) return;
    if (f.by == 0.0) {
        if (tid == 0) {
            a.out[2 * b] = f.j;
            a.out[2 * b + 1] = KDA_NO_TOKEN;
        }
        return;
    }
    // the piece: the first whose running sum passes the place (every wave finds it)
    if (f.drafted && __ballot(mass.w > 0.0) == 0) f.drafted = 0;
    const double mine = f.drafted ? mass.w : mass.p, upto = running_sum(mine);
    const double place = f.u * of_lane(upto, 63);
    uint64_t mask = __ballot(mine > 0.0 && upto > place);
    if (mask == 0) {   // a place at or behind the end: the last piece with weight
        mask = __ballot(mine > 0.0);
        mask = mask ? 1ull << (63 - __builtin_clzll(mask)) : 1ull;
    }
    const int piece = __builtin_ctzll(mask);
    double at = of_lane(upto - mine, piece);
    // the token in it: sums of each 64 tokens, their running sums, and those of the tokens where the
    // place lies
    const Weights weights = weights_of<BF16>(a, f);
    const int each = piece_tokens(a, w), begin = min(piece * each, a.V), end = min(begin + each, a.V);
    if (tid == 0) {
        token = a.V;
        behind = -1;
    }
    for (int v0 = begin; v0 < end; v0 += kChunk) {
        double x[N], e[N];
        by_kind(kind_of(a, f), [&](auto k) { weigh<BF16, k.value>(weights, v0 + tid, kTokenThreads, end, x, e); });
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = wave_sum(x[i]);
        __syncthreads();   // (behind the reads of the chunk before)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane == 0) sums[i * WAVES + wave] = e[i];
        __syncthreads();
        const double part = sums[lane], run = at + running_sum(part);
        const uint64_t parts = __ballot(part > 0.0), passed = __ballot(part > 0.0 && run > place);
        const int found = passed ? __builtin_ctzll(passed) : parts ? 63 - __builtin_clzll(parts) : -1;
        if (found >= 0 && found % WAVES == wave) {
            const double before = of_lane(run - part, found);
            double mine64 = 0.0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (found / WAVES == i) mine64 = x[i];
            const double here = before + running_sum(mine64);
            const int v = v0 + found * 64 + lane;
            const uint64_t some = __ballot(mine64 > 0.0), hit = __ballot(mine64 > 0.0 && here > place);
            if (hit && lane == __builtin_ctzll(hit)) token = v;
            if (some && lane == 63 - __builtin_clzll(some)) behind = v;
        }
        __syncthreads();
        if (token < a.V) break;
        at = of_lane(run, 63);
    }
    if (tid == 0) {
        a.out[2 * b] = f.j;
        a.out[2 * b + 1] = static_cast<uint32_t>(token < a.V ? token : behind);
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kAcceptThreads) sample_accept_kernel(SampledArgs a, Split w) {
    constexpr int WAVES = kAcceptThreads / 64;
    __shared__ int stop;
    __shared__ Found shared;
    __shared__ Mass waves[2][WAVES];
    const int group = blockIdx.x % w.groups, b = blockIdx.x / w.groups;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int first, last;
    sequence(a, b, first, last);
    const int n = last - first;
    if (n == 0) {
        if (group == 0 && tid == 0) w.found[b].row = -1;
        return;
    }
    const double u_last = a.u[last - 1];
    const double by = by_of(a, b);
    if (tid == 0) stop = by == 0.0 ? 0 : n - 1;
    __syncthreads();
    for (int i = wave; i < n - 1; i += WAVES) {
        const long long r = first + i;
        double p = __builtin_nan("");
        if (by != 0.0) {
            const uint32_t d = a.drafts[r];
            const bool real = d < static_cast<uint32_t>(a.V);
            const float x = real ? logit<BF16>(row_at<BF16>(a, r), d) : -kInf;
            const double q = a.probs && real ? a.probs[r * a.probs_ld + d] : 1.0, u = a.u[r];
            const Stat s = row_stat(w, r, by);
            if (s.m != -kInf) p = exp2((static_cast<double>(x) - s.m) * by) / s.z;
            if (lane == 0 && !(u * q < p)) atomicMin(&stop, i);
        }
        if (lane == 0 && group == 0 && a.p_draft) a.p_draft[r] = static_cast<float>(p);
    }
    __syncthreads();
    if (wave == 0) {
        const int j = stop;
        Stat s{0.0, -kInf, 0};
        if (by != 0.0) s = row_stat(w, first + j, by);
        const bool bad = s.m == -kInf || !(s.z < __builtin_inf());
        if (lane == 0) {
            shared = Found{s.z, u_last, bad ? 0.0 : by, s.m, first + j, j, j < n - 1};
            if (group == 0) w.found[b] = shared;
        }
    }
    __syncthreads();
    const Found f = shared;
    if (f.by == 0.0) return;
    const Weights weights = weights_of<BF16>(a, f);
    const int kind = kind_of(a, f);
    const int each = piece_tokens(a, w);
    const int p0 = static_cast<int>(static_cast<long long>(w.pieces) * group / w.groups);
    const int p1 = static_cast<int>(static_cast<long long>(w.pieces) * (group + 1) / w.groups);
    for (int piece = p0; piece < p1; ++piece) {
        const int begin = min(piece * each, a.V), end = min(begin + each, a.V);
        Mass sum{0.0, 0.0};
        by_kind(kind, [&](auto k) {
            constexpr int N = 8;
            for (int v = begin + tid; v < end; v += N * kAcceptThreads) {
                double x[N], e[N];
                weigh<BF16, k.value>(weights, v, kAcceptThreads, end, x, e);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    sum.w += x[n];
                    sum.p += e[n];
                }
            }
        });
        sum.w = wave_sum(sum.w);
        sum.p = wave_sum(sum.p);
        Mass* mine = waves[piece & 1];
        if (lane == 0) mine[wave] = sum;
        __syncthreads();   // (the next piece's sums go to the other half)
        if (tid == 0) {
            sum = mine[0];
#pragma unroll
            for (int i = 1; i < WAVES; ++i) {
                sum.w += mine[i].w;
                sum.p += mine[i].p;
            }
            w.mass[b * w.pieces + piece] = sum;
        }
    }
}

constexpr int kFill = 2048;   // workgroups that fill the chip

// Parts of a row that leave each four loads a lane at least.
int most_parts(int V, int es) {
    const long long loads = (static_cast<long long>(V) * es + 15) / 16, p = (loads + 4 * kThreads - 1) / (4 * kThreads);
    return static_cast<int>(p < kMostParts ? p : kMostParts);
}

// Of them as many as fill the chip.
int parts_of(int R, int V, int es) {
    const int p = most_parts(V, es), fill = (kFill + R - 1) / R;
    return p < fill ? p : fill;
}

int pieces_of(int V) {
    const int p = (V + kChunk - 1) / kChunk;
    return p > kMostParts ? kMostParts : p;
}

// Two workgroups a CU: each repeats its session's walk.
int groups_of(int B, int V) {
    const int p = pieces_of(V), fill = (512 + B - 1) / B;
    return p < fill ? p : fill;
}

template <bool BF16>
hipError_t launch(const SampledArgs& a, hipStream_t stream) {
    Split w{};
    w.parts = parts_of(a.R, a.V, BF16 ? 2 : 4);
    w.pieces = pieces_of(a.V);
    w.groups = groups_of(a.B, a.V);
    w.stats = static_cast<Stat*>(a.work);
    w.mass = reinterpret_cast<Mass*>(w.stats + static_cast<long long>(a.R) * w.parts);
    w.found = reinterpret_cast<Found*>(w.mass + static_cast<long long>(a.B) * w.pieces);
    sample_stats_kernel<BF16><<<dim3(static_cast<unsigned>(a.R + a.B) * w.parts), dim3(kThreads), 0, stream>>>(a, w);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sample_accept_kernel<BF16><<<dim3(static_cast<unsigned>(a.B) * w.groups), dim3(kAcceptThreads), 0, stream>>>(a, w);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    sample_token_kernel<BF16><<<dim3(static_cast<unsigned>(a.B)), dim3(kTokenThreads), 0, stream>>>(a, w);
    return hipGetLastError();
}

}  // namespace

// Grows with R, B and V, though the parts of a row become fewer with R: R rows have R * most_parts() statistics at
// most, and R * ceil(kFill / R) < kFill + R.  (f32 rows are the longer ones: never fewer parts than bf16 rows.)
long long sampled_work_bytes(int R, int B, int V) {
    const long long all = static_cast<long long>(R) * most_parts(V, 4), fill = static_cast<long long>(R) + kFill - 1;
    return (all < fill ? all : fill) * static_cast<long long>(sizeof(Stat)) +
           static_cast<long long>(B) * (pieces_of(V) * static_cast<long long>(sizeof(Mass)) + static_cast<long long>(sizeof(Found)));
}

long long sampled_workgroups(int R, int B, int V) {
    if (R < 1) return 0;
    const long long rows = (static_cast<long long>(R) + B) * parts_of(R, V, 4), groups = 2ll * B * groups_of(B, V);   // (of twice the threads)
    return rows > groups ? rows : groups;
}

hipError_t launch_sampled(const SampledArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace kda
