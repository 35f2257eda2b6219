// gfx950 kernels of kda_logprobs: log probabilities of given tokens, entropy
// and the top alternatives of logits rows.
//
// With m = max x, z = sum exp(x - m), y = x - m:
//   lp = y[token] - log z,   entropy = log z - (sum exp(y) y) / z
// and the top n by (value, lowest index first).
//
// One pass over the logits.  A lane carries its own running m, z and
// w = sum exp(y) y, moved to the new maximum once a 16-byte load; a wave keeps
// the best n keys it has seen, sorted, one a lane.  A step of the wave costs
// the list one compare a lane while nothing beats its last entry (a wave's
// steps rise in index, so an equal value never does); what does is inserted by
// a ballot for its place and a shift of the lanes behind it.  The first loads of
// a wave fill its list at once.
//
// Few rows are split over workgroups, whose waves leave their sums and lists
// in the workspace for a second launch; many rows take a workgroup each, which
// joins its waves through LDS.  The join takes, of W sorted lists, those whose
// head is among the n best heads, and ranks what is left by counting.  Keys
// are unique, so neither the order of the lists nor the positions that the
// candidates take change the result; sums are joined in a fixed order.
//
// 2048 rows of 150,000 logits, 8 alternatives: bf16 131 us, 4.7 TB/s, bound by
// VALU (0.85); f32 210 us, 5.85 TB/s.  15 rows of 150,000 f32, 20 alternatives: 9
// us for the parts and 6 for the join, latency of the lists and of the sums'
// exchanges.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_launch.h"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kInf = __builtin_inff();
constexpr float kSlack = 4.0f;
constexpr int kSplitThreads = 256;    // workgroup of a split row
constexpr int kMaxSplits = 64;        // workgroups of a row, at most
constexpr int kMaxLists = kMaxSplits * (kSplitThreads / 64);

using Key = unsigned long long;       // ordered value, then ~index: greater is better, 0 is none

// The value's bits in the order of the values, -0 as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(Key k) {
    const uint32_t o = static_cast<uint32_t>(k >> 32);
    return __builtin_bit_cast(float, o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Sums of a part of a row, relative to m, which no value exceeds by more than
// kSlack (a move costs an exponential; e^4 costs the sums nothing).  A NaN in z
// says that the part holds a NaN or +inf.
struct Sums {
    float m, z, w;
};

__device__ __forceinline__ float exp_of(float y) { return __builtin_amdgcn_exp2f(y * kLog2e); }

// Moves s to a maximum m >= s.m.
__device__ __forceinline__ void move_to(Sums& s, float m) {
    // (held above -1e30, whose exponential is 0 as well, so that z d stays finite)
    const float d = s.m == -kInf || s.m == m ? 0.f : fmaxf(s.m - m, -1e30f);
    const float c = s.m == -kInf ? 0.f : exp_of(d);
    s.w = c * fmaf(s.z, d, s.w);
    s.z *= c;
    s.m = m;
}

__device__ __forceinline__ void join(Sums& a, Sums b) {
    const bool bad = a.z != a.z || b.z != b.z;
    const float m = fmaxf(a.m, b.m);
    move_to(a, m);
    move_to(b, m);
    a.z = bad ? __builtin_nanf("") : a.z + b.z;
    a.w += b.w;
}

// The best n keys of a wave, best first, key i in lane i.
struct List {
    Key mine;
    float bar;    // a value has to be above it to enter
    Key last;     // the n-th key
};

__device__ __forceinline__ Key lane_key(Key k, int lane) {
    return static_cast<Key>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(k >> 32), lane))) << 32 |
           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(k), lane));
}

__device__ __forceinline__ void insert(List& l, Key k, int n) {
    const int lane = threadIdx.x & 63;
    const int at = __builtin_popcountll(__ballot(l.mine > k));
    // the key of the lane before (wave_shr:1)
    const Key up = static_cast<Key>(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
                       0, static_cast<int>(l.mine >> 32), 0x138, 0xF, 0xF, true))) << 32 |
                   static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(l.mine), 0x138, 0xF, 0xF, true));
    l.mine = lane < at ? l.mine : lane == at ? k : up;
    l.last = lane_key(l.mine, n - 1);
}

// Takes the lanes' values x, of index i each.
__device__ __forceinline__ void offer(List& l, float x, uint32_t i, int n) {
    const Key k = x > -kInf ? static_cast<Key>(ordered(x)) << 32 | static_cast<uint32_t>(~i) : 0;
    uint64_t mask = __ballot(k > l.last);
    while (mask) {
        insert(l, lane_key(k, __builtin_ctzll(mask)), n);
        mask &= mask - 1;
        mask &= __ballot(k > l.last);
    }
    l.bar = l.last == 0 ? -kInf : value_of(l.last);
}

// The list of a wave's first N values a lane, value e of index at(e).  Without
// it each of the first hundreds of values would be inserted.  The n-th largest
// of the lanes' maxima is found bit by bit; at least n values reach it, and few
// more: they are gathered in LDS and ranked by counting.  More than 64 (many
// equal values) are inserted one by one.  space: 64 keys of this wave's.
template <int N, typename At>
__device__ __forceinline__ void start(List& l, const float (&x)[N], At at, int n, volatile Key* space) {
    const int lane = threadIdx.x & 63;
    float top = x[0];
#pragma unroll
    for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
    const uint32_t o = ordered(top);
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t up = t | 1u << bit;
        if (__builtin_popcountll(__ballot(o >= up)) >= n) t = up;
    }
    const float least = value_of(static_cast<Key>(t) << 32);
    int c = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) c += __builtin_popcountll(__ballot(x[e] >= least && x[e] > -kInf));
    if (c > 64) {
#pragma unroll
        for (int e = 0; e < N; ++e) offer(l, x[e], at(e), n);
        return;
    }
    int p = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const bool in = x[e] >= least && x[e] > -kInf;
        const uint64_t mask = __ballot(in);
        const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
        if (in) space[p + before] = static_cast<Key>(ordered(x[e])) << 32 | static_cast<uint32_t>(~at(e));
        p += __builtin_popcountll(mask);
    }
    __builtin_amdgcn_wave_barrier();
    Key k = lane < c ? space[lane] : 0;
    int rank = 0;
    for (int i = 0; i < c; ++i) rank += lane_key(k, i) > k;
    if (lane < c) space[rank] = k;
    __builtin_amdgcn_wave_barrier();
    l.mine = lane < c ? space[lane] : 0;
    l.last = lane_key(l.mine, n - 1);
    l.bar = l.last == 0 ? -kInf : value_of(l.last);
}

// E values of a lane, whose indexes follow each other from i.
template <int E, bool TOP>
__device__ __forceinline__ void take(Sums& s, List& l, const float (&x)[E], uint32_t i, int n) {
    float top = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, x[e]);
    // m need not be the maximum: it follows once a value is well above it
    if (__ballot(top > s.m + kSlack || s.m == -kInf)) move_to(s, fmaxf(s.m, top));
    const float base = s.m == -kInf ? 0.f : s.m;
    // one add a load to the running sums: each add rounds by their size, and takes
    // nothing of what is under half a last place of them
    float z = 0.f, w = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float y = x[e] - base;
        const float p = exp_of(y);
        z += p;
        w = fmaf(p, fmaxf(y, -1e30f), w);
    }
    s.z += z;
    s.w += w;
    if constexpr (TOP) {
        if (__ballot(top > l.bar)) {
#pragma unroll
            for (int e = 0; e < E; ++e) offer(l, x[e], i + e, n);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, long long i) {
    if constexpr (BF16)
        return __builtin_bit_cast(float, static_cast<uint32_t>(static_cast<const uint16_t*>(row)[i]) << 16);
    else
        return static_cast<const float*>(row)[i];
}

template <bool BF16>
__device__ __forceinline__ void values(uint4 u, float (&x)[BF16 ? 8 : 4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (BF16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __builtin_bit_cast(float, e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __builtin_bit_cast(float, w[e]);
    }
}

__device__ __forceinline__ Sums wave_sums(Sums s) {
    float m = s.m;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    if (m > s.m) move_to(s, m);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        s.z += __shfl_xor(s.z, d);
        s.w += __shfl_xor(s.w, d);
    }
    return s;
}

// Part `part` of `parts` of a row, by one workgroup: the wave's sums (all lanes
// alike) and list.  The row is read from its first 16-byte boundary on in whole
// loads, four a lane in flight; what lies before and behind goes to one wave.
// FILL of a lane's first loads fill the list.
template <bool BF16, bool TOP, int THREADS, int LOADS, int FILL>
__device__ __forceinline__ void read_part(const LogprobArgs& a, const void* row, int part, int parts, Sums& s, List& l) {
    constexpr int E = BF16 ? 8 : 4, U = LOADS;
    const int tid = threadIdx.x, lane = tid & 63;
    const bool first = tid < 64;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row);
    const int head = min(a.V, static_cast<int>((16 - (at & 15)) & 15) / (BF16 ? 2 : 4));
    const int vectors = (a.V - head) / E;
    const int tail = a.V - head - vectors * E;
    const int each = (vectors + parts - 1) / parts;
    const int begin = min(part * each, vectors), end = min(begin + each, vectors);
    const uint4* body = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + head * (BF16 ? 2 : 4));
    s = Sums{-kInf, 0.f, 0.f};
    l = List{0, -kInf, 0};
    __shared__ Key space[TOP ? THREADS / 64 : 1][64];
    const float x0[1] = {first && part == 0 && lane < head ? logit<BF16>(row, lane) : -kInf};
    if (first && part == 0 && head > 0) take<1, false>(s, l, x0, lane, a.n_top);
    const uint32_t low = BF16 ? 0xFF80FF80u : 0xFF800000u;   // -inf
    const auto fetch = [&](int v0, uint4 (&u)[U]) {
        if (v0 + U * THREADS <= end) {
#pragma unroll
            for (int i = 0; i < U; ++i) u[i] = body[v0 + i * THREADS + tid];
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int v = v0 + i * THREADS + tid;
                u[i] = v < end ? body[v] : make_uint4(low, low, low, low);
            }
        }
    };
    uint4 u[U], next[U];
    if (begin < end) fetch(begin, next);
    for (int v0 = begin; v0 < end; v0 += U * THREADS) {
#pragma unroll
        for (int i = 0; i < U; ++i) u[i] = next[i];
        if (v0 + U * THREADS < end) fetch(v0 + U * THREADS, next);
        if (TOP && v0 == begin) {
            float x[FILL * E + 1];
            x[FILL * E] = x0[0];
#pragma unroll
            for (int i = 0; i < FILL; ++i) {
                float y[E];
                values<BF16>(u[i], y);
#pragma unroll
                for (int e = 0; e < E; ++e) x[i * E + e] = y[e];
            }
            const auto at = [&](int e) {
                return e == FILL * E ? lane : head + (v0 + e / E * THREADS + tid) * E + e % E;
            };
            start(l, x, at, a.n_top, space[tid >> 6]);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float y[E];
                values<BF16>(u[i], y);
                if (i < FILL)
                    take<E, false>(s, l, y, 0, 0);
                else
                    take<E, true>(s, l, y, head + (v0 + i * THREADS + tid) * E, a.n_top);
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int v = v0 + i * THREADS;
            if (v + (tid & ~63) >= end) break;
            float x[E];
            values<BF16>(u[i], x);
            take<E, TOP>(s, l, x, head + (v + tid) * E, a.n_top);
        }
    }
    if (TOP && begin >= end && part == 0 && first) offer(l, x0[0], lane, a.n_top);   // no whole load
    if (first && part == parts - 1 && tail > 0) {
        const int i = a.V - tail + lane;
        const float x[1] = {lane < tail ? logit<BF16>(row, i) : -kInf};
        take<1, TOP>(s, l, x, i, a.n_top);
    }
    s = wave_sums(s);
}

// Joins W lists and their sums to the outputs of row r.  sums and lists: W
// entries and W * n_top keys, W <= THREADS; AHEAD keys a thread are read at once.
template <bool BF16, int THREADS, int AHEAD>
__device__ __forceinline__ void finish(const LogprobArgs& a, const void* row, long long r, int W, const Sums* sums,
                                       const Key* lists) {
    __shared__ Sums waves[THREADS / 64];
    __shared__ Key heads[THREADS], found[KDA_TOP_MAX * KDA_TOP_MAX];
    __shared__ Key bar;
    __shared__ int count;
    const int tid = threadIdx.x, n = a.n_top;
    Sums s{-kInf, 0.f, 0.f};
    Key head = 0;
    uint32_t tok = kNoToken;
    float given = 0.f;
    if (a.lp && tid == 0) {
        tok = a.tokens[r];
        if (tok < static_cast<uint32_t>(a.V)) given = logit<BF16>(row, tok);
    }
    Key ahead[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ahead[i] = i * THREADS + tid < W * n ? lists[i * THREADS + tid] : 0;
    if (tid < W) {
        s = sums[tid];
        if (n > 0) head = lists[tid * n];
    }
    s = wave_sums(s);
    if ((tid & 63) == 0) waves[tid >> 6] = s;
    heads[tid] = head;
    if (tid == 0) {
        count = 0;
        bar = 1;
    }
    __syncthreads();
    s = waves[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) join(s, waves[w]);
    const bool bad = s.z != s.z, empty = s.m == -kInf;
    const float log_z = logf(s.z);
    if (tid == 0) {
        if (a.lp) {
            float lp = __builtin_nanf("");
            if (!bad && tok < static_cast<uint32_t>(a.V)) lp = empty ? -kInf : given - s.m - log_z;
            a.lp[r] = lp;
        }
        if (a.entropy) a.entropy[r] = bad ? __builtin_nanf("") : empty ? 0.f : log_z - s.w / s.z;
    }
    if (n == 0) return;
    // only keys at or above the n-th best head can be among the n best
    if (W > n && head != 0) {
        int rank = 0;
#pragma unroll 16
        for (int i = 0; i < W; ++i) rank += heads[i] > head;
        if (rank == n - 1) bar = head;
    }
    __syncthreads();
    if (!bad) {
        const Key least = bar;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (ahead[i] >= least) found[atomicAdd(&count, 1)] = ahead[i];
        for (int i = AHEAD * THREADS + tid; i < W * n; i += THREADS) {
            const Key k = lists[i];
            if (k >= least) found[atomicAdd(&count, 1)] = k;
        }
    }
    __syncthreads();
    const int c = count;
    for (int i = tid; i < c; i += THREADS) {
        const Key k = found[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < c; ++j) rank += found[j] > k;
        if (rank < n) {
            a.top_ids[r * n + rank] = ~static_cast<uint32_t>(k);
            a.top_lp[r * n + rank] = value_of(k) - s.m - log_z;
        }
    }
    for (int i = c + tid; i < n; i += THREADS) {
        a.top_ids[r * n + i] = kNoToken;
        a.top_lp[r * n + i] = bad ? __builtin_nanf("") : -kInf;
    }
}

template <bool BF16>
__device__ __forceinline__ const void* row_at(const LogprobArgs& a, long long r) {
    return static_cast<const char*>(a.logits) + r * a.ld * (BF16 ? 2 : 4);
}

// A workgroup a row.
template <bool BF16, bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 64 ? 4 : 6) logprob_row_kernel(LogprobArgs a) {
    constexpr int W = THREADS / 64;
    __shared__ Sums sums[W];
    __shared__ Key lists[TOP ? W * KDA_TOP_MAX : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long r = blockIdx.x;
    const void* row = row_at<BF16>(a, r);
    Sums s;
    List l;
    read_part<BF16, TOP, THREADS, THREADS == 64 ? 4 : 2, 1>(a, row, 0, 1, s, l);
    if (lane == 0) sums[wave] = s;
    if (TOP && lane < a.n_top) lists[wave * a.n_top + lane] = l.mine;
    __syncthreads();
    finish<BF16, THREADS, 1>(a, row, r, W, sums, lists);
}

// Where the waves of split rows leave their results.
struct Split {
    Sums* sums;     // [t][W]
    Key* lists;     // [t][W][n_top]
    int parts;      // workgroups a row; W = parts * 4
};

template <bool BF16, bool TOP>
__global__ void __launch_bounds__(kSplitThreads) logprob_part_kernel(LogprobArgs a, Split x) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long r = blockIdx.y;
    Sums s;
    List l;
    read_part<BF16, TOP, kSplitThreads, 4, 4>(a, row_at<BF16>(a, r), blockIdx.x, x.parts, s, l);
    const long long at = (r * x.parts + blockIdx.x) * (kSplitThreads / 64) + wave;
    if (lane == 0) x.sums[at] = s;
    if (TOP && lane < a.n_top) x.lists[at * a.n_top + lane] = l.mine;
}

template <bool BF16>
__global__ void __launch_bounds__(kMaxLists) logprob_join_kernel(LogprobArgs a, Split x) {
    const long long r = blockIdx.x;
    const int W = x.parts * (kSplitThreads / 64);
    finish<BF16, kMaxLists, 12>(a, row_at<BF16>(a, r), r, W, x.sums + r * W, x.lists + r * W * a.n_top);
}

// Workgroups a row: 1 (a row each, joined in place) from 256 rows on, where
// the rows alone fill the chip; below that enough for 1024 workgroups, but not
// with less than four loads a lane.
constexpr int kWholeRows = 256, kWaveRows = 2048;

int parts_of(int t, int V, int es) {
    if (t >= kWholeRows) return 1;
    const long long loads = (static_cast<long long>(V) * es + 15) / 16;
    long long p = (loads + 4 * kSplitThreads - 1) / (4 * kSplitThreads);
    const long long fill = (1024 + t - 1) / t;
    p = p < fill ? p : fill;
    return static_cast<int>(p > kMaxSplits ? kMaxSplits : p);
}

long long split_bytes(int t, int parts, int n_top) {
    if (parts == 1) return 0;
    return static_cast<long long>(t) * parts * (kSplitThreads / 64) *
           (static_cast<long long>(sizeof(Sums)) + 8ll * n_top);
}

template <bool BF16>
hipError_t launch(const LogprobArgs& a, hipStream_t stream) {
    Split x{};
    x.parts = parts_of(a.t, a.V, BF16 ? 2 : 4);
    const bool top = a.n_top > 0;
    if (x.parts == 1) {
        const dim3 grid(static_cast<unsigned>(a.t));
        // A wave a row from 2048 rows on (two waves a SIMD), four below: a list is
        // filled and joined for each wave, and a row's end waits for its slowest.
        // 150,000 bf16 logits, 8 alternatives: 2048 rows 130 us with a wave, 139
        // with four; 1024 rows 102 and 83; 512 rows 106 and 54.
        if (a.t >= kWaveRows) {
            if (top)
                logprob_row_kernel<BF16, true, 64><<<grid, dim3(64), 0, stream>>>(a);
            else
                logprob_row_kernel<BF16, false, 64><<<grid, dim3(64), 0, stream>>>(a);
        } else if (top) {
            logprob_row_kernel<BF16, true, 256><<<grid, dim3(256), 0, stream>>>(a);
        } else {
            logprob_row_kernel<BF16, false, 256><<<grid, dim3(256), 0, stream>>>(a);
        }
        return hipGetLastError();
    }
    // the keys first: they need 8-byte alignment
    const long long lists = static_cast<long long>(a.t) * x.parts * (kSplitThreads / 64);
    x.lists = static_cast<Key*>(a.work);
    x.sums = reinterpret_cast<Sums*>(x.lists + lists * a.n_top);
    const dim3 grid(static_cast<unsigned>(x.parts), static_cast<unsigned>(a.t));
    if (top)
        logprob_part_kernel<BF16, true><<<grid, dim3(kSplitThreads), 0, stream>>>(a, x);
    else
        logprob_part_kernel<BF16, false><<<grid, dim3(kSplitThreads), 0, stream>>>(a, x);
    logprob_join_kernel<BF16><<<dim3(static_cast<unsigned>(a.t)), dim3(kMaxLists), 0, stream>>>(a, x);
    return hipGetLastError();
}

}  // namespace

long long logprob_work_bytes(int t, int V, int n_top) {
    // f32 rows are the longer ones: never fewer parts than bf16 rows
    return split_bytes(t, parts_of(t, V, 4), n_top);
}

hipError_t launch_logprobs(const LogprobArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace kda
