// gfx950 kernels of the prompt and single-token operators: the KDA delta rule
// and linear attention with one decay for each head, over the same
// [H][128][128] f32 states as the verify scan.
//
// One row of one head (i = key channel, j = value channel):
//   KDA     S' = diag(exp(clamp(g, -5, 0))) S,  e = beta (v - S'^T k)
//   linear  S' = exp(min(g, 0)) S,              e = v
//   both    S  = S' + k e^T,  o = S^T q / sqrt(128)
//
// Prompts run in chunks of 32 rows, whose rows meet in matrix products.  On an
// MI355X, calls in a loop (the bytes that a call cannot do without, at the 4.69
// TB/s of a large copy, in brackets): KDA 4096 rows x 64 heads bf16 423 us (88),
// 8192 x 8 bf16 236 us (22), a ragged batch of 2,586 x 32 f32 162 us (52);
// linear 4096 x 64 bf16 155-164 us (74), 16384 x 8 f32 153-161 us (58); the
// single-token step over 34 x 15 x 64 states 836 us (919: it writes in place).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_launch.h"
#include "kda_ops.h"
#include "kda_seq.h"

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

// The sequence of a place in the order from long to short, so that the longest
// do not start last; beyond 64 sequences the place itself.
__device__ __forceinline__ int longest_first(const PromptArgs& a, int place) {
    if (a.B == 1 || a.B > 64) return place;
    const int lane = threadIdx.x & 63;
    const int first = running_max(lane < a.B ? min(max(a.offsets[lane], 0), a.R) : 0);
    const int last = lane < a.B ? min(max(a.offsets[lane + 1], first), a.R) : first;
    const int rows = lane < a.B ? last - first : -1;
    int rank = 0;
    for (int i = 0; i < a.B; ++i) {
        const int other = __builtin_amdgcn_readlane(rows, i);
        rank += other > rows || (other == rows && i < lane);
    }
    return __builtin_ctzll(__ballot(lane < a.B && rank == place));
}

// ------------------------------------------------------------------ linear attention, chunks
//
// Within a chunk of C = 32 rows, G_t = sum of log-decays up to and with row t:
//   O_t = [ e^{G_t} S_0^T q_t + sum_{j<=t} e^{G_t-G_j} (q_t.k_j) v_j ] / sqrt(128)
//   S_C = e^{G_C} S_0 + sum_j k_j (e^{G_C-G_j} v_j)^T
// Four matrix products on the bf16 matrix cores with f32 sums.  An operand that
// is not bf16 already is taken apart into three bf16 words whose sum is the f32
// value itself (24 bits = 3 x 8), so that every product keeps f32's precision:
// 3 products where one side is a bf16 input, 6 (all but those below 2^-24)
// where neither is.  G is summed in 64 bits: behind a row of strong decay a
// 32-bit running sum would lose the weak ones.
//
// A workgroup (8 waves) owns a head and a part of a sequence; a wave owns 16
// value columns, its 128 x 16 piece of the state stays in 32 registers.  The
// state's accumulator layout is an operand layout as it stands, with the key
// channels of a 32-block in the order p(16 h + 4 g + r) = 8 g + 4 h + r; q and
// k are stored in LDS in that order.
//
// Long sequences run in parts, side by side: a first launch leaves each part's
// own state (from zero), a second chains them to the state each part starts
// from, and a third computes the outputs.
//
// 4096 rows x 64 heads, bf16: states 43 us, chain 12, outputs 107 us (345 MB:
// 3.2 TB/s), bound by VALU (0.54: the state is taken apart for every chunk) and
// LDS (0.40, half of it bank conflicts: a half-wave's 8-byte writes of q and k by
// row lie on half of the banks) under two workgroups a CU; MFMA 0.27.

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float real(uint32_t x) { return __builtin_bit_cast(float, x); }

__device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// a . b over operands of NA and NB bf16 words each, the smallest products first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 product(const uint4 (&a)[NA], const uint4 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 2; i >= 0; --i)
            if (i < NA && s - i >= 0 && s - i < NB) c = mfma(a[i], b[s - i], c);
    return c;
}

// Two f32 values as three words of two bf16 each: x = w[0] + w[1] + w[2].
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& a, uint32_t& b, uint32_t& c) {
    a = __builtin_amdgcn_perm(bits(x1), bits(x0), 0x07060302u);
    const float y0 = x0 - real(bits(x0) & 0xFFFF0000u), y1 = x1 - real(bits(x1) & 0xFFFF0000u);
    b = __builtin_amdgcn_perm(bits(y1), bits(y0), 0x07060302u);
    const float z0 = y0 - real(bits(y0) & 0xFFFF0000u), z1 = y1 - real(bits(y1) & 0xFFFF0000u);
    c = __builtin_amdgcn_perm(bits(z1), bits(z0), 0x07060302u);
}

__device__ __forceinline__ void split4(const float (&x)[4], uint2 (&w)[3]) {
    split2(x[0], x[1], w[0].x, w[1].x, w[2].x);
    split2(x[2], x[3], w[0].y, w[1].y, w[2].y);
}

__device__ __forceinline__ void split8(const float (&x)[8], uint4 (&w)[3]) {
    split2(x[0], x[1], w[0].x, w[1].x, w[2].x);
    split2(x[2], x[3], w[0].y, w[1].y, w[2].y);
    split2(x[4], x[5], w[0].z, w[1].z, w[2].z);
    split2(x[6], x[7], w[0].w, w[1].w, w[2].w);
}

constexpr int kChunk = 32;
constexpr int kRowPitch = kD + 8;      // q and k by row: 16 rows of a 16-byte read on 64 banks
constexpr int kColPitch = kChunk + 8;  // k, v by channel and the chunk's weights: the same
constexpr float kGateOff = -104.0f;    // exp of it is 0 in f32

// min(g, 0), no lower than kGateOff; a NaN stays one.
__device__ __forceinline__ float log_decay(float g) { return g < kGateOff ? kGateOff : g > 0.f ? 0.f : g; }

// Up to 32 rows of one head as a buffer: reads past the last row give 0 and
// writes there are dropped, so that the row loops need no branches.
struct Rows {
    __amdgpu_buffer_rsrc_t buffer;
    int pitch;   // bytes from row to row
};

__device__ __forceinline__ Rows rows_of(const void* p, int es, long long row, int rows, int heads, int head) {
    const int pitch = heads * kD * es;
    char* at = static_cast<char*>(const_cast<void*>(p)) + row * pitch + static_cast<long long>(head) * kD * es;
    const int n = rows > 0 ? (min(rows, kChunk) - 1) * pitch + kD * es : 0;
    return Rows{__builtin_amdgcn_make_buffer_rsrc(at, 0, n, 0x00020000), pitch};
}

// Four rows x four channels of one thread, as they come from memory.
template <bool BF16>
struct Patch {
    uint4 r[BF16 ? 2 : 4];
};

template <bool BF16>
__device__ __forceinline__ void load_patch(Patch<BF16>& p, const Rows& x, int row, int col) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = (row + i) * x.pitch + col * (BF16 ? 2 : 4);
        if constexpr (BF16) {
            const uint2 y = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(x.buffer, at, 0, 0));
            if (i & 1) { p.r[i >> 1].z = y.x; p.r[i >> 1].w = y.y; }
            else       { p.r[i >> 1].x = y.x; p.r[i >> 1].y = y.y; }
        } else {
            p.r[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(x.buffer, at, 0, 0));
        }
    }
}

// One head's state as a buffer (one offset a lane, whatever the row).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t state_of(const float* s) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(s), 0, kD * kD * 4, 0x00020000);
}

// One element, raw; element() makes it a number.
template <bool BF16>
__device__ __forceinline__ uint32_t load_raw(const Rows& x, int row, int col) {
    if constexpr (BF16)
        return __builtin_amdgcn_raw_buffer_load_b16(x.buffer, row * x.pitch + col * 2, 0, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b32(x.buffer, row * x.pitch + col * 4, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ float element(uint32_t u) { return real(BF16 ? u << 16 : u); }

// The patch's four rows as bf16 words, plane by plane.
template <bool BF16>
__device__ __forceinline__ void patch_words(const Patch<BF16>& p, uint2 (&w)[4][BF16 ? 1 : 3]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const uint4 r = p.r[i >> 1];
            w[i][0] = i & 1 ? make_uint2(r.z, r.w) : make_uint2(r.x, r.y);
        } else {
            const float x[4] = {real(p.r[i].x), real(p.r[i].y), real(p.r[i].z), real(p.r[i].w)};
            split4(x, w[i]);
        }
    }
}

// True where one of the patch's values is a NaN or an infinity.
template <bool BF16>
__device__ __forceinline__ bool not_finite(const Patch<BF16>& p) {
    if constexpr (BF16) {
        using u16x2 = __attribute__((ext_vector_type(2))) uint16_t;
        u16x2 most{0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (const uint32_t u : {p.r[i].x, p.r[i].y, p.r[i].z, p.r[i].w})
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, u & 0x7FFF7FFFu));
        return max(most[0], most[1]) >= 0x7F80;
    } else {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            most = max(max(max(most, p.r[i].x & 0x7FFFFFFFu), max(p.r[i].y & 0x7FFFFFFFu, p.r[i].z & 0x7FFFFFFFu)),
                       p.r[i].w & 0x7FFFFFFFu);
        return most >= 0x7F800000u;
    }
}

template <int NS>
struct LinearTile {
    uint16_t q[NS][kChunk][kRowPitch];
    uint16_t k[NS][kChunk][kRowPitch];
    uint16_t kt[NS][kD][kColPitch];
    uint16_t vt[NS][kD][kColPitch];
    uint16_t p[3][kChunk][kColPitch];
    double G[kChunk];
    float eG[kChunk];   // e^{G_t}
    float w[kChunk];    // e^{G_C - G_t}
    __align__(16) uint32_t spoiled[4];   // v has a NaN or infinity: a flag of each wave that brings it
};

// By channel: word x of four rows of one plane.
template <int NS>
__device__ __forceinline__ void store_columns(uint16_t (&t)[NS][kD][kColPitch], int cg, int at,
                                              const uint2 (&w)[4][NS]) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t sel = x & 1 ? 0x07060302u : 0x05040100u;
            uint2 y;
            y.x = __builtin_amdgcn_perm(x < 2 ? w[1][s].x : w[1][s].y, x < 2 ? w[0][s].x : w[0][s].y, sel);
            y.y = __builtin_amdgcn_perm(x < 2 ? w[3][s].x : w[3][s].y, x < 2 ? w[2][s].x : w[2][s].y, sel);
            *reinterpret_cast<uint2*>(&t[s][4 * cg + x][at]) = y;
        }
    }
}

template <int NS>
__device__ __forceinline__ void store_rows(uint16_t (&t)[NS][kChunk][kRowPitch], int cg, int rg,
                                           const uint2 (&w)[4][NS]) {
    const int at = 32 * (cg >> 3) + 8 * (cg & 3) + 4 * ((cg >> 2) & 1);
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2*>(&t[s][4 * rg + i][at]) = w[i][s];
}

template <int NS>
__device__ __forceinline__ void read_rows(const uint16_t (&t)[NS][kChunk][kRowPitch], int row, int at,
                                          uint4 (&f)[NS]) {
#pragma unroll
    for (int s = 0; s < NS; ++s) f[s] = *reinterpret_cast<const uint4*>(&t[s][row][at]);
}

template <int NS, int ROWS>
__device__ __forceinline__ void read_columns(const uint16_t (&t)[NS][ROWS][kColPitch], int row, int at,
                                             uint4 (&f)[NS]) {
#pragma unroll
    for (int s = 0; s < NS; ++s) f[s] = *reinterpret_cast<const uint4*>(&t[s][row][at]);
}

// Eight rows (8 g4..) of a channel's values a lane: puts 0 in the place of what is
// not finite, and gives the first row of the chunk that has such a value.
template <int NS>
__device__ __forceinline__ int take_out(uint4 (&v)[NS]) {
    int first = kChunk;
    const int row = 8 * (threadIdx.x >> 4 & 3);
    const auto pair = [&](int i, auto part) {   // rows i and i + 1
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            const uint32_t mask = hi ? 0xFFFF0000u : 0xFFFFu;
            float x = 0.f;
#pragma unroll
            for (int s = NS - 1; s >= 0; --s) x += real(hi ? part(v[s]) & mask : part(v[s]) << 16);
            if (fabsf(x) < __builtin_inff()) continue;
            first = min(first, row + i + hi);
#pragma unroll
            for (int s = 0; s < NS; ++s) part(v[s]) &= ~mask;
        }
    };
    pair(0, [](uint4& u) -> uint32_t& { return u.x; });
    pair(2, [](uint4& u) -> uint32_t& { return u.y; });
    pair(4, [](uint4& u) -> uint32_t& { return u.z; });
    pair(6, [](uint4& u) -> uint32_t& { return u.w; });
    first = min(first, __shfl_xor(first, 16));
    return min(first, __shfl_xor(first, 32));
}

// Parts of a call: place s of head h has its state at states + (s * H + h) * 128 * 128
// and its summed log-decays at sums[s * H + h].  Only sequences of several parts
// take places, one for each part.  Of many short sequences few can be that long:
// they begin at twice the rows before them, in parts, which leaves each room for
// its own (ceil(x) <= floor(2 x) from one part on) and takes 2 R / rows places
// however many sequences there are.
struct Parts {
    float* states;
    double* sums;
    int rows;       // of a part
    bool twice;     // places by twice the rows, not by R / rows + B slots
    __device__ long long first_place(int b, int first) const {
        return twice ? 2 * first / rows : first / rows + b;   // first <= 2^28
    }
};

// STATES: the part's own state, from zero, into its slot (all but a sequence's
// last part).  Otherwise the outputs, and from a sequence's last part its state.
template <bool BF16, bool STATES>
__global__ void __launch_bounds__(512, BF16 ? 4 : 2) linear_chunk_kernel(PromptArgs a, Parts parts) {
    constexpr int NS = BF16 ? 1 : 3, es = BF16 ? 2 : 4;
    __shared__ __align__(16) LinearTile<NS> T;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int h = blockIdx.x % a.H, slot = blockIdx.x / a.H;
    const int hk = h / (a.H / a.Hk);
    const Part f = find_part(a, parts.rows, slot);
    if (f.b < 0) return;
    float* state = a.s_ptrs[f.b];
    if (state == nullptr) return;
    state += static_cast<long long>(h) * kD * kD;
    const int begin = f.first + f.index * parts.rows;
    const int end = min(f.last, begin + parts.rows);
    const bool last_part = end == f.last;
    const bool out = !STATES && a.o != nullptr;
    if (STATES ? last_part : !out && !last_part) return;

    const int col = 16 * wave + l16;
    f32x4 S[8];
    if constexpr (STATES) {
#pragma unroll
        for (int m = 0; m < 8; ++m) S[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
        // the chained states lie one place back; a first part's in the last place
        const float* from = state;
        if (f.index > 0 || !last_part) {
            const int back = f.index > 0 ? f.index - 1 : (f.last - f.first - 1) / parts.rows;
            from = parts.states + ((parts.first_place(f.b, f.first) + back) * a.H + h) * kD * kD;
        }
        const auto buffer = state_of(from);
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[m][r] = real(__builtin_amdgcn_raw_buffer_load_b32(buffer, (4 * g4 * kD + col) * 4, (16 * m + r) * kD * 4, 0));
        // the weights' upper block stays zero
        if (tid < 16)
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                *reinterpret_cast<uint4*>(&T.p[s][tid][16]) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(&T.p[s][tid][24]) = make_uint4(0, 0, 0, 0);
            }
    }

    // waves 0..3 bring k and g, 4..7 q and v
    const int x = tid & 255, rg = x & 7, cg = x >> 3;
    Patch<BF16> pa, pb;
    float pg = 0.f;
    const auto fetch = [&](int t0) {
        const int n = end - t0;
        if (wave < 4) {
            load_patch<BF16>(pa, rows_of(a.k, es, t0, n, a.Hk, hk), 4 * rg, 4 * cg);
            if (tid < kChunk)
                pg = t0 + tid < end ? static_cast<const float*>(a.g)[static_cast<long long>(t0 + tid) * a.H + h] : 0.f;
        } else {
            load_patch<BF16>(pa, rows_of(a.v, es, t0, n, a.H, h), 4 * rg, 4 * cg);
            if (out) load_patch<BF16>(pb, rows_of(a.q, es, t0, n, a.Hk, hk), 4 * rg, 4 * cg);
        }
    };
    fetch(begin);
    double sum = 0.0;

    for (int t0 = begin; t0 < end; t0 += kChunk) {
        __syncthreads();
        {
            uint2 w[4][NS];
            patch_words<BF16>(pa, w);
            if (wave < 4) {
                store_columns<NS>(T.kt, cg, 4 * rg, w);
                if (out) store_rows<NS>(T.k, cg, rg, w);
            } else {
                store_columns<NS>(T.vt, cg, 4 * rg, w);
                if (out) {
                    const uint64_t mask = __ballot(not_finite<BF16>(pa));
                    if (lane == 0) T.spoiled[wave - 4] = mask != 0;
                    patch_words<BF16>(pb, w);
                    store_rows<NS>(T.q, cg, rg, w);
                }
            }
        }
        if (wave == 0) {
            double x = lane < kChunk ? log_decay(pg) : 0.f;
#pragma unroll
            for (int d = 1; d < kChunk; d <<= 1) {
                const double y = __shfl_up(x, d);
                if (lane >= d) x += y;
            }
            const double all = __shfl(x, kChunk - 1);
            if (lane < kChunk) {
                T.G[lane] = x;
                T.eG[lane] = expf(static_cast<float>(x));
                T.w[lane] = expf(static_cast<float>(all - x));
            }
            sum += all;
        }
        if (t0 + kChunk < end) fetch(t0 + kChunk);
        __syncthreads();

        if (out) {
            // weights e^{G_t-G_j} q_t.k_j: three 16 x 16 blocks on or below the diagonal
            if (wave < 3) {
                const int jb = wave == 2, tb = wave > 0;
                f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    uint4 kf[NS], qf[NS];
                    read_rows<NS>(T.k, 16 * jb + l16, 32 * ks + 8 * g4, kf);
                    read_rows<NS>(T.q, 16 * tb + l16, 32 * ks + 8 * g4, qf);
                    x = product<NS, NS>(kf, qf, x);
                }
                const int t = 16 * tb + l16;
                const double Gt = T.G[t];
                float y[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * jb + 4 * g4 + r;
                    const float e = expf(static_cast<float>(fmin(Gt - T.G[j], 0.0)));
                    y[r] = j <= t ? x[r] * e : 0.f;
                }
                uint2 w[3];
                split4(y, w);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    *reinterpret_cast<uint2*>(&T.p[s][t][16 * jb + 4 * g4]) = w[s];
            }
            const Rows o = rows_of(a.o, 4, t0, end - t0, a.H, h);
            f32x4 O[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const f32x4 lo = S[2 * ks], hi = S[2 * ks + 1];
                const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                uint4 sf[3];
                split8(x, sf);
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    uint4 qf[NS];
                    read_rows<NS>(T.q, 16 * tb + l16, 32 * ks + 8 * g4, qf);
                    O[tb] = product<3, NS>(sf, qf, O[tb]);
                }
            }
            __syncthreads();
            uint4 vf[NS];
            read_columns<NS, kD>(T.vt, col, 8 * g4, vf);
            // a NaN or infinity in v would reach earlier rows through their weights
            // of 0: it is left out, and its channel's outputs from its row on are NaN
            const uint4 flags = *reinterpret_cast<const uint4*>(T.spoiled);
            const bool spoiled = __builtin_amdgcn_readfirstlane(flags.x | flags.y | flags.z | flags.w);
            int bad = kChunk;
            if (spoiled) bad = take_out<NS>(vf);
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const float e = T.eG[16 * tb + l16];
                uint4 pf[3];
                read_columns<3, kChunk>(T.p, 16 * tb + l16, 8 * g4, pf);
                O[tb] *= e;
                O[tb] = product<NS, 3>(vf, pf, O[tb]);
                f32x4 y = O[tb] * kScale;
                if (spoiled)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * tb + l16 >= __shfl(bad, 4 * g4 + r)) y[r] = __builtin_nanf("");
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), o.buffer,
                                                       (16 * tb + l16) * o.pitch + 4 * (16 * wave + 4 * g4), 0, 0);
            }
        }

        // the state: e^{G_C} S + k^T (weighted v)
        uint4 vw[3];
        {
            uint4 vf[NS];
            read_columns<NS, kD>(T.vt, col, 8 * g4, vf);
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v = 0.f;
#pragma unroll
                for (int s = NS - 1; s >= 0; --s) {
                    const uint32_t u = (i >> 1) == 0 ? vf[s].x : (i >> 1) == 1 ? vf[s].y : (i >> 1) == 2 ? vf[s].z : vf[s].w;
                    v += real(i & 1 ? u & 0xFFFF0000u : u << 16);
                }
                x[i] = v * T.w[8 * g4 + i];
            }
            split8(x, vw);
        }
        const float keep = T.eG[kChunk - 1];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            uint4 kf[NS];
            read_columns<NS, kD>(T.kt, 16 * m + l16, 8 * g4, kf);
            S[m] = product<NS, 3>(kf, vw, S[m] * keep);
        }
    }

    if (STATES || last_part) {
        const long long at = (parts.first_place(f.b, f.first) + f.index) * a.H + h;
        float* to = STATES ? parts.states + at * kD * kD : state;
        const auto buffer = state_of(to);
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                __builtin_amdgcn_raw_buffer_store_b32(bits(S[m][r]), buffer, (4 * g4 * kD + col) * 4, (16 * m + r) * kD * 4, 0);
        if (STATES && tid == 0) parts.sums[at] = sum;
    }
}

// Chains the parts of each (sequence, head): place i gets the state that part
// i + 1 starts from, the last place the one the sequence came with (its first
// part reads that copy, since the last part writes the state itself).
__global__ void __launch_bounds__(256) linear_chain_kernel(PromptArgs a, Parts parts) {
    const int h = blockIdx.x % a.H, b = blockIdx.x / a.H;
    int first, last;
    sequence(a, b, first, last);
    const float* state = a.s_ptrs[b];
    const int n = (last - first + parts.rows - 1) / parts.rows;
    if (state == nullptr || n < 2) return;
    const long long at = blockIdx.y * 256 + threadIdx.x;
    const long long place0 = parts.first_place(b, first);
    const long long step = static_cast<long long>(a.H) * kD * kD / 4;
    f32x4* p = reinterpret_cast<f32x4*>(parts.states) + place0 * step + static_cast<long long>(h) * (kD * kD / 4) + at;
    f32x4 S = reinterpret_cast<const f32x4*>(state + static_cast<long long>(h) * kD * kD)[at];
    p[(n - 1) * step] = S;
    constexpr int U = 4;
    for (int i = 0; i < n - 1; i += U) {
        f32x4 x[U];
        float e[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < n - 1) {
                x[u] = p[(i + u) * step];
                e[u] = expf(static_cast<float>(parts.sums[(place0 + i + u) * a.H + h]));
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < n - 1) {
                S = S * e[u] + x[u];
                p[(i + u) * step] = S;
            }
    }
}

// ------------------------------------------------------------------ KDA, chunks
//
// Within a chunk of 32 rows, G_t[c] = sum of the clamped gates of channel c up
// to and with row t, and
//   A_tj = sum_c k_t[c] k_j[c] e^{G_t[c]-G_j[c]}   (j < t)
//   B_tj = sum_c q_t[c] k_j[c] e^{G_t[c]-G_j[c]}   (j <= t)
// the rows' deltas e solve a triangular system, and the chunk is
//   E   = (I + diag(beta) A)^-1 diag(beta) (V - (k e^G) S_0)  =  M (V - (k e^G) S_0)
//   O   = [ (q e^G) S_0 + B E ] / sqrt(128)
//   S_C = diag(e^{G_C}) S_0 + (k e^{G_C-G})^T E
// Nothing but S_0 ties one chunk to the next: a first launch prepares all chunks
// side by side (M, B, k e^G, q e^G, k e^{G_C-G}, e^{G_C}), and a second walks the
// chunks of each sequence, where only the products are left.
//
// 4096 rows x 64 heads, bf16: prepare 165-185 us, 670 MB read and written at
// 3.6-4.0 TB/s (a copy: 4.69) beside 0.56 VALU and 0.37 LDS; the walk 255-265 us,
// 2.0 us a chunk, bound by the dependent chain of a chunk (MFMA 0.28, of which
// the f32 sums over rows are half; VALU 0.35).

using f16x8 = __attribute__((ext_vector_type(8))) _Float16;
using f16x2 = __attribute__((ext_vector_type(2))) _Float16;
using f32x2 = __attribute__((ext_vector_type(2))) float;

constexpr int kSub = 16;                        // rows of a block of A and B

// One chunk of one head, ready for the products: 16-byte operands of 64 lanes,
// the contracted index in the order of an accumulator.  k, q and kt are two f16
// words each of a value scaled by its row's power of two; M and B, whose rows
// meet values of any size, are f32 (in the same room).
struct KdaBlock {
    uint4 k[2][4][2][64];    // k e^G: 16-row block, 32-channel block, word, lane
    uint4 q[2][4][2][64];    // q e^G
    uint4 kt[8][2][64];      // k e^{G_C-G}: 16-channel block, word, lane
    float4 m[2][2][64];      // M: 16-row block, 16-column block, lane (the upper one is zero)
    float4 b[2][2][64];      // B
    float keep[kD];          // e^{G_C}
    float ki[kChunk], qi[kChunk], ti[kChunk];   // what undoes the rows' scales of k, q and kt
    float unused[32];
};
static_assert(sizeof(KdaBlock) == 57 * 1024, "whole kilobytes");

// A power of two that brings m into [2^13, 2^14): the largest f16 word then
// keeps 22 bits in two words, and what falls below f16's range is under 2^-38
// of the largest.  (Held to 2^126: values under 2^-126 keep fewer bits, as in f32.)
__device__ __forceinline__ float scale_of(float m) {
    const int e = static_cast<int>(bits(m) >> 23 & 0xFF);
    const int x = min(13 + 127 + 127 - e, 127 + 126);
    return real(static_cast<uint32_t>(max(x, 1)) << 23);
}

// 1 / s of a power of two from scale_of.
__device__ __forceinline__ float inverse_of(float s) { return real(0x7F000000u - bits(s)); }

// x0 s0 and x1 s1 as two words of two f16 each (22 bits).  The products are
// formed inside the two roundings: the second word holds what the first left of
// the exact product.
__device__ __forceinline__ void halves2(float x0, float s0, float x1, float s1, uint32_t& a, uint32_t& b) {
    const f16x2 h{static_cast<_Float16>(fmaf(x0, s0, 0.f)), static_cast<_Float16>(fmaf(x1, s1, 0.f))};
    const f16x2 l{static_cast<_Float16>(fmaf(x0, s0, -static_cast<float>(h[0]))),
                  static_cast<_Float16>(fmaf(x1, s1, -static_cast<float>(h[1])))};
    a = __builtin_bit_cast(uint32_t, h);
    b = __builtin_bit_cast(uint32_t, l);
}

__device__ __forceinline__ void halves4(const float (&x)[4], const float (&s)[4], uint2 (&w)[2]) {
    halves2(x[0], s[0], x[1], s[1], w[0].x, w[1].x);
    halves2(x[2], s[2], x[3], s[3], w[0].y, w[1].y);
}

__device__ __forceinline__ void halves8(const f32x4& lo, const f32x4& hi, float s, uint4 (&w)[2]) {
    halves2(lo[0], s, lo[1], s, w[0].x, w[1].x);
    halves2(lo[2], s, lo[3], s, w[0].y, w[1].y);
    halves2(hi[0], s, hi[1], s, w[0].z, w[1].z);
    halves2(hi[2], s, hi[3], s, w[0].w, w[1].w);
}

__device__ __forceinline__ float abs_max(float a, float b, float c) {
    return fmaxf(fmaxf(fabsf(a), fabsf(b)), c);
}

__device__ __forceinline__ float abs_max(const f32x4& x, float c) {
    return abs_max(x[0], x[1], abs_max(x[2], x[3], c));
}

// a . b over two f16 words each: all products but low x low (under 2^-22).
__device__ __forceinline__ f32x4 product16(const uint4 (&a)[2], const uint4 (&b)[2], f32x4 c) {
    const auto m = [](uint4 x, uint4 y, f32x4 z) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                      __builtin_bit_cast(f16x8, y), z, 0, 0, 0);
    };
    c = m(a[1], b[0], c);
    c = m(a[0], b[1], c);
    return m(a[0], b[0], c);
}

template <bool BF16>
__device__ __forceinline__ void patch_values(const Patch<BF16>& p, float (&x)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const uint4 r = p.r[i >> 1];
            const uint32_t u = i & 1 ? r.z : r.x, v = i & 1 ? r.w : r.y;
            x[i][0] = real(u << 16);
            x[i][1] = real(u & 0xFFFF0000u);
            x[i][2] = real(v << 16);
            x[i][3] = real(v & 0xFFFF0000u);
        } else {
            x[i][0] = real(p.r[i].x);
            x[i][1] = real(p.r[i].y);
            x[i][2] = real(p.r[i].z);
            x[i][3] = real(p.r[i].w);
        }
    }
}

// e^clamp(g): the rounding of g log2(e) is carried over to the result.
__device__ __forceinline__ float decay(float g) {
    constexpr float log2e = 1.44269504088896340736f, ln2 = 0.693147180559945309417f;
    g = fminf(fmaxf(g, kGateLow), 0.f);
    const float x = g * log2e;
    const float y = __builtin_amdgcn_exp2f(x);
    return fmaf(y, fmaf(g, log2e, -x) * ln2, y);
}

// Eight consecutive elements of a row.
template <bool BF16>
struct Eight {
    uint4 r[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ void load_eight(Eight<BF16>& p, const Rows& x, int row, int col) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i)
        p.r[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                               x.buffer, row * x.pitch + col * (BF16 ? 2 : 4) + 16 * i, 0, 0));
}

template <bool BF16>
__device__ __forceinline__ void eight_values(const Eight<BF16>& p, float (&x)[8]) {
    if constexpr (BF16) {
        const uint32_t w[4] = {p.r[0].x, p.r[0].y, p.r[0].z, p.r[0].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = real(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    } else {
        const uint32_t w[8] = {p.r[0].x, p.r[0].y, p.r[0].z, p.r[0].w, p.r[1].x, p.r[1].y, p.r[1].z, p.r[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = real(w[i]);
    }
}

// max over the four lanes that share a column.  (Written as asm: the swap
// builtins return the first register for both results.  The s_nop covers the
// wait states between a VALU write and a swap that reads it.)
__device__ __forceinline__ float column_max(float x) {
    float y = x;
    asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
    x = abs_max(x, y, 0.f);
    y = x;
    asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
    return abs_max(x, y, 0.f);
}

// x of the lane N before (or behind) this one, 0 where there is none in its row of 16.
template <int CTRL>
__device__ __forceinline__ float neighbour(float x) {
    return real(__builtin_amdgcn_update_dpp(0, bits(x), CTRL, 0xF, 0xF, true));
}
template <int N> __device__ __forceinline__ float lane_before(float x) { return neighbour<0x110 + N>(x); }
template <int N> __device__ __forceinline__ float lane_behind(float x) { return neighbour<0x100 + N>(x); }

// max over the eight lanes whose number is the same modulo 8.
__device__ __forceinline__ float eighth_max(float x) {
    return column_max(abs_max(x, neighbour<0x128>(x), 0.f));   // row_ror:8
}

// The rows of a chunk that a NaN or infinity is in: from first on in k or beta,
// after which nothing of the state is left, and a bit for each row of q.
struct Spoiled {
    int first;
    uint32_t queries;
};

// Rows of a patch, one bit each, that have a NaN or infinity.
template <bool BF16>
__device__ __forceinline__ uint32_t spoiled_rows(const Patch<BF16>& p) {
    float x[4][4];
    patch_values<BF16>(p, x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (!(fabsf(x[i][c]) < __builtin_inff())) m |= 1u << i;
    return m;
}

template <bool BF16>
__device__ __forceinline__ void clear_rows(Patch<BF16>& p, uint32_t rows) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!(rows >> i & 1)) continue;
        if constexpr (BF16) {
            if (i & 1) p.r[i >> 1].z = p.r[i >> 1].w = 0;
            else       p.r[i >> 1].x = p.r[i >> 1].y = 0;
        } else {
            p.r[i] = make_uint4(0, 0, 0, 0);
        }
    }
}

// Prepares one chunk of one head.
//
// e^{G_t-G_j} does not split into a factor of t and one of j over the chunk's
// whole range (e^{-5 * 32} leaves f32), so A and B are three blocks of 16 x 16:
// with f = e^{G - G_mid}, G_mid at the middle of a 16-row block, every factor
// stays within e^{-40}..e^{40}; the block below the diagonal takes the decay
// between the two middles with its rows.  The factors are running products of
// the rows' decays, which do not lose the weak gates behind strong ones as
// differences of sums would.
template <bool BF16>
__global__ void __launch_bounds__(256) kda_prepare_kernel(PromptArgs a, KdaBlock* blocks, int slot0) {
    struct Factors {
        float f[kChunk][kD + 4];      // e^{G-G_mid}
        float inverse[kChunk][kD + 4];
        float between[kD];
    };
    __shared__ __align__(16) union {
        Factors f;
        uint4 words[16 * 64];   // k, q or kt of the block, in turn
    } U;
    __shared__ float A[kChunk][kChunk + 1], B[kChunk][kChunk + 1], T[kChunk][kChunk + 1];
    __shared__ float beta[kChunk];
    __shared__ __align__(16) float top[3][4][kChunk];   // by wave: the rows' largest k e^G, q e^G, k e^{G_C-G}
    __shared__ __align__(16) uint32_t spoiled[4];
    __shared__ Spoiled rows_lost;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int h = blockIdx.x % a.H, slot = slot0 + blockIdx.x / a.H;
    const Part f = find_part(a, kChunk, slot);
    if (f.b < 0 || a.s_ptrs[f.b] == nullptr) return;
    const int t0 = f.first + f.index * kChunk;
    const int n = min(f.last - t0, kChunk);
    constexpr int es = BF16 ? 2 : 4;

    // a thread has 4 rows x 4 channels, 8 neighbouring lanes a channel's 32 rows
    const int rg = tid & 7, cg = tid >> 3;
    const Rows rk = rows_of(a.k, es, t0, n, a.H, h), rq = rows_of(a.q, es, t0, n, a.H, h);
    Patch<BF16> pg, pk, pq;
    load_patch<BF16>(pg, rows_of(a.g, es, t0, n, a.H, h), 4 * rg, 4 * cg);
    // waves 0, 1: the diagonal blocks; 2 and 3: A and B below it
    const int tb = wave != 0, jb = wave == 1;
    const bool low = wave >= 2, wantA = wave != 3, wantB = wave != 2;
    const int tr = 16 * tb + l16, jr = 16 * jb + l16;
    // (f32 rows are read one step ahead of their use: all at once they would take
    // 96 registers, and with them a third workgroup from the CU: 87 us against 74
    // for the ragged batch of 2,586 rows x 32 heads)
    Eight<BF16> ek[4], et[4], eq[4];
    const auto rows = [&](int ks) {
        load_eight<BF16>(ek[ks], rk, jr, 32 * ks + 8 * g4);
        if (low && wantA) load_eight<BF16>(et[ks], rk, tr, 32 * ks + 8 * g4);
        if (wantB) load_eight<BF16>(eq[ks], rq, tr, 32 * ks + 8 * g4);
    };
#pragma unroll
    for (int ks = 0; ks < (BF16 ? 4 : 1); ++ks) rows(ks);
    bool spoils = false;   // a NaN or infinity in the thread's part of the rows
    if (tid < kChunk) {
        const float x = tid < n ? load<BF16>(a.beta, static_cast<long long>(t0 + tid) * a.H + h) : 0.f;
        beta[tid] = x;
        spoils = !(fabsf(x) < __builtin_inff());
    }

    float pre[4][4], suf[4][4], keep[4];   // e^{G_t} and e^{G_C-G_t} of the thread's elements
    {
        float d[4][4];
        patch_values<BF16>(pg, d);
        const bool late = rg & 2;   // behind the middle of its block
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i][c] = decay(d[i][c]);
            pre[0][c] = d[0][c];
#pragma unroll
            for (int i = 1; i < 4; ++i) pre[i][c] = pre[i - 1][c] * d[i][c];
            suf[3][c] = 1.f;
#pragma unroll
            for (int i = 2; i >= 0; --i) suf[i][c] = suf[i + 1][c] * d[i + 1][c];
            const float all = pre[3][c];
            const float near = real(__builtin_amdgcn_update_dpp(0, bits(all), 0xB1, 0xF, 0xF, true));   // lane ^ 1
            // a late row's f is the product from the middle to it; an early row's
            // 1/f the product of what lies between it and the middle
            const float beyond = late == static_cast<bool>(rg & 1) ? near : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = (late ? pre[i][c] : suf[i][c]) * beyond;
                const float r = __builtin_amdgcn_rcpf(y);
                U.f.f[4 * rg + i][4 * cg + c] = late ? y : r;
                U.f.inverse[4 * rg + i][4 * cg + c] = late ? r : y;
            }
            // between the middles: row groups 2, 3 and 4, 5
            const float pair = all * near, next = lane_behind<2>(pair);
            if (rg == 2) U.f.between[4 * cg + c] = pair * next;
            // products over the row groups before and behind this one
            float up = all, down = all;
            float y = lane_before<1>(up), z = lane_behind<1>(down);
            up *= rg >= 1 ? y : 1.f;
            down *= rg < 7 ? z : 1.f;
            y = lane_before<2>(up), z = lane_behind<2>(down);
            up *= rg >= 2 ? y : 1.f;
            down *= rg < 6 ? z : 1.f;
            y = lane_before<4>(up), z = lane_behind<4>(down);
            up *= rg >= 4 ? y : 1.f;
            down *= rg < 4 ? z : 1.f;
            y = lane_before<1>(up), z = lane_behind<1>(down);
            keep[c] = up;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pre[i][c] *= rg >= 1 ? y : 1.f;
                suf[i][c] *= rg < 7 ? z : 1.f;
            }
        }
    }
    __syncthreads();

    // (f32 products: these operands would take three bf16 words and six
    // products, and taking them apart costs more than the matrix cores gain)
    f32x4 xa{0.f, 0.f, 0.f, 0.f}, xb{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
        const int c = 32 * ks + 8 * g4;
        float x[8], kj[8], ft[8];
        if (!BF16 && ks < 3) rows(ks + 1);
        eight_values<BF16>(ek[ks], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            kj[i] = x[i] * U.f.inverse[jr][c + i];
            ft[i] = U.f.f[tr][c + i];
        }
        if (low)
#pragma unroll
            for (int i = 0; i < 8; ++i) ft[i] *= U.f.between[c + i];
        if (wantA) {
            if (low) eight_values<BF16>(et[ks], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) xa = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i] * ft[i], kj[i], xa, 0, 0, 0);
        }
        if (wantB) {
            eight_values<BF16>(eq[ks], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) xb = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i] * ft[i], kj[i], xb, 0, 0, 0);
        }
    }
    load_patch<BF16>(pk, rk, 4 * rg, 4 * cg);
    load_patch<BF16>(pq, rq, 4 * rg, 4 * cg);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = 16 * tb + 4 * g4 + r, j = 16 * jb + l16;
        if (wantA) A[t][j] = j < t ? -beta[t] * xa[r] : 0.f;
        if (wantB) B[t][j] = j <= t ? xb[r] : 0.f;
        if (low) (wantA ? A : B)[l16][16 + 4 * g4 + r] = 0.f;
    }
    // Each row is scaled by its largest value with the decay in it: late rows
    // of a chunk can be e^{-5 * 32} of early ones, and where little is added to
    // a decaying state they are all that the state's products have.
    {
        float x[4][4], most[3][4];
        const auto largest = [&](const float (&f)[4][4], float (&m)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m[i] = eighth_max(abs_max(x[i][0] * f[i][0], x[i][1] * f[i][1], abs_max(x[i][2] * f[i][2], x[i][3] * f[i][3], 0.f)));
        };
        spoils = spoils || not_finite<BF16>(pk) || not_finite<BF16>(pq);
        const uint64_t mask = __ballot(spoils);
        if (lane == 0) spoiled[wave] = mask != 0;
        if (tid == 0) rows_lost = Spoiled{kChunk, 0};
        patch_values<BF16>(pk, x);
        largest(pre, most[0]);
        largest(suf, most[2]);
        patch_values<BF16>(pq, x);
        largest(pre, most[1]);
        if (lane < 8)
#pragma unroll
            for (int o = 0; o < 3; ++o)
                *reinterpret_cast<float4*>(&top[o][wave][4 * rg]) = make_float4(most[o][0], most[o][1], most[o][2], most[o][3]);
    }
    __syncthreads();

    // A row with a NaN or infinity would reach the rows before it through the zeros
    // above the diagonals.  Such a row of q, and all rows from the first of k or
    // beta on, are left out, and NaN comes back by their rows of B and, behind k
    // and beta, by the state's decay.
    Spoiled lost{kChunk, 0};
    const uint4 flags = *reinterpret_cast<const uint4*>(spoiled);
    if (__builtin_amdgcn_readfirstlane(flags.x | flags.y | flags.z | flags.w)) {
        uint32_t m = spoiled_rows<BF16>(pk);
        if (m) atomicMin(&rows_lost.first, 4 * rg + __builtin_ctz(m));
        if (tid < kChunk && !(fabsf(beta[tid]) < __builtin_inff())) atomicMin(&rows_lost.first, tid);
        m = spoiled_rows<BF16>(pq);
        if (m) atomicOr(&rows_lost.queries, m << 4 * rg);
        __syncthreads();
        lost = rows_lost;
        for (int i = tid; i < kChunk * kChunk; i += 256)
            if (i / kChunk >= lost.first) A[i / kChunk][i % kChunk] = 0.f;
        if (tid < kChunk && tid >= lost.first) beta[tid] = 0.f;
        clear_rows<BF16>(pk, 15u << min(max(lost.first - 4 * rg, 0), 4));
        clear_rows<BF16>(pq, lost.queries >> 4 * rg & 15);
        if (lost.first < kChunk)
#pragma unroll
            for (int c = 0; c < 4; ++c) keep[c] = __builtin_nanf("");
        __syncthreads();
    }

    // T = (I - A)^-1: the diagonal blocks column by column by the first wave ...
    if (tid < kChunk) {
        const int o = tid & 16, c = tid & 15;
        float x[kSub];
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            float s = t == c ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < t; ++j) s = fmaf(A[o + t][o + j], x[j], s);
            x[t] = s;
            T[o + t][o + c] = s;
        }
    }
    // ... and beside it the operands; the factors' memory is free
    KdaBlock& out = blocks[blockIdx.x];
    float sc[3][4];   // of the thread's rows
#pragma unroll
    for (int o = 0; o < 3; ++o) {
        f32x4 m[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) m[w] = *reinterpret_cast<const f32x4*>(&top[o][w][4 * rg]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[o][i] = scale_of(fmaxf(fmaxf(m[0][i], m[1][i]), fmaxf(m[2][i], m[3][i])));
        if (cg == 0)
            *reinterpret_cast<float4*>(&(o == 0 ? out.ki : o == 1 ? out.qi : out.ti)[4 * rg]) =
                make_float4(inverse_of(sc[o][0]), inverse_of(sc[o][1]), inverse_of(sc[o][2]), inverse_of(sc[o][3]));
    }
    if (rg == 7) *reinterpret_cast<float4*>(&out.keep[4 * cg]) = make_float4(keep[0], keep[1], keep[2], keep[3]);
    {
        float x[4][4];
        uint2 w[4][2];
        // (16-byte piece p of an operand lies at p ^ its lane group, so that the
        // writes of a wave spread over the banks)
        uint2* const to = reinterpret_cast<uint2*>(U.words);
        const int at = (cg >> 3) * 2 * 128 + (cg & 3) * 32 + (cg >> 2 & 1);   // channel part of a row operand
        const auto by_row = [&](const float (&sc)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) y[c] = pre[i][c] * sc[i];
                halves4(x[i], y, w[i]);
                const int t = 4 * rg + i;
#pragma unroll
                for (int s = 0; s < 2; ++s) to[(t >> 4) * 8 * 128 + s * 128 + at + 2 * ((t & 15) ^ (cg & 3))] = w[i][s];
            }
        };
        const auto copy = [&](uint4* to) {
#pragma unroll
            for (int i = 0; i < 4; ++i) to[256 * i + tid] = U.words[256 * i + (tid ^ g4)];
        };
        patch_values<BF16>(pq, x);
        by_row(sc[1]);
        __syncthreads();
        copy(&out.q[0][0][0][0]);
        __syncthreads();
        patch_values<BF16>(pk, x);
        by_row(sc[0]);
        __syncthreads();
        copy(&out.k[0][0][0][0]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = suf[i][c] * sc[2][i];
            halves4(x[i], y, w[i]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
                uint2 y;
                y.x = __builtin_amdgcn_perm(c < 2 ? w[1][s].x : w[1][s].y, c < 2 ? w[0][s].x : w[0][s].y, sel);
                y.y = __builtin_amdgcn_perm(c < 2 ? w[3][s].x : w[3][s].y, c < 2 ? w[2][s].x : w[2][s].y, sel);
                to[((cg >> 2) * 2 + s) * 128 + (rg & 3) * 32 + 2 * ((4 * (cg & 3) + c) ^ (rg & 3)) + (rg >> 2)] = y;
            }
        __syncthreads();
        copy(&out.kt[0][0][0]);
        // the block of T below the diagonal
        const int t = tid >> 4, j = tid & 15;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kSub; ++i) s = fmaf(A[16 + t][i], T[i][j], s);
        A[t][16 + j] = s;    // the upper block is free
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int i = 0; i < kSub; ++i) s = fmaf(T[16 + t][16 + i], A[i][16 + j], s);
        T[16 + t][j] = s;
        T[t][16 + j] = 0.f;
    }
    __syncthreads();

    const int t = tid >> 3, x = tid & 7;
    float m[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = T[t][4 * x + i] * beta[4 * x + i];
        b[i] = B[t][4 * x + i];
        if (t >= lost.first || lost.queries >> t & 1) b[i] = __builtin_nanf("");
    }
    const int at = 16 * (x & 3) + (t & 15);
    out.m[t >> 4][x >> 2][at] = make_float4(m[0], m[1], m[2], m[3]);
    out.b[t >> 4][x >> 2][at] = make_float4(b[0], b[1], b[2], b[3]);
}

// The chunks in slots slot0 .. slot1-1 of one sequence and head, 32 value columns.
//
// What ties the chunks together, S_0 -> R = V - (k e^G) S_0 -> E = M R -> S_C, is
// done by waves 0..3 and nothing else: wave 2 * half + c has columns 16 c.. and
// key channels 64 half.. of the state in 16 registers, and the two halves of a
// column block exchange their parts of R through LDS.  Waves 4..7 follow them:
// they bring the next chunk's operands and values from memory to LDS, and form
// the outputs of 16 rows x 16 columns each from the state's words and the
// deltas that waves 0..3 leave in LDS, one barrier behind.
//
// The products with the state and into it, 128 channels long, take two f16 words
// of a value scaled by a power of two (3 products, 22 bits; bf16 words would take
// six): the state by the largest of a column's 64 keys, k, q and kt by their
// row's, with the decays inside.  A sum over channels so keeps its precision
// however far the rows have decayed; what loses bits is a value under 2^-16 of
// the largest in its own row or column.  M R and B E sum over rows, which can be
// of any size against each other (a row that nothing is added to, behind one
// that was): f32 products.  For the sum of kt E over rows the deltas take the
// scales of kt's rows with them before they are scaled by column.
//
// Few sequences and heads leave most of the chip idle, and their chunks wait for
// each other.  Then a sequence runs in parts side by side: a part's end state is
// linear in the state it starts from, T S_0 + U, with T the end state from the
// identity without values, and U that from zero.  STATES leaves both (the
// slices behind the first four are T's columns); kda_chain_kernel chains them
// to the state that each part starts from; then the parts are walked again.
constexpr int kKdaCols = 32;
constexpr int kWhole = 1 << 30;   // rows of a part where sequences are not divided

// Slot s of head h: U, and later the next part's first state, at states +
// (s * H + h) * 128 * 128; T at moves likewise.
struct KdaParts {
    float* states;
    float* moves;
    int rows;
};

template <bool BF16, bool OUT, bool STATES>
__global__ void __launch_bounds__(512) kda_chunk_kernel(PromptArgs a, const KdaBlock* blocks, int slot0, int slot1,
                                                        KdaParts parts, int units) {
    static_assert(!(OUT && STATES), "a part's own states have no outputs");
    __shared__ __align__(16) KdaBlock tiles[2];
    __shared__ f32x4 xr[4][2][64];          // parts of R
    __shared__ f32x4 xv[2][2][64];          // V: column block, row block
    __shared__ uint4 sw[2][2][2][2][64];    // the state: column block, half, 32 channels, word
    __shared__ f32x4 ew[2][2][64];          // the deltas: column block, row block
    __shared__ float si[2][2][64];          // what undoes the state's scales
    __shared__ int from_row[2][64];         // the row from which a column's outputs are NaN
    constexpr int slices = kD / kKdaCols * (STATES ? 2 : 1), es = BF16 ? 2 : 4;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    // workgroups go round 8 XCDs: the slices of a head to one of them, whose L2
    // then has the operands that they share
    const int turn = blockIdx.x / (8 * slices), within = blockIdx.x % (8 * slices);
    const int unit = 8 * turn + (within & 7), slice = within >> 3 & 3;
    const bool move = STATES && within >> 3 > 3;
    if (unit >= units) return;
    const int h = unit % a.H;
    const int place = unit / a.H;
    Part f{0, 0, 0, 0};
    if (parts.rows == kWhole) {
        f.b = longest_first(a, place);
        sequence(a, f.b, f.first, f.last);
    } else {
        f = find_part(a, parts.rows, place);
        if (f.b < 0) return;
    }
    const int first = f.first, last = f.last;
    const int own = first / kChunk + f.b, chunks = (last - first + kChunk - 1) / kChunk;
    const int part_begin = f.index * (parts.rows / kChunk), part_end = min(part_begin + parts.rows / kChunk, chunks);
    const bool last_part = part_end == chunks;
    const int begin = max(slot0 - own, part_begin), end = min(slot1 - own, part_end);
    float* state = a.s_ptrs[f.b];
    if (state == nullptr || begin >= end) return;
    if (STATES ? last_part : !OUT && !last_part) return;
    state += static_cast<long long>(h) * kD * kD;
    const long long head = static_cast<long long>(kD) * kD;
    blocks += static_cast<long long>(own - slot0) * a.H + h;
    // the chained states lie one slot back; a first part's in the last slot
    const float* from = state;
    float* to = state;
    if (STATES) {
        to = (move ? parts.moves : parts.states) + unit * head;
    } else if (f.index > 0) {
        from = parts.states + (unit - a.H) * head;
    } else if (!last_part) {
        from = parts.states + (unit + static_cast<long long>((last - first - 1) / parts.rows) * a.H) * head;
    }
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};

    if (wave >= 4) {
        const int c = wave & 1, tb = (wave >> 1) & 1, x = tid - 256;
        const int col = kKdaCols * slice + 16 * c + l16;
        constexpr int pieces = sizeof(KdaBlock) / 4096, rest = sizeof(KdaBlock) % 4096 / 16;
        u32x4 next[pieces + 1];
        uint32_t v[4];
        const auto fetch = [&](int i) {
            const auto from = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<KdaBlock*>(blocks + static_cast<long long>(i) * a.H), 0, sizeof(KdaBlock), 0x00020000);
#pragma unroll
            for (int j = 0; j <= pieces; ++j)
                next[j] = __builtin_amdgcn_raw_buffer_load_b128(from, 16 * x, 4096 * j, 0);
            const int t0 = first + i * kChunk;
            const Rows rv = rows_of(a.v, es, t0, last - t0, a.H, h);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = move ? 0 : load_raw<BF16>(rv, 16 * tb + 4 * g4 + r, col);
        };
        const auto store = [&](KdaBlock& T) {
            u32x4* to = reinterpret_cast<u32x4*>(&T) + x;
#pragma unroll
            for (int j = 0; j < pieces; ++j) to[256 * j] = next[j];
            if (x < rest) to[256 * pieces] = next[pieces];
            xv[c][tb][lane] = f32x4{element<BF16>(v[0]), element<BF16>(v[1]), element<BF16>(v[2]), element<BF16>(v[3])};
        };
        fetch(begin);
        store(tiles[0]);
        if (begin + 1 < end) fetch(begin + 1);
        f32x4 Q = zero, bf[2] = {zero, zero};
        for (int i = begin; i <= end; ++i) {
            const KdaBlock& T = tiles[(i - begin) & 1];
            __syncthreads();
            // the chunk before: its deltas are there now
            f32x4 E[2] = {zero, zero};
            int bad = kChunk;
            if (OUT && i > begin) {
                bad = from_row[c][lane];
                E[0] = ew[c][0][lane];
                if (tb) E[1] = ew[c][1][lane];
            }
            uint4 qf[4][2], sf[4][2];
            float s0 = 0.f, s1 = 0.f;
            if (OUT && i < end) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        qf[ks][w] = T.q[tb][ks][w][lane];
                        sf[ks][w] = sw[c][ks >> 1][ks & 1][w][lane];
                    }
                s0 = si[c][0][lane];
                s1 = si[c][1][lane];
            }
            if (i < end) __syncthreads();
            if (OUT && i > begin) {
                f32x4 y = zero, z = zero;
#pragma unroll
                for (int r = 0; r < 4; ++r) y = __builtin_amdgcn_mfma_f32_16x16x4f32(bf[0][r], E[0][r], y, 0, 0, 0);
                if (tb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) z = __builtin_amdgcn_mfma_f32_16x16x4f32(bf[1][r], E[1][r], z, 0, 0, 0);
                y += z;
                const int t0 = first + (i - 1) * kChunk;
                const Rows ro = rows_of(a.o, 4, t0, last - t0, a.H, h);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * tb + 4 * g4 + r;
                    const float o = t < bad ? (y[r] + Q[r]) * kScale : __builtin_nanf("");
                    __builtin_amdgcn_raw_buffer_store_b32(bits(o), ro.buffer, t * ro.pitch + 4 * col, 0, 0);
                }
            }
            if (i == end) break;
            if (i + 1 < end) {
                store(tiles[(i + 1 - begin) & 1]);
                if (i + 2 < end) fetch(i + 2);
            }
            if (OUT) {
                f32x4 q0 = zero, q1 = zero;
                const f32x4 qi = *reinterpret_cast<const f32x4*>(&T.qi[16 * tb + 4 * g4]);
#pragma unroll
                for (int j = 0; j < 2; ++j) bf[j] = __builtin_bit_cast(f32x4, T.b[tb][j][lane]);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    q0 = product16(qf[ks], sf[ks], q0);
                    q1 = product16(qf[2 + ks], sf[2 + ks], q1);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) Q[r] = fmaf(q0[r], s0, q1[r] * s1) * qi[r];
            }
        }
        return;
    }

    const int half = wave >> 1, c = wave & 1, col = kKdaCols * slice + 16 * c + l16;
    f32x4 S[4];
    float smax = 0.f;
    const int at = ((64 * half + 4 * g4) * kD + col) * 4;
    {
        const auto buffer = state_of(from);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (STATES)
                    S[m][r] = move && 64 * half + 16 * m + 4 * g4 + r == col ? 1.f : 0.f;
                else
                    S[m][r] = real(__builtin_amdgcn_raw_buffer_load_b32(buffer, at, (16 * m + r) * kD * 4, 0));
            }
            smax = abs_max(S[m], smax);
        }
    }
    for (int i = begin; i < end; ++i) {
        const KdaBlock& T = tiles[(i - begin) & 1];
        const float ss = scale_of(column_max(smax)), s1 = inverse_of(ss);
        uint4 sf[2][2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            halves8(S[2 * ks], S[2 * ks + 1], ss, sf[ks]);
            if (OUT)
#pragma unroll
                for (int w = 0; w < 2; ++w) sw[c][half][ks][w][lane] = sf[ks][w];
        }
        if (OUT) si[c][half][lane] = s1;
        // The chain of products goes before the outputs' on the matrix cores that
        // they share, and the switches keep the reads from sinking into it: the walk
        // of 4096 rows x 64 heads 270 us under the profiler, 313 without them.
        __builtin_amdgcn_s_setprio(0);
        __syncthreads();
        __builtin_amdgcn_s_setprio(3);
        uint4 kf[2][2][2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
#pragma unroll
                for (int w = 0; w < 2; ++w) kf[ks][tb][w] = T.k[tb][2 * half + ks][w][lane];
        f32x4 R[2] = {zero, zero}, V[2] = {zero, zero};
        float z = 0.f;    // NaN if V has a NaN or infinity
        if (half == 0)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) V[tb] = xv[c][tb][lane];
        f32x4 ki[2], ti[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            ki[tb] = *reinterpret_cast<const f32x4*>(&T.ki[16 * tb + 4 * g4]);
            ti[tb] = *reinterpret_cast<const f32x4*>(&T.ti[16 * tb + 4 * g4]);
        }
        const f32x4 m00 = __builtin_bit_cast(f32x4, T.m[0][0][lane]), m10 = __builtin_bit_cast(f32x4, T.m[1][0][lane]),
                    m11 = __builtin_bit_cast(f32x4, T.m[1][1][lane]);
        __builtin_amdgcn_sched_barrier(0);   // all reads before the products that wait for the first of them
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) R[tb] = product16(kf[ks][tb], sf[ks], R[tb]);
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
            for (int r = 0; r < 4; ++r) z = fmaf(V[tb][r], 0.f, z);
#pragma unroll
            for (int r = 0; r < 4; ++r) R[tb][r] = fmaf(R[tb][r] * ki[tb][r], -s1, V[tb][r]);
            xr[wave][tb][lane] = R[tb];
        }
        __builtin_amdgcn_s_setprio(0);
        uint4 tf[4][2];
        f32x4 keep[4];
        __syncthreads();
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) R[tb] += xr[wave ^ 2][tb][lane];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int w = 0; w < 2; ++w) tf[m][w] = T.kt[4 * half + m][w][lane];
            keep[m] = *reinterpret_cast<const f32x4*>(&T.keep[64 * half + 16 * m + 4 * g4]);
        }
        __builtin_amdgcn_s_setprio(3);
        f32x4 E[2];    // the deltas
        const auto deltas = [&] {
            f32x4 x = zero;
            E[0] = E[1] = zero;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                E[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(m00[r], R[0][r], E[0], 0, 0, 0);
                E[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(m10[r], R[0][r], E[1], 0, 0, 0);
                x = __builtin_amdgcn_mfma_f32_16x16x4f32(m11[r], R[1][r], x, 0, 0, 0);
            }
            E[1] += x;
        };
        // A NaN or infinity in v has to reach the state, but not the deltas of earlier
        // rows, which it meets with M's zeros: those go to the outputs without it.
        if (OUT && half == 0) {
            int first = kChunk;
            if (__ballot(z != z)) {
                const f32x4 keep_R[2] = {R[0], R[1]};
#pragma unroll
                for (int tb = 0; tb < 2; ++tb)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!(fabsf(V[tb][r]) < __builtin_inff())) {
                            first = min(first, 16 * tb + 4 * g4 + r);
                            R[tb][r] = 0.f;
                        }
                first = min(first, __shfl_xor(first, 16));
                first = min(first, __shfl_xor(first, 32));
                deltas();
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    ew[c][tb][lane] = E[tb];
                    R[tb] = keep_R[tb];
                }
                deltas();
            } else {
                deltas();
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) ew[c][tb][lane] = E[tb];
            }
            from_row[c][lane] = first;
        } else {
            deltas();
        }
        float emax = 0.f;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            E[tb] *= ti[tb];
            emax = abs_max(E[tb], emax);
        }
        const float se = scale_of(column_max(emax)), ei = inverse_of(se);
        uint4 ef[2];
        halves8(E[0], E[1], se, ef);
        smax = 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 y = product16(tf[m], ef, zero);
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] = fmaf(y[r], ei, S[m][r] * keep[m][r]);
            smax = abs_max(S[m], smax);
        }
    }
    __syncthreads();
    if (!STATES && !last_part) return;
    const auto buffer = state_of(to);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            __builtin_amdgcn_raw_buffer_store_b32(bits(S[m][r]), buffer, at, (16 * m + r) * kD * 4, 0);
}

// Chains the parts of each (sequence, head): S <- T_i S + U_i, into slot i (the
// state that part i + 1 starts from); the last slot gets the state the sequence
// came with, for its first part.  A workgroup has 16 value columns, a wave 32
// rows of the product (f32 matrix products), and the rows meet in LDS.
__global__ void __launch_bounds__(256) kda_chain_kernel(PromptArgs a, KdaParts parts) {
    __shared__ f32x4 rows[2][8][64];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int h = blockIdx.x % a.H, b = blockIdx.x / a.H, col = 16 * blockIdx.y + l16;
    int first, last;
    sequence(a, b, first, last);
    const float* state = a.s_ptrs[b];
    const int n = (last - first + parts.rows - 1) / parts.rows;
    if (state == nullptr || n < 2) return;
    const long long step = static_cast<long long>(a.H) * kD * kD;
    const long long slot = (static_cast<long long>(first / parts.rows + b) * a.H + h) * kD * kD;
    float* states = parts.states + slot;
    const float* moves = parts.moves + slot;
    state += static_cast<long long>(h) * kD * kD;

    f32x4 S[8];
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[m][r] = state[(16 * m + 4 * g4 + r) * kD + col];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            states[(n - 1) * step + (32 * wave + 16 * m + 4 * g4 + r) * kD + col] =
                state[(32 * wave + 16 * m + 4 * g4 + r) * kD + col];
    f32x4 T[2][8], U[2];
    const auto fetch = [&](int i) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                T[m][k] = *reinterpret_cast<const f32x4*>(moves + i * step + (32 * wave + 16 * m + l16) * kD + 16 * k + 4 * g4);
#pragma unroll
            for (int r = 0; r < 4; ++r) U[m][r] = states[i * step + (32 * wave + 16 * m + 4 * g4 + r) * kD + col];
        }
    };
    fetch(0);
    for (int i = 0; i < n - 1; ++i) {
        f32x4 X[2] = {U[0], U[1]};
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int m = 0; m < 2; ++m) X[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(T[m][k][r], S[k][r], X[m], 0, 0, 0);
        if (i + 1 < n - 1) fetch(i + 1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            rows[i & 1][2 * wave + m][lane] = X[m];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                states[i * step + (32 * wave + 16 * m + 4 * g4 + r) * kD + col] = X[m][r];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) S[k] = rows[i & 1][k][lane];
    }
}

// ------------------------------------------------------------------ single token
//
// A workgroup owns one (layer, session, head): the head's 64 KiB state is read
// once and written once, 16 bytes a lane, all 16 loads of a lane in flight
// before the first use.  HBM-bound: 34 x 15 x 64 states, 4.31 GB in 837 us (5.15
// TB/s).
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
    const float d = expf(log_decay(a.g[r]));
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


// Rows of a part: 512, and more where the call has work for the chip without
// parts that short (each part but a sequence's last reads k and v twice).
static int part_rows(int R, int H) {
    int rows = 512;
    while (rows < 4096 && static_cast<long long>(R) * H > 1024ll * rows) rows *= 2;
    return rows;
}

static long long part_slots(int R, int B, int rows) { return R / rows + static_cast<long long>(B); }

// Places of part states: R / rows + B, or 2 R / rows if that is less.
static bool places_twice(int R, int B, int rows) { return B > R / rows; }

static long long part_places(int R, int B, int rows) {
    return places_twice(R, B, rows) ? 2ll * R / rows : part_slots(R, B, rows);
}

// For calls of up to R, B and H, whose parts can be of any size from 512 rows on:
// parts under 4096 rows have R * H / rows <= 1024, and there are at most twice as
// many places.
long long linear_work_bytes(int R, int B, int H) {
    if (R <= 512) return 0;
    const long long longest = static_cast<long long>(R) * H / 2048, shortest = part_places(R, B, 512) * H;
    const long long places = longest > 2048 ? longest : 2048;
    return (places < shortest ? places : shortest) * (kD * kD * 4ll + 8);
}

// The prepared chunks of a call, or of as many slots as fit kWorkCap: longer
// calls go through the workspace in turns.  Before them the parts' states.
constexpr long long kWorkCap = 2ll << 30;
constexpr int kFewHeads = 16, kPartRows = 512, kPartFill = 64;
constexpr long long kPartBytes = 2ll * (kPartFill + kFewHeads) * kD * kD * 4;

// Rows of a part.  Up to 16 (sequence, head) pairs of four workgroups each leave
// three CUs of four idle; parts of R * H / 64 rows give each of 256 CUs a
// workgroup of the outputs' walk, and two in turn of the walk for U and T, one of
// which fills a CU's LDS.  (The counts are a whole MI355X's and not the current
// device's: the workspace follows from R, B and H alone.)
// In parts every chunk but those of a sequence's last part is walked three times
// (U, T, outputs), so it takes four parts to gain: the three walks and the chain
// of 8192 rows x 8 heads 197 us in 8 parts when first measured, against 399 in one
// piece; 2048 x 32 would be 125 in 2 against 109.
static int kda_part_rows(int R, int B, int H) {
    if (static_cast<long long>(B) * H > kFewHeads || R < 4 * kPartRows) return kWhole;
    const long long rows = (static_cast<long long>(R) * H / kPartFill + kChunk - 1) / kChunk * kChunk;
    return static_cast<int>(rows > kPartRows ? rows : kPartRows);
}

static long long parts_bytes(int R) { return R < 4 * kPartRows ? 0 : kPartBytes; }

static long long blocks_bytes(int R, int B, int H) {
    const long long row = static_cast<long long>(H) * sizeof(KdaBlock), all = part_slots(R, B, kChunk) * row;
    const long long most = kWorkCap > row ? kWorkCap : row;
    return all < most ? all : most;
}

long long prompt_work_bytes(int R, int B, int H) { return R == 0 ? 0 : parts_bytes(R) + blocks_bytes(R, B, H); }

template <bool BF16>
static hipError_t launch_kda(const PromptArgs& a, hipStream_t stream) {
    const long long slots = part_slots(a.R, a.B, kChunk);
    const long long turn = blocks_bytes(a.R, a.B, a.H) / (static_cast<long long>(a.H) * sizeof(KdaBlock));
    KdaParts parts{};
    parts.rows = turn < slots ? kWhole : kda_part_rows(a.R, a.B, a.H);
    parts.states = static_cast<float*>(a.work);
    const int units = static_cast<int>(part_slots(a.R, a.B, parts.rows) * a.H);   // at most 80 in parts
    parts.moves = parts.states + static_cast<long long>(units) * kD * kD;
    KdaBlock* const blocks = reinterpret_cast<KdaBlock*>(static_cast<char*>(a.work) + parts_bytes(a.R));
    const auto grid = [&](int slices) { return dim3(static_cast<unsigned>((units + 7) / 8 * 8 * slices)); };
    constexpr int slices = kD / kKdaCols;
    for (long long s0 = 0; s0 < slots; s0 += turn) {
        const int slot0 = static_cast<int>(s0), slot1 = static_cast<int>(s0 + turn < slots ? s0 + turn : slots);
        kda_prepare_kernel<BF16><<<dim3(static_cast<unsigned>((slot1 - slot0) * static_cast<long long>(a.H))),
                                   dim3(256), 0, stream>>>(a, blocks, slot0);
        if (parts.rows != kWhole) {
            kda_chunk_kernel<BF16, false, true><<<grid(2 * slices), dim3(512), 0, stream>>>(a, blocks, slot0, slot1, parts, units);
            const dim3 chain(static_cast<unsigned>(a.B * a.H), 8);
            kda_chain_kernel<<<chain, dim3(256), 0, stream>>>(a, parts);
        }
        if (a.o)
            kda_chunk_kernel<BF16, true, false><<<grid(slices), dim3(512), 0, stream>>>(a, blocks, slot0, slot1, parts, units);
        else
            kda_chunk_kernel<BF16, false, false><<<grid(slices), dim3(512), 0, stream>>>(a, blocks, slot0, slot1, parts, units);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_prompt(const PromptArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch_kda<true>(a, stream) : launch_kda<false>(a, stream);
}

template <bool BF16>
static hipError_t launch_linear(const PromptArgs& a, hipStream_t stream) {
    Parts parts{};
    parts.rows = part_rows(a.R, a.H);
    const long long slots = part_slots(a.R, a.B, parts.rows);
    const long long blocks = slots * a.H;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (a.R > parts.rows) {   // a sequence may have several parts
        parts.twice = places_twice(a.R, a.B, parts.rows);
        parts.states = static_cast<float*>(a.work);
        parts.sums = reinterpret_cast<double*>(parts.states + part_places(a.R, a.B, parts.rows) * a.H * kD * kD);
        linear_chunk_kernel<BF16, true><<<grid, dim3(512), 0, stream>>>(a, parts);
        const dim3 chain(static_cast<unsigned>(static_cast<long long>(a.B) * a.H), kD * kD / 4 / 256);
        linear_chain_kernel<<<chain, dim3(256), 0, stream>>>(a, parts);
    }
    linear_chunk_kernel<BF16, false><<<grid, dim3(512), 0, stream>>>(a, parts);
    return hipGetLastError();
}

hipError_t launch_linear_prompt(const PromptArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch_linear<true>(a, stream) : launch_linear<false>(a, stream);
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
