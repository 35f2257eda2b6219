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

// Where a part of a packed batch lies.  Sequence b takes the slots
// first / part_rows + b, ... (one for each part of part_rows rows), so parts of
// different sequences never share a slot and R / part_rows + B slots are enough.
struct Part {
    int b;        // sequence, -1: the slot is empty
    int index;    // part within the sequence
    int first;    // the sequence's rows
    int last;
};

// The sequence of a slot: the last one whose slots begin at or before it.  The
// table is read with a running maximum, clamped to [0, R], so that any table
// gives disjoint rows and slots; every wave runs this by itself.
__device__ __forceinline__ Part find_part(const PromptArgs& a, int part_rows, int slot) {
    const int lane = threadIdx.x & 63;
    Part f{-1, 0, 0, 0};
    int carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        int x = b < a.B ? min(max(a.offsets[b], 0), a.R) : a.R;
        x = max(x, carry);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int y = __shfl_up(x, d);
            if (lane >= d) x = max(x, y);
        }
        const uint64_t before = __ballot(b < a.B && x / part_rows + b <= slot);
        if (before == 0) break;
        const int n = __builtin_popcountll(before) - 1;
        f.b = b0 + n;
        f.first = __builtin_amdgcn_readlane(x, n);
        carry = __builtin_amdgcn_readlane(x, 63);
        if (n < 63) break;
    }
    if (f.b < 0) return f;
    f.b = __builtin_amdgcn_readfirstlane(f.b);
    f.index = slot - (f.first / part_rows + f.b);
    f.last = min(max(a.offsets[f.b + 1], f.first), a.R);
    if (f.first + static_cast<long long>(f.index) * part_rows >= f.last) f.b = -1;
    return f;
}

// Rows of sequence b under the same reading of the table.
__device__ __forceinline__ void sequence(const PromptArgs& a, int b, int& first, int& last) {
    int x = 0;
    for (int i = threadIdx.x & 63; i <= b; i += 64) x = max(x, min(max(a.offsets[i], 0), a.R));
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x = max(x, __shfl_xor(x, m));
    first = __builtin_amdgcn_readfirstlane(x);
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
// A workgroup (4 waves) owns a head and a part of a sequence; a wave owns 32
// value columns, its 128 x 32 piece of the state stays in 64 registers.  The
// state's accumulator layout is an operand layout as it stands, with the key
// channels of a 32-block in the order p(16 h + 4 g + r) = 8 g + 4 h + r; q and
// k are stored in LDS in that order.
//
// Long sequences run in parts of seg_rows rows, side by side: a first launch
// leaves each part's own state (from zero), a second chains them to the state
// each part starts from, and a third computes the outputs.

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using f32x4 = __attribute__((ext_vector_type(4))) float;

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

// Four rows x four channels of one thread, as they come from memory.
template <bool BF16>
struct Patch {
    uint4 r[BF16 ? 2 : 4];
};

template <bool BF16>
__device__ __forceinline__ void load_patch(Patch<BF16>& p, const void* src, long long row0, int rows,
                                           long long pitch, long long col) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long at = (row0 + i) * pitch + col;
        if constexpr (BF16) {
            uint2 x = make_uint2(0, 0);
            if (i < rows) x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(src) + at);
            if (i & 1) { p.r[i >> 1].z = x.x; p.r[i >> 1].w = x.y; }
            else       { p.r[i >> 1].x = x.x; p.r[i >> 1].y = x.y; }
        } else {
            p.r[i] = make_uint4(0, 0, 0, 0);
            if (i < rows) p.r[i] = *reinterpret_cast<const uint4*>(static_cast<const float*>(src) + at);
        }
    }
}

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
};

// By channel: word x of four rows of one plane.
template <int NS>
__device__ __forceinline__ void store_columns(uint16_t (&t)[NS][kD][kColPitch], int cg, int rg,
                                              const uint2 (&w)[4][NS]) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t sel = x & 1 ? 0x07060302u : 0x05040100u;
            uint2 y;
            y.x = __builtin_amdgcn_perm(x < 2 ? w[1][s].x : w[1][s].y, x < 2 ? w[0][s].x : w[0][s].y, sel);
            y.y = __builtin_amdgcn_perm(x < 2 ? w[3][s].x : w[3][s].y, x < 2 ? w[2][s].x : w[2][s].y, sel);
            *reinterpret_cast<uint2*>(&t[s][4 * cg + x][4 * rg]) = y;
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

// Parts of a call: slot s of head h has its state at states + (s * H + h) * 128 * 128
// and its summed log-decays at sums[s * H + h].
struct Parts {
    float* states;
    double* sums;
    int rows;    // of a part
};

// STATES: the part's own state, from zero, into its slot (all but a sequence's
// last part).  Otherwise the outputs, and from a sequence's last part its state.
template <bool BF16, bool STATES>
__global__ void __launch_bounds__(256, BF16 ? 2 : 1) linear_chunk_kernel(PromptArgs a, Parts parts) {
    constexpr int NS = BF16 ? 1 : 3;
    __shared__ __align__(16) LinearTile<NS> T;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
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

    f32x4 S[8][2];
    if constexpr (STATES) {
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c) S[m][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
        // the chained states lie one slot back; a first part's in the last slot
        const float* from = state;
        if (f.index > 0 || !last_part) {
            const int back = f.index > 0 ? slot - 1 : slot + (f.last - f.first - 1) / parts.rows;
            from = parts.states + (static_cast<long long>(back) * a.H + h) * kD * kD;
        }
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[m][c][r] = from[(16 * m + 4 * g4 + r) * kD + 32 * wave + 16 * c + l16];
        // the weights' upper block stays zero
        if (tid < 16)
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                *reinterpret_cast<uint4*>(&T.p[s][tid][16]) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(&T.p[s][tid][24]) = make_uint4(0, 0, 0, 0);
            }
    }

    const int rg = tid & 7, cg = tid >> 3;
    const long long kpitch = static_cast<long long>(a.Hk) * kD, vpitch = static_cast<long long>(a.H) * kD;
    Patch<BF16> pq, pk, pv;
    float pg = 0.f;
    const auto fetch = [&](int t0) {
        const int r0 = t0 + 4 * rg, n = end - r0;
        if (out) load_patch<BF16>(pq, a.q, r0, n, kpitch, hk * kD + 4 * cg);
        load_patch<BF16>(pk, a.k, r0, n, kpitch, hk * kD + 4 * cg);
        load_patch<BF16>(pv, a.v, r0, n, vpitch, h * kD + 4 * cg);
        if (tid < kChunk)
            pg = t0 + tid < end ? static_cast<const float*>(a.g)[static_cast<long long>(t0 + tid) * a.H + h] : 0.f;
    };
    fetch(begin);
    double sum = 0.0;

    for (int t0 = begin; t0 < end; t0 += kChunk) {
        __syncthreads();
        {
            uint2 w[4][NS];
            if (out) {
                patch_words<BF16>(pq, w);
                store_rows<NS>(T.q, cg, rg, w);
            }
            patch_words<BF16>(pk, w);
            if (out) store_rows<NS>(T.k, cg, rg, w);
            store_columns<NS>(T.kt, cg, rg, w);
            patch_words<BF16>(pv, w);
            store_columns<NS>(T.vt, cg, rg, w);
        }
        if (tid < 64) {
            double x = lane < kChunk ? fminf(fmaxf(pg, kGateOff), 0.f) : 0.f;
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
                    y[r] = j <= t ? x[r] * expf(static_cast<float>(Gt - T.G[j])) : 0.f;
                }
                uint2 w[3];
                split4(y, w);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    *reinterpret_cast<uint2*>(&T.p[s][t][16 * jb + 4 * g4]) = w[s];
            }
            f32x4 O[2][2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) O[c][tb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint4 sf[2][3];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const f32x4 lo = S[2 * ks][c], hi = S[2 * ks + 1][c];
                    const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    split8(x, sf[c]);
                }
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    uint4 qf[NS];
                    read_rows<NS>(T.q, 16 * tb + l16, 32 * ks + 8 * g4, qf);
#pragma unroll
                    for (int c = 0; c < 2; ++c) O[c][tb] = product<3, NS>(sf[c], qf, O[c][tb]);
                }
            }
            __syncthreads();
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const float e = T.eG[16 * tb + l16];
                uint4 pf[3];
                read_columns<3, kChunk>(T.p, 16 * tb + l16, 8 * g4, pf);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint4 vf[NS];
                    read_columns<NS, kD>(T.vt, 32 * wave + 16 * c + l16, 8 * g4, vf);
                    O[c][tb] *= e;
                    O[c][tb] = product<NS, 3>(vf, pf, O[c][tb]);
                    const int t = t0 + 16 * tb + l16;
                    if (t < end)
                        *reinterpret_cast<f32x4*>(a.o + (static_cast<long long>(t) * a.H + h) * kD +
                                                  32 * wave + 16 * c + 4 * g4) = O[c][tb] * kScale;
                }
            }
        }

        // the state: e^{G_C} S + k^T (weighted v)
        uint4 vw[2][3];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint4 vf[NS];
            read_columns<NS, kD>(T.vt, 32 * wave + 16 * c + l16, 8 * g4, vf);
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
            split8(x, vw[c]);
        }
        const float keep = T.eG[kChunk - 1];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            uint4 kf[NS];
            read_columns<NS, kD>(T.kt, 16 * m + l16, 8 * g4, kf);
#pragma unroll
            for (int c = 0; c < 2; ++c) S[m][c] = product<NS, 3>(kf, vw[c], S[m][c] * keep);
        }
    }

    if (STATES || last_part) {
        float* to = STATES ? parts.states + (static_cast<long long>(slot) * a.H + h) * kD * kD : state;
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    to[(16 * m + 4 * g4 + r) * kD + 32 * wave + 16 * c + l16] = S[m][c][r];
        if (STATES && tid == 0) parts.sums[static_cast<long long>(slot) * a.H + h] = sum;
    }
}

// Chains the parts of each (sequence, head): slot i gets the state that part
// i + 1 starts from, the last slot the one the sequence came with (its first
// part reads that copy, since the last part writes the state itself).
__global__ void __launch_bounds__(256) linear_chain_kernel(PromptArgs a, Parts parts) {
    const int h = blockIdx.x % a.H, b = blockIdx.x / a.H;
    int first, last;
    sequence(a, b, first, last);
    const float* state = a.s_ptrs[b];
    const int n = (last - first + parts.rows - 1) / parts.rows;
    if (state == nullptr || n < 2) return;
    const long long at = blockIdx.y * 256 + threadIdx.x;
    const long long slot0 = first / parts.rows + b;
    const long long step = static_cast<long long>(a.H) * kD * kD / 4;
    f32x4* p = reinterpret_cast<f32x4*>(parts.states) + slot0 * step + static_cast<long long>(h) * (kD * kD / 4) + at;
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
                e[u] = expf(static_cast<float>(parts.sums[(slot0 + i + u) * a.H + h]));
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < n - 1) {
                S = S * e[u] + x[u];
                p[(i + u) * step] = S;
            }
    }
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

// Rows of a part: 512, and more where the call has work for the chip without
// parts that short (each part but a sequence's last reads k and v twice).
static int part_rows(int R, int H) {
    int rows = 512;
    while (rows < 4096 && static_cast<long long>(R) * H > 1024ll * rows) rows *= 2;
    return rows;
}

static long long part_slots(int R, int B, int rows) { return R / rows + static_cast<long long>(B); }

long long linear_work_bytes(int R, int B, int H) {
    if (R <= 512) return 0;
    return part_slots(R, B, 512) * H * (kD * kD * 4ll + 8);
}

hipError_t launch_prompt(const PromptArgs& a, bool bf16, hipStream_t stream) {
    return launch_rows<false>(a, bf16, stream);
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
        parts.states = static_cast<float*>(a.work);
        parts.sums = reinterpret_cast<double*>(parts.states + blocks * kD * kD);
        linear_chunk_kernel<BF16, true><<<grid, dim3(256), 0, stream>>>(a, parts);
        const dim3 chain(static_cast<unsigned>(static_cast<long long>(a.B) * a.H), kD * kD / 4 / 256);
        linear_chain_kernel<<<chain, dim3(256), 0, stream>>>(a, parts);
    }
    linear_chunk_kernel<BF16, false><<<grid, dim3(256), 0, stream>>>(a, parts);
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
