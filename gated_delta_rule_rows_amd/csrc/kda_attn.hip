// gfx950 kernels of the paged cache: the rows that are written to it, and the
// attention of new rows over it.
//
// Query row i of a sequence, at position p, and head h, with x_j = scale q . k_j:
//   o = sum_j e^{x_j - m} v_j / sum_j e^{x_j - m},   m = max_j x_j,
// over the keys j that the row sees: j <= p, its page there, and with a window
// j > p - window or j < sinks.  One pass over the keys, in tiles: O, the sum l
// and the maximum m are carried, and moved to a new maximum when one comes.
//
// The query heads of a key head and the rows of a sequence are the columns of
// one product: a tile of columns (32, or 128 of four waves) reads each key and
// value once for all of them.  A wave owns 32 columns.  It computes S^T = K Q^T,
// whose accumulators hold a column a lane, so that the softmax needs one
// exchange between the lane's two halves; the same registers are the operand of
// O^T += V^T P^T, with the keys of a step in the order in which the accumulators
// hold them.
//
// Where the tiles of columns are too few to fill the chip, the keys of a tile
// are split over workgroups, which leave O, m and l in the workspace for a
// second launch.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_cache.h"
#include "kda_launch.h"
#include "kda_seq.h"

namespace kda {
namespace {

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using s16x4 = __attribute__((ext_vector_type(4))) short;
using f32x16 = __attribute__((ext_vector_type(16))) float;

constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;        // the carried maximum may lag by this much (base 2)
constexpr int kColumns = 32;          // columns of a wave
constexpr int kTargetNarrow = 1024;   // workgroups that fill the chip: one wave each
constexpr int kTargetWide = 512;      // four waves each
constexpr int kLeastTiles = 4;        // a split has this many tiles at least
constexpr int kSplitKeys = 256;       // a cache of no more keys a sequence is never split
constexpr int kAppendThreads = 256;
constexpr int kJoinThreads = 256;

// ------------------------------------------------------------------ append

// A workgroup takes `rows` rows of one sequence; a thread moves 16 bytes of a
// key and a value at a time.
template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a, int rows) {
    constexpr int ES = BF16 ? 2 : 4, PIECES = kD * ES / 16;
    const Part f = find_part(a, rows, blockIdx.x);
    if (f.b < 0) return;
    const int begin = f.first + f.index * rows, n = min(rows, f.last - begin) * a.Hk * PIECES;
    const int len = a.c.lens[f.b];
    const int32_t* table = a.c.table + static_cast<long long>(f.b) * a.c.seq_pages;
    for (int i = threadIdx.x; i < n; i += kAppendThreads) {
        const int piece = i % PIECES, head = i / PIECES % a.Hk, row = begin + i / PIECES / a.Hk;
        const int pos = cache_pos(len, row, f.last), page = pos >> a.c.page_shift;
        if (pos < 0 || page >= a.c.seq_pages) continue;
        const long long at = cache_at(a.c, table[page], pos);
        if (at < 0) continue;
        const int in = head * kD * ES + piece * 16;
        const long long to = (at + head * a.c.head_stride) * ES + piece * 16;
        const uint4 k = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + row * a.k_ld * ES + in);
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + row * a.v_ld * ES + in);
        *reinterpret_cast<uint4*>(static_cast<char*>(a.c.k) + to) = k;
        *reinterpret_cast<uint4*>(static_cast<char*>(a.c.v) + to) = v;
    }
}

// ------------------------------------------------------------------ attention

// How a call is divided.
struct Plan {
    int cols;        // columns of a tile: 32 or 128
    int groups;      // parts of a key head's query heads (1 unless they are more than cols)
    int heads;       // query heads of a part
    int rows;        // rows of a tile
    int slots;       // tiles of columns, at most
    int parts;       // workgroups a (key head, part) that the keys are split for; 0: not split
};

__host__ __device__ inline int div_up(int a, int b) { return (a + b - 1) / b; }

Plan plan_of(int R, int B, int H, int Hk, bool wide) {
    Plan p{};
    const int G = H / Hk;
    p.cols = wide ? 4 * kColumns : kColumns;
    p.groups = div_up(G, p.cols);
    p.heads = div_up(G, p.groups);
    p.rows = p.cols / p.heads;
    p.slots = R / p.rows + B;
    const long long n = static_cast<long long>(p.slots) * Hk * p.groups;
    const int target = wide ? kTargetWide : kTargetNarrow;
    p.parts = n < target ? div_up(target, Hk * p.groups) : 0;
    return p;
}

// What a workgroup does: columns (rows from `row` on of sequence b), keys [t0, t1) of its tiles.
struct Item {
    int b;           // -1: nothing
    int row;         // first row of the tile of columns
    int last;        // end of the sequence's rows
    int split;
    int splits;
    int index;       // of the tile within the sequence
    int first;       // first row of the sequence
};

// The items of all sequences, one after the other: (tile of columns, split).
// Every wave runs it by itself; B < 64 * 64.
__device__ __forceinline__ Item find_item(const AttnArgs& a, const Plan& p, int kt, int item) {
    const int lane = threadIdx.x & 63;
    const int capacity = a.c.seq_pages << a.c.page_shift;
    const int each = div_up(a.B, 64), from = min(lane * each, a.B), to = min(from + each, a.B);
    const auto row = [&](int b) { return min(max(a.offsets[b], 0), a.R); };
    int most = 0;
    for (int b = from; b < to; ++b) most = max(most, row(b));
    int before = __shfl_up(running_max(most), 1);
    if (lane == 0) before = 0;
    // tiles of columns and of keys of sequence b, whose rows are first .. last-1
    const auto tiles = [&](int b, int first, int last, int& across, int& along) {
        across = div_up(last - first, p.rows);
        along = 0;
        if (across == 0) return;
        const int hi = cache_pos(a.c.lens[b], last - 1, last);
        along = key_tiles(max(hi - p.rows + 1, hi - (last - first) + 1), hi, capacity, a.window, a.sinks, kt).count;
    };
    long long units = 0;
    int run = before;
    for (int b = from; b < to; ++b) {
        const int first = max(run, row(b)), last = min(max(a.offsets[b + 1], first), a.R);
        run = first;
        int across, along;
        tiles(b, first, last, across, along);
        units += static_cast<long long>(across) * along;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) units += __shfl_xor(units, d);
    const int unit = max(kLeastTiles, static_cast<int>(min((units + p.parts - 1) / p.parts, 1ll << 30)));
    int mine = 0;
    run = before;
    for (int b = from; b < to; ++b) {
        const int first = max(run, row(b)), last = min(max(a.offsets[b + 1], first), a.R);
        run = first;
        int across, along;
        tiles(b, first, last, across, along);
        mine += across * max(1, div_up(along, unit));
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(upto, d);
        if (lane >= d) upto += y;
    }
    Item f{-1, 0, 0, 0, 1, 0, 0};
    const uint64_t mask = __ballot(item >= upto - mine && item < upto);
    if (mask == 0) return f;
    const int owner = __builtin_ctzll(mask);
    int base = upto - mine;
    run = before;
    for (int b = from; b < to; ++b) {
        const int first = max(run, row(b)), last = min(max(a.offsets[b + 1], first), a.R);
        run = first;
        int across, along;
        tiles(b, first, last, across, along);
        const int splits = max(1, div_up(along, unit));
        if (item >= base && item < base + across * splits) {
            f.b = b;
            f.first = first;
            f.index = (item - base) / splits;
            f.last = last;
            f.split = (item - base) % splits;
            f.splits = splits;
        }
        base += across * splits;
    }
    f.b = __builtin_amdgcn_readlane(f.b, owner);
    f.first = __builtin_amdgcn_readlane(f.first, owner);
    f.index = __builtin_amdgcn_readlane(f.index, owner);
    f.row = f.first + f.index * p.rows;
    f.last = __builtin_amdgcn_readlane(f.last, owner);
    f.split = __builtin_amdgcn_readlane(f.split, owner);
    f.splits = __builtin_amdgcn_readlane(f.splits, owner);
    return f;
}

// The tile of keys.
template <bool BF16, int WAVES>
struct Shape {
    static constexpr int kEs = BF16 ? 2 : 4;
    static constexpr int kKeys = BF16 && WAVES == 4 ? 64 : 32;
    static constexpr int kBlocks = kKeys / 32;
    static constexpr int kPieces = kD * kEs / 16;              // 16-byte pieces of a row
    // Pitches of the rows in LDS.  K: 16 rows of a 16-byte read lie on all banks.  V: four rows of 64
    // bytes (bf16), or rows 4 apart of 128 bytes (f32).
    static constexpr int kPitchK = kD * kEs + 16;
    static constexpr int kPitchV = kD * kEs + (BF16 ? 64 : 32);
    static constexpr int kTile = kKeys * (kPitchK + kPitchV);  // K, then V
    static constexpr int kThreads = WAVES * 64;
    static constexpr int kRowsAtOnce = kThreads / kPieces;     // rows that a load of all threads covers
    static constexpr int kLoads = kKeys / kRowsAtOnce;         // 16-byte loads a thread, for K and for V
};

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float real(uint32_t x) { return __builtin_bit_cast(float, x); }

// The two bf16 nearest to a and b (ties to even).
__device__ __forceinline__ uint32_t pack(float a, float b) {
    using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// x of this lane and of the lane 32 away.
__device__ __forceinline__ void halves(float x, float& a, float& b) {
    const auto p = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    a = real(p[0]);
    b = real(p[1]);
}

__device__ __forceinline__ f32x16 mfma(uint4 a, uint4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mfma(float a, float b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

// Four keys of the lane's channel, from V by row (transposed on the way): lane i of 16 brings piece
// i & 3 of row i >> 2, of 4 channels, and gets channel i.
__device__ __forceinline__ uint2 four_keys(const char* at) {
    using Lds = __attribute__((address_space(3))) s16x4;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)at));
}

// The workspace: for each tile of columns its first item and its splits, then
// for each item, head part and column m (base 2) and l, and O not divided by l.
// A tile's place is that of its rows among all packed parts (find_part).
struct Partials {
    int2* tiles;
    float2* ml;
    float* o;

    __host__ __device__ Partials(void* work, const Plan& p, int n_heads) {
        const long long all = static_cast<long long>(p.parts + p.slots) * n_heads * p.cols;
        o = static_cast<float*>(work);
        ml = reinterpret_cast<float2*>(o + all * kD);
        tiles = reinterpret_cast<int2*>(ml + all);
    }
};

// Makes what is not finite 0, and says in a bit a channel where that was.
template <bool BF16>
__device__ __forceinline__ uint32_t part_finite(uint4& u) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w}, bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const bool lo = (w[i] & 0x7F80u) == 0x7F80u, hi = (w[i] & 0x7F800000u) == 0x7F800000u;
            bad |= (lo ? 1u : 0u) << 2 * i | (hi ? 2u : 0u) << 2 * i;
            w[i] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
        } else {
            const bool all = (w[i] & 0x7F800000u) == 0x7F800000u;
            bad |= (all ? 1u : 0u) << i;
            w[i] = all ? 0u : w[i];
        }
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
    return bad;
}

// O^T += V^T P^T over a tile; v: the lane's place in its V.  P is rounded to bf16 for a bf16 cache, by
// half a step of 2^-8 at most; l sums it unrounded.
template <bool BF16, int NB, int PITCH>
__device__ __forceinline__ void add_values(f32x16 (&acc)[4], const f32x16 (&s)[NB], const char* v) {
    if constexpr (BF16) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int step = 0; step < 2; ++step) {
                const auto p = [&](int i) { return pack(s[b][8 * step + i], s[b][8 * step + i + 1]); };
                const uint4 w = make_uint4(p(0), p(2), p(4), p(6));
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const char* at = v + (32 * b + 16 * step) * PITCH + 64 * d;
                    const uint2 x = four_keys(at), y = four_keys(at + 8 * PITCH);
                    acc[d] = mfma(make_uint4(x.x, x.y, y.x, y.y), w, acc[d]);
                }
            }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                acc[d] = mfma(*reinterpret_cast<const float*>(v + (8 * (r >> 2) + (r & 3)) * PITCH + 128 * d), s[0][r], acc[d]);
    }
}

// Where a lane reads V: bf16, by four_keys, rows 4 half + (i >> 2), channels 16 (lane >> 4 & 1) + 4 (i & 3)
// on; f32, row 4 half, channel col.
template <bool BF16, int PITCH>
__device__ __forceinline__ int value_place() {
    const int lane = threadIdx.x & 63, i = lane & 15;
    if constexpr (BF16) return (4 * (lane >> 5) + (i >> 2)) * PITCH + 32 * (lane >> 4 & 1) + 8 * (i & 3);
    return 4 * (lane >> 5) * PITCH + 4 * (lane & 31);
}

template <bool BF16, int WAVES, bool SPLIT>
__global__ void __launch_bounds__(WAVES * 64, WAVES == 4 ? 2 : 1) attn_kernel(AttnArgs a, Plan p) {
    using Sh = Shape<BF16, WAVES>;
    constexpr int KT = Sh::kKeys, ES = Sh::kEs, NB = Sh::kBlocks, PIECES = Sh::kPieces, LOADS = Sh::kLoads;
    constexpr int NQ = BF16 ? 8 : 16;   // 16-byte pieces of q a lane
    constexpr int PK = Sh::kPitchK, PV = Sh::kPitchV;
    __shared__ __align__(16) char tiles[2][Sh::kTile];
    __shared__ uint32_t spoiled[2][WAVES];          // whether a row of V that the wave brought is in odd
    __shared__ uint8_t odd[2][KT * PIECES];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5, col = lane & 31;
    const int n_heads = a.Hk * p.groups;
    const int hd = blockIdx.x % n_heads, place = blockIdx.x / n_heads;
    Item f;
    if constexpr (SPLIT) {
        f = find_item(a, p, KT, place);
    } else {
        const Part part = find_part(a, p.rows, place);
        f = Item{part.b, part.first + part.index * p.rows, part.last, 0, 1, part.index, part.first};
    }
    if (f.b < 0) return;
    const int capacity = a.c.seq_pages << a.c.page_shift;
    const int len = a.c.lens[f.b];
    const int kh = hd / p.groups, g0 = hd % p.groups * p.heads, G = a.H / a.Hk;
    const int heads = min(p.heads, G - g0), rows = min(p.rows, f.last - f.row);
    // the tile's positions, and this wave's
    const int lo = cache_pos(len, f.row, f.last), hi = lo + rows - 1;
    const int c0 = wave * kColumns, row_lo = c0 / p.heads, row_hi = min((c0 + kColumns - 1) / p.heads, rows - 1);
    const int wave_lo = lo + row_lo, wave_hi = lo + row_hi;
    const bool active = row_lo < rows;
    const int my_row = (c0 + col) / p.heads, my_head = (c0 + col) % p.heads;
    const bool mine = my_row < rows && my_head < heads;
    const int pos = mine ? lo + my_row : -1;
    const long long q_head = static_cast<long long>(kh) * G + g0 + my_head;

    // which of the tiles
    const KeyTiles kt = key_tiles(lo, hi, capacity, a.window, a.sinks, KT);
    const int t0 = static_cast<int>(static_cast<long long>(kt.count) * f.split / f.splits);
    const int t1 = static_cast<int>(static_cast<long long>(kt.count) * (f.split + 1) / f.splits);
    const int keys = min(hi + 1, capacity);   // no row sees a key from here on
    const auto key_of = [&](int t) { return (t < kt.first ? t : t - kt.first + kt.from) * KT; };

    uint4 q[NQ];
    {
        const char* at = static_cast<const char*>(a.q) + ((f.row + my_row) * a.q_ld + q_head * kD) * ES + half * 16;
#pragma unroll
        for (int s = 0; s < NQ; ++s) q[s] = mine ? *reinterpret_cast<const uint4*>(at + s * 32) : make_uint4(0, 0, 0, 0);
    }

    f32x16 acc[4];
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.f;
    float m = -kInf, l = 0.f;   // m in base 2
    const float c = a.scale * kLog2e;

    // The table entry of a lane's key of tile t (-1: none), and where the row lies.
    const int32_t* table = a.c.table + static_cast<long long>(f.b) * a.c.seq_pages;
    const auto entry_of = [&](int t) {
        const int key = key_of(t) + lane % KT;
        return t < t1 && key < keys ? table[key >> a.c.page_shift] : -1;
    };
    const int piece = tid % PIECES, row0 = tid / PIECES;
    const int key_place = col * PK + half * 16, place_v = KT * PK + value_place<BF16, PV>();
    const char* k_base = static_cast<const char*>(a.c.k) + kh * a.c.head_stride * ES + piece * 16;
    const char* v_base = static_cast<const char*>(a.c.v) + kh * a.c.head_stride * ES + piece * 16;
    uint4 nk[LOADS], nv[LOADS];
    uint64_t there = 0, next_there = 0;   // the tile's rows that are
    // A row that is not there is read as the cache's first row: no row sees it.
    const auto fetch = [&](int t, int entry) {
        const long long off = cache_at(a.c, entry, key_of(t) + lane % KT);
        next_there = __ballot(off >= 0);
        const long long from = off >= 0 ? off * ES : 0;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const long long at = __shfl(from, row0 + j * Sh::kRowsAtOnce);
            nk[j] = *reinterpret_cast<const uint4*>(k_base + at);
            nv[j] = *reinterpret_cast<const uint4*>(v_base + at);
        }
    };
    // whether a row at positions from .. to does not see all of the tile's keys
    const auto partly = [&](int t, int from, int to) {
        const int key = key_of(t);
        return key + KT - 1 > from || (a.window > 0 && to - key >= a.window && key + KT > a.sinks);
    };
    const uint64_t all = KT == 64 ? ~0ull : 0xFFFFFFFFull;
    // A NaN or an infinity in V that some row does not see (0 x NaN would carry it there) is made 0 in
    // the tile, and its rows get a NaN afterwards: odd[] says which channels of which key.
    const auto keep = [&](int t, int buf) {
        there = next_there;
        if ((there & all) != all || partly(t, lo, hi)) {
            uint32_t bad[LOADS], any = 0;
#pragma unroll
            for (int j = 0; j < LOADS; ++j) any |= bad[j] = part_finite<BF16>(nv[j]);
            const bool some = __ballot(any != 0) != 0;
            if (some)
#pragma unroll
                for (int j = 0; j < LOADS; ++j) odd[buf][(row0 + j * Sh::kRowsAtOnce) * PIECES + piece] = static_cast<uint8_t>(bad[j]);
            if (lane == 0) spoiled[buf][wave] = some;
        }
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            char* at = tiles[buf] + j * Sh::kRowsAtOnce * PK;
            *reinterpret_cast<uint4*>(at + row0 * PK + piece * 16) = nk[j];
            at = tiles[buf] + KT * PK + j * Sh::kRowsAtOnce * PV;
            *reinterpret_cast<uint4*>(at + row0 * PV + piece * 16) = nv[j];
        }
    };

    int entry = entry_of(t0);
    if (t0 < t1) {
        fetch(t0, entry);
        entry = entry_of(t0 + 1);
        keep(t0, 0);
    }
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1;
        const uint64_t now = there;
        if (t + 1 < t1) {
            fetch(t + 1, entry);
            entry = entry_of(t + 2);
        }
        const int key0 = key_of(t);
        if (active && key0 <= wave_hi) {
            f32x16 s[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[b][r] = 0.f;
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const uint4 u = *reinterpret_cast<const uint4*>(tiles[buf] + key_place + 32 * b * PK + 32 * x);
                    if constexpr (BF16) {
                        s[b] = mfma(u, q[x], s[b]);
                    } else {
                        s[b] = mfma(real(u.x), real(q[x].x), s[b]);
                        s[b] = mfma(real(u.y), real(q[x].y), s[b]);
                        s[b] = mfma(real(u.z), real(q[x].z), s[b]);
                        s[b] = mfma(real(u.w), real(q[x].w), s[b]);
                    }
                }
            }
            const bool masked = (now & all) != all || partly(t, wave_lo, wave_hi);
            const auto sees = [&](int i) {   // key i of the tile, by this lane's column
                const int key = key0 + i;
                return (now >> i & 1) && key <= pos && (a.window <= 0 || pos - key < a.window || key < a.sinks);
            };
            if (masked) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[b][r] = sees(32 * b + 8 * (r >> 2) + 4 * half + (r & 3)) ? s[b][r] : -kInf;
            }
            float top = s[0][0];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
            float x, y;
            halves(top, x, y);
            top = fmaxf(x, y) * c;
            const bool up = top > m + kSlack || (m == -kInf && top > m);
            if (__ballot(up)) {   // each column by itself: no other column's values move its maximum
                const float to = up ? top : m;
                const float by = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - to);
                m = to;
                l *= by;
#pragma unroll
                for (int d = 0; d < 4; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[d][r] *= by;
            }
            const float base = m == -kInf ? 0.f : m;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], c, -base));
                    l += s[b][r];
                }
            add_values<BF16, NB, PV>(acc, s, tiles[buf] + place_v);
            uint32_t some = 0;
            if ((now & all) != all || partly(t, lo, hi))   // as in keep
#pragma unroll
                for (int w = 0; w < WAVES; ++w) some |= spoiled[buf][w];
            if (some) {
                constexpr int ROWS = 64 / PIECES;   // of a wave in each load
#pragma unroll 1
                for (int i = 0; i < KT; ++i) {
                    if (spoiled[buf][i / ROWS % WAVES] == 0 || !sees(i)) continue;
#pragma unroll
                    for (int d = 0; d < 4; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const uint32_t x = BF16 ? odd[buf][i * PIECES + 4 * d + (r >> 2)] >> (4 * half + (r & 3))
                                                    : odd[buf][i * PIECES + 8 * d + 2 * (r >> 2) + half] >> (r & 3);
                            acc[d][r] = x & 1 ? __builtin_nanf("") : acc[d][r];
                        }
                }
            }
        }
        if (t + 1 < t1) keep(t + 1, buf ^ 1);
        __syncthreads();
    }

    float x, y;
    halves(l, x, y);
    l = x + y;
    if (SPLIT && f.split == 0 && hd == 0 && tid == 0)
        Partials(a.work, p, n_heads).tiles[f.first / p.rows + f.b + f.index] = make_int2(place, f.splits);
    if (!mine) return;
    if (SPLIT && f.splits > 1) {
        const Partials w(a.work, p, n_heads);
        const long long at = (static_cast<long long>(place) * n_heads + hd) * p.cols + c0 + col;
        if (half == 0) w.ml[at] = make_float2(m, l);
        float* o = w.o + at * kD;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                *reinterpret_cast<float4*>(o + 32 * d + 2 * r + 4 * half) =
                    make_float4(acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]);
        return;
    }
    const float by = l == 0.f ? 0.f : 1.f / l;
    char* o = static_cast<char*>(a.o) + ((f.row + my_row) * static_cast<long long>(a.H) + q_head) * kD * ES;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const float z[4] = {acc[d][r] * by, acc[d][r + 1] * by, acc[d][r + 2] * by, acc[d][r + 3] * by};
            char* at = o + (32 * d + 2 * r + 4 * half) * ES;
            if constexpr (BF16)
                *reinterpret_cast<uint2*>(at) = make_uint2(pack(z[0], z[1]), pack(z[2], z[3]));
            else
                *reinterpret_cast<float4*>(at) = make_float4(z[0], z[1], z[2], z[3]);
        }
}

// Joins the splits of a column (row and head): a workgroup each, whose waves take every fourth
// split; a lane has two channels.
template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a, Plan p) {
    constexpr int WAVES = kJoinThreads / 64, AHEAD = 4;
    __shared__ float2 sums[WAVES][64];
    __shared__ float2 ml[WAVES];
    const int n_heads = a.Hk * p.groups, hd = blockIdx.x % n_heads, slot = blockIdx.x / n_heads, c = blockIdx.y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Part f = find_part(a, p.rows, slot);
    if (f.b < 0) return;
    const int row = f.first + f.index * p.rows + c / p.heads, kh = hd / p.groups, G = a.H / a.Hk;
    const int head = hd % p.groups * p.heads + c % p.heads;
    if (row >= f.last || head >= G) return;
    const Partials w(a.work, p, n_heads);
    const int2 tile = w.tiles[slot];
    if (tile.y <= 1) return;
    const long long step = static_cast<long long>(n_heads) * p.cols;
    const long long at = (static_cast<long long>(tile.x) * n_heads + hd) * p.cols + c;
    const float2* o = reinterpret_cast<const float2*>(w.o) + at * (kD / 2) + lane;
    float m = -kInf, l = 0.f;
    float2 x = make_float2(0.f, 0.f);
    for (int i0 = wave; i0 < tile.y; i0 += WAVES * AHEAD) {
        float2 part[AHEAD], got[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int n = i0 + i * WAVES;
            part[i] = n < tile.y ? w.ml[at + n * step] : make_float2(-kInf, 0.f);
            got[i] = n < tile.y ? o[n * step * (kD / 2)] : make_float2(0.f, 0.f);
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) top = fmaxf(top, part[i].x);
        const float base = top == -kInf ? 0.f : top;
        const float by = __builtin_amdgcn_exp2f(m - base);
        l *= by;
        x.x *= by;
        x.y *= by;
        m = top;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float e = __builtin_amdgcn_exp2f(part[i].x - base);
            l = fmaf(part[i].y, e, l);
            x.x = fmaf(got[i].x, e, x.x);
            x.y = fmaf(got[i].y, e, x.y);
        }
    }
    sums[wave][lane] = x;
    if (lane == 0) ml[wave] = make_float2(m, l);
    __syncthreads();
    if (wave != 0) return;
    m = ml[0].x;
#pragma unroll
    for (int i = 1; i < WAVES; ++i) m = fmaxf(m, ml[i].x);
    const float base = m == -kInf ? 0.f : m;
    l = 0.f;
    x = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        const float e = __builtin_amdgcn_exp2f(ml[i].x - base);
        l = fmaf(ml[i].y, e, l);
        x.x = fmaf(sums[i][lane].x, e, x.x);
        x.y = fmaf(sums[i][lane].y, e, x.y);
    }
    const float by = l == 0.f ? 0.f : 1.f / l;
    const long long to = (row * static_cast<long long>(a.H) + static_cast<long long>(kh) * G + head) * kD + 2 * lane;
    if constexpr (BF16)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + to) = pack(x.x * by, x.y * by);
    else
        *reinterpret_cast<float2*>(static_cast<float*>(a.o) + to) = make_float2(x.x * by, x.y * by);
}

// Four waves a tile where a sequence fills more than one wave's columns on average.
bool is_wide(int R, int B, int H, int Hk) { return static_cast<long long>(R) * (H / Hk) > static_cast<long long>(B) * kColumns; }

template <bool BF16, int WAVES>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
    Plan p = plan_of(a.R, a.B, a.H, a.Hk, WAVES == 4);
    const int n_heads = a.Hk * p.groups;
    if (static_cast<long long>(a.c.seq_pages) << a.c.page_shift <= kSplitKeys) p.parts = 0;
    if (p.parts == 0) {
        attn_kernel<BF16, WAVES, false><<<dim3(static_cast<unsigned>(p.slots) * n_heads), dim3(WAVES * 64), 0, stream>>>(a, p);
        return hipGetLastError();
    }
    attn_kernel<BF16, WAVES, true><<<dim3(static_cast<unsigned>(p.parts + p.slots) * n_heads), dim3(WAVES * 64), 0, stream>>>(a, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int columns = (a.R < p.rows ? a.R : p.rows) * p.heads;
    attn_join_kernel<BF16><<<dim3(static_cast<unsigned>(p.slots) * n_heads, static_cast<unsigned>(columns)), dim3(kJoinThreads), 0, stream>>>(a, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, bool bf16, hipStream_t stream) {
    // four 16-byte pieces a thread and more
    const int pieces = a.Hk * kD * (bf16 ? 2 : 4) / 16;
    const int rows = pieces >= 4 * kAppendThreads ? 1 : 4 * kAppendThreads / pieces;
    const dim3 grid(static_cast<unsigned>(a.R / rows + a.B));
    if (bf16)
        append_kernel<true><<<grid, dim3(kAppendThreads), 0, stream>>>(a, rows);
    else
        append_kernel<false><<<grid, dim3(kAppendThreads), 0, stream>>>(a, rows);
    return hipGetLastError();
}

long long attn_workgroups(int R, int B, int H, int Hk) {
    const Plan p = plan_of(R, B, H, Hk, is_wide(R, B, H, Hk));
    return (static_cast<long long>(p.slots) + p.parts) * Hk * p.groups;
}

// Grows with R and B, though the division of a call does not.
long long attn_work_bytes(int R, int B, int H, int Hk) {
    long long most = 0;
    for (const bool wide : {false, true}) {
        const Plan p = plan_of(R, B, H, Hk, wide);
        const int n_heads = Hk * p.groups, target = wide ? kTargetWide : kTargetNarrow;
        const long long parts = div_up(target, n_heads), slots = p.slots < parts ? p.slots : parts;
        const long long n = (parts + slots) * n_heads * p.cols * (kD + 2) * 4 + slots * 8;
        if (n > most) most = n;
    }
    return most;
}

hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t stream) {
    if (is_wide(a.R, a.B, a.H, a.Hk)) return bf16 ? launch<true, 4>(a, stream) : launch<false, 4>(a, stream);
    return bf16 ? launch<true, 1>(a, stream) : launch<false, 1>(a, stream);
}

}  // namespace kda
