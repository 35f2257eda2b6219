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
// one product: a tile of columns (128 of four waves; 32 for few f32 rows) reads
// each key and value once for all of them.  A wave owns 32 columns.  It computes
// S^T = K Q^T, whose accumulators hold a column a lane, so that the softmax needs
// one exchange between the lane's two halves; the same registers are the operand of
// O^T += V^T P^T, with the keys of a step in the order in which the accumulators
// hold them.
//
// Where the tiles of columns are too few to fill the chip, the keys of a tile
// are split over workgroups, which leave O, m and l in the workspace for a
// second launch.  Where they fill it, nothing is split, however uneven the
// sequences are: with 8 key heads bf16 from 64 tiles on (64 places; few shares
// are left from some 50 on).
//
// On an MI355X, calls in a loop (what a call cannot do without, at the 5.1 TB/s of
// a large copy or the 1,300 TFLOP/s of a large bf16 product, in brackets): a prompt
// of 4,096 rows x 64 heads bf16 317-334 us (211), 15 verify rows x 64 heads over
// 65,536 keys 74-76 us (53), one token of 15 sessions of 82,000 keys in all 74 us (66),
// ragged chunks of 1,420 rows x 12 heads 63-65 us (28), verify rounds of 8 sessions
// with a window of 1,024, 16 heads f32, 41 us (19), one token over 300 keys 10.7 us.
// The prompt is at 0.42 MFMA and 0.41 VALU activity: two waves a SIMD, whose
// products and softmax overlap in part, and its tiles start in the order of their rows, so that
// those with the most keys end alone: 160 tiles' times of a place where the
// mean is 130 (computed, not measured apart).  Two waves of 64 columns do not fit the
// registers, one a SIMD leaves every latency open (587 us against 360 then).  V is read
// in 8-byte transposing reads at half of LDS's rate; turning it on its way to LDS
// cost as much as that saves (360 against 357).  Tiles of 32 keys with three
// workgroups a CU took 376 us against 350.
// Batches of few columns are bound by memory: 4.5 TB/s over the steps.  The windowed
// rounds wait (0.33 MFMA, 0.12 VALU): two tiles a wave, behind the plan, a table entry and K.
// A step of 64 sessions, one of 65,536 keys and 63 of 300, takes 1,320 us (68): its
// longest sequence is read by one workgroup a key head.

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
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
using f32x16 = __attribute__((ext_vector_type(16))) float;

constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;        // the carried maximum may lag by this much (base 2)
constexpr float kFar = 16777216.0f;   // from here on (base 2) a step of f32 is a power of two or more
constexpr int kColumns = 32;          // columns of a wave
constexpr int kTargetNarrow = 2048;   // workgroups that run side by side: one wave each
constexpr int kTargetWide = 512;      // four waves each
constexpr int kLeastTiles = 1;        // a split has this many tiles at least
constexpr int kSplitKeys = 128;       // a cache of no more keys a sequence is never split
constexpr int kNarrowColumns = 96;    // of a sequence, up to which f32 rows take the narrow kernel
constexpr int kAppendThreads = 256;
constexpr int kJoinThreads = 256;
constexpr int kManySplits = 32;       // of a column: joined by four waves
constexpr int kJoinGroups = 2048;     // workgroups of the join, about

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
    int parts;       // workgroups a (key head, part) beside those of the tiles, for which the keys are split; 0: not split
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
    // parts + slots workgroups at most: as many as run side by side
    const int side = target / (Hk * p.groups);
    p.parts = n < target && side > p.slots ? side - p.slots : 0;
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
// Every wave runs it by itself; up to 64 sequences a lane.
__device__ __forceinline__ Item find_item(const AttnArgs& a, const Plan& p, int kt, int item) {
    const int lane = threadIdx.x & 63;
    const int capacity = a.c.seq_pages << a.c.page_shift;
    const int each = div_up(a.B, 64), from = min(lane * each, a.B), to = min(from + each, a.B);
    const auto row = [&](int b) { return min(max(a.offsets[b], 0), a.R); };
    int most = 0;
    for (int b = from; b < to; ++b) most = max(most, row(b));
    const int before = lane_before(running_max(most), 0);
    // Calls back for each of the lane's sequences: its rows, tiles of columns and tiles of keys.
    const auto visit = [&](auto&& with) {
        int run = before;
        for (int b = from; b < to; ++b) {
            const int first = max(run, row(b)), last = min(max(a.offsets[b + 1], first), a.R);
            run = first;
            const int across = div_up(last - first, p.rows);
            int along = 0;
            if (across > 0) {
                const int hi = cache_pos(a.c.lens[b], last - 1, last);
                along = key_tiles(max(hi - p.rows + 1, hi - (last - first) + 1), hi, capacity, a.window, a.sinks, kt).count;
            }
            with(b, first, last, across, along);
        }
    };
    // up to 64 sequences, one a lane, are read once
    int b1 = -1, first1 = 0, last1 = 0, across1 = 0, along1 = 0;
    if (each == 1)
        visit([&](int b, int first, int last, int across, int along) {
            b1 = b; first1 = first; last1 = last; across1 = across; along1 = along;
        });
    const auto again = [&](auto&& with) {
        if (each > 1) visit(with);
        else if (b1 >= 0) with(b1, first1, last1, across1, along1);
    };
    long long units = 0;
    again([&](int, int, int, int across, int along) { units += static_cast<long long>(across) * along; });
    units = of_lane(running_sum(units), 63);
    const int unit = max(kLeastTiles, static_cast<int>(min((units + p.parts - 1) / p.parts, 1ll << 30)));
    int mine = 0;
    again([&](int, int, int, int across, int along) { mine += across * max(1, div_up(along, unit)); });
    const int upto = running_sum(mine);
    Item f{-1, 0, 0, 0, 1, 0, 0};
    const uint64_t mask = __ballot(item >= upto - mine && item < upto);
    if (mask == 0) return f;
    const int owner = __builtin_ctzll(mask);
    int base = upto - mine;
    again([&](int b, int first, int last, int across, int along) {
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
    });
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
    static constexpr int kKeys = BF16 ? 64 : 32;
    static constexpr int kBlocks = kKeys / 32;
    static constexpr int kPieces = kD * kEs / 16;              // 16-byte pieces of a row
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
__device__ __forceinline__ uint32_t part_finite(u32x4& u) {
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = u[i];
        if constexpr (BF16) {
            const bool lo = (x & 0x7F80u) == 0x7F80u, hi = (x & 0x7F800000u) == 0x7F800000u;
            bad |= (lo ? 1u : 0u) << 2 * i | (hi ? 2u : 0u) << 2 * i;
            u[i] = x & ((lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u));
        } else {
            const bool all = (x & 0x7F800000u) == 0x7F800000u;
            bad |= (all ? 1u : 0u) << i;
            u[i] = all ? 0u : x;
        }
    }
    return bad;
}

// O^T += V^T P^T over a tile.  at(row, d): where the lane reads V from row `row` on (bf16: by four_keys; f32:
// a float), channels of block d.  P is rounded to bf16 for a bf16 cache, by half a step of 2^-8 at most; l sums
// it unrounded.
template <bool BF16, int NB, typename At>
__device__ __forceinline__ void add_values(f32x16 (&acc)[4], const f32x16 (&s)[NB], At&& at) {
    if constexpr (BF16) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int step = 0; step < 2; ++step) {
                const auto p = [&](int i) { return pack(s[b][8 * step + i], s[b][8 * step + i + 1]); };
                const uint4 w = make_uint4(p(0), p(2), p(4), p(6));
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint2 x = four_keys(at(32 * b + 16 * step, d)), y = four_keys(at(32 * b + 16 * step + 8, d));
                    acc[d] = mfma(make_uint4(x.x, x.y, y.x, y.y), w, acc[d]);
                }
            }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                acc[d] = mfma(*reinterpret_cast<const float*>(at(8 * (r >> 2) + (r & 3), d)), s[0][r], acc[d]);
    }
}

// What a workgroup computes: rows x heads columns, keys of tiles t0 .. t1-1.
struct Work {
    Item f;
    int hd;          // head part: key head and part of its query heads
    int kh;
    int heads;       // query heads of the part
    int rows;        // rows of the tile of columns
    int lo, hi;      // their positions
    int t0, t1;
    int keys;        // no row sees a key from here on
    KeyTiles tiles;
    long long head;  // first query head
};

template <int KT, bool SPLIT>
__device__ __forceinline__ Work work_of(const AttnArgs& a, const Plan& p) {
    Work w;
    const int n_heads = a.Hk * p.groups, place = blockIdx.x / n_heads;
    w.hd = blockIdx.x % n_heads;
    if constexpr (SPLIT) {
        w.f = find_item(a, p, KT, place);
    } else {
        const Part part = find_part(a, p.rows, place);
        w.f = Item{part.b, part.first + part.index * p.rows, part.last, 0, 1, part.index, part.first};
    }
    if (w.f.b < 0) return w;
    const int G = a.H / a.Hk, capacity = a.c.seq_pages << a.c.page_shift, g0 = w.hd % p.groups * p.heads;
    w.kh = w.hd / p.groups;
    w.head = static_cast<long long>(w.kh) * G + g0;
    w.heads = min(p.heads, G - g0);
    w.rows = min(p.rows, w.f.last - w.f.row);
    w.lo = cache_pos(a.c.lens[w.f.b], w.f.row, w.f.last);
    w.hi = w.lo + w.rows - 1;
    w.tiles = key_tiles(w.lo, w.hi, capacity, a.window, a.sinks, KT);
    w.t0 = static_cast<int>(static_cast<long long>(w.tiles.count) * w.f.split / w.f.splits);
    w.t1 = static_cast<int>(static_cast<long long>(w.tiles.count) * (w.f.split + 1) / w.f.splits);
    w.keys = min(w.hi + 1, capacity);
    return w;
}

// First key of tile t.
template <int KT>
__device__ __forceinline__ int key_of(const Work& w, int t) {
    return (t < w.tiles.first ? t : t - w.tiles.first + w.tiles.from) * KT;
}

// The table entry of tile t (WHOLE: a tile lies in one page) or of the lane's key of it; -1: none.
template <int KT, bool WHOLE>
__device__ __forceinline__ int entry_of(const AttnArgs& a, const Work& w, int t) {
    const int key = key_of<KT>(w, t) + (WHOLE ? 0 : static_cast<int>(threadIdx.x & 63) % KT);
    return t < w.t1 && key < w.keys ? a.c.table[static_cast<long long>(w.f.b) * a.c.seq_pages + (key >> a.c.page_shift)] : -1;
}

// Whether a row at positions from .. to does not see all keys of the tile that begins at key.
template <int KT>
__device__ __forceinline__ bool partly(const AttnArgs& a, int key, int from, int to) {
    return key + KT - 1 > from || (a.window > 0 && to - key >= a.window && key + KT > a.sinks);
}

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// Which of the 32 keys from key0 on a row at pos (-1: none) sees, of those that exist.
__device__ __forceinline__ uint32_t seen_by(const AttnArgs& a, uint32_t there, int pos, int key0) {
    uint32_t seen = there & low_bits(pos - key0 + 1);
    // (where the first difference wraps around, pos is before key0: nothing is seen)
    if (a.window > 0)
        seen &= ~low_bits(static_cast<int>(static_cast<uint32_t>(pos) - static_cast<uint32_t>(a.window) + 1u - static_cast<uint32_t>(key0))) |
                low_bits(a.sinks - key0);
    return seen;
}

// A wave's columns: a lane's column, in both halves, and what it carries.
template <bool BF16>
struct Columns {
    static constexpr int kQ = BF16 ? 8 : 16;   // 16-byte pieces of q a lane
    bool mine;       // the column exists
    int row, head;   // within the tile
    int pos;
    uint4 q[kQ];
    f32x16 acc[4];   // O^T
    float m, l;      // m in base 2; l of the half's keys
    bool far;        // |m| is kFar at least
    bool some_far;   // some column's is

    __device__ __forceinline__ void begin(const AttnArgs& a, const Plan& p, const Work& w, int c0) {
        constexpr int ES = BF16 ? 2 : 4;
        const int lane = threadIdx.x & 63, half = lane >> 5, c = c0 + (lane & 31);
        row = c / p.heads;
        head = c % p.heads;
        mine = row < w.rows && head < w.heads;
        pos = mine ? w.lo + row : -1;
        const char* at = static_cast<const char*>(a.q) + ((w.f.row + row) * a.q_ld + (w.head + head) * kD) * ES + half * 16;
#pragma unroll
        for (int x = 0; x < kQ; ++x) q[x] = mine ? *reinterpret_cast<const uint4*>(at + x * 32) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[d][r] = 0.f;
        m = -kInf;
        l = 0.f;
        far = some_far = false;
    }

    // S^T of 32 NB keys; read(b, i): 16 bytes of the lane's key of block b, pieces 2 i + half.  The blocks'
    // products alternate (each waits for the one before it in its block), K is read some products ahead.
    template <int NB, typename Read>
    __device__ __forceinline__ void scores(f32x16 (&s)[NB], Read&& read) const {
        constexpr int N = NB * kQ, AHEAD = 4;
        uint4 u[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) u[i] = read(i % NB, i / NB);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[b][r] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint4 w = u[i % AHEAD], y = q[i / NB];
            f32x16& z = s[i % NB];
            if (i + AHEAD < N) u[i % AHEAD] = read((i + AHEAD) % NB, (i + AHEAD) / NB);
            if constexpr (BF16) {
                z = mfma(w, y, z);
            } else {
                z = mfma(real(w.x), real(y.x), z);
                z = mfma(real(w.y), real(y.y), z);
                z = mfma(real(w.z), real(y.z), z);
                z = mfma(real(w.w), real(y.w), z);
            }
        }
        if constexpr (BF16 && NB > 1) {   // in this order
            __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (i + AHEAD < N) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
    }

    // Scores of keys that the column does not see (bits of `seen`) to -inf.
    __device__ __forceinline__ static void mask(f32x16& s, uint32_t seen) {
        const int here = static_cast<int>(seen >> (threadIdx.x & 32 ? 4 : 0));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const uint32_t on = static_cast<uint32_t>(__builtin_amdgcn_sbfe(here, 8 * (r >> 2) + (r & 3), 1));   // all ones or 0
            s[r] = real((bits(s[r]) & on) | (0xFF800000u & ~on));
        }
    }

    // Scores to weights 2^{c s - m}; O, l and m follow a new maximum.  Each column by itself: no other
    // column's values move its maximum.  c s - m in one operation is off by the rounding of m alone, the same
    // for all keys, which the quotient does not see.  From kFar on that is half a power of two and more, beyond
    // 2^31 the weights would leave f32's range: there c s is rounded by itself, as m was.  (A test of a scalar
    // a tile: the prompt of 4,096 rows 317 us, 315 without.)
    template <int NB>
    __device__ __forceinline__ void weights(f32x16 (&s)[NB], float c) {
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
        float x, y;
        halves(top, x, y);
        top = fmaxf(x, y) * c;
        const bool up = (top > m + kSlack) | ((m == -kInf) & (top > m));
        if (__ballot(up)) {
            const float to = up ? top : m;
            const float by = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - to);
            m = to;
            far = (fabsf(m) >= kFar) & (m != -kInf);
            some_far = __ballot(far) != 0;
            l *= by;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] *= by;
        }
        if (some_far) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[b][r] = far ? s[b][r] * c : s[b][r];
        }
        const float base = m == -kInf ? 0.f : m, per = far ? 1.f : c;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], per, -base));
                sum[r & 3] += s[b][r];
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }

    // A NaN in the channels of `odd` (a byte a piece).
    __device__ __forceinline__ void spoil(const uint8_t* odd) {
        const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t x = BF16 ? odd[4 * d + (r >> 2)] >> (4 * half + (r & 3)) : odd[8 * d + 2 * (r >> 2) + half] >> (r & 3);
                acc[d][r] = x & 1 ? __builtin_nanf("") : acc[d][r];
            }
    }

    // The result, or a split's part of it.
    template <bool SPLIT>
    __device__ __forceinline__ void finish(const AttnArgs& a, const Plan& p, const Work& w, int c0) {
        constexpr int ES = BF16 ? 2 : 4;
        const int lane = threadIdx.x & 63, half = lane >> 5, n_heads = a.Hk * p.groups, place = blockIdx.x / n_heads;
        float x, y;
        halves(l, x, y);
        l = x + y;
        if (SPLIT && w.f.split == 0 && w.hd == 0 && threadIdx.x == 0)
            Partials(a.work, p, n_heads).tiles[w.f.first / p.rows + w.f.b + w.f.index] = make_int2(place, w.f.splits);
        if (!mine) return;
        if (SPLIT && w.f.splits > 1) {
            const Partials parts(a.work, p, n_heads);
            const long long at = (static_cast<long long>(place) * n_heads + w.hd) * p.cols + c0 + (lane & 31);
            if (half == 0) parts.ml[at] = make_float2(m, l);
            float* o = parts.o + at * kD;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<float4*>(o + 32 * d + 2 * r + 4 * half) =
                        make_float4(acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]);
            return;
        }
        const float by = l == 0.f ? 0.f : 1.f / l;
        char* o = static_cast<char*>(a.o) + ((w.f.row + row) * static_cast<long long>(a.H) + w.head + head) * kD * ES;
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
};

template <int KT>
constexpr uint64_t kAll = KT == 64 ? ~0ull : (1ull << KT) - 1;

// Where a tile lies: the byte offset (head 0) of its first row (WHOLE) or of the row of the lane's key, and
// which of its rows exist.  What does not is read as the cache's first rows: no row sees it.
struct Place {
    long long off;
    uint64_t there;
};

template <int KT, int ES, bool WHOLE>
__device__ __forceinline__ Place place_of(const AttnArgs& a, const Work& w, int t, int entry) {
    const int key0 = key_of<KT>(w, t);
    if constexpr (WHOLE) {
        const long long at = cache_at(a.c, __builtin_amdgcn_readfirstlane(entry), key0);
        const int n = w.keys - key0;
        return at < 0 ? Place{0, 0} : Place{at * ES, n >= KT ? kAll<KT> : (1ull << (n & 63)) - 1};
    } else {
        const long long at = cache_at(a.c, entry, key0 + static_cast<int>(threadIdx.x & 63) % KT);
        return Place{at < 0 ? 0 : at * ES, __ballot(at >= 0) & kAll<KT>};
    }
}

// Rows of a tile that a thread brings to LDS: 16 bytes of row row0 + j * kRowsAtOnce in load j.
template <typename Sh, bool WHOLE>
struct Loader {
    struct Rows {
        u32x4 r[Sh::kLoads];
    };
    int piece, row0;
    const char* base;     // K's or V's, of the key head
    long long step;       // WHOLE: bytes from load to load
    uint32_t mine;        // bytes to the thread's piece of the tile's (WHOLE) or of any row

    __device__ __forceinline__ Loader(const void* p, const CacheView& c, int kh)
        : piece(threadIdx.x % Sh::kPieces), row0(threadIdx.x / Sh::kPieces),
          base(static_cast<const char*>(p) + kh * c.head_stride * Sh::kEs), step(Sh::kRowsAtOnce * c.row_stride * Sh::kEs),
          mine((WHOLE ? row0 * static_cast<uint32_t>(c.row_stride) * Sh::kEs : 0) + piece * 16) {}

    __device__ __forceinline__ Rows load(long long off) const {
        Rows u;
#pragma unroll
        for (int j = 0; j < Sh::kLoads; ++j) {
            const char* at = base + (WHOLE ? off + j * step : __shfl(off, row0 + j * Sh::kRowsAtOnce));
            u.r[j] = *reinterpret_cast<const u32x4*>(at + mine);
        }
        return u;
    }

    template <int PITCH>
    __device__ __forceinline__ void store(Rows u, char* to) const {
#pragma unroll
        for (int j = 0; j < Sh::kLoads; ++j)
            *reinterpret_cast<u32x4*>(to + row0 * PITCH + piece * 16 + j * Sh::kRowsAtOnce * PITCH) = u.r[j];
    }

    // Of V, where some row does not see all keys: what the wide kernel does in LDS, before the rows go
    // there.  Whether the wave brought any.
    __device__ __forceinline__ bool part(Rows& u, uint8_t* odd) const {
        uint32_t bad[Sh::kLoads], any = 0;
#pragma unroll
        for (int j = 0; j < Sh::kLoads; ++j) any |= bad[j] = part_finite<false>(u.r[j]);
        if (__ballot(any != 0) == 0) return false;
#pragma unroll
        for (int j = 0; j < Sh::kLoads; ++j) odd[(row0 + j * Sh::kRowsAtOnce) * Sh::kPieces + piece] = static_cast<uint8_t>(bad[j]);
        return true;
    }
};

// Waits for all loads: what a loop only reads would else be waited for in every turn, with what the turn loads.
__device__ __forceinline__ void arrived() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// The tiles of the wide kernel in LDS, row by row as they are loaded there: piece c of row r lies at
// c ^ turn(r), so that the 16-byte reads of K (16 or 8 rows), and those of V (four rows of 64 bytes, or
// rows 4 apart of 128 bytes) lie on all banks.
template <bool BF16>
__device__ __forceinline__ int turn_k(int row) { return BF16 ? row & 15 : row & 7; }
template <bool BF16>
__device__ __forceinline__ int turn_v(int row) { return BF16 ? (row & 3) << 2 : (row & 4) << 1; }

// 16 bytes a lane from global memory to LDS, lane after lane from `to` (the same in all lanes) on.
__device__ __forceinline__ void to_lds(const char* from, char* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// 128 columns: four waves share the tiles of keys, two of which lie in LDS.
template <bool BF16, bool SPLIT, bool WHOLE>
__global__ void __launch_bounds__(256, 2) attn_wide_kernel(AttnArgs a, Plan p) {
    using Sh = Shape<BF16, 4>;
    constexpr int KT = Sh::kKeys, NB = Sh::kBlocks, ES = Sh::kEs, ROW = kD * ES, PIECES = Sh::kPieces, BYTES = KT * ROW;
    // (arrays of their own: what is on its way to one does not hold up the reads of another)
    __shared__ __align__(16) char k0[BYTES], v0[BYTES], k1[BYTES], v1[BYTES];
    __shared__ uint32_t spoiled[4];      // whether the wave found values that are not finite: odd says which
    __shared__ uint8_t odd[KT * PIECES];
    const int lane = threadIdx.x & 63, half = lane >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c0 = wave * kColumns;
    const Work w = work_of<KT, SPLIT>(a, p);
    if (w.f.b < 0) return;
    // the wave's positions
    const int row_lo = c0 / p.heads, wave_lo = w.lo + row_lo, wave_hi = w.lo + min((c0 + kColumns - 1) / p.heads, w.rows - 1);
    Columns<BF16> x;
    x.begin(a, p, w, c0);
    const float c = a.scale * kLog2e;
    // what the thread brings: place `piece` of rows row0 + j * kRowsAtOnce, which has another piece
    const int piece = threadIdx.x % PIECES, row0 = threadIdx.x / PIECES;
    const int piece_k = piece ^ turn_k<BF16>(row0), piece_v = piece ^ turn_v<BF16>(row0);
    const long long step = Sh::kRowsAtOnce * a.c.row_stride * ES;
    const uint32_t mine = WHOLE ? row0 * static_cast<uint32_t>(a.c.row_stride) * ES : 0;
    const char* base_k = static_cast<const char*>(a.c.k) + w.kh * a.c.head_stride * ES;
    const char* base_v = static_cast<const char*>(a.c.v) + w.kh * a.c.head_stride * ES;
    const auto fetch = [&](const Place& at, char* k, char* v) {
#pragma unroll
        for (int j = 0; j < Sh::kLoads; ++j) {
            const long long off = WHOLE ? at.off + j * step : __shfl(at.off, row0 + j * Sh::kRowsAtOnce);
            const int to = (j * 4 + wave) * 1024;
            to_lds(base_k + off + (mine + piece_k * 16), k + to);
            to_lds(base_v + off + (mine + piece_v * 16), v + to);
        }
    };
    // where the lane reads
    const int key_at = (lane & 31) * ROW + ((half ^ turn_k<BF16>(lane & 31)) * 16);
    const int i16 = lane & 15, r0 = BF16 ? 4 * half + (i16 >> 2) : 4 * half;
    const int value_at = BF16 ? r0 * ROW + ((2 * (lane >> 4 & 1) + (i16 >> 1 & 1)) ^ turn_v<BF16>(r0)) * 16 + (i16 & 1) * 8
                              : r0 * ROW + (((lane & 31) >> 2) ^ turn_v<BF16>(r0)) * 16 + (lane & 3) * 4;
    uint64_t there = 0, next_there = 0;   // the tile's rows that exist
    int entry = entry_of<KT, WHOLE>(a, w, w.t0);
    const auto turn = [&](int t, char* k, char* v, char* next_k, char* next_v) {
        const int key0 = key_of<KT>(w, t);
        const bool uneven = there != kAll<KT> || partly<KT>(a, key0, w.lo, w.hi);
        if (t + 1 < w.t1) {
            const Place at = place_of<KT, ES, WHOLE>(a, w, t + 1, entry);
            next_there = at.there;
            fetch(at, next_k, next_v);
            entry = entry_of<KT, WHOLE>(a, w, t + 2);
        }
        // Some row does not see all keys: 0 x NaN would carry a NaN or an infinity of V into rows that do not
        // see it, so it is made 0, odd says which channels of which key it was, and the rows that see it get
        // a NaN afterwards.
        if (uneven) {
            bool any = false;
#pragma unroll
            for (int j = 0; j < Sh::kLoads; ++j) {
                const int row = row0 + j * Sh::kRowsAtOnce;
                u32x4* at = reinterpret_cast<u32x4*>(v + row * ROW + piece * 16);
                u32x4 u = *at;
                const uint32_t bad = part_finite<BF16>(u);
                if (bad) *at = u;
                odd[row * PIECES + piece_v] = static_cast<uint8_t>(bad);
                any |= bad != 0;
            }
            const bool some = __ballot(any) != 0;
            if (lane == 0) spoiled[wave] = some;
            __syncthreads();
        }
        if (row_lo < w.rows && key0 <= wave_hi) {
            f32x16 s[NB];
            __builtin_amdgcn_s_setprio(1);   // before the other wave's weights
            x.template scores<NB>(s, [&](int b, int i) { return *reinterpret_cast<const uint4*>(k + (key_at ^ (i * 32)) + b * 32 * ROW); });
            if (there != kAll<KT> || partly<KT>(a, key0, wave_lo, wave_hi))
#pragma unroll
                for (int b = 0; b < NB; ++b) x.mask(s[b], seen_by(a, static_cast<uint32_t>(there >> 32 * b), x.pos, key0 + 32 * b));
            __builtin_amdgcn_s_setprio(0);
            x.weights(s, c);
            add_values<BF16, NB>(x.acc, s, [&](int row, int d) { return v + (value_at ^ (d * (BF16 ? 64 : 128))) + row * ROW; });
            if (uneven && (spoiled[0] | spoiled[1] | spoiled[2] | spoiled[3])) {
#pragma unroll 1
                for (int i = 0; i < KT; ++i)
                    if (seen_by(a, static_cast<uint32_t>(there >> (i & 32)), x.pos, key0 + (i & 32)) >> (i & 31) & 1) x.spoil(odd + i * PIECES);
            }
        }
        there = next_there;
        arrived();
        __syncthreads();
    };
    if (w.t0 < w.t1) {
        const Place at = place_of<KT, ES, WHOLE>(a, w, w.t0, entry);
        there = at.there;
        fetch(at, k0, v0);
        entry = entry_of<KT, WHOLE>(a, w, w.t0 + 1);
    }
    arrived();
    __syncthreads();
    for (int t = w.t0; t < w.t1; t += 2) {
        turn(t, k0, v0, k1, v1);
        if (t + 1 < w.t1) turn(t + 1, k1, v1, k0, v0);
    }
    x.template finish<SPLIT>(a, p, w, c0);
}

// 32 columns of f32: a wave by itself, eight a CU.  K and V of a tile take turns in one region of LDS and in
// the registers that hold what is on its way: V comes while the scores are computed, the next K behind them.
template <bool SPLIT, bool WHOLE>
__global__ void __launch_bounds__(64, 2) attn_narrow_kernel(AttnArgs a, Plan p) {
    using Sh = Shape<false, 1>;
    // Pitches of the rows in LDS.  K: 16 rows of a 16-byte read lie on all banks; V: rows 4 apart of 128 bytes.
    constexpr int KT = Sh::kKeys, PK = kD * 4 + 16, PV = kD * 4 + 32;
    __shared__ __align__(16) char tile[KT * PV];
    __shared__ uint8_t odd[KT * Sh::kPieces];
    const int lane = threadIdx.x & 63;
    const Work w = work_of<KT, SPLIT>(a, p);
    if (w.f.b < 0) return;
    const Loader<Sh, WHOLE> from_k(a.c.k, a.c, w.kh), from_v(a.c.v, a.c, w.kh);
    Place at = place_of<KT, Sh::kEs, WHOLE>(a, w, w.t0, entry_of<KT, WHOLE>(a, w, w.t0));
    int entry = entry_of<KT, WHOLE>(a, w, w.t0 + 1);
    typename Loader<Sh, WHOLE>::Rows u;
    if (w.t0 < w.t1) u = from_k.load(at.off);
    Columns<false> x;
    x.begin(a, p, w, 0);
    const float c = a.scale * kLog2e;
    const int key_place = (lane & 31) * PK + (lane >> 5) * 16, value_at = 4 * (lane >> 5) * PV + 4 * (lane & 31);
    // (one wave: its LDS accesses are done in order)
    const auto order = [] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    if (w.t0 < w.t1) {
        from_k.template store<PK>(u, tile);
        u = from_v.load(at.off);
    }
    arrived();
    for (int t = w.t0; t < w.t1; ++t) {
        const int key0 = key_of<KT>(w, t);
        const uint64_t there = at.there;
        const bool masked = there != kAll<KT> || partly<KT>(a, key0, w.lo, w.hi);
        order();
        f32x16 s[1];
        x.template scores<1>(s, [&](int, int i) { return *reinterpret_cast<const uint4*>(tile + key_place + 32 * i); });
        order();
        bool odds = false;
        uint32_t seen = 0;
        if (masked) {
            seen = seen_by(a, static_cast<uint32_t>(there), x.pos, key0);
            x.mask(s[0], seen);
            odds = from_v.part(u, odd);
        }
        from_v.template store<PV>(u, tile);
        if (t + 1 < w.t1) {
            at = place_of<KT, Sh::kEs, WHOLE>(a, w, t + 1, entry);
            u = from_k.load(at.off);
            entry = entry_of<KT, WHOLE>(a, w, t + 2);
        }
        x.weights(s, c);
        order();
        add_values<false, 1>(x.acc, s, [&](int row, int d) { return tile + value_at + row * PV + d * 128; });
        if (odds) {
#pragma unroll 1
            for (int i = 0; i < KT; ++i)
                if (seen >> i & 1) x.spoil(odd + i * Sh::kPieces);
        }
        order();
        if (t + 1 < w.t1) {
            from_k.template store<PK>(u, tile);
            u = from_v.load(at.off);
        }
    }
    x.template finish<SPLIT>(a, p, w, 0);
}

// Joins the splits of columns (row and head).  TEAM waves take a column, each every TEAM-th split; a lane
// has two channels.
template <bool BF16, int TEAM>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a, Plan p, int columns, int per) {
    constexpr int WAVES = kJoinThreads / 64, AHEAD = 8;
    __shared__ float2 sums[WAVES][64];
    __shared__ float2 ml[WAVES];
    const int n_heads = a.Hk * p.groups, hd = blockIdx.x % n_heads, slot = blockIdx.x / n_heads;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, mate = wave % TEAM;
    const Partials w(a.work, p, n_heads);
    const int2 tile = w.tiles[slot];   // (anything, where the slot is empty)
    const Part f = find_part(a, p.rows, slot);
    if (f.b < 0 || tile.y <= 1) return;
    const int first = f.first + f.index * p.rows, kh = hd / p.groups, G = a.H / a.Hk, g0 = hd % p.groups * p.heads;
    const long long step = static_cast<long long>(n_heads) * p.cols;
    const int begin = blockIdx.y * per, end = min(begin + per, columns);
    for (int c = begin + wave / TEAM; c - wave / TEAM < end; c += WAVES / TEAM) {
        const int row = first + c / p.heads, head = g0 + c % p.heads;
        const bool there = c < end && row < f.last && head < G;
        const long long at = (static_cast<long long>(tile.x) * n_heads + hd) * p.cols + c;
        const float2* o = reinterpret_cast<const float2*>(w.o) + at * (kD / 2) + lane;
        float m = -kInf, l = 0.f;
        float2 x = make_float2(0.f, 0.f);
        for (int i0 = mate; there && i0 < tile.y; i0 += TEAM * AHEAD) {
            float2 part[AHEAD], got[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int n = i0 + i * TEAM;
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
        if constexpr (TEAM > 1) {   // (a column a workgroup: one turn)
            sums[wave][lane] = x;
            if (lane == 0) ml[wave] = make_float2(m, l);
            __syncthreads();
            m = ml[0].x;
#pragma unroll
            for (int i = 1; i < TEAM; ++i) m = fmaxf(m, ml[i].x);
            const float base = m == -kInf ? 0.f : m;
            l = 0.f;
            x = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < TEAM; ++i) {
                const float e = __builtin_amdgcn_exp2f(ml[i].x - base);
                l = fmaf(ml[i].y, e, l);
                x.x = fmaf(sums[i][lane].x, e, x.x);
                x.y = fmaf(sums[i][lane].y, e, x.y);
            }
        }
        if (!there || mate != 0) continue;
        const float by = l == 0.f ? 0.f : 1.f / l;
        const long long to = (row * static_cast<long long>(a.H) + static_cast<long long>(kh) * G + head) * kD + 2 * lane;
        if constexpr (BF16)
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + to) = pack(x.x * by, x.y * by);
        else
            *reinterpret_cast<float2*>(static_cast<float*>(a.o) + to) = make_float2(x.x * by, x.y * by);
    }
}

// The narrow kernel takes f32 rows of up to 96 columns a sequence on average: its matrix products are the
// bound there, and a tile of 32 columns has fewer that do not exist.  8 sequences of 8,192 keys x 8 key heads,
// 32 columns each: 126 us against the wide kernel's 172; 96 columns 262 against 311; 120 columns 346 against
// 314.  bf16 is bound by memory there, and the wide kernel holds more loads on their way with fewer
// registers: one token of 15 sessions x 8,192 keys x 64 heads 98 us against 103, of one with 65,536 keys 24
// against 39, 32 columns 62 against 76; there is no narrow kernel for it.  (The average is all that the host
// knows: a long chunk beside many single tokens is read in tiles of 32 columns too.)
bool is_wide(int R, int B, int H, int Hk, bool bf16) {
    return bf16 || static_cast<long long>(R) * (H / Hk) > static_cast<long long>(B) * kNarrowColumns;
}

template <bool BF16, bool WIDE, bool WHOLE>
void start(const AttnArgs& a, const Plan& p, unsigned grid, hipStream_t stream) {
    if constexpr (WIDE) {
        if (p.parts)
            attn_wide_kernel<BF16, true, WHOLE><<<dim3(grid), dim3(256), 0, stream>>>(a, p);
        else
            attn_wide_kernel<BF16, false, WHOLE><<<dim3(grid), dim3(256), 0, stream>>>(a, p);
    } else {
        if (p.parts)
            attn_narrow_kernel<true, WHOLE><<<dim3(grid), dim3(64), 0, stream>>>(a, p);
        else
            attn_narrow_kernel<false, WHOLE><<<dim3(grid), dim3(64), 0, stream>>>(a, p);
    }
}

template <bool BF16, bool WIDE>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
    Plan p = plan_of(a.R, a.B, a.H, a.Hk, WIDE);
    const int n_heads = a.Hk * p.groups;
    // A short cache in one launch: one token, 8 heads, 120 keys 9.6 us a call, 12.5 with the join; 248 keys
    // 12.6 and 12.4.
    if (static_cast<long long>(a.c.seq_pages) << a.c.page_shift <= kSplitKeys) p.parts = 0;
    const unsigned grid = static_cast<unsigned>(p.parts + p.slots) * n_heads;
    // Pages of whole tiles need one entry a tile, and no address of a row of its own (rows within 2^31 bytes):
    // a prompt of 2,048 rows x 64 heads bf16 102 us, row by row 110; 8 verify rounds of 15 rows over 4,096 keys
    // x 16 heads f32 117 and 129.
    constexpr int KT = Shape<BF16, WIDE ? 4 : 1>::kKeys, ES = BF16 ? 2 : 4;
    if (1 << a.c.page_shift >= KT && a.c.row_stride < (1ll << 31) / (KT * ES))
        start<BF16, WIDE, true>(a, p, grid, stream);
    else
        start<BF16, WIDE, false>(a, p, grid, stream);
    if (p.parts == 0) return hipGetLastError();
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // Columns of many splits take four waves each.  Of few, a wave each, and some of them a workgroup
    // where there are many (it begins with a search for its rows).  Whole calls with four waves and with one:
    // one token over 65,536 keys, 8 heads (256 splits) 39 and 103 us; of 4 sessions over 16,384 (50) 62 and 66;
    // of 15 over 8,192 (17) 110 and 104; ragged chunks (4) 106 and 65.
    const int columns = (a.R < p.rows ? a.R : p.rows) * p.heads;
    const unsigned tiles = static_cast<unsigned>(p.slots) * n_heads;
    if (p.parts > kManySplits * p.slots) {
        attn_join_kernel<BF16, kJoinThreads / 64><<<dim3(tiles, static_cast<unsigned>(columns)), dim3(kJoinThreads), 0, stream>>>(a, p, columns, 1);
    } else {
        const long long n = static_cast<long long>(tiles) * columns;
        const int per = 4 * static_cast<int>((n + 4 * kJoinGroups - 1) / (4 * kJoinGroups));
        attn_join_kernel<BF16, 1><<<dim3(tiles, static_cast<unsigned>(div_up(columns, per))), dim3(kJoinThreads), 0, stream>>>(a, p, columns, per);
    }
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
    long long most = 0;
    for (const bool bf16 : {false, true}) {
        const Plan p = plan_of(R, B, H, Hk, is_wide(R, B, H, Hk, bf16));
        const long long n = (static_cast<long long>(p.slots) + p.parts) * Hk * p.groups;
        if (n > most) most = n;
    }
    return most;
}

// Grows with R and B, though the division of a call does not.
long long attn_work_bytes(int R, int B, int H, int Hk) {
    long long most = 0;
    for (const bool wide : {false, true}) {
        const Plan p = plan_of(R, B, H, Hk, wide);
        const int n_heads = Hk * p.groups, side = div_up(wide ? kTargetWide : kTargetNarrow, n_heads);
        const long long slots = p.slots < side ? p.slots : side;
        const long long n = (side + 1ll) * n_heads * p.cols * (kD + 2) * 4 + slots * 8;
        if (n > most) most = n;
    }
    return most;
}

hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t stream) {
    if (bf16) return launch<true, true>(a, stream);
    return is_wide(a.R, a.B, a.H, a.Hk, false) ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace kda
