// Where the rows of a packed batch lie, read on the device: sequence b of B has
// rows offsets[b] .. offsets[b+1]-1 of R.  Args: any argument block with
// offsets, R and B.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"

namespace kda {
namespace {

// Where a part of a packed batch lies.  Sequence b takes the slots
// first / part_rows + b, ... (one for each part of part_rows rows), so parts of
// different sequences never share a slot and R / part_rows + B slots are enough.
struct Part {
    int b;        // sequence, -1: the slot is empty
    int index;    // part within the sequence
    int first;    // the sequence's rows
    int last;
};

// Inclusive running maximum over the lanes.
__device__ __forceinline__ int running_max(int x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x = max(x, y);
    }
    return x;
}

// The sequence of a slot: the last one whose slots begin at or before it.  The
// table is read with a running maximum, clamped to [0, R], so that any table
// gives disjoint rows and slots; every wave runs this by itself.  Beyond 64
// sequences each lane first takes 1/64 of the table (64 entries at most), to
// find the stretch of it that is searched.
template <typename Args>
__device__ __forceinline__ Part find_part(const Args& a, int part_rows, int slot) {
    static_assert(KDA_PROMPT_SEQS_MAX <= 64 * 64, "two levels of 64");
    const int lane = threadIdx.x & 63;
    const auto row = [&](int b) { return min(max(a.offsets[b], 0), a.R); };
    Part f{-1, 0, 0, 0};
    if (a.B == 1) {
        f.first = row(0);
        f.index = slot - f.first / part_rows;
        f.last = max(row(1), f.first);
        if (f.index >= 0 && f.first + static_cast<long long>(f.index) * part_rows < f.last) f.b = 0;
        return f;
    }
    int b0 = 0, n = min(a.B, 64), before = 0;   // the stretch, and the largest entry before it
    if (a.B > 64) {
        const int each = (a.B + 63) / 64, from = lane * each, to = min(from + each, a.B);
        int x = 0;
        for (int b = from; b < to; ++b) x = max(x, row(b));
        const int upto = running_max(x);
        int ahead = __shfl_up(upto, 1);
        if (lane == 0) ahead = 0;
        const uint64_t mask = __ballot(from < to && max(ahead, row(min(from, a.B - 1))) / part_rows + from <= slot);
        if (mask == 0) return f;
        const int at = 63 - __builtin_clzll(mask);
        b0 = at * each;
        n = min(each, a.B - b0);
        before = __builtin_amdgcn_readlane(ahead, at);
    }
    const int b = b0 + lane;
    const int x = running_max(max(before, lane < n ? row(b) : 0));
    const uint64_t mask = __ballot(lane < n && x / part_rows + b <= slot);
    if (mask == 0) return f;
    const int at = 63 - __builtin_clzll(mask);
    f.first = __builtin_amdgcn_readlane(x, at);
    f.index = slot - (f.first / part_rows + b0 + at);
    f.last = min(max(a.offsets[b0 + at + 1], f.first), a.R);
    if (f.first + static_cast<long long>(f.index) * part_rows < f.last) f.b = b0 + at;
    return f;
}

// Rows of sequence b under the same reading of the table.
template <typename Args>
__device__ __forceinline__ void sequence(const Args& a, int b, int& first, int& last) {
    int x = 0;
    for (int i = threadIdx.x & 63; i <= b; i += 64) x = max(x, min(max(a.offsets[i], 0), a.R));
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x = max(x, __shfl_xor(x, m));
    first = __builtin_amdgcn_readfirstlane(x);
    last = min(max(a.offsets[b + 1], first), a.R);
}

}  // namespace
}  // namespace kda
