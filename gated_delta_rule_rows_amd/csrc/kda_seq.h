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

// Inclusive running folds over the lanes of a wave, f(before, mine), without LDS: within rows of 16 lanes by
// shifts, then over the rows.  A lane that a step does not reach gets `none`.
template <int CTRL, int ROWS>
__device__ __forceinline__ int lane_step(int none, int x) {
    return __builtin_amdgcn_update_dpp(none, x, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float lane_step(float none, float x) {
    return __builtin_bit_cast(float, lane_step<CTRL, ROWS>(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x)));
}

template <int CTRL, int ROWS, typename T64>
__device__ __forceinline__ T64 lane_step(T64 none, T64 x) {
    static_assert(sizeof(T64) == 8, "two words");
    const long long n = __builtin_bit_cast(long long, none), y = __builtin_bit_cast(long long, x);
    const uint32_t lo = lane_step<CTRL, ROWS>(static_cast<int>(n), static_cast<int>(y));
    const uint32_t hi = lane_step<CTRL, ROWS>(static_cast<int>(n >> 32), static_cast<int>(y >> 32));
    return __builtin_bit_cast(T64, static_cast<long long>(static_cast<unsigned long long>(hi) << 32 | lo));
}

template <typename T, typename F>
__device__ __forceinline__ T running(T x, T none, F&& f) {
    x = f(lane_step<0x111, 0xF>(none, x), x);   // row_shr:1, 2, 4, 8
    x = f(lane_step<0x112, 0xF>(none, x), x);
    x = f(lane_step<0x114, 0xF>(none, x), x);
    x = f(lane_step<0x118, 0xF>(none, x), x);
    x = f(lane_step<0x142, 0xA>(none, x), x);   // row_bcast:15 into rows 1 and 3
    return f(lane_step<0x143, 0xC>(none, x), x);   // row_bcast:31 into rows 2 and 3
}

// The value of one lane in all.
template <typename T>
__device__ __forceinline__ T of_lane(T x, int lane) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
    } else {
        const long long y = __builtin_bit_cast(long long, x);
        const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(y), lane), hi = __builtin_amdgcn_readlane(static_cast<int>(y >> 32), lane);
        return __builtin_bit_cast(T, static_cast<long long>(static_cast<unsigned long long>(hi) << 32 | lo));
    }
}

template <typename T>
__device__ __forceinline__ T running_sum(T x) {
    return running(x, T(0), [](T a, T b) { return a + b; });
}

__device__ __forceinline__ int running_max(int x) {
    return running(x, -2147483647 - 1, [](int a, int b) { return max(a, b); });
}

// The value of the lane before; `first` in lane 0.
__device__ __forceinline__ int lane_before(int x, int first) {
    const int y = __shfl_up(x, 1);
    return (threadIdx.x & 63) == 0 ? first : y;
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
        const int ahead = lane_before(upto, 0);
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
    first = of_lane(running_max(x), 63);
    last = min(max(a.offsets[b + 1], first), a.R);
}

}  // namespace
}  // namespace kda
