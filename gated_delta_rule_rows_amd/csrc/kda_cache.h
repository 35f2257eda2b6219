// Internal interface between kda_cache_abi.cpp and the kernels of the paged
// cache, of the attention that reads it and of the sampled accept
// (kda_attn.hip, kda_sample.hip), with what host and device compute alike.
// Not installed; callers use include/kda.h.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace kda {

// The cache as kda_cache describes it; strides in elements.
struct CacheView {
    void* k;
    void* v;
    const int32_t* table;     // [B][seq_pages]
    const int32_t* lens;      // B
    long long page_stride;
    long long row_stride;
    long long head_stride;
    int pages;
    int page_shift;           // rows of a page = 1 << page_shift
    int seq_pages;
};

// Element offset of the row at position pos of a sequence whose table entry for
// that page is `entry` (head 0); -1 where the entry names no page.
__host__ __device__ inline long long cache_at(const CacheView& c, int entry, int pos) {
    if (entry < 0 || entry >= c.pages) return -1;
    return entry * c.page_stride + (pos & ((1 << c.page_shift) - 1)) * c.row_stride;
}

// Position of row `row` of a sequence that ends (not included) at row `last`.
// A length below zero counts as zero.
__host__ __device__ inline int cache_pos(int len, int row, int last) { return (len > 0 ? len : 0) - (last - row); }

// The tiles of KT keys that rows at positions lo .. hi (lo <= hi) can see:
// tiles 0 .. first-1 (the first keys that stay visible), then from .. from +
// count - first - 1.
struct KeyTiles {
    int count;
    int first;
    int from;
};

__host__ __device__ inline KeyTiles key_tiles(int lo, int hi, int capacity, int window, int sinks, int kt) {
    const int keys = hi + 1 < capacity ? hi + 1 : capacity;
    if (keys <= 0) return KeyTiles{0, 0, 0};
    const int end = (keys - 1) / kt + 1;
    const long long low = window > 0 ? static_cast<long long>(lo) - window + 1 : 0;
    int from = low > 0 ? static_cast<int>(low < keys ? low : keys) / kt : 0;
    if (from > end) from = end;
    const int s = sinks < keys ? sinks : keys;
    int first = s > 0 ? (s - 1) / kt + 1 : 0;
    if (first > from) first = from;
    return KeyTiles{end - from + first, first, from};
}

struct AppendArgs {
    CacheView c;
    const void* k;            // [R][Hk][128], rows k_ld elements apart
    const void* v;
    long long k_ld;
    long long v_ld;
    const int32_t* offsets;   // B + 1
    int R;
    int B;
    int Hk;
};

hipError_t launch_append(const AppendArgs& a, bool bf16, hipStream_t stream);

struct AttnArgs {
    CacheView c;
    const void* q;            // [R][H][128], rows q_ld elements apart
    long long q_ld;
    const int32_t* offsets;   // B + 1
    void* o;                  // [R][H][128] in the type of q
    void* work;
    int R;
    int B;
    int H;
    int Hk;
    float scale;
    int window;               // 0: none
    int sinks;
};

long long attn_work_bytes(int R, int B, int H, int Hk);
long long attn_workgroups(int R, int B, int H, int Hk);   // of the largest grid of such a call
hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t stream);

struct SampledArgs {
    const void* logits;       // row r at element r * ld
    long long ld;
    const float* probs;       // row r at element r * probs_ld, or null
    long long probs_ld;
    const int32_t* offsets;   // B + 1
    const uint32_t* drafts;   // R
    const float* u;           // R
    const float* temp;        // B, or null
    uint32_t* out;            // [B][2]
    float* p_draft;           // R, or null
    void* work;
    int R;
    int B;
    int V;
};

long long sampled_work_bytes(int R, int B, int V);
long long sampled_workgroups(int R, int B, int V);   // of the largest grid of such a call
hipError_t launch_sampled(const SampledArgs& a, bool bf16, hipStream_t stream);

}  // namespace kda
