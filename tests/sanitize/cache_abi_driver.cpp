// Drives kda_cache_abi.cpp's validation on the host, with the launchers
// replaced by stubs that record the call, and checks against brute force what
// the kernels share with the host: where a row of the cache lies (pages that do
// not exist among them) and which tiles of keys a tile of rows reads.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <string>
#include <thread>
#include <vector>

#include "kda.h"
#include "kda_cache.h"
#include "kda_check.h"

static int launches = 0;
static kda::CacheView seen;

namespace kda {
long long attn_work_bytes(int R, int B, int H, int) { return 64ll * (R + B) * H; }
long long attn_workgroups(int R, int B, int H, int Hk) { return (static_cast<long long>(R) / (H / Hk) + B) * Hk; }
long long sampled_work_bytes(int R, int B, int) { return 16ll * (R + B); }
long long sampled_workgroups(int R, int B, int) { return static_cast<long long>(R) + B; }
hipError_t launch_append(const AppendArgs& a, bool, hipStream_t) { ++launches; seen = a.c; return a.Hk == 7 ? hipErrorInvalidValue : hipSuccess; }
hipError_t launch_attn(const AttnArgs& a, bool, hipStream_t) { ++launches; seen = a.c; return hipSuccess; }
hipError_t launch_sampled(const SampledArgs&, bool, hipStream_t) { ++launches; return hipSuccess; }
}  // namespace kda

extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

static int bad = 0;

static void expect(long long got, long long want, const char* what) {
    if (got != want) {
        std::printf("FAIL %s: %lld, want %lld (%s)\n", what, got, want, kda::g_err);
        ++bad;
    }
}

static void* at(uintptr_t i) { return reinterpret_cast<void*>(uintptr_t{0x10000000} + i * (uintptr_t{1} << 44)); }

static kda_cache cache(int pages, int rows, int seq_pages, int heads) {
    kda_cache c{};
    c.k = at(1); c.v = at(2);
    c.table = static_cast<const int32_t*>(at(3)); c.lens = static_cast<const int32_t*>(at(4));
    c.head_stride = 128; c.row_stride = 128ll * heads; c.page_stride = c.row_stride * rows;
    c.pages = pages; c.page_rows = rows; c.seq_pages = seq_pages;
    return c;
}

// Every key of a tile that is not read must be one that no row sees, and no tile is read twice.
static void tiles(int lo, int hi, int capacity, int window, int sinks, int kt) {
    const kda::KeyTiles t = kda::key_tiles(lo, hi, capacity, window, sinks, kt);
    const int all = capacity / kt + 2;
    std::vector<int> read(all, 0);
    bool inside = t.count >= 0 && t.first >= 0 && t.first <= t.count;
    for (int i = 0; i < t.count && inside; ++i) {
        const int tile = i < t.first ? i : i - t.first + t.from;
        inside = tile >= 0 && tile < all && read[tile]++ == 0 && static_cast<long long>(tile) * kt < capacity && tile * kt <= hi;
    }
    bool whole = true;
    for (int p = lo; p <= hi; ++p)
        for (int j = 0; j <= p && j < capacity; ++j)
            if (window == 0 || j > p - window || j < sinks) whole = whole && read[j / kt] == 1;
    if (!inside || !whole) {
        std::printf("FAIL tiles lo %d hi %d capacity %d window %d sinks %d kt %d: count %d first %d from %d\n", lo, hi, capacity,
                    window, sinks, kt, t.count, t.first, t.from);
        ++bad;
    }
}

int main() {
    const int F32 = KDA_IN_F32, BF16 = KDA_IN_BF16;
    auto *x = at(5), *y = at(6), *o = at(8), *work = at(9);
    auto* off = static_cast<const int32_t*>(at(7));
    const long long big = 1ll << 39;
    kda_cache c = cache(10, 64, 6, 2);
    expect(kda_cache_append(x, 256, y, 640, &c, off, 40, 3, 2, BF16, nullptr), KDA_OK, "append");
    expect(seen.page_shift, 6, "shift");
    expect(kda_cache_append(x, 0, y, -5, &c, off, 1, 3, 2, F32, nullptr), KDA_OK, "one row has no stride");
    expect(kda_cache_append(nullptr, 0, nullptr, 0, &c, off, 0, 3, 2, F32, nullptr), KDA_OK, "no rows");
    expect(kda_cache_append(x, 256, y, 256, nullptr, off, 40, 3, 2, F32, nullptr), KDA_ERR_ARG, "no cache");
    kda_cache seven = cache(10, 64, 6, 7);
    expect(kda_cache_append(x, 896, y, 896, &seven, off, 40, 3, 7, F32, nullptr), KDA_ERR_HIP, "failed launch");
    kda_cache one = cache(10, 1, 6, 1);
    expect(kda_attn_rows(x, 512, &one, off, o, 40, 3, 4, 1, 0.1f, 0, 0, F32, work, big, nullptr), KDA_OK, "attn");
    expect(seen.page_shift, 0, "shift of one row");
    expect(kda_attn_rows(x, 512, &c, off, o, 40, 3, 4, 2, 0.1f, 7, 3, BF16, work, big, nullptr), KDA_OK, "attn window");
    expect(kda_attn_rows(x, 512, &c, off, o, 40, 3, 4, 2, 0.1f, 0, 3, BF16, work, big, nullptr), KDA_ERR_RANGE, "sinks alone");
    expect(kda_attn_rows(x, 512, &c, off, o, 40, 3, 4, 2, 0.1f, 0, 0, BF16, work, 64 * 43 * 4 - 1, nullptr), KDA_ERR_RANGE, "small work");
    expect(kda_attn_rows(x, 512, &c, off, o, KDA_PROMPT_ROWS_MAX, 3, 4, 2, 0.1f, 0, 0, BF16, work, big, nullptr), KDA_ERR_RANGE, "too many");
    kda_cache huge = cache(2147483647, 65536, 32767, 65535);
    expect(kda_attn_rows(x, 65535 * 128ll, &huge, off, o, 4, 3, 65535, 65535, 0.1f, 0, 0, BF16, work, big, nullptr), KDA_ERR_RANGE, "huge cache");
    auto* d = static_cast<uint32_t*>(at(10));
    auto *u = static_cast<float*>(at(11)), *t = static_cast<float*>(at(12)), *p = static_cast<float*>(at(13));
    auto* out = static_cast<uint32_t*>(at(14));
    expect(kda_accept_sampled(x, 100, BF16, u, 100, off, d, u, t, out, p, 9, 3, 100, work, big, nullptr), KDA_OK, "sampled");
    expect(kda_accept_sampled(x, 100, BF16, nullptr, -3, off, d, u, nullptr, out, nullptr, 9, 3, 100, work, big, nullptr), KDA_OK, "no probabilities");
    expect(kda_accept_sampled(x, 5, BF16, u, 5, off, d, u, t, out, p, 1, 3, 100, work, big, nullptr), KDA_OK, "one row");
    expect(kda_accept_sampled(x, 100, BF16, u, 99, off, d, u, t, out, p, 9, 3, 100, work, big, nullptr), KDA_ERR_RANGE, "probs_ld");
    expect(kda_accept_sampled(x, 100, BF16, u, 100, off, d, u, t, out, t, 9, 3, 100, work, big, nullptr), KDA_ERR_ALIAS, "alias");
    expect(launches, 8, "launches");

    // places in the cache
    kda::CacheView v{};
    v.pages = 5; v.page_shift = 3; v.page_stride = 1ll << 33; v.row_stride = 1000;
    for (int entry : {-2147483647 - 1, -1, 5, 2147483647}) expect(kda::cache_at(v, entry, 12), -1, "no page");
    expect(kda::cache_at(v, 4, 21), (4ll << 33) + 5000, "place");
    expect(kda::cache_at(v, 0, 2147483647), 7000, "last row");
    expect(kda::cache_pos(10, 3, 5), 8, "position");
    expect(kda::cache_pos(-2147483647 - 1, 0, KDA_PROMPT_ROWS_MAX), -KDA_PROMPT_ROWS_MAX, "negative length");
    expect(kda::cache_pos(2147483647, 0, 1), 2147483646, "longest");

    for (int kt : {4, 32})
        for (int capacity : {1, 5, 32, 70, 131})
            for (int lo = -9; lo < 140; lo += 7)
                for (int rows : {1, 2, 9, 33})
                    for (int window : {0, 1, 3, 31, 64, 2147483647})
                        for (int sinks : {0, 1, 5, 40, 2147483647})
                            if (window > 0 || sinks == 0) tiles(lo, lo + rows - 1, capacity, window, sinks, kt);
    // at the ends of the range: no overflow (the sanitizer watches), tiles within the keys
    for (int hi : {-1, 0, 2147483645, 2147483646})
        for (int window : {0, 1, 2147483647}) {
            const kda::KeyTiles k = kda::key_tiles(hi > 100 ? hi - 100 : -268435456, hi, 2147483647, window, window ? 2147483647 : 0, 32);
            if (k.count < 0 || k.first < 0 || k.from < 0) ++bad;
        }

    std::vector<std::thread> threads;
    bool mine[2] = {false, false};
    for (int i = 0; i < 2; ++i)
        threads.emplace_back([&, i] {
            bool ok = true;
            for (int n = 0; n < 2000; ++n) {
                if (i == 0) kda_cache_append(x, 256, y, 256, &c, off, -1, 3, 2, F32, nullptr);
                else kda_accept_sampled(x, 100, F32, nullptr, 0, off, d, u, t, out, p, 9, 0, 100, work, big, nullptr);
                ok = ok && std::strstr(kda::g_err, i == 0 ? "kda_cache_append: R=-1" : "kda_accept_sampled: B=0");
            }
            mine[i] = ok;
        });
    for (auto& th : threads) th.join();
    if (!mine[0] || !mine[1]) {
        std::printf("FAIL messages of two threads\n");
        ++bad;
    }
    if (!bad) std::printf("OK\n");
    return bad != 0;
}
