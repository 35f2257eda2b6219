// C ABI of the paged cache, the attention that reads it and the sampled accept:
// host-side argument validation, then one enqueue, as in kda_abi.cpp.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <utility>

#include "kda.h"
#include "kda_cache.h"
#include "kda_check.h"
#include "kda_launch.h"

using namespace kda;

namespace {

constexpr long long kStrideMax = 1ll << 40;     // elements
constexpr float kScaleMax = 2e38f;              // times log2(e) it has to be finite in f32: scores are kept in base 2
constexpr long long kGridMax = 1ll << 24;       // workgroups of 256 threads: 2^32 threads

int check_packed(const char* fn, int R, int B) {
    if (R < 0 || R > KDA_PROMPT_ROWS_MAX)
        return refuse(KDA_ERR_RANGE, "%s: R=%d outside 0..%d", fn, R, KDA_PROMPT_ROWS_MAX);
    if (B < 1 || B > KDA_PROMPT_SEQS_MAX)
        return refuse(KDA_ERR_RANGE, "%s: B=%d outside 1..%d", fn, B, KDA_PROMPT_SEQS_MAX);
    return KDA_OK;
}

int check_heads(const char* fn, int H, int Hk) {
    if (H < 1 || H > 65535) return refuse(KDA_ERR_RANGE, "%s: H=%d outside 1..65535", fn, H);
    if (Hk < 1 || H % Hk != 0)
        return refuse(KDA_ERR_RANGE, "%s: Hk=%d must be >= 1 and divide H=%d", fn, Hk, H);
    return KDA_OK;
}

// Rows of `heads` heads, ld elements apart (one row has no stride).
int check_ld(const char* fn, const char* name, int R, int heads, unsigned es, long long* ld) {
    const long long row = static_cast<long long>(heads) * kD;
    if (R <= 1) *ld = row;
    if (*ld < row) return refuse(KDA_ERR_RANGE, "%s: %s=%lld < %lld (rows would overlap)", fn, name, *ld, row);
    if (R > 0 && *ld > kStrideMax / R) return refuse(KDA_ERR_RANGE, "%s: %s=%lld too large for R=%d", fn, name, *ld, R);
    if (*ld % (16 / es) != 0)
        return refuse(KDA_ERR_ALIGN, "%s: rows %s=%lld elements apart are not 16-byte aligned", fn, name, *ld);
    return KDA_OK;
}

struct Axis {
    long long stride, count;
};

// Whether no two index combinations of the axes meet (`row` elements each), by
// nesting: each stride clears all that the smaller ones reach.
bool nested(Axis* axes, int n, long long row) {
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (axes[j].stride < axes[i].stride) std::swap(axes[i], axes[j]);
    long long reach = row;
    for (int i = 0; i < n; ++i) {
        if (axes[i].count <= 1) continue;
        if (axes[i].stride < reach) return false;
        reach += axes[i].stride * (axes[i].count - 1);
    }
    return true;
}

// The cache's description, as a view; its extent in bytes in *bytes.
int check_cache(const char* fn, const kda_cache* c, int B, int Hk, unsigned es, CacheView* v, unsigned long long* bytes) {
    if (!c) return refuse(KDA_ERR_ARG, "%s: cache is NULL", fn);
    if (c->pages < 1) return refuse(KDA_ERR_RANGE, "%s: cache.pages=%d, need >= 1", fn, c->pages);
    if (c->page_rows < 1 || (c->page_rows & (c->page_rows - 1)) != 0 || c->page_rows > KDA_PAGE_ROWS_MAX)
        return refuse(KDA_ERR_RANGE, "%s: cache.page_rows=%d is no power of two in 1..%d", fn, c->page_rows, KDA_PAGE_ROWS_MAX);
    if (c->seq_pages < 1 || static_cast<long long>(c->seq_pages) * c->page_rows > 1ll << 30)
        return refuse(KDA_ERR_RANGE, "%s: cache.seq_pages=%d: need 1 .. 2^30 rows in a sequence", fn, c->seq_pages);
    // (one page, row or head has no stride)
    Axis axes[3] = {{c->pages > 1 ? c->page_stride : 0, c->pages},
                    {c->page_rows > 1 ? c->row_stride : 0, c->page_rows},
                    {Hk > 1 ? c->head_stride : 0, Hk}};
    v->page_stride = axes[0].stride; v->row_stride = axes[1].stride; v->head_stride = axes[2].stride;
    long long last = kD;
    for (const Axis& x : axes) {
        if (x.stride < 0 || x.stride > kStrideMax || (x.count > 1 && x.stride > kStrideMax / (x.count - 1)))
            return refuse(KDA_ERR_RANGE, "%s: a cache stride of %lld elements is negative or too large", fn, x.stride);
        if (x.stride % (16 / es) != 0)
            return refuse(KDA_ERR_ALIGN, "%s: a cache stride of %lld elements is not 16-byte aligned", fn, x.stride);
        last += x.stride * (x.count - 1);
    }
    if (last > kStrideMax) return refuse(KDA_ERR_RANGE, "%s: the cache's extent is too large", fn);
    if (!nested(axes, 3, kD)) return refuse(KDA_ERR_RANGE, "%s: rows of the cache overlap by its strides", fn);
    *bytes = static_cast<unsigned long long>(last) * es;
    const Span spans[] = {
        {"cache.k", c->k, *bytes, 16, false},
        {"cache.v", c->v, *bytes, 16, false},
        {"cache.table", c->table, static_cast<unsigned long long>(B) * c->seq_pages * 4, 4, false},
        {"cache.lens", c->lens, B * 4ull, 4, false},
    };
    int rc;
    if ((rc = check_spans(fn, spans, 4))) return rc;
    v->k = c->k; v->v = c->v; v->table = c->table; v->lens = c->lens;
    v->pages = c->pages;
    v->page_shift = __builtin_ctz(static_cast<unsigned>(c->page_rows));
    v->seq_pages = c->seq_pages;
    return KDA_OK;
}

// Keys and values may share a buffer (each page, row or head with both), if no
// row of one meets a row of the other.
int check_apart(const char* fn, const kda_cache* c, int Hk, unsigned es, unsigned long long bytes) {
    const uintptr_t k = reinterpret_cast<uintptr_t>(c->k), v = reinterpret_cast<uintptr_t>(c->v);
    const uintptr_t apart = k < v ? v - k : k - v;
    if (apart >= bytes) return KDA_OK;
    Axis axes[4] = {{c->page_stride, c->pages}, {c->row_stride, c->page_rows}, {c->head_stride, Hk},
                    {static_cast<long long>(apart / es), 2}};
    if (apart % es != 0 || !nested(axes, 4, kD))
        return refuse(KDA_ERR_ALIAS, "%s: cache.k and cache.v overlap", fn);
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_cache_append(const void* k, long long k_ld, const void* v, long long v_ld, const kda_cache* cache,
                     const int32_t* offsets, int R, int B, int Hk, int in_dtype, void* stream) {
    const char* fn = "kda_cache_append";
    int rc;
    if ((rc = check_dtype(fn, in_dtype)) || (rc = check_heads(fn, Hk, Hk)) || (rc = check_packed(fn, R, B))) return rc;
    const unsigned es = in_dtype == KDA_IN_BF16 ? 2 : 4;
    if (static_cast<long long>(R) + B >= kGridMax)
        return refuse(KDA_ERR_RANGE, "%s: R=%d too large", fn, R);
    AppendArgs a{};
    unsigned long long bytes = 0;
    if ((rc = check_ld(fn, "k_ld", R, Hk, es, &k_ld)) || (rc = check_ld(fn, "v_ld", R, Hk, es, &v_ld)) ||
        (rc = check_cache(fn, cache, B, Hk, es, &a.c, &bytes)) || (rc = check_apart(fn, cache, Hk, es, bytes)))
        return rc;
    const bool none = R == 0;   // empty tensors have no address
    const unsigned long long rows = none ? 0 : static_cast<unsigned long long>(R - 1), row = static_cast<unsigned long long>(Hk) * kD;
    const Span in[] = {
        {"k", k, none ? 0 : (rows * k_ld + row) * es, 16, none},
        {"v", v, none ? 0 : (rows * v_ld + row) * es, 16, none},
        {"offsets", offsets, (B + 1) * 4ull, 4, false},
        {"cache.table", cache->table, static_cast<unsigned long long>(B) * cache->seq_pages * 4, 4, false},
        {"cache.lens", cache->lens, B * 4ull, 4, false},
    };
    const Span out_k = {"cache.k", cache->k, bytes, 16, false}, out_v = {"cache.v", cache->v, bytes, 16, false};
    if ((rc = check_spans(fn, in, 5)) || (rc = check_alias(fn, &out_k, 1, in, 5)) ||
        (rc = check_alias(fn, &out_v, 1, in, 5)))
        return rc;
    if (none) return launched(fn, hipSuccess);
    a.k = k; a.v = v; a.k_ld = k_ld; a.v_ld = v_ld; a.offsets = offsets; a.R = R; a.B = B; a.Hk = Hk;
    return launched(fn, launch_append(a, in_dtype == KDA_IN_BF16, static_cast<hipStream_t>(stream)));
}

long long kda_attn_rows_work_bytes(int R, int B, int H, int Hk) {
    const char* fn = "kda_attn_rows_work_bytes";
    if (check_heads(fn, H, Hk) || check_packed(fn, R, B)) return -1;
    return attn_work_bytes(R, B, H, Hk);
}

int kda_attn_rows(const void* q, long long q_ld, const kda_cache* cache, const int32_t* offsets, void* o, int R,
                  int B, int H, int Hk, float scale, int window, int sinks, int in_dtype, void* work,
                  long long work_bytes, void* stream) {
    const char* fn = "kda_attn_rows";
    int rc;
    if ((rc = check_dtype(fn, in_dtype)) || (rc = check_heads(fn, H, Hk)) || (rc = check_packed(fn, R, B))) return rc;
    if (!(scale > 0.f) || !(scale <= kScaleMax))
        return refuse(KDA_ERR_RANGE, "%s: scale=%g is no positive number up to %g", fn, static_cast<double>(scale),
                      static_cast<double>(kScaleMax));
    if (window < 0) return refuse(KDA_ERR_RANGE, "%s: window=%d, need >= 0 (0: none)", fn, window);
    if (sinks < 0 || (sinks > 0 && window == 0))
        return refuse(KDA_ERR_RANGE, "%s: sinks=%d: need >= 0, and 0 without a window", fn, sinks);
    if (attn_workgroups(R, B, H, Hk) >= kGridMax)
        return refuse(KDA_ERR_RANGE, "%s: R=%d rows of H=%d heads are too many", fn, R, H);
    const unsigned es = in_dtype == KDA_IN_BF16 ? 2 : 4;
    AttnArgs a{};
    unsigned long long bytes = 0;
    if ((rc = check_ld(fn, "q_ld", R, H, es, &q_ld)) || (rc = check_cache(fn, cache, B, Hk, es, &a.c, &bytes))) return rc;
    const long long need = attn_work_bytes(R, B, H, Hk);
    if (work_bytes < need) return refuse(KDA_ERR_RANGE, "%s: work_bytes=%lld, need %lld", fn, work_bytes, need);
    const bool none = R == 0;
    const unsigned long long row = static_cast<unsigned long long>(H) * kD;
    const Span in[] = {
        {"q", q, none ? 0 : (static_cast<unsigned long long>(R - 1) * q_ld + row) * es, 16, none},
        {"offsets", offsets, (B + 1) * 4ull, 4, false},
        {"cache.k", cache->k, bytes, 16, false},
        {"cache.v", cache->v, bytes, 16, false},
        {"cache.table", cache->table, static_cast<unsigned long long>(B) * cache->seq_pages * 4, 4, false},
        {"cache.lens", cache->lens, B * 4ull, 4, false},
    };
    const Span out[] = {
        {"o", o, R * row * es, 16, none},
        {"work", work, static_cast<unsigned long long>(need), 16, need == 0},
    };
    if ((rc = check_spans(fn, in, 6)) || (rc = check_spans(fn, out, 2)) || (rc = check_alias(fn, out, 2, in, 6)))
        return rc;
    if (none) return launched(fn, hipSuccess);
    a.q = q; a.q_ld = q_ld; a.offsets = offsets; a.o = o; a.work = work;
    a.R = R; a.B = B; a.H = H; a.Hk = Hk; a.scale = scale; a.window = window; a.sinks = sinks;
    return launched(fn, launch_attn(a, in_dtype == KDA_IN_BF16, static_cast<hipStream_t>(stream)));
}

long long kda_accept_sampled_work_bytes(int R, int B, int V) {
    const char* fn = "kda_accept_sampled_work_bytes";
    if (check_packed(fn, R, B)) return -1;
    if (V < 1 || V > 1 << 30) {
        refuse(KDA_ERR_RANGE, "%s: V=%d outside 1..2^30", fn, V);
        return -1;
    }
    return R == 0 ? 0 : sampled_work_bytes(R, B, V);
}

int kda_accept_sampled(const void* logits, long long ld, int in_dtype, const float* probs, long long probs_ld,
                       const int32_t* offsets, const uint32_t* drafts, const float* u, const float* temp,
                       uint32_t* out, float* p_draft, int R, int B, int V, void* work, long long work_bytes,
                       void* stream) {
    const char* fn = "kda_accept_sampled";
    int rc;
    if ((rc = check_dtype(fn, in_dtype)) || (rc = check_packed(fn, R, B))) return rc;
    if (V < 1 || V > 1 << 30) return refuse(KDA_ERR_RANGE, "%s: V=%d outside 1..2^30", fn, V);
    if (R <= 1) ld = probs_ld = V;
    if (ld < V) return refuse(KDA_ERR_RANGE, "%s: ld=%lld < V=%d (rows would overlap)", fn, ld, V);
    if (!probs) probs_ld = V;
    if (probs_ld < V) return refuse(KDA_ERR_RANGE, "%s: probs_ld=%lld < V=%d (rows would overlap)", fn, probs_ld, V);
    if (R > 0 && (ld > kStrideMax / R || probs_ld > kStrideMax / R))
        return refuse(KDA_ERR_RANGE, "%s: ld=%lld, probs_ld=%lld too large for R=%d", fn, ld, probs_ld, R);
    const bool none = R == 0;
    const long long need = none ? 0 : sampled_work_bytes(R, B, V);
    if (sampled_workgroups(R, B, V) >= kGridMax) return refuse(KDA_ERR_RANGE, "%s: R=%d too large", fn, R);
    if (work_bytes < need) return refuse(KDA_ERR_RANGE, "%s: work_bytes=%lld, need %lld", fn, work_bytes, need);
    const unsigned es = in_dtype == KDA_IN_BF16 ? 2 : 4;
    const unsigned long long rows = static_cast<unsigned long long>(R), gaps = none ? 0 : rows - 1;
    const Span in[] = {
        {"logits", logits, none ? 0 : (gaps * ld + V) * es, es, none},
        {"probs", probs, none ? 0 : (gaps * probs_ld + V) * 4, 4, true},
        {"offsets", offsets, (B + 1) * 4ull, 4, false},
        {"drafts", drafts, rows * 4, 4, none},
        {"u", u, rows * 4, 4, none},
        {"temp", temp, B * 4ull, 4, true},
    };
    const Span out_[] = {
        {"out", out, B * 8ull, 4, false},
        {"p_draft", p_draft, rows * 4, 4, true},
        {"work", work, static_cast<unsigned long long>(need), 16, need == 0},
    };
    if ((rc = check_spans(fn, in, 6)) || (rc = check_spans(fn, out_, 3)) || (rc = check_alias(fn, out_, 3, in, 6)))
        return rc;
    if (none) return launched(fn, hipSuccess);
    SampledArgs a{};
    a.logits = logits; a.ld = ld; a.probs = probs; a.probs_ld = probs_ld; a.offsets = offsets; a.drafts = drafts;
    a.u = u; a.temp = temp; a.out = out; a.p_draft = p_draft; a.work = work; a.R = R; a.B = B; a.V = V;
    return launched(fn, launch_sampled(a, in_dtype == KDA_IN_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
