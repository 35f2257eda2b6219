// Host-side argument checks shared by the C-ABI files.  A refusal formats its
// message into the calling thread's kda_last_error() buffer and returns the
// KDA_ERR_* status; nothing here touches the device.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "kda.h"

namespace kda {

inline thread_local char g_err[512] = "";   // message of the last refusal

inline int refuse(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

// A byte range [p, p + n) of device memory, with the alignment it needs.
struct Span {
    const char* name;
    const void* ptr;
    unsigned long long n;
    unsigned align;
    bool optional;   // may be NULL
};

inline uintptr_t addr(const Span& s) { return reinterpret_cast<uintptr_t>(s.ptr); }

inline bool overlap(const Span& a, const Span& b) {
    if (!a.ptr || !b.ptr || a.n == 0 || b.n == 0) return false;
    return addr(a) < addr(b) + b.n && addr(b) < addr(a) + a.n;
}

inline int check_spans(const char* fn, const Span* s, int n) {
    for (int i = 0; i < n; ++i) {
        if (!s[i].ptr) {
            if (s[i].optional) continue;
            return refuse(KDA_ERR_ARG, "%s: %s is NULL", fn, s[i].name);
        }
        if (addr(s[i]) % s[i].align != 0)
            return refuse(KDA_ERR_ALIGN, "%s: %s is not %u-byte aligned", fn, s[i].name, s[i].align);
    }
    return KDA_OK;
}

// No output may overlap an input or another output.  `same_out`/`same_in`
// name one (output, input) pair that may be the identical buffer (a state
// updated in place); a partial overlap of that pair is still refused.
inline int check_alias(const char* fn, const Span* out, int n_out, const Span* in, int n_in,
                       const Span* same_out = nullptr, const Span* same_in = nullptr) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j) {
            const bool pair = &out[i] == same_out && &in[j] == same_in;
            if (pair && out[i].ptr == in[j].ptr) continue;
            if (overlap(out[i], in[j])) {
                if (pair)
                    return refuse(KDA_ERR_ALIAS, "%s: %s partially overlaps %s", fn, out[i].name,
                                  in[j].name);
                return refuse(KDA_ERR_ALIAS, "%s: %s overlaps %s", fn, out[i].name, in[j].name);
            }
        }
        for (int j = i + 1; j < n_out; ++j) {
            if (overlap(out[i], out[j]))
                return refuse(KDA_ERR_ALIAS, "%s: %s overlaps %s", fn, out[i].name, out[j].name);
        }
    }
    return KDA_OK;
}

inline int check_counts(const char* fn, long long L, long long H) {
    if (L < 1) return refuse(KDA_ERR_RANGE, "%s: L=%lld, need L >= 1", fn, L);
    if (H < 1) return refuse(KDA_ERR_RANGE, "%s: H=%lld, need H >= 1", fn, H);
    if (L * H > INT_MAX) return refuse(KDA_ERR_RANGE, "%s: L*H=%lld too large", fn, L * H);
    return KDA_OK;
}

inline int check_dtype(const char* fn, int in_dtype) {
    if (in_dtype != KDA_IN_F32 && in_dtype != KDA_IN_BF16)
        return refuse(KDA_ERR_ARG, "%s: in_dtype=%d is neither KDA_IN_F32 nor KDA_IN_BF16", fn,
                      in_dtype);
    return KDA_OK;
}

inline int check_rows(const char* fn, const char* what, int T) {
    if (T < 1 || T > KDA_T_MAX)
        return refuse(KDA_ERR_RANGE, "%s: %s=%d outside 1..%d (K+1 verify rows, K <= 14)", fn, what,
                      T, KDA_T_MAX);
    return KDA_OK;
}

inline int launched(const char* fn, hipError_t e) {
    if (e != hipSuccess) return refuse(KDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
    g_err[0] = '\0';
    return KDA_OK;
}

}  // namespace kda
