// Argument checks and workspace of the C calls (host code shared by the api sources).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/selscan.h"

namespace selscan {

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t st);
hipError_t launch_fill(float* p, float v, int64_t n, hipStream_t st);
hipError_t launch_copy_f32(float* dst, const float* src, int64_t n, hipStream_t st);

inline bool aligned16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
    uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
};
inline Span span(const void* p, int64_t bytes) {
    Span s;
    if (p && bytes > 0) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + uintptr_t(bytes);
    }
    return s;
}
inline bool overlaps(const Span& a, const Span& b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

// Neither infinite nor a NaN.
inline bool finite_f32(float v) { return v - v == 0.0f; }

// dst = src (zeros without one), in pieces: a grid has fewer than 2^32 threads.
inline hipError_t pass_state(float* dst, const float* src, int64_t n, hipStream_t st) {
    const int64_t piece = int64_t(1) << 30;
    hipError_t e = hipSuccess;
    for (int64_t i = 0; dst && i < n && e == hipSuccess; i += piece) {
        const int64_t m = n - i < piece ? n - i : piece;
        e = src ? launch_copy_f32(dst + i, src + i, m, st) : launch_fill_zero(dst + i, m, st);
    }
    return e;
}

// The caller's workspace, or one taken on the stream.
struct Workspace {
    void* p = nullptr;
    bool own = false;
    int take(void* given, size_t bytes, hipStream_t st) {
        p = given;
        if (p || !bytes) return SELSCAN_OK;
        if (hipMallocAsync(&p, bytes, st) != hipSuccess || !p) {
            (void)hipGetLastError();
            return SELSCAN_ERR_ALLOC;
        }
        own = true;
        return SELSCAN_OK;
    }
    void give_back(hipStream_t st) {
        if (own) (void)hipFreeAsync(p, st);
    }
};

template <size_t NI, size_t NO>
bool any_alias(const Span (&ins)[NI], const Span (&outs)[NO]) {
    for (size_t i = 0; i < NO; ++i) {
        for (const Span& s : ins)
            if (overlaps(s, outs[i])) return true;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

}  // namespace selscan
