// Gated linear recurrence, its token step and its gradients.
//
// A token's decay a is held as a or as a - 1, whichever is smaller: formed without
// cancellation (a sigmoid, or the exponential's series), it keeps full relative
// accuracy of what is remembered where a is near 0, and of 1 - a, and with it of
// what the state settles to, where a is near 1.
#include "../../include/selscan.h"
#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

struct GaArgs {
    const void* x;
    const void* g;
    const void* r;
    const float* A;
    const void* z;
    const int32_t* lengths;
    const float* h0;
    void* y;
    float* last;
    float* ckpt;
    const void* dy;
    const float* dlast;
    void* dx;
    void* dg;
    void* dr;
    void* dz;
    float* dA_part;  // [batch][dim], null: not wanted
    float* dh0;
    int64_t B, L, D;
};

// sigmoid(v) and 1 - sigmoid(v), each to full relative accuracy.
struct Sig { float s, c; };
__device__ __forceinline__ Sig sigmoid2(float v) {
    const float t = exp2_hw(-fabsf(v) * kLog2e);
    const float w = rcp_hw(1.0f + t), m = t * w;
    return v >= 0.0f ? Sig{w, m} : Sig{m, w};
}

// A decay a in [0, 1], held so that it has full relative accuracy near 0 and 1 - a
// near 1: q is a itself (sign bit clear) or a - 1 (sign bit set), and p what is to
// be added, 0 or 1.
__device__ __forceinline__ float whole_of(float q) {
    return __int_as_float((__float_as_int(q) >> 31) & 0x3f800000);
}

// e^l for l <= 0 in that form. From -1/2 on, where a - 1 would cancel, a - 1 is the
// Taylor series up to l^8 / 8! (its rest is below 2^-26 of the sum).
__device__ __forceinline__ float decay_of(float l) {
    float s = 1.0f / 40320;
    s = fmaf(s, l, 1.0f / 5040);
    s = fmaf(s, l, 1.0f / 720);
    s = fmaf(s, l, 1.0f / 120);
    s = fmaf(s, l, 1.0f / 24);
    s = fmaf(s, l, 1.0f / 6);
    s = fmaf(s, l, 0.5f);
    return l < -0.5f ? exp2_hw(l * kLog2e) : -fabsf(fmaf(l * l, s, l));
}

// h after a token: a h + b.
__device__ __forceinline__ float step_of(float q, float p, float h, float b) {
    return fmaf(p, h, fmaf(q, h, b));
}

// A token of one channel: its decay, its input's weight f (b = f x), and what the gradients use.
struct Token {
    float q, p, f;
    Sig v, s;  // of g and r
    float w;   // sqrt(1 - a^2)
};
template <bool DECAY>
__device__ __forceinline__ Token token_of(float g, float r, float A) {
    Token k{};
    k.v = sigmoid2(g);
    if constexpr (!DECAY) {
        k.q = g > 0.0f ? k.v.c : -k.v.s;
        k.p = whole_of(k.q);
        k.f = k.v.s;
    } else {
        k.s = sigmoid2(r);
        k.q = decay_of(A * k.s.s);
        k.p = whole_of(k.q);
        k.w = __builtin_amdgcn_sqrtf(((1.0f - k.p) - k.q) * ((1.0f + k.p) + k.q));
        k.f = k.w * k.v.s;
    }
    return k;
}

// The channel's A, a NaN where it is above 0 (which has no sqrt(1 - a^2)).
__device__ __forceinline__ float rate_of(const float* A, int64_t d) {
    const float v = A[d];
    return v <= 0.0f ? v : __builtin_nanf("");
}

__device__ __forceinline__ int64_t entry_length(const int32_t* lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
}

template <typename T> __device__ __forceinline__ float at(const void* p, int64_t i) {
    return to_f32(static_cast<const T*>(p)[i]);
}
template <typename T> __device__ __forceinline__ void put(void* p, int64_t i, float v) {
    static_cast<T*>(p)[i] = from_f32<T>(v);
}

// One thread walks one channel of an entry.
template <typename T, bool DECAY>
__global__ __launch_bounds__(64) void fwd_kernel(GaArgs a) {
    const int64_t d = int64_t(blockIdx.x) * 64 + threadIdx.x, b = blockIdx.y;
    if (d >= a.D) return;
    const int64_t n = entry_length(a.lengths, b, a.L), row = b * a.D + d;
    const float A = DECAY ? rate_of(a.A, d) : 0.0f;
    double h = a.h0 ? a.h0[row] : 0.0;
    for (int64_t t = 0; t < a.L; ++t) {
        const int64_t i = (b * a.L + t) * a.D + d;
        if (a.ckpt && t % SELSCAN_GATED_CKPT == 0)
            a.ckpt[t / SELSCAN_GATED_CKPT * a.B * a.D + row] = float(h);
        if (t >= n) {
            if (a.y) put<T>(a.y, i, 0.0f);
            continue;
        }
        const Token k = token_of<DECAY>(at<T>(a.g, i), DECAY ? at<T>(a.r, i) : 0.0f, A);
        h = (double(k.p) + k.q) * h + double(k.f * at<T>(a.x, i));
        if (a.y) put<T>(a.y, i, a.z ? float(h) * silu(at<T>(a.z, i)) : float(h));
    }
    if (a.last) a.last[row] = float(h);
}

template <typename T, bool DECAY>
__global__ __launch_bounds__(64) void bwd_kernel(GaArgs a) {
    const int64_t d = int64_t(blockIdx.x) * 64 + threadIdx.x, b = blockIdx.y;
    if (d >= a.D) return;
    const int64_t n = entry_length(a.lengths, b, a.L), row = b * a.D + d;
    const float A = DECAY ? rate_of(a.A, d) : 0.0f;
    double C = a.dlast ? a.dlast[row] : 0.0, dA = 0.0;
    constexpr int64_t K = SELSCAN_GATED_CKPT;
    float before[K];
    for (int64_t t0 = (a.L - 1) / K * K; t0 >= 0; t0 -= K) {
        const int64_t t1 = t0 + K < a.L ? t0 + K : a.L;
        double h = a.ckpt[t0 / K * a.B * a.D + row];
        for (int64_t t = t0; t < t1 && t < n; ++t) {
            const int64_t i = (b * a.L + t) * a.D + d;
            const Token k = token_of<DECAY>(at<T>(a.g, i), DECAY ? at<T>(a.r, i) : 0.0f, A);
            before[t - t0] = float(h);
            h = (double(k.p) + k.q) * h + double(k.f * at<T>(a.x, i));
        }
        for (int64_t t = t1 - 1; t >= t0; --t) {
            const int64_t i = (b * a.L + t) * a.D + d;
            if (t >= n) {
                put<T>(a.dx, i, 0.0f);
                put<T>(a.dg, i, 0.0f);
                if (DECAY) put<T>(a.dr, i, 0.0f);
                if (a.z) put<T>(a.dz, i, 0.0f);
                continue;
            }
            const Token k = token_of<DECAY>(at<T>(a.g, i), DECAY ? at<T>(a.r, i) : 0.0f, A);
            const float x = at<T>(a.x, i), hb = before[t - t0];
            float dt = at<T>(a.dy, i);
            if (a.z) {
                const float z = at<T>(a.z, i), ha = step_of(k.q, k.p, hb, k.f * x);
                put<T>(a.dz, i, dt * ha * silu_grad(z));
                dt *= silu(z);
            }
            const float G = float(double(dt) + C);
            C = (double(k.p) + k.q) * G;
            put<T>(a.dx, i, G * k.f);
            if constexpr (!DECAY) {
                put<T>(a.dg, i, G * (x - hb) * (k.v.s * k.v.c));
            } else {
                put<T>(a.dg, i, G * k.w * x * (k.v.s * k.v.c));
                const float dec = k.p + k.q, ratio = k.w > 0.0f ? dec * rcp_hw(k.w) : 0.0f;
                const float dl = G * dec * (hb - ratio * (k.v.s * x));
                put<T>(a.dr, i, dl * A * (k.s.s * k.s.c));
                dA += double(dl * k.s.s);
            }
        }
    }
    if (a.dh0) a.dh0[row] = float(C);
    if (a.dA_part) a.dA_part[row] = float(dA);
}

// out[d] = the sum of part[i][d] over i, in order.
__global__ __launch_bounds__(64) void join_kernel(const float* part, int64_t n, int64_t D, float* out) {
    const int64_t d = int64_t(blockIdx.x) * 64 + threadIdx.x;
    if (d >= D) return;
    double s = 0.0;
    for (int64_t i = 0; i < n; ++i) s += part[i * D + d];
    out[d] = float(s);
}

template <typename T, bool DECAY>
__global__ __launch_bounds__(256) void step_kernel(float* state, GaArgs a) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.B * a.D) return;
    const Token k = token_of<DECAY>(at<T>(a.g, i), DECAY ? at<T>(a.r, i) : 0.0f, DECAY ? rate_of(a.A, i % a.D) : 0.0f);
    const float h = state[i], hn = step_of(k.q, k.p, h, k.f * at<T>(a.x, i));
    state[i] = hn;
    put<T>(a.y, i, a.z ? hn * silu(at<T>(a.z, i)) : hn);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
size_t ckpt_bytes(const GatedShape& s) {
    return up256(size_t(ceil_div(s.L, SELSCAN_GATED_CKPT)) * s.batch * s.dim * sizeof(float));
}

GaArgs args_of(const GatedTensors& t, const GatedShape& s) {
    GaArgs a{};
    a.x = t.x; a.g = t.g; a.r = t.r; a.A = t.A; a.z = t.z; a.lengths = t.lengths; a.h0 = t.h0;
    a.y = t.y; a.last = t.last_state; a.ckpt = t.ckpt; a.dy = t.dy; a.dlast = t.dlast;
    a.dx = t.dx; a.dg = t.dg; a.dr = t.dr; a.dz = t.dz; a.dh0 = t.dh0;
    a.B = s.batch; a.L = s.L; a.D = s.dim;
    return a;
}

// f(type, decay) with the call's type and kind as constants.
template <typename F> void dispatch(const GatedShape& s, F f) {
    const bool decay = s.kind == SELSCAN_GATED_DECAY;
    if (s.dtype == DType::BF16) {
        if (decay) f(bf16_bits{}, std::true_type{});
        else f(bf16_bits{}, std::false_type{});
    } else {
        if (decay) f(float{}, std::true_type{});
        else f(float{}, std::false_type{});
    }
}

}  // namespace

bool gated_plan(const GatedShape& s, int32_t, bool, GatedPlan* p) {
    *p = GatedPlan{1, s.L};
    return s.batch <= 65535;
}

size_t gated_fwd_workspace_bytes(const GatedShape&, const GatedPlan&) { return 0; }

size_t gated_bwd_workspace_bytes(const GatedShape& s, const GatedPlan&, bool ckpt_given) {
    return (ckpt_given ? 0 : ckpt_bytes(s)) + up256(size_t(s.batch) * s.dim * sizeof(float));
}

hipError_t launch_gated_fwd(const GatedTensors& t, const GatedShape& s, const GatedPlan&, void*, hipStream_t stream) {
    const GaArgs a = args_of(t, s);
    dispatch(s, [&](auto T, auto decay) {
        hipLaunchKernelGGL((fwd_kernel<decltype(T), decltype(decay)::value>),
                           dim3(unsigned(ceil_div(s.dim, 64)), unsigned(s.batch)), dim3(64), 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedTensors& t, const GatedShape& s, const GatedPlan&, void* workspace,
                            hipStream_t stream) {
    GaArgs a = args_of(t, s);
    char* ws = static_cast<char*>(workspace);
    float* part = reinterpret_cast<float*>(ws);
    if (!a.ckpt) {
        a.ckpt = reinterpret_cast<float*>(ws + up256(size_t(s.batch) * s.dim * sizeof(float)));
        GaArgs f = a;
        f.y = nullptr;
        f.last = nullptr;
        dispatch(s, [&](auto T, auto decay) {
            hipLaunchKernelGGL((fwd_kernel<decltype(T), decltype(decay)::value>),
                               dim3(unsigned(ceil_div(s.dim, 64)), unsigned(s.batch)), dim3(64), 0, stream, f);
        });
    }
    a.dA_part = t.dA ? part : nullptr;
    dispatch(s, [&](auto T, auto decay) {
        hipLaunchKernelGGL((bwd_kernel<decltype(T), decltype(decay)::value>),
                           dim3(unsigned(ceil_div(s.dim, 64)), unsigned(s.batch)), dim3(64), 0, stream, a);
    });
    if (t.dA)
        hipLaunchKernelGGL(join_kernel, dim3(unsigned(ceil_div(s.dim, 64))), dim3(64), 0, stream, part, s.batch, s.dim,
                           t.dA);
    return hipGetLastError();
}

hipError_t launch_gated_step(float* state, const GatedTensors& t, const GatedShape& s, hipStream_t stream) {
    const GaArgs a = args_of(t, s);
    dispatch(s, [&](auto T, auto decay) {
        hipLaunchKernelGGL((step_kernel<decltype(T), decltype(decay)::value>),
                           dim3(unsigned(ceil_div(s.batch * s.dim, 256))), dim3(256), 0, stream, state, a);
    });
    return hipGetLastError();
}

}  // namespace selscan
