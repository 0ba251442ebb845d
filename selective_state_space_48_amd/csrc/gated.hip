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

struct Stretch;
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
    float* dA_part;  // [segments][batch][dim], null: not wanted
    float* dh0;
    int64_t B, L, D;
    // runs of seg_len tokens
    int64_t seg_len;
    Stretch* runs;  // [segments][batch * dim]
    const double* enter;   // the states (gradients) entering the runs; null: h0 (dlast)
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

// ---- tiles -------------------------------------------------------------------
//
// A workgroup walks CL * V channels of an entry through tiles of tokens. A lane
// holds V channels (4 bytes of a row) of N tokens in a row; 64 / CL lanes of a
// wave, and the waves, hold the groups of N tokens after one another. A group
// steps its tokens from 0, which gives its state S and, as the product of its
// decays in 64 bits, what it leaves of the state that enters it: P. Groups are
// joined by h = P h + S in 64 bits, inside a wave by shuffles and over the waves
// through LDS, so that a tile costs one barrier (the LDS entries alternate) and
// every value is read once. The next tile's loads are in flight meanwhile.
constexpr int kWaves = 8;

template <int B> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <typename T, int V> using raw_t = typename RawOf<int(sizeof(T)) * V>::type;

template <typename T, int V> __device__ __forceinline__ void unpack(raw_t<T, V> r, float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(r);
    } else if constexpr (V == 2) {
        f[0] = bf16_lo(r);
        f[1] = bf16_hi(r);
    } else {
        f[0] = to_f32(r);
    }
}
template <typename T, int V> __device__ __forceinline__ raw_t<T, V> pack(const float (&f)[V]) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(f[0]);
    else if constexpr (V == 2) return pack_bf16x2(f[0], f[1]);
    else return from_f32<T>(f[0]);
}

// What a stretch of tokens does to the state that enters it: P h + S.
struct Stretch { double P, S; };
__device__ __forceinline__ Stretch after(const Stretch& first, const Stretch& then) {
    return {then.P * first.P, then.P * first.S + then.S};
}

// Where a thread stands: lane column c, group `first` of N tokens in the tile.
template <int V, int CL, int N> struct Place {
    static constexpr int kTile = kWaves * (64 / CL) * N, kChan = CL * V;
    int lane, wave, c, tg;
    int64_t d, b;     // first channel, entry
    bool live;
    __device__ __forceinline__ Place(int64_t block, int64_t D) {
        lane = threadIdx.x % 64; wave = threadIdx.x / 64;
        c = lane % CL; tg = lane / CL;
        const int64_t blocks = (D + kChan - 1) / kChan;
        d = block % blocks * kChan + c * V;
        b = block / blocks;
        live = d < D;
    }
    __device__ __forceinline__ int64_t token(int64_t t0) const { return t0 + (wave * (64 / CL) + tg) * N; }
};

// The group's stretch before this one in its wave (P 1, S 0 for the first), and the wave's own whole stretch in
// the lanes of its last group.
template <int CL> __device__ __forceinline__ Stretch before_in_wave(Stretch& own, int tg) {
#pragma unroll
    for (int s = 1; s < 64 / CL; s *= 2) {
        const Stretch prev = {__shfl_up(own.P, s * CL, 64), __shfl_up(own.S, s * CL, 64)};
        if (tg >= s) own = after(prev, own);
    }
    if constexpr (CL == 64) return {1.0, 0.0};
    const Stretch prev = {__shfl_up(own.P, CL, 64), __shfl_up(own.S, CL, 64)};
    return tg ? prev : Stretch{1.0, 0.0};
}
// The same against time.
template <int CL> __device__ __forceinline__ Stretch after_in_wave(Stretch& own, int tg) {
    constexpr int n = 64 / CL;
#pragma unroll
    for (int s = 1; s < n; s *= 2) {
        const Stretch next = {__shfl_down(own.P, s * CL, 64), __shfl_down(own.S, s * CL, 64)};
        if (tg + s < n) own = after(next, own);
    }
    if constexpr (CL == 64) return {1.0, 0.0};
    const Stretch next = {__shfl_down(own.P, CL, 64), __shfl_down(own.S, CL, 64)};
    return tg + 1 < n ? next : Stretch{1.0, 0.0};
}

// Loads of N tokens of one tensor at `at` (element of the group's first token), tokens from `last` on taken from it.
template <typename T, int V, int N>
__device__ __forceinline__ void fetch(const void* p, int64_t at, int64_t D, int last, raw_t<T, V> (&r)[N]) {
    const T* q = static_cast<const T*>(p) + at;
    if (last >= N - 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = *reinterpret_cast<const raw_t<T, V>*>(q + i * D);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = *reinterpret_cast<const raw_t<T, V>*>(q + (i < last ? i : last) * D);
    }
}

// Forward: outputs from the state entering the run (kOut), checkpoints alone (kKeep), or the run's own stretch (kRun).
enum { kOut = 0, kKeep = 1, kRun = 2 };

template <typename T, bool DECAY, bool GATE, int V, int CL, int N, int MODE>
__global__ __launch_bounds__(kWaves * 64) void fwd_kernel(GaArgs a) {
    using W = Place<V, CL, N>;
    using R = raw_t<T, V>;
    __shared__ Stretch whole[2][kWaves][W::kChan];
    __shared__ double carry[2][W::kChan];
    const int64_t per = (a.D + W::kChan - 1) / W::kChan * a.B, idx = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t run = idx / per;
    const W w(idx % per, a.D);
    const int64_t n = entry_length(a.lengths, w.b, a.L), row = w.b * a.D + w.d, rows = a.B * a.D;
    const int64_t begin = run * a.seg_len, end = begin + a.seg_len < a.L ? begin + a.seg_len : a.L;
    const bool last_wave = w.wave == kWaves - 1 && w.tg == 64 / CL - 1;
    float A[V];
    Stretch all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = DECAY && w.live ? rate_of(a.A, w.d + v) : 0.0f;
        all[v] = {1.0, 0.0};
    }
    if (w.wave == 0 && w.tg == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            carry[0][w.c * V + v] = MODE == kRun || !w.live ? 0.0
                                    : a.enter               ? a.enter[run * rows + row + v]
                                    : a.h0                  ? double(a.h0[row + v])
                                                            : 0.0;
    }
    R nx[N], ng[N], nr[DECAY ? N : 1], nz[GATE ? N : 1];
    auto load = [&](int64_t t0) {
        const int64_t t = w.token(t0);
        if (!w.live || t >= n) return;
        const int64_t at = (w.b * a.L + t) * a.D + w.d;
        const int left = int(n - t < N ? n - t : N) - 1;
        fetch<T, V, N>(a.x, at, a.D, left, nx);
        fetch<T, V, N>(a.g, at, a.D, left, ng);
        if constexpr (DECAY) fetch<T, V, N>(a.r, at, a.D, left, nr);
        if constexpr (GATE) fetch<T, V, N>(a.z, at, a.D, left, nz);
    };
    load(begin);
    int buf = 0;
    for (int64_t t0 = begin; t0 < end; t0 += W::kTile, buf ^= 1) {
        const int64_t t = w.token(t0);
        const int have = n - t < 0 ? 0 : n - t < N ? int(n - t) : N;
        float q[N][V], b[N][V];
        R z[GATE ? N : 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[V], g[V], r[V];
            unpack<T, V>(nx[i], x);
            unpack<T, V>(ng[i], g);
            if constexpr (DECAY) unpack<T, V>(nr[i], r);
            if constexpr (GATE) z[i] = nz[i];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Token k = token_of<DECAY>(g[v], DECAY ? r[v] : 0.0f, A[v]);
                q[i][v] = k.q;
                b[i][v] = k.f * x[v];
            }
        }
        if (have < N) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    q[i][v] = i < have ? q[i][v] : -0.0f;
                    b[i][v] = i < have ? b[i][v] : 0.0f;
                }
        }
        if (t0 + W::kTile < end) load(t0 + W::kTile);
        Stretch own[V], before[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            double P = 1.0;
            float S = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float p = whole_of(q[i][v]);
                P *= double(p) + double(q[i][v]);
                S = step_of(q[i][v], p, S, b[i][v]);
            }
            own[v] = {P, double(S)};
            before[v] = before_in_wave<CL>(own[v], w.tg);
            if (w.tg == 64 / CL - 1) whole[buf][w.wave][w.c * V + v] = own[v];
        }
        __syncthreads();
        double h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = carry[buf][w.c * V + v];
        for (int j = 0; j < w.wave; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Stretch s = whole[buf][j][w.c * V + v];
                h[v] = s.P * h[v] + s.S;
            }
        if (last_wave) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                carry[buf ^ 1][w.c * V + v] = own[v].P * h[v] + own[v].S;
                if constexpr (MODE == kRun) {
                    Stretch tile = own[v];
                    for (int j = kWaves - 2; j >= 0; --j) tile = after(whole[buf][j][w.c * V + v], tile);
                    all[v].P *= tile.P;
                }
            }
        }
        if constexpr (MODE != kRun) {
            float hf[V];
#pragma unroll
            for (int v = 0; v < V; ++v) hf[v] = float(before[v].P * h[v] + before[v].S);
            if (a.ckpt && w.live && t % SELSCAN_GATED_CKPT == 0 && t < a.L)
#pragma unroll
                for (int v = 0; v < V; ++v) a.ckpt[t / SELSCAN_GATED_CKPT * rows + row + v] = hf[v];
            if constexpr (MODE == kOut) {
                T* y = static_cast<T*>(a.y) + (w.b * a.L + t) * a.D + w.d;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        hf[v] = step_of(q[i][v], whole_of(q[i][v]), hf[v], b[i][v]);
                        o[v] = hf[v];
                    }
                    if constexpr (GATE) {
                        float f[V];
                        unpack<T, V>(z[i], f);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] *= silu(f[v]);
                    }
                    if (i >= have)
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] = 0.0f;
                    if (w.live && t + i < a.L) *reinterpret_cast<R*>(y + i * a.D) = pack<T, V>(o);
                }
            }
        }
    }
    if constexpr (MODE == kRun) {
        if (last_wave && w.live)
#pragma unroll
            for (int v = 0; v < V; ++v)
                a.runs[run * rows + row + v] = {all[v].P, carry[buf][w.c * V + v]};
    } else if (last_wave && w.live && a.last && end == a.L) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.last[row + v] = float(carry[buf][w.c * V + v]);
    }
}

// Backward: the gradients of a run (kOut), or what the run does to the gradient that enters it from behind (kRun):
// C = a (d + C), the same decays against time.
template <typename T, bool DECAY, bool GATE, int V, int CL, int N, int MODE>
__global__ __launch_bounds__(kWaves * 64) void bwd_kernel(GaArgs a) {
    using W = Place<V, CL, N>;
    using R = raw_t<T, V>;
    __shared__ Stretch fwd[2][MODE == kOut ? kWaves : 1][W::kChan], bwd[2][kWaves][W::kChan];
    __shared__ double carry[2][W::kChan];
    const int64_t per = (a.D + W::kChan - 1) / W::kChan * a.B, idx = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t run = idx / per;
    const W w(idx % per, a.D);
    const int64_t n = entry_length(a.lengths, w.b, a.L), row = w.b * a.D + w.d, rows = a.B * a.D;
    const int64_t begin = run * a.seg_len, end = begin + a.seg_len < a.L ? begin + a.seg_len : a.L;
    const int64_t tiles = (end - begin + W::kTile - 1) / W::kTile;
    const bool first_group = w.wave == 0 && w.tg == 0;
    float A[V], dA[V];
    double allP[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = DECAY && w.live ? rate_of(a.A, w.d + v) : 0.0f;
        dA[v] = 0.0f;
        allP[v] = 1.0;
        if (first_group)
            carry[0][w.c * V + v] = MODE == kRun || !w.live ? 0.0
                                    : a.enter               ? a.enter[run * rows + row + v]
                                    : a.dlast               ? double(a.dlast[row + v])
                                                            : 0.0;
    }
    constexpr bool OUT = MODE == kOut;
    R nx[OUT ? N : 1], ng[N], nr[DECAY ? N : 1], nz[GATE ? N : 1], nd[N];
    float nh[V];
    auto load = [&](int64_t t0) {
        const int64_t t = w.token(t0);
        if (!w.live || t >= n) return;
        const int64_t at = (w.b * a.L + t) * a.D + w.d;
        const int left = int(n - t < N ? n - t : N) - 1;
        if constexpr (OUT) fetch<T, V, N>(a.x, at, a.D, left, nx);
        if constexpr (OUT || !DECAY) fetch<T, V, N>(a.g, at, a.D, left, ng);
        if constexpr (DECAY) fetch<T, V, N>(a.r, at, a.D, left, nr);
        if constexpr (GATE) fetch<T, V, N>(a.z, at, a.D, left, nz);
        fetch<T, V, N>(a.dy, at, a.D, left, nd);
        if constexpr (OUT)
#pragma unroll
            for (int v = 0; v < V; ++v) nh[v] = a.ckpt[t0 / SELSCAN_GATED_CKPT * rows + row + v];
    };
    load(begin + (tiles - 1) * W::kTile);
    int buf = 0;
    for (int64_t k = tiles - 1; k >= 0; --k, buf ^= 1) {
        const int64_t t0 = begin + k * W::kTile, t = w.token(t0);
        const int have = n - t < 0 ? 0 : n - t < N ? int(n - t) : N;
        Token tok[N][V];
        float x[OUT ? N : 1][V], d[N][V], dy[OUT && GATE ? N : 1][V], h0[V];
        R z[OUT && GATE ? N : 1];
#pragma unroll
        for (int v = 0; v < V; ++v) h0[v] = OUT ? nh[v] : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float g[V], r[V], f[V];
            if constexpr (OUT) unpack<T, V>(nx[i], x[i]);
            if constexpr (OUT || !DECAY) unpack<T, V>(ng[i], g);
            if constexpr (DECAY) unpack<T, V>(nr[i], r);
            unpack<T, V>(nd[i], d[i]);
            if constexpr (GATE) unpack<T, V>(nz[i], f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                tok[i][v] = token_of<DECAY>(OUT || !DECAY ? g[v] : 0.0f, DECAY ? r[v] : 0.0f, A[v]);
                if constexpr (GATE) {
                    if constexpr (OUT) dy[i][v] = d[i][v];
                    d[i][v] *= silu(f[v]);
                }
            }
            if constexpr (OUT && GATE) z[i] = nz[i];
        }
        if (have < N) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (i < have) continue;
                    tok[i][v].q = -0.0f;
                    tok[i][v].p = 1.0f;
                    tok[i][v].f = 0.0f;
                    d[i][v] = 0.0f;
                    if constexpr (OUT) x[i][v] = 0.0f;
                }
        }
        if (k > 0) load(t0 - W::kTile);
        Stretch ownb[V], later[V], before[OUT ? V : 1];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            double P = 1.0;
            float S = 0.0f, C = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const Token& m = tok[i][v];
                P *= double(m.p) + double(m.q);
                if constexpr (OUT) S = step_of(m.q, m.p, S, m.f * x[i][v]);
            }
#pragma unroll
            for (int i = N - 1; i >= 0; --i) C = step_of(tok[i][v].q, tok[i][v].p, d[i][v] + C, 0.0f);
            ownb[v] = {P, double(C)};
            later[v] = after_in_wave<CL>(ownb[v], w.tg);
            if (w.tg == 0) bwd[buf][w.wave][w.c * V + v] = ownb[v];
            if constexpr (OUT) {
                Stretch own = {P, double(S)};
                before[v] = before_in_wave<CL>(own, w.tg);
                if (w.tg == 64 / CL - 1) fwd[buf][w.wave][w.c * V + v] = own;
            }
        }
        __syncthreads();
        double C[V];
#pragma unroll
        for (int v = 0; v < V; ++v) C[v] = carry[buf][w.c * V + v];
        for (int j = kWaves - 1; j > w.wave; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Stretch s = bwd[buf][j][w.c * V + v];
                C[v] = s.P * C[v] + s.S;
            }
        if (first_group) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                carry[buf ^ 1][w.c * V + v] = ownb[v].P * C[v] + ownb[v].S;
                if constexpr (!OUT) {
                    Stretch tile = ownb[v];
                    for (int j = 1; j < kWaves; ++j) tile = after(bwd[buf][j][w.c * V + v], tile);
                    allP[v] *= tile.P;
                }
            }
        }
        if constexpr (OUT) {
            double h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = h0[v];
            for (int j = 0; j < w.wave; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const Stretch s = fwd[buf][j][w.c * V + v];
                    h[v] = s.P * h[v] + s.S;
                }
            const int64_t at = (w.b * a.L + t) * a.D + w.d;
            float hb[N][V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float hf = float(before[v].P * h[v] + before[v].S);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    hb[i][v] = hf;
                    hf = step_of(tok[i][v].q, tok[i][v].p, hf, tok[i][v].f * x[i][v]);
                    if constexpr (GATE) dy[i][v] *= hf;  // (times silu' below)
                }
            }
            float Cf[V];
#pragma unroll
            for (int v = 0; v < V; ++v) Cf[v] = float(later[v].P * C[v] + later[v].S);
#pragma unroll
            for (int i = N - 1; i >= 0; --i) {
                float ox[V], og[V], orr[V], oz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const Token& m = tok[i][v];
                    const float G = d[i][v] + Cf[v];
                    Cf[v] = step_of(m.q, m.p, G, 0.0f);
                    ox[v] = G * m.f;
                    if constexpr (!DECAY) {
                        og[v] = G * (x[i][v] - hb[i][v]) * (m.v.s * m.v.c);
                    } else {
                        og[v] = G * m.w * x[i][v] * (m.v.s * m.v.c);
                        const float dec = m.p + m.q, ratio = m.w > 0.0f ? dec * rcp_hw(m.w) : 0.0f;
                        const float dl = G * dec * (hb[i][v] - ratio * (m.v.s * x[i][v]));
                        orr[v] = dl * A[v] * (m.s.s * m.s.c);
                        dA[v] += i < have ? dl * m.s.s : 0.0f;
                    }
                    if constexpr (GATE) {
                        float f[V];
                        unpack<T, V>(z[i], f);
                        oz[v] = dy[i][v] * silu_grad(f[v]);
                    }
                    if (i >= have) ox[v] = og[v] = orr[v] = oz[v] = 0.0f;
                }
                if (w.live && t + i < a.L) {
                    auto out = [&](void* p, const float (&o)[V]) {
                        *reinterpret_cast<R*>(static_cast<T*>(p) + at + i * a.D) = pack<T, V>(o);
                    };
                    out(a.dx, ox);
                    out(a.dg, og);
                    if constexpr (DECAY) out(a.dr, orr);
                    if constexpr (GATE) out(a.dz, oz);
                }
            }
        }
    }
    if constexpr (!OUT) {
        if (first_group && w.live)
#pragma unroll
            for (int v = 0; v < V; ++v) a.runs[run * rows + row + v] = {allP[v], carry[buf][w.c * V + v]};
        return;
    }
    if (first_group && w.live && a.dh0 && begin == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[row + v] = float(carry[buf][w.c * V + v]);
    }
    if constexpr (DECAY) {
        if (a.dA_part) {  // the groups' sums in order
            __shared__ float sums[kWaves * (64 / CL)][W::kChan];
#pragma unroll
            for (int v = 0; v < V; ++v) sums[w.wave * (64 / CL) + w.tg][w.c * V + v] = dA[v];
            __syncthreads();
            if (first_group && w.live)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s = 0.0f;
                    for (int j = 0; j < kWaves * (64 / CL); ++j) s += sums[j][w.c * V + v];
                    a.dA_part[(run * a.B + w.b) * a.D + w.d + v] = s;
                }
        }
    }
}

// The states entering the runs, from the first (against: the gradients, from the last) on, in 64 bits; in place of
// the runs' own.
__global__ __launch_bounds__(64) void carry_kernel(Stretch* runs, double* enter, const float* first, int64_t rows,
                                                   int segments, bool against) {
    const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
    if (i >= rows) return;
    double h = first ? first[i] : 0.0;
    for (int s = 0; s < segments; ++s) {
        const int64_t at = (against ? segments - 1 - s : s) * rows + i;
        const Stretch r = runs[at];
        enter[at] = h;
        h = r.P * h + r.S;
    }
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

GaArgs args_of(const GatedTensors& t, const GatedShape& s, const GatedPlan& p) {
    GaArgs a{};
    a.x = t.x; a.g = t.g; a.r = t.r; a.A = t.A; a.z = t.z; a.lengths = t.lengths; a.h0 = t.h0;
    a.y = t.y; a.last = t.last_state; a.ckpt = t.ckpt; a.dy = t.dy; a.dlast = t.dlast;
    a.dx = t.dx; a.dg = t.dg; a.dr = t.dr; a.dz = t.dz; a.dh0 = t.dh0;
    a.B = s.batch; a.L = s.L; a.D = s.dim; a.seg_len = p.seg_len;
    return a;
}

// Channels of a lane: 4 bytes of a row, where rows of an odd number of bfloat16 values allow it.
int lane_channels(const GatedShape& s) { return s.dtype == DType::BF16 && s.dim % 2 == 0 ? 2 : 1; }

constexpr int kCL = 32;               // lanes across channels
constexpr int kNF = 8, kNB = 8;       // tokens of a thread, forward and backward
constexpr int kTileF = kWaves * (64 / kCL) * kNF, kTileB = kWaves * (64 / kCL) * kNB;
static_assert(kTileF % SELSCAN_GATED_CKPT == 0 && kTileB % SELSCAN_GATED_CKPT == 0 && kNF <= SELSCAN_GATED_CKPT &&
                  SELSCAN_GATED_CKPT % kNF == 0,
              "a checkpoint is the state entering a group of tokens, and every tile's first");

int64_t blocks_of(const GatedShape& s) { return ceil_div(s.dim, kCL * lane_channels(s)) * s.batch; }

// f(type, decay, gate, channels of a lane) with the call's choices as constants.
template <typename F> void dispatch(const GatedShape& s, bool gate, F f) {
    auto kinds = [&](auto T, auto V) {
        const std::true_type yes;
        const std::false_type no;
        if (s.kind == SELSCAN_GATED_DECAY) {
            if (gate) f(T, yes, yes, V);
            else f(T, yes, no, V);
        } else {
            if (gate) f(T, no, yes, V);
            else f(T, no, no, V);
        }
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    if (s.dtype == DType::F32) kinds(float{}, one);
    else if (lane_channels(s) == 2) kinds(bf16_bits{}, two);
    else kinds(bf16_bits{}, one);
}

template <int MODE> void run_fwd(const GaArgs& a, const GatedShape& s, int segments, hipStream_t st) {
    dispatch(s, MODE == kOut && a.z, [&](auto T, auto decay, auto gate, auto V) {
        hipLaunchKernelGGL((fwd_kernel<decltype(T), decltype(decay)::value, MODE == kOut && decltype(gate)::value,
                                       decltype(V)::value, kCL, kNF, MODE>),
                           dim3(unsigned(blocks_of(s) * segments)), dim3(kWaves * 64), 0, st, a);
    });
}
template <int MODE> void run_bwd(const GaArgs& a, const GatedShape& s, int segments, hipStream_t st) {
    dispatch(s, a.z, [&](auto T, auto decay, auto gate, auto V) {
        hipLaunchKernelGGL((bwd_kernel<decltype(T), decltype(decay)::value, decltype(gate)::value, decltype(V)::value,
                                       kCL, kNB, MODE>),
                           dim3(unsigned(blocks_of(s) * segments)), dim3(kWaves * 64), 0, st, a);
    });
}
void run_carry(Stretch* runs, double* enter, const float* first, int64_t rows, int segments, bool against,
               hipStream_t st) {
    hipLaunchKernelGGL(carry_kernel, dim3(unsigned(ceil_div(rows, 64))), dim3(64), 0, st, runs, enter, first, rows,
                       segments, against);
}

// Workspace: the runs' stretches and entering states, then (backward) the checkpoints and the sums of dA.
struct Layout {
    size_t enter, ckpt, part, bytes;
};
Layout layout_of(const GatedShape& s, const GatedPlan& p, bool backward, bool ckpt_given) {
    const size_t rows = size_t(s.batch) * s.dim;
    Layout l{};
    size_t at = 0;
    if (p.segments > 1) {
        at = up256(rows * p.segments * sizeof(Stretch));
        l.enter = at;
        at += up256(rows * p.segments * sizeof(double));
    }
    l.ckpt = at;
    if (backward && !ckpt_given) at += up256(size_t(ceil_div(s.L, SELSCAN_GATED_CKPT)) * rows * sizeof(float));
    l.part = at;
    if (backward && s.kind == SELSCAN_GATED_DECAY) at += up256(rows * p.segments * sizeof(float));
    l.bytes = at;
    return l;
}

}  // namespace

bool gated_plan(const GatedShape& s, int32_t requested, bool backward, GatedPlan* p) {
    *p = GatedPlan{1, s.L};
    const int64_t tile = backward ? (kTileF > kTileB ? kTileF : kTileB) : kTileF;
    const int64_t blocks = blocks_of(s);
    int64_t want = requested;
    if (!requested) {
        // runs where workgroups leave CUs idle, of eight tiles at least
        want = blocks > 0 ? 512 / blocks : 1;
        const int64_t most = s.L / (8 * tile);
        want = want < most ? want : most;
    }
    if (want > 1 && s.L > tile) {
        p->seg_len = ceil_div(ceil_div(s.L, want), tile) * tile;
        p->segments = int32_t(ceil_div(s.L, p->seg_len));
    }
    // a grid has fewer than 2^32 threads
    return blocks * p->segments <= (int64_t(1) << 22);
}

size_t gated_fwd_workspace_bytes(const GatedShape& s, const GatedPlan& p) { return layout_of(s, p, false, false).bytes; }

size_t gated_bwd_workspace_bytes(const GatedShape& s, const GatedPlan& p, bool ckpt_given) {
    return layout_of(s, p, true, ckpt_given).bytes;
}

hipError_t launch_gated_fwd(const GatedTensors& t, const GatedShape& s, const GatedPlan& p, void* workspace,
                            hipStream_t stream) {
    GaArgs a = args_of(t, s, p);
    if (p.segments > 1) {
        char* ws = static_cast<char*>(workspace);
        a.runs = reinterpret_cast<Stretch*>(ws);
        double* enter = reinterpret_cast<double*>(ws + layout_of(s, p, false, false).enter);
        run_fwd<kRun>(a, s, p.segments, stream);
        run_carry(a.runs, enter, a.h0, s.batch * s.dim, p.segments, false, stream);
        a.enter = enter;
    }
    run_fwd<kOut>(a, s, p.segments, stream);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedTensors& t, const GatedShape& s, const GatedPlan& p, void* workspace,
                            hipStream_t stream) {
    GaArgs a = args_of(t, s, p);
    char* ws = static_cast<char*>(workspace);
    const Layout l = layout_of(s, p, true, t.ckpt != nullptr);
    const int64_t rows = s.batch * s.dim;
    double* enter = reinterpret_cast<double*>(ws + l.enter);
    a.runs = p.segments > 1 ? reinterpret_cast<Stretch*>(ws) : nullptr;
    if (!a.ckpt) {
        a.ckpt = reinterpret_cast<float*>(ws + l.ckpt);
        GaArgs f = a;
        f.last = nullptr;
        if (p.segments > 1) {
            run_fwd<kRun>(f, s, p.segments, stream);
            run_carry(f.runs, enter, f.h0, rows, p.segments, false, stream);
            f.enter = enter;
        }
        run_fwd<kKeep>(f, s, p.segments, stream);
    }
    if (p.segments > 1) {
        run_bwd<kRun>(a, s, p.segments, stream);
        run_carry(a.runs, enter, a.dlast, rows, p.segments, true, stream);
        a.enter = enter;
    }
    float* part = reinterpret_cast<float*>(ws + l.part);
    a.dA_part = t.dA ? part : nullptr;
    run_bwd<kOut>(a, s, p.segments, stream);
    if (t.dA)
        hipLaunchKernelGGL(join_kernel, dim3(unsigned(ceil_div(s.dim, 64))), dim3(64), 0, stream, part,
                           s.batch * p.segments, s.dim, t.dA);
    return hipGetLastError();
}

hipError_t launch_gated_step(float* state, const GatedTensors& t, const GatedShape& s, hipStream_t stream) {
    const GaArgs a = args_of(t, s, GatedPlan{1, 1});
    auto kind = [&](auto T, auto decay) {
        hipLaunchKernelGGL((step_kernel<decltype(T), decltype(decay)::value>),
                           dim3(unsigned(ceil_div(s.batch * s.dim, 256))), dim3(256), 0, stream, state, a);
    };
    const bool decay = s.kind == SELSCAN_GATED_DECAY;
    if (s.dtype == DType::BF16) {
        if (decay) kind(bf16_bits{}, std::true_type{});
        else kind(bf16_bits{}, std::false_type{});
    } else {
        if (decay) kind(float{}, std::true_type{});
        else kind(float{}, std::false_type{});
    }
    return hipGetLastError();
}

}  // namespace selscan
