// Gated linear recurrence, its token step and its gradients.
//
// Bound by memory where the vector units keep up: a bfloat16 value with a gate takes 47
// vector instructions forward and 100 backward, which hold the units 60 and 66 % of the
// time. 8 x 2048 x 4096 bf16, decay, gate: forward 175 to 186 us (3.6 to 3.8 TB/s), gradients
// 286 to 335 (3.6 to 4.2), where a copy reaches 4.9; 1 x 32771 x 2560, chained: 213 to 219;
// 256 x 5120 tokens: 6.1 (3.9).
//
// What a long memory settles to hangs on 1 - a, which a itself, near 1, does not
// hold: 1 - a is formed without cancellation, and what a group of tokens leaves of
// the state is held as the product of its decays or, near 1, as that less 1.
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

// sigmoid(v), and sigmoid'(v). The exponent's argument is rounded, so either is off by up to 2 |v| + 8 roundings of
// 2^-24, relative; what fp32 has no normal number for is 0 or as fp32 has it.
__device__ __forceinline__ float sigmoid(float v) { return rcp_hw(1.0f + exp2_hw(-v * kLog2e)); }
struct Sig { float s, slope; };
__device__ __forceinline__ Sig sigmoid_slope(float v) {
    const float t = exp2_hw(-fabsf(v) * kLog2e), w = rcp_hw(1.0f + t), m = t * w;
    return {v >= 0.0f ? w : m, m * w};
}

// A token of one channel: its decay a, e = a - 1 and its input's weight f: h = a h + f x.
struct Token { float a, e, f; };

// mix: a = 1 - sigmoid(g), f = sigmoid(g), neither by a difference. (slope: sigmoid'(g))
__device__ __forceinline__ Token mix_of(float g, float* slope) {
    const float t = exp2_hw(-fabsf(g) * kLog2e), w = rcp_hw(1.0f + t), m = t * w;
    const bool up = g >= 0.0f;
    const float u = up ? w : m;
    *slope = m * w;
    return {up ? m : w, -u, u};
}

// decay: a = exp(l), l = A sigmoid(r) <= 0. From -0.35 on, where a - 1 would cancel,
// a - 1 = l + l^2 p(l), p the best cubic for (e^l - 1 - l) / l^2 there (the sum's
// relative error with its roundings is below 1.4 of 2^-24). f = sqrt(1 - a^2) times
// the input gate, 1 - a^2 = -e (2 + e). ANY false: no channel of the wave has such l.
constexpr float kNear = -0.35f;
template <bool ANY> __device__ __forceinline__ Token decay_of(float l) {
    float p = 0.007231935393065214f;
    p = fmaf(p, l, 0.0413486510515213f);
    p = fmaf(p, l, 0.1666298657655716f);
    p = fmaf(p, l, 0.49999865889549255f);
    float e = fmaf(l * l, p, l), a = 1.0f + e;
    if constexpr (ANY) {
        const float far = exp2_hw(l * kLog2e);
        a = l < kNear ? far : a;
        e = l < kNear ? far - 1.0f : e;
    }
    return {a, e, __builtin_amdgcn_sqrtf(-e * (2.0f + e))};
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
// steps its tokens from 0, which gives its state S, and what it leaves of the
// state that enters it, P. Groups are joined by h = P h + S in 64 bits, inside a
// wave by shuffles and over the waves through LDS, so that a tile costs one
// barrier (the LDS entries alternate) and every value is read once. The next
// tile's loads are in flight meanwhile.
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

// The product of a group's decays: as it is, and less 1, which keeps what the first
// loses near 1 (as the first keeps what the second loses near 0).
struct Product {
    float D = 1.0f, E = 0.0f;
    __device__ __forceinline__ void step(float a, float e) {
        D *= a;
        E += fmaf(E, e, e);
    }
    __device__ __forceinline__ double value() const { return D < 0.5f ? double(D) : 1.0 + double(E); }
};

// Where a thread stands: lane column c of its workgroup's channels, group tg of its wave.
template <typename T, int V, int CL, int N> struct Place {
    static constexpr int kGroups = 64 / CL, kWaveTokens = kGroups * N, kTile = kWaves * kWaveTokens, kChan = CL * V;
    int wave, c, tg;
    int64_t d0, d, b;  // the workgroup's first channel, the lane's, the entry
    bool live;
    uint32_t off;      // bytes from the wave's first value in a tile to the lane's
    __device__ __forceinline__ Place(int64_t block, int64_t D) : Place(uint32_t(block), D, uint32_t((D + kChan - 1) / kChan)) {}
    // (fewer than 2^32 workgroups; 32-bit divisions)
    __device__ __forceinline__ Place(uint32_t block, int64_t D, uint32_t blocks) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        c = threadIdx.x % CL;
        tg = threadIdx.x % 64 / CL;
        d0 = int64_t(block % blocks) * kChan;
        d = d0 + c * V;
        b = block / blocks;
        live = d < D;
        // (a lane without channels reads the first ones)
        off = uint32_t((int64_t(tg) * N * D + (live ? c * V : 0)) * int64_t(sizeof(T)));
    }
    // The wave's first value in the tile at t0, and the lane's first token.
    __device__ __forceinline__ int64_t base(const GaArgs& a, int64_t t0) const {
        return (b * a.L + t0 + wave * kWaveTokens) * a.D + d0;
    }
    __device__ __forceinline__ int64_t token(int64_t t0) const { return t0 + wave * kWaveTokens + tg * N; }
};

// The group's stretch before this one in its wave (P 1, S 0 for the first), and the wave's own whole stretch in
// the lanes of its last group.
template <int CL> __device__ __forceinline__ Stretch before_in_wave(Stretch& own, int tg) {
#pragma unroll
    for (int s = 1; s < 64 / CL; s *= 2) {
        const Stretch prev = {__shfl_up(own.P, s * CL, 64), __shfl_up(own.S, s * CL, 64)};
        if (tg >= s) own = after(prev, own);
    }
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
    const Stretch next = {__shfl_down(own.P, CL, 64), __shfl_down(own.S, CL, 64)};
    return tg + 1 < n ? next : Stretch{1.0, 0.0};
}

// Global memory at a pointer that the whole wave shares, kept in scalar registers: rows then cost no vector additions
// (the compiler adds the lane's offset first, and then to every row in 64 bits).
#define SELSCAN_GLOBAL __attribute__((address_space(1)))
__device__ __forceinline__ SELSCAN_GLOBAL char* uniform(const void* p, int64_t bytes) {
    SELSCAN_GLOBAL char* q = (SELSCAN_GLOBAL char*)(static_cast<char*>(const_cast<void*>(p)) + bytes);
    asm("" : "+s"(q));
    return q;
}

// The lane's N tokens of one tensor, `base` the wave's first value; tokens past `left` (the last that exists)
// taken from it. `row`: bytes of a row.
template <typename T, int V, int N>
__device__ __forceinline__ void fetch(const void* p, int64_t base, uint32_t off, int64_t row, raw_t<T, V> (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        r[i] = *(const SELSCAN_GLOBAL raw_t<T, V>*)(uniform(p, base * int64_t(sizeof(T)) + i * row) + off);
}
template <typename T, int V, int N>
__device__ __forceinline__ void fetch_some(const void* p, int64_t base, uint32_t off, int64_t row, int left,
                                           raw_t<T, V> (&r)[N]) {
    const SELSCAN_GLOBAL char* q = uniform(p, base * int64_t(sizeof(T)));
#pragma unroll
    for (int i = 0; i < N; ++i)
        r[i] = *(const SELSCAN_GLOBAL raw_t<T, V>*)(q + (off + uint32_t(i < left ? i : left) * uint32_t(row)));
}
template <typename T, int V, int N>
__device__ __forceinline__ void store_rows(void* p, int64_t base, uint32_t off, int64_t row, int i, const float (&o)[V]) {
    *(SELSCAN_GLOBAL raw_t<T, V>*)(uniform(p, base * int64_t(sizeof(T)) + i * row) + off) = pack<T, V>(o);
}

// The state after the first `n` waves' stretches (against time: after those behind wave n), from h: their entries
// are read two waves at a time, ahead of the products that wait for them.
template <int V, int C>
__device__ __forceinline__ void join(const Stretch (&whole)[kWaves][C], int c, int n, double (&h)[V]) {
#pragma unroll
    for (int j = 0; j < kWaves - 1; j += 2) {
        if (j >= n) break;
        Stretch s[2][V];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) s[u][v] = whole[j + u][c + v];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (j + u < n)
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = s[u][v].P * h[v] + s[u][v].S;
    }
}
template <int V, int C>
__device__ __forceinline__ void join_back(const Stretch (&whole)[kWaves][C], int c, int n, double (&h)[V]) {
#pragma unroll
    for (int j = kWaves - 1; j > 0; j -= 2) {
        if (j <= n) break;
        Stretch s[2][V];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) s[u][v] = whole[j - u][c + v];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (j - u > n)
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = s[u][v].P * h[v] + s[u][v].S;
    }
}

// Forward: outputs from the state entering the run (kOut), checkpoints alone (kKeep), or the run's own stretch (kRun).
enum { kOut = 0, kKeep = 1, kRun = 2 };

// The forward's inputs of a lane's N tokens, as loaded.
template <typename T, bool DECAY, bool GATE, int V, int N> struct FwdInputs {
    raw_t<T, V> x[N], g[N], r[DECAY ? N : 1], z[GATE ? N : 1];
    __device__ __forceinline__ void load(const GaArgs& a, int64_t at, uint32_t off, int64_t row) {
        fetch<T, V, N>(a.x, at, off, row, x);
        fetch<T, V, N>(a.g, at, off, row, g);
        if constexpr (DECAY) fetch<T, V, N>(a.r, at, off, row, r);
        if constexpr (GATE) fetch<T, V, N>(a.z, at, off, row, z);
    }
    __device__ __forceinline__ void load_some(const GaArgs& a, int64_t at, uint32_t off, int64_t row, int left) {
        fetch_some<T, V, N>(a.x, at, off, row, left, x);
        fetch_some<T, V, N>(a.g, at, off, row, left, g);
        if constexpr (DECAY) fetch_some<T, V, N>(a.r, at, off, row, left, r);
        if constexpr (GATE) fetch_some<T, V, N>(a.z, at, off, row, left, z);
    }
};

// What the forward keeps of them: each token's decay and input, the gate, the group's stretch.
template <typename T, bool DECAY, bool GATE, int V, int N> struct FwdTokens {
    float dec[N][V], b[N][V];
    raw_t<T, V> z[GATE ? N : 1];
    double P[V];
    float S[V];

    template <bool FULL, bool FAR>
    __device__ __forceinline__ void eval_as(const FwdInputs<T, DECAY, GATE, V, N>& in, const float (&A)[V], int have) {
        Product prod[V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[V], g[V], r[V];
            unpack<T, V>(in.x[i], x);
            unpack<T, V>(in.g[i], g);
            if constexpr (DECAY) unpack<T, V>(in.r[i], r);
            if constexpr (GATE) z[i] = in.z[i];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Token k;
                float slope;
                if constexpr (DECAY) {
                    k = decay_of<FAR>(A[v] * sigmoid(r[v]));
                    k.f *= sigmoid(g[v]);
                } else {
                    k = mix_of(g[v], &slope);
                }
                dec[i][v] = k.a;
                b[i][v] = k.f * x[v];
                if constexpr (!FULL) {
                    const bool there = i < have;
                    k.e = there ? k.e : 0.0f;
                    dec[i][v] = there ? k.a : 1.0f;
                    b[i][v] = there ? b[i][v] : 0.0f;
                }
                prod[v].step(dec[i][v], k.e);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) P[v] = prod[v].value();
    }
    // FULL: all N tokens exist, else the first `have`. any: a channel of the wave has a rate below kNear.
    template <bool FULL>
    __device__ __forceinline__ void eval(const FwdInputs<T, DECAY, GATE, V, N>& in, const float (&A)[V], bool any,
                                         int have) {
        if (DECAY && !any) eval_as<FULL, false>(in, A, have);
        else eval_as<FULL, true>(in, A, have);
    }
    __device__ __forceinline__ void step_from_zero() {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            S[v] = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) S[v] = fmaf(dec[i][v], S[v], b[i][v]);
        }
    }
    // y from the state entering the group; `left` rows exist of the tensor.
    template <bool FULL>
    __device__ __forceinline__ void put(void* y, int64_t at, uint32_t off, int64_t row, float (&h)[V], int have,
                                        int64_t left) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = fmaf(dec[i][v], h[v], b[i][v]);
                o[v] = h[v];
            }
            if constexpr (GATE) {
                float f[V];
                unpack<T, V>(z[i], f);
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] *= silu(f[v]);
            }
            if constexpr (!FULL) {
                if (i >= left) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = i < have ? o[v] : 0.0f;
            }
            store_rows<T, V, N>(y, at, off, row, i, o);
        }
    }
};

template <typename T, bool DECAY, bool GATE, int V, int CL, int N, int MODE>
__global__ __launch_bounds__(kWaves * 64, N == 8 ? 4 : 2) void fwd_kernel(GaArgs a) {
    using W = Place<T, V, CL, N>;
    __shared__ Stretch whole[2][kWaves][W::kChan];
    __shared__ double carry[2][W::kChan];
    const int64_t per = (a.D + W::kChan - 1) / W::kChan * a.B, idx = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t run = idx / per;
    const W w(idx % per, a.D);
    const int64_t n = entry_length(a.lengths, w.b, a.L), lane = w.b * a.D + w.d, lanes = a.B * a.D;
    const int64_t begin = run * a.seg_len, end = begin + a.seg_len < a.L ? begin + a.seg_len : a.L;
    const int64_t stop = end < n ? end : n, row = a.D * int64_t(sizeof(T));
    const bool last_group = w.wave == kWaves - 1 && w.tg == W::kGroups - 1;
    float A[V];
    double allP[V];
    bool any = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = DECAY ? rate_of(a.A, w.live ? w.d + v : w.d0) : 0.0f;
        any |= A[v] < kNear;
        allP[v] = 1.0;
        if (w.wave == 0 && w.tg == 0)
            carry[0][w.c * V + v] = MODE == kRun || !w.live ? 0.0
                                    : a.enter               ? a.enter[run * lanes + lane + v]
                                    : a.h0                  ? double(a.h0[lane + v])
                                                            : 0.0;
    }
    any = __any(any);
    FwdInputs<T, DECAY, GATE, V, N> in;
    // One tile; all its tokens exist if `whole_tile`, and the next one's loads are sent off if `more`.
    int buf = 0;
    auto tile = [&](int64_t t0, auto whole_tile, bool more) {
        constexpr bool FULL = decltype(whole_tile)::value;
        const int64_t t = w.token(t0);
        const int have = FULL ? N : n - t < 0 ? 0 : n - t < N ? int(n - t) : N;
        FwdTokens<T, DECAY, GATE, V, N> tok;
        tok.template eval<FULL>(in, A, any, have);
        if (more) in.load(a, w.base(a, t0 + W::kTile), w.off, row);
        tok.step_from_zero();
        Stretch own[V], before[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            own[v] = {tok.P[v], double(tok.S[v])};
            before[v] = before_in_wave<CL>(own[v], w.tg);
            if (w.tg == W::kGroups - 1) whole[buf][w.wave][w.c * V + v] = own[v];
        }
        __syncthreads();
        double h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = carry[buf][w.c * V + v];
        join<V>(whole[buf], w.c * V, w.wave, h);
        if (last_group) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                carry[buf ^ 1][w.c * V + v] = own[v].P * h[v] + own[v].S;
                if constexpr (MODE == kRun) {
                    double P = own[v].P;
                    for (int j = 0; j < kWaves - 1; ++j) P *= whole[buf][j][w.c * V + v].P;
                    allP[v] *= P;
                }
            }
        }
        if constexpr (MODE != kRun) {
            float hf[V];
#pragma unroll
            for (int v = 0; v < V; ++v) hf[v] = float(before[v].P * h[v] + before[v].S);
            if (a.ckpt && w.live && t % SELSCAN_GATED_CKPT == 0 && t < a.L)
#pragma unroll
                for (int v = 0; v < V; ++v) a.ckpt[t / SELSCAN_GATED_CKPT * lanes + lane + v] = hf[v];
            if constexpr (MODE == kOut)
                if (w.live) tok.template put<FULL>(a.y, w.base(a, t0), w.off, row, hf, have, a.L - t);
        }
        buf ^= 1;
    };
    int64_t t0 = begin;
    const int64_t whole_end = begin + (stop > begin ? (stop - begin) / W::kTile * W::kTile : 0);
    if (t0 < whole_end) in.load(a, w.base(a, t0), w.off, row);
    for (; t0 < whole_end; t0 += W::kTile) tile(t0, std::true_type{}, t0 + W::kTile < whole_end);
    if (t0 < stop) {
        if (w.token(t0) < n) {
            const int64_t left = n - w.token(t0);
            in.load_some(a, w.base(a, t0), w.off, row, int(left < N ? left : N) - 1);
        }
        tile(t0, std::false_type{}, false);
        t0 += W::kTile;
    }
    __syncthreads();  // (without a tile, carry is what the first wave has put there)
    if constexpr (MODE == kRun) {
        if (last_group && w.live)
#pragma unroll
            for (int v = 0; v < V; ++v) a.runs[run * lanes + lane + v] = {allP[v], carry[buf][w.c * V + v]};
        return;
    }
    // tiles behind the entry's length
    for (; t0 < end; t0 += W::kTile) {
        const int64_t t = w.token(t0);
        if (!w.live || t >= a.L) continue;
        if (a.ckpt && t % SELSCAN_GATED_CKPT == 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
                a.ckpt[t / SELSCAN_GATED_CKPT * lanes + lane + v] = float(carry[buf][w.c * V + v]);
        if constexpr (MODE == kOut) {
            const float zero[V] = {};
            for (int i = 0; i < N && t + i < a.L; ++i)
                store_rows<T, V, N>(a.y, w.base(a, t0), w.off, row, i, zero);
        }
    }
    if (last_group && w.live && a.last && end == a.L) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.last[lane + v] = float(carry[buf][w.c * V + v]);
    }
}

// ---- chained tiles -------------------------------------------------------------
//
// Where the channels are too few for a workgroup each to fill the chip, workgroups
// take single tiles, all of a tile's channels before the next tile's, each tile by
// the order in which a counter hands them out. A tile publishes its own stretch; the
// state that enters it is folded from the state entering its link (kLink tiles) and
// the stretches of the link's tiles before it, always in that order, so that results
// do not depend on who came first; a link's last tile publishes the state entering
// the next one. Every value is again read once. What is published is a word of 64
// bits that says by itself whether it is there (kUnset, a NaN with low bits set,
// which no conversion of a 32-bit value and no operation on such gives), stored and
// read by atomics of the device's scope: no fence, and no order of several words.
//
// Every wait ends: a tile waits only for tiles that the counter handed out before
// it, whose workgroups therefore run (a workgroup takes its next tile before it
// finishes the one it has, but works on them in their order). Should a caller let two
// calls share a workspace, the waits give up after kPatience rounds and hand on NaN.
constexpr uint64_t kUnset = ~uint64_t(0);
constexpr int kLink = 8, kPatience = 1 << 18;

struct Chain {
    uint64_t* P;       // [tile][batch * dim], the tiles' stretches
    uint64_t* S;
    uint64_t* enter;   // [link][batch * dim], the states entering the links from the second on
    uint32_t* counter;
    uint32_t tiles;
};

// Words of tile or link `i` (uniform), `lane` the lane's channel from the first of the workgroup's, `row`.
struct Words {
    uint64_t* p;
    int64_t rows, row;
    uint32_t lane;
    __device__ __forceinline__ SELSCAN_GLOBAL uint64_t* at(uint32_t i) const {
        const uint64_t first = reinterpret_cast<uint64_t>(p) + uint64_t((int64_t(i) * rows + row) * 8);
        const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(first)),
                       hi = __builtin_amdgcn_readfirstlane(uint32_t(first >> 32));
        return (SELSCAN_GLOBAL uint64_t*)((SELSCAN_GLOBAL char*)(uint64_t(hi) << 32 | lo) + lane * 8u);
    }
    __device__ __forceinline__ void publish(uint32_t i, double v) const {
        uint64_t u = __builtin_bit_cast(uint64_t, v);
        if (u == kUnset) u = __builtin_bit_cast(uint64_t, __builtin_nan(""));
        __hip_atomic_store(at(i), u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ uint64_t look(uint32_t i) const {
        return __hip_atomic_load(at(i), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

// What a wave does for tile `k`, a lane for each channel (`live` of them): publishes the tile's own stretch, waits for
// the state that enters it (`from` enters tile 0), and returns that; a link's last tile hands on the next link's.
__device__ __forceinline__ double link_tile(const Words& P, const Words& S, const Words& enter, uint32_t k, uint32_t tiles,
                                            double from, bool live, const Stretch& own) {
    const uint32_t m = k % kLink, base = k - m;
    const bool more = k + 1 < tiles;
    if (live && more && m != kLink - 1) {
        P.publish(k, own.P);
        S.publish(k, own.S);
    }
    uint64_t e = __builtin_bit_cast(uint64_t, from), p[kLink - 1], s[kLink - 1];
    // Rounds over the words that come last, the state entering the link and the stretch of the tile before; then all
    // at once, one trip to memory. (For those of tiles from k on, an earlier one's. Rounds over all of them would
    // take the memory's time from everyone's inputs.)
    bool all = false;
    for (int round = 0;; ++round) {
        bool wait = false;
        if (live) {
            if (base && !all) e = enter.look(base / kLink - 1);
            if (m) {
                if (all) {
#pragma unroll
                    for (int j = 0; j < kLink - 1; ++j) {
                        p[j] = P.look(base + (j < int(m) ? j : m - 1));
                        s[j] = S.look(base + (j < int(m) ? j : m - 1));
                    }
#pragma unroll
                    for (int j = 0; j < kLink - 1; ++j) wait |= p[j] == kUnset || s[j] == kUnset;
                } else {
                    wait = S.look(k - 1) == kUnset;
                }
            }
            wait |= base && e == kUnset;
        }
        if (!__any(wait)) {
            if (all || !m) break;
            all = true;
            continue;
        }
        if (round == kPatience) {
            e = __builtin_bit_cast(uint64_t, __builtin_nan(""));
            break;
        }
        __builtin_amdgcn_s_sleep(4);
    }
    double h = __builtin_bit_cast(double, e);
#pragma unroll
    for (int j = 0; j < kLink - 1; ++j)
        if (j < int(m)) h = __builtin_bit_cast(double, p[j]) * h + __builtin_bit_cast(double, s[j]);
    if (live && more && m == kLink - 1) enter.publish(k / kLink, own.P * h + own.S);
    return h;
}

// A chain's words unset and its counter 0; `copy` the entering states (zeros without them), as last_state may take
// their place while tiles still start from them.
__global__ __launch_bounds__(256) void start_chain_kernel(Chain ch, int64_t words, const float* from, float* copy,
                                                          int64_t rows) {
    const int64_t i0 = int64_t(blockIdx.x) * 256 + threadIdx.x, step = int64_t(gridDim.x) * 256;
    if (i0 == 0) *ch.counter = 0;
    for (int64_t i = i0; i < words; i += step) ch.P[i] = kUnset;
    for (int64_t i = i0; i < rows; i += step) copy[i] = from ? from[i] : 0.0f;
}

// Eight waves compute; a ninth hands out the tiles and looks back. While it does that for a tile, the others
// evaluate the next one; the tile's tokens wait in LDS: one barrier a tile.
template <typename T, bool DECAY, bool GATE, int V, int CL, int N>
__global__ __launch_bounds__(kWaves * 64 + 64, 3) void fwd_chain_kernel(GaArgs a, Chain ch) {
    using W = Place<T, V, CL, N>;
    static_assert(W::kChan <= 64, "a lane of the ninth wave for each channel");
    __shared__ Stretch whole[3][kWaves][W::kChan];
    __shared__ double enter[3][W::kChan];
    __shared__ uint32_t tickets[3];
    const uint32_t blocks = uint32_t((a.D + W::kChan - 1) / W::kChan), per = blocks * uint32_t(a.B);
    const uint32_t total = ch.tiles * per;
    const int64_t lanes = a.B * a.D, row = a.D * int64_t(sizeof(T));
    const bool links = __builtin_amdgcn_readfirstlane(threadIdx.x / 64) == kWaves;
    if (threadIdx.x == kWaves * 64) tickets[0] = atomicAdd(ch.counter, 1u);
    __syncthreads();
    uint32_t item = __builtin_amdgcn_readfirstlane(tickets[0]), before_item = total;
    FwdInputs<T, DECAY, GATE, V, N> in;
    float A[V];
    auto load = [&](uint32_t it) {
        const W w(it % per, a.D, blocks);
        const int64_t n = entry_length(a.lengths, w.b, a.L), t0 = int64_t(it / per) * W::kTile;
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = DECAY ? rate_of(a.A, w.live ? w.d + v : w.d0) : 0.0f;
        if (t0 + W::kTile <= n) {
            in.load(a, w.base(a, t0), w.off, row);
        } else if (w.token(t0) < n) {
            const int64_t left = n - w.token(t0);
            in.load_some(a, w.base(a, t0), w.off, row, int(left < N ? left : N) - 1);
        }
    };
    // The tokens of the tile whose outputs are still to come: decays and inputs in LDS (a lane's own, two tiles in
    // turn), the gate in registers.
    constexpr int kQuads = N * V / 2;
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ f32x4 kept[2][kQuads][kWaves * 64];
    FwdTokens<T, DECAY, GATE, V, N> tok;
    raw_t<T, V> prev_z[GATE ? N : 1];
    Stretch before[V], prev_before[V];
    int side = 0;
    if (!links && item < total) load(item);
    for (int buf = 0;; buf = buf == 2 ? 0 : buf + 1) {
        const int after_buf = buf == 2 ? 0 : buf + 1, last_buf = buf == 0 ? 2 : buf - 1;
        if (!links) {
            if (item < total) {
                const W w(item % per, a.D, blocks);
                const int64_t n = entry_length(a.lengths, w.b, a.L), t0 = int64_t(item / per) * W::kTile, t = w.token(t0);
                const int have = n - t < 0 ? 0 : n - t < N ? int(n - t) : N;
                bool any = false;
#pragma unroll
                for (int v = 0; v < V; ++v) any |= A[v] < kNear;
                any = __any(any);
                if (t0 + W::kTile <= n) tok.template eval<true>(in, A, any, N);
                else tok.template eval<false>(in, A, any, have);
                tok.step_from_zero();
#pragma unroll
                for (int q = 0; q < kQuads; ++q) {
                    constexpr int per_quad = 2 / V;
                    f32x4 f;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        f[2 * j] = tok.dec[q * per_quad + (V == 1 ? j : 0)][V == 1 ? 0 : j];
                        f[2 * j + 1] = tok.b[q * per_quad + (V == 1 ? j : 0)][V == 1 ? 0 : j];
                    }
                    kept[side][q][threadIdx.x] = f;
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    Stretch own = {tok.P[v], double(tok.S[v])};
                    before[v] = before_in_wave<CL>(own, w.tg);
                    if (w.tg == W::kGroups - 1) whole[buf][w.wave][w.c * V + v] = own;
                }
            }
        } else if (item < total && threadIdx.x == kWaves * 64) {
            tickets[after_buf] = atomicAdd(ch.counter, 1u);
        }
        __syncthreads();
        const uint32_t next = item < total ? __builtin_amdgcn_readfirstlane(tickets[after_buf]) : total;
        if (!links) {
            if (next < total) load(next);
            if (before_item < total) {
                const W w(before_item % per, a.D, blocks);
                const int64_t n = entry_length(a.lengths, w.b, a.L), lane = w.b * a.D + w.d;
                const int64_t t0 = int64_t(before_item / per) * W::kTile, t = w.token(t0);
                const int have = n - t < 0 ? 0 : n - t < N ? int(n - t) : N;
                double h[V];
                float hf[V];
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = enter[last_buf][w.c * V + v];
                join<V>(whole[last_buf], w.c * V, w.wave, h);
#pragma unroll
                for (int v = 0; v < V; ++v) hf[v] = float(prev_before[v].P * h[v] + prev_before[v].S);
                if (a.ckpt && w.live && t % SELSCAN_GATED_CKPT == 0 && t < a.L)
#pragma unroll
                    for (int v = 0; v < V; ++v) a.ckpt[t / SELSCAN_GATED_CKPT * lanes + lane + v] = hf[v];
                const int64_t at = w.base(a, t0);
#pragma unroll
                for (int q = 0; q < kQuads; ++q) {
                    const f32x4 f = kept[side ^ 1][q][threadIdx.x];
#pragma unroll
                    for (int u = 0; u < 2 / V; ++u) {
                        const int i = q * (2 / V) + u;
                        float o[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const int j = V == 1 ? u : v;
                            hf[v] = fmaf(f[2 * j], hf[v], f[2 * j + 1]);
                            o[v] = i < have ? hf[v] : 0.0f;
                        }
                        if constexpr (GATE) {
                            float z[V];
                            unpack<T, V>(prev_z[i], z);
#pragma unroll
                            for (int v = 0; v < V; ++v) o[v] *= i < have ? silu(z[v]) : 1.0f;
                        }
                        if (w.live && t + i < a.L) store_rows<T, V, N>(a.y, at, w.off, row, i, o);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < (GATE ? N : 0); ++i) prev_z[i] = tok.z[i];
#pragma unroll
            for (int v = 0; v < V; ++v) prev_before[v] = before[v];
            side ^= 1;
        } else if (item < total) {
            const uint32_t k = item / per;
            const W w(item % per, a.D, blocks);
            const int c = threadIdx.x % 64;
            const bool live = c < W::kChan && w.d0 + c < a.D;
            const int64_t at = w.b * a.D + w.d0 + (live ? c : 0);
            Stretch s = whole[buf][0][live ? c : 0];
#pragma unroll
            for (int j = 1; j < kWaves; ++j) s = after(s, whole[buf][j][live ? c : 0]);
            const int64_t first = w.b * a.D + w.d0;
            const uint32_t lane = live ? c : 0;
            const double hin = link_tile(Words{ch.P, lanes, first, lane}, Words{ch.S, lanes, first, lane},
                                         Words{ch.enter, lanes, first, lane}, k, ch.tiles, a.h0[at], live, s);
            if (live) {
                enter[buf][c] = hin;
                if (k + 1 == ch.tiles && a.last) a.last[at] = float(s.P * hin + s.S);
            }
        }
        if (item >= total) break;
        before_item = item;
        item = next;
    }
}

// Backward: the gradients of a run (kOut), or what the run does to the gradient that enters it from behind (kRun):
// C = a (d + C), the same decays against time.
template <typename T, bool DECAY, bool GATE, int V, int CL, int N, int MODE>
__global__ __launch_bounds__(kWaves * 64) void bwd_kernel(GaArgs a) {
    using W = Place<T, V, CL, N>;
    using R = raw_t<T, V>;
    constexpr bool OUT = MODE == kOut;
    __shared__ Stretch fwd[2][OUT ? kWaves : 1][W::kChan], bwd[2][kWaves][W::kChan];
    __shared__ double carry[2][W::kChan];
    const int64_t per = (a.D + W::kChan - 1) / W::kChan * a.B, idx = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t run = idx / per;
    const W w(idx % per, a.D);
    const int64_t n = entry_length(a.lengths, w.b, a.L), lane = w.b * a.D + w.d, lanes = a.B * a.D;
    const int64_t begin = run * a.seg_len, end = begin + a.seg_len < a.L ? begin + a.seg_len : a.L;
    const int64_t stop = end < n ? end : n, row = a.D * int64_t(sizeof(T));
    const int64_t tiles = stop > begin ? (stop - begin + W::kTile - 1) / W::kTile : 0;
    const bool first_group = w.wave == 0 && w.tg == 0;
    float A[V];
    double dA[V], allP[V];
    bool any = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = DECAY ? rate_of(a.A, w.live ? w.d + v : w.d0) : 0.0f;
        any |= A[v] < kNear;
        dA[v] = 0.0;
        allP[v] = 1.0;
        if (first_group)
            carry[0][w.c * V + v] = MODE == kRun || !w.live ? 0.0
                                    : a.enter               ? a.enter[run * lanes + lane + v]
                                    : a.dlast               ? double(a.dlast[lane + v])
                                                            : 0.0;
    }
    any = __any(any);
    R nx[OUT ? N : 1], ng[N], nr[DECAY ? N : 1], nz[GATE ? N : 1], nd[N];
    float nh[V];
    auto enter_tile = [&](int64_t t0) {
        if constexpr (OUT)
#pragma unroll
            for (int v = 0; v < V; ++v)
                nh[v] = a.ckpt[t0 / SELSCAN_GATED_CKPT * lanes + (w.live ? lane + v : w.b * a.D + w.d0)];
    };
    auto load = [&](int64_t t0) {
        const int64_t at = w.base(a, t0);
        if constexpr (OUT) fetch<T, V, N>(a.x, at, w.off, row, nx);
        if constexpr (OUT || !DECAY) fetch<T, V, N>(a.g, at, w.off, row, ng);
        if constexpr (DECAY) fetch<T, V, N>(a.r, at, w.off, row, nr);
        if constexpr (GATE) fetch<T, V, N>(a.z, at, w.off, row, nz);
        fetch<T, V, N>(a.dy, at, w.off, row, nd);
        enter_tile(t0);
    };
    auto load_some = [&](int64_t t0, int left) {
        const int64_t at = w.base(a, t0);
        if constexpr (OUT) fetch_some<T, V, N>(a.x, at, w.off, row, left, nx);
        if constexpr (OUT || !DECAY) fetch_some<T, V, N>(a.g, at, w.off, row, left, ng);
        if constexpr (DECAY) fetch_some<T, V, N>(a.r, at, w.off, row, left, nr);
        if constexpr (GATE) fetch_some<T, V, N>(a.z, at, w.off, row, left, nz);
        fetch_some<T, V, N>(a.dy, at, w.off, row, left, nd);
        enter_tile(t0);
    };
    if constexpr (OUT) {  // tiles behind the entry's length
        for (int64_t t0 = begin + tiles * W::kTile; t0 < end; t0 += W::kTile) {
            const int64_t t = w.token(t0), at = w.base(a, t0);
            const float zero[V] = {};
            for (int i = 0; w.live && i < N && t + i < a.L; ++i) {
                store_rows<T, V, N>(a.dx, at, w.off, row, i, zero);
                store_rows<T, V, N>(a.dg, at, w.off, row, i, zero);
                if constexpr (DECAY) store_rows<T, V, N>(a.dr, at, w.off, row, i, zero);
                if constexpr (GATE) store_rows<T, V, N>(a.dz, at, w.off, row, i, zero);
            }
        }
    }
    int buf = 0;
    auto tile = [&](int64_t t0, auto whole_tile, bool more) {
        constexpr bool FULL = decltype(whole_tile)::value;
        const int64_t t = w.token(t0);
        const int have = FULL ? N : n - t < 0 ? 0 : n - t < N ? int(n - t) : N;
        // of each token: a; d, dy silu(z); and (OUT) b, then the state before it; f; and
        //   mix:   u', x
        //   decay: f' = w x v', dl = G (a h - rest), A s', s
        // with the gate dy silu'(z)
        constexpr int M = OUT ? N : 1, MD = OUT && DECAY ? N : 1, MG = OUT && GATE ? N : 1;
        float dec[N][V], d[N][V], hb[M][V], f[M][V], fs[M][V], rest[M][V], rs[MD][V], sr[MD][V], dz[MG][V], h0[V];
        Product prod[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h0[v] = OUT ? nh[v] : 0.0f;
        auto tokens = [&](auto far) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[V], g[V], r[V], z[V];
                if constexpr (OUT) unpack<T, V>(nx[i], x);
                if constexpr (OUT || !DECAY) unpack<T, V>(ng[i], g);
                if constexpr (DECAY) unpack<T, V>(nr[i], r);
                if constexpr (GATE) unpack<T, V>(nz[i], z);
                unpack<T, V>(nd[i], d[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool in = FULL || i < have;
                    Token k;
                    if constexpr (DECAY) {
                        const Sig s = sigmoid_slope(r[v]);
                        k = decay_of<decltype(far)::value>(A[v] * s.s);
                        if constexpr (OUT) {
                            const Sig u = sigmoid_slope(g[v]);
                            const float ux = u.s * x[v];
                            hb[i][v] = k.f * ux;
                            fs[i][v] = k.f * x[v] * u.slope;
                            // a^2 / w of w's derivative by l (0 where a rounds to 1)
                            rest[i][v] = k.f > 0.0f ? k.a * k.a * rcp_hw(k.f) * ux : 0.0f;
                            f[i][v] = k.f * u.s;
                            rs[i][v] = A[v] * s.slope;
                            sr[i][v] = in ? s.s : 0.0f;
                        }
                    } else {
                        float slope;
                        k = mix_of(g[v], &slope);
                        if constexpr (OUT) {
                            hb[i][v] = k.f * x[v];
                            f[i][v] = k.f;
                            fs[i][v] = slope;
                            rest[i][v] = x[v];
                        }
                    }
                    if constexpr (GATE) {
                        const float s = rcp_hw(1.0f + exp2_hw(-z[v] * kLog2e));
                        if constexpr (OUT) dz[i][v] = d[i][v] * (s * fmaf(z[v], 1.0f - s, 1.0f));
                        d[i][v] *= z[v] * s;
                    }
                    dec[i][v] = in ? k.a : 1.0f;
                    d[i][v] = in ? d[i][v] : 0.0f;
                    if constexpr (OUT) hb[i][v] = in ? hb[i][v] : 0.0f;
                    prod[v].step(dec[i][v], in ? k.e : 0.0f);
                }
            }
        };
        if (DECAY && !any) tokens(std::false_type{});
        else tokens(std::true_type{});
        if (more) load(t0 - W::kTile);
        Stretch own[V], later[V], before[OUT ? V : 1];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float S = 0.0f, C = 0.0f;
            if constexpr (OUT)
#pragma unroll
                for (int i = 0; i < N; ++i) S = fmaf(dec[i][v], S, hb[i][v]);
#pragma unroll
            for (int i = N - 1; i >= 0; --i) C = dec[i][v] * (d[i][v] + C);
            const double P = prod[v].value();
            own[v] = {P, double(C)};
            later[v] = after_in_wave<CL>(own[v], w.tg);
            if (w.tg == 0) bwd[buf][w.wave][w.c * V + v] = own[v];
            if constexpr (OUT) {
                Stretch s = {P, double(S)};
                before[v] = before_in_wave<CL>(s, w.tg);
                if (w.tg == W::kGroups - 1) fwd[buf][w.wave][w.c * V + v] = s;
            }
        }
        __syncthreads();
        double C[V];
#pragma unroll
        for (int v = 0; v < V; ++v) C[v] = carry[buf][w.c * V + v];
        join_back<V>(bwd[buf], w.c * V, w.wave, C);
        if (first_group) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                carry[buf ^ 1][w.c * V + v] = own[v].P * C[v] + own[v].S;
                if constexpr (!OUT) {
                    double P = own[v].P;
                    for (int j = 1; j < kWaves; ++j) P *= bwd[buf][j][w.c * V + v].P;
                    allP[v] *= P;
                }
            }
        }
        if constexpr (OUT) {
            double h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = h0[v];
            join<V>(fwd[buf], w.c * V, w.wave, h);
            const int64_t at = w.base(a, t0);
            float Cf[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Cf[v] = float(later[v].P * C[v] + later[v].S);
                float hf = float(before[v].P * h[v] + before[v].S);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float b = hb[i][v];
                    hb[i][v] = hf;
                    hf = fmaf(dec[i][v], hf, b);
                    if constexpr (GATE) dz[i][v] *= hf;
                }
            }
            if (w.live) {
                float sum[V] = {};  // a tile's share of dA; tiles are added in 64 bits
#pragma unroll
                for (int i = N - 1; i >= 0; --i) {
                    float ox[V], og[V], orr[V], oz[V];
                    const bool in = FULL || i < have;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float G = d[i][v] + Cf[v];
                        Cf[v] = dec[i][v] * G;
                        ox[v] = in ? G * f[i][v] : 0.0f;
                        if constexpr (!DECAY) {
                            og[v] = in ? G * (rest[i][v] - hb[i][v]) * fs[i][v] : 0.0f;
                        } else {
                            og[v] = in ? G * fs[i][v] : 0.0f;
                            const float dl = in ? G * fmaf(dec[i][v], hb[i][v], -rest[i][v]) : 0.0f;
                            sum[v] = fmaf(dl, sr[i][v], sum[v]);
                            orr[v] = in ? dl * rs[i][v] : 0.0f;
                        }
                        if constexpr (GATE) oz[v] = in ? dz[i][v] : 0.0f;
                    }
                    if (!FULL && t + i >= a.L) continue;
                    store_rows<T, V, N>(a.dx, at, w.off, row, i, ox);
                    store_rows<T, V, N>(a.dg, at, w.off, row, i, og);
                    if constexpr (DECAY) store_rows<T, V, N>(a.dr, at, w.off, row, i, orr);
                    if constexpr (GATE) store_rows<T, V, N>(a.dz, at, w.off, row, i, oz);
                }
                if constexpr (DECAY)
#pragma unroll
                    for (int v = 0; v < V; ++v) dA[v] += double(sum[v]);
            }
        }
        buf ^= 1;
    };
    int64_t k = tiles - 1;
    if (tiles && begin + tiles * W::kTile > n) {  // the last tile's tokens do not all exist
        const int64_t t0 = begin + k * W::kTile;
        if (w.token(t0) < n) {
            const int64_t left = n - w.token(t0);
            load_some(t0, int(left < N ? left : N) - 1);
        }
        tile(t0, std::false_type{}, false);
        --k;
    }
    if (k >= 0) load(begin + k * W::kTile);
    for (; k >= 0; --k) tile(begin + k * W::kTile, std::true_type{}, k > 0);
    if constexpr (!OUT) {
        if (first_group && w.live)
#pragma unroll
            for (int v = 0; v < V; ++v) a.runs[run * lanes + lane + v] = {allP[v], carry[buf][w.c * V + v]};
        return;
    }
    if (first_group && w.live && a.dh0 && begin == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[lane + v] = float(carry[buf][w.c * V + v]);
    }
    if constexpr (DECAY) {
        if (a.dA_part) {  // the groups' sums in order
            __shared__ double sums[kWaves * W::kGroups][W::kChan];
#pragma unroll
            for (int v = 0; v < V; ++v) sums[w.wave * W::kGroups + w.tg][w.c * V + v] = dA[v];
            __syncthreads();
            if (first_group && w.live)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    double s = 0.0;
                    for (int j = 0; j < kWaves * W::kGroups; ++j) s += sums[j][w.c * V + v];
                    a.dA_part[(run * a.B + w.b) * a.D + w.d + v] = float(s);
                }
        }
    }
}

// The states entering the runs, from the first (against: the gradients, from the last) on, in 64 bits: a thread goes
// through a channel's runs one by one.
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

// out[d] = the sum of part[i][d] over i: 64 columns a workgroup, sixteen interleaved sums joined in order.
__global__ __launch_bounds__(1024) void join_kernel(const float* part, int64_t n, int64_t D, float* out) {
    __shared__ double sums[16][64];
    const int c = threadIdx.x % 64, r = threadIdx.x / 64;
    const int64_t d = int64_t(blockIdx.x) * 64 + c;
    double s = 0.0;
    if (d < D)
#pragma unroll 4
        for (int64_t i = r; i < n; i += 16) s += part[i * D + d];
    sums[r][c] = s;
    __syncthreads();
    if (r || d >= D) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sums[k][c];
    out[d] = float(s);
}

template <typename T, bool DECAY>
__global__ __launch_bounds__(256) void step_kernel(float* state, GaArgs a) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.B * a.D) return;
    Token k;
    float slope;
    if constexpr (DECAY) {
        k = decay_of<true>(rate_of(a.A, i % a.D) * sigmoid(at<T>(a.r, i)));
        k.f *= sigmoid(at<T>(a.g, i));
    } else {
        k = mix_of(at<T>(a.g, i), &slope);
    }
    // near 1 from a - 1, as a token loop has no other way to keep what its state settles to
    const float h = state[i], b = k.f * at<T>(a.x, i);
    const float hn = k.a < 0.5f ? fmaf(k.a, h, b) : h + fmaf(k.e, h, b);
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

// Lanes across channels, and tokens of a thread, of the wide and the narrow split.
// Wide: 128-byte rows. Narrow: half of that, twice the workgroups, where the wide
// ones would leave CUs idle or take a round more (the work of a workgroup is bound
// by its CU; us, wide and narrow: bf16 4 x 2048 x 2048 74 and 40, 4 x 4096 x 5120
// 214 and 194; but 4 x 2048 x 4096 62 and 60, 3 x 4096 x 5120 132 and 155, 8 x 2048
// x 4096 with a gate 175 and 219, as two workgroups then read each line). Tokens of
// a thread are what the registers take: 4 backward, where 8 spill (331 against 858).
constexpr int kWide = 32, kNarrow = 16;
constexpr int kNF = 8, kNFNarrow = 16, kNB = 4;
constexpr int tile_of(int lanes, int tokens) { return kWaves * (64 / lanes) * tokens; }
constexpr int kTile = tile_of(kWide, kNF);  // runs are of whole tiles
constexpr int kChainGroups = 256;           // workgroups of a chain: one a CU
static_assert(kTile % tile_of(kWide, kNB) == 0 && tile_of(kWide, kNB) % SELSCAN_GATED_CKPT == 0 &&
                  tile_of(kNarrow, kNFNarrow) % SELSCAN_GATED_CKPT == 0 && tile_of(kNarrow, kNB) % SELSCAN_GATED_CKPT == 0 &&
                  SELSCAN_GATED_CKPT % kNFNarrow == 0 && SELSCAN_GATED_CKPT % kNF == 0,
              "a checkpoint is the state entering a group of tokens, and every tile's first");

int64_t blocks_of(const GatedShape& s, int lanes) { return ceil_div(s.dim, lanes * lane_channels(s)) * s.batch; }
// Rounds of workgroups over the CUs, weighed: a wide one 40; a narrow one half the work at 1.15 of its cost, or twice
// it where a lane's channel is 2 bytes and a row 32 (8 x 2048 x 2049 bf16 76 and 160).
int64_t wide_cost(const GatedShape& s) { return ceil_div(blocks_of(s, kWide), 256) * 40; }
bool thin(const GatedShape& s) { return s.dtype == DType::BF16 && lane_channels(s) == 1; }
int64_t narrow_cost(const GatedShape& s) { return ceil_div(blocks_of(s, kNarrow), 256) * (thin(s) ? 46 : 23); }
bool narrow(const GatedShape& s) { return narrow_cost(s) < wide_cost(s); }

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
        using E = decltype(T);
        constexpr bool D = decltype(decay)::value, G = MODE == kOut && decltype(gate)::value;
        constexpr int C = decltype(V)::value;
        if constexpr (MODE != kRun)
            if (segments == 1 && narrow(s)) {
                hipLaunchKernelGGL((fwd_kernel<E, D, G, C, kNarrow, kNFNarrow, MODE>), dim3(unsigned(blocks_of(s, kNarrow))),
                                   dim3(kWaves * 64), 0, st, a);
                return;
            }
        hipLaunchKernelGGL((fwd_kernel<E, D, G, C, kWide, kNF, MODE>), dim3(unsigned(blocks_of(s, kWide) * segments)),
                           dim3(kWaves * 64), 0, st, a);
    });
}
template <int MODE> void run_bwd(const GaArgs& a, const GatedShape& s, int segments, hipStream_t st) {
    dispatch(s, a.z, [&](auto T, auto decay, auto gate, auto V) {
        using E = decltype(T);
        constexpr bool D = decltype(decay)::value, G = decltype(gate)::value;
        constexpr int C = decltype(V)::value;
        if constexpr (MODE != kRun)
            if (segments == 1 && narrow(s)) {
                hipLaunchKernelGGL((bwd_kernel<E, D, G, C, kNarrow, kNB, MODE>), dim3(unsigned(blocks_of(s, kNarrow))),
                                   dim3(kWaves * 64), 0, st, a);
                return;
            }
        hipLaunchKernelGGL((bwd_kernel<E, D, G, C, kWide, kNB, MODE>), dim3(unsigned(blocks_of(s, kWide) * segments)),
                           dim3(kWaves * 64), 0, st, a);
    });
}
void run_carry(Stretch* runs, double* enter, const float* first, int64_t rows, int segments, bool against,
               hipStream_t st) {
    hipLaunchKernelGGL(carry_kernel, dim3(unsigned(ceil_div(rows, 64))), dim3(64), 0, st, runs, enter, first, rows,
                       segments, against);
}

// Workspace: the runs' stretches and entering states, or a chain's words, its counter and the states that it starts
// from, then (backward) the checkpoints and the sums of dA.
struct Layout {
    size_t enter, counter, from, ckpt, part, bytes;
};
int64_t chain_links(const GatedPlan& p) { return ceil_div(p.chain, kLink); }
int64_t chain_words(const GatedShape& s, const GatedPlan& p) { return (2 * p.chain + chain_links(p)) * s.batch * s.dim; }
Layout layout_of(const GatedShape& s, const GatedPlan& p, bool backward, bool ckpt_given) {
    const size_t rows = size_t(s.batch) * s.dim;
    Layout l{};
    size_t at = 0;
    if (p.segments > 1) {
        at = up256(rows * p.segments * sizeof(Stretch));
        l.enter = at;
        at += up256(rows * p.segments * sizeof(double));
    }
    if (p.chain) {
        l.counter = up256(size_t(chain_words(s, p)) * sizeof(uint64_t));
        l.from = l.counter + 256;
        at = l.from + up256(rows * sizeof(float));
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
    *p = GatedPlan{1, s.L, 0};
    const int64_t blocks = blocks_of(s, kWide);
    int64_t want = requested;
    if (!requested) {
        want = 1;
        const int64_t single = narrow(s) ? narrow_cost(s) : wide_cost(s);
        if (!backward) {
            // Chained tiles, which share out evenly what workgroups of whole sequences do not, at 1.3 of its cost (2.6 of
            // rows of 32 values of 2 bytes) and some 10 us (bf16, us, single and chained: 8 x 2048 x 64 31 and 17, 1 x
            // 2048 x 2560 33 and 24, 1 x 32771 x 2560 588 and 217, 2 x 4096 x 5120 135 and 113; but 2 x 1024 x 2560 20
            // and 23, 2 x 4096 x 4096 66 and 85, 3 x 4096 x 5120 143 and 163, 8 x 2048 x 2049 84 and 159). Runs, which
            // a caller can ask for, are not weighed; a link waits for the one before, so very long sequences of one block
            // of channels take less in runs (chained, 64 and 256 runs: 1 x 60000 x 64 100, 78, 87; 1 x 262144 x 64 401,
            // 234, 135; but 4 x 16384 x 32 35, 40, 56).
            if (s.L > 12 * kTile && blocks * (thin(s) ? 104 : 52) < single * 256) p->chain = ceil_div(s.L, kTile);
        } else if (blocks > 0 && blocks < 96) {
            // Runs, which read what the decays hang on twice, where even narrow workgroups leave CUs idle: for one round of
            // workgroups over the CUs, or for two and a half where that makes less than four runs; of a tile at least
            // (bf16, us, single and with runs: 1 x 16384 x 512 221 and 62, 1 x 8192 x 2560 270 and 130, 3 x 5000 x 300 110
            // and 46, 8 x 2048 x 64 67 and 28, in runs of two tiles 33; 1 x 1370 x 1152 48 and 27, of two tiles 33; but 3 x
            // 515 x 321 fp32, whose states are formed too, 20 and 31).
            const int64_t most = s.L > 6 * kTile ? ceil_div(s.L, kTile) : 1;
            want = blocks <= 64 ? 256 / blocks : 640 / blocks;
            want = want < most ? want : most;
            if (want < 4) want = 1;
        }
    }
    if (want > 1 && s.L > kTile) {
        p->seg_len = ceil_div(ceil_div(s.L, want), kTile) * kTile;
        p->segments = int32_t(ceil_div(s.L, p->seg_len));
    }
    // a grid has fewer than 2^32 threads
    return blocks_of(s, kNarrow) <= (int64_t(1) << 22) && blocks * p->segments <= (int64_t(1) << 22);
}

size_t gated_fwd_workspace_bytes(const GatedShape& s, const GatedPlan& p) { return layout_of(s, p, false, false).bytes; }

size_t gated_bwd_workspace_bytes(const GatedShape& s, const GatedPlan& p, bool ckpt_given) {
    return layout_of(s, p, true, ckpt_given).bytes;
}

namespace {
// The chain in `ws`, made ready: its words unset, and the states that it starts from copied; `from` then is the copy.
Chain start_chain(char* ws, const Layout& l, const GatedShape& s, const GatedPlan& p, const float** from,
                  hipStream_t st) {
    const int64_t rows = s.batch * s.dim, words = chain_words(s, p);
    Chain ch{};
    ch.P = reinterpret_cast<uint64_t*>(ws);
    ch.S = ch.P + p.chain * rows;
    ch.enter = ch.S + p.chain * rows;
    ch.counter = reinterpret_cast<uint32_t*>(ws + l.counter);
    ch.tiles = uint32_t(p.chain);
    float* copy = reinterpret_cast<float*>(ws + l.from);
    const int64_t groups = ceil_div(words, 1024);
    hipLaunchKernelGGL(start_chain_kernel, dim3(unsigned(groups < 4096 ? groups : 4096)), dim3(256), 0, st, ch, words,
                       *from, copy, rows);
    *from = copy;
    return ch;
}
void run_fwd_chain(const GaArgs& a, const Chain& ch, const GatedShape& s, hipStream_t st) {
    dispatch(s, a.z, [&](auto T, auto decay, auto gate, auto V) {
        const int64_t tiles = blocks_of(s, kWide) * int64_t(ch.tiles);
        hipLaunchKernelGGL((fwd_chain_kernel<decltype(T), decltype(decay)::value, decltype(gate)::value,
                                             decltype(V)::value, kWide, kNF>),
                           dim3(unsigned(tiles < kChainGroups ? tiles : kChainGroups)), dim3(kWaves * 64 + 64), 0, st, a, ch);
    });
}
}  // namespace

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
    if (p.chain) {
        const Chain ch = start_chain(static_cast<char*>(workspace), layout_of(s, p, false, false), s, p, &a.h0, stream);
        run_fwd_chain(a, ch, s, stream);
    } else {
        run_fwd<kOut>(a, s, p.segments, stream);
    }
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
        hipLaunchKernelGGL(join_kernel, dim3(unsigned(ceil_div(s.dim, 64))), dim3(1024), 0, stream, part,
                           s.batch * p.segments, s.dim, t.dA);
    return hipGetLastError();
}

hipError_t launch_gated_step(float* state, const GatedTensors& t, const GatedShape& s, hipStream_t stream) {
    const GaArgs a = args_of(t, s, GatedPlan{1, 1, 0});
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
