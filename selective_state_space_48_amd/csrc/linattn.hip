// Linear attention with a decay for each head: walks of the layer's
// recurrence (prompts and gradients) and its one-token step.
//
// A walk goes through an entry's tokens in chunks of Q (64 for bf16, 32 for
// fp32) with the K x P state of a head in matrix-core accumulators: inside a
// chunk the recurrence is a masked matrix product, between chunks the state
// carries it. The layer's output, dq, dk and dv are four walks over the same
// tensors in other roles (launch.hpp). One workgroup walks a run of one head's
// tokens for 64 or 128 state columns; where heads are few the sequence is cut
// into runs: the runs' own end states, their carries, then the outputs.
#include <initializer_list>

#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

constexpr int kCols = 64;   // state columns of a workgroup of the step
constexpr int kRun = 64;    // run lengths are multiples of this

// ---- operands of the matrix products ---------------------------------------
//
// All products are 16 x 16 tiles. Lane l = 16 g + m of an operand holds E
// consecutive contraction indices E g .. E g + E - 1 of row (or column) m, 16
// bytes; an accumulator holds rows 4 g + r, r = 0..3, of column m.

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T> struct Ops;

template <> struct Ops<bf16_bits> {
    using Frag = bf16x8;
    static constexpr int E = 8;    // contraction indices a lane holds
    static constexpr int KB = 32;  // of an operand
    // Terms that an fp32 operand is split into: scores and entering states
    // (outputs, rounded to bf16 at the end), weighted values (states, fp32).
    static constexpr int TP = 2, TS = 2, TU = 3;
    static __device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    template <int N> static __device__ __forceinline__ void split(const float (&v)[E], Frag (&t)[N]) {
        float r[E];
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = v[e];
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                t[k][e] = (__bf16)r[e];
                if (k + 1 < N) r[e] -= (float)t[k][e];
            }
    }
    static __device__ __forceinline__ float value(const Frag& f, int e) { return (float)f[e]; }
};

template <> struct Ops<float> {
    using Frag = f32x4;
    static constexpr int E = 4, KB = 16;
    static constexpr int TP = 1, TS = 1, TU = 1;
    static __device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    template <int N> static __device__ __forceinline__ void split(const float (&v)[E], Frag (&t)[N]) {
#pragma unroll
        for (int e = 0; e < E; ++e) t[0][e] = v[e];
    }
    static __device__ __forceinline__ float value(const Frag& f, int e) { return f[e]; }
};

// A tile in LDS: rows of W elements and a pad, so that 16 rows' same 16-byte
// piece (operands along rows) lie on 16 different pieces modulo 256 bytes (an
// odd number of pieces from row to row), and every address is a lane's base
// plus a constant. For bf16 the pad of 3 pieces keeps the transposed reads
// (rows j, j + 8, j < 4, of four pieces) to 3 lanes a bank; for fp32 one piece
// makes the reads of rows 4 g + e, columns m conflict-free.
template <typename T, int W> struct Tile {
    static constexpr int kStride = W + (sizeof(T) == 2 ? 24 : 4);
};
template <typename T, int W>
__device__ __forceinline__ int at(int row, int col) { return row * Tile<T, W>::kStride + col; }

__device__ __forceinline__ bf16x4 ldtr(const bf16_bits* p) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s4*)(const_cast<bf16_bits*>(p)));
    return __builtin_bit_cast(bf16x4, v);
}

// Operand along the tile's rows: row r0 + m, columns k0 + E g ...
template <typename T, int W>
__device__ __forceinline__ typename Ops<T>::Frag row_frag(const T* tile, int r0, int k0, int lane) {
    using O = Ops<T>;
    return *reinterpret_cast<const typename O::Frag*>(tile + at<T, W>(r0 + lane % 16, k0 + O::E * (lane / 16)));
}
// Operand down the tile's columns: the contraction runs over rows k0 + E g ..,
// index m is column c0 + (m / 4) step + m % 4. The LDS transpose read hands
// lane m of a 16-lane group the elements m % 4 of what lanes 4 e + m / 4 read,
// e = 0..3 (4 rows of 16 columns, transposed).
template <typename T, int W>
__device__ __forceinline__ typename Ops<T>::Frag col_frag(const T* tile, int k0, int c0, int step, int lane) {
    const int g = lane / 16, m = lane % 16;
    if constexpr (sizeof(T) == 2) {
        const int row = k0 + 8 * g + m / 4, col = c0 + (m % 4) * step;
        const bf16x4 lo = ldtr(tile + at<T, W>(row, col)), hi = ldtr(tile + at<T, W>(row + 4, col));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = tile[at<T, W>(k0 + 4 * g + e, c0 + (m / 4) * step + m % 4)];
        return v;
    }
}

// ---- powers of a head's decay ------------------------------------------------
//
// lambda^n = 2^(n log2 lambda): the exponent in 64 bits, its whole part by
// ldexp, so that the power is off by a rounding or two however large n is.
// log_decay of -inf counts as -1e30 (lambda^0 = 1, the rest 0).
struct Decay {
    double g2;  // log2 lambda
    __device__ __forceinline__ explicit Decay(float log_decay)
        : g2((log_decay < -1e30f ? -1e30 : double(log_decay)) * 1.4426950408889634074) {}
    __device__ __forceinline__ float pow(int64_t n) const {
        const double x = g2 * double(n), w = __builtin_rint(x > 2000.0 ? 2000.0 : x);
        return x < -160.0 ? 0.0f : ldexpf(exp2_hw(float(x - w)), int(w));  // (2^-150 rounds to 0)
    }
};

// ---- the walk ------------------------------------------------------------------

constexpr int kInvalid = int(0x80000000u);  // a buffer offset past every resource

struct WalkArgs {
    LinattnWalk w[3];
    int32_t roles, tiles, segments;  // segments of this launch
    int64_t seg_len;
    const float* log_decay;  // [H]
    const int32_t* lengths;  // [batch] or null
    float scale;
    int64_t L, H;
    // states of runs: [role][segment][batch * heads][K * P], local ends after
    // the state pass, the states leaving the runs after the carry pass
    float* run_state;
    int64_t run_stride;  // floats of one role and segment
    // slope: the derivatives by log_decay of the runs' states, the factor of
    // the outputs' derivatives [batch, L, H, P] (of o's kind), and the sums,
    // one per workgroup; dlast for the last state's, in s0's layout
    float* run_slope;
    const void* factor;
    const float* dlast;
    float* part;
};

__device__ __forceinline__ int64_t entry_length(const int32_t* lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < L ? n : L;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), short(0), bytes, 0x00020000);
}
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A run of a walk, chunk by chunk. KD: the width of a and b rounded up (64,
// 128, 256); PT: state columns of the workgroup, 16 per wave.
// STATE: only the run's end state, into run_state. SLOPE: with the outputs,
// their derivative by log_decay, summed against `factor`.
//
// Per chunk of Q (16, 32 or 64) tokens, with H the entering state, i, j positions in walk order:
//   P_ij = lambda^(i-j) (a_i . b_j), j <= i          (scores)
//   o_i  = scale sum_j P_ij c_j + (scale or 1) lambda^(i + e0) a_i H
//   H'   = lambda^n H + (1 or scale) sum_j lambda^(n-1-j+e1) b_j^T c_j
// (e0, e1) = (1, 0) forwards, (0, 1) backwards, n tokens in the chunk.
template <typename T, int Q, int KD, int PT, bool STATE, bool SLOPE, int WPE>
__global__ __launch_bounds__(PT * 4, WPE) void walk_kernel(WalkArgs g) {
    using O = Ops<T>;
    using Frag = typename O::Frag;
    constexpr int E = O::E, KB = O::KB, V = 16 / int(sizeof(T));
    constexpr int NW = PT / 16, NTH = 64 * NW;  // waves, threads
    constexpr int KT = KD / 16;           // 16-row tiles of the state
    constexpr int TT = Q / 16;            // 16-token tiles of a chunk
    constexpr int QB = Q / KB;            // operands along a chunk's tokens
    constexpr bool BF = sizeof(T) == 2;
    constexpr int NA = Q * KD / V / NTH;  // 16-byte pieces of a or b per thread
    constexpr int NC = Q * PT / V / NTH;
    __shared__ alignas(16) T As[STATE ? 16 : Q * Tile<T, KD>::kStride];
    __shared__ alignas(16) T Bs[Q * Tile<T, KD>::kStride];
    __shared__ alignas(16) T Cs[Q * Tile<T, PT>::kStride];
    constexpr int NPS = O::TP * (SLOPE ? 2 : 1);
    __shared__ alignas(16) T Ps[STATE ? 1 : NPS][STATE ? 16 : Q * Tile<T, Q>::kStride];
    __shared__ float red[NW];

    const int tid = threadIdx.x, lane = tid % 64, m = lane % 16, gq = lane / 16;
    const int wv = __builtin_amdgcn_readfirstlane(tid / 64);
    // Workgroups that read the same rows (column tiles, roles, heads of one kv head) run on one XCD.
    int idx = int(xcd_tile(blockIdx.x, gridDim.x));
    const int tile = idx % g.tiles; idx /= g.tiles;
    const int role = idx % g.roles; idx /= g.roles;
    const int seg = idx % g.segments;
    const int64_t bh = idx / g.segments, b = bh / g.H, h = bh % g.H;
    const LinattnWalk w = g.w[role];
    const int K = w.K, P = w.P;
    const int64_t len = entry_length(g.lengths, b, g.L);
    const Decay dec(g.log_decay[h]);
    const int e0 = w.rev ? 0 : 1, e1 = 1 - e0;
    const float sc_carry = w.rev ? 1.0f : g.scale, sc_upd = w.rev ? g.scale : 1.0f;

    // ---- state: tiles of 16 rows, one column of 16 per wave ----
    // An accumulator pair becomes one bf16 operand if its rows are dealt out as
    // n = 32 (kt / 2) + 8 (m / 4) + 4 (kt % 2) + m % 4.
    const int col0 = tile * PT + wv * 16;
    auto row_of = [&](int kt, int r) { return BF ? 32 * (kt / 2) + 8 * gq + 4 * (kt % 2) + r : 16 * kt + 4 * gq + r; };
    f32x4 S[KT];
    f32x4 D[SLOPE ? KT : 1];
    auto each_state = [&](auto f) {
        const int p = col0 + m;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = row_of(kt, r);
                f(kt, r, n, p, n < K && p < P);
            }
    };
    const int64_t run_at = (int64_t(role) * g.segments + seg) * g.run_stride + bh * K * P;  // STATE: of this run
    {
        // the output pass has one run more than the state pass
        const int64_t from = (int64_t(role) * (g.segments - 1) + seg - 1) * g.run_stride + bh * K * P;
        const bool own = seg == 0;
        const float* src = own ? (w.s0 ? w.s0 + bh * K * P : nullptr) : STATE ? nullptr : g.run_state + from;
        const int sn = own ? w.sn : P, sp = own ? w.sp : 1;
        const float* dsrc = SLOPE && !STATE && !own ? g.run_slope + from : nullptr;
        each_state([&](int kt, int r, int n, int p, bool ok) {
            S[kt][r] = src && ok ? src[int64_t(n) * sn + int64_t(p) * sp] : 0.0f;
            if (SLOPE) D[kt][r] = dsrc && ok ? dsrc[int64_t(n) * P + p] : 0.0f;
        });
    }

    // ---- powers of lambda by position ----
    float diag[4], base[4], up[TT], pw16 = 0.0f, pw32 = 0.0f;
    if (!STATE) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = m - 4 * gq - r;  // row minus column inside a 16 x 16 tile of scores
            diag[r] = d >= 0 ? g.scale * dec.pow(d) : 0.0f;
            base[r] = g.scale * dec.pow(16 + d);
        }
#pragma unroll
        for (int k = 0; k < TT; ++k) up[k] = sc_carry * dec.pow(16 * k + m + e0);
        pw16 = dec.pow(16);
        pw32 = dec.pow(32);
    }
    float wt[QB][E];  // weights of the chunk's tokens in the state
    auto weights = [&](int nv) {
#pragma unroll
        for (int q = 0; q < QB; ++q)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int s = KB * q + E * gq + e;
                wt[q][e] = s < nv ? sc_upd * dec.pow(nv - 1 - s + e1) : 0.0f;
            }
    };
    weights(Q);
    float keep = dec.pow(Q);

    // ---- the run's tokens: positions p0 .. p1 - 1; position i is token i, or len - 1 - i ----
    const int64_t p0 = int64_t(seg) * g.seg_len;
    const int64_t p1 = len < p0 + g.seg_len ? len : p0 + g.seg_len;
    const int nc = p1 > p0 ? int((p1 - p0 + Q - 1) / Q) : 0;
    const int64_t ra = h / (g.H / w.ha), rb = h / (g.H / w.hb), rc = h / (g.H / w.hc);
    const T* pa = static_cast<const T*>(w.a) + (b * g.L * w.ha + ra) * K;
    const T* pb = static_cast<const T*>(w.b) + (b * g.L * w.hb + rb) * K;
    const T* pc = static_cast<const T*>(w.c) + (b * g.L * w.hc + rc) * P;
    const int sa = w.ha * K, sb = w.hb * K, sc = w.hc * P, so = int(g.H) * P;  // elements from token to token
    auto valid = [&](int c) { const int64_t n = p1 - p0 - int64_t(c) * Q; return int(n < Q ? (n > 0 ? n : 0) : Q); };
    auto first = [&](int c, int nv) {  // lowest token of chunk c
        const int64_t p = p0 + int64_t(c) * Q;
        return w.rev ? len - p - nv : p;
    };
    auto span = [](int nv, int64_t stride, int row) { return nv > 0 ? int(((nv - 1) * stride + row) * int(sizeof(T))) : 0; };

    u32x4 ga[STATE ? 1 : NA], gb[NA], gc[NC];
    auto load = [&](int c) {
        const int nv = valid(c);
        const int64_t t0 = first(c, nv);
        const auto ra_ = buf_rsrc(pa + t0 * sa, span(nv, sa, K));
        const auto rb_ = buf_rsrc(pb + t0 * sb, span(nv, sb, K));
        const auto rc_ = buf_rsrc(pc + t0 * sc, span(nv, sc, P));
#pragma unroll
        for (int k = 0; k < NA; ++k) {
            const int i = (tid + NTH * k) / (KD / V), col = (tid + NTH * k) % (KD / V) * V;
            const int row = w.rev ? nv - 1 - i : i;
            const bool ok = i < nv && col < K;
            if (!STATE)
                ga[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                      ra_, ok ? (row * sa + col) * int(sizeof(T)) : kInvalid, 0, 0));
            gb[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rb_, ok ? (row * sb + col) * int(sizeof(T)) : kInvalid, 0, 0));
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int i = (tid + NTH * k) / (PT / V), col = tile * PT + (tid + NTH * k) % (PT / V) * V;
            const int row = w.rev ? nv - 1 - i : i;
            gc[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rc_, i < nv && col < P ? (row * sc + col) * int(sizeof(T)) : kInvalid, 0, 0));
        }
    };
    if (!STATE) {  // score tiles above the diagonal that an operand still covers stay zero
        for (int i = tid; i < Q * Tile<T, Q>::kStride * int(sizeof(T)) / 16; i += NTH)
#pragma unroll
            for (int k = 0; k < NPS; ++k) reinterpret_cast<u32x4*>(Ps[k])[i] = u32x4{0, 0, 0, 0};
    }
    float total = 0.0f;  // SLOPE
    if (nc > 0) load(0);
    for (int c = 0; c < nc; ++c) {
        const int nv = valid(c);
        if (nv < Q) {
            weights(nv);
            keep = dec.pow(nv);
        }
        __syncthreads();  // the reads of the last chunk's tiles are done
#pragma unroll
        for (int k = 0; k < NA; ++k) {
            const int i = (tid + NTH * k) / (KD / V), col = (tid + NTH * k) % (KD / V) * V;
            if (!STATE) *reinterpret_cast<u32x4*>(As + at<T, KD>(i, col)) = ga[k];
            *reinterpret_cast<u32x4*>(Bs + at<T, KD>(i, col)) = gb[k];
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int i = (tid + NTH * k) / (PT / V), col = (tid + NTH * k) % (PT / V) * V;
            *reinterpret_cast<u32x4*>(Cs + at<T, PT>(i, col)) = gc[k];
        }
        load(c + 1);  // in flight during this chunk (nothing past the last one)
        __syncthreads();

        f32x4 o[TT], o2[SLOPE && !STATE ? TT : 1];
        if (!STATE) {
            // ---- carry-in, transposed: o[p][t] = sum_n H[n][p] a[t][n] ----
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                o[t] = f32x4{};
                if (SLOPE) o2[t] = f32x4{};
            }
#pragma unroll
            for (int kb = 0; kb < KD / KB; ++kb) {
                Frag hs[O::TS], hd[O::TS];
                float v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = S[BF ? 2 * kb + e / 4 : kb][e % 4];
                O::split(v, hs);
                if (SLOPE) {
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] = D[BF ? 2 * kb + e / 4 : kb][e % 4];
                    O::split(v, hd);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const Frag f = row_frag<T, KD>(As, 16 * t, KB * kb, lane);
#pragma unroll
                    for (int k = 0; k < O::TS; ++k) {
                        o[t] = O::mfma(hs[k], f, o[t]);
                        if (SLOPE) o2[t] = O::mfma(hd[k], f, o2[t]);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (SLOPE) o2[t] = (o2[t] + o[t] * float(16 * t + m + 1)) * up[t];
                o[t] *= up[t];
            }
            // ---- scores, transposed: lane has 4 consecutive s of row t; tiles (t, s), s <= t, dealt to the waves ----
            for (int n = wv; n < TT * (TT + 1) / 2; n += NW) {
                const int ti = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3, si = n - ti * (ti + 1) / 2;
                f32x4 acc = {};
#pragma unroll
                for (int kb = 0; kb < KD / KB; ++kb)
                    acc = O::mfma(row_frag<T, KD>(Bs, 16 * si, KB * kb, lane), row_frag<T, KD>(As, 16 * ti, KB * kb, lane), acc);
                const int t = 16 * ti + m, s = 16 * si + 4 * gq;
                const float far = ti - si < 2 ? 1.0f : ti - si == 2 ? pw16 : pw32;
                float v[4], v2[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // (a masked score may be infinite or NaN: selected, not multiplied away)
                    v[r] = ti == si ? (m >= 4 * gq + r ? acc[r] * diag[r] : 0.0f) : acc[r] * (base[r] * far);
                    v2[r] = v[r] * float(t - s - r);
                }
                auto put = [&](int first_tile, const float (&x)[4]) {
                    if constexpr (BF) {
                        float y[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[r] = x[r];
#pragma unroll
                        for (int k = 0; k < O::TP; ++k) {
                            const u32x2 q = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
                            *reinterpret_cast<u32x2*>(Ps[first_tile + k] + at<T, Q>(t, s)) = q;
                            y[0] -= bf16_lo(q[0]); y[1] -= bf16_hi(q[0]);
                            y[2] -= bf16_lo(q[1]); y[3] -= bf16_hi(q[1]);
                        }
                    } else {
                        *reinterpret_cast<f32x4*>(Ps[first_tile] + at<T, Q>(t, s)) = f32x4{x[0], x[1], x[2], x[3]};
                    }
                };
                put(0, v);
                if (SLOPE) put(O::TP, v2);
            }
            __syncthreads();
        }
        // ---- outputs and state over the chunk's tokens ----
        Frag cf[QB];
#pragma unroll
        for (int q = 0; q < QB; ++q) cf[q] = col_frag<T, PT>(Cs, KB * q, wv * 16, 4, lane);
        if (!STATE) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int q = 0; q < QB; ++q) {
                    if (KB * q > 16 * t + 15) continue;
#pragma unroll
                    for (int k = 0; k < NPS; ++k) {
                        const Frag f = row_frag<T, Q>(Ps[k], 16 * t, KB * q, lane);
                        if (k < O::TP) o[t] = O::mfma(cf[q], f, o[t]);
                        else o2[t] = O::mfma(cf[q], f, o2[t]);
                    }
                }
            // ---- store: token 16 t + m, columns 4 gq .. 4 gq + 3 of the wave's 16 ----
            const int64_t t0 = first(c, nv);
            const int64_t row0 = ((b * g.L + t0) * g.H + h) * P;
            const int es = w.o_f32 ? 4 : int(sizeof(T));
            const auto ro = buf_rsrc(static_cast<char*>(w.o) + row0 * es, nv > 0 ? ((nv - 1) * so + P) * es : 0);
            const auto rf = buf_rsrc(SLOPE ? static_cast<const T*>(g.factor) + row0 : nullptr, SLOPE ? span(nv, so, P) : 0);
            const int p = col0 + 4 * gq;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int i = 16 * t + m, row = w.rev ? nv - 1 - i : i;
                const int off = i < nv && p < P ? row * so + p : -1;
                if (SLOPE) {
                    const int fo = off >= 0 ? off * int(sizeof(T)) : kInvalid;
                    f32x4 f;
                    if constexpr (BF) {
                        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rf, fo, 0, 0));
                        f = f32x4{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])};
                    } else {
                        f = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rf, fo, 0, 0));
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) total = off >= 0 ? fmaf(o2[t][r], f[r], total) : total;
                }
                if (!BF || w.o_f32) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[t]), ro, off >= 0 ? off * 4 : kInvalid, 0, 0);
                } else {
                    const u32x2 q = {pack_bf16x2(o[t][0], o[t][1]), pack_bf16x2(o[t][2], o[t][3])};
                    __builtin_amdgcn_raw_buffer_store_b64(q, ro, off >= 0 ? off * 2 : kInvalid, 0, 0);
                }
            }
        }
        // ---- state: H <- lambda^n H + B^T (w c) ----
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if (SLOPE) D[kt] = (D[kt] + S[kt] * float(nv)) * keep;
            S[kt] *= keep;
        }
#pragma unroll
        for (int q = 0; q < QB; ++q) {
            Frag cw[O::TU], cd[O::TU];
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = wt[q][e] * O::value(cf[q], e);
            O::split(v, cw);
            if (SLOPE) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] *= float(nv - 1 - (KB * q + E * gq + e) + e1);
                O::split(v, cd);
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const Frag f = BF ? col_frag<T, KD>(Bs, KB * q, 32 * (kt / 2) + 4 * (kt % 2), 8, lane)
                                  : col_frag<T, KD>(Bs, KB * q, 16 * kt, 4, lane);
#pragma unroll
                for (int k = 0; k < O::TU; ++k) {
                    S[kt] = O::mfma(f, cw[k], S[kt]);
                    if (SLOPE) D[kt] = O::mfma(f, cd[k], D[kt]);
                }
            }
        }
    }

    // ---- the state leaving the run ----
    if (STATE) {
        each_state([&](int kt, int r, int n, int p, bool ok) {
            if (ok) {
                g.run_state[run_at + int64_t(n) * P + p] = S[kt][r];
                if (SLOPE) g.run_slope[run_at + int64_t(n) * P + p] = D[kt][r];
            }
        });
        return;
    }
    if (seg == g.segments - 1) {
        if (w.s1) {
            float* dst = w.s1 + bh * K * P;
            each_state([&](int kt, int r, int n, int p, bool ok) {
                if (ok) dst[int64_t(n) * w.sn + int64_t(p) * w.sp] = S[kt][r];
            });
        }
        if (SLOPE && g.dlast) {
            const float* src = g.dlast + bh * K * P;
            each_state([&](int kt, int r, int n, int p, bool ok) {
                if (ok) total = fmaf(D[kt][r], src[int64_t(n) * w.sn + int64_t(p) * w.sp], total);
            });
        }
    }
    // ---- zeros behind the entry's tokens, as far as they lie in this run's stretch ----
    if (len < g.L && len < p0 + g.seg_len) {
        const int64_t z0 = len > p0 ? len : p0, z1 = p0 + g.seg_len < g.L ? p0 + g.seg_len : g.L;
        const int es = w.o_f32 ? 4 : int(sizeof(T)), v = 16 / es;  // columns of a 16-byte piece
        const int c1 = P - tile * PT < PT ? P - tile * PT : PT, np = (c1 + v - 1) / v;
        for (int64_t i = tid; i < (z1 - z0) * np; i += NTH) {
            const int64_t t = z0 + i / np;
            const int col = tile * PT + int(i % np) * v;
            *reinterpret_cast<u32x4*>(static_cast<char*>(w.o) + (((b * g.L + t) * g.H + h) * P + col) * es) = u32x4{0, 0, 0, 0};
        }
    }
    if (SLOPE) {
#pragma unroll
        for (int x = 32; x; x >>= 1) total += __shfl_xor(total, x, 64);
        __syncthreads();
        if (lane == 0) red[wv] = total;
        __syncthreads();
        // [batch][H][segment * tiles + tile]
        if (tid == 0) {
            for (int i = 1; i < NW; ++i) total += red[i];
            g.part[(bh * g.segments + seg) * g.tiles + tile] = total;
        }
    }
}

// dlog_decay[h] = sum over b and column tiles of the slope walk's sums, in order.
__global__ __launch_bounds__(64) void slope_sum_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                       int64_t batch, int64_t H, int tiles) {
    const int64_t h = int64_t(blockIdx.x) * 64 + threadIdx.x;
    if (h >= H) return;
    double s = 0.0;
    for (int64_t b = 0; b < batch; ++b)
        for (int i = 0; i < tiles; ++i) s += part[(b * H + h) * tiles + i];
    out[h] = float(s);
}

// out[row, j, :] = sum of the heads' partial gradients that read kv head j, in order.
template <typename T>
__global__ __launch_bounds__(256) void head_sum_kernel(const float* __restrict__ part, T* __restrict__ out,
                                                       int64_t n, int64_t H, int64_t hkv, int D) {
    const int64_t per = H / hkv;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t d = i % D, j = i / D % hkv, row = i / D / hkv;
        const float* p = part + (row * H + j * per) * D + d;
        float s = 0.0f;
        for (int64_t r = 0; r < per; ++r) s += p[r * D];
        out[i] = from_f32<T>(s);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void linattn_step_kernel(float* __restrict__ state, const T* __restrict__ q,
                                                           const T* __restrict__ k, const T* __restrict__ v,
                                                           const float* __restrict__ log_decay, T* __restrict__ y,
                                                           int64_t H, int64_t hkv, int dk, int dv, float scale) {
    __shared__ float red[4][kCols];
    const int tid = threadIdx.x, p = tid % kCols, r = tid / kCols;
    const int tiles = (dv + kCols - 1) / kCols;
    const int64_t bh = blockIdx.x / tiles, b = bh / H, h = bh % H, j = b * hkv + h / (H / hkv);
    const int col = int(blockIdx.x % tiles) * kCols + p;
    const bool live = col < dv;
    const float lam = expf(log_decay[h]);
    const float vv = live ? to_f32(v[j * dv + col]) : 0.0f;
    float o = 0.0f;
    if (live) {
        for (int n = r; n < dk; n += 4) {
            float* s = state + (bh * dk + n) * dv + col;
            const float u = fmaf(to_f32(k[j * dk + n]), vv, lam * *s);
            *s = u;
            o = fmaf(to_f32(q[bh * dk + n]), u, o);
        }
    }
    red[r][p] = o;
    __syncthreads();
    if (r == 0 && live) y[bh * dv + col] = from_f32<T>(scale * (red[0][p] + red[1][p] + red[2][p] + red[3][p]));
}

// Workgroups of 256 threads for n items taken in strides: a grid has fewer than 2^32 threads.
dim3 grid_of(int64_t n) { return dim3(unsigned(n < (int64_t(1) << 30) ? (n + 255) / 256 : int64_t(1) << 22)); }

int col_tiles(int64_t P) { return int((P + kCols - 1) / kCols); }

// Entering states of the runs: on entry run_state (and run_slope) hold the
// runs' own end states from zero (the first one's from the walk's entering
// state); on return the states leaving them. One thread per state element.
struct CarryArgs {
    float* state;
    float* slope;  // or null
    const float* log_decay;
    const int32_t* lengths;
    int64_t L, H, seg_len, stride;  // stride: floats of one run
    int32_t runs, KP;
};
__global__ __launch_bounds__(256) void carry_kernel(CarryArgs g) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= g.stride) return;
    float* x = g.state + int64_t(blockIdx.y) * g.runs * g.stride + i;
    float* y = g.slope ? g.slope + i : nullptr;
    const int64_t bh = i / g.KP;
    const int64_t len = entry_length(g.lengths, bh / g.H, g.L);
    const Decay dec(g.log_decay[bh % g.H]);
    float s = x[0], d = y ? y[0] : 0.0f;
    for (int r = 1; r < g.runs; ++r) {
        const int64_t left = len - r * g.seg_len, n = left < 0 ? 0 : left < g.seg_len ? left : g.seg_len;
        const float keep = dec.pow(n);
        if (y) y[r * g.stride] = d = fmaf(keep, fmaf(float(n), s, d), y[r * g.stride]);
        x[r * g.stride] = s = fmaf(keep, s, x[r * g.stride]);
    }
}

// Registers of two waves a SIMD hold a walk; the slope's second state at widths
// over 64 takes those of one (its workgroups have 4 waves then).
template <typename T, int Q, int KD, int PT, bool SLOPE>
void launch_walk(WalkArgs g, int64_t bh, bool state, hipStream_t st) {
    constexpr int WPE = PT == 64 && (KD == 256 || (SLOPE && KD == 128)) ? 1 : 2;
    if (state) --g.segments;
    const dim3 grid(unsigned(bh * g.segments * g.roles * g.tiles)), block(PT * 4);
    if (state) hipLaunchKernelGGL((walk_kernel<T, Q, KD, PT, true, SLOPE, WPE>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((walk_kernel<T, Q, KD, PT, false, SLOPE, WPE>), grid, block, 0, st, g);
}
template <typename T, int Q, int KD>
void launch_walk_pt(const WalkArgs& g, int64_t bh, int pt, bool state, bool slope, hipStream_t st) {
    if (slope) launch_walk<T, Q, KD, 64, true>(g, bh, state, st);
    else if (pt == 64) launch_walk<T, Q, KD, 64, false>(g, bh, state, st);
    else launch_walk<T, Q, KD, 128, false>(g, bh, state, st);
}
// The chunk is as long as its tiles fit: 64 tokens of bf16 up to width 128, 32 of fp32; half of that at width 256.
template <typename T>
void launch_walk_kd(const WalkArgs& g, int64_t bh, int pt, bool state, bool slope, hipStream_t st) {
    constexpr int Q = sizeof(T) == 2 ? 64 : 32;
    const int K = g.w[0].K;
    if (K <= 64) launch_walk_pt<T, Q, 64>(g, bh, pt, state, slope, st);
    else if (K <= 128) launch_walk_pt<T, Q, 128>(g, bh, pt, state, slope, st);
    else launch_walk_pt<T, Q / 2, 256>(g, bh, pt, state, slope, st);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t state_floats(const LinattnShape& s) { return s.batch * s.heads * s.dk * s.dv; }
// The runs' states of one role.
size_t run_bytes(const LinattnShape& s, const LinattnPlan& p) {
    return up256(size_t(p.segments - 1) * state_floats(s) * 4);
}
// The heads' own dk or dv where heads share keys and values.
size_t partial_bytes(const LinattnShape& s, int64_t D) {
    return s.heads == s.kv_heads ? 0 : up256(size_t(s.batch * s.L * s.heads * D) * 4);
}

int walk_cols(int64_t P, bool slope) { return slope || P <= 64 ? 64 : 128; }
int walk_tiles(int64_t P, bool slope) { return int((P + walk_cols(P, slope) - 1) / walk_cols(P, slope)); }

// Walks of one shape (K, P), at once: with several runs the state pass, the carries and the outputs.
template <typename T>
void walks(WalkArgs g, const LinattnShape& s, const LinattnPlan& p, bool slope, float* run_state, float* run_slope,
           hipStream_t st) {
    const int pt = walk_cols(g.w[0].P, slope);
    g.tiles = walk_tiles(g.w[0].P, slope);
    g.segments = p.segments;
    g.seg_len = p.seg_len;
    g.run_state = run_state;
    g.run_slope = slope ? run_slope : nullptr;
    g.run_stride = state_floats(s);
    const int64_t bh = s.batch * s.heads;
    if (p.segments > 1) {
        launch_walk_kd<T>(g, bh, pt, true, slope, st);
        const CarryArgs c{run_state, g.run_slope, g.log_decay, g.lengths, s.L, s.heads, p.seg_len, g.run_stride,
                          p.segments - 1, int(s.dk * s.dv)};
        hipLaunchKernelGGL(carry_kernel, dim3(unsigned((g.run_stride + 255) / 256), unsigned(g.roles)), dim3(256), 0,
                           st, c);
    }
    launch_walk_kd<T>(g, bh, pt, false, slope, st);
}

WalkArgs walk_args(const LinattnTensors& t, const LinattnShape& s) {
    WalkArgs g{};
    g.log_decay = t.log_decay;
    g.lengths = t.lengths;
    g.scale = t.scale;
    g.L = s.L;
    g.H = s.heads;
    return g;
}

template <typename T>
hipError_t bwd(const LinattnTensors& t, const LinattnShape& s, const LinattnPlan& p, void* workspace, hipStream_t st) {
    char* ws = static_cast<char*>(workspace);
    auto take = [&](size_t n) {
        float* r = reinterpret_cast<float*>(ws);
        ws += n;
        return r;
    };
    const bool shared = s.heads != s.kv_heads;
    float* pk = take(partial_bytes(s, s.dk));
    float* pv = take(partial_bytes(s, s.dv));
    const size_t run = run_bytes(s, p);
    float* runs = take(3 * run);  // one role's after the other
    float* run_slope = take(t.dlog_decay ? run : 0);
    const int H = int(s.heads), Hk = int(s.kv_heads), dk = int(s.dk), dv = int(s.dv);
    const LinattnWalk wq{t.dy, t.v, t.k, t.dq, t.h0, nullptr, H, Hk, Hk, dv, dk, 1, dv, false, false};
    const LinattnWalk wk{t.v, t.dy, t.q, shared ? pk : t.dk, t.dlast, nullptr, Hk, H, H, dv, dk, 1, dv, true, shared};
    const LinattnWalk wv{t.k, t.q, t.dy, shared ? pv : t.dv, t.dlast, t.dh0, Hk, H, H, dk, dv, dv, 1, true, shared};
    auto run_walks = [&](std::initializer_list<LinattnWalk> list) {
        WalkArgs g = walk_args(t, s);
        g.roles = 0;
        for (const LinattnWalk& w : list) g.w[g.roles++] = w;
        walks<T>(g, s, p, false, runs, nullptr, st);
    };
    if (t.dlog_decay) {
        WalkArgs g = walk_args(t, s);
        g.w[0] = wq;
        g.roles = 1;
        g.factor = t.q;
        g.dlast = t.dlast;
        g.part = take(0);
        walks<T>(g, s, p, true, runs, run_slope, st);
        hipLaunchKernelGGL(slope_sum_kernel, dim3(unsigned((H + 63) / 64)), dim3(64), 0, st, g.part, t.dlog_decay,
                           s.batch, s.heads, p.segments * walk_tiles(dk, true));
    }
    // walks of one width share a launch
    if (dk == dv && t.dlog_decay) run_walks({wk, wv});
    else if (dk == dv) run_walks({wq, wk, wv});
    else {
        if (t.dlog_decay) run_walks({wk});
        else run_walks({wq, wk});
        run_walks({wv});
    }
    if (shared) {
        const int64_t nk = s.batch * s.L * Hk * dk, nv = s.batch * s.L * Hk * dv;
        hipLaunchKernelGGL((head_sum_kernel<T>), grid_of(nk), dim3(256), 0, st, pk, static_cast<T*>(t.dk), nk, s.heads,
                           s.kv_heads, dk);
        hipLaunchKernelGGL((head_sum_kernel<T>), grid_of(nv), dim3(256), 0, st, pv, static_cast<T*>(t.dv), nv, s.heads,
                           s.kv_heads, dv);
    }
    return hipGetLastError();
}

}  // namespace

LinattnPlan linattn_plan(const LinattnShape& s, int32_t requested, bool backward) {
    int64_t S = requested;
    if (S == 0) {
        S = 1;
        const int64_t groups = s.batch * s.heads * ((s.dv + 127) / 128) * (backward ? 2 : 1);
        if (groups > 0 && groups < 512) S = (512 + groups - 1) / groups;
        const int64_t most = s.L / (4 * kRun);
        if (S > most) S = most;
        if (S > 1024) S = 1024;
        if (S < 1) S = 1;
    }
    LinattnPlan p{1, s.L};
    if (S > 1 && s.L > 0) {
        const int64_t len = ((s.L + S - 1) / S + kRun - 1) / kRun * kRun;
        p.segments = int32_t((s.L + len - 1) / len);
        if (p.segments > 1) p.seg_len = len;
    }
    return p;
}
size_t linattn_fwd_workspace_bytes(const LinattnShape& s, const LinattnPlan& p) { return run_bytes(s, p); }
size_t linattn_bwd_workspace_bytes(const LinattnShape& s, const LinattnPlan& p, bool slope) {
    return partial_bytes(s, s.dk) + partial_bytes(s, s.dv) + (slope ? 4 : 3) * run_bytes(s, p) +
           (slope ? up256(size_t(s.batch * s.heads * p.segments * walk_tiles(s.dk, true)) * 4) : 0);
}

hipError_t launch_linattn_fwd(const LinattnTensors& t, const LinattnShape& s, const LinattnPlan& p, void* workspace,
                              hipStream_t stream) {
    const int H = int(s.heads), Hk = int(s.kv_heads), dk = int(s.dk), dv = int(s.dv);
    WalkArgs g = walk_args(t, s);
    g.w[0] = {t.q, t.k, t.v, t.y, t.h0, t.last_state, H, Hk, Hk, dk, dv, dv, 1, false, false};
    g.roles = 1;
    if (s.dtype == DType::BF16) walks<bf16_bits>(g, s, p, false, static_cast<float*>(workspace), nullptr, stream);
    else walks<float>(g, s, p, false, static_cast<float*>(workspace), nullptr, stream);
    return hipGetLastError();
}

hipError_t launch_linattn_bwd(const LinattnTensors& t, const LinattnShape& s, const LinattnPlan& p, void* workspace,
                              hipStream_t stream) {
    return s.dtype == DType::BF16 ? bwd<bf16_bits>(t, s, p, workspace, stream) : bwd<float>(t, s, p, workspace, stream);
}

hipError_t launch_linattn_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                               void* y, const LinattnShape& s, float scale, hipStream_t stream) {
    const dim3 grid(unsigned(s.batch * s.heads * col_tiles(s.dv))), block(256);
    const int dk = int(s.dk), dv = int(s.dv);
    if (s.dtype == DType::BF16)
        hipLaunchKernelGGL((linattn_step_kernel<bf16_bits>), grid, block, 0, stream, state,
                           static_cast<const bf16_bits*>(q), static_cast<const bf16_bits*>(k),
                           static_cast<const bf16_bits*>(v), log_decay, static_cast<bf16_bits*>(y), s.heads,
                           s.kv_heads, dk, dv, scale);
    else
        hipLaunchKernelGGL((linattn_step_kernel<float>), grid, block, 0, stream, state, static_cast<const float*>(q),
                           static_cast<const float*>(k), static_cast<const float*>(v), log_decay,
                           static_cast<float*>(y), s.heads, s.kv_heads, dk, dv, scale);
    return hipGetLastError();
}

}  // namespace selscan
