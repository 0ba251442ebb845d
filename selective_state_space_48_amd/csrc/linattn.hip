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
//
// What bounds it (MI355X, b8 L2048, 32 heads of 128 x 128, bf16): the bytes, 554
// MB read and written once, take 117 us at the rate of a large copy (4.75
// TB/s); a call takes 135-157 us (3.5-4.1 TB/s; by the clock). Of its
// cycles the LDS is busy in 54 %, the vector units in 47 %, the matrix cores in
// 36 %: a chunk's dependent steps (stage, scores, outputs, state) come after one
// another in a workgroup that fills its CU. fp32 (b4, 1001 tokens at most, 12 heads of
// 64 x 128: 54-57 us against 14): of the outputs' walk, 34 us, the matrix cores of
// the 192 CUs that have a workgroup are busy in 35 %, the waves wait on LDS in 2 %.
// Its steps (us a call): 241 with
// every wave in every part and three barriers; 164 staged a chunk ahead (two
// barriers); 160 with supply waves, outputs in whole rows through LDS; 151 with
// them at a raised priority. One workgroup alone on the chip takes 3.3 us a
// chunk. Tried without gain: 64 state columns and two workgroups a CU (196); the
// two halves of the waves in different orders (174); products and vector
// instructions interleaved by hand (189); one bf16 term instead of two and two
// instead of three (147 against 163 then, but off by 2^-9 of the terms);
// non-temporal loads and stores (equal); 128 columns for the slope (gradients
// 290 -> 405).
#include <initializer_list>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

constexpr int kCols = 64;   // state columns of a workgroup of the step
constexpr int kRun = 64;    // run lengths are multiples of this
// States of more bytes than this are read and written past the caches in a
// step; the 256 MB cache keeps much of a smaller one from token to token (us per
// step past the caches and through them: 671 MB 236 and 256, 284 MB 97 and 89,
// 134 MB 49 and 41).
constexpr int64_t kStreamBytes = int64_t(384) << 20;

// ---- operands of the matrix products ---------------------------------------
//
// All products are 16 x 16 tiles. Lane l = 16 g + m of an operand holds E
// consecutive contraction indices E g .. E g + E - 1 of row (or column) m, 16
// bytes; an accumulator holds rows 4 g + r, r = 0..3, of column m.

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 fma4(const f32x4& a, float b, const f32x4& c) {
    return __builtin_elementwise_fma(a, f32x4{b, b, b, b}, c);
}

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
    // v in N bf16 terms: the upper halves of v and of what is left (a mask, a
    // subtraction and half a byte permutation each; the rounding conversion
    // takes twice as long). ROUND: the second term rounded instead. Two terms are
    // then off by 2^-16 of v at most; three hold all of its 24 bits either way.
    template <int N, bool ROUND> static __device__ __forceinline__ void split(const float (&v)[E], Frag (&t)[N]) {
        float r[E];
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = v[e];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            uint32_t p[E / 2];
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                p[e / 2] = k == 1 && ROUND ? pack_bf16x2(r[e], r[e + 1]) : upper_halves(r[e], r[e + 1]);
                if (k + 1 < N) {
                    r[e] -= bf16_lo(p[e / 2]);
                    r[e + 1] -= bf16_hi(p[e / 2]);
                }
            }
            struct A { uint32_t w[E / 2]; } a;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) a.w[e] = p[e];
            t[k] = __builtin_bit_cast(Frag, a);
        }
    }
    static __device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
        return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302);
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
    template <int N, bool ROUND> static __device__ __forceinline__ void split(const float (&v)[E], Frag (&t)[N]) {
#pragma unroll
        for (int e = 0; e < E; ++e) t[0][e] = v[e];
    }
    static __device__ __forceinline__ float value(const Frag& f, int e) { return f[e]; }
};

// A tile in LDS. Padded: rows of W elements and a pad, so that 16 rows' same
// 16-byte piece (operands along rows, 16 lanes at a time) lie on 16 different
// pieces modulo 256 bytes (an odd number of pieces from row to row), and every
// address is a lane's base plus a constant; for fp32 the pad of one piece
// makes the reads of rows 4 g + e, columns m conflict-free too. X (bf16 tiles
// that are mostly read transposed): no pad, a row's pieces permuted by an XOR
// with a function of the row, which spreads those rows just as well and puts
// the halves of four pieces of rows j, j + 8 (j < 4; 32 lanes at a time) on
// every bank twice, the least that half pieces allow (the pad: three times).
template <typename T, int W, bool X> struct Tile {
    static constexpr bool kX = X && sizeof(T) == 2;
    static constexpr int kStride = kX ? W : W + (sizeof(T) == 2 ? 24 : 4);
};
template <typename T, int W, bool X>
__device__ __forceinline__ int at(int row, int col) {
    if constexpr (Tile<T, W, X>::kX) {
        const int f = W == 64 ? ((row & 2) << 1) | ((row >> 2) & 1) | ((row >> 2) & 2)
                              : ((row & 3) << 2) | ((row >> 2) & 1) | ((row >> 2) & 2);
        return row * W + (((col >> 3) ^ f) << 3) + (col & 7);
    } else {
        return row * Tile<T, W, X>::kStride + col;
    }
}

__device__ __forceinline__ bf16x4 ldtr(const bf16_bits* p) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s4*)(const_cast<bf16_bits*>(p)));
    return __builtin_bit_cast(bf16x4, v);
}

// Operand along the tile's rows: row r0 + m, columns k0 + E g ...
template <typename T, int W, bool X = false>
__device__ __forceinline__ typename Ops<T>::Frag row_frag(const T* tile, int r0, int k0, int lane) {
    using O = Ops<T>;
    return *reinterpret_cast<const typename O::Frag*>(tile + at<T, W, X>(r0 + lane % 16, k0 + O::E * (lane / 16)));
}
// Operand down the tile's columns: the contraction runs over rows k0 + E g ..,
// index m is column c0 + (m / 4) step + m % 4 (step 8: every other four columns,
// the rows of one of a pair of accumulators). The LDS transpose read hands
// lane m of a 16-lane group the elements m % 4 of what lanes 4 e + m / 4 read,
// e = 0..3 (4 rows of 16 columns, transposed).
template <typename T, int W, bool X = false>
__device__ __forceinline__ typename Ops<T>::Frag col_frag(const T* tile, int k0, int c0, int step, int lane) {
    const int g = lane / 16, m = lane % 16;
    if constexpr (sizeof(T) == 2) {
        const int row = k0 + 8 * g + m / 4, col = c0 + (m % 4) * step;
        const bf16x4 lo = ldtr(tile + at<T, W, X>(row, col)), hi = ldtr(tile + at<T, W, X>(row + 4, col));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = tile[at<T, W, X>(k0 + 4 * g + e, c0 + (m / 4) * step + m % 4)];
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
    // In 64 bits, for a power that is applied again and again.
    __device__ __forceinline__ double exact(int64_t n) const { return exp2(g2 * double(n)); }
};

// The decay of a chunk, one fp32 number per chunk whose product from any chunk
// to any other is off by a rounding or two: what a rounding takes from one is
// given to the next. (lambda^Q rounded once and applied n times is off by n
// roundings of the same sign: 2.6e-5 over 1024 chunks of 32 at lambda = 1 - 2^-9.)
struct Keep {
    float hi, lo, debt;
    __device__ __forceinline__ explicit Keep(double r)
        : hi(float(r)), lo(r < 3e38 ? float(r - double(float(r))) : 0.0f), debt(lo) {}
    __device__ __forceinline__ float next() {
        const float k = hi + debt;
        debt = debt - (k - hi) + lo;
        return k;
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
    // sums of an earlier launch's part, joined here: sum_out[h] over the batch
    // and sum_n workgroups of each (entry, head)
    const float* sum_part;
    float* sum_out;
    int32_t sum_n;
    int64_t batch;
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

__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ bool not_finite(bf16_bits x) { return (x & 0x7f80u) == 0x7f80u; }

// A run of a walk, chunk by chunk. KD: the width of a and b rounded up (64,
// 128, 256); PT: state columns of the workgroup.
// STATE: only the run's end state, into run_state. SLOPE: with the outputs,
// their derivative by log_decay, summed against `factor`.
//
// Per chunk of Q (16, 32 or 64) tokens, with H the entering state, i, j positions in walk order:
//   P_ij = lambda^(i-j) (a_i . b_j), j <= i          (scores)
//   o_i  = scale sum_j P_ij c_j + (scale or 1) lambda^(i + e0) a_i H
//   H'   = lambda^n H + (1 or scale) sum_j lambda^(n-1-j+e1) b_j^T c_j
// (e0, e1) = (1, 0) forwards, (0, 1) backwards, n tokens in the chunk.
//
// Two kinds of waves. PT / 16 compute waves hold 16 state columns each and
// form outputs and state; 4 supply waves load, stage the next chunk in the
// other half of LDS and form its scores. Two barriers a chunk:
//   outputs of chunk c   beside  staging chunk c + 1, loading c + 2
//   state over chunk c   beside  scores of chunk c + 1
constexpr int kSupply = 4;

template <typename T, int Q, int KD, int PT, bool STATE, bool SLOPE>
__global__ __launch_bounds__(PT * 4 + kSupply * 64, (PT / 16 + kSupply) / 4) void walk_kernel(WalkArgs g) {
    using O = Ops<T>;
    using Frag = typename O::Frag;
    constexpr int E = O::E, KB = O::KB, V = 16 / int(sizeof(T)), ES = int(sizeof(T));
    constexpr int NW = PT / 16, NTH = 64 * (NW + kSupply);  // compute waves; all threads
    constexpr int NS = kSupply * 64;       // supply threads
    constexpr int KT = KD / 16;            // 16-row tiles of the state
    constexpr int TT = Q / 16;             // 16-token tiles of a chunk
    constexpr int QB = Q / KB;             // operands along a chunk's tokens
    constexpr bool BF = sizeof(T) == 2;
    constexpr int NA = Q * KD / V / NS;    // 16-byte pieces of a or b per supply thread
    constexpr int NC = Q * PT / V / NS;
    constexpr int SA = Q * Tile<T, KD, false>::kStride, SB = Q * Tile<T, KD, true>::kStride, SC = Q * Tile<T, PT, false>::kStride;
    // terms of the states in the outputs and of the scores; the slope is an fp32
    // result, so its operands (the entering states, its own scores) take three
    constexpr int TS = SLOPE && BF ? 3 : O::TS, TP = O::TP, TD = BF ? 3 : 1;
    constexpr int NPS = TP + (SLOPE ? TD : 0);
    constexpr bool VIA = BF && !SLOPE;  // outputs through LDS (SLOPE: no room left)
    __shared__ alignas(16) T As2[STATE ? 1 : 2][STATE ? 16 : SA];  // chunks c (even, odd)
    __shared__ alignas(16) T Bs2[2][SB];
    __shared__ alignas(16) T Cs2[2][SC];
    __shared__ alignas(16) T Ps[STATE ? 1 : NPS][STATE ? 16 : Q * Tile<T, Q, false>::kStride];
    // bf16 outputs go through LDS: stored in whole rows by the supply waves
    constexpr int SO = PT + 8;
    __shared__ alignas(16) T Os[STATE || !VIA ? 16 : Q * SO];
    __shared__ float red[NW];
    __shared__ int odds[2];  // number + 1 of the last (even, odd) chunk with a value that is not finite

    // Weights inside a chunk are cut at the largest number, so that where a state
    // grows an empty slot's weight times its zeros stays 0. Where a token's own
    // weight is cut, the decay of its chunk or the factor of the entering state is
    // an infinity, and what comes out is not finite (a scale above 1 is in the
    // first alone, so those calls are left uncut).
    const float most = fabsf(g.scale) <= 1.0f ? 3.4028235e38f : __builtin_inff();
    auto cut = [&](float x) { return __builtin_amdgcn_fmed3f(x, -most, most); };

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

    // ---- the run's tokens: positions p0 .. p1 - 1; position i is token i, or len - 1 - i ----
    // The first chunk is the partial one, its tokens in the last slots, so that
    // the weights of the slots in the state are the same for every chunk.
    const int64_t p0 = int64_t(seg) * g.seg_len;
    const int64_t p1 = len < p0 + g.seg_len ? len : p0 + g.seg_len;
    const int nc = p1 > p0 ? int((p1 - p0 + Q - 1) / Q) : 0;
    const int skip0 = int(nc * int64_t(Q) - (p1 > p0 ? p1 - p0 : 0));  // empty slots of chunk 0
    // Loads and stores go through buffer resources of a chunk's Q rows, based
    // at its lowest token; a lane's offsets stay the same from chunk to chunk
    // (kInvalid: a column past the width, which reads 0 and is not stored).
    // Chunk 0's empty slots are kInvalid too: nothing before the run is touched.
    const int64_t t_first = w.rev ? len - (p0 - skip0) - Q : p0 - skip0;
    const int64_t t_step = w.rev ? -Q : Q;
    const int oes = w.o_f32 ? 4 : ES;
    const int col0 = tile * PT + wv * 16;  // a compute wave's first state column
    float total = 0.0f;                    // SLOPE

    if (wv >= NW) {
        // ================================ supply ================================
        // (at a raised wave priority: what the other waves wait for is never behind
        // their products; 2 % of a layer's forward and gradients)
        __builtin_amdgcn_s_setprio(3);
        const int st = tid - 64 * NW;
        const int64_t ra = h / (g.H / w.ha), rb = h / (g.H / w.hb), rc = h / (g.H / w.hc);
        const T* pa = static_cast<const T*>(w.a) + (b * g.L * w.ha + ra) * K;
        const T* pb = static_cast<const T*>(w.b) + (b * g.L * w.hb + rb) * K;
        const T* pc = static_cast<const T*>(w.c) + (b * g.L * w.hc + rc) * P;
        const int sa = w.ha * K, sb = w.hb * K, sc = w.hc * P;  // elements from token to token
        constexpr int RA = NS / (KD / V), RC = NS / (PT / V);   // rows from one of a thread's pieces to the next
        const int ia = st / (KD / V), ca = st % (KD / V) * V, ic = st / (PT / V), cc = st % (PT / V) * V;
        const int rowa = w.rev ? Q - 1 - ia - (NA - 1) * RA : ia, rowc = w.rev ? Q - 1 - ic - (NC - 1) * RC : ic;
        const int va = ca < K ? (rowa * sa + ca) * ES : kInvalid, vb = ca < K ? (rowa * sb + ca) * ES : kInvalid;
        const int vc = tile * PT + cc < P ? (rowc * sc + tile * PT + cc) * ES : kInvalid;
        u32x4 ga[STATE ? 1 : NA], gb[NA], gc[NC];
        // Past the last chunk every lane's offset is kInvalid, which reads zeros and
        // touches nothing. (A resource of no bytes would not do: the rows go into the
        // scalar offset, and whether that counts against its length is not stated.)
        auto load = [&](int c, int skip) {
            const int64_t t0 = t_first + t_step * c;
            const bool on = c < nc;
            const int oa = on ? va : kInvalid, ob = on ? vb : kInvalid, oc = on ? vc : kInvalid;
            const auto ra_ = buf_rsrc(pa + t0 * sa, ((Q - 1) * sa + K) * ES);
            const auto rb_ = buf_rsrc(pb + t0 * sb, ((Q - 1) * sb + K) * ES);
            const auto rc_ = buf_rsrc(pc + t0 * sc, ((Q - 1) * sc + P) * ES);
            auto get = [](__amdgpu_buffer_rsrc_t r, int v, int s) {
                return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, v, s, 0));
            };
#pragma unroll
            for (int k = 0; k < NA; ++k) {
                const int up_ = (w.rev ? NA - 1 - k : k) * RA;
                const bool ok = ia + k * RA >= skip;
                if (!STATE) ga[k] = get(ra_, ok ? oa : kInvalid, up_ * sa * ES);
                gb[k] = get(rb_, ok ? ob : kInvalid, up_ * sb * ES);
            }
#pragma unroll
            for (int k = 0; k < NC; ++k)
                gc[k] = get(rc_, ic + k * RC >= skip ? oc : kInvalid, (w.rev ? NC - 1 - k : k) * RC * sc * ES);
        };
        auto stage = [&](int c) {
            T* As = As2[STATE ? 0 : c & 1];
            T* Bs = Bs2[c & 1];
            T* Cs = Cs2[c & 1];
#pragma unroll
            for (int k = 0; k < NA; ++k) {
                if (!STATE) *reinterpret_cast<u32x4*>(As + at<T, KD, false>(ia + k * RA, ca)) = ga[k];
                *reinterpret_cast<u32x4*>(Bs + at<T, KD, true>(ia + k * RA, ca)) = gb[k];
            }
#pragma unroll
            for (int k = 0; k < NC; ++k) *reinterpret_cast<u32x4*>(Cs + at<T, PT, false>(ic + k * RC, cc)) = gc[k];
        };
        // Chunks with a NaN or an infinity among the values leave their number.
        auto seek = [&] {
            uint32_t found = 0;
            constexpr uint32_t X = BF ? 0x7f807f80u : 0x7f800000u, ONE = BF ? 0x00800080u : 0x00800000u;
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) found |= (gc[k][i] & X) + ONE;
            return (found & (BF ? 0x80008000u : 0x80000000u)) != 0;
        };
        load(0, skip0);
        // powers of lambda inside a 16 x 16 tile of scores, by row minus column, and between tiles
        float diag[4], base[4], pw16 = 0.0f, pw32 = 0.0f;
        if (!STATE) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = m - 4 * gq - r;
                diag[r] = d >= 0 ? cut(g.scale * dec.pow(d)) : 0.0f;
                base[r] = g.scale * dec.pow(16 + d);
            }
            pw16 = dec.pow(16);
            pw32 = dec.pow(32);
            // score tiles above the diagonal that an operand still covers stay zero
            for (int i = st; i < Q * Tile<T, Q, false>::kStride * ES / 16; i += NS)
#pragma unroll
                for (int k = 0; k < NPS; ++k) reinterpret_cast<u32x4*>(Ps[k])[i] = u32x4{0, 0, 0, 0};
        }
        // Scores of chunk c, transposed: a lane has 4 consecutive s of row t; tiles (t, s), s <= t, dealt to the waves.
        auto scores = [&](int c) {
            const T* As = As2[STATE ? 0 : c & 1];
            const T* Bs = Bs2[c & 1];
            constexpr int N = TT * (TT + 1) / 2, R = (N + kSupply - 1) / kSupply;
            int ti[R], si[R];
            f32x4 acc[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {  // (a wave without a last tile forms another's again, to the same values)
                int n = r * kSupply + wv - NW;
                n = n < N ? n : N - 1;
                ti[r] = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3;
                si[r] = n - ti[r] * (ti[r] + 1) / 2;
                acc[r] = f32x4{};
            }
#pragma unroll
            for (int kb = 0; kb < KD / KB; ++kb) {
                Frag fa[R], fb[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    fb[r] = row_frag<T, KD, true>(Bs, 16 * si[r], KB * kb, lane);
                    fa[r] = row_frag<T, KD>(As, 16 * ti[r], KB * kb, lane);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r] = O::mfma(fb[r], fa[r], acc[r]);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = 16 * ti[i] + m, s = 16 * si[i] + 4 * gq, gap = ti[i] - si[i];
                const float far = gap < 2 ? 1.0f : gap == 2 ? pw16 : pw32;
                float v[4], v2[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // (a masked score may be infinite or NaN: selected, not multiplied away)
                    v[r] = gap == 0 ? (m >= 4 * gq + r ? acc[i][r] * diag[r] : 0.0f) : acc[i][r] * cut(base[r] * far);
                    v2[r] = v[r] * float(t - s - r);
                }
                auto put = [&](int first_tile, int terms, const float (&x)[4]) {
                    if constexpr (BF) {
                        float y[4];  // (as split)
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[r] = x[r];
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            if (k >= terms) break;
                            *reinterpret_cast<u32x2*>(Ps[first_tile + k] + at<T, Q, false>(t, s)) =
                                k == 1 && terms == 2 ? u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])}
                                                     : u32x2{O::upper_halves(y[0], y[1]), O::upper_halves(y[2], y[3])};
#pragma unroll
                            for (int r = 0; r < 4; ++r) y[r] -= bf16_hi(__float_as_uint(y[r]));
                        }
                    } else {
                        *reinterpret_cast<f32x4*>(Ps[first_tile] + at<T, Q, false>(t, s)) = f32x4{x[0], x[1], x[2], x[3]};
                    }
                };
                put(0, TP, v);
                if (SLOPE) put(TP, TD, v2);
            }
        };
        // Outputs of chunk c: whole rows of the workgroup's columns.
        const int so = int(g.H) * P;
        auto store = [&](int c) {
            const auto ro = buf_rsrc(static_cast<T*>(w.o) + ((b * g.L + t_first + t_step * c) * g.H + h) * P, ((Q - 1) * so + P) * ES);
            const int skip = c == 0 ? skip0 : 0;
            u32x4 x[NC];
#pragma unroll
            for (int k = 0; k < NC; ++k) x[k] = *reinterpret_cast<const u32x4*>(Os + (ic + k * RC) * SO + cc);
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int i = ic + k * RC, row = w.rev ? Q - 1 - i : i;
                // (no scalar offset: see the compute waves' stores)
                __builtin_amdgcn_raw_buffer_store_b128(
                    x[k], ro, i >= skip && tile * PT + cc < P ? (row * so + tile * PT + cc) * ES : kInvalid, 0, 0);
            }
        };
        if (nc > 0) {
            stage(0);
            const bool found = !STATE && seek();
            load(1, 0);
            __syncthreads();
            if (!STATE) {
                if (found) odds[0] = 1;
                scores(0);
                __syncthreads();
            }
        }
        for (int c = 0; c < nc; ++c) {
            stage(c + 1);  // (past the last chunk: zeros that nothing reads)
            if (!STATE && seek()) odds[(c + 1) & 1] = c + 2;
            load(c + 2, 0);
            if (!STATE) {
                __syncthreads();
                if (VIA && !w.o_f32) store(c);
                if (c + 1 < nc) scores(c + 1);
            }
            __syncthreads();
        }
        if (!STATE && !SLOPE && g.sum_out && wv == NW && b == 0 && seg == 0 && tile == 0 && role == 0) {
            double s = 0.0;  // (lanes in turn, then halves: a fixed order)
            for (int64_t i = lane; i < g.batch * g.sum_n; i += 64)
                s += g.sum_part[(i / g.sum_n * g.H + h) * g.sum_n + i % g.sum_n];
#pragma unroll
            for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x, 64);
            if (lane == 0) g.sum_out[h] = float(s);
        }
    } else {
        // ================================ compute ================================
        const int e0 = w.rev ? 0 : 1, e1 = 1 - e0;
        const float sc_carry = w.rev ? 1.0f : g.scale, sc_upd = w.rev ? g.scale : 1.0f;
        // ---- state: tiles of 16 rows, one column of 16 per wave ----
        // An accumulator pair becomes one bf16 operand if its rows are dealt out as
        // n = 32 (kt / 2) + 8 (m / 4) + 4 (kt % 2) + m % 4.
        f32x4 S[KT];
        f32x4 D[SLOPE ? KT : 1];
        auto each_state = [&](auto f) {
            int own = lane;  // (opaque: no address is kept from the entering state's loads to the leaving one's stores)
            asm volatile("" : "+v"(own));
            const int p = col0 + own % 16, g4 = own / 16;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = BF ? 32 * (kt / 2) + 8 * g4 + 4 * (kt % 2) + r : 16 * kt + 4 * g4 + r;
                    f(kt, r, n, p, n < K && p < P);
                }
        };
        const int64_t run_at = (int64_t(role) * g.segments + seg) * g.run_stride + bh * K * P;  // STATE: of this run
        // Where the last state replaces the entering one (one role then), the last
        // run may be through before the first begins: the state pass keeps a copy
        // behind the runs' states, and the first run reads that.
        const bool copied = seg == 0 && w.s0 && w.s0 == w.s1 && (STATE || g.segments > 1);
        const int64_t copy_at = int64_t(STATE ? g.segments : g.segments - 1) * g.run_stride + bh * K * P;
        {
            // the output pass has one run more than the state pass
            const int64_t from = (int64_t(role) * (g.segments - 1) + seg - 1) * g.run_stride + bh * K * P;
            const bool own = seg == 0;
            const float* src = own ? (w.s0 ? w.s0 + bh * K * P : nullptr) : STATE ? nullptr : g.run_state + from;
            int sn = own ? w.sn : P, sp = own ? w.sp : 1;
            if (copied && !STATE) {
                src = g.run_state + copy_at;
                sn = P;
                sp = 1;
            }
            const float* dsrc = SLOPE && !STATE && !own ? g.run_slope + from : nullptr;
            each_state([&](int kt, int r, int n, int p, bool ok) {
                S[kt][r] = src && ok ? src[int64_t(n) * sn + int64_t(p) * sp] : 0.0f;
                if (SLOPE) D[kt][r] = dsrc && ok ? dsrc[int64_t(n) * P + p] : 0.0f;
                if (STATE && copied && ok) g.run_state[copy_at + int64_t(n) * P + p] = S[kt][r];
            });
        }

        float up[TT];  // of the entering state in the outputs
        if (!STATE)
#pragma unroll
            for (int k = 0; k < TT; ++k) up[k] = sc_carry * dec.pow(16 * k + m + e0);
        // weights of the chunk's tokens in the state: token KB q + s by we[s] wq[q]
        float we[E], wq[QB];
#pragma unroll
        for (int e = 0; e < E; ++e) we[e] = dec.pow(KB - 1 - E * gq - e + e1);
#pragma unroll
        for (int q = 0; q < QB; ++q) wq[q] = sc_upd * dec.pow(KB * (QB - 1 - q));

        Keep whole(dec.exact(Q));  // of the entering state over a chunk
        const int so = int(g.H) * P, po = col0 + 4 * gq;  // a lane's 4 output columns
        const int vo = po < P ? (w.rev ? 15 - m : m) * so + po : kInvalid;  // (elements)
        if (!STATE && tid < 2) odds[tid] = 0;
        if (nc > 0) {
            __syncthreads();
            if (!STATE) __syncthreads();
        }
        for (int c = 0; c < nc; ++c) {
            const int skip = c == 0 ? skip0 : 0, nv = Q - skip;
            const T* As = As2[STATE ? 0 : c & 1];
            const T* Bs = Bs2[c & 1];
            const T* Cs = Cs2[c & 1];
            if (!STATE && c < 2 && skip0 > 0) {  // into, and out of, the partial chunk
#pragma unroll
                for (int k = 0; k < TT; ++k) {
                    const int n = 16 * k + m - skip;
                    up[k] = sc_carry * dec.pow((n > 0 ? n : 0) + e0);
                }
            }
            Frag cf[QB];
#pragma unroll
            for (int q = 0; q < QB; ++q) cf[q] = col_frag<T, PT>(Cs, KB * q, wv * 16, 4, lane);
            // A masked score is a 0 in the outputs' products. Times a NaN or an infinity
            // of a later token it would not be: in a chunk with one, those values are
            // left out there and added token by token. (The marks and branches cost up to 2 %.)
            const bool odd = !STATE && __builtin_amdgcn_readfirstlane(odds[c & 1]) == c + 1;
            if (odd)
#pragma unroll
                for (int q = 0; q < QB; ++q)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (not_finite(O::value(cf[q], e))) cf[q][e] = 0;
            if (!STATE) {
                // ---- carry-in, transposed: o[p][t] = sum_n H[n][p] a[t][n] ----
                f32x4 o[TT], o2[SLOPE ? TT : 1];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    o[t] = f32x4{};
                    if (SLOPE) o2[t] = f32x4{};
                }
#pragma unroll
                for (int kb = 0; kb < KD / KB; ++kb) {
                    Frag hs[TS], f[TT];
                    float v[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] = S[BF ? 2 * kb + e / 4 : kb][e % 4];
                    O::template split<TS, true>(v, hs);
#pragma unroll
                    for (int t = 0; t < TT; ++t) f[t] = row_frag<T, KD>(As, 16 * t, KB * kb, lane);
                    // (consecutive products go to different accumulators; the slope's third term apart)
#pragma unroll
                    for (int k = 0; k < TS; ++k)
#pragma unroll
                        for (int t = 0; t < TT; ++t) {
                            if (k < O::TS) o[t] = O::mfma(hs[k], f[t], o[t]);
                            else o2[t] = O::mfma(hs[k], f[t], o2[t]);
                        }
                }
                if (SLOPE) {
                    // (loads taken ahead over this line spill: gradients of b4 L2048, 32 heads 309 us with, 278 without)
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int t = 0; t < TT; ++t) o2[t] = (o2[t] + o[t]) * float(16 * t + m - skip + 1);
#pragma unroll
                    for (int kb = 0; kb < KD / KB; ++kb) {
                        Frag hd[TS], f[TT];
                        float v[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) v[e] = D[BF ? 2 * kb + e / 4 : kb][e % 4];
                        O::template split<TS, true>(v, hd);
#pragma unroll
                        for (int t = 0; t < TT; ++t) f[t] = row_frag<T, KD>(As, 16 * t, KB * kb, lane);
#pragma unroll
                        for (int k = 0; k < TS; ++k)
#pragma unroll
                            for (int t = 0; t < TT; ++t) o2[t] = O::mfma(hd[k], f[t], o2[t]);
                    }
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (SLOPE) o2[t] *= up[t];
                    o[t] *= up[t];
                }
                const int64_t row0 = ((b * g.L + t_first + t_step * c) * g.H + h) * P;
                // (asked for here, behind the next products)
                std::conditional_t<BF, u32x2, u32x4> fac[SLOPE ? TT : 1];
                if constexpr (SLOPE) {
                    const auto rf = buf_rsrc(static_cast<const T*>(g.factor) + row0, ((Q - 1) * so + P) * ES);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        const int fo = vo >= 0 && 16 * t + m >= skip ? (vo + (w.rev ? TT - 1 - t : t) * 16 * so) * ES : kInvalid;
                        if constexpr (BF) fac[t] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rf, fo, 0, 0));
                        else fac[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rf, fo, 0, 0));
                    }
                }
                // ---- scores times c ----
#pragma unroll
                for (int q = 0; q < QB; ++q)
#pragma unroll
                    for (int k = 0; k < NPS; ++k)
#pragma unroll
                        for (int t = 0; t < TT; ++t) {
                            if (KB * q > 16 * t + 15) continue;
                            const Frag f = row_frag<T, Q>(Ps[k], 16 * t, KB * q, lane);
                            if (k < TP) o[t] = O::mfma(cf[q], f, o[t]);
                            else o2[t] = O::mfma(cf[q], f, o2[t]);
                        }
                if (odd) {
                    int own = lane;  // (opaque: no address of this path is kept beside the other)
                    asm volatile("" : "+v"(own));
                    const int row = own % 16, col = wv * 16 + own / 16 * 4;
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll 1
                        for (int s = 0; s <= 16 * t + 15; ++s) {
                            float x = 0.0f, x2 = 0.0f;
#pragma unroll
                            for (int k = 0; k < NPS; ++k)
                                (k < TP ? x : x2) += to_f32(Ps[k][at<T, Q, false>(16 * t + row, s)]);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const T y = Cs[at<T, PT, false>(s, col + r)];
                                if (!not_finite(y)) continue;
                                if (s <= 16 * t + row) o[t][r] = fmaf(x, to_f32(y), o[t][r]);
                                if (SLOPE && s < 16 * t + row) o2[t][r] = fmaf(x2, to_f32(y), o2[t][r]);
                            }
                        }
                }
                // ---- store: token 16 t + m, columns 4 gq .. 4 gq + 3 of the wave's 16 ----
                if constexpr (SLOPE) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        f32x4 f;
                        if constexpr (BF) f = f32x4{bf16_lo(fac[t][0]), bf16_hi(fac[t][0]), bf16_lo(fac[t][1]), bf16_hi(fac[t][1])};
                        else f = __builtin_bit_cast(f32x4, fac[t]);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            total = vo >= 0 && 16 * t + m >= skip ? fmaf(o2[t][r], f[r], total) : total;
                    }
                }
                if (VIA && !w.o_f32) {
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        *reinterpret_cast<u32x2*>(Os + (16 * t + m) * SO + wv * 16 + 4 * gq) =
                            u32x2{pack_bf16x2(o[t][0], o[t][1]), pack_bf16x2(o[t][2], o[t][3])};
                } else {
                    const auto ro = buf_rsrc(static_cast<char*>(w.o) + row0 * oes, ((Q - 1) * so + P) * oes);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        // The row offset goes into the lane's offset, not into a scalar one: with a
                        // scalar offset the compiler lets the next instruction overwrite the 16
                        // bytes' registers, and gfx950 has then stored the new value (seen: the
                        // first of the four).
                        const bool ok = vo >= 0 && 16 * t + m >= skip;
                        const int at_ = ok ? (vo + (w.rev ? TT - 1 - t : t) * 16 * so) * oes : kInvalid;
                        if (BF && !w.o_f32)
                            __builtin_amdgcn_raw_buffer_store_b64(
                                u32x2{pack_bf16x2(o[t][0], o[t][1]), pack_bf16x2(o[t][2], o[t][3])}, ro, at_, 0, 0);
                        else
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[t]), ro, at_, 0, 0);
                    }
                }
                __syncthreads();
            }
            // ---- state: H <- lambda^n H + B^T (w c) ----
            const float keep = skip > 0 ? dec.pow(nv) : whole.next();
            if (odd)
#pragma unroll
                for (int q = 0; q < QB; ++q) cf[q] = col_frag<T, PT>(Cs, KB * q, wv * 16, 4, lane);
            Frag cw[QB][O::TU], cd[SLOPE ? QB : 1][O::TU];
#pragma unroll
            for (int q = 0; q < QB; ++q) {
                float v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = cut(we[e] * wq[q]) * O::value(cf[q], e);
                O::template split<O::TU, false>(v, cw[q]);
                if constexpr (SLOPE) {
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] *= float(Q - 1 - (KB * q + E * gq + e) + e1);
                    O::template split<O::TU, false>(v, cd[q]);
                }
            }
#pragma unroll
            for (int kt = 0; kt < KT; kt += 4) {
                // The products are summed from zero and added to the state by the vector
                // units, which round: a bf16 matrix product cuts off what its accumulator
                // does not hold, and a state that takes six of them a chunk loses 1.5e-5 at
                // lambda = 1 - 2^-16 (1.9e-6 at most this way, of either sign).
                f32x4 u[4], ud[SLOPE ? 4 : 1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = f32x4{};
                    if (SLOPE) ud[i] = f32x4{};
                }
#pragma unroll
                for (int q = 0; q < QB; ++q) {
                    Frag f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        f[i] = BF ? col_frag<T, KD, true>(Bs, KB * q, 32 * ((kt + i) / 2) + 4 * (i % 2), 8, lane)
                                  : col_frag<T, KD, true>(Bs, KB * q, 16 * (kt + i), 4, lane);
#pragma unroll
                    for (int k = 0; k < O::TU; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            u[i] = O::mfma(f[i], cw[q][k], u[i]);
                            if (SLOPE) ud[i] = O::mfma(f[i], cd[q][k], ud[i]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (SLOPE) D[kt + i] = fma4(fma4(S[kt + i], float(nv), D[kt + i]), keep, ud[i]);
                    S[kt + i] = fma4(S[kt + i], keep, u[i]);
                }
            }
            __syncthreads();
        }

        // ---- the state leaving the run ----
        if (STATE) {
            each_state([&](int kt, int r, int n, int p, bool ok) {
                if (ok) {
                    g.run_state[run_at + int64_t(n) * P + p] = S[kt][r];
                    if (SLOPE) g.run_slope[run_at + int64_t(n) * P + p] = D[kt][r];
                }
            });
        } else if (seg == g.segments - 1) {
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
    }
    if (STATE) return;
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
        if (lane == 0 && wv < NW) red[wv] = total;
        __syncthreads();
        // [batch][H][segment * tiles + tile]
        if (tid == 0) {
            for (int i = 1; i < NW; ++i) total += red[i];
            g.part[(bh * g.segments + seg) * g.tiles + tile] = total;
        }
    }
}

// out[row, j, :] = sum of the heads' partial gradients that read kv head j, in
// order; dk (grid y 0) and dv (1).
template <typename T>
__global__ __launch_bounds__(256) void head_sum_kernel(const float* __restrict__ pk, const float* __restrict__ pv,
                                                       T* __restrict__ dk, T* __restrict__ dv, int64_t rows,
                                                       int64_t H, int64_t hkv, int wk, int wv) {
    const float* part = blockIdx.y ? pv : pk;
    T* out = blockIdx.y ? dv : dk;
    const int D = blockIdx.y ? wv : wk;
    const int64_t per = H / hkv, n = rows * hkv * D;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t d = i % D, j = i / D % hkv, row = i / D / hkv;
        const float* p = part + (row * H + j * per) * D + d;
        float s = 0.0f;
        for (int64_t r = 0; r < per; ++r) s += p[r * D];
        out[i] = from_f32<T>(s);
    }
}

// One token: the state is read and written once (the step is bound by that
// traffic: 671 MB each way take 236-245 us, 5.5-5.7 TB/s, against 4.75 TB/s of a
// large copy). A workgroup takes 64 state columns of one head; thread (nq, p4) its
// columns 4 p4 .. 4 p4 + 3 of rows nq + 16 i, all loaded before the first is
// used, so that a wave moves four whole 256-byte rows per access; the outputs'
// 16 partial sums per column meet in LDS and are added in order. STREAM: past
// the caches (non-temporal).
template <typename T, int R, bool STREAM>
__global__ __launch_bounds__(256) void linattn_step_kernel(float* __restrict__ state, const T* __restrict__ q,
                                                           const T* __restrict__ k, const T* __restrict__ v,
                                                           const float* __restrict__ log_decay, T* __restrict__ y,
                                                           int64_t H, int64_t hkv, int dk, int dv, float scale) {
    __shared__ float red[16][kCols];
    const int tid = threadIdx.x, p4 = tid % 16, nq = tid / 16;
    const int tiles = (dv + kCols - 1) / kCols;
    const int64_t bh = blockIdx.x / tiles, b = bh / H, h = bh % H, j = b * hkv + h / (H / hkv);
    const int col = int(blockIdx.x % tiles) * kCols + 4 * p4;
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < dv) {  // (dv is a multiple of 4)
        f32x4* S = reinterpret_cast<f32x4*>(state + bh * dk * dv + col);
        f32x4 s[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int n = nq + 16 * i;
            if (n < dk) s[i] = STREAM ? __builtin_nontemporal_load(S + n * (dv / 4)) : S[n * (dv / 4)];
        }
        const float lam = Decay(log_decay[h]).pow(1);
        float vv[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) vv[c] = to_f32(v[j * dv + col + c]);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int n = nq + 16 * i;
            if (n >= dk) continue;
            const float kk = to_f32(k[j * dk + n]), qq = to_f32(q[bh * dk + n]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[i][c] = fmaf(kk, vv[c], lam * s[i][c]);
                o[c] = fmaf(qq, s[i][c], o[c]);
            }
            if (STREAM) __builtin_nontemporal_store(s[i], S + n * (dv / 4));
            else S[n * (dv / 4)] = s[i];
        }
    }
    *reinterpret_cast<f32x4*>(&red[nq][4 * p4]) = f32x4{o[0], o[1], o[2], o[3]};
    __syncthreads();
    const int c = int(blockIdx.x % tiles) * kCols + tid;
    if (tid < kCols && c < dv) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += red[i][tid];
        y[bh * dv + c] = from_f32<T>(scale * sum);
    }
}

int col_tiles(int64_t P) { return int((P + kCols - 1) / kCols); }

// Workgroups of 256 threads for n items taken in strides: a grid has fewer than 2^32 threads.
dim3 grid_of(int64_t n) { return dim3(unsigned(n < (int64_t(1) << 29) ? (n + 255) / 256 : int64_t(1) << 21)); }

// Entering states of the runs: on entry run_state (and run_slope) hold the
// runs' own end states from zero (the first one's from the walk's entering
// state); on return the states leaving them. One thread per state element, in
// 64 bits: there may be many runs.
struct CarryArgs {
    float* state;
    float* slope;  // or null
    const float* log_decay;
    const int32_t* lengths;
    int64_t L, H, seg_len, stride;  // stride: floats of one run
    int32_t runs, KP;
};
__global__ __launch_bounds__(256) void carry_kernel(CarryArgs g) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < g.stride; i += int64_t(gridDim.x) * 256) {
        float* x = g.state + int64_t(blockIdx.y) * g.runs * g.stride + i;
        float* y = g.slope ? g.slope + i : nullptr;
        const int64_t bh = i / g.KP;
        const int64_t len = entry_length(g.lengths, bh / g.H, g.L);
        const Decay dec(g.log_decay[bh % g.H]);
        double s = x[0], d = y ? y[0] : 0.0;
        const double whole = dec.exact(g.seg_len);
        for (int r = 1; r < g.runs; ++r) {
            const int64_t left = len - r * g.seg_len, n = left < 0 ? 0 : left < g.seg_len ? left : g.seg_len;
            const double keep = n == g.seg_len ? whole : dec.exact(n);
            if (y) y[r * g.stride] = float(d = fma(keep, fma(double(n), s, d), double(y[r * g.stride])));
            x[r * g.stride] = float(s = fma(keep, s, double(x[r * g.stride])));
        }
    }
}

template <typename T, int Q, int KD, int PT, bool SLOPE>
void launch_walk(WalkArgs g, int64_t bh, bool state, hipStream_t st) {
    if (state) --g.segments;
    const dim3 grid(unsigned(bh * g.segments * g.roles * g.tiles)), block(PT * 4 + kSupply * 64);
    if (state) hipLaunchKernelGGL((walk_kernel<T, Q, KD, PT, true, SLOPE>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((walk_kernel<T, Q, KD, PT, false, SLOPE>), grid, block, 0, st, g);
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
        hipLaunchKernelGGL(carry_kernel, dim3(grid_of(g.run_stride).x, unsigned(g.roles)), dim3(256), 0, st, c);
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
    g.batch = s.batch;
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
    const int sums = p.segments * walk_tiles(dk, true);
    float* part = take(0);
    auto run_walks = [&](std::initializer_list<LinattnWalk> list, bool join) {
        WalkArgs g = walk_args(t, s);
        g.roles = 0;
        for (const LinattnWalk& w : list) g.w[g.roles++] = w;
        if (join) {
            g.sum_part = part;
            g.sum_out = t.dlog_decay;
            g.sum_n = sums;
        }
        walks<T>(g, s, p, false, runs, nullptr, st);
    };
    // Walks of one width share a launch; the slope's sums are joined by the last one.
    const bool slope = t.dlog_decay != nullptr;
    if (slope) {
        WalkArgs g = walk_args(t, s);
        g.w[0] = wq;
        g.roles = 1;
        g.factor = t.q;
        g.dlast = t.dlast;
        g.part = part;
        walks<T>(g, s, p, true, runs, run_slope, st);
    }
    if (dk == dv) {
        if (slope) run_walks({wk, wv}, true);
        else run_walks({wq, wk, wv}, false);
    } else {
        if (slope) run_walks({wk}, false);
        else run_walks({wq, wk}, false);
        run_walks({wv}, slope);
    }
    if (shared) {
        const int64_t rows = s.batch * s.L;
        hipLaunchKernelGGL((head_sum_kernel<T>), dim3(grid_of(rows * Hk * (dk > dv ? dk : dv)).x, 2), dim3(256), 0, st,
                           pk, pv, static_cast<T*>(t.dk), static_cast<T*>(t.dv), rows, s.heads, s.kv_heads, dk, dv);
    }
    return hipGetLastError();
}

}  // namespace

// Runs: a workgroup fills a CU (its LDS), and a second round of workgroups
// costs as much as the first, while the state pass and the carries of runs
// cost about as much as half the outputs. So a launch that leaves CUs idle is
// cut into as many runs as still fit one round of the 256 CUs, of 128 tokens
// at least, if that is worth the two launches more: with n stretches of 64
// tokens, 3.5 us (bf16; fp32 6) each in the outputs and 2.2 us in the state
// pass, S runs save 3.5 n (1 - 1 / S) and cost 2.2 n / S + 12 us (measured, us at 1, 2, 4, 8, 16, 32 runs: b1 L32771, 16 heads of 128
// 1670 1166 597 315 200 226; b1 L2048, 16 heads 114 93 60 46 43 68; b4 L2048,
// 32 heads 117 105 135 182; b8, 32 heads 160 201 267).
LinattnPlan linattn_plan(const LinattnShape& s, int32_t requested, bool backward) {
    int64_t S = requested;
    if (S == 0) {
        // the backward's launches hold the walks of dk and dv, or one walk and its slope by halves
        const int64_t wide = backward && s.dk > s.dv ? s.dk : s.dv;
        const int64_t groups = s.batch * s.heads * ((wide + 127) / 128) * (backward && s.dk == s.dv ? 2 : 1);
        S = groups > 0 ? 256 / groups : 1;
        const int64_t most = s.L / 128;
        if (S > most) S = most;
        const int64_t n = (s.L + kRun - 1) / kRun, each = s.dtype == DType::BF16 ? 35 : 60;
        if (S < 2 || each * n * (S - 1) < 22 * n + 120 * S) S = 1;
    }
    LinattnPlan p{1, s.L};
    if (S > 1 && s.L > 0) {
        const int64_t len = ((s.L + S - 1) / S + kRun - 1) / kRun * kRun;
        p.segments = int32_t((s.L + len - 1) / len);
        if (p.segments > 1) p.seg_len = len;
    }
    return p;
}
// (with several runs one state more: the copy of an entering state that is replaced)
size_t linattn_fwd_workspace_bytes(const LinattnShape& s, const LinattnPlan& p) {
    return p.segments > 1 ? up256(size_t(p.segments) * state_floats(s) * 4) : 0;
}
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

namespace {
template <typename T, int R>
void step(float* state, const void* q, const void* k, const void* v, const float* log_decay, void* y,
          const LinattnShape& s, float scale, hipStream_t st) {
    const dim3 grid(unsigned(s.batch * s.heads * col_tiles(s.dv))), block(256);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, st, state, static_cast<const T*>(q), static_cast<const T*>(k),
                           static_cast<const T*>(v), log_decay, static_cast<T*>(y), s.heads, s.kv_heads, int(s.dk),
                           int(s.dv), scale);
    };
    if (state_floats(s) * 4 > kStreamBytes) go(linattn_step_kernel<T, R, true>);
    else go(linattn_step_kernel<T, R, false>);
}
template <typename T>
void step_rows(float* state, const void* q, const void* k, const void* v, const float* log_decay, void* y,
               const LinattnShape& s, float scale, hipStream_t st) {
    if (s.dk <= 64) step<T, 4>(state, q, k, v, log_decay, y, s, scale, st);
    else if (s.dk <= 128) step<T, 8>(state, q, k, v, log_decay, y, s, scale, st);
    else step<T, 16>(state, q, k, v, log_decay, y, s, scale, st);
}
}  // namespace

hipError_t launch_linattn_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                               void* y, const LinattnShape& s, float scale, hipStream_t stream) {
    if (s.dtype == DType::BF16) step_rows<bf16_bits>(state, q, k, v, log_decay, y, s, scale, stream);
    else step_rows<float>(state, q, k, v, log_decay, y, s, scale, stream);
    return hipGetLastError();
}

}  // namespace selscan
