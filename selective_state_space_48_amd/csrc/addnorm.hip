// Norms around a block with the residual sum between them, and the gradients.
//
// Bound by memory: a row is held in registers, read once and written once. A
// thread holds a vector of 8 values of a row (two above 8192), `lanes` threads a
// row: a power of two of a wave's lanes for narrow rows (several a workgroup),
// whole waves for wide ones (sums over the waves through LDS, one barrier each, as
// the entries alternate). Sums over lanes are moves of the vector unit: through LDS
// 8192 x 5120 bf16 took 131 us instead of 80. Workgroups go over their rows with the
// weights kept in registers and the next row's loads in flight.
//
// Statistics in fp32: a mean, then the squares about it. Backward, a workgroup adds
// what its rows give to the gradients of weights, biases and gate in registers and
// writes them once; join_kernel adds the workgroups' parts in order.
//
// 16384 x 4096 bf16, both norms, residual fp32: 145 to 148 us (5.5 TB/s; a large copy has 4.9);
// gradients with biases and 8 gate rows, residual bf16: 172 (4.8 with the parts).
#include "../../include/selscan.h"
#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

struct AnArgs {
    AddnormTensors t;
    int64_t R, C, per_gate;  // rows of a gate row (R without a gate)
    int32_t post, pre;
    float eps, scale, res_scale;
    int32_t lanes;  // threads of a row
    // backward: workgroups of a gate row (0: a workgroup takes whole gate rows), rows of a workgroup
    int64_t runs, per;
    float* part;       // [workgroup][kind of sum][C]
    float* gate_part;  // [workgroup][C], or dgate itself where a workgroup takes whole gate rows
    float* averages;   // [R][2], rows of more than 512 threads: what cols_kernel needs of a row
};

constexpr int kV = 8;  // values of a vector

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any element: rows of a width that is no multiple of 8 begin anywhere
struct __attribute__((packed, aligned(2))) Any16 { u32x4 v; };

template <typename T> struct Vec;
template <> struct Vec<float> {
    u32x4 a, b;
    __device__ __forceinline__ void get(float (&f)[kV]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __uint_as_float(a[i]);
            f[4 + i] = __uint_as_float(b[i]);
        }
    }
};
template <> struct Vec<bf16_bits> {
    u32x4 a;
    __device__ __forceinline__ void get(float (&f)[kV]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(a[i]);
            f[2 * i + 1] = bf16_hi(a[i]);
        }
    }
};

// Rows of whole vectors; of others (their last vector ends at the row's end, and the values before `lo` are another
// thread's: loads then take no branch, and what is loaded early stays in flight; value by value 50445 x 495 bf16 took
// 57 us instead of 34, its gradients 176 instead of 77); of fewer than 8 values.
enum { kWhole, kPart, kFew };

// A vector's first column (below 0 for kFew), and its first value that is the thread's own: 8 if it has none.
struct Column {
    int c, lo;
    __device__ __forceinline__ Column() {}
    __device__ __forceinline__ Column(int vector, int64_t C) {
        const int at = vector * kV, last = int(C) - kV;
        c = at < last ? at : last;
        lo = at - c < kV ? at - c : kV;
    }
};

template <int EDGE, typename T> __device__ __forceinline__ Vec<T> load(const void* base, int64_t at, int lo) {
    const T* p = static_cast<const T*>(base) + at;
    Vec<T> v{};
    if constexpr (EDGE != kFew) {
        v.a = reinterpret_cast<const Any16*>(p)->v;
        if constexpr (sizeof(T) == 4) v.b = reinterpret_cast<const Any16*>(p + 4)->v;
    } else {
        struct Values { T t[kV]; } s{};
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i >= lo) s.t[i] = p[i];
        v = __builtin_bit_cast(Vec<T>, s);
    }
    return v;
}
template <int EDGE, typename T>
__device__ __forceinline__ void store(void* base, int64_t at, int lo, const float (&f)[kV]) {
    T* p = static_cast<T*>(base) + at;
    if (EDGE != kFew && lo == 0) {
        if constexpr (sizeof(T) == 4) {
            u32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __float_as_uint(f[i]);
                b[i] = __float_as_uint(f[4 + i]);
            }
            reinterpret_cast<Any16*>(p)->v = a;
            reinterpret_cast<Any16*>(p + 4)->v = b;
        } else {
            u32x4 a;
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
            reinterpret_cast<Any16*>(p)->v = a;
        }
    } else if constexpr (EDGE != kWhole) {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i >= lo) p[i] = from_f32<T>(f[i]);
    }
}
// Weights, `dflt` without them.
template <int EDGE> __device__ __forceinline__ void weights(const float* w, const Column& c, float dflt, float (&f)[kV]) {
    if (w) {
        load<EDGE, float>(w, c.c, c.lo).get(f);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) f[i] = dflt;
    }
}
// A value's term of a row's sum: only the thread's own count. (Whole vectors: their sum at once, own().)
template <int EDGE> __device__ __forceinline__ float term(float t, int i, int lo) {
    return EDGE != kWhole && i < lo ? 0.0f : t;
}
template <int EDGE> __device__ __forceinline__ float own(float sum, int lo) { return EDGE == kWhole && lo ? 0.0f : sum; }

// Sums over the lanes of a wave, by moves inside the vector unit: every lane adds its partner's value (neighbours,
// then pairs, quads, ...), so that all end with the same bits. M: lanes that are summed, a power of two.
template <int CTRL> __device__ __forceinline__ float partner(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float add_16(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}
__device__ __forceinline__ float add_32(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}
__device__ __forceinline__ void lane_sums(int m, float& a, float& b) {
    if (m < 2) return;
    a += partner<0xB1>(a); b += partner<0xB1>(b);      // the neighbour
    if (m < 4) return;
    a += partner<0x4E>(a); b += partner<0x4E>(b);      // the other pair of four
    if (m < 8) return;
    a += partner<0x141>(a); b += partner<0x141>(b);    // mirrored in eight
    if (m < 16) return;
    a += partner<0x140>(a); b += partner<0x140>(b);   // mirrored in sixteen
    if (m < 32) return;
    a = add_16(a); b = add_16(b);
    if (m < 64) return;
    a = add_32(a); b = add_32(b);
}

// A thread's place, and sums over a row: in the lanes of a wave (WIDE false), or over the workgroup.
template <bool WIDE> struct Row {
    int l, ri, step, lanes;
    float2 (*red)[16];
    int slot = 0;
    __device__ __forceinline__ Row(int lanes_, float2 (*red_)[16]) : lanes(lanes_), red(red_) {
        l = WIDE ? threadIdx.x : threadIdx.x % lanes;
        ri = WIDE ? 0 : threadIdx.x / lanes;
        step = WIDE ? 1 : 256 / lanes;
    }
    __device__ __forceinline__ void sums(float& a, float& b) {
        if constexpr (WIDE) {
            lane_sums(64, a, b);
            if (threadIdx.x % 64 == 0) red[slot][threadIdx.x / 64] = {a, b};
            __syncthreads();
            const uint32_t i = threadIdx.x % 16;
            const float2 w = i < blockDim.x / 64 ? red[slot][i] : float2{0.0f, 0.0f};
            a = w.x;
            b = w.y;
            lane_sums(16, a, b);
            // an entry is written again only behind a barrier that follows every read of it
            slot ^= 1;
        } else {
            lane_sums(lanes, a, b);
        }
    }
    __device__ __forceinline__ float sum(float a) {
        float b = 0.0f;
        sums(a, b);
        return a;
    }
};

// mean and 1 / sqrt of a row's values.
template <int K, int EDGE, bool WIDE>
__device__ __forceinline__ void statistics(int kind, const float (&v)[K][kV], const Column (&c)[K], float inv, float eps,
                                           Row<WIDE>& row, float* mean, float* rstd) {
    *mean = 0.0f;
    float s = 0.0f;
    if (kind == SELSCAN_NORM_LAYER) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float p = 0.0f;
#pragma unroll
            for (int i = 0; i < kV; ++i) p += term<EDGE>(v[k][i], i, c[k].lo);
            s += own<EDGE>(p, c[k].lo);
        }
        *mean = row.sum(s) * inv;
        s = 0.0f;
    }
    // (an RMS norm's mean is 0)
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float p = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const float d = term<EDGE>(v[k][i] - *mean, i, c[k].lo);
            p = fmaf(d, d, p);
        }
        s += own<EDGE>(p, c[k].lo);
    }
    // (off by one rounding; what it would flush is left to the root and the division)
    const float q = row.sum(s) * inv + eps;
    *rstd = q < 1e-36f ? 1.0f / sqrtf(q) : __builtin_amdgcn_rsqf(q);
}

// K: vectors of a thread. With one, weights and the next row's loads stay in registers.
template <typename T, typename S, int K, bool WIDE, int EDGE>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void fwd_kernel(AnArgs a) {
    constexpr bool KEEP = K == 1;
    __shared__ float2 red[2][16];
    Row<WIDE> row(a.lanes, red);
    const AddnormTensors& t = a.t;
    const bool post = a.post != SELSCAN_NORM_NONE, pre = a.pre != SELSCAN_NORM_NONE;
    Column c[K];
    float w1[KEEP ? K : 1][kV], w2[KEEP ? K : 1][kV];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        c[k] = Column(row.l + a.lanes * k, a.C);
        if constexpr (KEEP) {
            weights<EDGE>(post ? t.post_w : nullptr, c[k], 1.0f, w1[k]);
            weights<EDGE>(pre ? t.pre_w : nullptr, c[k], 1.0f, w2[k]);
        }
    }
    const float inv = 1.0f / float(a.C > 0 ? a.C : 1);
    Vec<T> nx[K];
    Vec<S> ns[K];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t at = r * a.C + c[k].c;
            nx[k] = load<EDGE, T>(t.x, at, c[k].lo);
            if (t.res) ns[k] = load<EDGE, S>(t.res, at, c[k].lo);
        }
    };
    const int64_t stride = int64_t(gridDim.x) * row.step;
    int64_t r = int64_t(blockIdx.x) * row.step + row.ri;
    if (KEEP && r < a.R) fetch(r);
    for (; r < a.R; r += stride) {
        float v[K][kV], s[K][kV];
        if (!KEEP) fetch(r);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            nx[k].get(v[k]);
#pragma unroll
            for (int i = 0; i < kV; ++i) s[k][i] = 0.0f;
            if (t.res) {
                ns[k].get(s[k]);
#pragma unroll
                for (int i = 0; i < kV; ++i) s[k][i] *= a.res_scale;
            }
        }
        if (KEEP && r + stride < a.R) fetch(r + stride);
        float m1 = 0.0f, r1 = 1.0f, m2 = 0.0f, r2 = 1.0f;
        if (post) statistics<K, EDGE>(a.post, v, c, inv, a.eps, row, &m1, &r1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float (&u)[kV] = v[k];
            if (post) {
                float (&w)[kV] = w1[KEEP ? k : 0];
                if constexpr (!KEEP) weights<EDGE>(t.post_w, c[k], 1.0f, w);
#pragma unroll
                for (int i = 0; i < kV; ++i) u[i] = (u[i] - m1) * r1 * w[i];
                if (t.post_b) {
                    float b[kV];
                    load<EDGE, float>(t.post_b, c[k].c, c[k].lo).get(b);
#pragma unroll
                    for (int i = 0; i < kV; ++i) u[i] += b[i];
                }
            }
            if (t.gate) {
                float g[kV];
                load<EDGE, float>(t.gate + r / a.per_gate * a.C, c[k].c, c[k].lo).get(g);
#pragma unroll
                for (int i = 0; i < kV; ++i) s[k][i] = fmaf(u[i], a.scale * g[i], s[k][i]);
            } else {
#pragma unroll
                for (int i = 0; i < kV; ++i) s[k][i] = fmaf(u[i], a.scale, s[k][i]);
            }
            if (t.sum) store<EDGE, S>(t.sum, r * a.C + c[k].c, c[k].lo, s[k]);
        }
        if (pre) {
            statistics<K, EDGE>(a.pre, s, c, inv, a.eps, row, &m2, &r2);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float y[kV];
                float (&w)[kV] = w2[KEEP ? k : 0];
                if constexpr (!KEEP) weights<EDGE>(t.pre_w, c[k], 1.0f, w);
#pragma unroll
                for (int i = 0; i < kV; ++i) y[i] = (s[k][i] - m2) * r2 * w[i];
                if (t.pre_b) {
                    float b[kV];
                    load<EDGE, float>(t.pre_b, c[k].c, c[k].lo).get(b);
#pragma unroll
                    for (int i = 0; i < kV; ++i) y[i] += b[i];
                }
                if (t.y) store<EDGE, T>(t.y, r * a.C + c[k].c, c[k].lo, y);
            }
        }
        if (t.stats && row.l == 0) {
            const float st[4] = {m1, r1, m2, r2};
#pragma unroll
            for (int i = 0; i < 4; ++i) t.stats[r * 4 + i] = st[i];
        }
    }
}

// The sums that the backward pass forms over rows, by what is wanted of them: weights (0, 1), biases (2, 3).
enum { kPreW = 0, kPostW = 1, kPreB = 2, kPostB = 3 };

// ROWS: rows in a wave's lanes, of up to 512, 768 or 1024 threads (256, 168 and 128 registers), or of threads whose
// registers the sums do not fit, one vector each or two: the rows alone, and their averages for cols_kernel, which then
// writes dres.
enum { kLanes, k512, k768, k1024, kApart, kApart2 };
template <typename T, typename S, int ROWS, bool BIAS, bool GATE, int EDGE>
__global__ __launch_bounds__(ROWS == kLanes ? 256 : ROWS == k512 ? 512 : ROWS == k768 ? 768 : 1024,
                             ROWS == kLanes && sizeof(S) == 2 && !BIAS && !GATE ? 4 : 1) void bwd_kernel(AnArgs a) {
    constexpr bool WIDE = ROWS != kLanes, SUMS = ROWS < kApart;
    constexpr int K = ROWS == kApart2 ? 2 : 1;
    __shared__ float2 red[2][16];
    __shared__ float cols[WIDE ? 1 : 256 * kV];
    Row<WIDE> row(a.lanes, red);
    const AddnormTensors& t = a.t;
    const bool post = a.post != SELSCAN_NORM_NONE, pre = a.pre != SELSCAN_NORM_NONE;
    const bool use_x = post || (SUMS && GATE && t.dgate);
    constexpr int NS = BIAS ? 4 : 2, KW = SUMS ? K : 1;
    Column col[K];
    float w1[KW][kV], w2[KW][kV], acc[NS][KW][kV], accg[GATE ? KW : 1][kV];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        col[k] = Column(row.l + a.lanes * k, a.C);
        if constexpr (SUMS) {
            weights<EDGE>(post ? t.post_w : nullptr, col[k], 1.0f, w1[k]);
            weights<EDGE>(pre ? t.pre_w : nullptr, col[k], 1.0f, w2[k]);
        }
        if constexpr (SUMS)
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[j][k][i] = 0.0f;
    }
    const float inv = 1.0f / float(a.C);
    // The thread's sums of its columns joined over the workgroup's rows and written to out[0 .. C).
    auto flush = [&](const float (&f)[KW][kV], float* out) {
        if constexpr (!WIDE) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (i >= col[0].lo) cols[row.ri * a.lanes * kV + col[0].c + i] = f[0][i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.C; c += 256) {
                float s = cols[c];
                for (int j = 1; j < row.step; ++j) s += cols[j * a.lanes * kV + c];
                out[c] = s;
            }
        } else {
#pragma unroll
            for (int k = 0; k < KW; ++k) store<EDGE, float>(out, col[k].c, col[k].lo, f[k]);
        }
    };
    // Rows r0 .. r1 of the workgroup, one gate row's at a time.
    int64_t r0, r1;
    if (a.runs) {
        const int64_t g = blockIdx.x / a.runs;
        r0 = g * a.per_gate + blockIdx.x % a.runs * a.per;
        const int64_t e = (g + 1) * a.per_gate;
        r1 = r0 + a.per < e ? r0 + a.per : e;
    } else {
        r0 = blockIdx.x * a.per;
        r1 = r0 + a.per < a.R ? r0 + a.per : a.R;
    }
    Vec<T> nx[K], ny[K];
    Vec<S> ns[K], nd[K];
    float nst[4] = {0.0f, 1.0f, 0.0f, 1.0f};
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t at = r * a.C + col[k].c;
            if (use_x) nx[k] = load<EDGE, T>(t.x, at, col[k].lo);
            if (pre) {
                ns[k] = load<EDGE, S>(t.sum, at, col[k].lo);
                ny[k] = load<EDGE, T>(t.dy, at, col[k].lo);
            }
            if (t.dsum) nd[k] = load<EDGE, S>(t.dsum, at, col[k].lo);
        }
        if (t.stats)
#pragma unroll
            for (int i = 0; i < 4; ++i) nst[i] = t.stats[r * 4 + i];
    };
    // What else a row's vector needs: the gradient from behind, and x (normed by post).
    auto passed = [&](int k, float m1, float q1, float (&ds)[kV], float (&x1)[kV]) {
#pragma unroll
        for (int i = 0; i < kV; ++i) ds[i] = x1[i] = 0.0f;
        if (t.dsum) nd[k].get(ds);
        if (use_x) {
            nx[k].get(x1);
            if (post)
#pragma unroll
                for (int i = 0; i < kV; ++i) x1[i] = (x1[i] - m1) * q1;
        }
    };
    for (int64_t g0 = r0; g0 < r1;) {
        const int64_t gi = g0 / a.per_gate, end = (gi + 1) * a.per_gate, g1 = end < r1 ? end : r1;
        float gate[GATE ? KW : 1][kV];
        if constexpr (GATE && SUMS)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                weights<EDGE>(t.gate ? t.gate + gi * a.C : nullptr, col[k], 1.0f, gate[k]);
#pragma unroll
                for (int i = 0; i < kV; ++i) accg[k][i] = 0.0f;
            }
        int64_t r = g0 + row.ri;
        if (SUMS && r < g1) fetch(r);
        for (; r < g1; r += row.step) {
            // (without the sums two vectors' values would spill: each tensor is loaded where it is needed)
            if (!SUMS && t.stats)
#pragma unroll
                for (int i = 0; i < 4; ++i) nst[i] = t.stats[r * 4 + i];
            float ds[K][kV], xh[K][kV], e[K][kV], x1[K][kV];
            const float m1 = nst[0], q1 = nst[1], m2 = nst[2], q2 = nst[3];
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if constexpr (SUMS) passed(k, m1, q1, ds[k], x1[k]);
                if (pre) {
                    float dy[kV];
                    if constexpr (!SUMS) {
                        const int64_t at = r * a.C + col[k].c;
                        ns[k] = load<EDGE, S>(t.sum, at, col[k].lo);
                        ny[k] = load<EDGE, T>(t.dy, at, col[k].lo);
                    }
                    ns[k].get(xh[k]);
                    ny[k].get(dy);
                    float (&w)[kV] = w2[SUMS ? k : 0];
                    if constexpr (!SUMS) weights<EDGE>(t.pre_w, col[k], 1.0f, w);
                    float p1 = 0.0f, p2 = 0.0f;
#pragma unroll
                    for (int i = 0; i < kV; ++i) {
                        xh[k][i] = (xh[k][i] - m2) * q2;
                        e[k][i] = term<EDGE>(dy[i] * w[i], i, col[k].lo);
                        p1 += e[k][i];
                        p2 = fmaf(e[k][i], xh[k][i], p2);
                        if constexpr (SUMS) acc[kPreW][k][i] = fmaf(dy[i], xh[k][i], acc[kPreW][k][i]);
                        if constexpr (SUMS && BIAS) acc[kPreB][k][i] += dy[i];
                    }
                    s1 += own<EDGE>(p1, col[k].lo);
                    s2 += own<EDGE>(p2, col[k].lo);
                }
            }
            if (SUMS && r + row.step < g1) fetch(r + row.step);
            if (pre) {
                row.sums(s1, s2);
                const float a1 = a.pre == SELSCAN_NORM_LAYER ? s1 * inv : 0.0f, a2 = s2 * inv;
                if (!SUMS && a.averages && row.l == 0) {
                    a.averages[r * 2] = a1;
                    a.averages[r * 2 + 1] = a2;
                }
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < kV; ++i) {
                        e[k][i] = q2 * (e[k][i] - a1 - xh[k][i] * a2);
                        if constexpr (SUMS) ds[k][i] += e[k][i];
                    }
            }
            if constexpr (!SUMS)
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int64_t at = r * a.C + col[k].c;
                    if (use_x) nx[k] = load<EDGE, T>(t.x, at, col[k].lo);
                    if (t.dsum) nd[k] = load<EDGE, S>(t.dsum, at, col[k].lo);
                    passed(k, m1, q1, ds[k], x1[k]);
                    if (pre)
#pragma unroll
                        for (int i = 0; i < kV; ++i) ds[k][i] += e[k][i];
                }
            s1 = s2 = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int64_t at = r * a.C + col[k].c;
                if (t.dres && (SUMS || !a.averages)) {
                    float o[kV];
#pragma unroll
                    for (int i = 0; i < kV; ++i) o[i] = a.res_scale * ds[k][i];
                    store<EDGE, S>(t.dres, at, col[k].lo, o);
                }
                float b1[kV];
                if constexpr (GATE && SUMS) weights<EDGE>(post ? t.post_b : nullptr, col[k], 0.0f, b1);
                float (&w)[kV] = w1[SUMS ? k : 0];
                float (&gt)[kV] = gate[GATE && SUMS ? k : 0];
                if constexpr (!SUMS) {
                    weights<EDGE>(post ? t.post_w : nullptr, col[k], 1.0f, w);
                    if constexpr (GATE) weights<EDGE>(t.gate + gi * a.C, col[k], 1.0f, gt);
                }
                float p1 = 0.0f, p2 = 0.0f;
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    float du = a.scale * ds[k][i];
                    if constexpr (GATE) {
                        if constexpr (SUMS) accg[k][i] = fmaf(du, fmaf(x1[k][i], w[i], b1[i]), accg[k][i]);
                        du *= gt[i];
                    }
                    if (post) {
                        if constexpr (SUMS) acc[kPostW][k][i] = fmaf(du, x1[k][i], acc[kPostW][k][i]);
                        if constexpr (SUMS && BIAS) acc[kPostB][k][i] += du;
                        du = term<EDGE>(du * w[i], i, col[k].lo);
                        p1 += du;
                        p2 = fmaf(du, x1[k][i], p2);
                    }
                    ds[k][i] = du;
                }
                s1 += own<EDGE>(p1, col[k].lo);
                s2 += own<EDGE>(p2, col[k].lo);
            }
            if (post) {
                row.sums(s1, s2);
                const float a1 = a.post == SELSCAN_NORM_LAYER ? s1 * inv : 0.0f, a2 = s2 * inv;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < kV; ++i) ds[k][i] = q1 * (ds[k][i] - a1 - x1[k][i] * a2);
            }
            if (t.dx)
#pragma unroll
                for (int k = 0; k < K; ++k) store<EDGE, T>(t.dx, r * a.C + col[k].c, col[k].lo, ds[k]);
        }
        if constexpr (GATE && SUMS)
            if (t.dgate) flush(accg, a.gate_part + (a.runs ? int64_t(blockIdx.x) : gi) * a.C);
        g0 = g1;
    }
    if constexpr (SUMS) {
        if (!a.part) return;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            float* want = j == kPreW ? t.dpre_w : j == kPostW ? t.dpost_w : j == kPreB ? t.dpre_b : t.dpost_b;
            if (want) flush(acc[j], a.part + (int64_t(blockIdx.x) * NS + j) * a.C);
        }
    }
}

// The sums over rows where bwd_kernel does not form them: a thread takes a vector of columns down the rows of its
// workgroup (grid x), from the averages that bwd_kernel left. It writes dres too, which may stand in dsum's place.
template <typename T, typename S, int EDGE>
__global__ __launch_bounds__(64) void cols_kernel(AnArgs a, int NS) {
    const AddnormTensors& t = a.t;
    const int64_t blk = blockIdx.x;
    const Column c(int(blockIdx.y * 64 + threadIdx.x), a.C);
    const bool post = a.post != SELSCAN_NORM_NONE, pre = a.pre != SELSCAN_NORM_NONE;
    const bool use_x = post || t.dgate;
    if (c.lo == kV) return;
    int64_t r0, r1;
    if (a.runs) {
        const int64_t g = blk / a.runs, e = (g + 1) * a.per_gate;
        r0 = g * a.per_gate + blk % a.runs * a.per;
        r1 = r0 + a.per < e ? r0 + a.per : e;
    } else {
        r0 = blk * a.per;
        r1 = r0 + a.per < a.R ? r0 + a.per : a.R;
    }
    float w1[kV], b1[kV], w2[kV], gate[kV], acc[5][kV];
    weights<EDGE>(post ? t.post_w : nullptr, c, 1.0f, w1);
    weights<EDGE>(post ? t.post_b : nullptr, c, 0.0f, b1);
    weights<EDGE>(pre ? t.pre_w : nullptr, c, 1.0f, w2);
    weights<EDGE>(nullptr, c, 1.0f, gate);
#pragma unroll
    for (int j = 0; j < 5; ++j)
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[j][i] = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t at = r * a.C + c.c, gi = r / a.per_gate;
        if (t.gate && (r == r0 || r % a.per_gate == 0)) weights<EDGE>(t.gate + gi * a.C, c, 1.0f, gate);
        float st[4] = {0.0f, 1.0f, 0.0f, 1.0f}, x[kV] = {}, s[kV], dy[kV], ds[kV] = {};
        if (t.stats)
#pragma unroll
            for (int i = 0; i < 4; ++i) st[i] = t.stats[r * 4 + i];
        if (use_x) load<EDGE, T>(t.x, at, c.lo).get(x);
        if (t.dsum) load<EDGE, S>(t.dsum, at, c.lo).get(ds);
        if (pre) {
            load<EDGE, S>(t.sum, at, c.lo).get(s);
            load<EDGE, T>(t.dy, at, c.lo).get(dy);
            const float a1 = a.averages[r * 2], a2 = a.averages[r * 2 + 1];
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float xh = (s[i] - st[2]) * st[3];
                acc[kPreW][i] = fmaf(dy[i], xh, acc[kPreW][i]);
                acc[kPreB][i] += dy[i];
                ds[i] = fmaf(st[3], dy[i] * w2[i] - a1 - xh * a2, ds[i]);
            }
        }
        if (t.dres) {
            float o[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) o[i] = a.res_scale * ds[i];
            store<EDGE, S>(t.dres, at, c.lo, o);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const float du = a.scale * ds[i], xh = post ? (x[i] - st[0]) * st[1] : x[i];
            acc[4][i] = fmaf(du, fmaf(xh, w1[i], b1[i]), acc[4][i]);
            acc[kPostW][i] = fmaf(du * gate[i], xh, acc[kPostW][i]);
            acc[kPostB][i] = fmaf(du, gate[i], acc[kPostB][i]);
        }
        if (t.dgate && (r + 1 == r1 || (r + 1) % a.per_gate == 0)) {
            store<EDGE, float>(a.gate_part + (a.runs ? blk : gi) * a.C, c.c, c.lo, acc[4]);
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[4][i] = 0.0f;
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float* want = j == kPreW ? t.dpre_w : j == kPostW ? t.dpost_w : j == kPreB ? t.dpre_b : t.dpost_b;
        if (want) store<EDGE, float>(a.part + (blk * NS + j) * a.C, c.c, c.lo, acc[j]);
    }
}

// Sums of columns over parts that lie `pitch` apart: 64 columns a workgroup, 16 interleaved runs of parts joined in
// order. Grid y: which sum (its first part, `apart` behind the one before), z: which stretch of `count` parts.
struct JoinArgs {
    const float* part;
    int64_t pitch, apart, C;
    int32_t count, total;  // parts of a stretch, and of all
    float* out[4];         // of each sum, null: not wanted; stretch z at out + z * step
    int64_t step;
};
__global__ __launch_bounds__(1024) void join_kernel(JoinArgs a) {
    __shared__ float red[16][64];
    const int col = threadIdx.x % 64, r = threadIdx.x / 64;
    const int64_t c = int64_t(blockIdx.x) * 64 + col, z = blockIdx.z;
    float* out = a.out[blockIdx.y];
    if (!out) return;
    const int64_t p0 = z * a.count, p1 = p0 + a.count < a.total ? p0 + a.count : a.total;
    float s = 0.0f;
    if (c < a.C)
#pragma unroll 4
        for (int64_t p = p0 + r; p < p1; p += 16) s += a.part[p * a.pitch + blockIdx.y * a.apart + c];
    red[r][col] = s;
    __syncthreads();
    if (r == 0 && c < a.C) {
#pragma unroll
        for (int k = 1; k < 16; ++k) s += red[k][col];
        out[z * a.step + c] = s;
    }
}

// ---- the split of a call -----------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Threads of a row: a power of two up to a wave, then whole waves; a vector each in rows of up to kOne values, else two
// (8192 x 5120 bf16 136 us in two, 61 in one).
constexpr int64_t kOne = 1024 * kV;
int lanes_of(int64_t C) {
    const int64_t v = ceil_div(C, C <= kOne ? kV : 2 * kV);
    if (v > 64) return int(ceil_div(v, 64) * 64);
    int n = 1;
    while (n < v) n *= 2;
    return n;
}

AnArgs args_of(const AddnormTensors& t, const AddnormShape& s) {
    AnArgs a{};
    a.t = t;
    a.R = s.R; a.C = s.C; a.per_gate = s.G ? s.R / s.G : s.R > 0 ? s.R : 1;
    a.post = s.post; a.pre = s.pre; a.eps = s.eps; a.scale = s.scale; a.res_scale = s.res_scale;
    return a;
}

// f(type, residual's type, how rows end)
template <typename F> void dispatch(const AddnormShape& s, F f) {
    auto types = [&](auto edge) {
        if (s.dtype == DType::F32) f(float{}, float{}, edge);
        else if (s.res_dtype == DType::F32) f(bf16_bits{}, float{}, edge);
        else f(bf16_bits{}, bf16_bits{}, edge);
    };
    if (s.C % kV == 0 && s.C > 0) types(std::integral_constant<int, kWhole>{});
    else if (s.C > kV) types(std::integral_constant<int, kPart>{});
    else types(std::integral_constant<int, kFew>{});
}

// The backward's workgroups: their rows, and where their sums go.
struct BwdPlan {
    int rows, lanes, sums;  // rows: kLanes, ...
    bool apart;             // the sums in a launch of their own
    int64_t runs, per, blocks;
    size_t part, part2, gate, averages, bytes;  // places in the workspace
};
constexpr int kJoin = 512;
bool row_sums(const AddnormTensors& w) { return w.dpre_w || w.dpost_w || w.dpre_b || w.dpost_b; }

BwdPlan bwd_plan(const AddnormShape& s, const AddnormTensors& w) {
    BwdPlan p{};
    p.lanes = lanes_of(s.C);
    const bool wide = p.lanes > 64;
    p.sums = w.dpre_b || w.dpost_b ? 4 : 2;
    p.rows = !wide ? kLanes : p.lanes <= 512 ? k512 : s.C > kOne ? kApart2 : p.lanes <= 768 ? k768
             : !s.G && p.sums == 2 ? k1024 : kApart;
    p.apart = p.rows >= kApart;
    const int64_t step = wide ? 1 : 256 / p.lanes, groups = s.G ? s.G : 1, rows = s.R / groups;
    // workgroups for 512 threads a CU
    const int64_t want = 256 * (wide ? ceil_div(512, p.lanes) : 4);
    // A thread's sums of 256 rows at most (more where that would take more than 2^20 workgroups), so that long sums
    // lose no more than short ones.
    int64_t most = ceil_div(s.R, int64_t(1) << 20);
    most = most < 256 * step ? 256 * step : most;
    if (w.dgate && groups >= want && rows <= most) {  // whole gate rows, whose sums are then done
        const int64_t share = ceil_div(groups, want), fit = rows > 0 ? most / rows : 1;
        p.per = (share < fit ? share : fit) * rows;
        p.blocks = ceil_div(s.R, p.per);
    } else {  // runs of a gate row's rows; of all rows where the gate's gradient is not wanted
        const int64_t of = w.dgate ? rows : s.R, g = w.dgate ? groups : 1;
        const int64_t per = ceil_div(of, ceil_div(want, g));
        p.per = ceil_div(per < most ? per : most, step) * step;
        p.blocks = ceil_div(of, p.per) * g;
        p.runs = w.dgate ? ceil_div(of, p.per) : 0;
    }
    size_t at = 0;
    if (row_sums(w)) {
        at += up256(size_t(p.blocks) * p.sums * s.C * sizeof(float));
        p.part2 = at;
        if (p.blocks > kJoin) at += up256(size_t(ceil_div(p.blocks, kJoin)) * p.sums * s.C * sizeof(float));
    }
    p.gate = at;
    if (w.dgate && p.runs) at += up256(size_t(p.blocks) * s.C * sizeof(float));
    p.averages = at;
    if (p.apart && (row_sums(w) || w.dgate)) at += up256(size_t(s.R) * 2 * sizeof(float));
    p.bytes = at;
    return p;
}

}  // namespace

size_t addnorm_bwd_workspace_bytes(const AddnormShape& s, const AddnormTensors& wanted) {
    return bwd_plan(s, wanted).bytes;
}

hipError_t launch_addnorm(const AddnormTensors& t, const AddnormShape& s, hipStream_t stream) {
    AnArgs a = args_of(t, s);
    a.lanes = lanes_of(s.C);
    const bool wide = a.lanes > 64;
    const int threads = wide ? a.lanes : 256, step = wide ? 1 : 256 / a.lanes;
    // what a CU holds at once, 1280 threads or a row, so that all workgroups have the same rows to do (us, bf16, 2048 threads
    // and 1280: 8192 x 5120 80 and 62, 16384 x 4096 107 and 93)
    const int64_t blocks = ceil_div(s.R, step), most = int64_t(256) * (threads < 1280 ? 1280 / threads : 1);
    const dim3 grid(unsigned(blocks < most ? blocks : most)), block{unsigned(threads)};
    dispatch(s, [&](auto T, auto S, auto edge) {
        using X = decltype(T);
        using Y = decltype(S);
        constexpr int E = decltype(edge)::value;
        if (!wide) hipLaunchKernelGGL((fwd_kernel<X, Y, 1, false, E>), grid, block, 0, stream, a);
        if constexpr (E != kFew) {
            if (wide && s.C <= kOne) hipLaunchKernelGGL((fwd_kernel<X, Y, 1, true, E>), grid, block, 0, stream, a);
            else if (wide) hipLaunchKernelGGL((fwd_kernel<X, Y, 2, true, E>), grid, block, 0, stream, a);
        }
    });
    return hipGetLastError();
}

hipError_t launch_addnorm_bwd(const AddnormTensors& t, const AddnormShape& s, void* workspace, hipStream_t stream) {
    AnArgs a = args_of(t, s);
    const BwdPlan p = bwd_plan(s, t);
    char* ws = static_cast<char*>(workspace);
    const bool sums = row_sums(t);
    a.lanes = p.lanes; a.runs = p.runs; a.per = p.per;
    a.part = sums ? reinterpret_cast<float*>(ws) : nullptr;
    a.gate_part = p.runs ? reinterpret_cast<float*>(ws + p.gate) : t.dgate;
    a.averages = p.apart && (sums || t.dgate) ? reinterpret_cast<float*>(ws + p.averages) : nullptr;
    const dim3 grid(unsigned(p.blocks)), block(unsigned(p.rows == kLanes ? 256 : p.lanes));
    dispatch(s, [&](auto T, auto S, auto edge) {
        constexpr int E = decltype(edge)::value;
        auto with = [&](auto bias, auto gate) {
            using X = decltype(T);
            using Y = decltype(S);
            constexpr bool B = decltype(bias)::value, G = decltype(gate)::value;
            if (p.rows == kLanes) hipLaunchKernelGGL((bwd_kernel<X, Y, kLanes, B, G, E>), grid, block, 0, stream, a);
            if constexpr (E != kFew) {
                if (p.rows == k512) hipLaunchKernelGGL((bwd_kernel<X, Y, k512, B, G, E>), grid, block, 0, stream, a);
                else if (p.rows == k768) hipLaunchKernelGGL((bwd_kernel<X, Y, k768, B, G, E>), grid, block, 0, stream, a);
                else if (p.rows == k1024) hipLaunchKernelGGL((bwd_kernel<X, Y, k1024, false, false, E>), grid, block, 0, stream, a);
                else if (p.rows == kApart) hipLaunchKernelGGL((bwd_kernel<X, Y, kApart, false, G, E>), grid, block, 0, stream, a);
                else if (p.rows == kApart2) hipLaunchKernelGGL((bwd_kernel<X, Y, kApart2, false, G, E>), grid, block, 0, stream, a);
            }
        };
        const std::true_type yes;
        const std::false_type no;
        if (p.sums == 4) {
            if (t.gate) with(yes, yes);
            else with(yes, no);
        } else {
            if (t.gate) with(no, yes);
            else with(no, no);
        }
        if constexpr (E != kFew)
            if (a.averages)
                hipLaunchKernelGGL((cols_kernel<decltype(T), decltype(S), E>),
                                   dim3(unsigned(p.blocks), unsigned(ceil_div(s.C, 64 * kV))), dim3(64), 0, stream, a, p.sums);
    });
    const unsigned cols = unsigned(ceil_div(s.C, 64));
    if (sums) {
        float* const outs[4] = {t.dpre_w, t.dpost_w, t.dpre_b, t.dpost_b};
        JoinArgs j{};
        j.part = a.part;
        j.pitch = int64_t(p.sums) * s.C; j.apart = s.C; j.C = s.C;
        j.count = j.total = int32_t(p.blocks);
        if (p.blocks > kJoin) {  // in two stages
            float* mid = reinterpret_cast<float*>(ws + p.part2);
            const int64_t stretches = ceil_div(p.blocks, kJoin);
            j.count = kJoin;
            j.step = j.pitch;
            for (int i = 0; i < p.sums; ++i) j.out[i] = outs[i] ? mid + i * s.C : nullptr;
            hipLaunchKernelGGL(join_kernel, dim3(cols, unsigned(p.sums), unsigned(stretches)), dim3(1024), 0, stream, j);
            j.part = mid;
            j.count = j.total = int32_t(stretches);
        }
        for (int i = 0; i < p.sums; ++i) j.out[i] = outs[i];
        hipLaunchKernelGGL(join_kernel, dim3(cols, unsigned(p.sums)), dim3(1024), 0, stream, j);
    }
    if (t.dgate && p.runs) {
        JoinArgs j{};
        j.part = a.gate_part;
        j.pitch = s.C; j.C = s.C;
        j.count = int32_t(p.runs); j.total = int32_t(p.blocks);
        j.step = s.C;
        const int64_t most = 65535;  // workgroups along z
        for (int64_t g = 0; g < s.G; g += most) {
            const int64_t n = s.G - g < most ? s.G - g : most;
            j.part = a.gate_part + g * p.runs * s.C;
            j.total = int32_t(n * p.runs);
            j.out[0] = t.dgate + g * s.C;
            hipLaunchKernelGGL(join_kernel, dim3(cols, 1, unsigned(n)), dim3(1024), 0, stream, j);
        }
    }
    return hipGetLastError();
}

}  // namespace selscan
