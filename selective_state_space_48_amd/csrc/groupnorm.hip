// Group norm with an activation, channels last, and its gradients. Bound by
// memory: x (and z) is read once and y written once where an instance (the
// S x D values of one n and group, D = C / G) fits the registers of a
// workgroup; else statistics are formed by slabs of rows first and the slabs
// read again. Three kernels, by the shape of an instance:
//   rows  (S = 1, D up to 64 or 256 vectors): a power of two of lanes per
//         instance, sums by shuffles, weights kept in registers over many rows;
//   block (a row of the group fits a workgroup's threads): one workgroup per
//         instance or slab, its values in registers;
//   plain (groups of more than 1024 vectors): one workgroup per instance, three
//         passes, scalar accesses.
// Measured (MI355X; bytes moved once over the time; a large copy 4.75 TB/s):
// 16384 rows of 4096 in 32 groups, bf16, gated: 88-97 us (4.2-4.6 TB/s),
// gradients 152 us (4.4 TB/s); 8 x 2048 x 512 fp32 in 32 groups (64-byte rows),
// SiLU: 17 us (4.0 TB/s), gradients 30 us (3.4 TB/s). Far from the copy rate:
// slabs (8 x 16384 x 512 bf16 in 32 groups: 97 us, 2.8 TB/s, gradients 266 us, 1.5
// TB/s), plain (4096 x 16384 fp32: 450 us, 1.2 TB/s, gradients 542 us, 1.5 TB/s),
// and maps of few positions, whose workgroups hold one instance however small
// (131072 x 2 x 512 bf16 in 64 groups: 2.8 ms, 0.2 TB/s, gradients 5.2 ms).
// Statistics in fp32: the mean, a sum of the values (off by its roundings: some
// 2^-24 of the average magnitude), then the squares about it (slabs: their own
// means, joined by n_i (mean_i - mean)^2).
#include "../../include/selscan.h"
#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

struct GnArgs {
    const void* x;
    const float* weight;
    const float* bias;
    const void* z;
    void* y;
    float* mean;
    float* rstd;
    const void* dy;
    void* dx;
    void* dz;
    int64_t N, S, C, G;
    int32_t act;
    float eps;
    // work split
    int32_t D, lanes;   // channels of a group; vectors of a row of it
    int32_t sub, gb;    // rows kernel: lanes of an instance, groups of a workgroup
    int64_t per;        // rows kernel: rows of a workgroup; block kernel: entries of a run, or rows of a slab
    int32_t slabs;
    float* stats;       // per instance and slab: (mean, M2), backward (sum e, sum e xh)
    float* part;        // partial column sums: [part][2][C] of du xh and du; null: not wanted
};

// ---- vectors of V values -----------------------------------------------------

template <int B> struct Raw;
template <> struct Raw<2> { using type = uint16_t; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };

template <typename T, int V> using raw_t = typename Raw<int(sizeof(T)) * V>::type;
template <typename T, int V>
__device__ __forceinline__ raw_t<T, V> load_raw(const void* p, int64_t i) {
    return *reinterpret_cast<const raw_t<T, V>*>(static_cast<const T*>(p) + i);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const raw_t<T, V>& r, float (&f)[V]) {
    struct A { T t[V]; };
    const A a = __builtin_bit_cast(A, r);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(a.t[i]);
}
// STREAM: 16-byte vectors past the caches
template <typename T, int V, bool STREAM = false>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&f)[V]) {
    struct A { T t[V]; } a;
#pragma unroll
    for (int j = 0; j < V; ++j) a.t[j] = from_f32<T>(f[j]);
    if constexpr (STREAM && V * sizeof(T) == 16) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, a), reinterpret_cast<u32x4*>(static_cast<T*>(p) + i));
    } else {
        *reinterpret_cast<raw_t<T, V>*>(static_cast<T*>(p) + i) = __builtin_bit_cast(raw_t<T, V>, a);
    }
}
template <int V>
__device__ __forceinline__ void load_affine(const float* p, int64_t c, float dflt, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = p ? p[c + i] : dflt;
}

// ---- the functions -------------------------------------------------------------

__device__ __forceinline__ float activate(float u, int act, float z) {
    return act == SELSCAN_ACT_SILU ? silu(u) : act == SELSCAN_ACT_GATE ? u * silu(z) : u;
}
// du and (gate) dz of one value.
__device__ __forceinline__ float grad_u(int act, float u, float dy, float z, float* dz) {
    if (act == SELSCAN_ACT_SILU) return dy * silu_grad(u);
    if (act == SELSCAN_ACT_GATE) {
        *dz = dy * u * silu_grad(z);
        return dy * silu(z);
    }
    return dy;
}

// Sum over the workgroup's threads, in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* red) {
    const int tid = threadIdx.x, waves = (blockDim.x + 63) / 64;
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if (tid % 64 == 0) red[tid / 64] = v;
    __syncthreads();
    float s = red[0];
    for (int i = 1; i < waves; ++i) s += red[i];
    return s;
}

// cols[0][i] = the sum over r < n of cols[r][i], i < width: halves folded onto
// each other, a fixed order. Called by all threads.
__device__ __forceinline__ void fold_rows(float* cols, int n, int width) {
    while (n > 1) {
        const int half = (n + 1) / 2;
        __syncthreads();
        for (int i = threadIdx.x; i < (n - half) * width; i += blockDim.x) cols[i] += cols[half * width + i];
        n = half;
    }
    __syncthreads();
}

// ---- rows: S = 1 ----------------------------------------------------------------
//
// `sub` lanes (a power of two) hold an instance, KV vectors each; a workgroup
// covers gb groups and 256 / sub / gb rows at once, and goes down `per` rows
// with its columns fixed, the next row's loads in flight.
template <typename T, int V, int KV, bool BWD, bool STREAM>
__global__ __launch_bounds__(256) void rows_kernel(GnArgs a) {
    __shared__ float cols[BWD ? 256 * KV * V : 1];
    const int tid = threadIdx.x, j = tid / a.sub, l = tid % a.sub, step = 256 / a.sub / a.gb;
    const int gi = j % a.gb, ri = j / a.gb;
    const int64_t g = int64_t(blockIdx.x) * a.gb + gi;
    const bool live = g < a.G && ri < step;
    const int64_t r0 = int64_t(blockIdx.y) * a.per, r1 = r0 + a.per < a.N ? r0 + a.per : a.N;
    const bool gate = a.act == SELSCAN_ACT_GATE;
    float w[KV][V], b[KV][V], sw[KV][V], sb[KV][V];
    bool in[KV];
#pragma unroll
    for (int k = 0; k < KV; ++k) {
        in[k] = live && l + a.sub * k < a.lanes;
        const int64_t c = g * a.D + int64_t(l + a.sub * k) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[k][i] = in[k] && a.weight ? a.weight[c + i] : 1.0f;
            b[k][i] = in[k] && a.bias ? a.bias[c + i] : 0.0f;
            sw[k][i] = sb[k][i] = 0.0f;
        }
    }
    raw_t<T, V> nx[KV], nz[KV], ny[KV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            if (!in[k] || r >= r1) continue;
            const int64_t at = r * a.C + g * a.D + int64_t(l + a.sub * k) * V;
            nx[k] = load_raw<T, V>(a.x, at);
            if (gate) nz[k] = load_raw<T, V>(a.z, at);
            if (BWD) ny[k] = load_raw<T, V>(a.dy, at);
        }
    };
    auto sum = [&](float v) {
        for (int m = a.sub / 2; m; m >>= 1) v += __shfl_xor(v, m, 64);
        return v;
    };
    if (live) {
        const float inv = 1.0f / float(a.D);
        fetch(r0 + ri);
        for (int64_t r = r0 + ri; r < r1; r += step) {
            float x[KV][V], z[KV][V], dy[KV][V];
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                unpack<T, V>(nx[k], x[k]);
                if (gate) unpack<T, V>(nz[k], z[k]);
                if (BWD) unpack<T, V>(ny[k], dy[k]);
            }
            fetch(r + step);
            float mean, rstd;
            if (!BWD) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < KV; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) s += in[k] ? x[k][i] : 0.0f;
                mean = sum(s) * inv;
                s = 0.0f;
#pragma unroll
                for (int k = 0; k < KV; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float d = in[k] ? x[k][i] - mean : 0.0f;
                        s = fmaf(d, d, s);
                    }
                rstd = 1.0f / sqrtf(sum(s) * inv + a.eps);
                if (a.mean && l == 0) {
                    a.mean[r * a.G + g] = mean;
                    a.rstd[r * a.G + g] = rstd;
                }
            } else {
                mean = a.mean[r * a.G + g];
                rstd = a.rstd[r * a.G + g];
            }
            const int64_t at = r * a.C + g * a.D + int64_t(l) * V;
            if (!BWD) {
#pragma unroll
                for (int k = 0; k < KV; ++k) {
                    float y[V];
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        y[i] = activate(fmaf((x[k][i] - mean) * rstd, w[k][i], b[k][i]), a.act, gate ? z[k][i] : 0.0f);
                    if (in[k]) store_vec<T, V, STREAM>(a.y, at + int64_t(a.sub) * k * V, y);
                }
            } else {
                float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
                for (int k = 0; k < KV; ++k) {
                    float dz[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float xh = (x[k][i] - mean) * rstd;
                        const float du = grad_u(a.act, fmaf(xh, w[k][i], b[k][i]), dy[k][i], gate ? z[k][i] : 0.0f, &dz[i]);
                        const float e = in[k] ? du * w[k][i] : 0.0f;
                        sw[k][i] = fmaf(du, xh, sw[k][i]);
                        sb[k][i] += du;
                        s1 += e;
                        s2 = in[k] ? fmaf(e, xh, s2) : s2;
                        x[k][i] = xh;
                        dy[k][i] = e;
                    }
                    if (gate && in[k]) store_vec<T, V, STREAM>(a.dz, at + int64_t(a.sub) * k * V, dz);
                }
                const float m1 = sum(s1) * inv, m2 = sum(s2) * inv;
#pragma unroll
                for (int k = 0; k < KV; ++k) {
                    float dx[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) dx[i] = rstd * (dy[k][i] - m1 - x[k][i] * m2);
                    if (in[k]) store_vec<T, V, STREAM>(a.dx, at + int64_t(a.sub) * k * V, dx);
                }
            }
        }
    }
    if (BWD && a.part) {  // the workgroup's column sums: its `step` rows at a time joined in order
        const int width = a.gb * a.D;
        float* out = a.part + int64_t(blockIdx.y) * 2 * a.C + int64_t(blockIdx.x) * width;
        const int64_t have = a.C - int64_t(blockIdx.x) * width;
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < KV; ++k)
                if (in[k])
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        cols[ri * width + gi * a.D + (l + a.sub * k) * V + i] = which ? sb[k][i] : sw[k][i];
            fold_rows(cols, step, width);
            for (int c = tid; c < width && c < have; c += 256) out[which * a.C + c] = cols[c];
        }
    }
}

// ---- block: an instance or a slab of its rows per workgroup ----------------------
//
// Thread (r, v) takes vector v of rows r, r + rs, ... of the slab, K of them in
// registers; threads past the last whole row idle.
enum { kFused = 0, kStats = 1, kApply = 2 };
// Vectors of V values a thread holds of each tensor: 32 values (16 of the three
// tensors of a gated backward), which the registers of 16 waves a CU take; and
// two where that is enough, for more waves.
constexpr int held(bool bwd, bool gate, int V) {
    const int k = (bwd && gate ? 16 : 32) / V;
    return k < 16 ? k : 16;
}

// Where a whole instance fits (kFused), a workgroup takes `per` entries of its
// group one after the other, the weights kept and the column sums joined once.
template <typename T, int V, int K, bool BWD, bool GATE, int MODE>
__global__ __launch_bounds__(1024) void block_kernel(GnArgs a) {
    __shared__ float red[16];
    extern __shared__ float cols[];  // backward: V values a thread, sized by the launch
    const int tid = threadIdx.x, rs = int(blockDim.x) / a.lanes, r0 = tid / a.lanes, v = tid % a.lanes;
    // kFused: group g of entries n0 .. n1 - 1; else slab `slab` of instance (n0, g).
    // The groups of the same rows, which share cache lines where they are narrow,
    // are neighbours and run on one XCD.
    const int64_t idx = xcd_tile(blockIdx.x, gridDim.x), g = idx % a.G;
    const int64_t slab = MODE == kFused ? 0 : idx / a.G % a.slabs;
    const int64_t n0 = MODE == kFused ? idx / a.G * a.per : idx / a.G / a.slabs;
    const int64_t n1 = MODE != kFused ? n0 + 1 : n0 + a.per < a.N ? n0 + a.per : a.N;
    const int64_t s0 = MODE == kFused ? 0 : slab * a.per;
    const int64_t s1 = MODE == kFused || s0 + a.per > a.S ? a.S : s0 + a.per;
    const bool live = r0 < rs;
    const int64_t c = g * a.D + int64_t(v) * V;
    const float cnt = float(s1 - s0) * float(a.D), all = float(a.S) * float(a.D);
    float w[V], b[V], sw[BWD ? V : 1], sb[BWD ? V : 1];
    if (BWD || MODE != kStats) {
        load_affine<V>(live ? a.weight : nullptr, c, 1.0f, w);
        load_affine<V>(live ? a.bias : nullptr, c, 0.0f, b);
    }
    if (BWD)
#pragma unroll
        for (int i = 0; i < V; ++i) sw[i] = sb[i] = 0.0f;
    for (int64_t n = n0; n < n1; ++n) {
        const int64_t inst = n * a.G + g, base = n * a.S * a.C + c;
        raw_t<T, V> x[K], z[GATE ? K : 1], dy[BWD ? K : 1];
        bool in[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t s = s0 + r0 + int64_t(rs) * k;
            in[k] = live && s < s1;
            if (!in[k]) continue;
            x[k] = load_raw<T, V>(a.x, base + s * a.C);
            if ((BWD || MODE != kStats) && GATE) z[k] = load_raw<T, V>(a.z, base + s * a.C);
            if (BWD) dy[k] = load_raw<T, V>(a.dy, base + s * a.C);
        }
        if constexpr (!BWD) {
            float mean, var;
            if (MODE != kApply) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float f[V];
                    if (!in[k]) continue;
                    unpack<T, V>(x[k], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) s += f[i];
                }
                mean = block_sum(s, red) / cnt;
                s = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float f[V];
                    if (!in[k]) continue;
                    unpack<T, V>(x[k], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) s = fmaf(f[i] - mean, f[i] - mean, s);
                }
                var = block_sum(s, red);
                if (MODE == kStats) {
                    if (tid == 0) {
                        a.stats[2 * (inst * a.slabs + slab)] = mean;
                        a.stats[2 * (inst * a.slabs + slab) + 1] = var;
                    }
                    return;
                }
            } else {
                const float* st = a.stats + 2 * inst * a.slabs;
                auto rows = [&](int i) { return float(i + 1 < a.slabs ? a.per : a.S - int64_t(i) * a.per) * float(a.D); };
                float s = 0.0f;
                for (int i = tid; i < a.slabs; i += blockDim.x) s = fmaf(st[2 * i], rows(i), s);
                mean = block_sum(s, red) / all;
                s = 0.0f;
                for (int i = tid; i < a.slabs; i += blockDim.x) {
                    const float d = st[2 * i] - mean;
                    s += fmaf(d * d, rows(i), st[2 * i + 1]);
                }
                var = block_sum(s, red);
            }
            const float rstd = 1.0f / sqrtf(var / all + a.eps);
            if (a.mean && slab == 0 && tid == 0) {
                a.mean[inst] = mean;
                a.rstd[inst] = rstd;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k]) continue;
                float f[V], zz[V], y[V];
                unpack<T, V>(x[k], f);
                if constexpr (GATE) unpack<T, V>(z[k], zz);
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = activate(fmaf((f[i] - mean) * rstd, w[i], b[i]), a.act, GATE ? zz[i] : 0.0f);
                store_vec<T, V>(a.y, base + (s0 + r0 + int64_t(rs) * k) * a.C, y);
            }
        } else {
            const float mean = a.mean[inst], rstd = a.rstd[inst];
            // xh, du and dz of vector k
            auto grads = [&](int k, float (&xh)[V], float (&du)[V], float (&dz)[V]) {
                float f[V], zz[V], gy[V];
                unpack<T, V>(x[k], f);
                unpack<T, V>(dy[k], gy);
                if constexpr (GATE) unpack<T, V>(z[k], zz);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[i] = (f[i] - mean) * rstd;
                    du[i] = grad_u(a.act, fmaf(xh[i], w[i], b[i]), gy[i], GATE ? zz[i] : 0.0f, &dz[i]);
                }
            };
            float m1, m2;
            if (MODE != kApply) {
                float p1 = 0.0f, p2 = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!in[k]) continue;
                    float xh[V], du[V], dz[V];
                    grads(k, xh, du, dz);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        p1 = fmaf(du[i], w[i], p1);
                        p2 = fmaf(du[i] * w[i], xh[i], p2);
                        sw[i] = fmaf(du[i], xh[i], sw[i]);
                        sb[i] += du[i];
                    }
                }
                m1 = block_sum(p1, red);
                m2 = block_sum(p2, red);
                if (MODE == kStats && tid == 0) {
                    a.stats[2 * (inst * a.slabs + slab)] = m1;
                    a.stats[2 * (inst * a.slabs + slab) + 1] = m2;
                }
            } else {
                const float* st = a.stats + 2 * inst * a.slabs;
                float p1 = 0.0f, p2 = 0.0f;
                for (int i = tid; i < a.slabs; i += blockDim.x) {
                    p1 += st[2 * i];
                    p2 += st[2 * i + 1];
                }
                m1 = block_sum(p1, red);
                m2 = block_sum(p2, red);
            }
            m1 /= all;
            m2 /= all;
            if (MODE != kStats) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!in[k]) continue;
                    float xh[V], du[V], dz[V], dx[V];
                    grads(k, xh, du, dz);
#pragma unroll
                    for (int i = 0; i < V; ++i) dx[i] = rstd * (du[i] * w[i] - m1 - xh[i] * m2);
                    const int64_t at = base + (s0 + r0 + int64_t(rs) * k) * a.C;
                    store_vec<T, V>(a.dx, at, dx);
                    if (GATE) store_vec<T, V>(a.dz, at, dz);
                }
            }
        }
    }
    if constexpr (BWD && MODE != kApply) {
        if (a.part) {  // the column sums, the threads' rows joined in a fixed order
            const int64_t at = MODE == kFused ? idx / a.G : n0 * a.slabs + slab;
            float* out = a.part + at * 2 * a.C + g * a.D;
            for (int which = 0; which < 2; ++which) {
                __syncthreads();
                if (live)
#pragma unroll
                    for (int i = 0; i < V; ++i) cols[(r0 * a.lanes + v) * V + i] = which ? sb[i] : sw[i];
                fold_rows(cols, rs, a.D);
                for (int i = tid; i < a.D; i += blockDim.x) out[which * a.C + i] = cols[i];
            }
        }
    }
}

// ---- plain: groups wider than a workgroup's vectors -------------------------------
//
// A thread's own sums are as long as the instance is large, so they are kept in 64
// bits (in 32, what is small beside the sum is lost: 7e-6 of the variance of
// 65536 values a thread, always to the same side).

template <typename T, bool BWD>
__global__ __launch_bounds__(1024) void plain_kernel(GnArgs a) {
    __shared__ float red[16];
    for (int64_t inst = blockIdx.x; inst < a.N * a.G; inst += gridDim.x) {
        const int64_t n = inst / a.G, g = inst % a.G, cnt = a.S * a.D;
        const int64_t base = n * a.S * a.C + g * a.D;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* z = static_cast<const T*>(a.z) + base;
        const bool gate = a.act == SELSCAN_ACT_GATE;
        auto each = [&](auto f) {
            for (int64_t i = threadIdx.x; i < cnt; i += blockDim.x) f(i / a.D * a.C + i % a.D, g * a.D + i % a.D);
        };
        if (!BWD) {
            T* y = static_cast<T*>(a.y) + base;
            double s = 0.0;
            each([&](int64_t i, int64_t) { s += to_f32(x[i]); });
            const float mean = block_sum(float(s), red) / float(cnt);
            s = 0.0;
            each([&](int64_t i, int64_t) {
                const float d = to_f32(x[i]) - mean;
                s += d * d;
            });
            const float rstd = 1.0f / sqrtf(block_sum(float(s), red) / float(cnt) + a.eps);
            each([&](int64_t i, int64_t c) {
                const float u = fmaf((to_f32(x[i]) - mean) * rstd, a.weight ? a.weight[c] : 1.0f, a.bias ? a.bias[c] : 0.0f);
                y[i] = from_f32<T>(activate(u, a.act, gate ? to_f32(z[i]) : 0.0f));
            });
            if (a.mean && threadIdx.x == 0) {
                a.mean[inst] = mean;
                a.rstd[inst] = rstd;
            }
        } else {
            const T* dy = static_cast<const T*>(a.dy) + base;
            T* dx = static_cast<T*>(a.dx) + base;
            T* dz = static_cast<T*>(a.dz) + base;
            const float mean = a.mean[inst], rstd = a.rstd[inst];
            double s1 = 0.0, s2 = 0.0;
            auto grad = [&](int64_t i, int64_t c, float* xh, float* d) {
                const float w = a.weight ? a.weight[c] : 1.0f;
                *xh = (to_f32(x[i]) - mean) * rstd;
                return w * grad_u(a.act, fmaf(*xh, w, a.bias ? a.bias[c] : 0.0f), to_f32(dy[i]), gate ? to_f32(z[i]) : 0.0f, d);
            };
            each([&](int64_t i, int64_t c) {
                float xh, d;
                const float e = grad(i, c, &xh, &d);
                s1 += e;
                s2 += e * xh;
            });
            const float m1 = block_sum(float(s1), red) / float(cnt), m2 = block_sum(float(s2), red) / float(cnt);
            each([&](int64_t i, int64_t c) {
                float xh, d;
                const float e = grad(i, c, &xh, &d);
                dx[i] = from_f32<T>(rstd * (e - m1 - xh * m2));
                if (gate) dz[i] = from_f32<T>(d);
            });
        }
    }
}

// Its column sums: part[k][0..1][c] over run k's rows (n, s).
template <typename T>
__global__ __launch_bounds__(256) void plain_cols_kernel(GnArgs a) {
    const int64_t c = int64_t(blockIdx.y) * 256 + threadIdx.x, rows = a.N * a.S;
    if (c >= a.C) return;
    const int64_t g = c / a.D, r0 = int64_t(blockIdx.x) * a.per, r1 = r0 + a.per < rows ? r0 + a.per : rows;
    const float w = a.weight ? a.weight[c] : 1.0f, b = a.bias ? a.bias[c] : 0.0f;
    double sw = 0.0, sb = 0.0;
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t n = r / a.S, j = r * a.C + c;
        const float xh = (to_f32(static_cast<const T*>(a.x)[j]) - a.mean[n * a.G + g]) * a.rstd[n * a.G + g];
        float dz;
        const float du = grad_u(a.act, fmaf(xh, w, b), to_f32(static_cast<const T*>(a.dy)[j]),
                                a.act == SELSCAN_ACT_GATE ? to_f32(static_cast<const T*>(a.z)[j]) : 0.0f, &dz);
        sw += du * xh;
        sb += du;
    }
    a.part[(int64_t(blockIdx.x) * 2 + 0) * a.C + c] = float(sw);
    a.part[(int64_t(blockIdx.x) * 2 + 1) * a.C + c] = float(sb);
}

// Column sums over runs of kJoin parts (grid z), 16 interleaved rows of them
// joined in order; 64 columns per workgroup, du xh (y 0) and du (y 1). The
// last stage (one run) writes dweight and dbias, the others out[run][2][C].
constexpr int kJoin = 512;
__global__ __launch_bounds__(1024) void cols_sum_kernel(const float* __restrict__ part, int parts, int64_t C,
                                                        float* __restrict__ out, float* __restrict__ dweight,
                                                        float* __restrict__ dbias) {
    __shared__ float red[16][64];
    const int col = threadIdx.x % 64, r = threadIdx.x / 64, run = blockIdx.z;
    const int64_t c = int64_t(blockIdx.x) * 64 + col;
    float* to = out ? out + (int64_t(run) * 2 + blockIdx.y) * C : blockIdx.y ? dbias : dweight;
    if (!to) return;
    const int k1 = (run + 1) * kJoin < parts ? (run + 1) * kJoin : parts;
    float s = 0.0f;
    if (c < C) {
#pragma unroll 4
        for (int k = run * kJoin + r; k < k1; k += 16) s += part[(int64_t(k) * 2 + blockIdx.y) * C + c];
    }
    red[r][col] = s;
    __syncthreads();
    if (r == 0 && c < C) {
#pragma unroll
        for (int k = 1; k < 16; ++k) s += red[k][col];
        to[c] = s;
    }
}

// ---- the split of a call -----------------------------------------------------------

struct Plan {
    enum Kind { kRows, kBlock, kPlain } kind;
    int V, KV;  // values of a vector; vectors a thread holds
    int sub, gb;
    int64_t per;
    int slabs, threads;
    int64_t parts;  // backward: partial column sums
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

Plan plan_of(const GroupnormShape& s, bool bwd) {
    Plan p{};
    const int64_t D = s.C / s.G;
    // the widest vector (16 bytes at most) that divides a group: rows are then aligned to it too
    const int full = s.dtype == DType::BF16 ? 8 : 4;
    p.V = full;
    while (D % p.V) p.V /= 2;
    const int64_t lanes = D / p.V;
    p.KV = 1;
    if (s.S == 1 && (lanes <= 64 || (lanes <= 256 && p.V == full))) {
        p.kind = Plan::kRows;
        if (lanes > 64) p.KV = 4;
        p.sub = 1;
        while (p.sub * p.KV < lanes) p.sub *= 2;
        const int n = 256 / p.sub;
        p.gb = int(s.G < n ? s.G : n);
        const int step = n / p.gb;
        // about 8 workgroups a CU; the backward's partial sums are written per
        // workgroup, so it takes half as many
        const int64_t blocks = ceil_div(s.G, p.gb), want = ceil_div(bwd ? 1024 : 2048, blocks);
        p.per = ceil_div(ceil_div(s.N, want), step) * step;
        p.slabs = 1;
        p.parts = ceil_div(s.N, p.per);
    } else if (lanes <= 1024) {
        p.kind = Plan::kBlock;
        const int K = held(bwd, s.act == SELSCAN_ACT_GATE, p.V);
        // threads for two vectors each, whole waves, at least one row
        int64_t t = ceil_div(s.S * lanes, 2);
        t = t < lanes ? lanes : t;
        t = t > 1024 ? 1024 : t;
        p.threads = int(ceil_div(t, 64) * 64);
        const int64_t rs = p.threads / lanes;
        p.slabs = int(ceil_div(s.S, rs * K));
        p.KV = s.S <= 2 * rs ? 2 : K;
        if (p.slabs == 1) {
            // runs of entries: workgroups for the threads the chip holds, twice those in the forward
            const int64_t want = ceil_div(int64_t(256) * (bwd ? 2048 : 4096) / p.threads, s.G);
            p.per = ceil_div(s.N, want);
            p.parts = ceil_div(s.N, p.per);
        } else {
            p.per = rs * K;
            p.parts = s.N * p.slabs;
        }
    } else {
        p.kind = Plan::kPlain;
        p.threads = 1024;
        p.slabs = 1;
        p.per = ceil_div(s.N * s.S, 256);
        p.parts = ceil_div(s.N * s.S, p.per);
    }
    return p;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
size_t stats_bytes(const GroupnormShape& s, const Plan& p) {
    return p.slabs > 1 ? up256(size_t(s.N * s.G) * p.slabs * 2 * sizeof(float)) : 0;
}

GnArgs args_of(const GroupnormTensors& t, const GroupnormShape& s, const Plan& p) {
    GnArgs a{};
    a.x = t.x; a.weight = t.weight; a.bias = t.bias; a.z = t.z; a.y = t.y;
    a.mean = t.mean; a.rstd = t.rstd; a.dy = t.dy; a.dx = t.dx; a.dz = t.dz;
    a.N = s.N; a.S = s.S; a.C = s.C; a.G = s.G; a.act = s.act; a.eps = s.eps;
    a.D = int32_t(s.C / s.G);
    a.lanes = a.D / p.V;
    a.sub = p.sub; a.gb = p.gb; a.per = p.per; a.slabs = p.slabs;
    return a;
}

template <typename T, int V, bool BWD, bool GATE>
void launch_block(const GnArgs& a, const Plan& p, hipStream_t st) {
    constexpr int K = held(BWD, GATE, V);
    const dim3 block(unsigned(p.threads));
    const unsigned lds = BWD ? unsigned(p.threads) * V * 4 : 0;  // at most 32 KB
    if (a.slabs == 1) {
        const dim3 grid(unsigned(ceil_div(a.N, a.per) * a.G));
        if (p.KV == 2) hipLaunchKernelGGL((block_kernel<T, V, 2, BWD, GATE, kFused>), grid, block, lds, st, a);
        else hipLaunchKernelGGL((block_kernel<T, V, K, BWD, GATE, kFused>), grid, block, lds, st, a);
    } else {
        const dim3 grid(unsigned(a.N * a.G * a.slabs));
        hipLaunchKernelGGL((block_kernel<T, V, K, BWD, GATE, kStats>), grid, block, lds, st, a);
        hipLaunchKernelGGL((block_kernel<T, V, K, BWD, GATE, kApply>), grid, block, 0, st, a);
    }
}

template <typename T, int V, bool BWD>
void launch_v(const GnArgs& a, const Plan& p, hipStream_t st) {
    if (p.kind == Plan::kRows) {
        const dim3 grid(unsigned(ceil_div(a.G, a.gb)), unsigned(ceil_div(a.N, a.per)));
        // An output that no cache would keep whole goes past them (us with and
        // without, forward: 16384 x 4096 bf16 gate 88 and 99, SiLU 65 and 75; 2048
        // rows 22 and 23).
        if constexpr (V * sizeof(T) == 16) {
            const bool stream = a.N * a.C * int64_t(sizeof(T)) > (int64_t(64) << 20);
            if (p.KV == 4 && stream) hipLaunchKernelGGL((rows_kernel<T, V, 4, BWD, true>), grid, dim3(256), 0, st, a);
            else if (p.KV == 4) hipLaunchKernelGGL((rows_kernel<T, V, 4, BWD, false>), grid, dim3(256), 0, st, a);
            else if (stream) hipLaunchKernelGGL((rows_kernel<T, V, 1, BWD, true>), grid, dim3(256), 0, st, a);
            else hipLaunchKernelGGL((rows_kernel<T, V, 1, BWD, false>), grid, dim3(256), 0, st, a);
        } else {
            hipLaunchKernelGGL((rows_kernel<T, V, 1, BWD, false>), grid, dim3(256), 0, st, a);
        }
        return;
    }
    if (a.act == SELSCAN_ACT_GATE) launch_block<T, V, BWD, true>(a, p, st);
    else launch_block<T, V, BWD, false>(a, p, st);
}

template <typename T, bool BWD>
void launch(const GnArgs& a, const Plan& p, hipStream_t st) {
    if (p.kind == Plan::kPlain) {
        const int64_t inst = a.N * a.G, most = int64_t(1) << 21;
        hipLaunchKernelGGL((plain_kernel<T, BWD>), dim3(unsigned(inst < most ? inst : most)), dim3(unsigned(p.threads)),
                           0, st, a);
        if (BWD && a.part)
            hipLaunchKernelGGL((plain_cols_kernel<T>), dim3(unsigned(p.parts), unsigned(ceil_div(a.C, 256))), dim3(256),
                               0, st, a);
        return;
    }
    if (p.V == 1) launch_v<T, 1, BWD>(a, p, st);
    else if (p.V == 2) launch_v<T, 2, BWD>(a, p, st);
    else if (p.V == 4) launch_v<T, 4, BWD>(a, p, st);
    else if constexpr (sizeof(T) == 2) launch_v<T, 8, BWD>(a, p, st);
}

}  // namespace

// A grid has fewer than 2^32 threads, and fewer than 2^16 workgroups along z (runs of partial sums).
bool groupnorm_fits(const GroupnormShape& s, bool backward) {
    if (s.N * s.S * s.C == 0) return true;
    const Plan p = plan_of(s, backward);
    if (p.kind != Plan::kBlock) return true;
    const int64_t grid = p.slabs == 1 ? ceil_div(s.N, p.per) * s.G : s.N * s.G * p.slabs;
    return grid * p.threads < (int64_t(1) << 32) && (!backward || p.parts <= int64_t(65535) * kJoin);
}

size_t groupnorm_workspace_bytes(const GroupnormShape& s, bool backward) {
    const Plan p = plan_of(s, backward);
    // the partial column sums, and where they are joined in stages those of the first stage
    const size_t cols = size_t(2) * s.C * sizeof(float);
    return stats_bytes(s, p) +
           (backward ? (size_t(p.parts) + (p.parts > kJoin ? size_t(ceil_div(p.parts, kJoin)) : 0)) * cols : 0);
}

hipError_t launch_groupnorm(const GroupnormTensors& t, const GroupnormShape& s, void* workspace, hipStream_t stream) {
    const Plan p = plan_of(s, false);
    GnArgs a = args_of(t, s, p);
    a.stats = static_cast<float*>(workspace);
    if (s.dtype == DType::BF16) launch<bf16_bits, false>(a, p, stream);
    else launch<float, false>(a, p, stream);
    return hipGetLastError();
}

hipError_t launch_groupnorm_bwd(const GroupnormTensors& t, const GroupnormShape& s, void* workspace,
                                hipStream_t stream) {
    const Plan p = plan_of(s, true);
    GnArgs a = args_of(t, s, p);
    a.stats = static_cast<float*>(workspace);
    float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(s, p));
    a.part = t.dweight || t.dbias ? part : nullptr;
    if (s.dtype == DType::BF16) launch<bf16_bits, true>(a, p, stream);
    else launch<float, true>(a, p, stream);
    if (a.part) {
        // Joined in stages of kJoin. The parts of a stage lie where those of the
        // stage before last did: at most 1 / kJoin of them each time.
        const dim3 block(1024);
        float* from = part;
        float* to = part + p.parts * 2 * s.C;
        int64_t n = p.parts;
        while (n > kJoin) {
            const int64_t m = ceil_div(n, kJoin);
            hipLaunchKernelGGL(cols_sum_kernel, dim3(unsigned(ceil_div(s.C, 64)), 2, unsigned(m)), block, 0, stream,
                               from, int(n), s.C, to, nullptr, nullptr);
            float* t_ = from;
            from = to;
            to = t_;
            n = m;
        }
        hipLaunchKernelGGL(cols_sum_kernel, dim3(unsigned(ceil_div(s.C, 64)), 2), block, 0, stream, from, int(n), s.C,
                           nullptr, t.dweight, t.dbias);
    }
    return hipGetLastError();
}

}  // namespace selscan
