// Rotary positions: pairs of a head's values turned by position * inv_freq.
//
// Bound by memory: every value is read once and written once, in vectors of 16
// bytes where the widths allow it. A workgroup takes a few tokens: it forms their
// cosines and sines once, in LDS, for all heads of queries and keys. 8 x 2048 tokens of
// 32 + 8 heads of 128 bf16: 64 us (5.2 TB/s).
#include "../../include/selscan.h"
#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

struct RoArgs {
    const void* q;
    const void* k;
    const float* inv_freq;
    const int32_t* positions;
    void* q_out;
    void* k_out;
    int64_t tokens, L, offset;
    int32_t H, Hk, W, rot, per;  // per: tokens of a workgroup
    float scale, sign;
};

// cos and sin of 2 pi f, f in turns. Whole quarters are taken off in 64 bits, which
// leaves |x| <= pi / 4 with full relative accuracy; there the Taylor sums up to
// x^10 / 10! and x^9 / 9! are off by less than 2^-26.
__device__ __forceinline__ float2 turn_of(double f) {
    const double quarters = rint(4.0 * f);
    const float x = float((f - 0.25 * quarters) * 6.283185307179586477);
    const float z = x * x;
    float s = 1.0f / 362880, c = -1.0f / 3628800;
    s = fmaf(s, z, -1.0f / 5040);
    s = fmaf(s, z, 1.0f / 120);
    s = fmaf(s, z, -1.0f / 6);
    s = fmaf(s * z, x, x);
    c = fmaf(c, z, 1.0f / 40320);
    c = fmaf(c, z, -1.0f / 720);
    c = fmaf(c, z, 1.0f / 24);
    c = fmaf(c, z, -0.5f);
    c = fmaf(c, z, 1.0f);
    const int n = int(quarters - 4.0 * floor(0.25 * quarters));
    const float a = n & 1 ? s : c, b = n & 1 ? c : s;
    return {n == 1 || n == 2 ? -a : a, n >= 2 ? -b : b};
}

template <int B> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
template <typename T, int V> struct Pack {
    using raw = typename RawOf<int(sizeof(T)) * V>::type;
    struct Values { T t[V]; };
    static __device__ __forceinline__ void get(const raw& r, float (&f)[V]) {
        const Values v = __builtin_bit_cast(Values, r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f32(v.t[i]);
    }
    static __device__ __forceinline__ raw put(const float (&f)[V]) {
        Values v;
#pragma unroll
        for (int i = 0; i < V; ++i) v.t[i] = from_f32<T>(f[i]);
        return __builtin_bit_cast(raw, v);
    }
};

constexpr int kCs = 2048;  // cosines and sines that a workgroup holds

// V values at once: of halves, V of either half (V divides rot / 2); of neighbours, V / 2 pairs (V divides rot). V
// divides the head's width too. (V 1: one pair either way.)
template <typename T, int V, bool PAIRS>
__global__ __launch_bounds__(256) void rotary_kernel(RoArgs a) {
    using P = Pack<T, V>;
    using R = typename P::raw;
    __shared__ float2 cs[kCs];
    const int half = a.rot / 2, turned = PAIRS && V > 1 ? a.rot / V : half / V, units = turned + (a.W - a.rot) / V;
    const int heads = a.H + a.Hk, row = heads * units;
    for (int64_t first = int64_t(blockIdx.x) * a.per; first < a.tokens; first += int64_t(gridDim.x) * a.per) {
        const int here = int(a.tokens - first < a.per ? a.tokens - first : a.per);
        __syncthreads();
        for (int i = threadIdx.x; i < here * half; i += 256) {
            const int64_t token = first + i / half;
            const int64_t p = a.offset + (a.positions ? int64_t(a.positions[token]) : token % a.L);
            float2 t = turn_of(double(p) * (double(a.inv_freq[i % half]) * 0.15915494309189533577));
            t.x *= a.scale;
            t.y *= a.scale * a.sign;
            cs[i] = t;
        }
        __syncthreads();
        for (int j = threadIdx.x; j < here * row; j += 256) {
            const int tt = j / row, head = j % row / units, u = j % units;
            const bool isq = head < a.H;
            const int64_t token = first + tt, base = (isq ? token * a.H + head : token * a.Hk + head - a.H) * a.W;
            const T* src = static_cast<const T*>(isq ? a.q : a.k) + base;
            T* dst = static_cast<T*>(isq ? a.q_out : a.k_out) + base;
            if (u >= turned) {  // passed on
                const int at = a.rot + (u - turned) * V;
                *reinterpret_cast<R*>(dst + at) = *reinterpret_cast<const R*>(src + at);
            } else if constexpr (PAIRS && V > 1) {
                const float2* t = cs + tt * half + u * (V / 2);
                float x[V], y[V];
                P::get(*reinterpret_cast<const R*>(src + u * V), x);
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 c = t[i / 2];
                    y[i] = fmaf(x[i], c.x, -x[i + 1] * c.y);
                    y[i + 1] = fmaf(x[i], c.y, x[i + 1] * c.x);
                }
                *reinterpret_cast<R*>(dst + u * V) = P::put(y);
            } else {
                const float2* t = cs + tt * half + u * V;
                const int at = PAIRS ? 2 * u : u * V, to = PAIRS ? 1 : half;
                float x[V], z[V], lo[V], hi[V];
                P::get(*reinterpret_cast<const R*>(src + at), x);
                P::get(*reinterpret_cast<const R*>(src + at + to), z);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 c = t[i];
                    lo[i] = fmaf(x[i], c.x, -z[i] * c.y);
                    hi[i] = fmaf(x[i], c.y, z[i] * c.x);
                }
                *reinterpret_cast<R*>(dst + at) = P::put(lo);
                *reinterpret_cast<R*>(dst + at + to) = P::put(hi);
            }
        }
    }
}

template <typename T, int V> void launch(const RoArgs& a, bool pairs, unsigned grid, hipStream_t st) {
    if (pairs) hipLaunchKernelGGL((rotary_kernel<T, V, true>), dim3(grid), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((rotary_kernel<T, V, false>), dim3(grid), dim3(256), 0, st, a);
}

}  // namespace

hipError_t launch_rotary(const void* q, const void* k, const float* inv_freq, const int32_t* positions, void* q_out,
                         void* k_out, const RotaryShape& s, hipStream_t stream) {
    RoArgs a{};
    a.q = q; a.k = k; a.inv_freq = inv_freq; a.positions = positions; a.q_out = q_out; a.k_out = k_out;
    a.tokens = s.batch * s.L; a.L = s.L; a.H = int32_t(s.heads); a.Hk = int32_t(s.kv_heads); a.offset = s.offset;
    a.W = int32_t(s.W); a.rot = int32_t(s.rot);
    a.scale = s.scale; a.sign = s.inverse ? -1.0f : 1.0f;
    const bool pairs = s.layout == SELSCAN_ROTARY_INTERLEAVED;
    // the widest vector that divides a head, and what is turned of it
    int V = s.dtype == DType::BF16 ? 8 : 4;
    while (s.W % V || (pairs ? s.rot : s.rot / 2) % V) V /= 2;
    // tokens for an angle a thread, and some 2048 workgroups
    const int64_t half = s.rot / 2, fill = (s.batch * s.L + 2047) / 2048;
    int64_t per = half < 256 ? 256 / half : 1;
    per = per < fill ? per : fill;
    a.per = int32_t(per < 1 ? 1 : per);
    const int64_t groups = (a.tokens + a.per - 1) / a.per;
    const unsigned grid = unsigned(groups < 1 << 20 ? groups : 1 << 20);
    if (s.dtype == DType::BF16) {
        if (V == 8) launch<bf16_bits, 8>(a, pairs, grid, stream);
        else if (V == 4) launch<bf16_bits, 4>(a, pairs, grid, stream);
        else if (V == 2) launch<bf16_bits, 2>(a, pairs, grid, stream);
        else launch<bf16_bits, 1>(a, pairs, grid, stream);
    } else {
        if (V == 4) launch<float, 4>(a, pairs, grid, stream);
        else if (V == 2) launch<float, 2>(a, pairs, grid, stream);
        else launch<float, 1>(a, pairs, grid, stream);
    }
    return hipGetLastError();
}

}  // namespace selscan
