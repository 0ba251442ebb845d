// Rotary positions: pairs of a head's values turned by position * inv_freq.
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
    int64_t tokens, L, H, Hk, offset;
    int32_t W, rot, interleaved;
    float scale, sign;
};

// cos and sin of 2 pi f for |f| <= 1/2, f from 64 bits with whole turns taken off.
__device__ __forceinline__ void turn(const RoArgs& a, int64_t token, int i, float* c, float* s) {
    const int64_t p = a.offset + (a.positions ? int64_t(a.positions[token]) : token % a.L);
    const double f = double(p) * (double(a.inv_freq[i]) * 0.15915494309189533577);
    double sn, cs;
    sincospi(2.0 * (f - rint(f)), &sn, &cs);
    *c = float(cs) * a.scale;
    *s = float(sn) * a.scale * a.sign;
}

// A workgroup per token: its angles once, then all heads.
template <typename T>
__global__ __launch_bounds__(256) void rotary_kernel(RoArgs a) {
    __shared__ float2 cs[2048];
    const int half = a.rot / 2, rest = a.W - a.rot, per = half + rest;
    for (int64_t token = blockIdx.x; token < a.tokens; token += gridDim.x) {
        __syncthreads();
        for (int i = threadIdx.x; i < half; i += 256) turn(a, token, i, &cs[i].x, &cs[i].y);
        __syncthreads();
        for (int64_t j = threadIdx.x; j < (a.H + a.Hk) * per; j += 256) {
            const int64_t head = j / per;
            const int i = int(j % per);
            const bool isq = head < a.H;
            const int64_t base = (isq ? token * a.H + head : token * a.Hk + head - a.H) * a.W;
            const T* src = static_cast<const T*>(isq ? a.q : a.k) + base;
            T* dst = static_cast<T*>(isq ? a.q_out : a.k_out) + base;
            if (i >= half) {
                dst[a.rot + i - half] = src[a.rot + i - half];
                continue;
            }
            const int lo = a.interleaved ? 2 * i : i, hi = a.interleaved ? 2 * i + 1 : i + half;
            const float u = to_f32(src[lo]), v = to_f32(src[hi]);
            dst[lo] = from_f32<T>(fmaf(u, cs[i].x, -v * cs[i].y));
            dst[hi] = from_f32<T>(fmaf(u, cs[i].y, v * cs[i].x));
        }
    }
}

}  // namespace

hipError_t launch_rotary(const void* q, const void* k, const float* inv_freq, const int32_t* positions, void* q_out,
                         void* k_out, const RotaryShape& s, hipStream_t stream) {
    RoArgs a{};
    a.q = q; a.k = k; a.inv_freq = inv_freq; a.positions = positions; a.q_out = q_out; a.k_out = k_out;
    a.tokens = s.batch * s.L; a.L = s.L; a.H = s.heads; a.Hk = s.kv_heads; a.offset = s.offset;
    a.W = int32_t(s.W); a.rot = int32_t(s.rot); a.interleaved = s.layout == SELSCAN_ROTARY_INTERLEAVED;
    a.scale = s.scale; a.sign = s.inverse ? -1.0f : 1.0f;
    const dim3 grid(unsigned(a.tokens < 1 << 20 ? a.tokens : 1 << 20));
    if (s.dtype == DType::BF16) hipLaunchKernelGGL((rotary_kernel<bf16_bits>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((rotary_kernel<float>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace selscan
