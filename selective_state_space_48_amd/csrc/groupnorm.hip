// Group norm with an activation, channels last, and its gradients.
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
};

// Sum over the 256 threads of a workgroup, in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* red) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if (tid % 64 == 0) red[tid / 64] = v;
    __syncthreads();
    return red[0] + red[1] + red[2] + red[3];
}

__device__ __forceinline__ float activate(float u, int act, float z) {
    return act == SELSCAN_ACT_SILU ? silu(u) : act == SELSCAN_ACT_GATE ? u * silu(z) : u;
}

// One workgroup per (n, group), over its S x D values three times.
template <typename T>
__global__ __launch_bounds__(256) void gn_kernel(GnArgs a) {
    __shared__ float red[4];
    for (int64_t i0 = blockIdx.x; i0 < a.N * a.G; i0 += gridDim.x) {
        const int64_t n = i0 / a.G, g = i0 % a.G, D = a.C / a.G, cnt = a.S * D;
        const T* x = static_cast<const T*>(a.x) + n * a.S * a.C + g * D;
        const T* z = static_cast<const T*>(a.z) + n * a.S * a.C + g * D;
        T* y = static_cast<T*>(a.y) + n * a.S * a.C + g * D;
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < cnt; i += 256) s += to_f32(x[i / D * a.C + i % D]);
        const float mean = block_sum(s, red) / float(cnt);
        s = 0.0f;
        for (int64_t i = threadIdx.x; i < cnt; i += 256) {
            const float d = to_f32(x[i / D * a.C + i % D]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, red) / float(cnt) + a.eps);
        for (int64_t i = threadIdx.x; i < cnt; i += 256) {
            const int64_t at = i / D * a.C + i % D, c = g * D + i % D;
            const float u = fmaf((to_f32(x[at]) - mean) * rstd, a.weight ? a.weight[c] : 1.0f, a.bias ? a.bias[c] : 0.0f);
            y[at] = from_f32<T>(activate(u, a.act, a.act == SELSCAN_ACT_GATE ? to_f32(z[at]) : 0.0f));
        }
        if (a.mean && threadIdx.x == 0) {
            a.mean[i0] = mean;
            a.rstd[i0] = rstd;
        }
    }
}

// du and (gate) dz of one value.
struct Grad {
    float xh, du, dz;
};
__device__ __forceinline__ Grad grad_of(const GnArgs& a, float x, float dy, float z, float mean, float rstd, float w,
                                        float b) {
    Grad r;
    r.xh = (x - mean) * rstd;
    r.dz = 0.0f;
    const float u = fmaf(r.xh, w, b);
    if (a.act == SELSCAN_ACT_SILU) {
        r.du = dy * silu_grad(u);
    } else if (a.act == SELSCAN_ACT_GATE) {
        r.du = dy * silu(z);
        r.dz = dy * u * silu_grad(z);
    } else {
        r.du = dy;
    }
    return r;
}

template <typename T>
__global__ __launch_bounds__(256) void gn_bwd_kernel(GnArgs a) {
    __shared__ float red[4];
    for (int64_t i0 = blockIdx.x; i0 < a.N * a.G; i0 += gridDim.x) {
        const int64_t n = i0 / a.G, g = i0 % a.G, D = a.C / a.G, cnt = a.S * D;
        const int64_t base = n * a.S * a.C + g * D;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* z = static_cast<const T*>(a.z) + base;
        const T* dy = static_cast<const T*>(a.dy) + base;
        T* dx = static_cast<T*>(a.dx) + base;
        T* dz = static_cast<T*>(a.dz) + base;
        const float mean = a.mean[i0], rstd = a.rstd[i0];
        const bool gate = a.act == SELSCAN_ACT_GATE;
        float s1 = 0.0f, s2 = 0.0f;
        auto at = [&](int64_t i) { return i / D * a.C + i % D; };
        auto get = [&](int64_t i, float* w) {
            const int64_t c = g * D + i % D, j = at(i);
            *w = a.weight ? a.weight[c] : 1.0f;
            return grad_of(a, to_f32(x[j]), to_f32(dy[j]), gate ? to_f32(z[j]) : 0.0f, mean, rstd, *w,
                           a.bias ? a.bias[c] : 0.0f);
        };
        for (int64_t i = threadIdx.x; i < cnt; i += 256) {
            float w;
            const Grad r = get(i, &w);
            s1 += r.du * w;
            s2 = fmaf(r.du * w, r.xh, s2);
        }
        const float m1 = block_sum(s1, red) / float(cnt), m2 = block_sum(s2, red) / float(cnt);
        for (int64_t i = threadIdx.x; i < cnt; i += 256) {
            float w;
            const Grad r = get(i, &w);
            if (gate) dz[at(i)] = from_f32<T>(r.dz);
            dx[at(i)] = from_f32<T>(rstd * (r.du * w - m1 - r.xh * m2));
        }
    }
}

constexpr int kParts = 256;  // runs of rows whose column sums are formed apart

// part[k][0..1][c]: the sums of du xh and du over run k's rows (n, s).
template <typename T>
__global__ __launch_bounds__(256) void gn_cols_kernel(GnArgs a, int64_t rows, int64_t per, float* part) {
    const int64_t c = int64_t(blockIdx.y) * 256 + threadIdx.x;
    if (c >= a.C) return;
    const int64_t g = c / (a.C / a.G), r0 = int64_t(blockIdx.x) * per, r1 = min(r0 + per, rows);
    const float w = a.weight ? a.weight[c] : 1.0f, b = a.bias ? a.bias[c] : 0.0f;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t n = r / a.S, j = r * a.C + c;
        const Grad v = grad_of(a, to_f32(static_cast<const T*>(a.x)[j]), to_f32(static_cast<const T*>(a.dy)[j]),
                               a.act == SELSCAN_ACT_GATE ? to_f32(static_cast<const T*>(a.z)[j]) : 0.0f,
                               a.mean[n * a.G + g], a.rstd[n * a.G + g], w, b);
        sw = fmaf(v.du, v.xh, sw);
        sb += v.du;
    }
    part[(int64_t(blockIdx.x) * 2 + 0) * a.C + c] = sw;
    part[(int64_t(blockIdx.x) * 2 + 1) * a.C + c] = sb;
}

__global__ __launch_bounds__(256) void gn_cols_sum_kernel(const float* part, int parts, int64_t C, float* dweight,
                                                          float* dbias) {
    const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (c >= C) return;
    float sw = 0.0f, sb = 0.0f;
    for (int k = 0; k < parts; ++k) {
        sw += part[(int64_t(k) * 2 + 0) * C + c];
        sb += part[(int64_t(k) * 2 + 1) * C + c];
    }
    if (dweight) dweight[c] = sw;
    if (dbias) dbias[c] = sb;
}

GnArgs args_of(const GroupnormTensors& t, const GroupnormShape& s) {
    return {t.x, t.weight, t.bias, t.z, t.y, t.mean, t.rstd, t.dy, t.dx, t.dz, s.N, s.S, s.C, s.G, s.act, s.eps};
}
int64_t rows_per_part(const GroupnormShape& s) { return (s.N * s.S + kParts - 1) / kParts; }
int parts_of(const GroupnormShape& s) {
    const int64_t per = rows_per_part(s);
    return int((s.N * s.S + per - 1) / per);
}

}  // namespace

size_t groupnorm_workspace_bytes(const GroupnormShape& s, bool backward) {
    return backward ? size_t(parts_of(s)) * 2 * s.C * sizeof(float) : 0;
}

hipError_t launch_groupnorm(const GroupnormTensors& t, const GroupnormShape& s, void*, hipStream_t stream) {
    // a grid has fewer than 2^32 threads
    const dim3 grid(unsigned(s.N * s.G < (1 << 20) ? s.N * s.G : (1 << 20))), block(256);
    const GnArgs a = args_of(t, s);
    if (s.dtype == DType::BF16) hipLaunchKernelGGL((gn_kernel<bf16_bits>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((gn_kernel<float>), grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_groupnorm_bwd(const GroupnormTensors& t, const GroupnormShape& s, void* workspace,
                                hipStream_t stream) {
    // a grid has fewer than 2^32 threads
    const dim3 grid(unsigned(s.N * s.G < (1 << 20) ? s.N * s.G : (1 << 20))), block(256);
    const GnArgs a = args_of(t, s);
    float* part = static_cast<float*>(workspace);
    const int parts = parts_of(s);
    const unsigned cb = unsigned((s.C + 255) / 256);
    if (s.dtype == DType::BF16) {
        hipLaunchKernelGGL((gn_bwd_kernel<bf16_bits>), grid, block, 0, stream, a);
        hipLaunchKernelGGL((gn_cols_kernel<bf16_bits>), dim3(unsigned(parts), cb), block, 0, stream, a, s.N * s.S,
                           rows_per_part(s), part);
    } else {
        hipLaunchKernelGGL((gn_bwd_kernel<float>), grid, block, 0, stream, a);
        hipLaunchKernelGGL((gn_cols_kernel<float>), dim3(unsigned(parts), cb), block, 0, stream, a, s.N * s.S,
                           rows_per_part(s), part);
    }
    if (t.dweight || t.dbias)
        hipLaunchKernelGGL(gn_cols_sum_kernel, dim3(cb), block, 0, stream, part, parts, s.C, t.dweight, t.dbias);
    return hipGetLastError();
}

}  // namespace selscan
