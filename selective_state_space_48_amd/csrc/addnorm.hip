// Norms around a block with the residual sum between them, and the gradients.
#include "../../include/selscan.h"
#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

struct AnArgs {
    AddnormTensors t;
    int64_t R, C, per_gate;  // rows of a gate row
    int32_t post, pre;
    float eps, scale, res_scale;
};

template <typename T> __device__ __forceinline__ float at(const void* p, int64_t i) {
    return to_f32(static_cast<const T*>(p)[i]);
}
template <typename T> __device__ __forceinline__ void put(void* p, int64_t i, float v) {
    static_cast<T*>(p)[i] = from_f32<T>(v);
}

// Sum over the workgroup's 256 threads, in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename T, typename S>
__global__ __launch_bounds__(256) void fwd_kernel(AnArgs a) {
    __shared__ float red[4];
    extern __shared__ float row[];
    const AddnormTensors& t = a.t;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
        float st[4] = {0.0f, 1.0f, 0.0f, 1.0f};
        auto stats = [&](int kind, float* mean, float* rstd) {
            if (kind == SELSCAN_NORM_NONE) return;
            float s = 0.0f;
            if (kind == SELSCAN_NORM_LAYER) {
                for (int64_t c = threadIdx.x; c < a.C; c += 256) s += row[c];
                *mean = block_sum(s, red) / float(a.C > 0 ? a.C : 1);
                s = 0.0f;
            }
            for (int64_t c = threadIdx.x; c < a.C; c += 256) s += (row[c] - *mean) * (row[c] - *mean);
            *rstd = 1.0f / sqrtf(block_sum(s, red) / float(a.C > 0 ? a.C : 1) + a.eps);
        };
        for (int64_t c = threadIdx.x; c < a.C; c += 256) row[c] = at<T>(t.x, r * a.C + c);
        stats(a.post, &st[0], &st[1]);
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            float u = (row[c] - st[0]) * st[1];
            if (t.post_w) u *= t.post_w[c];
            if (t.post_b) u += t.post_b[c];
            u *= a.scale;
            if (t.gate) u *= t.gate[r / a.per_gate * a.C + c];
            if (t.res) u = fmaf(a.res_scale, at<S>(t.res, r * a.C + c), u);
            row[c] = u;
            if (t.sum) put<S>(t.sum, r * a.C + c, u);
        }
        stats(a.pre, &st[2], &st[3]);
        if (t.y)
            for (int64_t c = threadIdx.x; c < a.C; c += 256) {
                float u = (row[c] - st[2]) * st[3];
                if (t.pre_w) u *= t.pre_w[c];
                if (t.pre_b) u += t.pre_b[c];
                put<T>(t.y, r * a.C + c, u);
            }
        if (t.stats && threadIdx.x < 4) t.stats[r * 4 + threadIdx.x] = st[threadIdx.x];
    }
}

template <typename T, typename S>
__global__ __launch_bounds__(256) void bwd_kernel(AnArgs a, float* ds_out) {
    __shared__ float red[4];
    extern __shared__ float row[];
    const AddnormTensors& t = a.t;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
        const float* st = t.stats + r * 4;
        const int64_t o = r * a.C;
        float m1 = 0.0f, m2 = 0.0f;
        auto e_of = [&](int64_t c) { return at<T>(t.dy, o + c) * (t.pre_w ? t.pre_w[c] : 1.0f); };
        auto xh_of = [&](int64_t c) { return (at<S>(t.sum, o + c) - st[2]) * st[3]; };
        if (a.pre != SELSCAN_NORM_NONE) {
            for (int64_t c = threadIdx.x; c < a.C; c += 256) {
                m1 += e_of(c);
                m2 += e_of(c) * xh_of(c);
            }
            m1 = a.pre == SELSCAN_NORM_LAYER ? block_sum(m1, red) / float(a.C) : 0.0f;
            m2 = block_sum(m2, red) / float(a.C);
        }
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            float ds = t.dsum ? at<S>(t.dsum, o + c) : 0.0f;
            if (a.pre != SELSCAN_NORM_NONE) ds += st[3] * (e_of(c) - m1 - xh_of(c) * m2);
            row[c] = ds;
        }
        m1 = m2 = 0.0f;
        auto f_of = [&](int64_t c) {
            return row[c] * a.scale * (t.gate ? t.gate[r / a.per_gate * a.C + c] : 1.0f) * (t.post_w ? t.post_w[c] : 1.0f);
        };
        auto x_of = [&](int64_t c) { return (at<T>(t.x, o + c) - st[0]) * st[1]; };
        if (a.post != SELSCAN_NORM_NONE) {
            for (int64_t c = threadIdx.x; c < a.C; c += 256) {
                m1 += f_of(c);
                m2 += f_of(c) * x_of(c);
            }
            m1 = a.post == SELSCAN_NORM_LAYER ? block_sum(m1, red) / float(a.C) : 0.0f;
            m2 = block_sum(m2, red) / float(a.C);
        }
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            if (ds_out) ds_out[o + c] = row[c];
            if (t.dx)
                put<T>(t.dx, o + c, a.post != SELSCAN_NORM_NONE ? st[1] * (f_of(c) - m1 - x_of(c) * m2) : f_of(c));
            if (t.dres) put<S>(t.dres, o + c, a.res_scale * row[c]);
        }
    }
}

// Column sums, one thread a column of a gate's rows.
template <typename T, typename S>
__global__ __launch_bounds__(64) void cols_kernel(AnArgs a, const float* ds, int gates, int mode) {
    const AddnormTensors& t = a.t;
    const int64_t c = int64_t(blockIdx.x) * 64 + threadIdx.x;
    if (c >= a.C) return;
    double s[5] = {};
    for (int64_t r = 0; r < a.R; ++r) {
        if (mode && r % a.per_gate == 0) s[4] = 0.0;
        const int64_t i = r * a.C + c;
        const float* st = t.stats + r * 4;
        const float g = t.gate ? t.gate[r / a.per_gate * a.C + c] : 1.0f;
        if (t.dpre_w || t.dpre_b) {
            const float dy = at<T>(t.dy, i);
            s[0] += dy * ((at<S>(t.sum, i) - st[2]) * st[3]);
            s[1] += dy;
        }
        const bool post = a.post != SELSCAN_NORM_NONE;
        const float du = a.scale * g * ds[i], xh = t.x ? (post ? (at<T>(t.x, i) - st[0]) * st[1] : at<T>(t.x, i)) : 0.0f;
        s[2] += du * xh;
        s[3] += du;
        if (mode) {
            const float u = fmaf(xh, t.post_w ? t.post_w[c] : 1.0f, t.post_b ? t.post_b[c] : 0.0f);
            s[4] += a.scale * u * ds[i];
            if (r % a.per_gate == a.per_gate - 1) t.dgate[r / a.per_gate * a.C + c] = float(s[4]);
        }
    }
    if (t.dpre_w) t.dpre_w[c] = float(s[0]);
    if (t.dpre_b) t.dpre_b[c] = float(s[1]);
    if (t.dpost_w) t.dpost_w[c] = float(s[2]);
    if (t.dpost_b) t.dpost_b[c] = float(s[3]);
}

AnArgs args_of(const AddnormTensors& t, const AddnormShape& s) {
    return AnArgs{t, s.R, s.C, s.G ? s.R / s.G : 1, s.post, s.pre, s.eps, s.scale, s.res_scale};
}

// f(type, residual's type)
template <typename F> void dispatch(const AddnormShape& s, F f) {
    if (s.dtype == DType::F32) f(float{}, float{});
    else if (s.res_dtype == DType::F32) f(bf16_bits{}, float{});
    else f(bf16_bits{}, bf16_bits{});
}

bool any_sum(const AddnormTensors& t) { return t.dpost_w || t.dpost_b || t.dpre_w || t.dpre_b || t.dgate; }

}  // namespace

size_t addnorm_bwd_workspace_bytes(const AddnormShape& s, const AddnormTensors& wanted) {
    return any_sum(wanted) ? size_t(s.R) * s.C * sizeof(float) : 0;
}

hipError_t launch_addnorm(const AddnormTensors& t, const AddnormShape& s, hipStream_t stream) {
    const AnArgs a = args_of(t, s);
    dispatch(s, [&](auto T, auto S) {
        hipLaunchKernelGGL((fwd_kernel<decltype(T), decltype(S)>), dim3(unsigned(s.R < 1 << 16 ? s.R : 1 << 16)),
                           dim3(256), unsigned(s.C * 4), stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_addnorm_bwd(const AddnormTensors& t, const AddnormShape& s, void* workspace, hipStream_t stream) {
    const AnArgs a = args_of(t, s);
    float* ds = any_sum(t) ? static_cast<float*>(workspace) : nullptr;
    dispatch(s, [&](auto T, auto S) {
        hipLaunchKernelGGL((bwd_kernel<decltype(T), decltype(S)>), dim3(unsigned(s.R < 1 << 16 ? s.R : 1 << 16)),
                           dim3(256), unsigned(s.C * 4), stream, a, ds);
        if (ds)
            hipLaunchKernelGGL((cols_kernel<decltype(T), decltype(S)>), dim3(unsigned((s.C + 63) / 64)), dim3(64), 0,
                               stream, a, ds, int(s.G), t.dgate ? 1 : 0);
    });
    return hipGetLastError();
}

}  // namespace selscan
