// Linear attention with a decay for each head: walks of the layer's
// recurrence (prompts and gradients) and its one-token step.
#include "common.hpp"
#include "launch.hpp"

namespace selscan {
namespace {

constexpr int kCols = 64;  // state columns of a workgroup

struct WalkArgs {
    LinattnWalk w;
    const float* log_decay;  // [H]
    const int32_t* lengths;  // [batch] or null
    float scale;
    int64_t L, H;
    const void* dy;      // slope walk: [batch, L, H, P]
    const float* dlast;  // slope walk: the state's strides, or null
    float* part;         // slope walk: one sum per workgroup
};

__device__ __forceinline__ int64_t entry_length(const int32_t* lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < L ? n : L;
}

// Token by token: thread (p, r) holds the state rows n = r + 4 i of column p.
// SLOPE: the derivative of the outputs by log_decay, summed against dy.
template <typename T, bool SLOPE>
__global__ __launch_bounds__(256) void walk_kernel(WalkArgs g) {
    __shared__ float as[256], bs[256], red[2][4][kCols];
    const int tid = threadIdx.x, p = tid % kCols, r = tid / kCols;
    const int tiles = (g.w.P + kCols - 1) / kCols;
    const int64_t bh = blockIdx.x / tiles, b = bh / g.H, h = bh % g.H;
    const int col = int(blockIdx.x % tiles) * kCols + p;
    const bool live = col < g.w.P;
    const int64_t len = entry_length(g.lengths, b, g.L);
    const float lam = expf(g.log_decay[h]);
    const int64_t ra = h / (g.H / g.w.ha), rb = h / (g.H / g.w.hb), rc = h / (g.H / g.w.hc);
    float S[64], D[64];
    const int64_t sbase = bh * g.w.K * g.w.P + int64_t(col) * g.w.sp;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        const int n = r + 4 * i;
        S[i] = g.w.s0 && live && n < g.w.K ? g.w.s0[sbase + int64_t(n) * g.w.sn] : 0.0f;
        D[i] = 0.0f;
    }
    float total = 0.0f;
    for (int64_t i = 0; i < g.L; ++i) {
        const int64_t t = g.w.rev ? g.L - 1 - i : i;
        const int64_t row = b * g.L + t;
        const int64_t at = (row * g.H + h) * g.w.P + col;
        if (t >= len) {
            if (!SLOPE && live && r == 0) {
                if (g.w.o_f32) static_cast<float*>(g.w.o)[at] = 0.0f;
                else static_cast<T*>(g.w.o)[at] = from_f32<T>(0.0f);
            }
            continue;
        }
        __syncthreads();
        if (tid < g.w.K) {
            as[tid] = to_f32(static_cast<const T*>(g.w.a)[(row * g.w.ha + ra) * g.w.K + tid]);
            bs[tid] = to_f32(static_cast<const T*>(g.w.b)[(row * g.w.hb + rb) * g.w.K + tid]);
        }
        const float c0 = live ? to_f32(static_cast<const T*>(g.w.c)[(row * g.w.hc + rc) * g.w.P + col]) : 0.0f;
        const float c = g.w.rev ? c0 * g.scale : c0;
        __syncthreads();
        float y = 0.0f, y2 = 0.0f;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
            const int n = r + 4 * j;
            if (n < g.w.K) {
                if (SLOPE) D[j] = lam * (D[j] + S[j]);
                S[j] = fmaf(bs[n], c, g.w.rev ? S[j] : lam * S[j]);
                y = fmaf(as[n], S[j], y);
                if (SLOPE) y2 = fmaf(as[n], D[j], y2);
                if (g.w.rev) S[j] *= lam;
            }
        }
        red[0][r][p] = SLOPE ? y2 : y;
        __syncthreads();
        if (r == 0 && live) {
            float o = red[0][0][p] + red[0][1][p] + red[0][2][p] + red[0][3][p];
            if (!g.w.rev) o *= g.scale;
            if (SLOPE) total = fmaf(o, to_f32(static_cast<const T*>(g.dy)[at]), total);
            else if (g.w.o_f32) static_cast<float*>(g.w.o)[at] = o;
            else static_cast<T*>(g.w.o)[at] = from_f32<T>(o);
        }
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            const int n = r + 4 * i;
            if (n < g.w.K) {
                if (SLOPE) {
                    if (g.dlast) total = fmaf(D[i], g.dlast[sbase + int64_t(n) * g.w.sn], total);
                } else if (g.w.s1) {
                    g.w.s1[sbase + int64_t(n) * g.w.sn] = S[i];
                }
            }
        }
    }
    if (SLOPE) {
        __syncthreads();
        red[0][r][p] = total;
        __syncthreads();
        if (tid == 0) {
            float s = 0.0f;
            for (int i = 0; i < 256; ++i) s += red[0][i / kCols][i % kCols];
            g.part[blockIdx.x] = s;
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

template <typename T>
void walk(const LinattnWalk& w, const LinattnTensors& t, const LinattnShape& s, hipStream_t st) {
    WalkArgs g{w, t.log_decay, t.lengths, t.scale, s.L, s.heads, nullptr, nullptr, nullptr};
    hipLaunchKernelGGL((walk_kernel<T, false>), dim3(unsigned(s.batch * s.heads * col_tiles(w.P))), dim3(256), 0, st, g);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of the backward: the heads' partial dk and dv where heads share
// keys and values, and the slope walk's sums.
size_t partial_bytes(const LinattnShape& s, int64_t D) {
    return s.heads == s.kv_heads ? 0 : up256(size_t(s.batch * s.L * s.heads * D) * 4);
}

template <typename T>
hipError_t bwd(const LinattnTensors& t, const LinattnShape& s, void* workspace, hipStream_t st) {
    char* ws = static_cast<char*>(workspace);
    const bool shared = s.heads != s.kv_heads;
    float* pk = reinterpret_cast<float*>(ws);
    float* pv = reinterpret_cast<float*>(ws + partial_bytes(s, s.dk));
    float* part = reinterpret_cast<float*>(ws + partial_bytes(s, s.dk) + partial_bytes(s, s.dv));
    const int H = int(s.heads), Hk = int(s.kv_heads), dk = int(s.dk), dv = int(s.dv);
    walk<T>({t.dy, t.v, t.k, t.dq, t.h0, nullptr, H, Hk, Hk, dv, dk, 1, dv, false, false}, t, s, st);
    walk<T>({t.v, t.dy, t.q, shared ? pk : t.dk, t.dlast, nullptr, Hk, H, H, dv, dk, 1, dv, true, shared}, t, s, st);
    walk<T>({t.k, t.q, t.dy, shared ? pv : t.dv, t.dlast, t.dh0, Hk, H, H, dk, dv, dv, 1, true, shared}, t, s, st);
    if (shared) {
        const int64_t nk = s.batch * s.L * Hk * dk, nv = s.batch * s.L * Hk * dv;
        hipLaunchKernelGGL((head_sum_kernel<T>), grid_of(nk), dim3(256), 0, st, pk,
                           static_cast<T*>(t.dk), nk, s.heads, s.kv_heads, dk);
        hipLaunchKernelGGL((head_sum_kernel<T>), grid_of(nv), dim3(256), 0, st, pv,
                           static_cast<T*>(t.dv), nv, s.heads, s.kv_heads, dv);
    }
    if (t.dlog_decay) {
        WalkArgs g{{t.q, t.k, t.v, nullptr, t.h0, nullptr, H, Hk, Hk, dk, dv, dv, 1, false, false},
                   t.log_decay, t.lengths, t.scale, s.L, s.heads, t.dy, t.dlast, part};
        hipLaunchKernelGGL((walk_kernel<T, true>), dim3(unsigned(s.batch * H * col_tiles(dv))), dim3(256), 0, st, g);
        hipLaunchKernelGGL(slope_sum_kernel, dim3(unsigned((H + 63) / 64)), dim3(64), 0, st, part, t.dlog_decay,
                           s.batch, s.heads, col_tiles(dv));
    }
    return hipGetLastError();
}

}  // namespace

LinattnPlan linattn_plan(const LinattnShape& s, int32_t requested, bool backward) {
    (void)requested;
    (void)backward;
    return {1, s.L};
}
size_t linattn_fwd_workspace_bytes(const LinattnShape&, const LinattnPlan&) { return 0; }
size_t linattn_bwd_workspace_bytes(const LinattnShape& s, const LinattnPlan&, bool slope) {
    return partial_bytes(s, s.dk) + partial_bytes(s, s.dv) +
           (slope ? up256(size_t(s.batch * s.heads * col_tiles(s.dv)) * 4) : 0);
}

hipError_t launch_linattn_fwd(const LinattnTensors& t, const LinattnShape& s, const LinattnPlan&, void*,
                              hipStream_t stream) {
    const int H = int(s.heads), Hk = int(s.kv_heads), dk = int(s.dk), dv = int(s.dv);
    const LinattnWalk w{t.q, t.k, t.v, t.y, t.h0, t.last_state, H, Hk, Hk, dk, dv, dv, 1, false, false};
    if (s.dtype == DType::BF16) walk<bf16_bits>(w, t, s, stream);
    else walk<float>(w, t, s, stream);
    return hipGetLastError();
}

hipError_t launch_linattn_bwd(const LinattnTensors& t, const LinattnShape& s, const LinattnPlan&, void* workspace,
                              hipStream_t stream) {
    return s.dtype == DType::BF16 ? bwd<bf16_bits>(t, s, workspace, stream) : bwd<float>(t, s, workspace, stream);
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
