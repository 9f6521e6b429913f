// block_norm.cu — the norms between one block and the next (include/moe_ops.h).
//
//   z = y r_y w_post,  x_out = alpha residual + gate z,  normed = x_out r_x w_next,
//   r = rsqrt(mean(v^2) + eps)
// Each element of y and the residual is read once and each of x_out and normed
// written once; a token stays in its block's registers between the two norms.
#include <cuda_runtime.h>
#include <stdint.h>

#include "once.cuh"
#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

constexpr int kNormParts = 296;        // blocks of the backward pass, each with a partial of every weight gradient

// Sum of v over the block's threads, the same value in every thread; fixed
// order (lanes, then warps).  `buf` is 32 floats used by this call only until
// the next __syncthreads.
MOE_DEVINL float block_sum(float v, float* buf) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) buf[w] = v;
    __syncthreads();
    return warp_sum(lane < nw ? buf[lane] : 0.f);
}

struct NormArgs {
    const void *y, *residual;
    const float* gate;
    int gate_mode;
    float alpha;
    const float *w_post, *w_next;
    float eps;
    int D;
    void *x_out, *normed;
    float *rstd_post, *rstd_next;
};

// One block per token, ITER packs of V elements per thread.
template <typename T, int V, int ITER>
__global__ void __launch_bounds__(1024) block_norm_kernel(NormArgs a) {
    __shared__ float buf[2][32];
    pdl_wait();
    const size_t t = blockIdx.x, at = t * a.D;
    const T* y = static_cast<const T*>(a.y) + at;
    const T* res = static_cast<const T*>(a.residual) + at;
    float v[ITER][V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < a.D) {
            load_f32<T, V>(y + c, v[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) ss = __fmaf_rn(v[i][j], v[i][j], ss);
        }
    }
    float ry = 1.f;
    if (a.w_post) {
        ry = rsqrtf(block_sum(ss, buf[0]) / a.D + a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = ry;
    }
    const float gt = a.gate_mode == MOE_GATE_TOKEN ? __ldg(a.gate + t) : 1.f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= a.D) continue;
        float m[V];
        if (a.w_post) {
            load_f32<float, V>(a.w_post + c, m);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] *= ry * m[j];
        }
        if (a.gate_mode == MOE_GATE_CHANNEL) {
            load_f32<float, V>(a.gate + c, m);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] *= m[j];
        } else if (a.gate_mode == MOE_GATE_TOKEN) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] *= gt;
        }
        if (a.residual) {
            load_f32<T, V>(res + c, m);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = __fmaf_rn(a.alpha, m[j], v[i][j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[i][j] = as_stored<T>(v[i][j]);         // x_out as it is stored
            ss = __fmaf_rn(v[i][j], v[i][j], ss);
        }
        if (a.x_out) store_f32<T, V>(static_cast<T*>(a.x_out) + at + c, v[i]);
    }
    if (!a.w_next) return;
    const float rx = rsqrtf(block_sum(ss, buf[1]) / a.D + a.eps);
    if (a.rstd_next && threadIdx.x == 0) a.rstd_next[t] = rx;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= a.D) continue;
        float m[V];
        load_f32<float, V>(a.w_next + c, m);
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] *= v[i][j] * rx;
        store_f32<T, V>(static_cast<T*>(a.normed) + at + c, m);
    }
}

struct NormGradArgs {
    const void *dx_out, *dnormed, *x_out, *y;
    const float* gate;
    int gate_mode;
    float alpha;
    const float *w_post, *rstd_post, *w_next, *rstd_next;
    int T, D;
    void *dy, *dresidual;
    float *dgate, *dw_post, *dw_next;
    float* part;                        // [gridDim.x][3][D]: dw_next, dw_post, dgate (channel)
};

// Blocks walk over the tokens t = blockIdx.x, + gridDim.x, ...; a thread owns
// the same columns of all of them and keeps their weight gradients.
template <typename T, int V, int ITER>
__global__ void __launch_bounds__(1024) block_norm_backward_kernel(NormGradArgs a) {
    __shared__ float buf[3][32];
    pdl_wait();
    float s_next[ITER][V], s_post[ITER][V], s_gate[ITER][V];
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s_next[i][j] = s_post[i][j] = s_gate[i][j] = 0.f;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t at = (size_t)t * a.D;
        const float rx = a.w_next ? __ldg(a.rstd_next + t) : 0.f;
        const float ry = a.w_post ? __ldg(a.rstd_post + t) : 1.f;
        float g[ITER][V], xh[ITER][V];
        float c1 = 0.f;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) g[i][j] = xh[i][j] = 0.f;
            if (c >= a.D || !a.w_next) continue;
            float w[V];
            load_f32<T, V>(static_cast<const T*>(a.x_out) + at + c, xh[i]);
            load_f32<T, V>(static_cast<const T*>(a.dnormed) + at + c, g[i]);
            load_f32<float, V>(a.w_next + c, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[i][j] *= rx;
                s_next[i][j] = __fmaf_rn(g[i][j], xh[i][j], s_next[i][j]);
                g[i][j] *= w[j];
                c1 = __fmaf_rn(xh[i][j], g[i][j], c1);
            }
        }
        if (a.w_next) c1 = block_sum(c1, buf[0]) / a.D;
        const float gt = a.gate_mode == MOE_GATE_TOKEN ? __ldg(a.gate + t) : 1.f;
        float c2 = 0.f, dot = 0.f;
        float yh[ITER][V];
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c >= a.D) continue;
            float m[V];
#pragma unroll
            for (int j = 0; j < V; ++j) g[i][j] = rx * (g[i][j] - xh[i][j] * c1);
            if (a.dx_out) {
                load_f32<T, V>(static_cast<const T*>(a.dx_out) + at + c, m);
#pragma unroll
                for (int j = 0; j < V; ++j) g[i][j] += m[j];
            }
            if (a.dresidual) {
#pragma unroll
                for (int j = 0; j < V; ++j) m[j] = a.alpha * g[i][j];
                store_f32<T, V>(static_cast<T*>(a.dresidual) + at + c, m);
            }
            float wp[V];
#pragma unroll
            for (int j = 0; j < V; ++j) wp[j] = 1.f, yh[i][j] = 0.f;
            if (a.w_post) load_f32<float, V>(a.w_post + c, wp);
            if (a.w_post || a.dgate) {
                load_f32<T, V>(static_cast<const T*>(a.y) + at + c, yh[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) yh[i][j] *= ry;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gz = g[i][j] * yh[i][j] * wp[j];
                s_gate[i][j] += gz;
                dot += gz;
                m[j] = gt;
            }
            if (a.gate_mode == MOE_GATE_CHANNEL) load_f32<float, V>(a.gate + c, m);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                g[i][j] *= m[j];                            // dz
                s_post[i][j] = __fmaf_rn(g[i][j], yh[i][j], s_post[i][j]);
                g[i][j] *= wp[j];
                c2 = __fmaf_rn(yh[i][j], g[i][j], c2);
            }
        }
        if (a.gate_mode == MOE_GATE_TOKEN && a.dgate) {
            dot = block_sum(dot, buf[2]);
            if (threadIdx.x == 0) a.dgate[t] = dot;
        }
        if (a.w_post) c2 = block_sum(c2, buf[1]) / a.D;
        else c2 = 0.f;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c >= a.D) continue;
            float m[V];
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] = ry * (g[i][j] - yh[i][j] * c2);
            store_f32<T, V>(static_cast<T*>(a.dy) + at + c, m);
        }
        __syncthreads();                                    // buf is used again by the next token
    }
    float* part = a.part + (size_t)blockIdx.x * 3 * a.D;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= a.D) continue;
        if (a.dw_next) store_f32<float, V>(part + c, s_next[i]);
        if (a.dw_post) store_f32<float, V>(part + a.D + c, s_post[i]);
        if (a.dgate && a.gate_mode == MOE_GATE_CHANNEL) store_f32<float, V>(part + 2 * a.D + c, s_gate[i]);
    }
}

// Column sums of the blocks' partials, in block order.
__global__ void __launch_bounds__(256) block_norm_join_kernel(const float* __restrict__ part, int n, int D,
                                                              float* dw_next, float* dw_post, float* dgate) {
    pdl_wait();
    float* out = blockIdx.y == 0 ? dw_next : blockIdx.y == 1 ? dw_post : dgate;
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (!out || c >= D) return;
    float s = 0.f;
    for (int i = 0; i < n; ++i) s += __ldg(part + ((size_t)i * 3 + blockIdx.y) * D + c);
    out[c] = s;
}

template <typename T, int V, int ITER>
cudaError_t run_norm(const NormArgs& a, int T_, int threads, cudaStream_t s) {
    return launch_pdl(block_norm_kernel<T, V, ITER>, dim3(T_), dim3(threads), 0, s, a);
}
template <typename T, int V, int ITER>
cudaError_t run_norm_backward(const NormGradArgs& a, int blocks, int threads, cudaStream_t s) {
    return launch_pdl(block_norm_backward_kernel<T, V, ITER>, dim3(blocks), dim3(threads), 0, s, a);
}

inline int warps_of(int n) { return (n + 31) / 32 * 32; }

template <typename T, int V>
cudaError_t pick_norm(const NormArgs& a, int T_, cudaStream_t s) {
    const int n = (a.D + V - 1) / V;            // packs per token
    if (n <= 1024) return run_norm<T, V, 1>(a, T_, warps_of(n), s);
    if (n <= 2048) return run_norm<T, V, 2>(a, T_, 1024, s);
    if (n <= 4096) return run_norm<T, V, 4>(a, T_, 1024, s);
    return run_norm<T, V, 8>(a, T_, 1024, s);
}
template <typename T, int V>
cudaError_t pick_norm_backward(const NormGradArgs& a, int blocks, cudaStream_t s) {
    const int n = (a.D + V - 1) / V;
    if (n <= 1024) return run_norm_backward<T, V, 1>(a, blocks, warps_of(n), s);
    if (n <= 2048) return run_norm_backward<T, V, 2>(a, blocks, 1024, s);
    if (n <= 4096) return run_norm_backward<T, V, 4>(a, blocks, 1024, s);
    return run_norm_backward<T, V, 8>(a, blocks, 1024, s);
}

moe_status norm_shapes(int T, int D) { return ops_shapes(T, 1, D); }

bool gate_ok(const float* gate, int mode) {
    if (mode == MOE_GATE_NONE) return !gate;
    return (mode == MOE_GATE_CHANNEL || mode == MOE_GATE_TOKEN) && gate && ops_aligned(gate, 4);
}

// |v| < infinity, and not NaN
bool finite(float v) { return v - v == 0.f; }

size_t norm_ws_bytes(int T, int D) { return (size_t)(T < kNormParts ? T : kNormParts) * 3 * D * 4 + 256; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_norm(const void* y, const void* residual, const float* gate, int gate_mode,
                                     float alpha, const float* w_post, const float* w_next, float eps, int T, int D,
                                     int dtype, void* x_out, void* normed, float* rstd_post, float* rstd_next,
                                     moe_stream_t stream) {
    moe_status st = norm_shapes(T, D);
    if (st != MOE_OK) return st;
    if (!dtype_ok(dtype) || !(eps >= 0.f) || !finite(eps) || !finite(alpha)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const size_t es = dtype_size(dtype);
    if (!y || !gate_ok(gate, gate_mode) || !w_next != !normed || (!x_out && !normed)) return MOE_ERR_INVALID_ARG;
    if ((rstd_post && !w_post) || (rstd_next && !w_next)) return MOE_ERR_INVALID_ARG;
    if (normed && (normed == y || normed == residual || normed == x_out)) return MOE_ERR_INVALID_ARG;
    if (!ops_aligned(y, es) || !ops_aligned(residual, es) || !ops_aligned(x_out, es) || !ops_aligned(normed, es) ||
        !ops_aligned(w_post, 4) || !ops_aligned(w_next, 4) || !ops_aligned(rstd_post, 4) || !ops_aligned(rstd_next, 4))
        return MOE_ERR_INVALID_ARG;
    const bool wide = (D * es) % 16 == 0 && ops_aligned(y, 16) && ops_aligned(residual, 16) && ops_aligned(x_out, 16) &&
                      ops_aligned(normed, 16) && ops_aligned(w_post, 16) && ops_aligned(w_next, 16) &&
                      (gate_mode != MOE_GATE_CHANNEL || ops_aligned(gate, 16));
    const NormArgs a{y, residual, gate, gate_mode, alpha, w_post, w_next, eps, D, x_out, normed, rstd_post, rstd_next};
    cudaStream_t s = (cudaStream_t)stream;
    return with_dtype(dtype, [&](auto e) {
        using Tp = decltype(e);
        return ops_status(wide ? pick_norm<Tp, 16 / sizeof(Tp)>(a, T, s) : pick_norm<Tp, 1>(a, T, s));
    });
}

extern "C" size_t moe_block_norm_backward_workspace_size(int T, int D) {
    return norm_shapes(T, D) == MOE_OK ? norm_ws_bytes(T, D) : 0;
}

extern "C" moe_status moe_block_norm_backward(const void* dx_out, const void* dnormed, const void* x_out,
                                              const void* y, const float* gate, int gate_mode, float alpha,
                                              const float* w_post, const float* rstd_post, const float* w_next,
                                              const float* rstd_next, int T, int D, int dtype, void* dy,
                                              void* dresidual, float* dgate, float* dw_post, float* dw_next, void* ws,
                                              size_t ws_bytes, moe_stream_t stream) {
    moe_status st = norm_shapes(T, D);
    if (st != MOE_OK) return st;
    if (!dtype_ok(dtype) || !finite(alpha)) return MOE_ERR_INVALID_ARG;
    if ((dgate && gate_mode == MOE_GATE_NONE) || (dw_post && !w_post) || (dw_next && !w_next))
        return MOE_ERR_INVALID_ARG;
    if (!ops_aligned(dgate, 4) || !ops_aligned(dw_post, 4) || !ops_aligned(dw_next, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t cols = (size_t)D * 4;
    float* dgate_cols = gate_mode == MOE_GATE_CHANNEL ? dgate : nullptr;
    if (T == 0) {
        for (float* p : {dw_next, dw_post, dgate_cols})
            if (p && cudaMemsetAsync(p, 0, cols, s) != cudaSuccess) return ops_status(cudaErrorUnknown);
        return MOE_OK;
    }
    const size_t es = dtype_size(dtype);
    if (!dy || !gate_ok(gate, gate_mode) || !w_next != !dnormed || (!dx_out && !dnormed)) return MOE_ERR_INVALID_ARG;
    if ((w_next && (!x_out || !rstd_next)) || (w_post && !rstd_post) || ((w_post || dgate) && !y))
        return MOE_ERR_INVALID_ARG;
    for (const void* in : {dx_out, dnormed, x_out, y})
        if (in && (dy == in || (dresidual == in && in != dx_out))) return MOE_ERR_INVALID_ARG;
    if (dy == dresidual) return MOE_ERR_INVALID_ARG;
    if (!ops_aligned(dx_out, es) || !ops_aligned(dnormed, es) || !ops_aligned(x_out, es) || !ops_aligned(y, es) ||
        !ops_aligned(dy, es) || !ops_aligned(dresidual, es) || !ops_aligned(w_post, 4) || !ops_aligned(w_next, 4) ||
        !ops_aligned(rstd_post, 4) || !ops_aligned(rstd_next, 4) || !ws || !ops_aligned(ws, 256))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < norm_ws_bytes(T, D)) return MOE_ERR_WORKSPACE;
    const bool wide = (D * es) % 16 == 0 && ops_aligned(dx_out, 16) && ops_aligned(dnormed, 16) &&
                      ops_aligned(x_out, 16) && ops_aligned(y, 16) && ops_aligned(dy, 16) &&
                      ops_aligned(dresidual, 16) && ops_aligned(w_post, 16) && ops_aligned(w_next, 16) &&
                      (gate_mode != MOE_GATE_CHANNEL || ops_aligned(gate, 16));
    const int blocks = T < kNormParts ? T : kNormParts;
    const NormGradArgs a{dx_out,    dnormed, x_out, y,  gate, gate_mode, alpha, w_post,  rstd_post, w_next,
                         rstd_next, T,       D,     dy, dresidual, dgate, dw_post, dw_next, static_cast<float*>(ws)};
    st = with_dtype(dtype, [&](auto e) {
        using Tp = decltype(e);
        return ops_status(wide ? pick_norm_backward<Tp, 16 / sizeof(Tp)>(a, blocks, s)
                               : pick_norm_backward<Tp, 1>(a, blocks, s));
    });
    if (st != MOE_OK || (!dw_next && !dw_post && !dgate_cols)) return st;
    return ops_status(launch_pdl(block_norm_join_kernel, dim3((D + 255) / 256, 3), dim3(256), 0, s,
                                 (const float*)ws, blocks, D, dw_next, dw_post, dgate_cols));
}
