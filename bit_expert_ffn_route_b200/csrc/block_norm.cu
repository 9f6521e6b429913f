// block_norm.cu — the norms between one block and the next (include/moe_ops.h).
//
//   z = y r_y w_post,  x_out = alpha residual + gate z,  normed = x_out r_x w_next,
//   r = rsqrt(mean(v^2) + eps)
// Each element of y and the residual is read once and each of x_out and normed
// written once; a token stays in registers between the two norms.  Gradients
// likewise: four rows in, two out.  HBM bounds both.
//
// Threads: a group of whole warps takes a token, each thread the same columns of
// every token it takes, so that the sums over tokens stay in its registers;
// short rows put several groups in a block.  Groups walk over the tokens and
// fetch the rows of their next tokens with cp.async while they work: a thread
// copies just what it will read itself, so no barrier guards the copies.
#include <cuda_runtime.h>
#include <stdint.h>

#include "once.cuh"
#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

constexpr int kNormParts = 296;        // most blocks of the backward pass: two per SM, a partial of each weight gradient from every one
constexpr int kNormThreads = 384;      // threads that the groups of a block fill, about
constexpr int kMaxDynamic = 227 * 1024;
constexpr int kMaxGroups = 12;         // named barriers 1..12

template <int N>
MOE_DEVINL void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
MOE_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
MOE_DEVINL void cp_async16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// A group's threads: rank in the group, its warps, and sums over them.
struct Group {
    int g, rank, size;                          // group in the block, thread in the group, threads per group
    MOE_DEVINL explicit Group(int threads) : g(threadIdx.x / threads), rank(threadIdx.x % threads), size(threads) {}
    // N sums over the group, the same bits in every thread: lanes, then warps, in
    // a fixed order.  buf: [2][N][32] floats of this group; parity alternates
    // from call to call, so one barrier per call is enough.
    template <int N>
    MOE_DEVINL void sum(float (&v)[N], float* buf, int parity) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if (size == 32) return;
        float* b = buf + parity * N * 32;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) b[i * 32 + rank / 32] = v[i];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(size) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < size / 32 ? b[i * 32 + lane] : 0.f);
    }
};

// The rows of a group's coming tokens: STAGES tokens ahead in shared memory
// (16-byte packs), or read when they are wanted (STAGES 0).
template <typename T, int V, int ITER, int ROWS, int STAGES>
struct Rows {
    const T* src[ROWS];                         // null: no such row
    T* ring;                                    // [STAGES][ROWS][D] of this group
    int D, rank, size, stage = 0;
    MOE_DEVINL void fetch(int t, int T_, int to) {
        if constexpr (STAGES > 0) {
            if (t < T_) {
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
#pragma unroll
                    for (int i = 0; i < ITER; ++i) {
                        const int c = (i * size + rank) * V;
                        if (src[r] && c < D) cp_async16(ring + (size_t)(to * ROWS + r) * D + c, src[r] + (size_t)t * D + c);
                    }
            }
            cp_async_commit();
        }
    }
    MOE_DEVINL void begin(int t0, int step, int T_) {
        if constexpr (STAGES > 0) {
#pragma unroll
            for (int i = 0; i < STAGES; ++i) fetch(t0 + i * step, T_, i);
        }
    }
    MOE_DEVINL void wait() const {
        if constexpr (STAGES > 0) cp_async_wait<STAGES - 1>();
    }
    MOE_DEVINL void read(int r, int i, int t, float (&v)[V]) const {
        const int c = (i * size + rank) * V;
        if constexpr (STAGES > 0) load_f32<T, V>(ring + (size_t)(stage * ROWS + r) * D + c, v);
        else load_f32<T, V>(src[r] + (size_t)t * D + c, v);
    }
    // The token's rows have been read and used: fetch those of a later one in their place.
    MOE_DEVINL void refill(int t, int step, int T_) {
        if constexpr (STAGES > 0) {
            fetch(t + STAGES * step, T_, stage);
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }
    }
};

struct NormArgs {
    const void *y, *residual;
    const float* gate;
    int gate_mode;
    float alpha;
    const float *w_post, *w_next;
    float eps;
    int T, D, group;                            // group: threads per token
    void *x_out, *normed;
    float *rstd_post, *rstd_next;
};

template <typename T, int V, int ITER, int STAGES, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(NormArgs a) {
    extern __shared__ __align__(16) float dyn[];        // of every group: [2][32] for its sums; its ring
    const Group grp(a.group);
    const int groups = blockDim.x / a.group, step = gridDim.x * groups, t0 = blockIdx.x * groups + grp.g;
    Rows<T, V, ITER, 2, STAGES> in;
    in.src[0] = static_cast<const T*>(a.y);
    in.src[1] = static_cast<const T*>(a.residual);
    float* buf = dyn + grp.g * 64;
    in.ring = reinterpret_cast<T*>(dyn + groups * 64) + (size_t)grp.g * STAGES * 2 * a.D;
    in.D = a.D;
    in.rank = grp.rank;
    in.size = a.group;
    pdl_wait();
    in.begin(t0, step, a.T);
    const float inv = 1.f / a.D;
    int parity = 0;
    for (int t = t0; t < a.T; t += step) {
        float v[ITER][V], ss[1] = {0.f};
        in.wait();
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            if ((i * a.group + grp.rank) * V >= a.D) continue;
            in.read(0, i, t, v[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) ss[0] = __fmaf_rn(v[i][j], v[i][j], ss[0]);
        }
        float ry = 1.f;
        if (a.w_post) {
            grp.sum(ss, buf, parity ^= 1);
            ry = rsqrtf(__fmaf_rn(ss[0], inv, a.eps));
            if (a.rstd_post && grp.rank == 0) a.rstd_post[t] = ry;
        }
        if (a.gate_mode == MOE_GATE_TOKEN) ry *= __ldg(a.gate + t);
        ss[0] = 0.f;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * a.group + grp.rank) * V;
            if (c >= a.D) continue;
            float m[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] *= ry;
            if (a.w_post) {
                load_f32<float, V>(a.w_post + c, m);
#pragma unroll
                for (int j = 0; j < V; ++j) v[i][j] *= m[j];
            }
            if (a.gate_mode == MOE_GATE_CHANNEL) {
                load_f32<float, V>(a.gate + c, m);
#pragma unroll
                for (int j = 0; j < V; ++j) v[i][j] *= m[j];
            }
            if (a.residual) {
                in.read(1, i, t, m);
#pragma unroll
                for (int j = 0; j < V; ++j) v[i][j] = __fmaf_rn(a.alpha, m[j], v[i][j]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] = as_stored<T>(v[i][j]);
                ss[0] = __fmaf_rn(v[i][j], v[i][j], ss[0]);
            }
            if (a.x_out) store_f32<T, V>(static_cast<T*>(a.x_out) + (size_t)t * a.D + c, v[i]);
        }
        if (a.w_next) {
            grp.sum(ss, buf, parity ^= 1);
            const float rx = rsqrtf(__fmaf_rn(ss[0], inv, a.eps));
            if (a.rstd_next && grp.rank == 0) a.rstd_next[t] = rx;
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                const int c = (i * a.group + grp.rank) * V;
                if (c >= a.D) continue;
                float m[V];
                load_f32<float, V>(a.w_next + c, m);
#pragma unroll
                for (int j = 0; j < V; ++j) m[j] *= v[i][j] * rx;
                store_f32<T, V>(static_cast<T*>(a.normed) + (size_t)t * a.D + c, m);
            }
        }
        in.refill(t, step, a.T);
    }
}

struct NormGradArgs {
    const void *dx_out, *dnormed, *x_out, *y;   // dnormed, x_out: null without w_next; y: null if it is not read
    const float* gate;
    int gate_mode;
    float alpha;
    const float *w_post, *rstd_post, *w_next, *rstd_next;
    int T, D, group;
    void *dy, *dresidual;
    float *dgate, *dw_post, *dw_next;
    float* part;                        // [gridDim.x][3][D]: dw_next, dw_post, dgate (channel)
};

// With q = yh w_post gate and G = b - r c1 xh, b = dx_out + r u, c1 = mean(xh u),
// the second mean's sum is  sum(q G) = sum(q b) - r c1 sum(q xh):  all three sums
// of a token are formed at once, with one barrier.  A token gate stays outside
// of q: sum(q G) is then its gradient.
//   SMEM: the sums over tokens are kept in shared memory, for rows too wide for
//   the registers.
template <typename T, int V, int ITER, int STAGES, int THREADS, bool SMEM>
__global__ void __launch_bounds__(THREADS, THREADS == kNormThreads ? 2 : 1) block_norm_backward_kernel(NormGradArgs a) {
    extern __shared__ __align__(16) float dyn[];        // [2][3][32] per group, [3][D] sums, the groups' rings
    const Group grp(a.group);
    const int groups = blockDim.x / a.group, step = gridDim.x * groups, t0 = blockIdx.x * groups + grp.g;
    float *buf = dyn + grp.g * 192, *sums = dyn + groups * 192;         // the sums: with SMEM or several groups
    const bool joined = SMEM || groups > 1;
    Rows<T, V, ITER, 4, STAGES> in;
    in.src[0] = static_cast<const T*>(a.x_out);
    in.src[1] = static_cast<const T*>(a.dnormed);
    in.src[2] = static_cast<const T*>(a.dx_out);
    in.src[3] = static_cast<const T*>(a.y);
    in.ring = reinterpret_cast<T*>(sums + (joined ? 3 * a.D : 0)) + (size_t)grp.g * STAGES * 4 * a.D;
    in.D = a.D;
    in.rank = grp.rank;
    in.size = a.group;
    constexpr int N = SMEM ? 1 : ITER;
    float s_next[N][V], s_post[N][V], s_gate[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s_next[i][j] = s_post[i][j] = s_gate[i][j] = 0.f;
    if (SMEM) {
        for (int i = threadIdx.x; i < 3 * a.D; i += blockDim.x) sums[i] = 0.f;
        __syncthreads();
    }
    pdl_wait();
    in.begin(t0, step, a.T);
    const float inv = 1.f / a.D;
    int parity = 0;
    for (int t = t0; t < a.T; t += step, parity ^= 1) {
        const float rx = a.w_next ? __ldg(a.rstd_next + t) : 0.f;
        const float ry = a.w_post ? __ldg(a.rstd_post + t) : 1.f;
        const float gt = a.gate_mode == MOE_GATE_TOKEN ? __ldg(a.gate + t) : 1.f;
        float b[ITER][V], xh[ITER][V], yh[ITER][V];
        float s[3] = {0.f, 0.f, 0.f};           // xh u, q b, q xh
        in.wait();
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * a.group + grp.rank) * V;
            if (c >= a.D) continue;
            float m[V];
#pragma unroll
            for (int j = 0; j < V; ++j) b[i][j] = xh[i][j] = yh[i][j] = 0.f;
            if (a.w_next) {
                float w[V];
                in.read(0, i, t, xh[i]);
                in.read(1, i, t, m);
                load_f32<float, V>(a.w_next + c, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xh[i][j] *= rx;
                    if (!SMEM) s_next[i][j] = __fmaf_rn(m[j], xh[i][j], s_next[i][j]);
                    w[j] *= m[j];
                    s[0] = __fmaf_rn(xh[i][j], w[j], s[0]);
                    b[i][j] = rx * w[j];
                }
                if (SMEM && a.dw_next) {
                    load_f32<float, V>(sums + c, w);
#pragma unroll
                    for (int j = 0; j < V; ++j) w[j] = __fmaf_rn(m[j], xh[i][j], w[j]);
                    store_f32<float, V>(sums + c, w);
                }
            }
            if (a.dx_out) {
                in.read(2, i, t, m);
#pragma unroll
                for (int j = 0; j < V; ++j) b[i][j] += m[j];
            }
            if (a.y) {
                in.read(3, i, t, yh[i]);
                float q[V];
#pragma unroll
                for (int j = 0; j < V; ++j) q[j] = yh[i][j] *= ry;
                if (a.w_post) {
                    load_f32<float, V>(a.w_post + c, m);
#pragma unroll
                    for (int j = 0; j < V; ++j) q[j] *= m[j];
                }
                if (a.gate_mode == MOE_GATE_CHANNEL) {
                    load_f32<float, V>(a.gate + c, m);
#pragma unroll
                    for (int j = 0; j < V; ++j) q[j] *= m[j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    s[1] = __fmaf_rn(q[j], b[i][j], s[1]);
                    s[2] = __fmaf_rn(q[j], xh[i][j], s[2]);
                }
            }
        }
        grp.sum(s, buf, parity);
        in.refill(t, step, a.T);
        const float rc1 = rx * s[0] * inv, sq = __fmaf_rn(-rc1, s[2], s[1]);
        const float c2 = a.w_post ? gt * sq * inv : 0.f;
        if (a.gate_mode == MOE_GATE_TOKEN && a.dgate && grp.rank == 0) a.dgate[t] = sq;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * a.group + grp.rank) * V;
            if (c >= a.D) continue;
            const size_t at = (size_t)t * a.D + c;
            float m[V], wp[V];
#pragma unroll
            for (int j = 0; j < V; ++j) b[i][j] = __fmaf_rn(-rc1, xh[i][j], b[i][j]);       // G
            if (a.dresidual) {
#pragma unroll
                for (int j = 0; j < V; ++j) m[j] = a.alpha * b[i][j];
                store_f32<T, V>(static_cast<T*>(a.dresidual) + at, m);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) wp[j] = 1.f;
            if (a.w_post) load_f32<float, V>(a.w_post + c, wp);
            if (a.gate_mode == MOE_GATE_CHANNEL) {
                float sg[V];
                if (SMEM && a.dgate) load_f32<float, V>(sums + 2 * a.D + c, sg);
                load_f32<float, V>(a.gate + c, m);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float z = yh[i][j] * wp[j];
                    if (SMEM) sg[j] = __fmaf_rn(b[i][j], z, sg[j]);
                    else s_gate[i][j] = __fmaf_rn(b[i][j], z, s_gate[i][j]);
                    b[i][j] *= m[j];                                                        // dz
                }
                if (SMEM && a.dgate) store_f32<float, V>(sums + 2 * a.D + c, sg);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) b[i][j] *= gt;
            }
            if (SMEM && a.dw_post) {
                load_f32<float, V>(sums + a.D + c, m);
#pragma unroll
                for (int j = 0; j < V; ++j) m[j] = __fmaf_rn(b[i][j], yh[i][j], m[j]);
                store_f32<float, V>(sums + a.D + c, m);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!SMEM) s_post[i][j] = __fmaf_rn(b[i][j], yh[i][j], s_post[i][j]);
                m[j] = ry * __fmaf_rn(b[i][j], wp[j], -yh[i][j] * c2);
            }
            store_f32<T, V>(static_cast<T*>(a.dy) + at, m);
        }
    }
    // The block's sums: from the registers, or those of its groups added in order.
    float* part = a.part + (size_t)blockIdx.x * 3 * a.D;
    for (int g = 0; !SMEM && g < groups; ++g) {
        if (g == grp.g) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (i * a.group + grp.rank) * V;
                if (c >= a.D) continue;
                auto put = [&](int n, float (&v)[V]) {
                    if (g > 0) {
                        float w[V];
                        load_f32<float, V>(sums + n * a.D + c, w);
#pragma unroll
                        for (int j = 0; j < V; ++j) v[j] += w[j];
                    }
                    store_f32<float, V>((g == groups - 1 ? part : sums) + n * a.D + c, v);
                };
                if (a.dw_next) put(0, s_next[i]);
                if (a.dw_post) put(1, s_post[i]);
                if (a.dgate && a.gate_mode == MOE_GATE_CHANNEL) put(2, s_gate[i]);
            }
        }
        if (groups > 1) __syncthreads();
    }
    if (SMEM) {
        __syncthreads();
        for (int i = threadIdx.x; i < 3 * a.D; i += blockDim.x) part[i] = sums[i];
    }
}

// Column sums of the blocks' partials: 32 columns per block, an eighth of the
// partials per warp, the eighths added in order.
__global__ void __launch_bounds__(256) block_norm_join_kernel(const float* __restrict__ part, int n, int D,
                                                              float* dw_next, float* dw_post, float* dgate) {
    __shared__ float sums[8][32];
    float* out = blockIdx.y == 0 ? dw_next : blockIdx.y == 1 ? dw_post : dgate;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    pdl_wait();
    if (!out) return;
    const int each = (n + 7) / 8, i1 = min(n, (w + 1) * each);
    float s = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int i = w * each; i < i1; ++i) s += __ldg(part + ((size_t)i * 3 + blockIdx.y) * D + c);
    }
    sums[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][lane];
        out[c] = s;
    }
}

// Threads per token and tokens per block for rows of n packs per thread-iteration.
struct NormShape {
    int group, groups;
    NormShape(int D, int per_thread) {
        group = ((D + per_thread - 1) / per_thread + 31) / 32 * 32;
        groups = group >= kNormThreads ? 1 : kNormThreads / group;
        if (groups > kMaxGroups) groups = kMaxGroups;
    }
    int blocks(int T, int most) const {
        const int n = (T + groups - 1) / groups;
        return n < most ? n : most;
    }
};

template <typename T, int V, int ITER, int STAGES, int THREADS>
cudaError_t run_norm(NormArgs a, cudaStream_t s) {
    auto kernel = block_norm_kernel<T, V, ITER, STAGES, THREADS>;
    const NormShape n(a.D, V * ITER);
    const size_t smem = (size_t)n.groups * (256 + STAGES * 2 * a.D * sizeof(T));
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic) == cudaSuccess;
        }))
        return cudaErrorUnknown;
    a.group = n.group;
    const int per_sm = THREADS > 512 ? 1 : n.group * n.groups > kNormThreads ? 2 : 3;      // as their registers allow
    return launch_pdl(kernel, dim3(n.blocks(a.T, device_sm_count() * per_sm)), dim3(n.group * n.groups), smem, s, a);
}
template <typename T, int V, int ITER, int STAGES, int THREADS, bool SMEM>
cudaError_t run_norm_backward(NormGradArgs a, int* blocks, cudaStream_t s) {
    auto kernel = block_norm_backward_kernel<T, V, ITER, STAGES, THREADS, SMEM>;
    const NormShape n(a.D, V * ITER);
    const size_t smem = (SMEM || n.groups > 1 ? (size_t)3 * a.D * 4 : 0) +
                        (size_t)n.groups * (768 + STAGES * 4 * a.D * sizeof(T));
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic) == cudaSuccess;
        }))
        return cudaErrorUnknown;
    a.group = n.group;
    const int sms = device_sm_count() < kNormParts / 2 ? device_sm_count() : kNormParts / 2;
    *blocks = n.blocks(a.T, THREADS == kNormThreads ? 2 * sms : sms);
    return launch_pdl(kernel, dim3(*blocks), dim3(n.group * n.groups), smem, s, a);
}

// Rows up to 4,096 elements keep their sums over tokens in registers (8 of each
// per thread with 16-bit types, 4 with fp32); wider ones, and single elements
// where the rows are not of 16-byte packs, as the limits of threads and
// registers allow.
template <typename T>
cudaError_t pick_norm(const NormArgs& a, bool wide, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (!wide) {
        if (a.D <= 2048) return run_norm<T, 1, 4, 0, 512>(a, s);
        return run_norm<T, 1, 8, 0, 1024>(a, s);
    }
    if (a.D <= 512 * V) return run_norm<T, V, 1, 3, 512>(a, s);
    if (a.D <= 1024 * V) return run_norm<T, V, 1, 3, 1024>(a, s);
    return run_norm<T, V, sizeof(T) == 4 ? 2 : 1, 3, 1024>(a, s);
}
template <typename T>
cudaError_t pick_norm_backward(const NormGradArgs& a, bool wide, int* blocks, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (!wide) {
        if (a.D <= 4 * kNormThreads) return run_norm_backward<T, 1, 4, 0, kNormThreads, false>(a, blocks, s);
        if (a.D <= 2048) return run_norm_backward<T, 1, 4, 0, 512, false>(a, blocks, s);
        return run_norm_backward<T, 1, 8, 0, 1024, true>(a, blocks, s);
    }
    if (a.D <= kNormThreads * V) return run_norm_backward<T, V, 1, 3, kNormThreads, false>(a, blocks, s);
    if (a.D <= 512 * V) return run_norm_backward<T, V, 1, 3, 512, false>(a, blocks, s);
    if constexpr (sizeof(T) == 2) return run_norm_backward<T, V, 1, 2, 1024, true>(a, blocks, s);
    else if (a.D <= 1024 * V) return run_norm_backward<T, V, 1, 2, 1024, false>(a, blocks, s);
    else return run_norm_backward<T, V, 2, 0, 1024, true>(a, blocks, s);
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
    const NormArgs a{y, residual, gate, gate_mode, alpha, w_post, w_next, eps, T, D, 0, x_out, normed, rstd_post, rstd_next};
    return with_dtype(dtype, [&](auto e) { return ops_status(pick_norm<decltype(e)>(a, wide, (cudaStream_t)stream)); });
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
    const NormGradArgs a{dx_out, w_next ? dnormed : nullptr, w_next ? x_out : nullptr, w_post || dgate ? y : nullptr,
                         gate, gate_mode, alpha, w_post, rstd_post, w_next, rstd_next, T, D, 0, dy, dresidual, dgate,
                         dw_post, dw_next, static_cast<float*>(ws)};
    int blocks = 0;
    st = with_dtype(dtype, [&](auto e) { return ops_status(pick_norm_backward<decltype(e)>(a, wide, &blocks, s)); });
    if (st != MOE_OK || (!dw_next && !dw_post && !dgate_cols)) return st;
    return ops_status(launch_pdl(block_norm_join_kernel, dim3((D + 31) / 32, 3), dim3(256), 0, s,
                                 (const float*)ws, blocks, D, dw_next, dw_post, dgate_cols));
}
