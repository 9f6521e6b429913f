// permute.cu — tokens sorted by expert and back, weighted, with the gradients of
// both (include/moe_ops.h).
//
// With row(p) the place of pair p = t*k + r among the taken pairs, ordered by
// expert and then by p:
//   permute            rows[row(p)] = x[t]
//   unpermute          out[t] = sum_r w[t,r] rows[row(t,r)]
//   permute backward   the same sum with w = 1, of the rows' gradients
//   unpermute backward drows[row(p)] = w[p] dout[t],  dw[p] = <dout[t], rows[row(p)]>
// Every one of them moves each row once and each token once: HBM bounds them.
#include <cuda_runtime.h>
#include <stdint.h>

#include "once.cuh"
#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// The expert of pair p, or -1 if the pair is not taken.
MOE_DEVINL int taken_expert(const int32_t* ids, int p, int E, const int32_t* slot_table, int n_slots) {
    const int e = __ldg(ids + p);
    if (e < 0 || e >= E) return -1;
    if (slot_table) {
        const int s = __ldg(slot_table + e);
        if (s >= 0 && s < n_slots) return -1;
    }
    return e;
}

// The plan: a stable counting sort of the P pairs by expert in one block.  Warp
// w owns the pairs of segment w, 32 at a time in order; lanes with the same
// expert find one another (match), the first of them adds their number to the
// warp's counter of that expert.  An exclusive scan over (expert, warp) turns
// the counters into first rows, and the second walk over the pairs hands them out.
__global__ void __launch_bounds__(kPlanThreads) permute_plan_kernel(const int32_t* __restrict__ ids, int P, int E,
                                                                    const int32_t* __restrict__ slot_table,
                                                                    int n_slots, int32_t* __restrict__ offsets,
                                                                    int32_t* __restrict__ pair_row,
                                                                    int32_t* __restrict__ row_pair) {
    extern __shared__ int32_t count[];          // [warp][E]
    __shared__ int wsum[32];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kPlanWarps * E; i += kPlanThreads) count[i] = 0;
    __syncthreads();
    const int seg = ((P + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int p0 = w * seg, p1 = min(P, p0 + seg);
    int32_t* mine = count + w * E;
    for (int p = p0; p < p1; p += 32) {
        const int e = p + lane < p1 ? taken_expert(ids, p + lane, E, slot_table, n_slots) : -1;
        const uint32_t peers = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    // thread e: the expert's total, and its warps' counters as offsets inside the expert
    int total = 0;
    if (threadIdx.x < E) {
        for (int i = 0; i < kPlanWarps; ++i) {
            const int c = count[i * E + threadIdx.x];
            count[i * E + threadIdx.x] = total;
            total += c;
        }
    }
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    if (w == 0) {
        int t = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        wsum[lane] = t;
    }
    __syncthreads();
    if (threadIdx.x < E) {
        const int base = incl - total + (w ? wsum[w - 1] : 0);
        offsets[threadIdx.x] = base;
        if (threadIdx.x == E - 1) offsets[E] = base + total;
        for (int i = 0; i < kPlanWarps; ++i) count[i * E + threadIdx.x] += base;
    }
    __syncthreads();
    for (int p = p0; p < p1; p += 32) {
        const int e = p + lane < p1 ? taken_expert(ids, p + lane, E, slot_table, n_slots) : -1;
        const uint32_t peers = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = mine[e] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
        __syncwarp();
        if (p + lane < p1) {
            pair_row[p + lane] = row;
            if (row >= 0) row_pair[row] = p + lane;
        }
    }
}

// rows[pair_row[t][r]] = x[t]: one block per token, the token read once.
template <typename T, int V>
__global__ void __launch_bounds__(256) permute_rows_kernel(const T* __restrict__ x,
                                                           const int32_t* __restrict__ pair_row, int k, int D,
                                                           T* __restrict__ rows) {
    pdl_wait();
    const int t = blockIdx.x;
    for (int c = threadIdx.x * V; c < D; c += blockDim.x * V) {
        const Pack<T, V> a = load_pack<T, V>(x + (size_t)t * D + c);
        for (int r = 0; r < k; ++r) {
            const int row = __ldg(pair_row + t * k + r);
            if (row >= 0) store_pack<T, V>(rows + (size_t)row * D + c, a);
        }
    }
}

// out[t] = sum_r w[t,r] rows[row(t,r)], r ascending in fp32 (w NULL: 1).
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(256) unpermute_kernel(const T* __restrict__ rows, int n_rows,
                                                        const int32_t* __restrict__ pair_row,
                                                        const float* __restrict__ weights, int k, int D,
                                                        TO* __restrict__ out) {
    pdl_wait();
    const int t = blockIdx.x;
    for (int c = threadIdx.x * V; c < D; c += blockDim.x * V) {
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        for (int r = 0; r < k; ++r) {
            const int row = __ldg(pair_row + t * k + r);
            if (row < 0 || row >= n_rows) continue;
            const float w = weights ? __ldg(weights + t * k + r) : 1.f;
            float y[V];
            load_f32<T, V>(rows + (size_t)row * D + c, y);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(w, y[i], acc[i]);
        }
        store_f32<TO, V>(out + (size_t)t * D + c, acc);
    }
}

// drows[row(t,r)] = w[t,r] dout[t] and dw[t,r] = <dout[t], rows[row(t,r)]>.
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(256) unpermute_backward_kernel(const TO* __restrict__ dout,
                                                                 const T* __restrict__ rows, int n_rows,
                                                                 const int32_t* __restrict__ pair_row,
                                                                 const float* __restrict__ weights, int k, int D,
                                                                 T* __restrict__ drows, float* __restrict__ dweights) {
    __shared__ float part[kMaxTopK][8];
    pdl_wait();
    const int t = blockIdx.x, lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    float dot[kMaxTopK];
#pragma unroll
    for (int r = 0; r < kMaxTopK; ++r) dot[r] = 0.f;
    for (int c = threadIdx.x * V; c < D; c += blockDim.x * V) {
        float d[V];
        load_f32<TO, V>(dout + (size_t)t * D + c, d);
#pragma unroll
        for (int r = 0; r < kMaxTopK; ++r) {
            if (r >= k) continue;
            const int row = __ldg(pair_row + t * k + r);
            if (row < 0 || row >= n_rows) continue;
            if (dweights) {
                float y[V];
                load_f32<T, V>(rows + (size_t)row * D + c, y);
#pragma unroll
                for (int i = 0; i < V; ++i) dot[r] = __fmaf_rn(d[i], y[i], dot[r]);
            }
            if (drows) {
                const float w = weights ? __ldg(weights + t * k + r) : 1.f;
                float g[V];
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = w * d[i];
                store_f32<T, V>(drows + (size_t)row * D + c, g);
            }
        }
    }
    if (!dweights) return;
#pragma unroll
    for (int r = 0; r < kMaxTopK; ++r) {
        if (r >= k) continue;
        const float s = warp_sum(dot[r]);
        if (lane == 0) part[r][wp] = s;
    }
    __syncthreads();
    if (threadIdx.x < k) {
        float s = 0.f;
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += part[threadIdx.x][i];
        dweights[(size_t)t * k + threadIdx.x] = s;
    }
}

// Threads for a row of n packs: one pack per thread, whole warps, at most 256.
inline int row_threads(int n) { return n >= 256 ? 256 : (n + 31) / 32 * 32; }

// Rows whose bytes are a multiple of 16, in 16-byte aligned buffers.
template <typename... P>
inline bool wide_rows(int D, size_t elem, P... p) {
    return (D * elem) % 16 == 0 && (ops_aligned(p, 16) && ...);
}

template <typename T, typename TO, int V>
cudaError_t run_unpermute(const void* rows, int n_rows, const int32_t* pair_row, const float* weights, int T_, int k,
                          int D, void* out, cudaStream_t s) {
    return launch_pdl(unpermute_kernel<T, TO, V>, dim3(T_), dim3(row_threads((D + V - 1) / V)), 0, s,
                      static_cast<const T*>(rows), n_rows, pair_row, weights, k, D, static_cast<TO*>(out));
}
template <typename T, typename TO, int V>
cudaError_t run_unpermute_backward(const void* dout, const void* rows, int n_rows, const int32_t* pair_row,
                                   const float* weights, int T_, int k, int D, void* drows, float* dweights,
                                   cudaStream_t s) {
    return launch_pdl(unpermute_backward_kernel<T, TO, V>, dim3(T_), dim3(row_threads((D + V - 1) / V)), 0, s,
                      static_cast<const TO*>(dout), static_cast<const T*>(rows), n_rows, pair_row, weights, k, D,
                      static_cast<T*>(drows), dweights);
}

moe_status launch_unpermute(const void* rows, int n_rows, const int32_t* pair_row, const float* weights, int T_, int k,
                            int D, int dtype, void* out, int out_dtype, cudaStream_t s) {
    const bool wide = wide_rows(D, dtype_size(dtype), rows, out);
    return with_dtype(dtype, [&](auto e) {
        using T = decltype(e);
        constexpr int V = 16 / sizeof(T);
        if (out_dtype == MOE_F32)
            return ops_status(wide ? run_unpermute<T, float, V>(rows, n_rows, pair_row, weights, T_, k, D, out, s)
                                   : run_unpermute<T, float, 1>(rows, n_rows, pair_row, weights, T_, k, D, out, s));
        return ops_status(wide ? run_unpermute<T, T, V>(rows, n_rows, pair_row, weights, T_, k, D, out, s)
                               : run_unpermute<T, T, 1>(rows, n_rows, pair_row, weights, T_, k, D, out, s));
    });
}

bool out_dtype_ok(int dtype, int out_dtype) { return out_dtype == dtype || out_dtype == MOE_F32; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_permute(const int32_t* ids, int T, int k, int E, const int32_t* slot_table, int n_slots,
                                  const void* x, int D, int dtype, void* rows, int32_t* offsets, int32_t* pair_row,
                                  int32_t* row_pair, moe_stream_t stream) {
    moe_status st = ops_shapes(T, k, D);
    if (st != MOE_OK) return st;
    if (E <= 0 || n_slots < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (E > kOpsMaxE) return MOE_ERR_UNSUPPORTED;
    if (!offsets || !ops_aligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) return ops_status(cudaMemsetAsync(offsets, 0, (E + 1) * sizeof(int32_t), s));
    if (!ids || !pair_row || !row_pair || !x != !rows) return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_size(dtype);
    if (!ops_aligned(ids, 4) || !ops_aligned(pair_row, 4) || !ops_aligned(row_pair, 4) || !ops_aligned(slot_table, 4) ||
        !ops_aligned(x, es) || !ops_aligned(rows, es) || (x && x == rows))
        return MOE_ERR_INVALID_ARG;
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [] {
            return cudaFuncSetAttribute(permute_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kPlanWarps * kOpsMaxE * 4) == cudaSuccess;
        }))
        return MOE_ERR_CUDA;
    cudaError_t e = launch_pdl(permute_plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)kPlanWarps * E * 4, s, ids,
                               T * k, E, slot_table, n_slots, offsets, pair_row, row_pair);
    if (e != cudaSuccess || !x) return ops_status(e);
    const bool wide = wide_rows(D, es, x, rows);
    return with_dtype(dtype, [&](auto el) {
        using Tp = decltype(el);
        constexpr int V = 16 / sizeof(Tp);
        const Tp* xt = static_cast<const Tp*>(x);
        Tp* rt = static_cast<Tp*>(rows);
        return ops_status(wide ? launch_pdl(permute_rows_kernel<Tp, V>, dim3(T), dim3(row_threads(D / V)), 0, s, xt,
                                            (const int32_t*)pair_row, k, D, rt)
                               : launch_pdl(permute_rows_kernel<Tp, 1>, dim3(T), dim3(row_threads(D)), 0, s, xt,
                                            (const int32_t*)pair_row, k, D, rt));
    });
}

extern "C" moe_status moe_unpermute(const void* rows, int n_rows, const int32_t* pair_row, const float* weights, int T,
                                    int k, int D, int dtype, void* out, int out_dtype, moe_stream_t stream) {
    moe_status st = ops_shapes(T, k, D);
    if (st != MOE_OK) return st;
    if (n_rows < 0 || !dtype_ok(dtype) || !out_dtype_ok(dtype, out_dtype)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!pair_row || !out || (n_rows > 0 && !rows) || out == rows) return MOE_ERR_INVALID_ARG;
    if (!ops_aligned(rows, dtype_size(dtype)) || !ops_aligned(out, dtype_size(out_dtype)) ||
        !ops_aligned(pair_row, 4) || !ops_aligned(weights, 4))
        return MOE_ERR_INVALID_ARG;
    return launch_unpermute(rows, n_rows, pair_row, weights, T, k, D, dtype, out, out_dtype, (cudaStream_t)stream);
}

extern "C" moe_status moe_permute_backward(const void* drows, int n_rows, const int32_t* pair_row, int T, int k, int D,
                                           int dtype, void* dx, moe_stream_t stream) {
    return moe_unpermute(drows, n_rows, pair_row, nullptr, T, k, D, dtype, dx, dtype, stream);
}

extern "C" moe_status moe_unpermute_backward(const void* dout, int out_dtype, const void* rows, int n_rows,
                                             const int32_t* pair_row, const float* weights, int T, int k, int D,
                                             int dtype, void* drows, float* dweights, moe_stream_t stream) {
    moe_status st = ops_shapes(T, k, D);
    if (st != MOE_OK) return st;
    if (n_rows < 0 || !dtype_ok(dtype) || !out_dtype_ok(dtype, out_dtype)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!dout || !pair_row || (!drows && !dweights)) return MOE_ERR_INVALID_ARG;
    if (dweights && n_rows > 0 && !rows) return MOE_ERR_INVALID_ARG;
    if (n_rows > 0 && drows && (drows == rows || drows == dout)) return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_size(dtype);
    if (!ops_aligned(dout, dtype_size(out_dtype)) || !ops_aligned(rows, es) || !ops_aligned(drows, es) ||
        !ops_aligned(pair_row, 4) || !ops_aligned(weights, 4) || !ops_aligned(dweights, 4))
        return MOE_ERR_INVALID_ARG;
    const bool wide = wide_rows(D, es, dout, rows, drows);
    cudaStream_t s = (cudaStream_t)stream;
    return with_dtype(dtype, [&](auto e) {
        using Tp = decltype(e);
        constexpr int V = 16 / sizeof(Tp);
        if (out_dtype == MOE_F32)
            return ops_status(
                wide ? run_unpermute_backward<Tp, float, V>(dout, rows, n_rows, pair_row, weights, T, k, D, drows, dweights, s)
                     : run_unpermute_backward<Tp, float, 1>(dout, rows, n_rows, pair_row, weights, T, k, D, drows, dweights, s));
        return ops_status(
            wide ? run_unpermute_backward<Tp, Tp, V>(dout, rows, n_rows, pair_row, weights, T, k, D, drows, dweights, s)
                 : run_unpermute_backward<Tp, Tp, 1>(dout, rows, n_rows, pair_row, weights, T, k, D, drows, dweights, s));
    });
}
