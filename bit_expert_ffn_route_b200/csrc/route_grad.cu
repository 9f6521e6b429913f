// route_grad.cu — gradient of the router (include/moe_ops.h): from the gates'
// gradient to the selected logits', and from those to x, Wr and the bias.
//
//   dl[t,r] = g (dg - sum_j g_j dg_j),  dx[t] = sum_r dl[t,r] Wr[id],
//   dWr[e] = sum over the pairs of e of dl x[t],  dbias[e] = sum of dl
//
// Only k of E logits of a token have a gradient, so both products run over the
// pairs (2 P D multiply-adds) and not over all experts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "once.cuh"
#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

using B16 = __nv_bfloat16;

constexpr int kSliceThreads = 1024;
constexpr int kSliceSmem = 200 * 1024;     // a slice of Wr: all experts, 128 columns (64 beyond 800 experts)
constexpr int kDwThreads = 128;            // columns of dWr per block: 8 per thread
constexpr int kDwChunks = 1280;            // chunks of pairs that the dWr sums are cut into, about
constexpr int kDwDepth = 8;                // rows of x in flight per thread
constexpr int kDwMaxChunk = 1024;

// Lane r < k: the gradient of the token's r-th selected logit, and its expert
// (-1: id outside [0, E), gradient 0).
MOE_DEVINL float token_dlogit(const float* dgates, const float* gates, const int32_t* ids, size_t t, int k, int E,
                              int lane, int& id) {
    id = -1;
    float g = 0.f, dg = 0.f;
    if (lane < k) {
        id = __ldg(ids + t * k + lane);
        g = __ldg(gates + t * k + lane);
        dg = __ldg(dgates + t * k + lane);
        if (id < 0 || id >= E) id = -1, g = dg = 0.f;
    }
    return g * (dg - warp_sum(g * dg));
}

// The logits' gradients alone: a warp per token.
__global__ void __launch_bounds__(256) route_dlogits_kernel(const float* __restrict__ dgates,
                                                            const float* __restrict__ gates,
                                                            const int32_t* __restrict__ ids, int T, int E, int k,
                                                            float* __restrict__ dlogits) {
    pdl_wait();
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= T) return;
    int id;
    const float dl = token_dlogit(dgates, gates, ids, t, k, E, lane, id);
    if (lane < k) dlogits[(size_t)t * k + lane] = dl;
}

// Few tokens: a block per token and 1024 columns, the rows of Wr straight from L2.
template <int R>
__global__ void __launch_bounds__(128) route_dx_kernel(const float* __restrict__ dgates,
                                                       const float* __restrict__ gates,
                                                       const int32_t* __restrict__ ids, const B16* __restrict__ Wr,
                                                       int D, int E, int k, const B16* dx_add,
                                                       float* __restrict__ dlogits, B16* dx) {
    pdl_wait();
    const size_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, c = (blockIdx.y * 128 + threadIdx.x) * 8;
    int id;
    const float dl = token_dlogit(dgates, gates, ids, t, k, E, lane, id);
    if (blockIdx.y == 0 && threadIdx.x < k) dlogits[t * k + threadIdx.x] = dl;
    Pack<B16, 8> w[R];
    int e[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        e[r] = __shfl_sync(0xffffffffu, id, r);
        if (e[r] >= 0 && c < D) w[r] = load_pack<B16, 8>(Wr + (size_t)e[r] * D + c);
    }
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (dx_add && c < D) load_f32<B16, 8>(dx_add + t * D + c, acc);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float d = __shfl_sync(0xffffffffu, dl, r);
        if (e[r] < 0 || c >= D) continue;
        float v[8];
        unpack<B16, 8>(w[r], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(d, v[i], acc[i]);
    }
    if (c < D) store_f32<B16, 8>(dx + t * D + c, acc);
}

// Many tokens: block (slice, group) keeps 32 N columns of all experts' rows in
// shared memory and its warps walk over the group's tokens, one row of the
// slice per pair.
template <int N>
__global__ void __launch_bounds__(kSliceThreads) route_dx_slice_kernel(const float* __restrict__ dgates,
                                                                       const float* __restrict__ gates,
                                                                       const int32_t* __restrict__ ids,
                                                                       const B16* __restrict__ Wr, int T, int D, int E,
                                                                       int k, const B16* dx_add,
                                                                       float* __restrict__ dlogits, B16* dx) {
    extern __shared__ __align__(16) B16 slice[];        // [E][32 N]
    constexpr int W = 32 * N, kCopies = W * 2 / 16;     // 16-byte copies per expert
    const int lane = threadIdx.x & 31, c = blockIdx.x * W;
    pdl_wait();
    for (int i = threadIdx.x; i < E * kCopies; i += kSliceThreads) {
        const int e = i / kCopies, j = i % kCopies * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slice + e * W + j)),
                     "l"(Wr + (size_t)e * D + c + j)
                     : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const int step = gridDim.y * (kSliceThreads / 32);
    for (int t = blockIdx.y * (kSliceThreads / 32) + (threadIdx.x >> 5); t < T; t += step) {
        int id;
        const float dl = token_dlogit(dgates, gates, ids, t, k, E, lane, id);
        if (blockIdx.x == 0 && lane < k) dlogits[(size_t)t * k + lane] = dl;
        const size_t at = (size_t)t * D + c + lane * N;
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        if (dx_add) load_f32<B16, N>(dx_add + at, acc);
#pragma unroll 4
        for (int r = 0; r < k; ++r) {
            const int e = __shfl_sync(0xffffffffu, id, r);
            const float d = __shfl_sync(0xffffffffu, dl, r);
            if (e < 0) continue;
            float v[N];
            load_f32<B16, N>(slice + e * W + lane * N, v);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = __fmaf_rn(d, v[i], acc[i]);
        }
        store_f32<B16, N>(dx + at, acc);
    }
}

// dWr.  The rows of the plan (the pairs by expert) are cut into chunks of equal
// length whatever the experts' loads are; block (chunk, columns) sums dl x[t]
// over its rows and stores the sum at each change of expert: into dWr where all
// of the expert's rows are in the chunk, otherwise into part[2 chunk] (the
// expert began before the chunk) or part[2 chunk + 1] (it goes on after it).
// The next kernel adds those up in chunk order.
__global__ void __launch_bounds__(kDwThreads) route_dw_kernel(const float* __restrict__ dlogits,
                                                              const int32_t* __restrict__ ids,
                                                              const B16* __restrict__ x,
                                                              const int32_t* __restrict__ offsets,
                                                              const int32_t* __restrict__ row_pair, int P, int D, int E,
                                                              int k, int chunk, float* __restrict__ dWr,
                                                              float* __restrict__ part) {
    __shared__ int s_tok[kDwMaxChunk], s_exp[kDwMaxChunk];
    __shared__ float s_dl[kDwMaxChunk];
    pdl_wait();
    const int j0 = blockIdx.x * chunk;
    const int n = min(chunk, min(P, __ldg(offsets + E)) - j0);
    if (n <= 0) return;
    for (int j = threadIdx.x; j < n; j += kDwThreads) {
        const int p = __ldg(row_pair + j0 + j);
        int e = -1;
        if (p >= 0 && p < P) e = __ldg(ids + p);
        if (e < 0 || e >= E) e = -1;            // not what a plan of these ids holds
        s_exp[j] = e;
        s_tok[j] = e >= 0 ? p / k : 0;
        s_dl[j] = e >= 0 ? __ldg(dlogits + p) : 0.f;
    }
    __syncthreads();
    const int c = (blockIdx.y * kDwThreads + threadIdx.x) * 8;
    if (c >= D) return;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto flush = [&](int e) {
        if (e < 0) return;
        float* to = dWr + (size_t)e * D;
        if (__ldg(offsets + e) < j0) to = part + (size_t)(2 * blockIdx.x) * D;
        else if (__ldg(offsets + e + 1) > j0 + n) to = part + (size_t)(2 * blockIdx.x + 1) * D;
        store_f32<float, 8>(to + c, acc);
    };
    int cur = s_exp[0];
    for (int j = 0; j < n; j += kDwDepth) {
        Pack<B16, 8> a[kDwDepth];
#pragma unroll
        for (int i = 0; i < kDwDepth; ++i)
            if (j + i < n) a[i] = load_pack<B16, 8>(x + (size_t)s_tok[j + i] * D + c);
#pragma unroll
        for (int i = 0; i < kDwDepth; ++i) {
            if (j + i >= n) break;
            if (s_exp[j + i] != cur) {
                flush(cur);
                cur = s_exp[j + i];
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = 0.f;
            }
            const float dl = s_dl[j + i];
            float v[8];
            unpack<B16, 8>(a[i], v);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] = __fmaf_rn(dl, v[q], acc[q]);
        }
    }
    flush(cur);
}

// Block (e, columns): the sums of an expert whose rows lie in several chunks, a
// zero row for an expert without any, and dbias.
__global__ void __launch_bounds__(kDwThreads) route_join_kernel(const float* __restrict__ dlogits,
                                                                const int32_t* __restrict__ offsets,
                                                                const int32_t* __restrict__ row_pair, int P, int D,
                                                                int chunk, const float* __restrict__ part,
                                                                float* __restrict__ dWr, float* __restrict__ dbias) {
    __shared__ float wsum[kDwThreads / 32];
    pdl_wait();
    const int e = blockIdx.x;
    const int r0 = max(0, __ldg(offsets + e)), r1 = min(P, __ldg(offsets + e + 1));
    if (dbias && blockIdx.y == 0) {
        float s = 0.f;
        for (int j = r0 + threadIdx.x; j < r1; j += kDwThreads) {
            const int p = __ldg(row_pair + j);
            if (p >= 0 && p < P) s += __ldg(dlogits + p);
        }
        s = warp_sum(s);
        if ((threadIdx.x & 31) == 0) wsum[threadIdx.x >> 5] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kDwThreads / 32; ++i) s += wsum[i];
            dbias[e] = s;
        }
    }
    const int c = (blockIdx.y * kDwThreads + threadIdx.x) * 8;
    if (!dWr || c >= D) return;
    const int a = r0 / chunk, b = (r1 - 1) / chunk;
    if (r1 > r0 && a == b) return;              // stored by its block
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r1 > r0) {
        load_f32<float, 8>(part + (size_t)(2 * a + 1) * D + c, acc);
#pragma unroll 4
        for (int i = a + 1; i <= b; ++i) {
            float v[8];
            load_f32<float, 8>(part + (size_t)(2 * i) * D + c, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += v[q];
        }
    }
    store_f32<float, 8>(dWr + (size_t)e * D + c, acc);
}

// Rows per chunk: a multiple of 16.
int dw_chunk(int P) {
    const int n = (P + kDwChunks - 1) / kDwChunks;
    return (n + 15) / 16 * 16;
}

moe_status route_grad_shapes(int T, int D, int E, int k) {
    moe_status st = ops_shapes(T, k, D);
    if (st != MOE_OK) return st;
    if (E <= 0) return MOE_ERR_INVALID_ARG;
    if (D % 256 || E > kOpsMaxE || E < k) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t route_grad_ws_bytes(int T, int D, int k) {
    const int P = T * k, chunk = P ? dw_chunk(P) : 16;
    return 256 + (size_t)2 * ((P + chunk - 1) / chunk) * D * 4;
}

cudaError_t launch_dx(const float* dgates, const float* gates, const int32_t* ids, const B16* Wr, int T, int D, int E,
                      int k, const B16* dx_add, float* dlogits, B16* dx, cudaStream_t s) {
    if (!dx) return launch_pdl(route_dlogits_kernel, dim3((T + 7) / 8), dim3(256), 0, s, dgates, gates, ids, T, E, k, dlogits);
    // A slice block reads its columns of all E rows once, the direct kernel one row per pair: the slices' reads are
    // `groups` times Wr.
    const int N = E * 256 <= kSliceSmem ? 4 : 2, slices = D / (32 * N);
    const int groups = slices < device_sm_count() ? device_sm_count() / slices : 1;
    if ((long long)T * k < 2ll * groups * E) {
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3(T, (D + 1023) / 1024), dim3(128), 0, s, dgates, gates, ids, Wr, D, E, k, dx_add,
                              dlogits, dx);
        };
        if (k <= 4) return go(route_dx_kernel<4>);
        if (k <= 8) return go(route_dx_kernel<8>);
        if (k <= 12) return go(route_dx_kernel<12>);
        return go(route_dx_kernel<16>);
    }
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [] {
            return cudaFuncSetAttribute(route_dx_slice_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kSliceSmem) == cudaSuccess &&
                   cudaFuncSetAttribute(route_dx_slice_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kSliceSmem) == cudaSuccess;
        }))
        return cudaErrorUnknown;
    auto kernel = N == 4 ? route_dx_slice_kernel<4> : route_dx_slice_kernel<2>;
    return launch_pdl(kernel, dim3(slices, groups), dim3(kSliceThreads), (size_t)E * 64 * N, s, dgates, gates, ids, Wr, T,
                      D, E, k, dx_add, dlogits, dx);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_backward_workspace_size(int T, int D, int E, int k) {
    return route_grad_shapes(T, D, E, k) == MOE_OK ? route_grad_ws_bytes(T, D, k) : 0;
}

extern "C" moe_status moe_route_backward(const float* dgates, const float* gates, const int32_t* ids,
                                         const uint16_t* x, const uint16_t* Wr, const int32_t* offsets,
                                         const int32_t* row_pair, int T, int D, int E, int k, const uint16_t* dx_add,
                                         float* dlogits, uint16_t* dx, float* dWr, float* dbias, void* ws,
                                         size_t ws_bytes, moe_stream_t stream) {
    moe_status st = route_grad_shapes(T, D, E, k);
    if (st != MOE_OK) return st;
    if (!ops_aligned(x, 16) || !ops_aligned(Wr, 16) || !ops_aligned(dx_add, 16) || !ops_aligned(dx, 16) ||
        !ops_aligned(dWr, 16) || !ops_aligned(dbias, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        if (dWr && cudaMemsetAsync(dWr, 0, (size_t)E * D * 4, s) != cudaSuccess) return ops_status(cudaErrorUnknown);
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)E * 4, s) != cudaSuccess) return ops_status(cudaErrorUnknown);
        return MOE_OK;
    }
    if (!dgates || !gates || !ids || !dlogits || !ws || !ops_aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    if (!ops_aligned(dgates, 4) || !ops_aligned(gates, 4) || !ops_aligned(ids, 4) || !ops_aligned(dlogits, 4) ||
        !ops_aligned(offsets, 4) || !ops_aligned(row_pair, 4))
        return MOE_ERR_INVALID_ARG;
    if ((dx && !Wr) || (dx_add && !dx) || (dWr && !x) || ((dWr || dbias) && (!offsets || !row_pair)))
        return MOE_ERR_INVALID_ARG;
    if (dx && (dx == x || dx == Wr)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < route_grad_ws_bytes(T, D, k)) return MOE_ERR_WORKSPACE;
    const B16 *xb = reinterpret_cast<const B16*>(x), *Wb = reinterpret_cast<const B16*>(Wr);
    cudaError_t e = launch_dx(dgates, gates, ids, Wb, T, D, E, k, reinterpret_cast<const B16*>(dx_add), dlogits,
                              reinterpret_cast<B16*>(dx), s);
    if (e != cudaSuccess || (!dWr && !dbias)) return ops_status(e);
    const int P = T * k, chunk = dw_chunk(P), cols = dWr ? (D + kDwThreads * 8 - 1) / (kDwThreads * 8) : 1;
    float* part = static_cast<float*>(ws);
    if (dWr)
        e = launch_pdl(route_dw_kernel, dim3((P + chunk - 1) / chunk, cols), dim3(kDwThreads), 0, s,
                       (const float*)dlogits, ids, xb, offsets, row_pair, P, D, E, k, chunk, dWr, part);
    if (e != cudaSuccess) return ops_status(e);
    return ops_status(launch_pdl(route_join_kernel, dim3(E, cols), dim3(kDwThreads), 0, s, (const float*)dlogits,
                                 offsets, row_pair, P, D, chunk, (const float*)part, dWr, dbias));
}
