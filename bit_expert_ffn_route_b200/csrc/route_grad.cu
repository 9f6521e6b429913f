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

#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

// One block per token: the logits' gradients, then dx.
__global__ void __launch_bounds__(256) route_dx_kernel(const float* __restrict__ dgates,
                                                       const float* __restrict__ gates,
                                                       const int32_t* __restrict__ ids,
                                                       const __nv_bfloat16* __restrict__ Wr, int D, int E, int k,
                                                       const __nv_bfloat16* dx_add, float* __restrict__ dlogits,
                                                       __nv_bfloat16* dx) {
    pdl_wait();
    const size_t t = blockIdx.x;
    float dl[kMaxTopK];
    int id[kMaxTopK];
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxTopK; ++r) {
        id[r] = r < k ? __ldg(ids + t * k + r) : -1;
        const bool in = id[r] >= 0 && id[r] < E;
        if (!in) id[r] = -1;
        dl[r] = in ? __ldg(gates + t * k + r) : 0.f;
        if (in) s = __fmaf_rn(dl[r], __ldg(dgates + t * k + r), s);
    }
#pragma unroll
    for (int r = 0; r < kMaxTopK; ++r) {
        if (id[r] >= 0) dl[r] *= __ldg(dgates + t * k + r) - s;
        if (r < k && threadIdx.x == r) dlogits[t * k + r] = dl[r];
    }
    if (!dx) return;
    for (int c = threadIdx.x * 8; c < D; c += blockDim.x * 8) {
        float acc[8];
        if (dx_add) {
            load_f32<__nv_bfloat16, 8>(dx_add + t * D + c, acc);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < kMaxTopK; ++r) {
            if (id[r] < 0) continue;
            float w[8];
            load_f32<__nv_bfloat16, 8>(Wr + (size_t)id[r] * D + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(dl[r], w[i], acc[i]);
        }
        store_f32<__nv_bfloat16, 8>(dx + t * D + c, acc);
    }
}

// Block (e, columns): dWr of one expert, over its pairs in order.
__global__ void __launch_bounds__(256) route_dw_kernel(const float* __restrict__ dlogits,
                                                       const __nv_bfloat16* __restrict__ x,
                                                       const int32_t* __restrict__ offsets,
                                                       const int32_t* __restrict__ row_pair, int P, int D, int k,
                                                       float* __restrict__ dWr, float* __restrict__ dbias) {
    pdl_wait();
    const int e = blockIdx.x;
    const int r0 = max(0, __ldg(offsets + e)), r1 = min(P, __ldg(offsets + e + 1));
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    float acc[8], b = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int j = r0; j < r1; ++j) {
        const int p = __ldg(row_pair + j);
        if (p < 0 || p >= P) continue;
        const float dl = __ldg(dlogits + p);
        b += dl;
        if (!dWr || c >= D) continue;
        float v[8];
        load_f32<__nv_bfloat16, 8>(x + (size_t)(p / k) * D + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(dl, v[i], acc[i]);
    }
    if (dWr && c < D) store_f32<float, 8>(dWr + (size_t)e * D + c, acc);
    if (dbias && blockIdx.y == 0 && threadIdx.x == 0) dbias[e] = b;
}

moe_status route_grad_shapes(int T, int D, int E, int k) {
    moe_status st = ops_shapes(T, k, D);
    if (st != MOE_OK) return st;
    if (E <= 0) return MOE_ERR_INVALID_ARG;
    if (D % 256 || E > kOpsMaxE || E < k) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t route_grad_ws_bytes(int, int, int, int) { return 256; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_backward_workspace_size(int T, int D, int E, int k) {
    return route_grad_shapes(T, D, E, k) == MOE_OK ? route_grad_ws_bytes(T, D, E, k) : 0;
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
    if (ws_bytes < route_grad_ws_bytes(T, D, E, k)) return MOE_ERR_WORKSPACE;
    using B = __nv_bfloat16;
    cudaError_t e = launch_pdl(route_dx_kernel, dim3(T), dim3(256), 0, s, dgates, gates, ids,
                               reinterpret_cast<const B*>(Wr), D, E, k, reinterpret_cast<const B*>(dx_add), dlogits,
                               reinterpret_cast<B*>(dx));
    if (e != cudaSuccess || (!dWr && !dbias)) return ops_status(e);
    return ops_status(launch_pdl(route_dw_kernel, dim3(E, dWr ? (D + 2047) / 2048 : 1), dim3(256), 0, s,
                                 (const float*)dlogits, reinterpret_cast<const B*>(x), offsets, row_pair, T * k, D, k,
                                 dWr, dbias));
}
