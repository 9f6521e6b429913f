// rows.cuh — typed rows for the operators of moe_ops.h: element types, packs of
// elements moved by one load or store, block sums, and the host-side choice of
// pack width.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "moe.h"
#include "moe_ops.h"

namespace moe {

constexpr int kOpsMaxD = 8192;
constexpr int kOpsMaxE = 1024;
constexpr int kOpsMaxT = 65536;

MOE_DEVINL float to_f32(float v) { return v; }
MOE_DEVINL float to_f32(__half v) { return __half2float(v); }
MOE_DEVINL float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
// Round to nearest even, the one rounding between an fp32 result and its store.
template <typename T> MOE_DEVINL T from_f32(float v);
template <> MOE_DEVINL float from_f32<float>(float v) { return v; }
template <> MOE_DEVINL __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> MOE_DEVINL __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V elements moved by one access (16 bytes, or one element: V = 1).
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

template <typename T, int V>
MOE_DEVINL Pack<T, V> load_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
MOE_DEVINL void store_pack(T* p, const Pack<T, V>& a) {
    *reinterpret_cast<Pack<T, V>*>(p) = a;
}
// V fp32 values rounded to T and stored (V * sizeof(T) may be 8, 16 or 32 bytes).
template <typename T, int V>
MOE_DEVINL void store_f32(T* p, const float (&f)[V]) {
    constexpr int W = V * sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        Pack<T, W> a;
#pragma unroll
        for (int j = 0; j < W; ++j) a.v[j] = from_f32<T>(f[i + j]);
        store_pack<T, W>(p + i, a);
    }
}
template <typename T, int V>
MOE_DEVINL void load_f32(const T* p, float (&f)[V]) {
    constexpr int W = V * sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        const Pack<T, W> a = load_pack<T, W>(p + i);
#pragma unroll
        for (int j = 0; j < W; ++j) f[i + j] = to_f32(a.v[j]);
    }
}

MOE_DEVINL float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Host side.
inline bool ops_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool dtype_ok(int d) { return d == MOE_BF16 || d == MOE_F16 || d == MOE_F32; }
inline size_t dtype_size(int d) { return d == MOE_F32 ? 4 : 2; }
inline moe_status ops_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    (void)cudaGetLastError();                   // the status reports it: clear it for the caller's next call
    return MOE_ERR_CUDA;
}
// T, k and D within the limits of moe_ops.h
inline moe_status ops_shapes(int T, int k, int D) {
    if (T < 0 || k <= 0 || D <= 0) return MOE_ERR_INVALID_ARG;
    if (T > kOpsMaxT || k > kMaxTopK || D > kOpsMaxD) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// fn(Elem) with an object of the element type of a moe_dtype
template <typename Fn>
inline moe_status with_dtype(int dtype, Fn&& fn) {
    switch (dtype) {
        case MOE_BF16: return fn(__nv_bfloat16{});
        case MOE_F16: return fn(__half{});
        default: return fn(float{});
    }
}

}  // namespace moe
