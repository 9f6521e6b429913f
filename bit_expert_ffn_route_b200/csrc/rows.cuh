// rows.cuh — typed rows for the operators of moe_ops.h: element types, packs of
// elements moved by one load or store, warp sums, and the host's checks of types,
// alignment and limits.
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

// Round to nearest even: the one rounding between an fp32 result and its store.
template <typename T> MOE_DEVINL T from_f32(float v);
template <> MOE_DEVINL float from_f32<float>(float v) { return v; }
template <> MOE_DEVINL __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> MOE_DEVINL __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V elements moved by one access: 16 bytes, or one element (V = 1).  Packs of
// 16-bit elements stay packed in 32-bit words until they are used.
template <int BYTES> struct RawOf { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
template <typename T, int V> using Pack = typename RawOf<V * (int)sizeof(T)>::type;

template <typename T, int V>
MOE_DEVINL Pack<T, V> load_pack(const T* p) {
    if constexpr (V * sizeof(T) == 2) return *reinterpret_cast<const uint16_t*>(p);
    else return *reinterpret_cast<const Pack<T, V>*>(p);
}
// Past the L1 cache: for what is read before the kernel's dependency wait.
template <typename T, int V>
MOE_DEVINL Pack<T, V> load_pack_l2(const T* p) {
    if constexpr (V * sizeof(T) == 2) return __ldcg(reinterpret_cast<const unsigned short*>(p));
    else return __ldcg(reinterpret_cast<const Pack<T, V>*>(p));
}
template <typename T, int V>
MOE_DEVINL void store_pack(T* p, const Pack<T, V>& a) {
    if constexpr (V * sizeof(T) == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)a;
    else *reinterpret_cast<Pack<T, V>*>(p) = a;
}

// Between loads under a condition and their use under the same one: without it the
// compiler moves the conversion to fp32 into the load's branch, and each load is
// waited for before the next is issued (unpermute of 4,096 x 10 rows of 3,071
// bf16: 179 us against 68 us; its gradient 130 us against 107 us).
template <typename P>
MOE_DEVINL void hold(P& a) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
    for (int i = 0; i < (int)sizeof(P) / 4; ++i) asm volatile("" : "+r"(w[i]));
}

MOE_DEVINL void unpack_word(float, uint32_t w, float* f) { f[0] = __uint_as_float(w); }
MOE_DEVINL void unpack_word(__half, uint32_t w, float* f) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    f[0] = v.x;
    f[1] = v.y;
}
MOE_DEVINL void unpack_word(__nv_bfloat16, uint32_t w, float* f) {
    f[0] = bf16lo(w);
    f[1] = bf16hi(w);
}
template <typename T, int V>
MOE_DEVINL void unpack(const Pack<T, V>& a, float (&f)[V]) {
    if constexpr (V * sizeof(T) == 2) {
        float g[2];
        unpack_word(T{}, a, g);
        f[0] = g[0];
    } else {
        constexpr int N = V * (int)sizeof(T) / 4, PER = 4 / (int)sizeof(T);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&a);
#pragma unroll
        for (int i = 0; i < N; ++i) unpack_word(T{}, w[i], f + i * PER);
    }
}

MOE_DEVINL uint32_t pack_word(float, const float* f) { return __float_as_uint(f[0]); }
MOE_DEVINL uint32_t pack_word(__half, const float* f) {
    const __half2 h = __floats2half2_rn(f[0], f[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
}
MOE_DEVINL uint32_t pack_word(__nv_bfloat16, const float* f) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// V fp32 values rounded to T and stored, or V elements loaded as fp32, in
// accesses of at most 16 bytes (V fp32 values for V elements of 2 bytes are 32).
template <typename T, int V>
MOE_DEVINL void store_f32(T* p, const float (&f)[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(f[0]);
    } else {
        constexpr int W = V * sizeof(T) > 16 ? 16 / (int)sizeof(T) : V, PER = 4 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < V; i += W) {
            Pack<T, W> a;
            uint32_t* w = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
            for (int j = 0; j < W / PER; ++j) w[j] = pack_word(T{}, f + i + j * PER);
            store_pack<T, W>(p + i, a);
        }
    }
}
template <typename T, int V>
MOE_DEVINL void load_f32(const T* p, float (&f)[V]) {
    constexpr int W = V * sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        float g[W];
        unpack<T, W>(load_pack<T, W>(p + i), g);
#pragma unroll
        for (int j = 0; j < W; ++j) f[i + j] = g[j];
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
