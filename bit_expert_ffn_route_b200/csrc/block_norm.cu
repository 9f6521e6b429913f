// block_norm.cu — the norms between one block and the next (include/moe_ops.h).
//
//   z = y r_y w_post,  x_out = alpha residual + gate z,  normed = x_out r_x w_next,
//   r = rsqrt(mean(v^2) + eps)
// Each element of y and the residual is read once and each of x_out and normed
// written once; a token stays in registers between the two norms.  Gradients
// likewise: four rows in, two out.  HBM is the floor of both; what bounds them is
// the chain of a token's steps (rows out of shared memory, a sum over the block's
// warps, the rest) with as many warps as the registers leave.  4,096 tokens of
// 3,072 bf16: 19 us forward (100 MB, 5.3 TB/s) and 36 us backward (151 MB, 4.2
// TB/s; 31 us of it the tokens, the rest the join of the partial sums).
//
// Threads: a group of whole warps takes a token, each thread the same columns of
// every token it takes, so that the sums over tokens stay in its registers; short
// rows put several groups in a block.  Groups walk over the tokens and fetch the
// rows of their next tokens with cp.async while they work (loads at the start of
// a block per token: 26 and 71 us).
// Rows of whole 16-byte packs: a thread copies just what it will read itself, so
// no barrier guards the copies.  Other rows start anywhere: the 16-byte blocks
// that cover the row are copied (elements where such a block reaches over the
// buffer's ends), and read back an element at a time, or a pair, behind a barrier.
#include <cuda_runtime.h>
#include <stdint.h>

#include "once.cuh"
#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

constexpr int kNormParts = 148;        // most blocks of the backward pass, one per SM: each leaves a partial of every
                                       // sum over tokens
constexpr int kJoinEach = (kNormParts + 7) / 8;     // of which a warp of the join adds up so many
constexpr int kNormThreads = 384;      // threads that the groups of a block fill, about
constexpr int kGradThreads = 768;      // and of the backward pass: one block per SM, half the partials of blocks of
                                       // 384, and three tokens where D is 2,048 (59 us, with 384 71 us, of 12,288 bf16)
constexpr int kMaxDynamic = 227 * 1024;

template <int N>
MOE_DEVINL void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
MOE_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
MOE_DEVINL void cp_async16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// Elementwise on N (even) fp32 values, two per instruction; each product and
// multiply-add rounds as the scalar instruction does.
#define MOE_F32X2(OP, D0, D1, A0, A1, B0, B1)                                                                     \
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t" OP                             \
        " a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"                                                                  \
        : "=f"(D0), "=f"(D1)                                                                                      \
        : "f"(A0), "f"(A1), "f"(B0), "f"(B1))
template <int N>
MOE_DEVINL void mul(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) MOE_F32X2("mul.rn.f32x2", d[i], d[i + 1], a[i], a[i + 1], b[i], b[i + 1]);
}
template <int N>
MOE_DEVINL void mul(float (&d)[N], const float (&a)[N], float b) {
#pragma unroll
    for (int i = 0; i < N; i += 2) MOE_F32X2("mul.rn.f32x2", d[i], d[i + 1], a[i], a[i + 1], b, b);
}
MOE_DEVINL void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
// d = a b + c
template <int N>
MOE_DEVINL void fma(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) fma2(d[i], d[i + 1], a[i], a[i + 1], b[i], b[i + 1], c[i], c[i + 1]);
}
template <int N>
MOE_DEVINL void fma(float (&d)[N], const float (&a)[N], float b, const float (&c)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) fma2(d[i], d[i + 1], a[i], a[i + 1], b, b, c[i], c[i + 1]);
}
// sum of a b over the N values
template <int N>
MOE_DEVINL float dot(const float (&a)[N], const float (&b)[N]) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) fma2(s0, s1, a[i], a[i + 1], b[i], b[i + 1], s0, s1);
    return s0 + s1;
}

// v as it reads back after a store as T
template <typename T, int N>
MOE_DEVINL void round_stored(float (&v)[N]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < N; i += 2) unpack_word(T{}, pack_word(T{}, v + i), v + i);
    }
}

// A group's threads, and sums over them: the same bits in every thread, formed
// in a fixed order (lanes, then warps).  buf: [2][4][32] floats of this group;
// parity alternates from call to call, so one barrier per call is enough.
struct Group {
    int g, rank, size;                          // group in the block, thread in the group, threads per group
    float* buf;
    int parity = 0;
    MOE_DEVINL void sync() const {
        if (size == 32) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(size) : "memory");
    }
    MOE_DEVINL float sum(float v) {
        const int lane = threadIdx.x & 31;
        v = warp_sum(v);
        if (size == 32) return v;
        float* b = buf + (parity ^= 128);
        if (lane == 0) b[rank / 32] = v;
        sync();
        return warp_sum(lane < size / 32 ? b[lane] : 0.f);
    }
    // Three sums at once: lanes hand halves over, so that after two steps a lane
    // is left with one of the three (or zero).
    MOE_DEVINL void sum3(float& v0, float& v1, float& v2) {
        const int lane = threadIdx.x & 31;
        const bool hi = lane & 16, odd = lane & 8;
        const float k0 = (hi ? v2 : v0) + __shfl_xor_sync(0xffffffffu, hi ? v0 : v2, 16);
        const float k1 = (hi ? 0.f : v1) + __shfl_xor_sync(0xffffffffu, hi ? v1 : 0.f, 16);
        float v = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 8);
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (size > 32) {                        // lane 8 i holds sum 0, 1, 2, -, of this warp
            float* b = buf + (parity ^= 128);
            if (lane % 8 == 0) b[rank / 32 * 4 + lane / 8] = v;
            sync();
            v = 0.f;
#pragma unroll
            for (int w = 0; w < 32; w += 8)
                if (w * 32 < size && lane % 8 + w < size / 32) v += b[(lane % 8 + w) * 4 + lane / 8];
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        v0 = __shfl_sync(0xffffffffu, v, 0);
        v1 = __shfl_sync(0xffffffffu, v, 8);
        v2 = __shfl_sync(0xffffffffu, v, 16);
    }
};
constexpr int kSumFloats = 256;

// How rows lie: they start anywhere (ANY), they are of whole PAIRS of 16-bit
// elements (13,519 x 2,482 fp16 forward 72 us, 92 us as single elements; 6,000 x
// 6,002 bf16 backward 147 against 221) or of whole 16-byte packs (WIDE), or besides
// every thread of the group has all its columns and the call has every operand but
// a token gate (FULL: no test of these in the token's path; 4,096 x 3,072 bf16
// forward 19.1 us against 21.7 us, backward 36 against 47; 12,288 x 2,048 backward 58
// against 75).  Other sets of operands are WIDE: a pre-norm step (residual and next
// norm alone) 18.1 us forward, 40 backward, a token gate 21.4 and 46.
enum { ANY, PAIRS, WIDE, FULL };

// Thread `rank` of a group of `size` owns N elements of a row: packs of V, at
// (i size + rank) V (V = 1: single elements of rows that start anywhere).
template <typename T, int N, int KIND>
struct Cols {
    static constexpr int V = KIND == ANY     ? 1
                             : KIND == PAIRS ? 2
                             : N < 16 / (int)sizeof(T) ? N : 16 / (int)sizeof(T),
                         ITER = N / V;
    int rank, size, D;
    MOE_DEVINL int at(int i) const { return (i * size + rank) * V; }
    MOE_DEVINL bool in(int i) const { return KIND == FULL || at(i) < D; }
    // Elements outside the row are zero.
    template <typename S>
    MOE_DEVINL void load(const S* p, float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            float w[V];
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = 0.f;
            if (in(i)) load_f32<S, V>(p + at(i), w);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i * V + j] = w[j];
        }
    }
    template <typename S>
    MOE_DEVINL void store(S* p, const float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            float w[V];
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = v[i * V + j];
            if (in(i)) store_f32<S, V>(p + at(i), w);
        }
    }
};

// The rows of a group's coming tokens, STAGES tokens ahead in shared memory, out
// of the ROWS matrices a.rows (null: not there).  Offsets into the [T][D]
// matrices are bytes in 32 bits (at most 2^31).
template <typename T, int N, int ROWS, int STAGES, int KIND, typename Args>
struct Ring {
    const Args& a;
    const Cols<T, N, KIND>& col;
    char* ring;                                 // [STAGES][ROWS][pitch] of this group
    int slot = 0;                               // offset in the ring of the token to read next, then to fetch into
    // bytes from the row's place in its slot to its first element
    MOE_DEVINL int lead(int r, uint32_t at) const {
        return KIND >= WIDE ? 0 : (int)(((uint32_t)(uintptr_t)a.rows[r] + at) & 15);
    }
    // Fetch the token at offset `at`, if there is one.
    MOE_DEVINL void fetch(uint32_t at, bool live) {
        if (live) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (KIND != FULL && !a.rows[r]) continue;
                const char* src = static_cast<const char*>(a.rows[r]);
                char* to = ring + slot + r * a.pitch;
                if constexpr (KIND >= WIDE) {
#pragma unroll
                    for (int i = 0; i < Cols<T, N, KIND>::ITER; ++i)
                        if (col.in(i))
                            cp_async16(to + col.at(i) * sizeof(T), src + (at + col.at(i) * (uint32_t)sizeof(T)));
                } else {
                    const uint32_t row_bytes = a.D * (uint32_t)sizeof(T);
                    const char *lo = src, *hi = lo + (size_t)a.T * row_bytes;           // the buffer
                    const char* from = src + at - lead(r, at);
                    const int bytes = lead(r, at) + (int)row_bytes;
                    for (int j = col.rank * 16; j < bytes; j += a.group * 16) {
                        if (from + j >= lo && from + j + 16 <= hi) {
                            cp_async16(to + j, from + j);
                        } else {
                            for (int q = j; q < j + 16; q += sizeof(T))
                                if (from + q >= lo && from + q < hi)
                                    *reinterpret_cast<T*>(to + q) = *reinterpret_cast<const T*>(from + q);
                        }
                    }
                }
            }
        }
        cp_async_commit();
        slot = slot == (STAGES - 1) * ROWS * a.pitch ? 0 : slot + ROWS * a.pitch;
    }
    MOE_DEVINL void wait(const Group& grp) const {
        cp_async_wait<STAGES - 1>();
        if (KIND < WIDE) grp.sync();
    }
    MOE_DEVINL void read(int r, uint32_t at, float (&v)[N]) const {
        col.load(reinterpret_cast<const T*>(ring + slot + r * a.pitch + lead(r, at)), v);
    }
};

// A thread's factors of its columns: w_post times a channel gate, and w_next
// (1 where absent).  Kept in shared memory, a thread's N values in packs of four
// that neighbouring threads hold next to one another (in registers the backward
// pass spilled: 44 us against 40).
template <int N>
struct Factors {
    float4* at;                                 // [2][N / 4][threads per token]
    int rank, size;
    template <typename Col, typename Args>
    MOE_DEVINL void make(const Col& col, const Args& a, bool write) {
        float v[N], w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = 1.f;
        if (a.w_post) col.load(a.w_post, v);
        if (a.gate_mode == MOE_GATE_CHANNEL) {
            col.load(a.gate, w);
            mul(v, v, w);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = 1.f;
        if (a.w_next) col.load(a.w_next, w);
        if (!write) return;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            at[j / 4 * size + rank] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            at[(N / 4 + j / 4) * size + rank] = make_float4(w[j], w[j + 1], w[j + 2], w[j + 3]);
        }
    }
    MOE_DEVINL void get(int n, float (&v)[N]) const {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 q = at[(n * (N / 4) + j / 4) * size + rank];
            v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
        }
    }
};

template <typename T>
MOE_DEVINL T* at_bytes(void* p, uint32_t at) { return reinterpret_cast<T*>(static_cast<char*>(p) + at); }

struct NormArgs {
    const void* rows[2];                        // y, residual or null
    const float* gate;
    int gate_mode;
    float alpha;
    const float *w_post, *w_next;
    float eps;
    int T, D, group, pitch;                     // group: threads per token; pitch: bytes of a row's slot
    void *x_out, *normed;
    float *rstd_post, *rstd_next;
};

template <typename T, int N, int STAGES, int THREADS, int KIND>
__global__ void __launch_bounds__(THREADS, THREADS == kNormThreads ? 3 : 1)
    block_norm_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) float dyn[];        // the groups' sums, the factors, the groups' rings
    const int groups = blockDim.x / a.group, g = threadIdx.x / a.group, rank = threadIdx.x % a.group;
    const int step = gridDim.x * groups, t0 = blockIdx.x * groups + g;
    Group grp{g, rank, a.group, dyn + g * kSumFloats};
    const Cols<T, N, KIND> col{rank, a.group, a.D};
    char* rings = reinterpret_cast<char*>(dyn + groups * kSumFloats + 2 * N * a.group);
    Ring<T, N, 2, STAGES, KIND, NormArgs> in{a, col, rings + g * STAGES * 2 * a.pitch};
    const uint32_t skip = step * a.D * (uint32_t)sizeof(T);
    uint32_t at = t0 * a.D * (uint32_t)sizeof(T);       // the token's offset in every matrix
    pdl_wait();
#pragma unroll
    for (int i = 0; i < STAGES; ++i) in.fetch(at + i * skip, t0 + i * step < a.T);
    Factors<N> fac{reinterpret_cast<float4*>(dyn + groups * kSumFloats), rank, a.group};
    fac.make(col, a, g == 0);
    __syncthreads();
    const float inv = 1.f / a.D;
    const bool per_token = KIND != FULL && a.gate_mode == MOE_GATE_TOKEN;
    const bool post = KIND == FULL || a.w_post, next = KIND == FULL || a.w_next;
    float gt = per_token && t0 < a.T ? __ldg(a.gate + t0) : 1.f;    // loaded a token ahead
    for (int t = t0; t < a.T; t += step) {
        float v[N], r[N];
        float f = gt;
        if (per_token && t + step < a.T) gt = __ldg(a.gate + t + step);
        in.wait(grp);
        in.read(0, at, v);
        if (KIND == FULL || a.rows[1]) {
            in.read(1, at, r);
            mul(r, r, a.alpha);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) r[j] = 0.f;
        }
        if (post) {
            const float ry = rsqrtf(__fmaf_rn(grp.sum(dot(v, v)), inv, a.eps));
            if (a.rstd_post && rank == 0) a.rstd_post[t] = ry;
            f *= ry;
        }
        float w[N];
        fac.get(0, w);
        mul(v, v, w);
        fma(v, v, f, r);
        round_stored<T>(v);
        if (KIND == FULL || a.x_out) col.store(at_bytes<T>(a.x_out, at), v);
        if (next) {
            const float rx = rsqrtf(__fmaf_rn(grp.sum(dot(v, v)), inv, a.eps));
            if (a.rstd_next && rank == 0) a.rstd_next[t] = rx;
            fac.get(1, w);
            mul(v, v, w);
            mul(v, v, rx);
            col.store(at_bytes<T>(a.normed, at), v);
        } else if (KIND < WIDE) {
            grp.sync();                         // all of the group have read the token
        }
        if (KIND < WIDE && a.group == 32) __syncwarp();     // the sums above had no barrier
        in.fetch(at + STAGES * skip, t + STAGES * step < a.T);
        at += skip;
    }
}

struct NormGradArgs {
    const void* rows[4];                        // x_out, dnormed (null without w_next), dx_out or null, y (null: not read)
    const float* gate;
    int gate_mode;
    float alpha;
    const float *w_post, *rstd_post, *w_next, *rstd_next;
    int T, D, group, pitch;
    void *dy, *dresidual;
    float* dgate;                               // of a token gate
    bool want_next, want_post;                  // the sums over tokens that part gets
    float* part;                                // [gridDim.x][2][D]: of dnormed xh, of G yh (times a token gate)
};

// With q = yh w_post gate and G = b - r c1 xh, b = dx_out + r u, c1 = mean(xh u),
// the second mean's sum is  sum(q G) = sum(q b) - r c1 sum(q xh):  all three sums
// of a token are formed at once, with one barrier.  A token gate stays outside
// of q: sum(q G) is then its gradient.  A channel gate and w_post are the same
// for all tokens, so both their gradients come from the sums of G yh.
template <typename T, int N, int STAGES, int THREADS, int KIND>
__global__ void __launch_bounds__(THREADS, 1)
    block_norm_backward_kernel(const __grid_constant__ NormGradArgs a) {
    extern __shared__ __align__(16) float dyn[];        // the groups' sums, the factors, the groups' rings
    const int groups = blockDim.x / a.group, g = threadIdx.x / a.group, rank = threadIdx.x % a.group;
    const int step = gridDim.x * groups, t0 = blockIdx.x * groups + g;
    Group grp{g, rank, a.group, dyn + g * kSumFloats};
    const Cols<T, N, KIND> col{rank, a.group, a.D};
    char* rings = reinterpret_cast<char*>(dyn + groups * kSumFloats + 2 * N * a.group);
    Ring<T, N, 4, STAGES, KIND, NormGradArgs> in{a, col, rings + g * STAGES * 4 * a.pitch};
    const uint32_t skip = step * a.D * (uint32_t)sizeof(T);
    uint32_t at = t0 * a.D * (uint32_t)sizeof(T);
    float s_next[N], s_gy[N];                   // the sums over tokens
#pragma unroll
    for (int j = 0; j < N; ++j) s_next[j] = s_gy[j] = 0.f;
    pdl_wait();
#pragma unroll
    for (int i = 0; i < STAGES; ++i) in.fetch(at + i * skip, t0 + i * step < a.T);
    Factors<N> fac{reinterpret_cast<float4*>(dyn + groups * kSumFloats), rank, a.group};
    fac.make(col, a, g == 0);
    __syncthreads();
    const float inv = 1.f / a.D;
    const bool next = KIND == FULL || a.w_next, post = KIND == FULL || a.w_post;
    const bool per_token = KIND != FULL && a.gate_mode == MOE_GATE_TOKEN;
    float rx_next = 0.f, ry_next = 1.f, gt_next = 1.f;  // loaded a token ahead
    auto scalars = [&](int t) {
        if (t >= a.T) return;
        if (next) rx_next = __ldg(a.rstd_next + t);
        if (post) ry_next = __ldg(a.rstd_post + t);
        if (per_token) gt_next = __ldg(a.gate + t);
    };
    scalars(t0);
    for (int t = t0; t < a.T; t += step) {
        const float rx = rx_next, ry = ry_next, gt = gt_next;
        scalars(t + step);
        float b[N], xh[N], yh[N], m[N], w[N];
        float s0 = 0.f, s1 = 0.f, s2 = 0.f;     // sums of xh u, q b, q xh
        in.wait(grp);
#pragma unroll
        for (int j = 0; j < N; ++j) b[j] = xh[j] = yh[j] = 0.f;
        if (KIND == FULL || a.rows[2]) in.read(2, at, b);
        if (next) {
            in.read(0, at, xh);
            in.read(1, at, m);
            mul(xh, xh, rx);
            fma(s_next, m, xh, s_next);
            fac.get(1, w);
            mul(m, m, w);                       // u
            s0 = dot(xh, m);
            fma(b, m, rx, b);
        }
        if (KIND == FULL || a.rows[3]) {
            in.read(3, at, yh);
            mul(yh, yh, ry);
            fac.get(0, w);
            mul(m, yh, w);                      // q
            s1 = dot(m, b);
            s2 = dot(m, xh);
        }
        grp.sum3(s0, s1, s2);
        if (KIND < WIDE && a.group == 32) __syncwarp();     // the sums had no barrier
        in.fetch(at + STAGES * skip, t + STAGES * step < a.T);  // all of the group have read the token
        const float rc1 = rx * s0 * inv, sq = __fmaf_rn(-rc1, s2, s1);
        const float c2 = post ? gt * sq * inv : 0.f;
        if (KIND != FULL && a.dgate && rank == 0) a.dgate[t] = sq;
        fma(b, xh, -rc1, b);                    // G
        if (KIND == FULL || a.dresidual) {
            mul(m, b, a.alpha);
            col.store(at_bytes<T>(a.dresidual, at), m);
        }
        if (per_token) mul(b, b, gt);
        fma(s_gy, b, yh, s_gy);
        fac.get(0, w);
        mul(b, b, w);
        if (post) fma(b, yh, -c2, b);
        mul(b, b, ry);
        col.store(at_bytes<T>(a.dy, at), b);
        at += skip;
    }
    // The block's sums: those of its groups added in order.
    float* part = a.part + (size_t)blockIdx.x * 2 * a.D;
    if (groups == 1) {
        if (a.want_next) col.store(part, s_next);
        if (a.want_post) col.store(part + a.D, s_gy);
    } else {
        const int pitch = STAGES * 4 * a.pitch / 4;     // floats from ring to ring: 2 D and more
        __syncthreads();                        // the rings are read out
        float* mine = reinterpret_cast<float*>(rings) + g * pitch;
        if (a.want_next) col.store(mine, s_next);
        if (a.want_post) col.store(mine + a.D, s_gy);
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
            if (!(i < a.D ? a.want_next : a.want_post)) continue;
            float v = 0.f;
            for (int q = 0; q < groups; ++q) v += reinterpret_cast<const float*>(rings)[q * pitch + i];
            part[i] = v;
        }
    }
}

// Column sums of the blocks' partials: 32 columns per block, an eighth of the
// partials per warp, the eighths added in order.
__global__ void __launch_bounds__(256) block_norm_join_kernel(const float* __restrict__ part, int n, int D,
                                                              const float* w_post, const float* gate, float* dw_next,
                                                              float* dw_post, float* dgate) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const bool next = blockIdx.y == 0;
    pdl_wait();
    if (next ? !dw_next : !dw_post && !dgate) return;
    const int each = (n + 7) / 8, i0 = w * each, i1 = c < D ? min(n, i0 + each) : 0;
    float v[kJoinEach], s = 0.f;                // all loads in flight: one round trip (8 at a time: 2 us more)
#pragma unroll
    for (int i = 0; i < kJoinEach; ++i)
        v[i] = i0 + i < i1 ? __ldg(part + ((size_t)(i0 + i) * 2 + blockIdx.y) * D + c) : 0.f;
#pragma unroll
    for (int i = 0; i < kJoinEach; ++i) s += v[i];
    sums[w][lane] = s;
    __syncthreads();
    if (w > 0 || c >= D) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][lane];
    if (next) {
        dw_next[c] = s;
    } else {
        if (dw_post) dw_post[c] = gate ? s * __ldg(gate + c) : s;
        if (dgate) dgate[c] = w_post ? s * __ldg(w_post + c) : s;
    }
}

// Threads per token, tokens per block and bytes of a row's slot.
struct NormShape {
    int group, groups, pitch;
    NormShape(int D, int per_thread, size_t elem, bool wide, int threads) {
        group = ((D + per_thread - 1) / per_thread + 31) / 32 * 32;
        groups = group >= threads ? 1 : threads / group;
        pitch = (int)((D * elem + 15) / 16 * 16) + (wide ? 0 : 16);
    }
    int blocks(int T, int most) const {
        const int n = (T + groups - 1) / groups;
        return n < most ? n : most;
    }
};

template <typename T, int N, int STAGES, int THREADS, int KIND>
cudaError_t run_norm(NormArgs a, cudaStream_t s) {
    auto kernel = block_norm_kernel<T, N, STAGES, THREADS, KIND>;
    const NormShape n(a.D, N, sizeof(T), KIND >= WIDE, kNormThreads);
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic) ==
                   cudaSuccess;
        }))
        return cudaErrorUnknown;
    a.group = n.group;
    a.pitch = n.pitch;
    const int per_sm = THREADS > 512 ? 1 : THREADS == kNormThreads ? 3 : 2;
    return launch_pdl(kernel, dim3(n.blocks(a.T, device_sm_count() * per_sm)), dim3(n.group * n.groups),
                      (size_t)n.groups * (kSumFloats * 4 + STAGES * 2 * n.pitch) + (size_t)n.group * N * 8, s, a);
}
template <typename T, int N, int STAGES, int THREADS, int KIND>
cudaError_t run_norm_backward(NormGradArgs a, int* blocks, cudaStream_t s) {
    auto kernel = block_norm_backward_kernel<T, N, STAGES, THREADS, KIND>;
    const NormShape n(a.D, N, sizeof(T), KIND >= WIDE, THREADS);
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic) ==
                   cudaSuccess;
        }))
        return cudaErrorUnknown;
    a.group = n.group;
    a.pitch = n.pitch;
    *blocks = n.blocks(a.T, device_sm_count() < kNormParts ? device_sm_count() : kNormParts);
    return launch_pdl(kernel, dim3(*blocks), dim3(n.group * n.groups),
                      (size_t)n.groups * (kSumFloats * 4 + STAGES * 4 * n.pitch) + (size_t)n.group * N * 8, s, a);
}

// A thread has 16 bytes of a row (twice that for fp32 rows beyond 4,096).  Forward
// blocks of 384 threads leave room for three per SM; 768 threads of the backward
// pass, two tokens or more, for the sums over tokens in registers.  Those of rows
// beyond 4,096 elements need 16 elements per thread and 512 threads (3,072 x 8,192
// bf16 62 us; 8 elements with the sums in shared memory 81 us).
template <typename T, int KIND>
cudaError_t pick_norm(const NormArgs& a, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    if (a.D <= kNormThreads * N) return run_norm<T, N, 3, kNormThreads, KIND>(a, s);
    if (a.D <= 512 * N) return run_norm<T, N, 3, 512, KIND>(a, s);
    if constexpr (N == 4) {
        if (a.D > 1024 * N) return run_norm<T, 8, 2, 1024, KIND>(a, s);
    }
    return run_norm<T, N, 3, 1024, KIND>(a, s);
}
template <typename T, int KIND>
cudaError_t pick_norm_backward(const NormGradArgs& a, int* blocks, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    if (a.D <= kGradThreads / 2 * N) return run_norm_backward<T, N, 3, kGradThreads, KIND>(a, blocks, s);
    if (a.D <= 512 * N) return run_norm_backward<T, N, 3, 512, KIND>(a, blocks, s);
    if constexpr (N == 4) {
        if (a.D <= 1024 * N) return run_norm_backward<T, N, 2, 1024, KIND>(a, blocks, s);
    }
    if constexpr (KIND == FULL) return cudaErrorInvalidValue;           // not beyond 4096: see whole_groups
    else return run_norm_backward<T, 16, N / 4, 512, KIND>(a, blocks, s);
}

// Whether every thread of the groups has all its columns: D a multiple of 32 N,
// with the N that the D takes above.  Not for the widest rows' gradient: its
// registers spill in that form (3,072 x 8,192 bf16 73 us against 62 us).
bool whole_groups(int D, size_t elem, bool grad) {
    return !(grad && D > 4096) && D % (elem == 4 && D <= 4096 ? 128 : 256) == 0;
}

moe_status norm_shapes(int T, int D) { return ops_shapes(T, 1, D); }

bool gate_ok(const float* gate, int mode) {
    if (mode == MOE_GATE_NONE) return !gate;
    return (mode == MOE_GATE_CHANNEL || mode == MOE_GATE_TOKEN) && gate && ops_aligned(gate, 4);
}

// |v| < infinity, and not NaN
bool finite(float v) { return v - v == 0.f; }

size_t norm_ws_bytes(int T, int D) { return (size_t)(T < kNormParts ? T : kNormParts) * 2 * D * 4 + 256; }

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
    // rows of whole units of n bytes, in buffers that start with one; fp32 arrays likewise
    auto units = [&](size_t n, size_t fp32) {
        return (D * es) % n == 0 && ops_aligned(y, n) && ops_aligned(residual, n) && ops_aligned(x_out, n) &&
               ops_aligned(normed, n) && ops_aligned(w_post, fp32) && ops_aligned(w_next, fp32) &&
               (gate_mode != MOE_GATE_CHANNEL || ops_aligned(gate, fp32));
    };
    const bool wide = units(16, 16), pairs = units(4, 8);
    const bool full =
        wide && whole_groups(D, es, false) && residual && w_post && w_next && x_out && gate_mode != MOE_GATE_TOKEN;
    const NormArgs a{{y, residual}, gate, gate_mode, alpha, w_post, w_next,   eps,
                     T,             D,    0,         0,     x_out,  normed,   rstd_post, rstd_next};
    cudaStream_t s = (cudaStream_t)stream;
    return with_dtype(dtype, [&](auto e) {
        using Tp = decltype(e);
        if constexpr (sizeof(Tp) == 2)
            if (!wide && pairs) return ops_status(pick_norm<Tp, PAIRS>(a, s));
        return ops_status(full   ? pick_norm<Tp, FULL>(a, s)
                          : wide ? pick_norm<Tp, WIDE>(a, s)
                                 : pick_norm<Tp, ANY>(a, s));
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
    auto units = [&](size_t n, size_t fp32) {   // as in the forward pass
        return (D * es) % n == 0 && ops_aligned(dx_out, n) && ops_aligned(dnormed, n) && ops_aligned(x_out, n) &&
               ops_aligned(y, n) && ops_aligned(dy, n) && ops_aligned(dresidual, n) && ops_aligned(w_post, fp32) &&
               ops_aligned(w_next, fp32) && (gate_mode != MOE_GATE_CHANNEL || ops_aligned(gate, fp32));
    };
    const bool wide = units(16, 16), pairs = units(4, 8);
    const bool per_token = gate_mode == MOE_GATE_TOKEN;
    const bool full = wide && whole_groups(D, es, true) && dx_out && w_post && w_next && dresidual && !per_token;
    const NormGradArgs a{{w_next ? x_out : nullptr, w_next ? dnormed : nullptr, dx_out, w_post || dgate ? y : nullptr},
                         gate, gate_mode, alpha, w_post, rstd_post, w_next, rstd_next, T, D, 0, 0, dy, dresidual,
                         per_token ? dgate : nullptr, dw_next != nullptr, dw_post || dgate_cols,
                         static_cast<float*>(ws)};
    int blocks = 0;
    st = with_dtype(dtype, [&](auto e) {
        using Tp = decltype(e);
        if constexpr (sizeof(Tp) == 2)
            if (!wide && pairs) return ops_status(pick_norm_backward<Tp, PAIRS>(a, &blocks, s));
        return ops_status(full   ? pick_norm_backward<Tp, FULL>(a, &blocks, s)
                          : wide ? pick_norm_backward<Tp, WIDE>(a, &blocks, s)
                                 : pick_norm_backward<Tp, ANY>(a, &blocks, s));
    });
    if (st != MOE_OK || (!dw_next && !dw_post && !dgate_cols)) return st;
    return ops_status(launch_pdl(block_norm_join_kernel, dim3((D + 31) / 32, 2), dim3(256), 0, s, (const float*)ws,
                                 blocks, D, w_post, per_token ? nullptr : gate, dw_next, dw_post, dgate_cols));
}
