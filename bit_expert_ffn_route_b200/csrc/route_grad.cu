// route_grad.cu — gradient of the router (include/moe_ops.h): from the gates'
// gradient to the selected logits', and from those to x, Wr and the bias.
//
//   dl[t,r] = g (dg - sum_j g_j dg_j),  dx[t] = sum_r dl[t,r] Wr[id],
//   dWr[e] = sum over the pairs of e of dl x[t],  dbias[e] = sum of dl
//
// Only k of E logits of a token have a gradient, so both products run over the
// pairs (2 P D multiply-adds in fp32) and not over all experts, unless these are few
// (route_dense.cuh): as dense products on the tensor cores they would be 51 times the
// work at 512 experts and 10 per token, three times over for dl in three bf16 terms.
// HBM sees little (x, Wr, dx, dWr once each); what bounds the two is reading a row of
// x or Wr per pair, 251 MB each at 40,960 pairs of 3,072, out of L2 or shared memory,
// with its unpacking.
// 4,096 tokens, 512 experts, 10 x 3,072: 54 us in all (logits 3, dx 23, dWr 28,
// join 6, overlapping at their ends).
#include <cuda_runtime.h>
#include <stdint.h>

#include "once.cuh"
#include "route_dense.cuh"
#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

using B16 = __nv_bfloat16;

constexpr int kSlicePairs = 12288;         // pairs from which on dx is made from slices of Wr
constexpr int kSliceThreads = 1024;
constexpr int kSliceTile = 64;             // tokens whose pairs a slice block holds at a time (a pair per thread)
constexpr int kSliceMaxE = 800;            // experts whose 128 columns fit beside the pairs in shared memory; 64 beyond
constexpr int kDwThreads = 128;            // most threads of a dWr block: 8 columns each
constexpr int kDwSmallT = 32;              // tokens whose experts' rows are summed whole (13.2 us of 24 tokens
                                           // against 15.4 us cut and joined; 21.3 us of 100 against 15.4 us)
constexpr int kDwMaxChunk = 3328;          // rows whose places fit in 40 KB of shared memory
constexpr int kDwSums = 320 * 3072;        // partial sums that the dWr chunks make, about
constexpr int kDwDepth = 4;                // rows of x in flight per thread
constexpr int kDenseMinT = 16;             // tokens from which on few experts go to the tensor cores
constexpr int kJoinThreads = 256;
constexpr int kJoinFew = 8;                // chunks per expert, on average, from which on 16 shares join them, not 4

// Eight fp32 sums as four pairs: fma.rn.f32x2 makes two multiply-adds, each
// rounded as fmaf rounds it.
struct Sum8 {
    unsigned long long v[4] = {0, 0, 0, 0};     // +0, +0
    MOE_DEVINL void add(float d, const Pack<B16, 8>& a) {
        unsigned long long m;
        asm("mov.b64 %0, {%1, %1};" : "=l"(m) : "f"(d));
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            unsigned long long x;
            asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(bf16lo(w[i])), "f"(bf16hi(w[i])));
            asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(v[i]) : "l"(m), "l"(x));
        }
    }
    MOE_DEVINL void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("mov.b64 {%0, %1}, %2;" : "=f"(f[2 * i]), "=f"(f[2 * i + 1]) : "l"(v[i]));
    }
    MOE_DEVINL void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("mov.b64 %0, {%1, %2};" : "=l"(v[i]) : "f"(f[2 * i]), "f"(f[2 * i + 1]));
    }
};

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
    pdl_launch_dependents();
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
    Sum8 sum;
    float acc[8];
    if (dx_add && c < D) {
        load_f32<B16, 8>(dx_add + t * D + c, acc);
        sum.set(acc);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float d = __shfl_sync(0xffffffffu, dl, r);
        if (e[r] >= 0 && c < D) sum.add(d, w[r]);
    }
    sum.get(acc);
    if (c < D) store_f32<B16, 8>(dx + t * D + c, acc);
}

// Many tokens: block (slice, group) keeps W = 256 / G columns of all experts'
// rows in shared memory and walks over the group's tokens, 64 at a time.  A warp
// takes a token: G groups of lanes each add up every G-th pair over all W columns
// (16 bytes per lane, S steps), then exchange halves so that a lane ends with
// 8 / G columns.  Shared memory reads each pair's row once, at 128 bytes per
// clock; the instructions (unpacking, two multiply-adds each) are the larger
// part.  The row past the last expert is zero: pairs without expert, and the pairs
// that round k up to S G, point there.
template <int G, int S>
__global__ void __launch_bounds__(kSliceThreads, 1) route_dx_slice_kernel(const float* __restrict__ dlogits,
                                                                          const int32_t* __restrict__ ids,
                                                                          const B16* __restrict__ Wr, int T, int D,
                                                                          int E, int k, const B16* dx_add, B16* dx) {
    extern __shared__ __align__(16) B16 slice[];        // [E + 1][W], then the tile's pairs, twice
    constexpr int W = 256 / G, kCopies = W * 2 / 16, L = 32 / G;
    constexpr int S2 = (S + 1) / 2 * 2, kPairs = G * S2;    // a group's pairs of a token, read two at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * W;
    int2* pairs = reinterpret_cast<int2*>(slice + (size_t)(E + 1) * W);
    // Wr was complete before the kernel in front of this one began
    for (int i = threadIdx.x; i < E * kCopies; i += kSliceThreads) {
        const int e = i / kCopies, j = i % kCopies * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slice + e * W + j)),
                     "l"(Wr + (size_t)e * D + c + j)
                     : "memory");
    }
    for (int i = threadIdx.x; i < W; i += kSliceThreads) slice[E * W + i] = from_f32<B16>(0.f);
    pdl_wait();
    // thread: the pair (token of the tile, rank) that it fetches for every tile
    const int my_tok = threadIdx.x / kPairs, my_r = threadIdx.x % S2 * G + threadIdx.x % kPairs / S2;
    const bool mine = my_tok < kSliceTile, real = mine && threadIdx.x % S2 < S && my_r < k;
    const int step = gridDim.y * kSliceTile;
    auto fetch = [&](int t0) {
        int2 q = {E * W, 0};
        if (real && t0 + my_tok < T) {
            const size_t p = (size_t)(t0 + my_tok) * k + my_r;
            const int e = __ldg(ids + p);
            const float dl = __ldg(dlogits + p);
            if (e >= 0 && e < E) q = {e * W, __float_as_int(dl)};
        }
        return q;
    };
    int2 next = fetch(blockIdx.y * kSliceTile);
    asm volatile("cp.async.wait_all;" ::: "memory");
    int buf = 0;
    for (int t0 = blockIdx.y * kSliceTile; t0 < T; t0 += step, buf ^= 1) {
        int2* tile = pairs + buf * kSliceTile * kMaxTopK;
        if (mine) tile[threadIdx.x] = next;
        __syncthreads();                                // two buffers: the tile before last is done with by all
        next = fetch(t0 + step);
        const B16* col = slice + lane % L * 8;
        for (int i = warp; i < kSliceTile && t0 + i < T; i += kSliceThreads / 32) {
            const int4* q = reinterpret_cast<const int4*>(tile + i * kPairs + lane / L * S2);
            Sum8 sum;
#pragma unroll
            for (int s = 0; s < S; s += 2) {
                const int4 v = q[s / 2];
                sum.add(__int_as_float(v.y), load_pack<B16, 8>(col + v.x));
                if (s + 1 < S) sum.add(__int_as_float(v.w), load_pack<B16, 8>(col + v.z));
            }
            float acc[8];
            sum.get(acc);
            int at = lane % L * 8;
#pragma unroll
            for (int n = 4, bit = 16; n * G >= 8; n /= 2, bit /= 2) {
                const bool up = lane & bit;
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const float give = up ? acc[j] : acc[j + n], keep = up ? acc[j + n] : acc[j];
                    acc[j] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
                }
                at += up ? n : 0;
            }
            float out[8 / G];
            const size_t to = (size_t)(t0 + i) * D + c + at;
#pragma unroll
            for (int j = 0; j < 8 / G; ++j) out[j] = acc[j];
            if (dx_add) {
                float add[8 / G];
                load_f32<B16, 8 / G>(dx_add + to, add);
#pragma unroll
                for (int j = 0; j < 8 / G; ++j) out[j] += add[j];
            }
            store_f32<B16, 8 / G>(dx + to, out);
        }
    }
}

// dWr and dbias of few tokens, in one launch: block (e, 1024 columns) sums over
// all rows of its expert (at most one per token where a token's ids differ).
__global__ void __launch_bounds__(kDwThreads) route_dw_small_kernel(const float* __restrict__ dlogits,
                                                                    const B16* __restrict__ x,
                                                                    const int32_t* __restrict__ offsets,
                                                                    const int32_t* __restrict__ row_pair, int P, int D,
                                                                    int k, float* __restrict__ dWr,
                                                                    float* __restrict__ dbias) {
    pdl_wait();
    const int e = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    const int r0 = max(0, __ldg(offsets + e)), r1 = min(P, __ldg(offsets + e + 1));
    Sum8 sum;
    float b = 0.f;
    for (int j = r0; j < r1; j += kDwDepth) {
        Pack<B16, 8> a[kDwDepth];
        float dl[kDwDepth];
        bool held[kDwDepth];
#pragma unroll
        for (int i = 0; i < kDwDepth; ++i) {
            const int p = j + i < r1 ? __ldg(row_pair + j + i) : -1;
            dl[i] = 0.f;
            held[i] = p >= 0 && p < P;
            if (!held[i]) continue;
            dl[i] = __ldg(dlogits + p);
            if (dWr && c < D) a[i] = load_pack<B16, 8>(x + (size_t)(p / k) * D + c);
        }
#pragma unroll
        for (int i = 0; i < kDwDepth; ++i) {
            b += dl[i];
            if (dWr && c < D && held[i]) {
                hold(a[i]);
                sum.add(dl[i], a[i]);
            }
        }
    }
    if (dWr && c < D) {
        float acc[8];
        sum.get(acc);
        store_f32<float, 8>(dWr + (size_t)e * D + c, acc);
    }
    if (dbias && blockIdx.y == 0 && threadIdx.x == 0) dbias[e] = b;
}

// dWr.  The rows of the plan (the pairs by expert) are cut into chunks of equal
// length whatever the experts' loads are; block (chunk, columns) sums dl x[t]
// over its rows and stores the sum at each change of expert: into dWr where all
// of the expert's rows are in the chunk, otherwise into part[2 chunk] (the
// expert began before the chunk) or part[2 chunk + 1] (it goes on after it).
// The next kernel adds those up in chunk order.  The sums of dl alone go the same
// way, from the first columns' blocks (SUMS false: only these).  A block per expert instead, over
// all its rows, took 1,146 us of the same 40,960 pairs: the largest expert's load.
template <bool SUMS>
__global__ void __launch_bounds__(kDwThreads) route_dw_kernel(const float* __restrict__ dlogits,
                                                              const int32_t* __restrict__ ids,
                                                              const B16* __restrict__ x,
                                                              const int32_t* __restrict__ offsets,
                                                              const int32_t* __restrict__ row_pair, int P, int D, int E,
                                                              int k, int chunk, float* __restrict__ dWr,
                                                              float* __restrict__ part, float* __restrict__ dbias,
                                                              float* __restrict__ bias_part) {
    // of every row: the offset of its token in x, with bit 0 set where an expert begins, and dl
    extern __shared__ uint2 s_row[];
    int* s_exp = reinterpret_cast<int*>(s_row + chunk);
    pdl_wait();
    const int j0 = blockIdx.x * chunk;
    const int n = min(chunk, min(P, __ldg(offsets + E)) - j0);
    for (int j = threadIdx.x; j < min(chunk, P - j0); j += blockDim.x) {
        const int p = __ldg(row_pair + j0 + j);     // anything beyond the plan's rows
        int e = -1;
        float dl = 0.f;
        if (p >= 0 && p < P) {
            e = __ldg(ids + p);
            dl = __ldg(dlogits + p);
        }
        if (e < 0 || e >= E) e = -1;            // not what a plan of these ids holds
        s_exp[j] = e;
        s_row[j] = e >= 0 ? make_uint2((uint32_t)(p / k) * (uint32_t)D, __float_as_uint(dl)) : make_uint2(0u, 0u);
    }
    if (n <= 0) return;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += blockDim.x)
        if (j > 0 && s_exp[j] != s_exp[j - 1]) s_row[j].x |= 1u;
    __syncthreads();
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    if (c >= D) return;
    Sum8 sum;
    const bool first = blockIdx.y == 0 && dbias;
    float b = 0.f;
    auto flush = [&](int e) {
        float acc[8];
        sum.get(acc);
        sum = Sum8();
        const float bias = b;
        b = 0.f;
        if (e < 0) return;
        const bool before = __ldg(offsets + e) < j0, behind = !before && __ldg(offsets + e + 1) > j0 + n;
        const int slot = 2 * blockIdx.x + behind;
        if (SUMS) store_f32<float, 8>((before || behind ? part + (size_t)slot * D : dWr + (size_t)e * D) + c, acc);
        if (first && c == 0) *(before || behind ? bias_part + slot : dbias + e) = bias;
    };
    const B16* xc = x + c;
    int j = 0;
    for (; j + kDwDepth <= n; j += kDwDepth) {
        Pack<B16, 8> a[kDwDepth];
        uint2 row[kDwDepth];
#pragma unroll
        for (int i = 0; i < kDwDepth; ++i) {
            row[i] = s_row[j + i];
            if (SUMS) a[i] = load_pack<B16, 8>(xc + (row[i].x & ~1u));
        }
#pragma unroll
        for (int i = 0; i < kDwDepth; ++i) {
            if (row[i].x & 1u) flush(s_exp[j + i - 1]);
            if (first) b += __uint_as_float(row[i].y);
            if (SUMS) sum.add(__uint_as_float(row[i].y), a[i]);
        }
    }
    for (; j < n; ++j) {
        const uint2 row = s_row[j];
        if (row.x & 1u) flush(s_exp[j - 1]);
        if (first) b += __uint_as_float(row.y);
        if (SUMS) sum.add(__uint_as_float(row.y), load_pack<B16, 8>(xc + (row.x & ~1u)));
    }
    flush(s_exp[n - 1]);
}

// Block (e, columns): the sums of an expert whose rows lie in several chunks (one
// PARTS-th of them per share of the threads, then the shares in order), and a zero row
// for an expert without any; the last block of an expert sums dbias.  Few experts have
// many chunks each: 8,324 x 8 of 51 x 512 in 4 shares, with dbias from the pairs, 28 us
// in all, in 16 shares 22 us.
template <int PARTS>
__global__ void __launch_bounds__(kJoinThreads) route_join_kernel(const int32_t* __restrict__ offsets, int P, int D,
                                                                  int chunk, const float* __restrict__ part,
                                                                  const float* __restrict__ bias_part,
                                                                  float* __restrict__ dWr, float* __restrict__ dbias) {
    constexpr int COLS = kJoinThreads / PARTS * 8;
    __shared__ float sums[PARTS][COLS];
    pdl_wait();
    const int e = blockIdx.x;
    const int r0 = max(0, __ldg(offsets + e)), r1 = min(P, __ldg(offsets + e + 1));
    // partial a is the expert's beginning (odd slot), the others' rows go on from the chunk before
    const int a = r0 / chunk, b = (r1 - 1) / chunk;
    if (r1 > r0 && a == b) return;              // stored by its block
    if (blockIdx.y == gridDim.y - 1) {
        if (!dbias) return;
        float s = 0.f;
        for (int i = a + threadIdx.x; r1 > r0 && i <= b; i += kJoinThreads) s += __ldg(bias_part + 2 * i + (i == a));
        s = warp_sum(s);
        if (threadIdx.x % 32 == 0) sums[0][threadIdx.x / 32] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kJoinThreads / 32; ++i) s += sums[0][i];
            dbias[e] = s;
        }
        return;
    }
    const int g = threadIdx.x / (COLS / 8), col = threadIdx.x % (COLS / 8) * 8;
    const int c = blockIdx.y * COLS;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r1 > r0 && c + col < D) {
        const int each = (b - a + PARTS) / PARTS, i0 = a + g * each, i1 = min(b + 1, i0 + each);
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
            float v[8];
            load_f32<float, 8>(part + (size_t)(2 * i + (i == a)) * D + c + col, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += v[q];
        }
    }
    store_f32<float, 8>(&sums[g][col], acc);
    __syncthreads();
    for (int i = threadIdx.x * 2; i < COLS && c + i < D; i += kJoinThreads * 2) {
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < PARTS; ++j) {
            s[0] += sums[j][i];
            s[1] += sums[j][i + 1];
        }
        store_f32<float, 2>(dWr + (size_t)e * D + c + i, s);
    }
}

// Rows per chunk, a multiple of 16: about kDwSums / D chunks, so that the columns'
// threads of all chunks are as many whatever D is.
int dw_chunk(int P, int D) {
    const int chunks = kDwSums / D, n = (P + chunks - 1) / chunks;
    return n > kDwMaxChunk ? kDwMaxChunk : (n + 15) / 16 * 16;
}

moe_status route_grad_shapes(int T, int D, int E, int k) {
    moe_status st = ops_shapes(T, k, D);
    if (st != MOE_OK) return st;
    if (E <= 0) return MOE_ERR_INVALID_ARG;
    if (D % 256 || E > kOpsMaxE || E < k) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Few experts, or few more of which a token takes five and more: dense products.
// Whole calls, dense against pair by pair: 8,266 x 16 of 19 x 256 13.5 us and 21.5 us,
// 20,000 x 2 of 8 x 1,024 26 and 43, 32 x 8 of 16 x 2,048 5.3 and 12.3; of 32 experts,
// 1,024 x 4,096, 6 per token 15.0 and 16.5, 4 per token 14.7 and 13.5, 3 per token 14.8
// and 12.6; of 64 (an experts' tile twice as wide, by mma.sync as here) 4,096 x 8 x
// 2,048 38 and 34.  The crossing also moves with T and D, which the rule does not look
// at: 4,096 x 4 of 32 x 4,096 would be 35 dense and is 42 by pairs, 16,000 x 2 of 32 x
// 2,048 53 and 60, 4,096 x 4 of 20 x 1,024 14.4 and 16.2; 300 x 1 of 16 x 8,192 is 9.3
// dense and would be 9.0 by pairs.
bool route_dense(int T, int E, int k) { return T >= kDenseMinT && (E <= 16 || (E <= kDenseMaxE && k >= 5)); }

// What T tokens need and fewer: the chunks are no more than the blocks of 16 rows, and than kDwSums / D or what chunks
// of the greatest length leave.  Their own number falls wherever a chunk becomes longer.
size_t dw_part_bytes(int P, int D) {
    int chunks = kDwSums / D;
    if (chunks < (P + kDwMaxChunk - 1) / kDwMaxChunk) chunks = (P + kDwMaxChunk - 1) / kDwMaxChunk;
    if (chunks > (P + 15) / 16) chunks = (P + 15) / 16;
    return (size_t)2 * chunks * (D + 1) * 4;
}
size_t route_grad_ws_bytes(int T, int D, int E, int k) {
    if (!route_dense(T, E, k)) return 256 + dw_part_bytes(T * k, D);
    const size_t dense = dense_part_bytes(T, D, E), few = dw_part_bytes((kDenseMinT - 1) * k, D);
    return 256 + (dense > few ? dense : few);
}

size_t slice_smem(int E, int G) {
    return (size_t)(E + 1) * (256 / G) * 2 + (size_t)2 * kSliceTile * kMaxTopK * sizeof(int2);
}

template <int G, int S>
cudaError_t slice_steps(const float* dlogits, const int32_t* ids, const B16* Wr, int T, int D, int E, int k, int groups,
                        const B16* dx_add, B16* dx, cudaStream_t s) {
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [] {
            return cudaFuncSetAttribute(route_dx_slice_kernel<G, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)slice_smem(G == 2 ? kSliceMaxE : kOpsMaxE, G)) == cudaSuccess;
        }))
        return cudaErrorUnknown;
    return launch_pdl(route_dx_slice_kernel<G, S>, dim3(D / (256 / G), groups), dim3(kSliceThreads), slice_smem(E, G), s,
                      dlogits, ids, Wr, T, D, E, k, dx_add, dx);
}

cudaError_t launch_dx(const float* dgates, const float* gates, const int32_t* ids, const B16* Wr, int T, int D, int E,
                      int k, const B16* dx_add, float* dlogits, B16* dx, cudaStream_t s) {
    // A slice block reads its columns of all E rows once, the direct kernel one row per pair: the slices' reads are
    // `groups` times Wr.  They also take a launch more (whole calls, 512 experts, 10 x 3,072: 600 tokens 17.1 us
    // direct and 18.2 us sliced, 1,200 tokens 25.6 and 25.5, 3,000 tokens 47.8 and 43.8).
    const int G = E <= kSliceMaxE ? 2 : 4, slices = D / (256 / G);
    const int groups = slices < device_sm_count() ? device_sm_count() / slices : 1;
    const bool sliced = dx && T * k >= kSlicePairs && T * k >= 2 * groups * E;
    if (dx && !sliced) {
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3(T, (D + 1023) / 1024), dim3(128), 0, s, dgates, gates, ids, Wr, D, E, k, dx_add,
                              dlogits, dx);
        };
        if (k <= 4) return go(route_dx_kernel<4>);
        if (k <= 8) return go(route_dx_kernel<8>);
        if (k <= 12) return go(route_dx_kernel<12>);
        return go(route_dx_kernel<16>);
    }
    cudaError_t e = launch_pdl(route_dlogits_kernel, dim3((T + 7) / 8), dim3(256), 0, s, dgates, gates, ids, T, E, k,
                               dlogits);
    if (!sliced || e != cudaSuccess) return e;
    if (G == 4) return k <= 4 ? slice_steps<4, 1>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s)
                     : k <= 8 ? slice_steps<4, 2>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s)
                     : k <= 12 ? slice_steps<4, 3>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s)
                               : slice_steps<4, 4>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
    switch ((k + 1) / 2) {
        case 1: return slice_steps<2, 1>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
        case 2: return slice_steps<2, 2>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
        case 3: return slice_steps<2, 3>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
        case 4: return slice_steps<2, 4>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
        case 5: return slice_steps<2, 5>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
        case 6: return slice_steps<2, 6>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
        case 7: return slice_steps<2, 7>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
        default: return slice_steps<2, 8>(dlogits, ids, Wr, T, D, E, k, groups, dx_add, dx, s);
    }
}

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
    const B16 *xb = reinterpret_cast<const B16*>(x), *Wb = reinterpret_cast<const B16*>(Wr);
    if (route_dense(T, E, k)) {
        const DenseArgs a{dgates, gates, ids, dWr ? xb : nullptr, Wb, T, D, E, k, dense_chunk(T, D, E),
                          reinterpret_cast<const B16*>(dx_add), dlogits, reinterpret_cast<B16*>(dx), static_cast<float*>(ws)};
        return ops_status(E <= 16   ? run_route_dense<16>(a, dWr, dbias, s)
                                    : run_route_dense<32>(a, dWr, dbias, s));
    }
    cudaError_t e = launch_dx(dgates, gates, ids, Wb, T, D, E, k, reinterpret_cast<const B16*>(dx_add), dlogits,
                              reinterpret_cast<B16*>(dx), s);
    if (e != cudaSuccess || (!dWr && !dbias)) return ops_status(e);
    if (T <= kDwSmallT)
        return ops_status(launch_pdl(route_dw_small_kernel, dim3(E, dWr ? (D + kDwThreads * 8 - 1) / (kDwThreads * 8) : 1),
                                     dim3(D / 8 < kDwThreads ? D / 8 : kDwThreads), 0, s, (const float*)dlogits, xb, offsets,
                                     row_pair, T * k, D, k, dWr, dbias));
    const int P = T * k, chunk = dw_chunk(P, D), chunks = (P + chunk - 1) / chunk;
    float *part = static_cast<float*>(ws), *bias_part = part + (size_t)2 * chunks * D;
    auto sums = [&](auto kernel, int blocks, int threads) {
        return launch_pdl(kernel, dim3(chunks, blocks), dim3(threads), (size_t)chunk * (sizeof(uint2) + sizeof(int)), s,
                          (const float*)dlogits, ids, xb, offsets, row_pair, P, D, E, k, chunk, dWr, part, dbias, bias_part);
    };
    e = dWr ? sums(route_dw_kernel<true>, (D + kDwThreads * 8 - 1) / (kDwThreads * 8), D / 8 < kDwThreads ? D / 8 : kDwThreads)
            : sums(route_dw_kernel<false>, 1, 32);
    if (e != cudaSuccess) return ops_status(e);
    auto join = [&](auto kernel, int parts) {
        const int cols = kJoinThreads / parts * 8;
        return ops_status(launch_pdl(kernel, dim3(E, (dWr ? (D + cols - 1) / cols : 0) + 1), dim3(kJoinThreads), 0, s, offsets,
                                     P, D, chunk, (const float*)part, (const float*)bias_part, dWr, dbias));
    };
    return chunks >= kJoinFew * E ? join(route_join_kernel<16>, 16) : join(route_join_kernel<4>, 4);
}
