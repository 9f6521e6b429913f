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
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "once.cuh"
#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 512;          // two experts per thread
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBlocks = 16;            // one cluster (of the size that a kernel has to ask for), where one of
constexpr int kPlanFewBlocks = 8;          // these fits on the device: a partition of one may have room for eight only
constexpr int kPlanHeld = 8;               // rounds of 32 pairs that a warp loads together
constexpr int kSmallPairs = 2816;          // up to here every block makes its part of the plan itself (2,500 pairs of
                                           // 3,072 bf16: 8.6 us against 11.1 us with the plan; 4,000: 15.6 against 11.0)
constexpr int kSmallThreads = 256;
constexpr int kNoExpert = 0x7fffffff;
constexpr int kShiftBytes = 256;           // rows that start anywhere: moved in shifted blocks from this length on,
constexpr int kShiftCopyBytes = 512;       // and copied so from this on
constexpr int kCopyThreads = 256;          // of a block that copies several short tokens
constexpr int kSumThreads = 128;           // of an unpermute block
constexpr int kDotThreads = 256;           // of a block of its gradient
constexpr int kManyPairs = 2048;           // from here on a warp per pair fills the GPU

// The expert of pair p, or kNoExpert if the pair is not taken.
MOE_DEVINL int taken_expert(const int32_t* ids, int p, int E, const int32_t* slot_table, int n_slots) {
    const int e = __ldg(ids + p);
    if (e < 0 || e >= E) return kNoExpert;
    if (slot_table) {
        const int s = __ldg(slot_table + e);
        if (s >= 0 && s < n_slots) return kNoExpert;
    }
    return e;
}

// Inclusive prefix sum over the block's threads (a multiple of 32, at most 1024).
MOE_DEVINL int block_scan(int v, int* wsum) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) wsum[w] = v;
    __syncthreads();
    int s = lane < w && lane < nw ? wsum[lane] : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return v + s;
}

// The plan: a stable counting sort of the P pairs by expert, in one cluster.
// Warp w of block b owns the pairs of segment (b, w), 32 at a time in order.
// Lanes with the same expert find one another by a ballot for each bit of the
// expert's number (with 32 warps per SM a round took 1,430 clocks so and 1,960
// with __match_any_sync); the first of them adds their number to the
// warp's counter of that expert and tells the others what it held, so that every
// pair knows its rank among the warp's pairs of its expert.  An exclusive scan
// over (expert, block, warp) gives the ranks their first row.  A chain of
// latencies bounds it, so the ids of 8 rounds are loaded together, and the ranks
// of the first 8 rounds stay in registers (those of longer segments wait in
// pair_row): one walk does all the matching.  row_pair null: the next kernel
// writes it (scattered words, which few SMs write slowly).  40,960 pairs take 8 us
// alone, 6 us in front of the copies; in a cluster of BLOCKS = 8 11 us.
template <int BLOCKS>
__global__ void __cluster_dims__(BLOCKS, 1, 1) __launch_bounds__(kPlanThreads)
    permute_plan_kernel(const int32_t* __restrict__ ids, int P, int E, const int32_t* __restrict__ slot_table,
                        int n_slots, int32_t* __restrict__ offsets, int32_t* __restrict__ pair_row,
                        int32_t* __restrict__ row_pair) {
    extern __shared__ __align__(8) int32_t count[];     // [warp][Ep]
    __shared__ __align__(8) int block_total[kOpsMaxE];       // of each expert, read by the cluster's other blocks
    __shared__ __align__(8) int first[kOpsMaxE];           // first row of the block's pairs of each expert
    __shared__ int wsum[32];
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, b = (int)cluster.block_rank();
    const int Ep = (E + 1) & ~1, e0 = 2 * threadIdx.x;  // this thread's experts: e0, e0 + 1
    for (int i = threadIdx.x; i < kPlanWarps * Ep / 2; i += kPlanThreads) reinterpret_cast<int2*>(count)[i] = {0, 0};
    pdl_wait();
    pdl_launch_dependents();
    const int rounds = (P + BLOCKS * kPlanThreads - 1) / (BLOCKS * kPlanThreads);
    const int p0 = (b * kPlanWarps + w) * rounds * 32 + lane;
    int32_t* mine = count + w * Ep;
    int key[kPlanHeld], rank[kPlanHeld];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i) {
            const int p = p0 + (i0 + i) * 32;
            key[i] = i0 + i < rounds && p < P ? __ldg(ids + p) : -1;
        }
        if (slot_table) {
            int slot[kPlanHeld];
#pragma unroll
            for (int i = 0; i < kPlanHeld; ++i)
                slot[i] = (uint32_t)key[i] < (uint32_t)E ? __ldg(slot_table + key[i]) : 0;
#pragma unroll
            for (int i = 0; i < kPlanHeld; ++i)
                if (slot[i] >= 0 && slot[i] < n_slots) key[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i)
            if ((uint32_t)key[i] >= (uint32_t)E) key[i] = E;        // no expert
    };
    load(0);
    __syncthreads();
    for (int i0 = 0; i0 < rounds; i0 += kPlanHeld) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i) {
            if (i0 + i >= rounds) break;
            uint32_t peers = 0xffffffffu;
#pragma unroll
            for (int j = 0; j < 11; ++j) {              // of the numbers 0..E, E <= 1024
                if (E >> j == 0) break;
                const bool one = key[i] & (1 << j);
                peers &= __ballot_sync(0xffffffffu, one) ^ (one ? 0u : 0xffffffffu);
            }
            const int leader = __ffs(peers) - 1;
            int held = 0;
            if (lane == leader && key[i] < E) {
                held = mine[key[i]];
                mine[key[i]] = held + __popc(peers);
            }
            rank[i] = __shfl_sync(0xffffffffu, held, leader) + __popc(peers & ((1u << lane) - 1u));
            __syncwarp();                       // the counter is read by another lane next
            const int p = p0 + (i0 + i) * 32;
            if (rounds > kPlanHeld && p < P) pair_row[p] = rank[i];
        }
    }
    __syncthreads();
    // the experts' totals in this block, and their warps' counters as offsets inside it
    if (e0 < E) {
        int2 c[kPlanWarps], sum = {0, 0};
#pragma unroll
        for (int i = 0; i < kPlanWarps; ++i) c[i] = *reinterpret_cast<const int2*>(count + i * Ep + e0);
#pragma unroll
        for (int i = 0; i < kPlanWarps; ++i) {
            *reinterpret_cast<int2*>(count + i * Ep + e0) = sum;
            sum.x += c[i].x, sum.y += c[i].y;
        }
        *reinterpret_cast<int2*>(block_total + e0) = sum;
    }
    cluster.sync();
    int2 total = {0, 0}, before = {0, 0};
    if (e0 < E) {
        int2 c[BLOCKS];
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
            c[i] = *reinterpret_cast<const int2*>(cluster.map_shared_rank(block_total, i) + e0);
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i) {
            total.x += c[i].x, total.y += c[i].y;
            if (i < b) before.x += c[i].x, before.y += c[i].y;
        }
    }
    const int base = block_scan(total.x + total.y, wsum) - total.x - total.y;
    if (e0 < E) {
        *reinterpret_cast<int2*>(first + e0) = {base + before.x, base + total.x + before.y};
        if (b == 0) {
            offsets[e0] = base;
            offsets[e0 + 1] = base + total.x;           // offsets[E], if e0 is the last expert
            if (e0 + 2 == E) offsets[E] = base + total.x + total.y;
        }
    }
    cluster.sync();                             // `first` is there, and no block leaves while another reads its totals
    for (int i0 = 0; i0 < rounds; i0 += kPlanHeld) {
        if (rounds > kPlanHeld) load(i0);
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i) {
            const int p = p0 + (i0 + i) * 32;
            if (i0 + i >= rounds || p >= P) break;
            int row = -1;
            if (key[i] < E) {
                row = first[key[i]] + mine[key[i]] + (rounds > kPlanHeld ? pair_row[p] : rank[i]);
                if (row_pair) row_pair[row] = p;
            }
            pair_row[p] = row;
        }
    }
}

// A small batch in one launch: block t places the pairs of token t itself, by
// counting the pairs that come before each of them (a warp per pair, the pairs'
// experts in shared memory), then copies its token; block T writes the offsets.
template <typename T, int V>
__global__ void __launch_bounds__(kSmallThreads) permute_small_kernel(
    const int32_t* __restrict__ ids, int P, int E, const int32_t* __restrict__ slot_table, int n_slots,
    const T* __restrict__ x, int k, int D, T* __restrict__ rows, int32_t* __restrict__ offsets,
    int32_t* __restrict__ pair_row, int32_t* __restrict__ row_pair) {
    __shared__ __align__(16) int key[kSmallPairs];
    __shared__ int hist[kOpsMaxE];
    __shared__ int32_t row[kMaxTopK];
    __shared__ int wsum[32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, t = blockIdx.x;
    const bool last = t == (int)gridDim.x - 1;
    if (last)
        for (int e = threadIdx.x; e < E; e += kSmallThreads) hist[e] = 0;
    pdl_wait();
    const int P4 = (P + 3) / 4;
    for (int p = threadIdx.x; p < P4 * 4; p += kSmallThreads)
        key[p] = p < P ? taken_expert(ids, p, E, slot_table, n_slots) : kNoExpert;
    __syncthreads();
    if (last) {
        for (int p = threadIdx.x; p < P; p += kSmallThreads)
            if (key[p] != kNoExpert) atomicAdd(hist + key[p], 1);
        __syncthreads();
        constexpr int N = kOpsMaxE / kSmallThreads;
        int c[N], sum = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = threadIdx.x * N + i;
            c[i] = e < E ? hist[e] : 0;
            sum += c[i];
        }
        int at = block_scan(sum, wsum) - sum;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = threadIdx.x * N + i;
            if (e < E) offsets[e] = at;
            at += c[i];
            if (e == E - 1) offsets[E] = at;
        }
        return;
    }
    for (int r = w; r < k; r += kSmallThreads / 32) {
        const int p = t * k + r, e = key[p];
        int n = 0;
        for (int q = lane; q < P4; q += 32) {
            const int4 v = reinterpret_cast<const int4*>(key)[q];
            const int vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) n += vs[j] < e || (vs[j] == e && q * 4 + j < p);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (e == kNoExpert) n = -1;
        if (lane == 0) {
            row[r] = n;
            pair_row[p] = n;
            if (n >= 0) row_pair[n] = p;
        }
    }
    if (!x) return;
    __syncthreads();
    for (int c = threadIdx.x * V; c < D; c += kSmallThreads * V) {
        const Pack<T, V> a = load_pack<T, V>(x + (size_t)t * D + c);
        for (int r = 0; r < k; ++r)
            if (row[r] >= 0) store_pack<T, V>(rows + (size_t)row[r] * D + c, a);
    }
}

// The copies behind the plan, and row_pair: a block per token, or `each` threads
// where rows are SHORT (12,525 tokens x 12 x 32 fp16: 16 us against 22 us; 10,019 x
// 8 x 81 fp32 18 us, in shifted blocks 21 us; x 576 bf16 31 us against 28 us).  The
// first columns of x are read while the plan is still made: its blocks let this
// kernel start once they have waited for the kernels that may have written x.
// 4,096 tokens x 10 x 3,072 bf16: 44 us, 277 MB at 6.3 TB/s.
template <typename T, int V, bool SHORT>
__global__ void __launch_bounds__(512) permute_rows_kernel(const T* __restrict__ x,
                                                           const int32_t* __restrict__ pair_row, int T_, int k, int D,
                                                           int each, T* __restrict__ rows,
                                                           int32_t* __restrict__ row_pair) {
    __shared__ int32_t row[(SHORT ? kCopyThreads / 8 : 1) * kMaxTopK];
    const int tokens = SHORT ? kCopyThreads / each : 1, mine = SHORT ? threadIdx.x / each : 0;
    const int step = SHORT ? each : blockDim.x, rank = SHORT ? threadIdx.x % each : threadIdx.x;
    const int t0 = blockIdx.x * tokens, t = t0 + mine;
    int c = rank * V;
    Pack<T, V> a;
    if ((!SHORT || t < T_) && c < D) a = load_pack_l2<T, V>(x + (size_t)t * D + c);
    pdl_wait();
    if constexpr (SHORT) {
        for (int i = threadIdx.x; i < tokens * k; i += blockDim.x) {
            const int p = t0 * k + i, r = p < T_ * k ? __ldg(pair_row + p) : -1;
            row[i] = r;
            if (r >= 0) row_pair[r] = p;
        }
    } else if (threadIdx.x < k) {
        const int p = t * k + threadIdx.x, r = __ldg(pair_row + p);
        row[threadIdx.x] = r;
        if (r >= 0) row_pair[r] = p;
    }
    __syncthreads();
    if (SHORT && t >= T_) return;
    const int32_t* to = row + mine * k;
    if (c < D)
        for (int r = 0; r < k; ++r)
            if (to[r] >= 0) store_pack<T, V>(rows + (size_t)to[r] * D + c, a);
    for (c += step * V; c < D; c += step * V) {
        a = load_pack<T, V>(x + (size_t)t * D + c);
        for (int r = 0; r < k; ++r)
            if (to[r] >= 0) store_pack<T, V>(rows + (size_t)to[r] * D + c, a);
    }
}

// Rows that start anywhere.  A matrix row's bytes from its first 16-byte boundary
// on are `body` blocks of 16; `head` bytes come before and `tail` bytes after them.
struct Row16 {
    int head, body, tail;
    MOE_DEVINL Row16(const void* row, int bytes) {
        head = (16 - (int)((uintptr_t)row & 15)) & 15;
        body = (bytes - head) / 16;
        tail = bytes - head - 16 * body;
    }
};

// 16 bytes from byte `at` (any) of a buffer in shared memory; at % 16 is the same
// in all lanes.
template <int Q>
MOE_DEVINL uint4 shifted_words(const uint32_t (&w)[8], int bits) {
    return {__funnelshift_r(w[Q], w[Q + 1], bits), __funnelshift_r(w[Q + 1], w[Q + 2], bits),
            __funnelshift_r(w[Q + 2], w[Q + 3], bits), __funnelshift_r(w[Q + 3], w[Q + 4], bits)};
}
MOE_DEVINL uint4 bytes16(const uint4* buf, int at) {
    const uint4 a = buf[at / 16];
    if (at % 16 == 0) return a;
    const uint4 b = buf[at / 16 + 1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int bits = at % 4 * 8;
    switch (at % 16 / 4) {
        case 0: return shifted_words<0>(w, bits);
        case 1: return shifted_words<1>(w, bits);
        case 2: return shifted_words<2>(w, bits);
        default: return shifted_words<3>(w, bits);
    }
}

// Row t of a [T][D] matrix into shared memory by the block: the 16-byte blocks
// that cover it, element by element where one reaches over the matrix's ends.
// Returns the byte of `buf` at which the row starts (0..15).
template <typename T>
MOE_DEVINL int stage_row(const T* m, int t, int T_, int D, uint4* buf) {
    const char *lo = reinterpret_cast<const char*>(m), *hi = lo + (size_t)T_ * D * sizeof(T);
    const char* row = reinterpret_cast<const char*>(m + (size_t)t * D);
    const int lead = (int)((uintptr_t)row & 15), bytes = lead + D * (int)sizeof(T);
    const char* from = row - lead;
    for (int j = threadIdx.x * 16; j < bytes; j += blockDim.x * 16) {
        if (from + j >= lo && from + j + 16 <= hi) {
            buf[j / 16] = __ldcg(reinterpret_cast<const uint4*>(from + j));
        } else {
            for (int q = j; q < j + 16; q += sizeof(T))
                if (from + q >= lo && from + q < hi)
                    store_pack<T, 1>(reinterpret_cast<T*>(reinterpret_cast<char*>(buf) + q),
                                     load_pack_l2<T, 1>(reinterpret_cast<const T*>(from + q)));
        }
    }
    return lead;
}

// The copies of rows that start anywhere: the token goes to shared memory, and
// each of its rows gets whole 16-byte blocks, shifted into place, besides its few
// elements at either end (4,096 x 10 rows of 3,071 bf16: 54 us with the plan
// against 88 us with single elements; of 1,535 fp32 54 us against 69 us).
template <typename T>
__global__ void __launch_bounds__(512) permute_rows_shifted_kernel(const T* __restrict__ x,
                                                                   const int32_t* __restrict__ pair_row, int T_, int k,
                                                                   int D, T* __restrict__ rows,
                                                                   int32_t* __restrict__ row_pair) {
    extern __shared__ __align__(16) uint4 buf[];
    __shared__ int32_t row[kMaxTopK];
    const int t = blockIdx.x, bytes = D * (int)sizeof(T);
    const int lead = stage_row(x, t, T_, D, buf);       // x may be read early: see permute_rows_kernel
    pdl_wait();
    if (threadIdx.x < k) {
        const int p = t * k + threadIdx.x, i = __ldg(pair_row + p);
        row[threadIdx.x] = i;
        if (i >= 0) row_pair[i] = p;
    }
    __syncthreads();
    for (int r = 0; r < k; ++r) {
        if (row[r] < 0) continue;
        char* to = reinterpret_cast<char*>(rows + (size_t)row[r] * D);
        const Row16 at(to, bytes);
        for (int j = threadIdx.x; j < at.body; j += blockDim.x)
            *reinterpret_cast<uint4*>(to + at.head + 16 * j) = bytes16(buf, lead + at.head + 16 * j);
        // elements: threads 0..7 before the body, 8..15 after it
        const int q = threadIdx.x % 8 * (int)sizeof(T) + (threadIdx.x < 8 ? 0 : bytes - at.tail);
        if (threadIdx.x < 16 && q < (threadIdx.x < 8 ? at.head : bytes))
            *reinterpret_cast<T*>(to + q) = *reinterpret_cast<const T*>(reinterpret_cast<const char*>(buf) + lead + q);
    }
}

// out[t] = sum_r w[t,r] rows[row(t,r)], r ascending in fp32 (w NULL: 1).  `each`
// threads take a token, each of them U packs of it, `each` packs apart, and load
// them from all of the token's up to R rows before they add the first; short rows
// put several tokens in a block.  4,096 tokens x 10 x 3,072 bf16: 45 us, 277 MB at
// 6.1 TB/s.  EACH: `each` as a constant where U > 1, so that a thread's packs
// differ by constant offsets (20,011 x 3 x 1,001 fp32: 54 to 55 us, 5.9 TB/s; with
// `each` in a register 72 us).
template <typename T, typename TO, int V, int U, int R, int EACH>
__global__ void __launch_bounds__(kSumThreads) unpermute_kernel(const T* __restrict__ rows, int n_rows,
                                                                const int32_t* __restrict__ pair_row,
                                                                const float* __restrict__ weights, int T_, int k, int D,
                                                                int each_, TO* __restrict__ out) {
    const int each = EACH ? EACH : each_;
    __shared__ int s_row[kSumThreads / 8 * kMaxTopK];
    __shared__ float s_w[kSumThreads / 8 * kMaxTopK];
    pdl_wait();
    const int tokens = blockDim.x / each, t0 = blockIdx.x * tokens, mine = threadIdx.x / each;
    for (int i = threadIdx.x; i < tokens * k; i += blockDim.x) {
        const int p = t0 * k + i;
        int row = -1;
        if (p < T_ * k) {
            row = __ldg(pair_row + p);
            s_w[i] = weights ? __ldg(weights + p) : 1.f;
        }
        s_row[i] = row < n_rows ? row : -1;
    }
    __syncthreads();
    const int t = t0 + mine, c0 = (blockIdx.y * U * each + threadIdx.x % each) * V;
    if (t >= T_) return;
    int row[R];
    Pack<T, V> y[U][R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        row[r] = r < k ? s_row[mine * k + r] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * each * V;
            if (row[r] >= 0 && c < D) y[u][r] = load_pack<T, V>(rows + (size_t)row[r] * D + c);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u) hold(y[u][r]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * each * V;
        if (c >= D) continue;
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row[r] < 0) continue;
            const float w = s_w[mine * k + r];
            float v[V];
            unpack<T, V>(y[u][r], v);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(w, v[i], acc[i]);
        }
        store_f32<TO, V>(out + (size_t)t * D + c, acc);
    }
}

// drows[row(p)] = w[p] dout[t] and dw[p] = <dout[t], rows[row(p)]>: EACH threads
// per pair, U packs in flight per thread.  The pairs of a token read dout[t] after
// one another, so all but the first find it in the caches.  4,096 tokens x 10 x
// 3,072 bf16: 83 us, 528 MB at 6.4 TB/s.
template <typename T, typename TO, int V, int U, int EACH>
__global__ void __launch_bounds__(kDotThreads) unpermute_backward_kernel(const TO* __restrict__ dout,
                                                                         const T* __restrict__ rows, int n_rows,
                                                                         const int32_t* __restrict__ pair_row,
                                                                         const float* __restrict__ weights, int P, int k,
                                                                         int D, T* __restrict__ drows,
                                                                         float* __restrict__ dweights) {
    constexpr int each = EACH;
    __shared__ float part[kDotThreads / 32];
    pdl_wait();
    const int p = blockIdx.x * (kDotThreads / each) + threadIdx.x / each, rank = threadIdx.x % each;
    const int row = p < P ? __ldg(pair_row + p) : -1;
    float dot = 0.f;
    if (row >= 0 && row < n_rows) {
        const float w = weights ? __ldg(weights + p) : 1.f;
        const TO* d = dout + (size_t)(p / k) * D;
        const size_t at = (size_t)row * D;
        for (int c0 = rank * V; c0 < D; c0 += U * each * V) {
            constexpr int H = V * (int)sizeof(TO) > 16 ? 2 : 1, W = V / H;      // dout's accesses per pack
            Pack<T, V> y[U];
            Pack<TO, W> e[U][H];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * each * V;
                if (c < D && dweights) y[u] = load_pack<T, V>(rows + at + c);
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (c < D) e[u][h] = load_pack<TO, W>(d + c + h * W);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                hold(y[u]);
#pragma unroll
                for (int h = 0; h < H; ++h) hold(e[u][h]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + u * each * V >= D) continue;
                float g[V];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float v[W];
                    unpack<TO, W>(e[u][h], v);
#pragma unroll
                    for (int i = 0; i < W; ++i) g[h * W + i] = v[i];
                }
                if (dweights) {
                    float v[V];
                    unpack<T, V>(y[u], v);
#pragma unroll
                    for (int i = 0; i < V; ++i) dot = __fmaf_rn(g[i], v[i], dot);
                }
                if (drows) {
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] *= w;
                    store_f32<T, V>(drows + at + c0 + u * each * V, g);
                }
            }
        }
    }
    if (!dweights) return;
#pragma unroll
    for (int o = (each < 32 ? each : 32) / 2; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if constexpr (each > 32) {
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = dot;
        __syncthreads();
        if (rank == 0)
            for (int i = 1; i < each / 32; ++i) dot += part[threadIdx.x / 32 + i];
    }
    if (rank == 0 && p < P) dweights[p] = dot;
}

// The same for rows that start anywhere, a block per token: dout[t] in shared
// memory, rows and drows (which start alike: their buffers are apart by a multiple
// of 16 bytes) in whole 16-byte blocks, four rows in flight (4,096 x 10 rows of
// 3,071 bf16: 105 us against 168 us with single elements).
template <typename T, typename TO>
__global__ void __launch_bounds__(512) unpermute_backward_shifted_kernel(const TO* __restrict__ dout,
                                                                         const T* __restrict__ rows, int n_rows,
                                                                         const int32_t* __restrict__ pair_row,
                                                                         const float* __restrict__ weights, int T_, int k,
                                                                         int D, T* __restrict__ drows,
                                                                         float* __restrict__ dweights) {
    extern __shared__ __align__(16) uint4 buf[];
    // of every rank: the first block's place in rows and drows, the blocks (0: no row), the first's place in buf
    __shared__ size_t s_at[kMaxTopK];
    __shared__ int s_body[kMaxTopK], s_from[kMaxTopK];
    __shared__ float s_w[kMaxTopK], part[kMaxTopK][16 + 1];
    constexpr int V = 16 / sizeof(T), B = 4, E = sizeof(T), EO = sizeof(TO);
    const int t = blockIdx.x, bytes = D * E, lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const char* from = reinterpret_cast<const char*>(rows);
    char* to = reinterpret_cast<char*>(drows);
    pdl_wait();
    int held = 0;
    const int lead = stage_row(dout, t, T_, D, buf);
    if (threadIdx.x < kMaxTopK) {
        const int p = t * k + threadIdx.x, i = (int)threadIdx.x < k ? __ldg(pair_row + p) : -1;
        held = i >= 0 && i < n_rows;
        const size_t at = (size_t)(i < 0 ? 0 : i) * bytes;
        const Row16 r((dweights ? from : to) + at, bytes);
        s_at[threadIdx.x] = at + r.head;
        s_body[threadIdx.x] = held ? r.body : 0;
        s_from[threadIdx.x] = lead + r.head / E * EO;
        s_w[threadIdx.x] = weights && (int)threadIdx.x < k ? __ldg(weights + p) : 1.f;
    }
    if (!__syncthreads_or(held)) {
        if (dweights && threadIdx.x < k) dweights[(size_t)t * k + threadIdx.x] = 0.f;
        return;
    }
    for (int r0 = 0; r0 < k; r0 += B) {
        float dot[B];
#pragma unroll
        for (int b = 0; b < B; ++b) dot[b] = 0.f;
        for (int j = threadIdx.x; j < bytes / 16; j += blockDim.x) {        // a row's blocks are this many or one less
            uint4 y[B];
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (dweights && j < s_body[r0 + b]) y[b] = *reinterpret_cast<const uint4*>(from + s_at[r0 + b] + 16 * j);
#pragma unroll
            for (int b = 0; b < B; ++b) hold(y[b]);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (j >= s_body[r0 + b]) continue;
                float g[V];                     // the elements of dout that belong to the block
#pragma unroll
                for (int h = 0; h < V * EO / 16; ++h) {
                    constexpr int W = 16 / EO;
                    float v[W];
                    unpack<TO, W>(bytes16(buf, s_from[r0 + b] + j * V * EO + 16 * h), v);
#pragma unroll
                    for (int q = 0; q < W; ++q) g[h * W + q] = v[q];
                }
                if (dweights) {
                    float v[V];
                    unpack<T, V>(y[b], v);
#pragma unroll
                    for (int q = 0; q < V; ++q) dot[b] = __fmaf_rn(g[q], v[q], dot[b]);
                }
                if (drows) {
#pragma unroll
                    for (int q = 0; q < V; ++q) g[q] *= s_w[r0 + b];
                    store_f32<T, V>(reinterpret_cast<T*>(to + s_at[r0 + b] + 16 * j), g);
                }
            }
        }
        if (dweights) {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                dot[b] = warp_sum(dot[b]);
                if (lane == 0) part[r0 + b][w] = dot[b];
            }
        }
    }
    // the elements at the rows' ends, a warp per row: lanes 0..7 before the blocks, 8..15 after them
    for (int r = w; r < k; r += warps) {
        float dot = 0.f;
        if (s_body[r] > 0 && lane < 16) {
            const int head = (s_from[r] - lead) / EO, tail = head + s_body[r] * V;
            const int q = lane < 8 ? lane : tail + lane - 8;
            if (q < (lane < 8 ? head : D)) {
                const size_t at = s_at[r] + (size_t)((q - head) * E);       // head may exceed q: the sum wraps back
                float g[1], v[1];
                load_f32<TO, 1>(reinterpret_cast<const TO*>(reinterpret_cast<const char*>(buf) + lead) + q, g);
                if (dweights) {
                    load_f32<T, 1>(reinterpret_cast<const T*>(from + at), v);
                    dot = g[0] * v[0];
                }
                if (drows) {
                    g[0] *= s_w[r];
                    store_f32<T, 1>(reinterpret_cast<T*>(to + at), g);
                }
            }
        }
        if (dweights) {
            dot = warp_sum(dot);
            if (lane == 0) part[r][16] = dot;
        }
    }
    if (!dweights) return;
    __syncthreads();
    if (threadIdx.x < k) {
        float s = 0.f;
        for (int i = 0; i < warps; ++i) s += part[threadIdx.x][i];
        dweights[(size_t)t * k + threadIdx.x] = s + part[threadIdx.x][16];
    }
}

// The least power of two >= n, in [lo, hi].
inline int threads_for(int n, int lo, int hi) {
    while (lo < n && lo < hi) lo *= 2;
    return lo;
}

// Threads for a row of n packs: whole warps, at most 512, the row's passes equally full.
inline int row_threads(int n) {
    const int passes = (n + 511) / 512;
    return ((n + passes - 1) / passes + 31) / 32 * 32;
}

// Rows whose bytes are a multiple of 16, in 16-byte aligned buffers.
template <typename... P>
inline bool wide_rows(int D, size_t elem, P... p) {
    return (D * elem) % 16 == 0 && (ops_aligned(p, 16) && ...);
}

// Shared memory for a row that starts anywhere, read two blocks at a time.
inline size_t staged_bytes(int D, size_t elem) { return (D * elem + 15) / 16 * 16 + 32; }

template <typename T, typename TO, int V, int U>
cudaError_t run_unpermute(const void* rows, int n_rows, const int32_t* pair_row, const float* weights, int T_, int k,
                          int D, void* out, cudaStream_t s) {
    const int packs = (D + V - 1) / V, need = (packs + U - 1) / U;
    // U == 1, long rows: a token per block, its packs dealt evenly to blocks of at most 128 threads
    const int slices = (need + kSumThreads - 1) / kSumThreads, even = ((need + slices - 1) / slices + 31) / 32 * 32;
    const int each = U > 1 ? (need <= 8 ? 8 : need <= 32 ? 32 : kSumThreads) : need > 64 ? even : threads_for(need, 8, 64);
    const int tokens = kSumThreads / each;
    const dim3 grid((T_ + tokens - 1) / tokens, (packs + U * each - 1) / (U * each));
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(tokens * each), 0, s, static_cast<const T*>(rows), n_rows, pair_row, weights,
                          T_, k, D, each, static_cast<TO*>(out));
    };
    auto by_rank = [&](auto e) {
        constexpr int EACH = decltype(e)::value;
        if (k <= 4) return go(unpermute_kernel<T, TO, V, U, 4, EACH>);
        if (k <= 8) return go(unpermute_kernel<T, TO, V, U, 8, EACH>);
        if (k <= 12) return go(unpermute_kernel<T, TO, V, U, 12, EACH>);
        return go(unpermute_kernel<T, TO, V, U, 16, EACH>);
    };
    if constexpr (U == 1) return by_rank(std::integral_constant<int, 0>{});
    else if (each == 8) return by_rank(std::integral_constant<int, 8>{});
    else if (each == 32) return by_rank(std::integral_constant<int, 32>{});
    else return by_rank(std::integral_constant<int, kSumThreads>{});
}
template <typename T, typename TO, int V, int U>
cudaError_t run_unpermute_backward(const void* dout, const void* rows, int n_rows, const int32_t* pair_row,
                                   const float* weights, int P, int k, int D, void* drows, float* dweights,
                                   cudaStream_t s) {
    if constexpr (V == 1) {
        const bool alike = !drows || !dweights || ((uintptr_t)drows - (uintptr_t)rows) % 16 == 0;
        if (alike && D * (int)sizeof(T) >= kShiftBytes)
            return launch_pdl(unpermute_backward_shifted_kernel<T, TO>, dim3(P / k),
                              dim3(row_threads(D * (int)sizeof(T) / 16)), staged_bytes(D, sizeof(TO)), s,
                              static_cast<const TO*>(dout), static_cast<const T*>(rows), n_rows, pair_row, weights, P / k,
                              k, D, static_cast<T*>(drows), dweights);
    }
    const int need = (D + V * U - 1) / (V * U);
    auto go = [&](auto e) {
        constexpr int EACH = decltype(e)::value;
        return launch_pdl(unpermute_backward_kernel<T, TO, V, U, EACH>,
                          dim3((P + kDotThreads / EACH - 1) / (kDotThreads / EACH)), dim3(kDotThreads), 0, s,
                          static_cast<const TO*>(dout), static_cast<const T*>(rows), n_rows, pair_row, weights, P, k, D,
                          static_cast<T*>(drows), dweights);
    };
    // Threads per pair: as many as its packs ask for, but a warp where the pairs alone fill the GPU (packs of 16 bytes,
    // 6,000 pairs of 3,072 bf16: 16.4 us against 20.9 us with 128 threads; 240 pairs: 8.9 us with 128).  Single
    // elements take all they can get (5,439 pairs of 2,055 fp16: 12.6 us with 256 threads, 18.2 us with 128).
    if (need <= 8) return go(std::integral_constant<int, 8>{});
    if (need <= 32 || (V > 1 && P >= kManyPairs)) return go(std::integral_constant<int, 32>{});
    if (need <= 160) return go(std::integral_constant<int, 128>{});
    return go(std::integral_constant<int, 256>{});
}

moe_status launch_unpermute(const void* rows, int n_rows, const int32_t* pair_row, const float* weights, int T_, int k,
                            int D, int dtype, void* out, int out_dtype, cudaStream_t s) {
    const bool wide = wide_rows(D, dtype_size(dtype), rows, out);
    return with_dtype(dtype, [&](auto e) {
        using T = decltype(e);
        constexpr int V = 16 / sizeof(T);
        if (out_dtype == MOE_F32)
            return ops_status(wide ? run_unpermute<T, float, V, 1>(rows, n_rows, pair_row, weights, T_, k, D, out, s)
                                   : run_unpermute<T, float, 1, 4>(rows, n_rows, pair_row, weights, T_, k, D, out, s));
        return ops_status(wide ? run_unpermute<T, T, V, 1>(rows, n_rows, pair_row, weights, T_, k, D, out, s)
                               : run_unpermute<T, T, 1, 4>(rows, n_rows, pair_row, weights, T_, k, D, out, s));
    });
}

constexpr size_t plan_smem(int E) { return (size_t)kPlanWarps * ((E + 1) / 2 * 2) * 4; }

// The plan kernel's launch attributes on the current device
template <int BLOCKS>
bool plan_ready() {
    static std::atomic<uint64_t> set{0};
    return once_per_device(set, [] {
        return cudaFuncSetAttribute(permute_plan_kernel<BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)plan_smem(kOpsMaxE)) == cudaSuccess &&
               (BLOCKS <= 8 || cudaFuncSetAttribute(permute_plan_kernel<BLOCKS>,
                                                    cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess);
    });
}

// The blocks of the plan on the current device: kPlanBlocks where such a cluster fits at all, looked up once per device.
int plan_blocks() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return kPlanFewBlocks;
    const bool kept = dev >= 0 && dev < 64;
    if (const int n = kept ? known[dev].load(std::memory_order_relaxed) : 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanBlocks);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = plan_smem(kOpsMaxE);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {kPlanBlocks, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (!plan_ready<kPlanBlocks>() ||
        cudaOccupancyMaxActiveClusters(&clusters, permute_plan_kernel<kPlanBlocks>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        clusters = 0;
    }
    const int n = clusters > 0 ? kPlanBlocks : kPlanFewBlocks;
    if (kept) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_plan(const int32_t* ids, int P, int E, const int32_t* slot_table, int n_slots, int32_t* offsets,
                        int32_t* pair_row, int32_t* row_pair, int blocks, cudaStream_t s) {
    if (!(blocks == kPlanBlocks ? plan_ready<kPlanBlocks>() : plan_ready<kPlanFewBlocks>())) return cudaErrorUnknown;
    return launch_pdl(blocks == kPlanBlocks ? permute_plan_kernel<kPlanBlocks> : permute_plan_kernel<kPlanFewBlocks>,
                      dim3(blocks), dim3(kPlanThreads), plan_smem(E), s, ids, P, E, slot_table, n_slots, offsets, pair_row,
                      row_pair);
}

template <typename T>
moe_status launch_permute(const int32_t* ids, int T_, int k, int E, const int32_t* slot_table, int n_slots,
                          const T* x, int D, T* rows, int32_t* offsets, int32_t* pair_row, int32_t* row_pair,
                          cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int P = T_ * k;
    const bool wide = wide_rows(D, sizeof(T), x, rows);
    if (P <= kSmallPairs) {
        auto kernel = wide ? permute_small_kernel<T, V> : permute_small_kernel<T, 1>;
        return ops_status(launch_pdl(kernel, dim3(T_ + 1), dim3(kSmallThreads), 0, s, ids, P, E, slot_table, n_slots, x,
                                     k, D, rows, offsets, pair_row, row_pair));
    }
    const cudaError_t e = launch_plan(ids, P, E, slot_table, n_slots, offsets, pair_row, x ? nullptr : row_pair,
                                      plan_blocks(), s);
    if (e != cudaSuccess || !x) return ops_status(e);
    if (!wide && D * (int)sizeof(T) >= kShiftCopyBytes)
        return ops_status(launch_pdl(permute_rows_shifted_kernel<T>, dim3(T_), dim3(row_threads(D / V)),
                                     staged_bytes(D, sizeof(T)), s, x, (const int32_t*)pair_row, T_, k, D, rows,
                                     row_pair));
    const int packs = wide ? D / V : D;
    const bool few = packs <= (wide ? 64 : 128);
    const int each = few ? threads_for(packs, 8, 64) : row_threads(packs), tokens = few ? kCopyThreads / each : 1;
    auto kernel = wide ? (few ? permute_rows_kernel<T, V, true> : permute_rows_kernel<T, V, false>)
                       : (few ? permute_rows_kernel<T, 1, true> : permute_rows_kernel<T, 1, false>);
    return ops_status(launch_pdl(kernel, dim3((T_ + tokens - 1) / tokens), dim3(tokens * each), 0, s, x,
                                 (const int32_t*)pair_row, T_, k, D, each, rows, row_pair));
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
    return with_dtype(dtype, [&](auto el) {
        using Tp = decltype(el);
        return launch_permute<Tp>(ids, T, k, E, slot_table, n_slots, static_cast<const Tp*>(x), D,
                                  static_cast<Tp*>(rows), offsets, pair_row, row_pair, s);
    });
}

extern "C" moe_status moe_debug_permute_plan(const int32_t* ids, int T, int k, int E, int blocks, int32_t* offsets,
                                             int32_t* pair_row, int32_t* row_pair, moe_stream_t stream) {
    moe_status st = ops_shapes(T, k, 1);
    if (st != MOE_OK) return st;
    if (T == 0 || E <= 0 || (blocks != kPlanBlocks && blocks != kPlanFewBlocks)) return MOE_ERR_INVALID_ARG;
    if (E > kOpsMaxE) return MOE_ERR_UNSUPPORTED;
    if (!ids || !offsets || !pair_row || !row_pair) return MOE_ERR_INVALID_ARG;
    if (!ops_aligned(ids, 4) || !ops_aligned(offsets, 4) || !ops_aligned(pair_row, 4) || !ops_aligned(row_pair, 4))
        return MOE_ERR_INVALID_ARG;
    return ops_status(launch_plan(ids, T * k, E, nullptr, 0, offsets, pair_row, row_pair, blocks, (cudaStream_t)stream));
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
        const int P = T * k;
        if (out_dtype == MOE_F32)
            return ops_status(wide ? run_unpermute_backward<Tp, float, V, 4>(dout, rows, n_rows, pair_row, weights, P, k,
                                                                             D, drows, dweights, s)
                                   : run_unpermute_backward<Tp, float, 1, 8>(dout, rows, n_rows, pair_row, weights, P,
                                                                              k, D, drows, dweights, s));
        return ops_status(wide ? run_unpermute_backward<Tp, Tp, V, 4>(dout, rows, n_rows, pair_row, weights, P, k, D,
                                                                      drows, dweights, s)
                               : run_unpermute_backward<Tp, Tp, 1, 8>(dout, rows, n_rows, pair_row, weights, P, k, D,
                                                                       drows, dweights, s));
    });
}
