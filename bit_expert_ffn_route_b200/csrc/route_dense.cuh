// route_dense.cuh — the router's gradient of few experts as dense products on the
// tensor cores (see route_grad.cu for the formulas):
//   dx = dl Wr  ([T, E] x [E, D]),  dWr = dl^T x  ([E, T] x [T, D])
// with dl zero where an expert is not selected.  Of few experts that costs less than
// a row of x and of Wr per pair: a block reads its tokens' columns of x once for all
// of them and keeps its columns of Wr in registers.  HBM is the floor (x and dx once);
// what bounds the kernel is the chain of a tile's steps (the tile's dl, then products
// of three terms one behind the other) with 16 to 24 warps per SM: 20,000 tokens x 2
// of 8 experts x 1,024 26 us in all, 82 MB at 3.2 TB/s.
//
// dl stays exact: it is cut into three bf16 terms of 8 bits each (h + m + l = dl; below
// 2^-110 bits of l fall under bf16's smallest number, 2^-133), products of bf16 are
// exact in fp32, sums are fp32.  Zero times an infinity or NaN
// would reach experts and tokens that were not paired, so columns of Wr and tiles of x
// that hold one are added up pair by pair instead.
#pragma once

#include "rows.cuh"
#include "sync.cuh"

namespace moe {
namespace {

constexpr int kDenseMaxE = 32;
constexpr int kDenseTok = 32;              // tokens of a tile
constexpr int kDenseStages = 3;            // tiles of x, two of them on their way
constexpr int kDenseThreads = 256;
constexpr int kDenseCols = 256;            // columns of a block, 32 per warp
constexpr int kDenseBlocks = 296;          // blocks of a wave, two per SM;
constexpr int kDenseBlocks16 = 444;        // three where the tile has 16 experts

template <int EP>
struct DenseTile {
    static constexpr int TOK = kDenseTok, MINE = TOK / (kDenseThreads / 32);    // tokens a warp makes the dl of
    static constexpr int XP = kDenseCols + 8, AP = EP + 8;      // eight rows lie in different banks
    __nv_bfloat16 x[kDenseStages][TOK][XP];
    uint16_t a[2][3][TOK][AP];                          // h, m, l of dl
    uint32_t mask[2][TOK];                              // the token's experts
    int2 pair[TOK][kMaxTopK];                           // expert (-1: none), dl
};

MOE_DEVINL void ldsm4(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
MOE_DEVINL void ldsm4t(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
MOE_DEVINL void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
MOE_DEVINL float high16(uint32_t bits) { return __uint_as_float(bits << 16); }
// Whether a bf16 of the two is infinite or NaN
MOE_DEVINL bool not_finite(uint32_t two) {
    return (two & 0x7f80u) == 0x7f80u || (two & 0x7f800000u) == 0x7f800000u;
}

// v = h + m + l, each the first 8 bits of what is left of v (an infinity or NaN: h alone)
MOE_DEVINL void cut3(float v, uint16_t (&q)[3]) {
    const uint32_t u = __float_as_uint(v);
    q[0] = (uint16_t)(u >> 16);
    q[1] = q[2] = 0;
    if ((u & 0x7f800000u) == 0x7f800000u) {
        if (u & 0x7fffffu) q[0] |= 0x40;
        return;
    }
    const float r = v - high16(q[0]);
    q[1] = (uint16_t)(__float_as_uint(r) >> 16);
    q[2] = (uint16_t)(__float_as_uint(r - high16(q[1])) >> 16);
}

MOE_DEVINL float whole(uint16_t h, uint16_t m, uint16_t l) { return high16(h) + (high16(m) + high16(l)); }

struct DenseArgs {
    const float *dgates, *gates;
    const int32_t* ids;
    const __nv_bfloat16 *x, *Wr;                // x null: no dWr; Wr null: no dx
    int T, D, E, k, chunk;                      // chunk: tokens of a block, whole tiles
    const __nv_bfloat16* dx_add;
    float* dlogits;
    __nv_bfloat16* dx;
    float* part;                                // [chunks][E D + E]: dWr, then dbias
};
MOE_DEVINL size_t dense_stride(int D, int E) { return (size_t)E * D + (E + 3) / 4 * 4; }

// Block (256 columns, chunk).  A warp has 32 columns for both products, and makes the
// dl of TOK / 8 tokens of the next tile behind those of this one.
template <int EP>
__global__ void __launch_bounds__(kDenseThreads, EP == 16 ? 3 : 2) route_dense_kernel(const __grid_constant__ DenseArgs a) {
    using Tile = DenseTile<EP>;
    constexpr int TOK = Tile::TOK, MINE = Tile::MINE, K = EP / 16;
    extern __shared__ __align__(16) char smem[];
    Tile& s = *reinterpret_cast<Tile*>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q4 = lane & 3;
    const int c0 = blockIdx.x * kDenseCols, cw = c0 + warp * 32;
    const int t0 = blockIdx.y * a.chunk, t1 = min(a.T, t0 + a.chunk);
    pdl_wait();

    // The warp's four tokens of the tile at t, eight lanes each: lane r has ranks r and r + 8 ...
    int id[2];
    float gv[2], dv[2];
    auto load_pairs = [&](int t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = lane % 8 + 8 * j, tok = t + warp * MINE + lane / 8;
            id[j] = -1;
            gv[j] = dv[j] = 0.f;
            if (r >= a.k || tok >= t1) continue;
            const int p = tok * a.k + r;
            id[j] = __ldg(a.ids + p);
            gv[j] = __ldg(a.gates + p);
            dv[j] = __ldg(a.dgates + p);
            if (id[j] < 0 || id[j] >= a.E) id[j] = -1, gv[j] = dv[j] = 0.f;
        }
    };
    // ... and their dl into buffer `buf`: a lane takes an expert, and adds up the token's pairs that name it (a token
    // may name one twice).
    constexpr int AT_ONCE = 32 / EP;
    float bias = 0.f;
    auto make_dl = [&](int t, int buf) {
        float sum = gv[0] * dv[0] + gv[1] * dv[1];
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncwarp();                           // the pairs before are read
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = lane % 8 + 8 * j, tok = warp * MINE + lane / 8;
            if (r >= a.k) continue;
            const float v = gv[j] * (dv[j] - sum);
            s.pair[tok][r] = make_int2(id[j], __float_as_int(v));
            if (blockIdx.x == 0 && t + tok < t1) a.dlogits[(t + tok) * a.k + r] = v;
        }
        __syncwarp();
        const int e = lane % EP;
#pragma unroll
        for (int i = 0; i < MINE / AT_ONCE; ++i) {
            const int tok = warp * MINE + i * AT_ONCE + lane / EP;
            float v = 0.f;
            bool named = false;
#pragma unroll 4
            for (int r = 0; r < a.k; ++r) {
                const int2 p = s.pair[tok][r];
                if (p.x == e) v += __int_as_float(p.y), named = true;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, named);
            if (e == 0) s.mask[buf][tok] = EP == 32 ? m : m >> (lane / EP * EP) & ((1u << (EP % 32)) - 1);
            uint16_t part[3];
            cut3(v, part);
            bias += v;
#pragma unroll
            for (int q = 0; q < 3; ++q) s.a[buf][q][tok][e] = part[q];
        }
    };
    auto load_x = [&](int t, int buf) {
        if (a.x && t < t1) {
            for (int i = threadIdx.x; i < TOK * kDenseCols / 8; i += kDenseThreads) {
                const int row = i / (kDenseCols / 8), col = i % (kDenseCols / 8) * 8, in = t + row < t1;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(&s.x[buf][row][col])),
                             "l"(a.x + (size_t)(in ? t + row : t0) * a.D + c0 + col), "r"(in ? 16 : 0)
                             : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // The block's columns of Wr, through the last buffer of x, and the first tiles.
    if (a.dx) {
        for (int i = threadIdx.x; i < EP * kDenseCols / 8; i += kDenseThreads) {
            const int e = i / (kDenseCols / 8), col = i % (kDenseCols / 8) * 8, in = e < a.E;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(&s.x[kDenseStages - 1][e][col])),
                         "l"(a.Wr + (size_t)(in ? e : 0) * a.D + c0 + col), "r"(in ? 16 : 0)
                         : "memory");
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
    for (int i = 0; i < kDenseStages - 1; ++i) load_x(t0 + i * TOK, i);
    load_pairs(t0);
    make_dl(t0, 0);
    load_pairs(t0 + TOK);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDenseStages - 1) : "memory");
    __syncthreads();
    // A warp's columns of Wr as the second operand, in registers.  Its columns are taken in an order that leaves a
    // lane 8 that follow one another in the sums: column 2 q + i of fragment j is column 8 q + 2 j + i.
    uint32_t w[K][4][2];
    uint32_t most = 0;                          // of the absolute values' bits: an infinity or NaN is above the others
    if (a.dx) {
#pragma unroll
        for (int kk = 0; kk < K; ++kk)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = kk * 16 + h * 8 + 2 * q4, col = warp * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
                    const uint32_t lo = reinterpret_cast<const uint16_t*>(s.x[kDenseStages - 1][e])[col];
                    const uint32_t hi = reinterpret_cast<const uint16_t*>(s.x[kDenseStages - 1][e + 1])[col];
                    w[kk][j][h] = lo | hi << 16;
                    most = __vmaxu2(most, w[kk][j][h] & 0x7fff7fffu);
                }
    }
    const bool by_pair = __any_sync(0xffffffffu, not_finite(most));
    float dw[K][4][4] = {};
    most = 0;
    int buf = 0, xb = 0;
    for (int t = t0; t < t1; t += TOK, buf ^= 1, xb = (xb + 1) % kDenseStages) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDenseStages - 2) : "memory");
        __syncthreads();                        // this tile is there, the one before (Wr) is done with
        load_x(t + (kDenseStages - 1) * TOK, (xb + kDenseStages - 1) % kDenseStages);
        if (a.dx && !by_pair) {
#pragma unroll
            for (int mt = 0; mt < TOK / 16; ++mt) {
                float acc[4][4] = {};
#pragma unroll
                for (int q = 2; q >= 0; --q)
#pragma unroll
                    for (int kk = 0; kk < K; ++kk) {
                        uint32_t f[4];
                        ldsm4(f, &s.a[buf][q][mt * 16 + lane % 16][kk * 16 + lane / 16 * 8]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma16816(acc[j], f, w[kk][j][0], w[kk][j][1]);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = t + mt * 16 + h * 8 + g;
                    if (tok >= t1) continue;
                    const size_t at = (size_t)tok * a.D + cw + 8 * q4;
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[2 * j] = acc[j][2 * h], o[2 * j + 1] = acc[j][2 * h + 1];
                    if (a.dx_add) {
                        float add[8];
                        load_f32<__nv_bfloat16, 8>(a.dx_add + at, add);
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] += add[j];
                    }
                    store_f32<__nv_bfloat16, 8>(a.dx + at, o);
                }
            }
        } else if (a.dx) {
            for (int i = 0; i < TOK && t + i < t1; ++i) {
                const size_t at = (size_t)(t + i) * a.D + cw + lane;
                float v = 0.f;
                for (uint32_t m = s.mask[buf][i]; m; m &= m - 1) {
                    const int e = __ffs(m) - 1;
                    v += whole(s.a[buf][0][i][e], s.a[buf][1][i][e], s.a[buf][2][i][e]) * __bfloat162float(a.Wr[(size_t)e * a.D + cw + lane]);
                }
                if (a.dx_add) v += __bfloat162float(a.dx_add[at]);
                a.dx[at] = from_f32<__nv_bfloat16>(v);
            }
        }
        if (a.x) {
#pragma unroll
            for (int ks = 0; ks < TOK / 16; ++ks) {
                uint32_t b[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    ldsm4t(b[n], &s.x[xb][ks * 16 + lane % 16][warp * 32 + n * 16 + lane / 16 * 8]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) most = __vmaxu2(most, b[n][i] & 0x7fff7fffu);
                }
#pragma unroll
                for (int q = 2; q >= 0; --q)
#pragma unroll
                    for (int mt = 0; mt < K; ++mt) {
                        uint32_t f[4];
                        ldsm4t(f, &s.a[buf][q][ks * 16 + lane / 16 * 8 + lane % 8][mt * 16 + lane / 8 % 2 * 8]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma16816(dw[mt][j], f, b[j / 2][j % 2 * 2], b[j / 2][j % 2 * 2 + 1]);
                    }
            }
        }
        if (t + TOK < t1) {
            make_dl(t + TOK, buf ^ 1);
            load_pairs(t + 2 * TOK);
        }
    }

    float* part = a.part + blockIdx.y * dense_stride(a.D, a.E);
    const bool again = __syncthreads_or(not_finite(most));
    if (blockIdx.x == 0) {                      // dbias: the warps' sums in order
        float* sums = reinterpret_cast<float*>(s.x);
        if (EP < 32) bias += __shfl_xor_sync(0xffffffffu, bias, EP % 32);
        if (lane < EP) sums[warp * EP + lane] = bias;
        __syncthreads();
        if ((int)threadIdx.x < a.E) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kDenseThreads / 32; ++i) v += sums[i * EP + threadIdx.x];
            part[(size_t)a.E * a.D + threadIdx.x] = v;
        }
    }
    if (!a.x) return;
    if (!again) {
#pragma unroll
        for (int mt = 0; mt < K; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e = mt * 16 + h * 8 + g;
                if (e >= a.E) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float2*>(part + (size_t)e * a.D + cw + j * 8 + 2 * q4) =
                        make_float2(dw[mt][j][2 * h], dw[mt][j][2 * h + 1]);
            }
        return;
    }
    float* col = part + c0 + threadIdx.x;       // the chunk again, a column per thread
    for (int e = 0; e < a.E; ++e) col[(size_t)e * a.D] = 0.f;
    for (int t = t0; t < t1; t += TOK) {
        __syncthreads();
        load_pairs(t);
        make_dl(t, 0);
        __syncthreads();
        for (int i = 0; i < TOK && t + i < t1; ++i) {
            const float v = __bfloat162float(a.x[(size_t)(t + i) * a.D + c0 + threadIdx.x]);
            for (uint32_t m = s.mask[0][i]; m; m &= m - 1) {
                const int e = __ffs(m) - 1;
                col[(size_t)e * a.D] += whole(s.a[0][0][i][e], s.a[0][1][i][e], s.a[0][2][i][e]) * v;
            }
        }
    }
}

// The chunks' partials: a thread adds up four columns of [E D + E], or with SHARES a
// share of them, and the shares in order.
template <int SHARES>
__global__ void __launch_bounds__(256) route_dense_join_kernel(const float* __restrict__ part, int n, int D, int E,
                                                               float* __restrict__ dWr, float* __restrict__ dbias) {
    constexpr int COLS = 256 / SHARES, BATCH = 10;
    __shared__ float4 sums[SHARES][COLS];
    const int w = threadIdx.x / COLS, lane = threadIdx.x % COLS, i = (blockIdx.x * COLS + lane) * 4;
    const size_t stride = dense_stride(D, E);
    pdl_wait();
    const bool row = i < E * D, live = row ? dWr != nullptr : i < E * D + E && dbias;
    const int each = (n + SHARES - 1) / SHARES, j1 = live ? min(n, (w + 1) * each) : 0;
    float4 s = {0.f, 0.f, 0.f, 0.f};
    for (int j = w * each; j < j1; j += BATCH) {
        float4 v[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j + q < j1) v[q] = __ldg(reinterpret_cast<const float4*>(part + (j + q) * stride + i));
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) s.x += v[q].x, s.y += v[q].y, s.z += v[q].z, s.w += v[q].w;
    }
    if (SHARES > 1) {
        sums[w][lane] = s;
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int q = 1; q < SHARES; ++q) {
            const float4 v = sums[q][lane];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    if (!live) return;
    if (row) {
        *reinterpret_cast<float4*>(dWr + i) = s;
    } else {
        const float v[4] = {s.x, s.y, s.z, s.w};
        for (int q = 0; q < 4 && i + q < E * D + E; ++q) dbias[i + q - E * D] = v[q];
    }
}

// Tokens of a block: about a wave of blocks.
inline int dense_chunks(int D, int E) {
    const int chunks = (E <= 16 ? kDenseBlocks16 : kDenseBlocks) / (D / kDenseCols);
    return chunks < 1 ? 1 : chunks;
}
inline int dense_chunk(int T, int D, int E) {
    const int chunks = dense_chunks(D, E);
    return ((T + chunks - 1) / chunks + kDenseTok - 1) / kDenseTok * kDenseTok;
}
// Of the partials of T tokens and of fewer: whole tiles per block leave at most this many blocks, and sometimes fewer
// of more tokens.
inline size_t dense_part_bytes(int T, int D, int E) {
    const int tiles = (T + kDenseTok - 1) / kDenseTok, chunks = dense_chunks(D, E);
    return (size_t)(tiles < chunks ? tiles : chunks) * ((size_t)E * D + (E + 3) / 4 * 4) * 4;
}

template <int EP>
cudaError_t run_route_dense(const DenseArgs& a, float* dWr, float* dbias, cudaStream_t s) {
    static std::atomic<uint64_t> set{0};
    if (!once_per_device(set, [] {
            return cudaFuncSetAttribute(route_dense_kernel<EP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)sizeof(DenseTile<EP>)) == cudaSuccess;
        }))
        return cudaErrorUnknown;
    const int chunks = (a.T + a.chunk - 1) / a.chunk;
    cudaError_t e = launch_pdl(route_dense_kernel<EP>, dim3(a.dx || a.x ? a.D / kDenseCols : 1, chunks),
                               dim3(kDenseThreads),
                               sizeof(DenseTile<EP>), s, a);
    if (e != cudaSuccess || (!dWr && !dbias)) return e;
    const int quads = (a.E * a.D + a.E + 3) / 4;
    auto join = [&](auto kernel, int shares) {  // ten partials or fewer per thread
        return launch_pdl(kernel, dim3((quads * shares + 255) / 256), dim3(256), 0, s, (const float*)a.part, chunks, a.D,
                          a.E, dWr, dbias);
    };
    if (chunks <= 10) return join(route_dense_join_kernel<1>, 1);
    return chunks <= 80 ? join(route_dense_join_kernel<8>, 8) : join(route_dense_join_kernel<32>, 32);
}

}  // namespace
}  // namespace moe
