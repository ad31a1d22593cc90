// zero_gated.cu -- the gated feed-forward block's products on the 5th-generation
// tensor cores (tcgen05, kind::f16), forward and backward.
//
//   forward   h = act(x Wg^T) (x Wu^T): both projections, the activation and the
//             product in one kernel; G = x Wg^T and U = x Wu^T are stored too
//             where a backward pass follows
//   backward  dG = dh U act'(G), dU = dh act(G)       (k_gated_slopes, stored)
//             dx = dG Wg + dU Wu                      one sum over both
//             dWg = dG^T x, dWu = dU^T x              one launch for both
//
// One kernel template does the three products.  Two blocks on neighbouring SMs
// (cta_group::2) share a tile of 256 x 256: each loads 128 rows of A and 128 of
// B, keeps 128 rows of the accumulator in its tensor memory, and the first one
// issues the products for both.  Alone, a block with 128 x 256 reads 96 bytes of
// shared memory a cycle for its products and writes as many for its loads, of
// 128 that there are; a pair halves B's share of both.  In the forward pass the
// first block's rows of B are Wg's and the second's Wu's, so that gate and up
// of one element come to lie in one lane of tensor memory, 128 columns apart,
// and neither is stored unless it is asked for.
//
// A block stays and walks tiles.  Warp 0's first lane copies stages of 64
// elements of k into shared memory (TMA, 128-byte swizzle), warp 1's first lane
// (of the first block) issues the four products of a stage, warps 2 to 5 read
// the accumulator back and finish it; two accumulators of 256 columns fill the
// tensor memory, so that one tile's end runs beside the next one's products.
// Operands whose k runs along the rows (Wg, Wu in dx; all in dW) are read where
// they lie, as chunks of 64 columns by 64 rows (the "MN-major" layout).
//
// Every wait is bounded.  A block whose wait runs out sets bit 0 of *status, its
// roles stop, what the pair has in flight is waited for (bounded again), the
// tensor memory is freed, and both leave; the outputs are then incomplete.
#include <cstdlib>

#include "zero_tc.cuh"

namespace zdp {

constexpr int GT_THREADS = 192;
constexpr int GT_TILE = 256;                  // rows and columns of a pair's tile
constexpr int GT_HALF = 128;                  // of a block's operands
constexpr int GT_K = 64;                      // elements of k in a stage: 128 bytes
constexpr int GT_OPERAND = GT_HALF * GT_K * 2;
constexpr int GT_CHUNK = GT_K * 128;          // 64 columns by 64 rows of an operand whose k runs along the rows
constexpr int GT_STAGE = 2 * GT_OPERAND;
constexpr int GT_STAGES = 6;
constexpr int GT_HEADER = 1024;
constexpr int GT_EPI = 4 * 32 * 17 * 4;       // a 32 x 16 piece for each epilogue warp, padded
constexpr int GT_SMEM = GT_STAGES * GT_STAGE + 2048 + GT_EPI;
static_assert(GT_SMEM <= 232448, "shared memory of a block");

enum { GT_FORWARD = 0, GT_DX = 1, GT_DW = 2 };

struct GatedOut {
    void* p;
    int64_t ld;
    int dt, store;                            // store: bytes of an aligned store of its rows (32, 16, or 0: unaligned)
};
struct GatedArgs {
    GatedOut o[3];                            // forward: h, gate, up; dx; dWg, dWu
    int64_t rows, cols;                       // of an output
    int m_tiles, n_tiles, half_tiles;         // tiles; dW: m_tiles of dWg
    int k_steps, k_half;                      // stages of a tile; dx: of them with gate
    int act, accumulate;
    int32_t* status;
    unsigned spin_limit, drain_limit;
};

// ---------------------------------------------------------------- PTX
// A tile to this block's shared memory, its bytes counted by a barrier of the pair's first block.
__device__ __forceinline__ void tma_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Arrives at the barrier of both blocks once what was issued before is done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((int)add)
        : "memory");
}
__device__ __forceinline__ uint32_t block_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ int read_at(uint32_t addr) {
    int v;
    asm volatile("ld.volatile.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// As mm_wait, for a barrier at which the other block arrives.
template <bool POLL>
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, unsigned limit, volatile int* stop) {
    if (POLL && limit) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
    }
#pragma unroll 1
    for (unsigned it = 0; it < limit; ++it) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if ((it & 255) == 255 && stop && *stop) return false;
    }
    return false;
}

// Shared-memory descriptor of an operand in the 128-byte swizzle.  k along the
// columns: rows of 128 bytes, 8 rows from one group to the next.  k along the
// rows: chunks of 64 columns (128 bytes), 8 rows of k a group.
template <bool K_ROWS>
__device__ __forceinline__ uint64_t gt_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)((K_ROWS ? GT_CHUNK >> 4 : 1) & 0x3FFF) << 16 |
           (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// 16 elements of k further on, in the descriptor's units of 16 bytes
template <bool K_ROWS> constexpr int GT_K16 = K_ROWS ? 16 * 128 >> 4 : 16 * 2 >> 4;
// Instruction descriptor: 16-bit operands, fp32 accumulator, 256 x 256.
template <int DT, bool A_ROWS, bool B_ROWS>
constexpr uint32_t GT_IDESC = 1u << 4 | (DT == ZERO_BF16 ? 1u << 7 | 1u << 10 : 0u) | (A_ROWS ? 1u << 15 : 0u) |
                              (B_ROWS ? 1u << 16 : 0u) | (uint32_t)(GT_TILE >> 3) << 17 | (uint32_t)(GT_TILE >> 4) << 24;

// ---------------------------------------------------------------- activations
// Both are g times a sigmoid s; the slope is s + g s (1 - s) t' with t the
// sigmoid's argument.  exp and the quotient are the fast ones: off by some
// 2^-20, of a result with 8 or 11 bits.
struct Act {
    float value, slope;
};
constexpr float GELU_A = 1.5957691216057308f, GELU_B = 0.044715f;       // 2 sqrt(2 / pi)
__device__ __forceinline__ float sigmoid(float t) { return __fdividef(1.f, 1.f + __expf(-t)); }
__device__ __forceinline__ float act_value(float g, int act) {
    float t = g;
    if (act == ZERO_GELU_TANH) {
        const float c = fminf(fmaxf(g, -100.f), 100.f);     // beyond, s is 0 or 1, and g^3 stays finite
        t = GELU_A * c * fmaf(GELU_B * c, c, 1.f);
    }
    return g * sigmoid(t);
}
__device__ __forceinline__ Act act_both(float g, int act) {
    float t = g, d = 1.f;
    if (act == ZERO_GELU_TANH) {
        const float c = fminf(fmaxf(g, -100.f), 100.f);
        t = GELU_A * c * fmaf(GELU_B * c, c, 1.f);
        d = GELU_A * fmaf(3.f * GELU_B * c, c, 1.f);
    }
    const float s = sigmoid(t), v = g * s;
    return {v, fmaf(v * (1.f - s), d, s)};
}

// ---------------------------------------------------------------- the end of a tile
// 16 columns of an output from column `col`, of this lane's row: rounded and
// stored, added to what is there if `add`.  The whole warp calls it; buf: its
// piece of shared memory.
template <int DT>
__device__ __forceinline__ void gt_put16(const GatedOut& o, int64_t rows, int64_t cols, int64_t row, int64_t col,
                                         float (&v)[16], bool add, float* buf) {
    const int lane = threadIdx.x & 31;
    if (col >= cols) return;
    if (o.store && col + 16 <= cols) {
        if (row >= rows) return;
        const int64_t at = row * o.ld + col;
        if (o.dt == ZERO_F32) {
            float* p = static_cast<float*>(o.p) + at;
            if (add)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 t = *reinterpret_cast<const float4*>(p + e);
                    v[e] += t.x;
                    v[e + 1] += t.y;
                    v[e + 2] += t.z;
                    v[e + 3] += t.w;
                }
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                const uint4 a = make_uint4(__float_as_uint(v[e]), __float_as_uint(v[e + 1]), __float_as_uint(v[e + 2]), __float_as_uint(v[e + 3]));
                const uint4 b = make_uint4(__float_as_uint(v[e + 4]), __float_as_uint(v[e + 5]), __float_as_uint(v[e + 6]), __float_as_uint(v[e + 7]));
                if (o.store == 32) {
                    st32(p + e, a, b);
                } else {
                    *reinterpret_cast<uint4*>(p + e) = a;
                    *reinterpret_cast<uint4*>(p + e + 4) = b;
                }
            }
            return;
        }
        uint16_t* p = static_cast<uint16_t*>(o.p) + at;
        if (add)
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                float t[8];
                widen8<DT>(ld8<DT>(p, e), t);
#pragma unroll
                for (int f = 0; f < 8; ++f) v[e + f] += t[f];
            }
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = Half16<DT>::narrow2(v[2 * e], v[2 * e + 1]);
        if (o.store == 32) {
            st32(p, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
        } else {
            reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return;
    }
    // rows that start anywhere, and the last columns: by shared memory, 16 neighbouring columns of two rows a store
#pragma unroll
    for (int e = 0; e < 16; ++e) buf[lane * 17 + e] = v[e];
    __syncwarp();
    const int64_t c = col + (lane & 15), r0 = row - lane;
    if (c < cols)
#pragma unroll 4
        for (int r = lane >> 4; r < 32; r += 2)
            if (r0 + r < rows) {
                const int64_t at = (r0 + r) * o.ld + c;
                float t = buf[r * 17 + (lane & 15)];
                if (add) t += o.dt == ZERO_F32 ? ld1<ZERO_F32>(o.p, at) : ld1<DT>(o.p, at);
                if (o.dt == ZERO_F32) st1<ZERO_F32>(o.p, at, t);
                else st1<DT>(o.p, at, t);
            }
    __syncwarp();
}

// Tiles in order, in groups of 8 tiles of columns so that the pairs that run
// together share both operands in L2.
__device__ __forceinline__ void gt_tile(const GatedArgs& a, int t, int& m, int& n) {
    const int per = 8 * a.m_tiles, g = t / per, n0 = g * 8;
    const int w = min(8, a.n_tiles - n0), r = t - g * per;
    m = r / w;
    n = n0 + r % w;
}

template <int MODE, int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GT_THREADS, 1)
    k_gated(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap a1,
            const __grid_constant__ CUtensorMap b0, const __grid_constant__ CUtensorMap b1,
            const __grid_constant__ GatedArgs a) {
    constexpr bool A_ROWS = MODE == GT_DW, B_ROWS = MODE != GT_FORWARD;      // k along the rows
    constexpr int N_TILE = MODE == GT_FORWARD ? GT_HALF : GT_TILE;           // columns of the output
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023) & ~1023u;
    uint8_t* head = smem_raw + (base - raw);
    // header: full[8] (the first block's count for both), empty[8], acc_full[2], acc_free[2] (the first block's), drained,
    // then the tensor-memory address, stop flag and count of loads issued
    const uint32_t full = base, empty = base + 64, acc_full = base + 128, acc_free = base + 144, drained = base + 160;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(head + 200);
    volatile int* stop = reinterpret_cast<volatile int*>(head + 204);
    volatile int* loaded = reinterpret_cast<volatile int*>(head + 208);
    const uint32_t stages = base + GT_HEADER;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3;                            // the 32 lanes of tensor memory this warp can reach
    const uint32_t rank = blockIdx.x & 1;                    // in the pair
    float* epi = reinterpret_cast<float*>(head + GT_HEADER + GT_STAGES * GT_STAGE) + quarter * 32 * 17;

    if (threadIdx.x == 0) {
        for (int s = 0; s < GT_STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + 8 * s, 1);
            mbar_init(acc_free + 8 * s, 8);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
        *stop = 0;
        *loaded = 0;
    }
    // Both blocks run before either allocates, and neither leaves before both have freed: the allocation is the pair's.
    // Without the first barrier, a block that had started well before its partner (beside a kernel whose blocks were still
    // on the partner's SM) was through, and the partner's allocation never returned.
    cluster_arrive();
    cluster_wait();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + 200) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();                                          // both blocks' barriers stand
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_next();

    const int n_tiles = a.m_tiles * a.n_tiles, first = blockIdx.x >> 1, step = gridDim.x >> 1, K = a.k_steps;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = block_addr(full, 0);
            int st = 0, count = 0;
            uint32_t phase = 0;
            for (int t = first; t < n_tiles && ok; t += step) {
                int m, n;
                gt_tile(a, t, m, n);
                const bool second = MODE == GT_DW && m >= a.half_tiles;
                const int am = (second ? m - a.half_tiles : m) * GT_TILE + (int)rank * GT_HALF;
                const int bn = MODE == GT_FORWARD ? n * GT_HALF : n * GT_TILE + (int)rank * GT_HALF;
                for (int k = 0; k < K; ++k) {
                    if (count >= GT_STAGES && !pair_wait<false>(empty + 8 * st, phase ^ 1, a.spin_limit, stop)) {
                        ok = false;
                        break;
                    }
                    const bool up = MODE == GT_DX && k >= a.k_half;
                    const int kk = (up ? k - a.k_half : k) * GT_K;
                    const CUtensorMap* A = second || up ? &a1 : &a0;
                    const CUtensorMap* B = (MODE == GT_FORWARD && rank) || up ? &b1 : &b0;
                    // rows and columns past the end read as 0
                    const uint32_t bar = full0 + 8 * st, at = stages + st * GT_STAGE;
                    if (rank == 0) mbar_expect_tx(full + 8 * st, 2 * GT_STAGE);
                    if (A_ROWS) {
                        tma_pair(at, A, am, kk, bar);
                        tma_pair(at + GT_CHUNK, A, am + 64, kk, bar);
                    } else {
                        tma_pair(at, A, kk, am, bar);
                    }
                    if (B_ROWS) {
                        tma_pair(at + GT_OPERAND, B, bn, kk, bar);
                        tma_pair(at + GT_OPERAND + GT_CHUNK, B, bn + 64, kk, bar);
                    } else {
                        tma_pair(at + GT_OPERAND, B, kk, bn, bar);
                    }
                    *loaded = ++count;
                    if (++st == GT_STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // the last stages' releases come from the first block: this one does not leave before them
            for (int c = max(0, count - GT_STAGES); c < count && ok; ++c)
                ok = pair_wait<false>(empty + 8 * (c % GT_STAGES), (uint32_t)(c / GT_STAGES) & 1, a.spin_limit, stop);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int st = 0, n = 0;
            uint32_t phase = 0;
            for (int t = first; t < n_tiles && ok; t += step, ++n) {
                const int acc = n & 1;
                if (n >= 2 && !pair_wait<true>(acc_free + 8 * acc, ((n - 2) >> 1) & 1, a.spin_limit, stop)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + acc * GT_TILE;
                for (int k = 0; k < K; ++k) {
                    if (!pair_wait<true>(full + 8 * st, phase, a.spin_limit, stop)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = stages + st * GT_STAGE;
                    const uint64_t da = gt_desc<A_ROWS>(at), db = gt_desc<B_ROWS>(at + GT_OPERAND);
#pragma unroll
                    for (int q = 0; q < GT_K / 16; ++q)
                        pair_mma(d, da + q * GT_K16<A_ROWS>, db + q * GT_K16<B_ROWS>, GT_IDESC<DT, A_ROWS, B_ROWS>, k > 0 || q > 0);
                    pair_commit(empty + 8 * st);
                    if (++st == GT_STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                if (ok) pair_commit(acc_full + 8 * acc);
            }
            pair_commit(drained);
        }
    } else {
        const uint32_t free0 = block_addr(acc_free, 0);
        int n = 0;
        for (int t = first; t < n_tiles; t += step, ++n) {
            int m, nt;
            gt_tile(a, t, m, nt);
            const int acc = n & 1;
            ok = pair_wait<false>(acc_full + 8 * acc, (n >> 1) & 1, a.spin_limit, stop);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + acc * GT_TILE + ((uint32_t)(quarter * 32) << 16);
            const bool second = MODE == GT_DW && m >= a.half_tiles;
            const int64_t row = (int64_t)(second ? m - a.half_tiles : m) * GT_TILE + (int)rank * GT_HALF + quarter * 32 + lane;
            const int64_t c0 = (int64_t)nt * N_TILE;
#pragma unroll 1
            for (int col = 0; col < N_TILE; col += 16) {
                uint32_t v[16], w[16];
                float f[16];
                __syncwarp();
                tc_ld16(d + col, v);
                if (MODE == GT_FORWARD) tc_ld16(d + GT_HALF + col, w);
                tc_wait_ld();
                if (col + 16 == N_TILE) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(free0 + 8 * acc);
                }
                if (MODE == GT_FORWARD) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = act_value(__uint_as_float(v[e]), a.act) * __uint_as_float(w[e]);
                    gt_put16<DT>(a.o[0], a.rows, a.cols, row, c0 + col, f, false, epi);
                    if (a.o[1].p) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(v[e]);
                        gt_put16<DT>(a.o[1], a.rows, a.cols, row, c0 + col, f, false, epi);
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(w[e]);
                        gt_put16<DT>(a.o[2], a.rows, a.cols, row, c0 + col, f, false, epi);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(v[e]);
                    gt_put16<DT>(a.o[second], a.rows, a.cols, row, c0 + col, f, a.accumulate, epi);
                }
            }
        }
    }
    if (!ok && lane == 0) {
        *stop = 1;
        atomicOr(a.status, 1);
    }
    __syncwarp();
    // what was issued and not waited for: the products
    if (threadIdx.x == 32) pair_wait<false>(drained, 0, a.drain_limit, nullptr);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    // after a stop of either block, the loads of both, which the first block's barriers count
    if (rank == 0 && threadIdx.x == 0 && (*stop || read_at(block_addr(base + 204, 1)))) {
        const int most = max(*loaded, read_at(block_addr(base + 208, 1)));
        for (int c = max(0, most - GT_STAGES); c < most; ++c)
            pair_wait<false>(full + 8 * (c % GT_STAGES), (uint32_t)(c / GT_STAGES) & 1, a.drain_limit, nullptr);
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
}

// ---------------------------------------------------------------- the slopes
struct SlopesArgs {
    const void *dh, *gate, *up;
    void *dgate, *dup, *pgate, *pup;          // pgate, pup: rows ldp apart for the products, or NULL
    int64_t lddh, ldg, ldu, lddg, lddu, ldp, rows, cols, tiles;
    int act;
};
constexpr int SL_THREADS = 256;

__device__ __forceinline__ void slopes(float dh, float g, float u, int act, float& dg, float& du) {
    const Act s = act_both(g, act);
    dg = dh * u * s.slope;
    du = dh * s.value;
}

// Rows on 16-byte boundaries, columns a multiple of 8: a tile is SL_THREADS
// units of 8 columns of a row (rows without gaps come as one).
template <int DT>
__global__ void __launch_bounds__(SL_THREADS) k_gated_slopes(const __grid_constant__ SlopesArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int64_t n = a.rows * a.tiles;
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x) {
        const int64_t row = a.rows == 1 ? 0 : t / a.tiles, c = ((t - row * a.tiles) * SL_THREADS + threadIdx.x) * 8;
        if (c >= a.cols) continue;
        float d[8], g[8], u[8];
        widen8<DT>(ld8_stream<DT>(a.dh, row * a.lddh + c), d);
        widen8<DT>(ld8_stream<DT>(a.gate, row * a.ldg + c), g);
        widen8<DT>(ld8_stream<DT>(a.up, row * a.ldu + c), u);
#pragma unroll
        for (int e = 0; e < 8; ++e) slopes(d[e], g[e], u[e], a.act, g[e], u[e]);
        st8<DT>(a.dgate, row * a.lddg + c, narrow8<DT>(g));
        st8<DT>(a.dup, row * a.lddu + c, narrow8<DT>(u));
    }
}
// Rows that start anywhere: neighbouring lanes, neighbouring elements.
template <int DT>
__global__ void __launch_bounds__(SL_THREADS) k_gated_slopes_any(const __grid_constant__ SlopesArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int64_t n = a.rows * a.tiles;
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x) {
        const int64_t row = t / a.tiles, c0 = (t - row * a.tiles) * (SL_THREADS * 4) + threadIdx.x;
        float d[4], g[4], u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = c0 + j * SL_THREADS;
            const bool in = c < a.cols;
            d[j] = in ? ld1<DT>(a.dh, row * a.lddh + c) : 0.f;
            g[j] = in ? ld1<DT>(a.gate, row * a.ldg + c) : 0.f;
            u[j] = in ? ld1<DT>(a.up, row * a.ldu + c) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = c0 + j * SL_THREADS;
            if (c >= a.cols) break;
            float dg, du;
            slopes(d[j], g[j], u[j], a.act, dg, du);
            st1<DT>(a.dgate, row * a.lddg + c, dg);
            st1<DT>(a.dup, row * a.lddu + c, du);
            if (a.pgate) st1<DT>(a.pgate, row * a.ldp + c, dg);
            if (a.pup) st1<DT>(a.pup, row * a.ldp + c, du);
        }
    }
}

// A matrix whose rows start anywhere, copied to rows that the tensor maps can
// name: 16-byte boundaries, ldp apart.
__global__ void __launch_bounds__(256) k_gated_pack(const void* src, int64_t ld, int64_t rows, int64_t cols, void* dst, int64_t ldp) {
    pdl_wait();
    pdl_launch_next();
    const int64_t units = (cols + 7) / 8, n = rows * units;
    const Extent x = extent_of<ZERO_BF16>(src, ld, rows, cols);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / units, c = (i - row * units) * 8;
        st8<ZERO_BF16>(dst, row * ldp + c, ld8_shifted<ZERO_BF16>(static_cast<const uint16_t*>(src) + row * ld, c, cols, x));
    }
}
// zeros, where a sum has no terms
__global__ void __launch_bounds__(256) k_gated_zero(void* d, int64_t ld, int64_t rows, int64_t cols, int size) {
    pdl_wait();
    pdl_launch_next();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rows * cols; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t at = i / cols * ld + i % cols;
        if (size == 4) static_cast<uint32_t*>(d)[at] = 0;
        else static_cast<uint16_t*>(d)[at] = 0;
    }
}

// ---------------------------------------------------------------- host
constexpr unsigned GT_TYPES = 1u << ZERO_F16 | 1u << ZERO_BF16;
constexpr int64_t GT_MOST = INT32_MAX / 2;

// Row distance and bytes of a matrix packed for the tensor maps.
static int64_t packed_ld(int64_t cols) { return (cols + 63) / 64 * 64; }
static size_t packed_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (size_t)packed_ld(cols) * 2; }
static size_t room_for(const zero_mat* m, int64_t rows, int64_t cols) {
    return m && !rows_aligned(*m, rows) ? packed_bytes(rows, cols) : 0;
}

struct Maker {
    const char* call;
    uint8_t* ws;
    cudaStream_t s;
    int sms, dt, rc = ZERO_OK;
    // m as the products read it: where it lies, or packed into the workspace
    zero_mat packed(const zero_mat& m, int64_t rows, int64_t cols, bool copy = true) {
        if (rc != ZERO_OK || rows_aligned(m, rows)) return m;
        zero_mat p = {ws, packed_ld(cols), m.dtype, 0};
        ws += packed_bytes(rows, cols);
        if (!copy) return p;
        const void* src = m.data;
        int64_t ld = m.ld, ldp = p.ld;
        void* args[] = {&src, &ld, &rows, &cols, &p.data, &ldp};
        rc = cuda_fail(launch_after_previous((const void*)k_gated_pack, sms * 8, 256, args, 0, s), call);
        return p;
    }
    void zero(const zero_mat& m, int64_t rows, int64_t cols) {
        if (rc != ZERO_OK || rows == 0 || cols == 0) return;
        void* d = m.data;
        int64_t ld = m.ld;
        int size = elem_size(m.dtype);
        void* args[] = {&d, &ld, &rows, &cols, &size};
        rc = cuda_fail(launch_after_previous((const void*)k_gated_zero, sms * 4, 256, args, 0, s), call);
    }
    // boxes of 64 columns by box_rows rows, 128-byte swizzle; what lies outside reads as 0
    CUtensorMap map(const zero_mat& m, int64_t rows, int64_t cols, int box_rows) {
        CUtensorMap t = {};
        if (rc != ZERO_OK) return t;
        EncodeFn fn = encode_fn();
        if (!fn) {
            rc = refuse(ZERO_ECUDA, call, "the driver", " has no cuTensorMapEncodeTiled");
            return t;
        }
        // with one row any distance is right, and it must be a multiple of 16 bytes
        const cuuint64_t ld = rows == 1 ? (cuuint64_t)packed_ld(cols) : (cuuint64_t)m.ld;
        const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {ld * 2};
        const cuuint32_t box[2] = {GT_K, (cuuint32_t)box_rows}, one[2] = {1, 1};
        const CUresult r = fn(&t, dt == ZERO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, m.data,
                              dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) rc = refuse(ZERO_ECUDA, call, "cuTensorMapEncodeTiled", " failed");
        return t;
    }
    static GatedOut out(const zero_mat& m, int64_t rows) {
        const auto on = [&](int n) { return aligned(m.data, n) && (rows <= 1 || m.ld * elem_size(m.dtype) % n == 0); };
        return {m.data, m.ld, m.dtype, on(32) ? 32 : on(16) ? 16 : 0};
    }
    void product(int mode, const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0, const CUtensorMap& b1, GatedArgs& a,
                 int32_t* status) {
        if (rc != ZERO_OK) return;
        a.status = status;
        const char* e = std::getenv("ZERO_GB300_SPIN_LIMIT");
        a.spin_limit = e ? (unsigned)std::strtoul(e, nullptr, 10) : SPIN_LIMIT;
        a.drain_limit = SPIN_LIMIT;
        const bool bf = dt == ZERO_BF16;
        const void* f = mode == GT_FORWARD ? (bf ? (const void*)k_gated<GT_FORWARD, ZERO_BF16> : (const void*)k_gated<GT_FORWARD, ZERO_F16>)
                        : mode == GT_DX    ? (bf ? (const void*)k_gated<GT_DX, ZERO_BF16> : (const void*)k_gated<GT_DX, ZERO_F16>)
                                           : (bf ? (const void*)k_gated<GT_DW, ZERO_BF16> : (const void*)k_gated<GT_DW, ZERO_F16>);
        rc = raise_smem(f, GT_SMEM, call);
        if (rc != ZERO_OK) return;
        const int tiles = a.m_tiles * a.n_tiles, pairs = sms / 2;
        void* args[] = {const_cast<CUtensorMap*>(&a0), const_cast<CUtensorMap*>(&a1), const_cast<CUtensorMap*>(&b0),
                        const_cast<CUtensorMap*>(&b1), &a};
        rc = cuda_fail(launch_after_previous(f, 2 * (tiles < pairs ? tiles : pairs), GT_THREADS, args, GT_SMEM, s), call);
    }
};

static int tiles_of(int64_t n, int tile) { return (int)((n + tile - 1) / tile); }

static int check_sizes(int64_t rows, int64_t cols, int64_t ff, int act, const char* call) {
    if (rows < 0 || cols < 0 || ff < 0) return refuse(ZERO_EINVAL, call, "rows, cols or ff", " negative");
    if (rows > GT_MOST || cols > GT_MOST || ff > GT_MOST) return refuse(ZERO_ELIMIT, call, "sizes", ": more than 2^30 - 1 rows or columns");
    // tiles are counted in 32 bits: the largest of the three products' counts
    const int64_t r = tiles_of(rows, GT_TILE), c = tiles_of(cols, GT_TILE), f = tiles_of(ff, GT_HALF);
    if (r * f > GT_MOST || r * c > GT_MOST || 2 * f * c > GT_MOST) return refuse(ZERO_ELIMIT, call, "sizes", ": more than 2^30 tiles");
    if (act != ZERO_SILU && act != ZERO_GELU_TANH) return refuse(ZERO_EINVAL, call, "act", ": unknown activation");
    return ZERO_OK;
}
static int check_status(const int32_t* status, const char* call) {
    return status && aligned(status, 4) ? ZERO_OK : refuse(ZERO_EINVAL, call, "status", ": NULL or not 4-byte aligned");
}
static int check_room(const void* ws, size_t have, size_t need, const char* call) {
    if (need == 0) return ZERO_OK;
    if (!ws || !aligned(ws, 16) || have < need)
        return refuse(ZERO_EWORKSPACE, call, "workspace", ": NULL, not 16-byte aligned, or smaller than the call needs");
    return ZERO_OK;
}

}  // namespace zdp

using namespace zdp;

extern "C" {

size_t zero_gated_forward_workspace_bytes(const zero_mat* x, const zero_mat* gate_w, const zero_mat* up_w, int64_t rows,
                                          int64_t cols, int64_t ff) {
    if (rows <= 0 || cols <= 0 || ff <= 0) return 0;
    return room_for(x, rows, cols) + room_for(gate_w, ff, cols) + room_for(up_w, ff, cols);
}

int zero_gated_forward(const zero_mat* x, const zero_mat* gate_w, const zero_mat* up_w, int64_t rows, int64_t cols,
                       int64_t ff, int act, const zero_mat* h, const zero_mat* gate, const zero_mat* up, void* workspace,
                       size_t workspace_bytes, int32_t* status, void* stream) {
    const char* me = "zero_gated_forward";
    int rc = check_sizes(rows, cols, ff, act, me);
    if (rc == ZERO_OK) rc = check_mat(x, rows, cols, GT_TYPES, me, "x");
    if (rc == ZERO_OK) rc = check_mat(gate_w, ff, cols, GT_TYPES, me, "gate_w");
    if (rc == ZERO_OK) rc = check_mat(up_w, ff, cols, GT_TYPES, me, "up_w");
    if (rc == ZERO_OK) rc = check_mat(h, rows, ff, GT_TYPES, me, "h");
    if (rc == ZERO_OK && gate) rc = check_mat(gate, rows, ff, GT_TYPES, me, "gate");
    if (rc == ZERO_OK && up) rc = check_mat(up, rows, ff, GT_TYPES, me, "up");
    if (rc == ZERO_OK) rc = check_status(status, me);
    if (rc != ZERO_OK) return rc;
    const int dt = x->dtype;
    if (gate_w->dtype != dt || up_w->dtype != dt || h->dtype != dt || (gate && gate->dtype != dt) || (up && up->dtype != dt))
        return fail(ZERO_EINVAL, "zero_gated_forward: all matrices are of one type");
    if (!gate != !up) return fail(ZERO_EINVAL, "zero_gated_forward: gate and up: both or neither");
    rc = check_room(workspace, workspace_bytes, zero_gated_forward_workspace_bytes(x, gate_w, up_w, rows, cols, ff), me);
    if (rc != ZERO_OK || rows == 0 || ff == 0) return rc;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    Maker mk = {me, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream), sms, dt};
    if (cols == 0) {
        for (const zero_mat* o : {h, gate, up})
            if (o) mk.zero(*o, rows, ff);
        return mk.rc;
    }
    const zero_mat X = mk.packed(*x, rows, cols), G = mk.packed(*gate_w, ff, cols), U = mk.packed(*up_w, ff, cols);
    const CUtensorMap xm = mk.map(X, rows, cols, GT_HALF), gm = mk.map(G, ff, cols, GT_HALF), um = mk.map(U, ff, cols, GT_HALF);
    GatedArgs a = {};
    a.o[0] = Maker::out(*h, rows);
    if (gate) {
        a.o[1] = Maker::out(*gate, rows);
        a.o[2] = Maker::out(*up, rows);
    }
    a.rows = rows;
    a.cols = ff;
    a.m_tiles = tiles_of(rows, GT_TILE);
    a.n_tiles = tiles_of(ff, GT_HALF);
    a.k_steps = tiles_of(cols, GT_K);
    a.act = act;
    mk.product(GT_FORWARD, xm, xm, gm, um, a, status);
    return mk.rc;
}

size_t zero_gated_backward_workspace_bytes(const zero_mat* x, const zero_mat* gate_w, const zero_mat* up_w,
                                           const zero_mat* dgate, const zero_mat* dup, int64_t rows, int64_t cols,
                                           int64_t ff) {
    if (rows <= 0 || cols <= 0 || ff <= 0) return 0;
    return room_for(x, rows, cols) + room_for(gate_w, ff, cols) + room_for(up_w, ff, cols) + room_for(dgate, rows, ff) +
           room_for(dup, rows, ff);
}

int zero_gated_backward(const zero_mat* dh, const zero_mat* gate, const zero_mat* up, const zero_mat* x,
                        const zero_mat* gate_w, const zero_mat* up_w, int64_t rows, int64_t cols, int64_t ff, int act,
                        const zero_mat* dgate, const zero_mat* dup, const zero_mat* dx, const zero_mat* dgate_w,
                        const zero_mat* dup_w, int accumulate, void* workspace, size_t workspace_bytes, int32_t* status,
                        void* stream) {
    const char* me = "zero_gated_backward";
    constexpr unsigned W_TYPES = GT_TYPES | 1u << ZERO_F32;
    int rc = check_sizes(rows, cols, ff, act, me);
    if (rc == ZERO_OK) rc = check_mat(dh, rows, ff, GT_TYPES, me, "dh");
    if (rc == ZERO_OK) rc = check_mat(gate, rows, ff, GT_TYPES, me, "gate");
    if (rc == ZERO_OK) rc = check_mat(up, rows, ff, GT_TYPES, me, "up");
    if (rc == ZERO_OK) rc = check_mat(dgate, rows, ff, GT_TYPES, me, "dgate");
    if (rc == ZERO_OK) rc = check_mat(dup, rows, ff, GT_TYPES, me, "dup");
    if (rc == ZERO_OK && dx) rc = check_mat(dx, rows, cols, GT_TYPES, me, "dx");
    if (rc == ZERO_OK && dx) rc = check_mat(gate_w, ff, cols, GT_TYPES, me, "gate_w");
    if (rc == ZERO_OK && dx) rc = check_mat(up_w, ff, cols, GT_TYPES, me, "up_w");
    if (rc == ZERO_OK && dgate_w) rc = check_mat(dgate_w, ff, cols, W_TYPES, me, "dgate_w");
    if (rc == ZERO_OK && dup_w) rc = check_mat(dup_w, ff, cols, W_TYPES, me, "dup_w");
    if (rc == ZERO_OK && dgate_w) rc = check_mat(x, rows, cols, GT_TYPES, me, "x");
    if (rc == ZERO_OK) rc = check_status(status, me);
    if (rc != ZERO_OK) return rc;
    if (!dgate_w != !dup_w) return fail(ZERO_EINVAL, "zero_gated_backward: dgate_w and dup_w: both or neither");
    const int dt = dh->dtype;
    for (const zero_mat* m : {gate, up, dgate, dup, dx, dx ? gate_w : nullptr, dx ? up_w : nullptr, dgate_w ? x : nullptr})
        if (m && m->dtype != dt) return fail(ZERO_EINVAL, "zero_gated_backward: all matrices but the weights' gradients are of one type");
    if (dgate_w && (dgate_w->dtype != dup_w->dtype || (dgate_w->dtype != dt && dgate_w->dtype != ZERO_F32)))
        return fail(ZERO_EINVAL, "zero_gated_backward: dgate_w and dup_w are both in dh's type or both in fp32");
    rc = check_room(workspace, workspace_bytes,
                    zero_gated_backward_workspace_bytes(dgate_w ? x : nullptr, dx ? gate_w : nullptr, dx ? up_w : nullptr, dgate,
                                                        dup, rows, cols, ff), me);
    if (rc != ZERO_OK) return rc;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    Maker mk = {me, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream), sms, dt};
    if (rows == 0 || ff == 0) {                  // sums of nothing
        if (dx) mk.zero(*dx, rows, cols);
        if (dgate_w && !accumulate) {
            mk.zero(*dgate_w, ff, cols);
            mk.zero(*dup_w, ff, cols);
        }
        return mk.rc;
    }
    // what the products read; the slopes write their own packed form
    const bool products = cols > 0 && (dx || dgate_w);
    const zero_mat DG = products ? mk.packed(*dgate, rows, ff, false) : *dgate, DU = products ? mk.packed(*dup, rows, ff, false) : *dup;
    SlopesArgs sl = {};
    sl.dh = dh->data;
    sl.lddh = dh->ld;
    sl.gate = gate->data;
    sl.ldg = gate->ld;
    sl.up = up->data;
    sl.ldu = up->ld;
    sl.dgate = dgate->data;
    sl.lddg = dgate->ld;
    sl.dup = dup->data;
    sl.lddu = dup->ld;
    sl.pgate = DG.data != dgate->data ? DG.data : nullptr;
    sl.pup = DU.data != dup->data ? DU.data : nullptr;
    sl.ldp = packed_ld(ff);
    sl.rows = rows;
    sl.cols = ff;
    sl.act = act;
    bool v8 = ff % 8 == 0, whole = true;
    for (const zero_mat* m : {dh, gate, up, dgate, dup}) {
        v8 = v8 && rows_aligned(*m, rows);
        whole = whole && m->ld == ff;
    }
    if (v8 && whole) {
        sl.cols *= rows;
        sl.rows = 1;
    }
    const int64_t per_tile = v8 ? SL_THREADS * 8 : SL_THREADS * 4;
    sl.tiles = (sl.cols + per_tile - 1) / per_tile;
    const int64_t most = (int64_t)sms * 16, blocks = sl.rows * sl.tiles;
    const bool bf = dt == ZERO_BF16;
    const void* f = v8 ? (bf ? (const void*)k_gated_slopes<ZERO_BF16> : (const void*)k_gated_slopes<ZERO_F16>)
                       : (bf ? (const void*)k_gated_slopes_any<ZERO_BF16> : (const void*)k_gated_slopes_any<ZERO_F16>);
    void* args[] = {&sl};
    if (mk.rc == ZERO_OK)
        mk.rc = cuda_fail(launch_after_previous(f, (int)(blocks < most ? blocks : most), SL_THREADS, args, 0, mk.s), me);
    if (!products) return mk.rc;
    if (dx) {
        const zero_mat G = mk.packed(*gate_w, ff, cols), U = mk.packed(*up_w, ff, cols);
        GatedArgs a = {};
        a.o[0] = Maker::out(*dx, rows);
        a.rows = rows;
        a.cols = cols;
        a.m_tiles = tiles_of(rows, GT_TILE);
        a.n_tiles = tiles_of(cols, GT_TILE);
        a.k_half = tiles_of(ff, GT_K);
        a.k_steps = 2 * a.k_half;
        mk.product(GT_DX, mk.map(DG, rows, ff, GT_HALF), mk.map(DU, rows, ff, GT_HALF), mk.map(G, ff, cols, GT_K),
                   mk.map(U, ff, cols, GT_K), a, status);
    }
    if (dgate_w) {
        const zero_mat X = mk.packed(*x, rows, cols);
        GatedArgs a = {};
        a.o[0] = Maker::out(*dgate_w, ff);
        a.o[1] = Maker::out(*dup_w, ff);
        a.rows = ff;
        a.cols = cols;
        a.half_tiles = tiles_of(ff, GT_TILE);
        a.m_tiles = 2 * a.half_tiles;
        a.n_tiles = tiles_of(cols, GT_TILE);
        a.k_steps = tiles_of(rows, GT_K);
        a.accumulate = accumulate;
        const CUtensorMap xm = mk.map(X, rows, cols, GT_K);
        mk.product(GT_DW, mk.map(DG, rows, ff, GT_K), mk.map(DU, rows, ff, GT_K), xm, xm, a, status);
    }
    return mk.rc;
}

}  // extern "C"
