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
// (of the first block) issues the four products of a stage, warps 2 to 9 read
// the accumulator back and finish it; two accumulators of 256 columns fill the
// tensor memory, so that one tile's end runs beside the next one's products.
// Operands whose k runs along the rows (Wg, Wu in dx; all in dW) are read where
// they lie, as chunks of 64 columns by 64 rows (the "MN-major" layout).
//
// Measured (GB300, bf16, through 4096 x 14336): 8192 rows in 1.09 to 1.18 ms, 1.77 to
// 1.64 PFLOP/s, at the card's power limit (a library product: 1.71 sustained, 1.87 in
// a burst); 1.00 where the limit does not hold yet; with gate and up stored 1.20; dx
// and dW 1.18 and 1.20 each, dW added to a bucket 1.21, in fp32 1.25, added in fp32
// 1.26; the slopes 186 us, 6.3 TB/s.
// 512 rows in 73 us, 129 to 256 in 53: 8.5 to start and end, then two rounds of 112
// tiles on 76 pairs, the first bound by HBM, the second by its 36 pairs' products.
// A stage takes 512 cycles of products whatever the rows, and whether B has 256
// rows or 128 (tiles of 64 columns: 63 us), so shorter rounds do not help.  With up
// to 128 rows a block alone has a tile where that takes fewer rounds (one of 112
// blocks): 44 us for the 51 to 52 of pairs, HBM at 0.80.  Weights asked for
// ahead towards L2, and sums that start at different places of k, made it slower
// (56 to 67 us; 56).  Outputs whose rows start on 16 bytes but not on 32 are stored
// half a sector at a time: with gate and up 2001 x 1600 x 4264 takes 56 us, 2048 x
// 1600 x 4352 44.  Odd widths are copied first: 2001 x 1601 x 4263 in 65 us, 94
// with gate and up, its slopes, dx and dW in 25, 70 and 65.
//
// Every wait on an mbarrier is bounded.  A block whose wait runs out sets bit 0 of
// *status, its roles stop, what the pair has in flight is waited for (bounded again),
// the tensor memory is freed, and both leave; the outputs are then incomplete.  The
// cluster barriers and the tensor-memory allocation have no limit of their own.
// They end because a cluster's blocks are scheduled together and each of their
// threads reaches every barrier, bounded waits in between; and because a block's 216
// KB of shared memory keep any other of these kernels, or of the 4-bit product's,
// off its SM while it holds tensor memory.
#include <cstdlib>

#include "zero_tc.cuh"

namespace zdp {

constexpr int GT_EPI_WARPS = 8;               // two for each 32 lanes of tensor memory, a half of the columns each
constexpr int GT_THREADS = 64 + 32 * GT_EPI_WARPS;
constexpr int GT_TILE = 256;                  // rows and columns of a pair's tile
constexpr int GT_HALF = 128;                  // of a block's operands
constexpr int GT_K = 64;                      // elements of k in a stage: 128 bytes
constexpr int GT_A = GT_HALF * GT_K * 2;      // bytes of a block's A in a stage
constexpr int GT_CHUNK = GT_K * 128;          // 64 columns by 64 rows of an operand whose k runs along the rows
constexpr int GT_HEADER = 1024;
constexpr int GT_EPI = GT_EPI_WARPS * 32 * 17 * 4;      // a 32 x 16 piece for each of its warps, padded

// Alone, a block has all 256 rows of B.
template <bool PAIR>
struct GtShape {
    static constexpr int B = PAIR ? GT_A : 2 * GT_A, STAGE = GT_A + B, STAGES = PAIR ? 6 : 4;
    static constexpr int SMEM = STAGES * STAGE + 2048 + GT_EPI;
    static_assert(SMEM <= 232448 && STAGES <= 8, "shared memory of a block");
};

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
    int split;                                // dx: parts of its sum, each to rows of its own (the parts' outputs follow one another)
    int a_rows;                               // rows of A's boxes: 128, or what few rows need (the second block then has none)
    int act, accumulate;
    int32_t* status;
    unsigned spin_limit, drain_limit;
};

// ---------------------------------------------------------------- PTX
// A tile to this block's shared memory, its bytes counted by a barrier of the pair's first block.
template <bool PAIR>
__device__ __forceinline__ void gt_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        tma_tile(dst, map, x, y, bar);
}
// All threads of the pair, or of the block.
template <bool PAIR>
__device__ __forceinline__ void gt_meet() {
    if constexpr (PAIR) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}
// Arrives at the barrier (of both blocks) once what was issued before is done.
template <bool PAIR>
__device__ __forceinline__ void gt_commit(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void gt_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((int)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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
// Instruction descriptor: 16-bit operands, fp32 accumulator, 256 columns and 256 rows, or 128.
template <int DT, bool PAIR, bool A_ROWS, bool B_ROWS>
constexpr uint32_t GT_IDESC = 1u << 4 | (DT == ZERO_BF16 ? 1u << 7 | 1u << 10 : 0u) | (A_ROWS ? 1u << 15 : 0u) |
                              (B_ROWS ? 1u << 16 : 0u) | (uint32_t)(GT_TILE >> 3) << 17 | (uint32_t)((PAIR ? GT_TILE : GT_HALF) >> 4) << 24;

// ---------------------------------------------------------------- activations
// Both are g times a sigmoid s; the slope is s + g s (1 - s) t' with t the
// sigmoid's argument.  s and 1 - s are taken from exp(-|t|), which is at most 1:
// far below zero s is exp(t) down to the smallest number (by 1 / (1 + exp(-t)) it
// was 0 from t = -87.4 on, where __fdividef's divisor passes 2^126, and bf16 holds
// g s down to t = -96).  exp and the quotient are the fast ones: s is off by some
// (4 + 1.2 |t|) 2^-23 of itself (exp's error grows with its argument), GELU's t by
// |t| 2^-22 more, of a result with 8 or 11 bits.
struct Act {
    float value, slope;
};
struct Sigmoid {
    float s, rest;                            // rest: 1 - s
};
constexpr float GELU_A = 1.5957691216057308f, GELU_B = 0.044715f;       // 2 sqrt(2 / pi)
__device__ __forceinline__ Sigmoid sigmoid(float t) {
    const float e = __expf(-fabsf(t)), most = __fdividef(1.f, 1.f + e), least = e * most;
    return t < 0.f ? Sigmoid{least, most} : Sigmoid{most, least};
}
__device__ __forceinline__ float act_value(float g, int act) {
    float t = g;
    if (act == ZERO_GELU_TANH) {
        const float c = fminf(fmaxf(g, -100.f), 100.f);     // beyond, s is 0 or 1, and g^3 stays finite
        t = GELU_A * c * fmaf(GELU_B * c, c, 1.f);
    }
    return g * sigmoid(t).s;
}
__device__ __forceinline__ Act act_both(float g, int act) {
    float t = g, d = 1.f;
    if (act == ZERO_GELU_TANH) {
        const float c = fminf(fmaxf(g, -100.f), 100.f);
        t = GELU_A * c * fmaf(GELU_B * c, c, 1.f);
        d = GELU_A * fmaf(3.f * GELU_B * c, c, 1.f);
    }
    const Sigmoid s = sigmoid(t);
    const float v = g * s.s;
    return {v, fmaf(v * s.rest, d, s.s)};
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

// PAIR: two blocks a tile of 256 rows; else (forward, up to 128 rows) one.
template <int MODE, int DT, bool PAIR>
__device__ __forceinline__ void gated(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0, const CUtensorMap& b1,
                                      const GatedArgs& a) {
    using S = GtShape<PAIR>;
    constexpr int STAGES = S::STAGES;
    static_assert(PAIR || MODE == GT_FORWARD, "one block a tile");
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
    const uint32_t rank = PAIR ? blockIdx.x & 1 : 0;         // in the pair
    float* epi = reinterpret_cast<float*>(head + GT_HEADER + STAGES * S::STAGE) + (warp & 7) * 32 * 17;

    if (threadIdx.x == 0) {
        for (const CUtensorMap* m : {&a0, &a1, &b0, &b1}) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + 8 * s, 1);
            mbar_init(acc_free + 8 * s, (PAIR ? 2 : 1) * GT_EPI_WARPS);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
        *stop = 0;
        *loaded = 0;
    }
    // Both blocks run before either allocates, and neither leaves before both have freed: the allocation is the pair's.
    // Without the first barrier, a block that had started well before its partner (beside a kernel whose blocks were still
    // on the partner's SM) was through, and the partner's allocation never returned.
    gt_meet<PAIR>();
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + 200) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + 200) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    gt_meet<PAIR>();                                          // both blocks' barriers stand
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_next();

    // this pair's tiles, and the stages of the part of the sum that a tile stands for
    const int n_parts = a.m_tiles * a.n_tiles, n_tiles = n_parts * a.split, first = PAIR ? blockIdx.x >> 1 : blockIdx.x,
              step = PAIR ? gridDim.x >> 1 : gridDim.x;
    const auto part_of = [&](int t, int& tile, int& k0, int& k1) {
        const int part = MODE == GT_DX ? t / n_parts : 0;
        tile = MODE == GT_DX ? t - part * n_parts : t;
        k0 = MODE == GT_DX ? (int)((int64_t)a.k_steps * part / a.split) : 0;
        k1 = MODE == GT_DX ? (int)((int64_t)a.k_steps * (part + 1) / a.split) : a.k_steps;
        return part;
    };
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = PAIR ? block_addr(full, 0) : full;
            int st = 0, count = 0;
            uint32_t phase = 0;
            for (int t = first; t < n_tiles && ok; t += step) {
                int m, n, tile, k0, k1;
                part_of(t, tile, k0, k1);
                gt_tile(a, tile, m, n);
                const bool second = MODE == GT_DW && m >= a.half_tiles;
                const int am = (second ? m - a.half_tiles : m) * GT_TILE + (int)rank * GT_HALF;
                const int bn = MODE == GT_FORWARD ? n * N_TILE : n * GT_TILE + (int)rank * GT_HALF;
                const uint32_t bytes = (a.a_rows < GT_HALF ? a.a_rows * (GT_K * 2) : (PAIR ? 2 : 1) * GT_A) + 2 * GT_A;
                for (int k = k0; k < k1; ++k) {
                    if (count >= STAGES && !pair_wait<true>(empty + 8 * st, phase ^ 1, a.spin_limit, stop)) {
                        ok = false;
                        break;
                    }
                    const bool up = MODE == GT_DX && k >= a.k_half;
                    const int kk = (up ? k - a.k_half : k) * GT_K;
                    const CUtensorMap* A = second || up ? &a1 : &a0;
                    const CUtensorMap* B = (MODE == GT_FORWARD && rank) || up ? &b1 : &b0;
                    // rows and columns past the end read as 0
                    const uint32_t bar = full0 + 8 * st, at = stages + st * S::STAGE;
                    if (rank == 0) mbar_expect_tx(full + 8 * st, bytes);
                    if (A_ROWS) {
                        gt_load<PAIR>(at, A, am, kk, bar);
                        gt_load<PAIR>(at + GT_CHUNK, A, am + 64, kk, bar);
                    } else if (rank == 0 || a.a_rows == GT_HALF) {
                        // of few rows only the boxes' are loaded; what else lies in A's place is multiplied, but not stored
                        gt_load<PAIR>(at, A, kk, am, bar);
                    }
                    if (B_ROWS) {
                        gt_load<PAIR>(at + GT_A, B, bn, kk, bar);
                        gt_load<PAIR>(at + GT_A + GT_CHUNK, B, bn + 64, kk, bar);
                    } else {
                        gt_load<PAIR>(at + GT_A, B, kk, bn, bar);
                        if (!PAIR) gt_load<PAIR>(at + 2 * GT_A, &b1, kk, bn, bar);
                    }
                    *loaded = ++count;
                    if (++st == STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // the last stages' releases come from the first block: this one does not leave before them
            for (int c = max(0, count - STAGES); c < count && ok; ++c)
                ok = pair_wait<false>(empty + 8 * (c % STAGES), (uint32_t)(c / STAGES) & 1, a.spin_limit, stop);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int st = 0, n = 0;
            uint32_t phase = 0;
            for (int t = first; t < n_tiles && ok; t += step, ++n) {
                const int acc = n & 1;
                int tile, k0, k1;
                part_of(t, tile, k0, k1);
                if (n >= 2 && !pair_wait<true>(acc_free + 8 * acc, ((n - 2) >> 1) & 1, a.spin_limit, stop)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + acc * GT_TILE;
                for (int k = k0; k < k1; ++k) {
                    if (!pair_wait<true>(full + 8 * st, phase, a.spin_limit, stop)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = stages + st * S::STAGE;
                    const uint64_t da = gt_desc<A_ROWS>(at), db = gt_desc<B_ROWS>(at + GT_A);
#pragma unroll
                    for (int q = 0; q < GT_K / 16; ++q)
                        gt_mma<PAIR>(d, da + q * GT_K16<A_ROWS>, db + q * GT_K16<B_ROWS>, GT_IDESC<DT, PAIR, A_ROWS, B_ROWS>, k > k0 || q > 0);
                    gt_commit<PAIR>(empty + 8 * st);
                    if (++st == STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                if (ok) gt_commit<PAIR>(acc_full + 8 * acc);
            }
            gt_commit<PAIR>(drained);
        }
    } else {
        const uint32_t free0 = PAIR ? block_addr(acc_free, 0) : acc_free;
        constexpr int HALF = N_TILE / 2;
        const int from = (warp - 2) / 4 * HALF;               // this warp's columns of the tile
        int n = 0;
        for (int t = first; t < n_tiles; t += step, ++n) {
            int m, nt, tile, k0, k1;
            const int part = part_of(t, tile, k0, k1);
            gt_tile(a, tile, m, nt);
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
            GatedOut o = a.o[MODE == GT_DW && second ? 1 : 0];
            if (MODE == GT_DX && a.split > 1) o.p = static_cast<float*>(o.p) + part * a.rows * o.ld;
            const auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(free0 + 8 * acc);
            };
            // a warp whose rows are all past the end has nothing to store
            if (row - lane >= a.rows) {
                release();
                continue;
            }
            if constexpr (MODE == GT_FORWARD) {
#pragma unroll 1
                for (int col = from; col < from + HALF; col += 16) {
                    uint32_t v[16], w[16];
                    float f[16];
                    __syncwarp();
                    tc_ld16(d + col, v);
                    tc_ld16(d + GT_HALF + col, w);
                    tc_wait_ld();
                    if (col + 16 == from + HALF) release();
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = act_value(__uint_as_float(v[e]), a.act) * __uint_as_float(w[e]);
                    gt_put16<DT>(o, a.rows, a.cols, row, c0 + col, f, false, epi);
                    if (a.o[1].p) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(v[e]);
                        gt_put16<DT>(a.o[1], a.rows, a.cols, row, c0 + col, f, false, epi);
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(w[e]);
                        gt_put16<DT>(a.o[2], a.rows, a.cols, row, c0 + col, f, false, epi);
                    }
                }
            } else {
                // 64 columns at a time: a lane's stores fill whole lines of 128 bytes one behind the other
#pragma unroll 1
                for (int col = from; col < from + HALF; col += 64) {
                    uint32_t v[4][16];
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_ld16(d + col + 16 * q, v[q]);
                    tc_wait_ld();
                    if (col + 64 == from + HALF) release();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float f[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(v[q][e]);
                        gt_put16<DT>(o, a.rows, a.cols, row, c0 + col + 16 * q, f, a.accumulate, epi);
                    }
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
    gt_meet<PAIR>();
    // after a stop of either block, the loads of both, which the first block's barriers count
    if (rank == 0 && threadIdx.x == 0 && (*stop || (PAIR && read_at(block_addr(base + 204, 1))))) {
        const int most = PAIR ? max(*loaded, read_at(block_addr(base + 208, 1))) : *loaded;
        for (int c = max(0, most - STAGES); c < most; ++c)
            pair_wait<false>(full + 8 * (c % STAGES), (uint32_t)(c / STAGES) & 1, a.drain_limit, nullptr);
    }
    __syncthreads();
    gt_meet<PAIR>();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    __syncwarp();
    gt_meet<PAIR>();
}

template <int MODE, int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GT_THREADS, 1)
    k_gated(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap a1,
            const __grid_constant__ CUtensorMap b0, const __grid_constant__ CUtensorMap b1,
            const __grid_constant__ GatedArgs a) {
    gated<MODE, DT, true>(a0, a1, b0, b1, a);
}
// Up to 128 rows, where one block a tile needs fewer rounds (112 tiles: one of 152 blocks, two of 76 pairs).
template <int DT>
__global__ void __launch_bounds__(GT_THREADS, 1)
    k_gated_alone(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap a1,
                  const __grid_constant__ CUtensorMap b0, const __grid_constant__ CUtensorMap b1,
                  const __grid_constant__ GatedArgs a) {
    gated<GT_FORWARD, DT, false>(a0, a1, b0, b1, a);
}

// ---------------------------------------------------------------- few rows
// Up to 4 rows: the weights are read once, and the sums are fp32 ones of the
// ordinary units.  A warp has two columns of h, that is four rows of weights, of
// which a lane reads every 32nd unit of 8; x lies in shared memory as it is.
// Bound: HBM (the weights' bytes): through 4096 x 14336 bf16 one row in 35.7 us,
// 6.57 TB/s (0.97 of the measured copy bandwidth), two in 36.1, four in 42.6.
// The products above take 43 us for any number up to 128.  Eight rows here take
// 78: their sums leave half the registers for loads.
constexpr int FEW_ROWS = 4, FEW_THREADS = 256;
constexpr size_t FEW_SMEM = 96 * 1024;        // of x: two blocks an SM

struct FewArgs {
    const void *x, *wg, *wu;
    int64_t ldx, ldg, ldu, ff;
    int rows, cols, units, act;
    GatedOut o[3];
};

template <int DT, int R, bool V8>
__global__ void __launch_bounds__(FEW_THREADS, 2) k_gated_few(const __grid_constant__ FewArgs a) {
    extern __shared__ __align__(16) uint4 xs[];              // [row][unit]
    pdl_wait();
    pdl_launch_next();
    const Extent ex = extent_of<DT>(a.x, a.ldx, a.rows, a.cols), eg = extent_of<DT>(a.wg, a.ldg, a.ff, a.cols),
                 eu = extent_of<DT>(a.wu, a.ldu, a.ff, a.cols);
    for (int i = threadIdx.x; i < R * a.units; i += FEW_THREADS) {
        const int r = i / a.units, u = i - r * a.units;
        const uint16_t* row = static_cast<const uint16_t*>(a.x) + r * a.ldx;
        xs[i] = r >= a.rows ? make_uint4(0, 0, 0, 0) : V8 ? ld8<DT>(row, u * 8).w[0] : ld8_shifted<DT>(row, u * 8, a.cols, ex).w[0];
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int64_t pairs = (a.ff + 1) / 2, step = (int64_t)gridDim.x * (FEW_THREADS / 32);
    for (int64_t p = (int64_t)blockIdx.x * (FEW_THREADS / 32) + (threadIdx.x >> 5); p < pairs; p += step) {
        const int64_t f = 2 * p, f1 = f + 1 < a.ff ? f + 1 : f;          // an odd last column twice
        const uint16_t* const w[4] = {static_cast<const uint16_t*>(a.wg) + f * a.ldg, static_cast<const uint16_t*>(a.wu) + f * a.ldu,
                                      static_cast<const uint16_t*>(a.wg) + f1 * a.ldg, static_cast<const uint16_t*>(a.wu) + f1 * a.ldu};
        uint64_t sum[4][R] = {};
        constexpr int AT_ONCE = R <= 2 ? 4 : 2;              // units whose loads are under way, beside 8 R registers of sums
        for (int u0 = lane; u0 < a.units; u0 += 32 * AT_ONCE) {
            Raw8<DT> v[AT_ONCE][4];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                const int u = u0 + 32 * j;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[j][q].w[0] = make_uint4(0, 0, 0, 0);
                    if (u < a.units) {
                        if (V8) v[j][q] = ld8_stream<DT>(w[q], u * 8);
                        else v[j][q] = ld8_shifted<DT>(w[q], u * 8, a.cols, q & 1 ? eu : eg);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                const int u = u0 + 32 * j;
                if (u >= a.units) break;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    Raw8<DT> x;
                    x.w[0] = xs[r * a.units + u];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[q][r] = fma2(pair8<DT>(v[j][q], e), pair8<DT>(x, e), sum[q][r]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float t[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 s = unpack2(sum[q][r]);
                t[q] = warp_sum(s.x + s.y);
            }
            if (lane == 0 && r < a.rows) {
                const int n = f1 > f ? 2 : 1;
                for (int c = 0; c < n; ++c) {
                    const float g = t[2 * c], u = t[2 * c + 1];
                    st1<DT>(a.o[0].p, r * a.o[0].ld + f + c, act_value(g, a.act) * u);
                    if (a.o[1].p) {
                        st1<DT>(a.o[1].p, r * a.o[1].ld + f + c, g);
                        st1<DT>(a.o[2].p, r * a.o[2].ld + f + c, u);
                    }
                }
            }
        }
    }
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
        const int64_t row = a.rows == 1 ? 0 : quotient(t, a.tiles), c = ((t - row * a.tiles) * SL_THREADS + threadIdx.x) * 8;
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
        const int64_t row = quotient(t, a.tiles), c0 = (t - row * a.tiles) * (SL_THREADS * 4) + threadIdx.x;
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
        const int64_t row = quotient(i, units), c = (i - row * units) * 8;
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

// The parts of a sum over k added in order and rounded.  A thread four columns of
// a row; the parts' columns are padded to a multiple of 8.
__global__ void __launch_bounds__(256) k_gated_join(const float* parts, int n, int64_t ldp, int64_t rows, int64_t cols, GatedOut o) {
    pdl_wait();
    pdl_launch_next();
    const int64_t quads = ldp / 4;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rows * quads; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = quotient(i, quads), c = (i - row * quads) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < n; ++p) {
            const float4 v = *reinterpret_cast<const float4*>(parts + (p * rows + row) * ldp + c);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        const float f[4] = {s.x, s.y, s.z, s.w};
        if (o.store && c + 4 <= cols) {
            const uint2 w = o.dt == ZERO_BF16 ? make_uint2(Half16<ZERO_BF16>::narrow2(f[0], f[1]), Half16<ZERO_BF16>::narrow2(f[2], f[3]))
                                              : make_uint2(Half16<ZERO_F16>::narrow2(f[0], f[1]), Half16<ZERO_F16>::narrow2(f[2], f[3]));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(o.p) + row * o.ld + c) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < cols) st1_any(o.p, row * o.ld + c + e, f[e], o.dt);
        }
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
                 int32_t* status, bool alone = false) {
        if (rc != ZERO_OK) return;
        a.status = status;
        const char* e = std::getenv("ZERO_GB300_SPIN_LIMIT");
        a.spin_limit = e ? (unsigned)std::strtoul(e, nullptr, 10) : SPIN_LIMIT;
        a.drain_limit = SPIN_LIMIT;
        if (a.split < 1) a.split = 1;
        if (!a.a_rows) a.a_rows = GT_HALF;
        const bool bf = dt == ZERO_BF16;
        const void* f = mode == GT_FORWARD ? (bf ? (const void*)k_gated<GT_FORWARD, ZERO_BF16> : (const void*)k_gated<GT_FORWARD, ZERO_F16>)
                        : mode == GT_DX    ? (bf ? (const void*)k_gated<GT_DX, ZERO_BF16> : (const void*)k_gated<GT_DX, ZERO_F16>)
                                           : (bf ? (const void*)k_gated<GT_DW, ZERO_BF16> : (const void*)k_gated<GT_DW, ZERO_F16>);
        if (alone) f = bf ? (const void*)k_gated_alone<ZERO_BF16> : (const void*)k_gated_alone<ZERO_F16>;
        const size_t smem = alone ? GtShape<false>::SMEM : GtShape<true>::SMEM;
        rc = raise_smem(f, smem, call);
        if (rc != ZERO_OK) return;
        const int tiles = a.m_tiles * a.n_tiles * a.split, at_once = alone ? sms : sms / 2;
        void* args[] = {const_cast<CUtensorMap*>(&a0), const_cast<CUtensorMap*>(&a1), const_cast<CUtensorMap*>(&b0),
                        const_cast<CUtensorMap*>(&b1), &a};
        rc = cuda_fail(launch_after_previous(f, (alone ? 1 : 2) * (tiles < at_once ? tiles : at_once), GT_THREADS, args, smem, s), call);
    }
};

static int tiles_of(int64_t n, int tile) { return (int)((n + tile - 1) / tile); }

// Whether the few rows' kernel takes them: its x must fit shared memory.
static int few_of(int64_t rows) { return rows <= 1 ? 1 : rows <= 2 ? 2 : 4; }
static bool is_few(int64_t rows, int64_t cols) {
    return rows <= FEW_ROWS && cols <= 1 << 20 && (size_t)few_of(rows) * (size_t)((cols + 7) / 8) * 16 <= FEW_SMEM;
}
template <int DT>
static const void* few_fn(int r, bool v8) {
    if (v8)
        return r == 1 ? (const void*)k_gated_few<DT, 1, true> : r == 2 ? (const void*)k_gated_few<DT, 2, true>
                                                                       : (const void*)k_gated_few<DT, 4, true>;
    return r == 1 ? (const void*)k_gated_few<DT, 1, false> : r == 2 ? (const void*)k_gated_few<DT, 2, false>
                                                                    : (const void*)k_gated_few<DT, 4, false>;
}

// Rows of A's boxes: of up to 128 rows the multiple of 8 that holds them.
// Rows past the end cost the loads as much as others, and more (one token
// through 4096 x 14336: 81 us with boxes of 128 rows, where 100 tokens took 52).
static int boxes_of(int64_t rows) { return rows > GT_HALF ? GT_HALF : (int)((rows + 7) / 8 * 8); }

// Parts of dx's sum where its tiles leave more than half of the pairs idle:
// as many as all run at once, of 8 stages at least.  Counted in a GB300's 76 pairs,
// whatever the device, since the workspace's size follows from it.
constexpr int GT_PAIRS = 76;
static int parts_of(int64_t rows, int64_t cols, int64_t ff) {
    const int64_t tiles = (int64_t)tiles_of(rows, GT_TILE) * tiles_of(cols, GT_TILE), steps = 2 * (int64_t)tiles_of(ff, GT_K);
    int64_t n = tiles < GT_PAIRS ? GT_PAIRS / tiles : 1;
    if (n > steps / 8) n = steps / 8;
    return n < 2 ? 1 : (int)n;
}
static int64_t parts_ld(int64_t cols) { return (cols + 7) / 8 * 8; }
static size_t parts_bytes(int64_t rows, int64_t cols, int64_t ff) {
    const int n = parts_of(rows, cols, ff);
    return n > 1 ? (size_t)n * (size_t)rows * (size_t)parts_ld(cols) * 4 : 0;
}

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
    if (rows <= 0 || cols <= 0 || ff <= 0 || is_few(rows, cols)) return 0;
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
    if (is_few(rows, cols)) {
        FewArgs a = {x->data, gate_w->data, up_w->data, x->ld, gate_w->ld, up_w->ld, ff, (int)rows, (int)cols, (int)((cols + 7) / 8), act, {}};
        a.o[0] = Maker::out(*h, rows);
        if (gate) {
            a.o[1] = Maker::out(*gate, rows);
            a.o[2] = Maker::out(*up, rows);
        }
        const bool v8 = cols % 8 == 0 && rows_aligned(*x, rows) && rows_aligned(*gate_w, ff) && rows_aligned(*up_w, ff);
        const void* f = dt == ZERO_BF16 ? few_fn<ZERO_BF16>(few_of(rows), v8) : few_fn<ZERO_F16>(few_of(rows), v8);
        const size_t smem = (size_t)few_of(rows) * a.units * 16;
        rc = raise_smem(f, smem, me);
        if (rc != ZERO_OK) return rc;
        const int64_t blocks = (ff + 2 * (FEW_THREADS / 32) - 1) / (2 * (FEW_THREADS / 32)), most = 2 * (int64_t)sms;
        void* args[] = {&a};
        return cuda_fail(launch_after_previous(f, (int)(blocks < most ? blocks : most), FEW_THREADS, args, smem, mk.s), me);
    }
    const zero_mat X = mk.packed(*x, rows, cols), G = mk.packed(*gate_w, ff, cols), U = mk.packed(*up_w, ff, cols);
    const CUtensorMap xm = mk.map(X, rows, cols, boxes_of(rows)), gm = mk.map(G, ff, cols, GT_HALF), um = mk.map(U, ff, cols, GT_HALF);
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
    a.a_rows = boxes_of(rows);
    a.act = act;
    const int pairs = sms / 2;
    const bool alone = rows <= GT_HALF && (a.n_tiles + sms - 1) / sms < (a.n_tiles + pairs - 1) / pairs;
    mk.product(GT_FORWARD, xm, xm, gm, um, a, status, alone);
    return mk.rc;
}

size_t zero_gated_backward_workspace_bytes(const zero_mat* x, const zero_mat* gate_w, const zero_mat* up_w,
                                           const zero_mat* dgate, const zero_mat* dup, int64_t rows, int64_t cols,
                                           int64_t ff) {
    if (rows <= 0 || cols <= 0 || ff <= 0) return 0;
    return room_for(x, rows, cols) + room_for(gate_w, ff, cols) + room_for(up_w, ff, cols) + room_for(dgate, rows, ff) +
           room_for(dup, rows, ff) + (gate_w && up_w ? parts_bytes(rows, cols, ff) : 0);
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
        a.rows = rows;
        a.cols = cols;
        a.m_tiles = tiles_of(rows, GT_TILE);
        a.n_tiles = tiles_of(cols, GT_TILE);
        a.k_half = tiles_of(ff, GT_K);
        a.k_steps = 2 * a.k_half;
        a.a_rows = boxes_of(rows);
        a.split = parts_of(rows, cols, ff);
        const GatedOut to = Maker::out(*dx, rows);
        const int64_t ldp = parts_ld(cols);
        float* parts = reinterpret_cast<float*>(mk.ws);
        if (a.split > 1) mk.ws += parts_bytes(rows, cols, ff);
        a.o[0] = a.split > 1 ? GatedOut{parts, ldp, ZERO_F32, aligned(parts, 32) ? 32 : 16} : to;
        mk.product(GT_DX, mk.map(DG, rows, ff, a.a_rows), mk.map(DU, rows, ff, a.a_rows), mk.map(G, ff, cols, GT_K),
                   mk.map(U, ff, cols, GT_K), a, status);
        if (mk.rc == ZERO_OK && a.split > 1) {
            int n = a.split;
            int64_t r = rows, c = cols, ld = ldp;
            GatedOut o = to;
            void* jargs[] = {&parts, &n, &ld, &r, &c, &o};
            const int64_t all = (rows * (ldp / 4) + 255) / 256, at_once = (int64_t)sms * 8;
            mk.rc = cuda_fail(launch_after_previous((const void*)k_gated_join, (int)(all < at_once ? all : at_once), 256, jargs, 0, mk.s), me);
        }
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
