// zero_mx4_matmul.cu -- D[m][n] = alpha * sum_k A[m][k] B[n][k] of two
// microscaled 4-bit matrices on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4, a scale for 32 elements of each operand).
//
// A persistent block per SM walks tiles of 128 rows of one operand (X) by BN
// rows of the other (Y).  Warp 0's first lane copies stages of 256 elements
// of k into shared memory (TMA tiles of 128-byte rows, 128-byte swizzle), the
// last four warps load the stage's scales ahead into registers and store them
// to tensor memory, warp 1's first lane issues the four products of a stage,
// and warps 2 to 5 read the fp32 accumulator back, scale it and store it.
//
// Measured (GB300): 8192 x 14336 x 4096 in 171 us, 5.6 PFLOP/s (2.9 times the
// measured bf16 rate).  A stage takes 850 cycles at 1.94 GHz: its four products
// need 512 (102 us if nothing else took time),
// and shared memory, from which they read 48 KB and into which the loads write
// 48 KB, 770 at 128 bytes a cycle.  So the scales go by registers: copied to
// shared memory by TMA and on by tcgen05.cp, in order with the products, they
// cost 250 cycles more a stage (232 us).  Two blocks on one tile of 256 x 256
// (cta_group::2) load two thirds of the bytes each, but took 250 us with the
// quantisation of A, where one block took 236 (both with scales by tcgen05.cp).
//
// With BN = 256 the two accumulators of 256 columns and three sets of scales
// do not fit the 512 columns of tensor memory side by side, so the accumulators
// overlap by 80 columns: a tile's epilogue reads those first and then lets
// the next tile start.
//
// X is A, and Y is B, unless A has few rows (tokens, up to 128): then X is B,
// the weights, so that the 128 rows of a tile are all used, and the accumulator
// is stored transposed.  Few tiles share their sum over k: clusters of 2 to 8
// blocks, each with a stretch of k (16 x 4096 x 14336 in 14 to 16 us, 22
// without).  One token through 14336 x 4096 takes 8 to 9 us, its 31 MB 4.6; 128
// take 16: 112 tiles of 128 rows leave a quarter of the SMs idle, and are too
// many to share k.  Rows a multiple of 128 bytes apart are the fast ones: 4096 x
// 4104 x 4104 takes 51 us where 4096 of each takes 34, and an n that is no
// multiple of 8 costs the wide stores (4096 x 4097 x 4096: 82).
//
// Every wait is bounded.  A block whose wait runs out sets bit 0 of *status,
// its roles stop, what they have in flight is waited for (bounded again), the
// tensor memory is freed, and the block leaves; D is then incomplete.
#include <cuda.h>

#include <cstdlib>
#include <mutex>

#include "zero_layer.cuh"
#include "zero_mx4.cuh"
#include "zero_tma.cuh"

namespace zdp {

constexpr int MM_THREADS = 320;
constexpr int MM_BX = 128;
constexpr int MM_KB = 128;                    // bytes of k in a stage: 256 elements
constexpr int MM_HEADER = 1024;
constexpr int MM_SF_COL = 432;                // tensor-memory column of the scales: sets of 24 columns, used by turns
constexpr int MM_SF_SET = 24, MM_SF_SETS = 3;
constexpr int MM_MAX_STAGES = 8;
constexpr int MM_EPI = 4 * 32 * 17 * 4;       // a 32 x 16 piece of D for each epilogue warp, padded
constexpr int MM_SPLIT = 8;                   // most blocks that share a tile's sum over k (the portable cluster size)

template <int BN>
struct MmShape {
    static constexpr int Y_TILES = (BN + 127) / 128;           // 128-row scale tiles of Y
    static constexpr int X_BYTES = MM_BX * MM_KB, Y_BYTES = BN * MM_KB;
    // a stage starts on 1024 bytes (the swizzle's period)
    static constexpr int STAGE = X_BYTES + Y_BYTES;
    static constexpr int FIT = (232448 - 2048 - MM_EPI) / STAGE;
    static constexpr int STAGES = FIT < MM_MAX_STAGES ? FIT : MM_MAX_STAGES;
    static constexpr int SMEM = STAGES * STAGE + 2048 + MM_EPI;
    // with the sum over k shared out, the other blocks' parts of this block's columns lie where the stages were
    static_assert((MM_SPLIT - 1) * MM_BX * (BN / MM_SPLIT) * 4 <= STAGES * STAGE, "parts fit");
    static constexpr bool OVERLAP = BN == 256;
    static constexpr int ACC1 = OVERLAP ? 176 : BN;            // column of the second accumulator
    static constexpr int EARLY = OVERLAP ? 80 : BN;            // columns read before the next tile may start
    static constexpr int SF_WORDS = 8 + 8 * Y_TILES;           // columns of a stage's scales: X, then Y
    static_assert(STAGE % 1024 == 0 && SF_WORDS <= MM_SF_SET, "layout");
};

struct MmArgs {
    const uint8_t *xs, *ys;                   // tiled scales
    void* d;
    int64_t ldd;
    int x_rows, y_rows;                       // rows of X and Y
    int x_tiles, y_tiles, k_steps;            // tiles of 128 and BN rows, stages of 256 elements
    int xs_tiles, ys_tiles;                   // 128-row tiles of scales
    int dt, swap, store;                      // store: bytes of an aligned store of D's rows (32, 16, or 0: unaligned)
    int split;                                // blocks that share a tile's sum over k
    float alpha;
    int32_t* status;
    unsigned spin_limit, drain_limit;
};

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((int)add)
        : "memory");
}
// A thread's words to its lane's consecutive columns.
__device__ __forceinline__ void tc_st8(uint32_t taddr, const uint4& a, const uint4& b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 32 lanes by 16 columns: a thread gets its lane's 16 consecutive columns.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Shared-memory descriptor of an operand tile: rows of 128 bytes in the
// 128-byte swizzle, 8 rows (1024 bytes) from one group to the next.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | 1ull << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: both operands e2m1, scales e8m0, the shape, and
// which half of a 4-byte word of scales is used.
__device__ __forceinline__ constexpr uint32_t mma_desc(int bn, int half) {
    return (uint32_t)(half * 2) << 4 | 1u << 7 | 1u << 10 | (uint32_t)(bn >> 3) << 17 | 1u << 23 |
           (uint32_t)(MM_BX >> 4) << 24 | (uint32_t)(half * 2) << 29;
}

__device__ __forceinline__ bool mm_poll(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done;
}
// A bounded wait that also ends when another role of the block has given up.
// A try suspends the thread for 1 us at most, so that SPIN_LIMIT tries end
// after a few seconds.  The lane that issues the products polls first (POLL):
// with data at hand a poll takes 25 cycles and mbarrier.try_wait 260, twice a
// stage (8192 x 14336 x 4096: 170 us, 198 without the poll).
template <bool POLL = false>
__device__ __forceinline__ bool mm_wait(uint32_t bar, uint32_t parity, unsigned limit, volatile int* stop) {
    if (POLL && limit && mm_poll(bar, parity)) return true;
#pragma unroll 1
    for (unsigned it = 0; it < limit; ++it) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if ((it & 255) == 255 && stop && *stop) return false;
    }
    return false;
}

// Tiles in order, in groups of 8 tiles of Y so that the blocks that run
// together share both operands in L2.
__device__ __forceinline__ void tile_at(const MmArgs& a, int t, int& x, int& y) {
    const int per = 8 * a.x_tiles, g = t / per, y0 = g * 8;
    const int w = min(8, a.y_tiles - y0), r = t - g * per;
    x = r / w;
    y = y0 + r % w;
}

// 16 columns of D from column y0 + col, of this lane's row xr of X: scaled,
// rounded and stored.  buf: this warp's piece of shared memory.  The whole warp
// calls it.
__device__ __forceinline__ void put16(const MmArgs& a, int64_t xr, int64_t y0, int col, int n, const uint32_t (&v)[16],
                                      float* buf) {
    const int lane = threadIdx.x & 31;
    if (a.swap) {
        // a lane holds one column of D: the warp stores 32 consecutive ones of each row
        if (xr < a.x_rows)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e < n && y0 + col + e < a.y_rows)
                    st1_any(a.d, (y0 + col + e) * a.ldd + xr, __uint_as_float(v[e]) * a.alpha, a.dt);
        return;
    }
    if (a.store && n == 16 && y0 + col + 16 <= a.y_rows) {
        if (xr >= a.x_rows) return;
        const int64_t at = xr * a.ldd + y0 + col;
        float lo[8], hi[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo[e] = __uint_as_float(v[e]) * a.alpha;
            hi[e] = __uint_as_float(v[8 + e]) * a.alpha;
        }
        if (a.dt == ZERO_F32) {
            const Raw8<ZERO_F32> l = narrow8<ZERO_F32>(lo), h = narrow8<ZERO_F32>(hi);
            if (a.store == 32) {
                st32(static_cast<float*>(a.d) + at, l.w[0], l.w[1]);
                st32(static_cast<float*>(a.d) + at + 8, h.w[0], h.w[1]);
            } else {
                st8<ZERO_F32>(a.d, at, l);
                st8<ZERO_F32>(a.d, at + 8, h);
            }
        } else {
            const uint4 l = a.dt == ZERO_BF16 ? narrow8<ZERO_BF16>(lo).w[0] : narrow8<ZERO_F16>(lo).w[0];
            const uint4 h = a.dt == ZERO_BF16 ? narrow8<ZERO_BF16>(hi).w[0] : narrow8<ZERO_F16>(hi).w[0];
            uint16_t* p = static_cast<uint16_t*>(a.d) + at;
            if (a.store == 32) {
                st32(p, l, h);
            } else {
                reinterpret_cast<uint4*>(p)[0] = l;
                reinterpret_cast<uint4*>(p)[1] = h;
            }
        }
        return;
    }
    // rows that start anywhere, and the last columns: by shared memory, 16 neighbouring columns of two rows a store
#pragma unroll
    for (int e = 0; e < 16; ++e) buf[lane * 17 + e] = __uint_as_float(v[e]) * a.alpha;
    __syncwarp();
    const int64_t c = y0 + col + (lane & 15), r0 = xr - lane;
    if ((lane & 15) < n && c < a.y_rows)
#pragma unroll 4
        for (int r = lane >> 4; r < 32; r += 2)
            if (r0 + r < a.x_rows) st1_any(a.d, (r0 + r) * a.ldd + c, buf[r * 17 + (lane & 15)], a.dt);
    __syncwarp();
}

__device__ __forceinline__ void st_remote4(uint32_t addr, const uint32_t* v) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ uint32_t remote_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

// SPLIT: a cluster of a.split blocks shares one tile, each a stretch of k; see
// the end of the kernel.
template <int BN, bool SPLIT>
__global__ void __launch_bounds__(MM_THREADS, 1)
    k_mx4_matmul(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap,
                 const __grid_constant__ MmArgs a) {
    using S = MmShape<BN>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023) & ~1023u;
    uint8_t* head = smem_raw + (base - raw);
    // header: full[8], empty[8], acc_full[2], acc_free[2], drained, sf_full[4], then the tensor-memory address, stop
    // flag and count
    const uint32_t full = base, empty = base + 64, acc_full = base + 128, acc_free = base + 144, drained = base + 160,
                   sf_full = base + 168;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(head + 200);
    volatile int* stop = reinterpret_cast<volatile int*>(head + 204);
    volatile int* loaded = reinterpret_cast<volatile int*>(head + 208);   // stages whose loads were issued
    const uint32_t stages = base + MM_HEADER;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3;                            // the 32 lanes of tensor memory this warp can reach
    float* epi = reinterpret_cast<float*>(head + MM_HEADER + S::STAGES * S::STAGE) + quarter * 32 * 17;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + 8 * s, 1);
            mbar_init(acc_free + 8 * s, 4);
        }
        for (int s = 0; s < MM_SF_SETS; ++s) mbar_init(sf_full + 8 * s, 4);
        mbar_init(drained, 1);
        fence_mbar_init();
        *stop = 0;
        *loaded = 0;
    }
    if (warp == 1)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + 200) : "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_next();

    // this block's tiles and its stretch of k
    const int rank = SPLIT ? (int)(blockIdx.x % (unsigned)a.split) : 0;
    const int first = SPLIT ? blockIdx.x / (unsigned)a.split : blockIdx.x, step = SPLIT ? a.x_tiles * a.y_tiles : gridDim.x;
    const int n_tiles = a.x_tiles * a.y_tiles, K = a.k_steps;
    const int k0 = SPLIT ? (int)((int64_t)K * rank / a.split) : 0, k1 = SPLIT ? (int)((int64_t)K * (rank + 1) / a.split) : K;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int st = 0, count = 0;
            uint32_t phase = 0;
            for (int t = first; t < n_tiles && ok; t += step) {
                int x, y;
                tile_at(a, t, x, y);
                for (int k = k0; k < k1; ++k) {
                    if (count >= S::STAGES && !mm_wait(empty + 8 * st, phase ^ 1, a.spin_limit, stop)) {
                        ok = false;
                        break;
                    }
                    // rows past the end read as 0
                    const uint32_t bar = full + 8 * st, at = stages + st * S::STAGE;
                    mbar_expect_tx(bar, S::STAGE);
                    tma_tile(at, &xmap, k * MM_KB, x * MM_BX, bar);
                    tma_tile(at + S::X_BYTES, &ymap, k * MM_KB, y * BN, bar);
                    *loaded = ++count;
                    if (++st == S::STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int st = 0, set = 0, n = 0;
            uint32_t phase = 0, set_phase = 0;
            for (int t = first; t < n_tiles && ok; t += step, ++n) {
                // the accumulator of tile n was last used by tile n - 2; overlapping ones wait for tile n - 1's first
                // columns (its epilogue began after tile n - 2's ended)
                const int need = S::OVERLAP ? n - 1 : n - 2;
                if (need >= 0 && !mm_wait<true>(acc_free + 8 * (need & 1), (need >> 1) & 1, a.spin_limit, stop)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (n & 1 ? S::ACC1 : 0);
                for (int k = k0; k < k1; ++k) {
                    if (!mm_wait<true>(sf_full + 8 * set, set_phase, a.spin_limit, stop) ||
                        !mm_wait<true>(full + 8 * st, phase, a.spin_limit, stop)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = stages + st * S::STAGE, sf = tmem + MM_SF_COL + set * MM_SF_SET;
                    const uint64_t dx = operand_desc(at), dy = operand_desc(at + S::X_BYTES);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tc_mma(d, dx + 2 * q, dy + 2 * q, mma_desc(BN, q & 1), sf + 4 * (q >> 1),
                               sf + 8 + 4 * S::Y_TILES * (q >> 1), k > k0 || q > 0);
                    tc_commit(empty + 8 * st);
                    if (++st == S::STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                    if (++set == MM_SF_SETS) {
                        set = 0;
                        set_phase ^= 1;
                    }
                }
                if (ok) tc_commit(acc_full + 8 * (n & 1));
            }
            tc_commit(drained);
        }
    } else if (warp >= 6) {
        // Stage i's scales: lane l of every quarter holds rows l, 32 + l, 64 + l and 96 + l of a tile, a word of 4 blocks
        // each, 16 bytes as they lie in the tile.  Loaded two stages ahead; a set is free when the stage that used it last is done.
        const uint32_t sf0 = tmem + MM_SF_COL + ((uint32_t)(quarter * 32) << 16);
        struct Words {
            uint4 x[2], y[2][S::Y_TILES];
        };
        int lt = first, lk = k0, lx = 0, ly = 0;              // the next stage to load
        if (lt < n_tiles) tile_at(a, lt, lx, ly);
        auto load = [&](Words& w) {
            if (lt >= n_tiles) return;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const int yt = BN >= 128 ? ly * S::Y_TILES : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w.x[h] = lx < a.xs_tiles ? __ldg(reinterpret_cast<const uint4*>(a.xs + ((int64_t)lx * K + lk) * 1024 + h * 512) + lane)
                                         : zero;
#pragma unroll
                for (int q = 0; q < S::Y_TILES; ++q)
                    w.y[h][q] = yt + q < a.ys_tiles
                                    ? __ldg(reinterpret_cast<const uint4*>(a.ys + ((int64_t)(yt + q) * K + lk) * 1024 + h * 512) + lane)
                                    : zero;
            }
            if (++lk == k1) {
                lk = k0;
                lt += step;
                if (lt < n_tiles) tile_at(a, lt, lx, ly);
            }
        };
        const int total = first < n_tiles ? ((n_tiles - 1 - first) / step + 1) * (k1 - k0) : 0;
        static_assert(S::STAGES > MM_SF_SETS, "a barrier of the ring is waited for within its turn");
        int set = 0, old = 0;                                 // the set of stage i, and the ring's place of stage i - sets
        uint32_t old_phase = 0;
        auto put = [&](int i, const Words& w) {
            if (i >= MM_SF_SETS) {
                ok = mm_wait(empty + 8 * old, old_phase, a.spin_limit, stop);
                if (++old == S::STAGES) {
                    old = 0;
                    old_phase ^= 1;
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    return false;
                }
                tc_fence_after();
            }
            const uint32_t sf = sf0 + set * MM_SF_SET;
            tc_st8(sf, w.x[0], w.x[1]);
            if constexpr (S::Y_TILES == 2) {
                tc_st8(sf + 8, w.y[0][0], w.y[0][1]);
                tc_st8(sf + 16, w.y[1][0], w.y[1][1]);
            } else {
                tc_st8(sf + 8, w.y[0][0], w.y[1][0]);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sf_full + 8 * set);
            if (++set == MM_SF_SETS) set = 0;
            return true;
        };
        Words w0, w1;
        load(w0);
        load(w1);
        for (int i = 0; i < total; i += 2) {
            if (!put(i, w0)) break;
            load(w0);
            if (i + 1 == total || !put(i + 1, w1)) break;
            load(w1);
        }
    } else if (SPLIT) {
        ok = mm_wait(acc_full, 0, a.spin_limit, stop);
        ok = __all_sync(0xFFFFFFFFu, ok);
    } else {
        int n = 0;
        for (int t = first; t < n_tiles; t += step, ++n) {
            int x, y;
            tile_at(a, t, x, y);
            const int acc = n & 1;
            ok = mm_wait(acc_full + 8 * acc, (n >> 1) & 1, a.spin_limit, stop);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + (acc ? S::ACC1 : 0) + ((uint32_t)(quarter * 32) << 16);
            const int64_t xr = (int64_t)x * MM_BX + quarter * 32 + lane;
            const int64_t y0 = (int64_t)y * BN;
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_free + 8 * acc);
            };
            int col = 0, end = BN;
            if constexpr (S::OVERLAP) {
                // the columns that the other accumulator shares first, all at once: the next tile waits for them
                uint32_t v[S::EARLY / 16][16];
                const int at = acc ? 0 : BN - S::EARLY;
#pragma unroll
                for (int c = 0; c < S::EARLY / 16; ++c) tc_ld16(d + at + 16 * c, v[c]);
                tc_wait_ld();
                release();
#pragma unroll
                for (int c = 0; c < S::EARLY / 16; ++c) put16(a, xr, y0, at + 16 * c, 16, v[c], epi);
                if (acc) col = S::EARLY;
                else end = BN - S::EARLY;
            }
#pragma unroll 1
            for (; col < end; col += 16) {
                uint32_t v[16];
                __syncwarp();
                tc_ld16(d + col, v);
                tc_wait_ld();
                if (!S::OVERLAP && col + 16 == end) release();
                put16(a, xr, y0, col, 16, v, epi);
            }
        }
    }
    if (!ok && lane == 0) {
        *stop = 1;
        atomicOr(a.status, 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // what was issued and not waited for: the products, and after a stop the loads
    if (threadIdx.x == 32) {
        mm_wait(drained, 0, a.drain_limit, nullptr);
        if (*stop)
            for (int c = max(0, *loaded - S::STAGES); c < *loaded; ++c)
                mm_wait(full + 8 * (c % S::STAGES), (uint32_t)(c / S::STAGES) & 1, a.drain_limit, nullptr);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (SPLIT) {
        // Every block of the cluster finishes BN / split of the tile's columns: it gets the others' parts of them where
        // its stages were, and adds all in the order of k, so that the sum does not depend on who comes first.
        cluster_arrive();
        cluster_wait();                        // all products and loads of the cluster are done
        tc_fence_after();
        const int own = BN / a.split;          // a multiple of 4
        const uint32_t d = tmem + ((uint32_t)(quarter * 32) << 16);
        const int row = quarter * 32 + lane;
        const bool epilogue = warp >= 2 && warp < 6;
        if (epilogue)
            for (int col = 0; col < BN; col += 16) {
                uint32_t v[16];
                __syncwarp();
                tc_ld16(d + col, v);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const int to = (col + e) / own;
                    if (to == rank) continue;
                    // this block's place among the other blocks' parts there; four columns of a row together
                    const int slot = rank < to ? rank : rank - 1, c = (col + e) - to * own;
                    st_remote4(remote_addr(stages, to) + (((slot * own + c) >> 2) * MM_BX + row) * 16, v + e);
                }
            }
        __syncwarp();
        cluster_arrive();
        cluster_wait();                        // all parts are there; no block leaves before its last one has been sent
        if (epilogue) {
            int x, y;
            tile_at(a, first, x, y);
            const float4* parts = reinterpret_cast<const float4*>(head + MM_HEADER);
            for (int col = 0; col < own; col += 16) {
                // columns c0 .. c0 + n - 1 are this block's; they lie in the 16 from base16 on, at `at`
                const int n = min(16, own - col), c0 = rank * own + col, at = c0 & 15;
                uint32_t t[16], v[16];
                __syncwarp();
                tc_ld16(d + c0 - at, t);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float4 mine = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int f = 0; f < 16; f += 4)
                        if (f == at + e)
                            mine = make_float4(__uint_as_float(t[f]), __uint_as_float(t[f + 1]), __uint_as_float(t[f + 2]),
                                               __uint_as_float(t[f + 3]));
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (e < n)
                        for (int r = 0; r < a.split; ++r) {
                            const float4 p = r == rank ? mine : parts[(((r < rank ? r : r - 1) * own + col + e) >> 2) * MM_BX + row];
                            sum.x += p.x;
                            sum.y += p.y;
                            sum.z += p.z;
                            sum.w += p.w;
                        }
                    v[e] = __float_as_uint(sum.x);
                    v[e + 1] = __float_as_uint(sum.y);
                    v[e + 2] = __float_as_uint(sum.z);
                    v[e + 3] = __float_as_uint(sum.w);
                }
                put16(a, (int64_t)x * MM_BX + row, (int64_t)y * BN, c0, n, v, epi);
            }
        }
        tc_fence_before();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

// Packed rows as bytes: boxes of 128 bytes by box_rows rows, 128-byte swizzle;
// bytes and rows past the end read as 0.
static int make_map(CUtensorMap* map, const zero_mx4& m, int box_rows) {
    EncodeFn fn = encode_fn();
    if (!fn) return fail(ZERO_ECUDA, "zero_mx4_matmul: the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t dims[2] = {(cuuint64_t)(mx4_blocks(m.cols) * 16), (cuuint64_t)m.rows}, strides[1] = {(cuuint64_t)m.ld};
    const cuuint32_t box[2] = {MM_KB, (cuuint32_t)box_rows}, step[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.data, dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ZERO_OK : fail(ZERO_ECUDA, "zero_mx4_matmul: cuTensorMapEncodeTiled failed");
}

template <int BN, bool SPLIT>
static int launch_matmul(const CUtensorMap& xm, const CUtensorMap& ym, const MmArgs& a, int grid, cudaStream_t s) {
    using S = MmShape<BN>;
    const void* f = (const void*)k_mx4_matmul<BN, SPLIT>;
    int rc = raise_smem(f, S::SMEM, "zero_mx4_matmul shared-memory size");
    if (rc != ZERO_OK) return rc;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(MM_THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    void* args[] = {const_cast<CUtensorMap*>(&xm), const_cast<CUtensorMap*>(&ym), const_cast<MmArgs*>(&a)};
    return cuda_fail(cudaLaunchKernelExC(&cfg, f, args), "zero_mx4_matmul launch");
}

template <int BN>
static int matmul(const zero_mx4& x, const zero_mx4& y, MmArgs& a, int sms, cudaStream_t s) {
    const int64_t x_tiles = (x.rows + MM_BX - 1) / MM_BX, y_tiles = (y.rows + BN - 1) / BN, tiles = x_tiles * y_tiles;
    if (tiles > INT32_MAX / 2) return fail(ZERO_ELIMIT, "zero_mx4_matmul: too many tiles");
    a.x_tiles = (int)x_tiles;
    a.y_tiles = (int)y_tiles;
    CUtensorMap xm, ym;
    int rc = make_map(&xm, x, MM_BX);
    if (rc == ZERO_OK) rc = make_map(&ym, y, BN);
    if (rc != ZERO_OK) return rc;
    // Few tiles and a long sum: blocks share it while the GPU has room for all
    // of them at once and each keeps 7 stages (clusters of 4 and 8 do not fill
    // every SM of a GPC).
    a.split = 1;
    while (a.split < MM_SPLIT && BN / (2 * a.split) >= 4 && tiles * 2 * a.split <= (a.split == 1 ? sms : sms * 5 / 6) && a.k_steps / (2 * a.split) >= 7)
        a.split *= 2;
    if (a.split > 1) return launch_matmul<BN, true>(xm, ym, a, (int)tiles * a.split, s);
    return launch_matmul<BN, false>(xm, ym, a, tiles < sms ? (int)tiles : sms, s);
}

__global__ void k_fill_zero(void* d, int64_t ld, int64_t rows, int64_t cols, int dt) {
    pdl_wait();
    pdl_launch_next();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rows * cols; i += (int64_t)gridDim.x * blockDim.x)
        st1_any(d, i / cols * ld + i % cols, 0.f, dt);
}

}  // namespace zdp

using namespace zdp;

extern "C" {

int zero_mx4_matmul(const zero_mx4* a, const zero_mx4* b, float alpha, const zero_mat* d, int32_t* status, void* stream) {
    int rc = check_mx4(a, "zero_mx4_matmul", "a");
    if (rc == ZERO_OK) rc = check_mx4(b, "zero_mx4_matmul", "b");
    if (rc != ZERO_OK) return rc;
    if (a->cols != b->cols) return fail(ZERO_EINVAL, "zero_mx4_matmul: a and b have as many columns");
    if (a->layout != ZERO_MX4_TILES || b->layout != ZERO_MX4_TILES)
        return fail(ZERO_EINVAL, "zero_mx4_matmul: scales in ZERO_MX4_TILES (zero_mx4_tile_scales)");
    if (a->rows > INT32_MAX / 2 || b->rows > INT32_MAX / 2 || a->cols > INT32_MAX / 2)
        return fail(ZERO_ELIMIT, "zero_mx4_matmul: more than 2^30 rows or columns");
    rc = check_mat(d, a->rows, b->rows, FLOAT_TYPES, "zero_mx4_matmul", "d");
    if (rc != ZERO_OK) return rc;
    if (!status || !aligned(status, 4)) return fail(ZERO_EINVAL, "zero_mx4_matmul: status NULL or not 4-byte aligned");
    if (!(alpha - alpha == 0.f)) return fail(ZERO_EINVAL, "zero_mx4_matmul: alpha must be finite");
    if (a->rows == 0 || b->rows == 0) return ZERO_OK;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->cols == 0) {                      // a sum of nothing
        void* dp = d->data;
        int64_t ld = d->ld, rows = a->rows, cols = b->rows;
        int dt = d->dtype;
        void* args[] = {&dp, &ld, &rows, &cols, &dt};
        return cuda_fail(launch_after_previous((const void*)k_fill_zero, sms * 4, 256, args, 0, s), "zero_mx4_matmul launch");
    }
    MmArgs m = {};
    m.swap = a->rows <= 128;
    const zero_mx4 &x = m.swap ? *b : *a, &y = m.swap ? *a : *b;
    m.xs = static_cast<const uint8_t*>(x.scales);
    m.ys = static_cast<const uint8_t*>(y.scales);
    m.xs_tiles = (int)((x.rows + 127) / 128);
    m.ys_tiles = (int)((y.rows + 127) / 128);
    m.d = d->data;
    m.ldd = d->ld;
    m.x_rows = (int)x.rows;
    m.y_rows = (int)y.rows;
    m.k_steps = (int)((a->cols + 255) / 256);
    m.dt = d->dtype;
    const auto rows_on = [&](int n) { return aligned(d->data, n) && (a->rows == 1 || d->ld * elem_size(d->dtype) % n == 0); };
    m.store = rows_on(32) ? 32 : rows_on(16) ? 16 : 0;
    m.alpha = alpha;
    m.status = status;
    const char* e = std::getenv("ZERO_GB300_SPIN_LIMIT");
    m.spin_limit = e ? (unsigned)std::strtoul(e, nullptr, 10) : SPIN_LIMIT;
    m.drain_limit = SPIN_LIMIT;
    if (!m.swap) {
        // 256 columns a tile, or 128 where that gives more tiles in as many rounds: a tile of 128 columns takes 0.9 of the
        // time (4001 x 1600 x 6400: three rounds of them 33.6 us, two of 256 columns 24.9)
        const int64_t xt = (x.rows + MM_BX - 1) / MM_BX;
        const auto rounds = [&](int bn) { return (xt * ((y.rows + bn - 1) / bn) + sms - 1) / sms; };
        return rounds(256) * 10 <= rounds(128) * 9 ? matmul<256>(x, y, m, sms, s) : matmul<128>(x, y, m, sms, s);
    }
    if (y.rows <= 16) return matmul<16>(x, y, m, sms, s);
    if (y.rows <= 64) return matmul<64>(x, y, m, sms, s);
    return matmul<128>(x, y, m, sms, s);
}

}  // extern "C"
