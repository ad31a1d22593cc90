// zero_layernorm.cuh -- the layer norm's arguments and what its forward and
// backward passes share.
#pragma once

#include "zero_drop.cuh"
#include "zero_rows.cuh"

namespace zdp {

struct LayerNormArgs {
    const void *x, *r, *w, *b;          // backward: dy, dh, w
    const void* hin;                    // backward: the stored h
    void *h, *y;                        // backward: dx, dr (either may be NULL)
    int64_t ldx, ldr, ldhin, ldh, ldy, rows;
    int cols, units;                    // units of 8 columns of a row
    float eps;
    int wdt, bdt, w_aligned, b_aligned, stages;
    int T;                              // threads that share a row (rows on 16-byte boundaries)
    int h32, y32;                       // rows of h and y start on 32-byte boundaries
    float *mean, *rstd;
    float* part;                        // backward: [grid][2][cols] partial dw and db
    int part16;                         // its rows start on 16-byte boundaries
    DropArgs drop;
};

// dropout(x) + r of one unit, rounded to the type h is stored in.
template <int XT, int RT, bool V8>
__device__ __forceinline__ Unit<RT, V8> drop_add_unit(const Unit<XT, V8>& x, const Unit<RT, V8>& r, bool has_r,
                                                      const DropArgs& d, uint32_t step, int64_t unit) {
    const uint4 bits = drop_bits(d, step, unit);
    const uint64_t s = pack2(d.scale, d.scale);
    Unit<RT, V8> h;
    float v[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint64_t k = drop2(x.pair(q), bits, q, d.above);
        const float2 p = unpack2(has_r ? fma2(k, s, r.pair(q)) : mul2(k, s));
        v[2 * q] = p.x;
        v[2 * q + 1] = p.y;
    }
    h.hold(v);
    return h;
}

// ---------------------------------------------------------------- rows that all start on 16-byte boundaries
// A block of up to 512 threads stays on its SM.  T of them (whole warps) share a
// row: G = blockDim.x / T rows are under way at a time, each with its own
// barrier.  A warp has NV * 32 neighbouring units of 8 columns, a lane every 32nd
// of them, so that the places of its NV units differ by constants.  The rows that
// follow are on their way to shared memory; weight and bias stay there, in fp32
// (16-bit ones packed where rows are too long for that).  These kernels are
// bound by the instructions they issue before HBM, so all that is not arithmetic
// is done once a row, not once a unit: one block a row, its weights fetched for
// every 2 rows, took 45 instructions an element and 28 us (8192 x 1600 bf16).
constexpr int LN_THREADS = 512;

// One matrix of a stage.  16-bit units are one 16-byte word, copied and read by
// the same lane.  fp32 units are two, and a lane that copied its own two would
// touch every sector twice: the lanes copy neighbouring words instead, and read
// what other lanes of the warp copied.
template <int DT, int NV>
struct Lane {
    static constexpr int W = DT == ZERO_F32 ? 2 : 1, WORDS = NV * W * 32;    // of a warp
    // from: the warp's first unit of the row; left: units from there to the row's end
    static __device__ __forceinline__ void copy(uint32_t at, const char* from, int left) {
        const int lane = threadIdx.x & 31;
        left = left * W - lane;
#pragma unroll
        for (int k = 0; k < NV * W; ++k)
            if (32 * k < left) copy16(at + (32 * k + lane) * 16, from + (32 * k + lane) * 16);
    }
    static __device__ __forceinline__ Raw8<DT> read(const uint4* at, int j) {
        const int lane = threadIdx.x & 31;
        Raw8<DT> v;
#pragma unroll
        for (int w = 0; w < W; ++w) v.w[w] = at[(32 * j + lane) * W + w];
        return v;
    }
};
// Eight columns of a row, an fp32 unit by one 32-byte store where its rows allow it.
template <int DT>
__device__ __forceinline__ void put8(void* row, int u, const Raw8<DT>& r, bool on32) {
    if constexpr (DT == ZERO_F32) {
        if (on32) {
            st32(static_cast<char*>(row) + (int64_t)u * 32, r.w[0], r.w[1]);
            return;
        }
    }
    st8<DT>(row, (int64_t)u * 8, r);
}
// A vector of all columns in shared memory: words w of the units side by side.
template <int WT>
struct Vector {
    static constexpr int W = WT == ZERO_F32 ? 2 : 1;
    static __device__ __forceinline__ void fill(uint4* to, const void* v, int dt, bool aligned16, int cols, int units, float none) {
        for (int u = threadIdx.x; u < units; u += blockDim.x) {
            float t[8];
            vector8(v, dt, aligned16, cols, u, none, t);
            const Raw8<WT> r = narrow8<WT>(t);
#pragma unroll
            for (int w = 0; w < W; ++w) to[w * units + u] = r.w[w];
        }
    }
    static __device__ __forceinline__ Raw8<WT> read(const uint4* from, int u, int units) {
        Raw8<WT> r;
#pragma unroll
        for (int w = 0; w < W; ++w) r.w[w] = from[w * units + u];
        return r;
    }
};
// Barrier of the T threads that share a row.
__device__ __forceinline__ void row_barrier(int group, int T) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
}

inline bool rows_on_32(const zero_mat& m, int64_t rows) {
    return aligned(m.data, 32) && (rows <= 1 || (m.ld * elem_size(m.dtype)) % 32 == 0);
}
// Threads a row, rows a block, blocks and stages.  words: 16-byte words of a
// unit of all matrices read; vectors: of all vectors.  threads 0: a row needs
// more than 512 threads, or two stages of it more than shared memory.
struct RowsShape {
    int threads, T, stages, grid;
    size_t smem;
};
inline RowsShape rows_shape(int64_t rows, int64_t cols, int nv, int words, int vectors, int sms) {
    RowsShape s = {};
    const int64_t units = cols / 8, t = (units + 32 * nv - 1) / (32 * nv) * 32;
    if (t > LN_THREADS) return s;
    s.T = (int)t;
    int64_t g = (rows + sms - 1) / sms;
    if (g > LN_THREADS / t) g = LN_THREADS / t;
    const size_t stage = (size_t)words * nv * 16 * (size_t)t;      // of one row
    const size_t fixed = (size_t)vectors * 16 * (size_t)units;
    while (g > 1 && 2 * stage * g + fixed > NORM_SM_SMEM) --g;
    if (2 * stage * g + fixed > NORM_SM_SMEM) return s;
    s.threads = (int)(g * t);
    s.stages = 2;
    while (s.stages < NORM_MAX_STAGES && (s.stages + 1) * stage * g + fixed <= NORM_SM_SMEM) ++s.stages;
    s.smem = s.stages * stage * g + fixed;
    const int64_t blocks = (rows + g - 1) / g;
    s.grid = (int)(blocks < sms ? blocks : sms);
    return s;
}

// Four units a lane, so that what is done once a row counts less (backward 16384
// x 3456 bf16 in 84 us, 92 with two); two where four leave the block fewer
// threads: rows too wide to have as many under way (backward 8192 x 8192 bf16 in
// 105 us, 129 with four; 8192 x 4096 fp32 in 86, 120), few rows, which then
// have more threads each, and rows that four a lane would leave half a warp of.
inline RowsShape rows_shape(int64_t rows, int64_t cols, int words, int vectors, int sms, int* nv) {
    const RowsShape two = rows_shape(rows, cols, 2, words, vectors, sms), four = rows_shape(rows, cols, 4, words, vectors, sms);
    *nv = cols > 512 && four.threads >= two.threads ? 4 : 2;
    return *nv == 4 ? four : two;
}

}  // namespace zdp
