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
// barrier, and what a block keeps in registers (weights, the weights'
// gradients) it loads and writes once.  The rows that follow are on their way
// to each thread's own slots of shared memory.  Against the general form, a
// block a row and several times as many blocks: 8192 x 1600 bf16 forward 28 us
// there (weights fetched for every 2 rows, 727 instructions a warp and row).
constexpr int LN_THREADS = 512;

// One matrix of a stage: NV units a thread.  16-bit units are one 16-byte word,
// copied and read by the same thread.  fp32 units are two, and a thread that
// copied its own two would touch every sector twice: a warp's lanes copy
// neighbouring words instead, and read what other lanes copied.
template <int DT, int NV>
struct Lane {
    static constexpr int W = DT == ZERO_F32 ? 2 : 1;
    static __device__ __forceinline__ int words() { return NV * W * blockDim.x; }
    static __device__ __forceinline__ void copy(uint4* at, const void* row, int u0, int T, int units) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                // word `from` of the warp's W * 32, which is of unit u
                const int from = w * 32 + lane, u = u0 - lane + j * T + from / W;
                if (u < units)
                    copy16((uint32_t)__cvta_generic_to_shared(at + j * W * blockDim.x + (threadIdx.x - lane) * W + from),
                           static_cast<const char*>(row) + ((int64_t)(u0 - lane + j * T) * W + from) * 16);
            }
    }
    static __device__ __forceinline__ Raw8<DT> read(const uint4* at, int j, int u0, int T, int units) {
        Raw8<DT> v;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v.w[w] = u0 + j * T < units ? at[j * W * blockDim.x + threadIdx.x * W + w] : make_uint4(0, 0, 0, 0);
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
// Keeps what is computed of v's words inside the loop: the compiler would widen
// 16-bit weights once, before it, and hold twice the registers.
template <int DT>
__device__ __forceinline__ void stay_packed(Raw8<DT>& v) {
    if constexpr (DT != ZERO_F32) asm("" : "+r"(v.w[0].x), "+r"(v.w[0].y), "+r"(v.w[0].z), "+r"(v.w[0].w));
}
// Barrier of the T threads that share a row.
__device__ __forceinline__ void row_barrier(int group, int T) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
}

// Threads a row, rows a block, blocks and stages.  words: 16-byte words of a
// unit of all matrices read.  threads 0: the row does not fit NV units of 512
// threads, or two stages of it shared memory.
struct RowsShape {
    int threads, T, stages, grid;
    size_t smem;
};
inline bool rows_on_32(const zero_mat& m, int64_t rows) {
    return aligned(m.data, 32) && (rows <= 1 || (m.ld * elem_size(m.dtype)) % 32 == 0);
}
inline RowsShape rows_shape(int64_t rows, int64_t cols, int nv, int words, int sms) {
    RowsShape s = {};
    const int64_t units = cols / 8, t = ((units + nv - 1) / nv + 31) / 32 * 32;
    if (t > LN_THREADS) return s;
    s.T = (int)t;
    int64_t g = (rows + sms - 1) / sms;
    if (g > LN_THREADS / t) g = LN_THREADS / t;
    const size_t stage = (size_t)words * nv * 16 * (size_t)t;      // of one row
    while (g > 1 && 2 * stage * g > NORM_SM_SMEM) --g;
    if (2 * stage * g > NORM_SM_SMEM) return s;
    s.threads = (int)(g * t);
    s.stages = 2;
    while (s.stages < NORM_MAX_STAGES && (s.stages + 1) * stage * g <= NORM_SM_SMEM) ++s.stages;
    s.smem = s.stages * stage * g;
    const int64_t blocks = (rows + g - 1) / g;
    s.grid = (int)(blocks < sms ? blocks : sms);
    return s;
}

}  // namespace zdp
