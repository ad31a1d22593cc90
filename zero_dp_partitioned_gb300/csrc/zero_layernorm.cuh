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
    int T;                              // threads that share a row
    int h32, y32;                       // rows of h and y start on 32-byte boundaries (no SHIFT)
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

// ---------------------------------------------------------------- blocks that stay
// A block of up to 512 threads stays on its SM.  T of them (whole warps) share a
// row: G = blockDim.x / T rows are under way at a time, each with its own
// barrier.  A warp has NV * 32 neighbouring units of 8 columns, a lane every 32nd
// of them, so that the places of its NV units differ by constants.  The rows that
// follow are on their way to shared memory; weight and bias stay there, in fp32
// (16-bit ones packed where rows are too long for that).  These kernels are
// bound by the instructions they issue before HBM, so all that is not arithmetic
// is done once a row, not once a unit: one block a row, its weights fetched for
// every 2 rows, took 45 instructions an element and 28 us (8192 x 1600 bf16).
//
// SHIFT: rows that start anywhere, or widths that are no multiple of 8.  Memory
// is still read and written in aligned 16-byte words: a warp copies the words
// that its columns lie in, a lane takes the words that its unit touches and
// shifts them, and gives what it stores the end of the unit before it (from the
// neighbouring lane, or lane 31's last unit); only a warp's first and last
// words of a row, which it shares, go element by element.
constexpr int LN_THREADS = 512;

// One matrix of a stage.  Without SHIFT, 16-bit units are one 16-byte word, copied
// and read by the same lane.  fp32 units are two, and a lane that copied its own
// two would touch every sector twice: the lanes copy neighbouring words instead,
// and read what other lanes of the warp copied.
template <int DT, int NV, bool SHIFT>
struct Lane {
    static constexpr int W = DT == ZERO_F32 ? 2 : 1, N = 4 * W, SIZE = Elem<DT>::SIZE;
    static constexpr int WORDS = NV * W * 32 + SHIFT;                        // of a warp
    static constexpr bool SHARED = SHIFT || DT == ZERO_F32;                 // lanes read what others copied
    // from: the warp's first column of the row; cols: columns from there to the row's end; x: what may be read
    static __device__ __forceinline__ void copy(uint4* to, const char* from, int cols, const Extent& x) {
        const int lane = threadIdx.x & 31;
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
        if (!SHIFT) {
            const int left = cols / 8 * W - lane;
#pragma unroll
            for (int k = 0; k < NV * W; ++k)
                if (32 * k < left) copy16(at + (32 * k + lane) * 16, from + (32 * k + lane) * 16);
            return;
        }
        if (cols <= 0) return;
        const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15u), all = min(cols, NV * 256) * SIZE + off;
        const int words = (all + 15) / 16, left = words - lane;              // words from this lane's first
        from -= off;
        const bool edge = from < x.lo || from + words * 16 > x.hi;
#pragma unroll
        for (int k = 0; k < NV * W + 1; ++k)
            if (32 * k < left) {
                const char* p = from + (32 * k + lane) * 16;
                if (!edge || (p >= x.lo && p + 16 <= x.hi)) {
                    copy16(at + (32 * k + lane) * 16, p);
                } else {
                    // partly outside the matrix: element by element
#pragma unroll 1
                    for (int e = 0; e < 16 / SIZE; ++e) {
                        const char* q = p + e * SIZE;
                        const bool in = q >= x.lo && q + SIZE <= x.hi;
                        if constexpr (DT == ZERO_F32)
                            reinterpret_cast<uint32_t*>(to + 32 * k + lane)[e] = in ? *reinterpret_cast<const uint32_t*>(q) : 0u;
                        else
                            reinterpret_cast<uint16_t*>(to + 32 * k + lane)[e] = in ? *reinterpret_cast<const uint16_t*>(q) : (uint16_t)0;
                    }
                }
            }
    }
    // This lane's j-th unit.  SHIFT: off: the row's byte in its first word; cols: columns from the unit on, what follows reads as 0.
    static __device__ __forceinline__ Raw8<DT> read(const uint4* at, int j, int off, int cols) {
        const int lane = threadIdx.x & 31;
        Raw8<DT> v;
        if constexpr (!SHIFT) {
#pragma unroll
            for (int w = 0; w < W; ++w) v.w[w] = at[(32 * j + lane) * W + w];
        } else {
            uint32_t u[N + 4];
#pragma unroll
            for (int k = 0; k < W + 1; ++k) {
                const uint4 t = at[(32 * j + lane) * W + k];
                u[4 * k] = t.x;
                u[4 * k + 1] = t.y;
                u[4 * k + 2] = t.z;
                u[4 * k + 3] = t.w;
            }
            shift_words<N>(u, off);
            if (cols < 8)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= cols) {
                        if constexpr (DT == ZERO_F32) u[e] = 0;
                        else u[e / 2] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                    }
#pragma unroll
            for (int k = 0; k < W; ++k) v.w[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
        }
        return v;
    }
    // The unit shifted into place, in the stead of what read() took; all lanes have read their j-th (and no earlier) before.
    static __device__ __forceinline__ void write(uint4* at, int j, const Raw8<DT>& v) {
#pragma unroll
        for (int w = 0; w < W; ++w) at[(32 * j + (threadIdx.x & 31)) * W + w] = v.w[w];
    }
};

// A warp's units of a row, stored one j after the other; the whole warp calls
// put() where any of its lanes has a unit.
template <int DT, bool SHIFT>
struct Put {
    static constexpr int N = DT == ZERO_F32 ? 8 : 4, SIZE = Elem<DT>::SIZE;
    uint32_t last[4];                                                        // of the unit before: its last 16 bytes
    // row: the warp's first column of it; on32: rows start on 32-byte boundaries; cols: columns from this lane's unit to the
    // row's end (none: at most 0); lasts: the warp's last j
    __device__ __forceinline__ void put(char* row, int j, int cols, bool on32, bool lasts, const Raw8<DT>& r) {
        const int lane = threadIdx.x & 31;
        if constexpr (!SHIFT) {
            if (cols <= 0) return;
            char* p = row + (32 * j + lane) * (8 * SIZE);
            if constexpr (DT == ZERO_F32) {
                if (on32) {
                    st32(p, r.w[0], r.w[1]);
                    return;
                }
            }
            st8<DT>(p, 0, r);
        } else {
            uint32_t v[N], w[N + 4];
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                v[4 * k] = r.w[k].x;
                v[4 * k + 1] = r.w[k].y;
                v[4 * k + 2] = r.w[k].z;
                v[4 * k + 3] = r.w[k].w;
            }
            char* p = row + (32 * j + lane) * (8 * SIZE);
            const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u), cut = 8 - off / SIZE;      // elements up to the last word
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = __shfl_sync(0xFFFFFFFFu, lane == 31 ? last[i] : v[N - 4 + i], (lane + 31) & 31);
                last[i] = v[N - 4 + i];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) w[4 + i] = v[i];
            if (cols <= 0) return;
            const bool whole = cols >= 8, before = j > 0 || lane > 0, after = cols >= 16 && !(lasts && lane == 31);
            int from = 0;
            if (whole && (before || off == 0)) {
                if (off) {
                    shift_words<N>(w, 16 - off);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) w[i] = v[i];
                }
#pragma unroll
                for (int k = 0; k < N / 4; ++k)
                    reinterpret_cast<uint4*>(p - off)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                from = cut;
            }
            const int to = whole && after ? cut : min(cols, 8);
            if (from < to)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= from && e < to) {
                        if constexpr (DT == ZERO_F32) reinterpret_cast<uint32_t*>(p)[e] = v[e];
                        else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
                    }
        }
    }
};
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
    const int64_t units = (cols + 7) / 8, t = (units + 32 * nv - 1) / (32 * nv) * 32;
    if (t > LN_THREADS) return s;
    s.T = (int)t;
    int64_t g = (rows + sms - 1) / sms;
    if (g > LN_THREADS / t) g = LN_THREADS / t;
    const size_t stage = ((size_t)words * nv * 32 + 3) * 16 * (size_t)(t / 32);      // of one row; a word after each of up to three matrices
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
