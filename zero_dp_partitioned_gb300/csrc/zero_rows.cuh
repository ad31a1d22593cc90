// zero_rows.cuh -- rows walked by blocks that stay, for the norms: units of 8
// columns, the next rows on their way to shared memory, and what is computed of
// a unit at both of them.
#pragma once

#include "zero_layer.cuh"

namespace zdp {

constexpr int NORM_THREADS = 512;       // most threads that share a row
constexpr int64_t NORM_MAX_COLS = 1 << 20;
constexpr int NORM_MAX_STAGES = 4;      // rows a thread has on their way or at hand
constexpr int NORM_SM_SMEM = 216 * 1024;
constexpr int NORM_MAX_GRID = 608;      // blocks of the backward pass, each with partial sums of the weight's gradient

// Units of 8 columns (zero_layer.cuh).  V8: every row of every matrix starts on
// a 16-byte boundary and the columns are a multiple of 8.
struct Map {
    static constexpr int E = 8, LANES = 16;         // elements of a unit, lanes that share 128 columns
    // this thread's j-th unit
    static __device__ __forceinline__ int unit(int j) { return threadIdx.x + j * blockDim.x; }
    static __device__ __forceinline__ int col(int u, int e) { return u * 8 + e; }
    static __device__ __forceinline__ bool any(int u, int cols) { return u * 8 < cols; }
};

// One unit of a row, as it lies in memory.  A warp's lanes hold consecutive
// units, and call store() together.
template <int DT, bool V8>
struct Unit {
    Raw8<DT> raw;
    __device__ __forceinline__ void load(const void* row, int u, int cols, const Extent& x) {
        if (u * 8 < cols) {
            raw = V8 ? ld8<DT>(row, u * 8) : ld8_shifted<DT>(row, u * 8, cols, x);
        } else {
#pragma unroll
            for (auto& w : raw.w) w = make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ uint64_t pair(int q) const { return pair8<DT>(raw, q); }
    __device__ __forceinline__ void hold(const float (&v)[8]) { raw = narrow8<DT>(v); }
    __device__ __forceinline__ void store(void* row, int u, int cols) const {
        if constexpr (!V8) st8_shifted<DT>(row, u * 8, cols, u * 8 < cols, raw);
        else if (u * 8 < cols) st8<DT>(row, u * 8, raw);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const { widen8<DT>(raw, v); }
};

// Rows on their way: a thread copies its own units of the next rows to its own
// slots of shared memory (cp.async, 16 bytes each, past the registers and L1)
// and, where rows are aligned, waits for its own copies alone.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void copies_wait_all_but(int n) {     // n = stages - 1
    if (n == 1) copies_wait<1>();
    else if (n == 2) copies_wait<2>();
    else copies_wait<3>();
}

// One matrix of a stage: NV units a thread, each of 1 word (fp32: 2) of shared
// memory.  Where rows start anywhere, the words are the aligned ones that the
// row lies in, and one more at its end; a unit then begins in its thread's own
// words and ends in the next one's, so a barrier stands between copy and read.
template <int DT, int NV, bool V8>
struct Slots {
    static constexpr int N = DT == ZERO_F32 ? 8 : 4, W = N / 4, PER_WORD = 16 / Elem<DT>::SIZE;
    static __device__ __forceinline__ int words() { return NV * W * blockDim.x + (V8 ? 0 : 1); }
    uint4* at;                                        // the matrix's part of the stage
    // word w of this thread's j-th unit: a thread's words blockDim.x apart, or in the row's order
    static __device__ __forceinline__ int word(int j, int w) {
        return V8 ? (j * W + w) * blockDim.x + threadIdx.x : Map::unit(j) * W + w;
    }
    __device__ __forceinline__ void copy(const void* row, int cols, const Extent& x) const {
        const char* p = static_cast<const char*>(row);
        const int off = V8 ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int u = Map::unit(j);
            if (u * 8 >= cols) continue;
            const char* q = p + (int64_t)u * 8 * Elem<DT>::SIZE - off;
            const int n = V8 || (u + 1) * 8 < cols ? W : W + 1;       // the row's last unit takes the word after it too
#pragma unroll
            for (int w = 0; w < W + 1; ++w) {
                if (w >= n) break;
                uint4* to = at + word(j, w);
                if (V8 || (q + 16 * w >= x.lo && q + 16 * w + 16 <= x.hi)) {
                    copy16((uint32_t)__cvta_generic_to_shared(to), q + 16 * w);
                } else {
                    // partly outside the matrix: element by element
#pragma unroll 1
                    for (int e = 0; e < PER_WORD; ++e) {
                        const char* from = q + 16 * w + e * Elem<DT>::SIZE;
                        const bool in = from >= x.lo && from + Elem<DT>::SIZE <= x.hi;
                        if constexpr (DT == ZERO_F32)
                            reinterpret_cast<uint32_t*>(to)[e] = in ? *reinterpret_cast<const uint32_t*>(from) : 0u;
                        else
                            reinterpret_cast<uint16_t*>(to)[e] = in ? *reinterpret_cast<const uint16_t*>(from) : (uint16_t)0;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void read(Unit<DT, V8> (&u)[NV], const void* row, int cols) const {
        const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int left = cols - Map::unit(j) * 8;       // columns from this unit's first
            uint32_t w[N + 4];
#pragma unroll
            for (int k = 0; k < W + (V8 ? 0 : 1); ++k) {
                const uint4 v = left > 0 ? at[word(j, k)] : make_uint4(0, 0, 0, 0);
                w[4 * k] = v.x;
                w[4 * k + 1] = v.y;
                w[4 * k + 2] = v.z;
                w[4 * k + 3] = v.w;
            }
            if constexpr (!V8) {
                shift_words<N>(w, off);
                if (left < 8)                               // what follows the row's last column is not the row's
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e >= left) {
                            if constexpr (DT == ZERO_F32) w[e] = 0;
                            else w[e / 2] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        }
            }
#pragma unroll
            for (int k = 0; k < N / 4; ++k) u[j].raw.w[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
    }
};

template <int DT, bool V8>
__device__ __forceinline__ void store_unit(void* row, int u, int cols, const float (&v)[8]) {
    Unit<DT, V8> o;
    o.hold(v);
    o.store(row, u, cols);
}

template <int DT>
__device__ __forceinline__ const void* row_of(const void* p, int64_t ld, int64_t r) {
    return static_cast<const char*>(p) + r * ld * Elem<DT>::SIZE;
}
template <int DT>
__device__ __forceinline__ void* row_of(void* p, int64_t ld, int64_t r) {
    return static_cast<char*>(p) + r * ld * Elem<DT>::SIZE;
}

// x + r of one unit, rounded to the type h is stored in.
template <int XT, int RT, bool V8>
__device__ __forceinline__ Unit<RT, V8> add_unit(const Unit<XT, V8>& x, const Unit<RT, V8>& r, bool has_r) {
    Unit<RT, V8> h;
    uint32_t w[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 p = unpack2(has_r ? add2(x.pair(q), r.pair(q)) : x.pair(q));
        if constexpr (RT == ZERO_F32) {
            w[2 * q] = __float_as_uint(p.x);
            w[2 * q + 1] = __float_as_uint(p.y);
        } else {
            w[q] = Half16<RT>::narrow2(p.x, p.y);
        }
    }
    h.raw.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (RT == ZERO_F32) h.raw.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return h;
}

// Columns 8 u .. 8 u + 7 of a vector that every row reads (a weight), 0 past the
// end; `none` where there is no vector.
__device__ __forceinline__ void vector8(const void* w, int dt, bool aligned16, int cols, int u, float none, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = none;
    } else if (u * 8 + 8 <= cols) {
        ld8_any(w, u * 8, dt, aligned16, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = u * 8 + e < cols ? ld1_any(w, u * 8 + e, dt) : 0.f;
    }
}

// ---------------------------------------------------------------- choice of the launch
inline int words_of(int dt) { return dt == ZERO_F32 ? 2 : 1; }

// How a row is shared out: units per thread (0: the row does not fit the
// registers, or two stages of it shared memory), threads per row, blocks per
// multiprocessor, stages and their bytes.  words: 16-byte words of a unit of
// all matrices read.
struct NormShape {
    int nv, threads, per_sm, stages;
    size_t smem;
};
inline NormShape shape_of(int64_t cols, int words, int sm_threads) {
    NormShape s;
    const int64_t units = (cols + 7) / 8;
    s.nv = units <= 2 * NORM_THREADS ? 2 : units <= 4 * NORM_THREADS ? 4 : 0;
    const int64_t t = s.nv ? (units + s.nv - 1) / s.nv : NORM_THREADS;
    s.threads = (int)((t + 31) / 32 * 32);
    s.per_sm = sm_threads / s.threads < 1 ? 1 : sm_threads / s.threads;
    s.stages = 2;
    s.smem = 0;
    if (!s.nv) return s;
    const size_t stage = ((size_t)words * s.nv * s.threads + 3) * 16;      // and a word after each of up to three rows
    const int fit = (int)(NORM_SM_SMEM / (2 * stage));         // blocks with two stages each
    if (s.per_sm > fit) s.per_sm = fit < 1 ? 1 : fit;
    while (s.stages < NORM_MAX_STAGES && (s.stages + 1) * stage * s.per_sm <= NORM_SM_SMEM) ++s.stages;
    s.smem = s.stages * stage;
    if (s.smem <= NORM_SM_SMEM) return s;
    return NormShape{0, NORM_THREADS, sm_threads / NORM_THREADS, 2, 0};
}
}  // namespace zdp
