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

// dropout(x) + r of one unit, rounded to the type h is stored in: the bits of
// zero_dropout.
template <int XT, int RT, bool V8>
__device__ __forceinline__ Unit<RT, V8> drop_add_unit(const Unit<XT, V8>& x, const Unit<RT, V8>& r, bool has_r,
                                                      const DropArgs& d, uint32_t step, int64_t unit) {
    const uint4 bits = drop_bits(d, step, unit);
    Unit<RT, V8> h;
    float v[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint64_t k = drop2(x.pair(q), bits, q, d.above);
        const float2 p = unpack2(has_r ? scaled_onto2(k, d, r.pair(q)) : mul2(k, pack2(d.scale, d.scale)));
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
// (16-bit ones packed where rows are too long for that).  What is not arithmetic
// is done once a row, not once a unit: one block a row, its weights fetched for
// every 2 rows, took 58 instructions an element and 28 us (8192 x 1600 bf16; 20 us
// now).  Wide rows are bound by HBM; narrow ones by latency: 8192 x 1600 fills half
// of the issue slots, and its four warps a scheduler wait for fixed latencies, the
// row's barrier and shared memory (200 units on 64 lanes of four leave 22 % of the
// places empty).
//
// SHIFT: rows that start anywhere, or widths that are no multiple of 8.  fp32
// rows are copied by words of 4 bytes, neighbouring lanes neighbouring ones, so
// that they lie aligned in shared memory, and stored the same way from there.
// 16-bit rows are copied and stored in aligned 16-byte words: a lane takes the
// words that its unit touches and shifts them, and gives what it stores the end
// of the unit before it (from the neighbouring lane, or lane 31's last unit);
// only a warp's first and last words of a row, which it shares, go element by
// element.  Each the other way was slower (8192 x 4097, forward and backward:
// bf16 92 and 167 us, by 4 bytes 109 and 191; fp32 134 and 168, by shifts 159 and
// 224).
constexpr int LN_THREADS = 512;

__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// One matrix of a stage.  Without SHIFT, 16-bit units are one 16-byte word, copied
// and read by the same lane.  fp32 units are two, and a lane that copied its own
// two would touch every sector twice: the lanes copy neighbouring words instead,
// and read what other lanes of the warp copied.
template <int DT, int NV, bool SHIFT>
struct Lane {
    static constexpr bool F32 = DT == ZERO_F32;
    static constexpr int W = F32 ? 2 : 1, SIZE = Elem<DT>::SIZE;
    static constexpr int WORDS = NV * W * 32 + (SHIFT && !F32);              // of a warp
    static constexpr bool SHARED = SHIFT || F32;                            // lanes read what others copied
    // The byte in its first word at which a row lies in shared memory.
    static __device__ __forceinline__ int off(const char* row) {
        return SHIFT && !F32 ? (int)(reinterpret_cast<uintptr_t>(row) & 15u) : 0;
    }
    // from: the warp's first column of the row; cols: columns from there to the row's end; x: what may be read
    static __device__ __forceinline__ void copy(uint4* to, const char* from, int cols, const Extent& x) {
        const int lane = threadIdx.x & 31;
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
        if constexpr (!SHIFT) {
            const int left = cols / 8 * W - lane;
#pragma unroll
            for (int k = 0; k < NV * W; ++k)
                if (32 * k < left) copy16(at + (32 * k + lane) * 16, from + (32 * k + lane) * 16);
        } else if constexpr (F32) {
            const int left = min(cols, NV * 256) - lane;
#pragma unroll
            for (int k = 0; k < NV * 8; ++k)
                if (32 * k < left) copy4(at + (32 * k + lane) * 4, from + (32 * k + lane) * 4);
        } else {
            if (cols <= 0) return;
            const int o = off(from), words = (min(cols, NV * 256) * SIZE + o + 15) / 16, left = words - lane;
            from -= o;
            const bool edge = from < x.lo || from + words * 16 > x.hi;
#pragma unroll
            for (int k = 0; k < NV + 1; ++k)
                if (32 * k < left) {
                    const char* p = from + (32 * k + lane) * 16;
                    if (!edge || (p >= x.lo && p + 16 <= x.hi)) {
                        copy16(at + (32 * k + lane) * 16, p);
                    } else {
                        // partly outside the matrix: element by element
#pragma unroll 1
                        for (int e = 0; e < 8; ++e) {
                            const char* q = p + e * SIZE;
                            reinterpret_cast<uint16_t*>(to + 32 * k + lane)[e] =
                                q >= x.lo && q + SIZE <= x.hi ? *reinterpret_cast<const uint16_t*>(q) : (uint16_t)0;
                        }
                    }
                }
        }
    }
    // This lane's j-th unit.  SHIFT: o: off() of the row; cols: columns from the unit on, what follows reads as 0.
    static __device__ __forceinline__ Raw8<DT> read(const uint4* at, int j, int o, int cols) {
        const int lane = threadIdx.x & 31;
        Raw8<DT> v;
#pragma unroll
        for (int w = 0; w < W; ++w) v.w[w] = at[(32 * j + lane) * W + w];
        if constexpr (SHIFT) {
            uint32_t u[4 * W + 4];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                u[4 * k] = v.w[k].x;
                u[4 * k + 1] = v.w[k].y;
                u[4 * k + 2] = v.w[k].z;
                u[4 * k + 3] = v.w[k].w;
            }
            if constexpr (!F32) {
                const uint4 t = at[32 * j + lane + 1];
                u[4] = t.x;
                u[5] = t.y;
                u[6] = t.z;
                u[7] = t.w;
                shift_words<4>(u, o);
            }
            if (cols < 8)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= cols) {
                        if constexpr (F32) u[e] = 0;
                        else u[e / 2] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                    }
#pragma unroll
            for (int k = 0; k < W; ++k) v.w[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
        }
        return v;
    }
    // A unit into its lane's place: what no lane reads any more.
    static __device__ __forceinline__ void write(uint4* at, int j, const Raw8<DT>& v) {
#pragma unroll
        for (int w = 0; w < W; ++w) at[(32 * j + (threadIdx.x & 31)) * W + w] = v.w[w];
    }
};

// A warp's units of a row, stored one j after the other; the whole warp calls
// put() where any of its lanes has a unit, and with SHIFT end() at the end.
template <int DT, int NV, bool SHIFT>
struct Put {
    static constexpr bool F32 = DT == ZERO_F32;
    static constexpr int SIZE = Elem<DT>::SIZE;
    uint32_t last[4];                                                        // of the unit before: its 16 bytes
    // row: the warp's first column of it; at: the warp's part of a stage, of which no lane reads its j-th units any more; on32:
    // rows start on 32-byte boundaries; cols: columns from this lane's unit to the row's end (none: at most 0)
    __device__ __forceinline__ void put(char* row, uint4* at, int j, int cols, bool on32, const Raw8<DT>& r) {
        const int lane = threadIdx.x & 31;
        char* p = row + (32 * j + lane) * (8 * SIZE);
        if constexpr (!SHIFT) {
            if constexpr (F32) {
                if (on32) {
                    st32(p, r.w[0], r.w[1]);
                    return;
                }
            }
            st8<DT>(p, 0, r);
        } else if constexpr (F32) {
            Lane<DT, NV, SHIFT>::write(at, j, r);
        } else {
            const uint32_t v[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
            uint32_t w[8];
            const int o = (int)(reinterpret_cast<uintptr_t>(p) & 15u), cut = 8 - o / SIZE;          // elements up to the last word
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = __shfl_sync(0xFFFFFFFFu, lane == 31 ? last[i] : v[i], (lane + 31) & 31);
                last[i] = v[i];
                w[4 + i] = v[i];
            }
            if (cols <= 0) return;
            const bool whole = cols >= 8, before = j > 0 || lane > 0, after = cols >= 16 && !(j == NV - 1 && lane == 31);
            int from = 0;
            if (whole && (before || o == 0)) {
                if (o) {
                    shift_words<4>(w, 16 - o);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = v[i];
                }
                *reinterpret_cast<uint4*>(p - o) = make_uint4(w[0], w[1], w[2], w[3]);
                from = cut;
            }
            const int to = whole && after ? cut : min(cols, 8);
            if (from < to)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= from && e < to) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
        }
    }
    // cols: columns from the warp's first to the row's end
    __device__ __forceinline__ void end(char* row, const uint4* at, int cols) const {
        if constexpr (SHIFT && F32) {
            __syncwarp();
            const int lane = threadIdx.x & 31, left = min(cols, NV * 256) - lane;
            const uint32_t* u = reinterpret_cast<const uint32_t*>(at) + lane;
            uint32_t* p = reinterpret_cast<uint32_t*>(row) + lane;
#pragma unroll
            for (int k = 0; k < NV * 8; ++k)
                if (32 * k < left) p[32 * k] = u[32 * k];
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
