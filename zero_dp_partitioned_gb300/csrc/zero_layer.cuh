// zero_layer.cuh -- what the layer operators (norm, distillation, 4-bit
// matrices) share: element types, row access of any alignment, block
// reductions, and the host checks of a zero_mat.
//
// A row is walked in units of 8 consecutive elements, the units of a warp's
// lanes one after another: 128 consecutive columns belong to 16 lanes.  Where
// every row of every matrix starts on a 16-byte boundary a unit is one 16-byte
// access (two for fp32).  Rows that start anywhere are still read and written
// in aligned 16-byte words: a load takes the two words that a unit touches and
// shifts them, a store takes the unit before it from the neighbouring lane;
// only the ends of a row, and of a warp, go element by element.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zdp {

template <int DT> struct Elem;
template <> struct Elem<ZERO_F16> { static constexpr int SIZE = 2; };
template <> struct Elem<ZERO_BF16> { static constexpr int SIZE = 2; };
template <> struct Elem<ZERO_F32> { static constexpr int SIZE = 4; };

__host__ __device__ __forceinline__ int elem_size(int dt) {
    return dt == ZERO_F32 || dt == ZERO_I32 ? 4 : dt == ZERO_I64 ? 8 : dt == ZERO_E4M3 ? 1 : 2;
}

// ---------------------------------------------------------------- elements
template <int DT>
__device__ __forceinline__ float ld1(const void* p, int64_t i) {
    if constexpr (DT == ZERO_F32) return static_cast<const float*>(p)[i];
    else return Half16<DT>::widen(static_cast<const uint16_t*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void st1(void* p, int64_t i, float v) {
    if constexpr (DT == ZERO_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)Half16<DT>::narrow(v);
}
__device__ __forceinline__ float ld1_any(const void* p, int64_t i, int dt) {
    return dt == ZERO_F32 ? ld1<ZERO_F32>(p, i) : dt == ZERO_BF16 ? ld1<ZERO_BF16>(p, i) : ld1<ZERO_F16>(p, i);
}
__device__ __forceinline__ void st1_any(void* p, int64_t i, float v, int dt) {
    if (dt == ZERO_F32) st1<ZERO_F32>(p, i, v);
    else if (dt == ZERO_BF16) st1<ZERO_BF16>(p, i, v);
    else st1<ZERO_F16>(p, i, v);
}

// Eight packed elements as they lie in memory: one 16-byte word, or two.
template <int DT> struct Raw8 { uint4 w[DT == ZERO_F32 ? 2 : 1]; };

template <int DT>
__device__ __forceinline__ Raw8<DT> ld8(const void* p, int64_t i) {
    Raw8<DT> r;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * Elem<DT>::SIZE);
    r.w[0] = q[0];
    if constexpr (DT == ZERO_F32) r.w[1] = q[1];
    return r;
}
template <int DT>
__device__ __forceinline__ Raw8<DT> ld8_stream(const void* p, int64_t i) {
    Raw8<DT> r;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * Elem<DT>::SIZE);
    r.w[0] = __ldcs(q);
    if constexpr (DT == ZERO_F32) r.w[1] = __ldcs(q + 1);
    return r;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&v)[8]) {
    if constexpr (DT == ZERO_F32) {
        const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
    } else {
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = Half16<DT>::widen(u[q] & 0xFFFFu);
            v[2 * q + 1] = Half16<DT>::widen(u[q] >> 16);
        }
    }
}
template <int DT>
__device__ __forceinline__ Raw8<DT> narrow8(const float (&v)[8]) {
    Raw8<DT> r;
    if constexpr (DT == ZERO_F32) {
        r.w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        r.w[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
        r.w[0] = make_uint4(Half16<DT>::narrow2(v[0], v[1]), Half16<DT>::narrow2(v[2], v[3]),
                            Half16<DT>::narrow2(v[4], v[5]), Half16<DT>::narrow2(v[6], v[7]));
    }
    return r;
}
template <int DT>
__device__ __forceinline__ void st8(void* p, int64_t i, const Raw8<DT>& r) {
    uint4* q = reinterpret_cast<uint4*>(static_cast<char*>(p) + i * Elem<DT>::SIZE);
    q[0] = r.w[0];
    if constexpr (DT == ZERO_F32) q[1] = r.w[1];
}
// 32 bytes to global memory, 32-byte aligned: a whole sector a lane.
__device__ __forceinline__ void st32(void* p, const uint4& lo, const uint4& hi) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w),
                 "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                 : "memory");
}

// Eight elements of a vector that other rows read too (a weight), whatever its alignment.
__device__ __forceinline__ void ld8_any(const void* p, int64_t i, int dt, bool aligned16, float (&v)[8]) {
    if (!aligned16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = ld1_any(p, i + e, dt);
    } else if (dt == ZERO_F32) {
        widen8<ZERO_F32>(ld8<ZERO_F32>(p, i), v);
    } else if (dt == ZERO_BF16) {
        widen8<ZERO_BF16>(ld8<ZERO_BF16>(p, i), v);
    } else {
        widen8<ZERO_F16>(ld8<ZERO_F16>(p, i), v);
    }
}

// ---------------------------------------------------------------- rows that start anywhere
// N words from byte `by` (below 16) of the words w[0 .. N + 3].  `by` is the
// same for a whole row, so the branches do not diverge.
template <int N>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N + 4], int by) {
    if (by & 8)
#pragma unroll
        for (int i = 0; i < N + 2; ++i) w[i] = w[i + 2];
    if (by & 4)
#pragma unroll
        for (int i = 0; i < N + 1; ++i) w[i] = w[i + 1];
    if (by & 3)
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (by & 3));
}

// The bytes a matrix occupies, first row to last element: no access leaves them.
struct Extent {
    const char *lo, *hi;
};
template <int DT>
__device__ __forceinline__ Extent extent_of(const void* p, int64_t ld, int64_t rows, int64_t cols) {
    return Extent{static_cast<const char*>(p), static_cast<const char*>(p) + ((rows - 1) * ld + cols) * Elem<DT>::SIZE};
}

// 8 elements of a row from column c (a multiple of 8); columns past the end are 0.
template <int DT>
__device__ __forceinline__ Raw8<DT> ld8_shifted(const void* row, int64_t c, int64_t cols, const Extent& x) {
    constexpr int N = DT == ZERO_F32 ? 8 : 4;
    const char* p = static_cast<const char*>(row) + c * Elem<DT>::SIZE;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
    const char* q = p - off;
    Raw8<DT> r;
    if (c + 8 <= cols && q >= x.lo && q + 4 * N + 16 <= x.hi) {
        uint32_t w[N + 4];
#pragma unroll
        for (int k = 0; k < N / 4 + 1; ++k) {
            const uint4 u = reinterpret_cast<const uint4*>(q)[k];
            w[4 * k] = u.x;
            w[4 * k + 1] = u.y;
            w[4 * k + 2] = u.z;
            w[4 * k + 3] = u.w;
        }
        shift_words<N>(w, off);
#pragma unroll
        for (int k = 0; k < N / 4; ++k) r.w[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    } else {
        uint32_t w[N] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < cols) {
                if constexpr (DT == ZERO_F32) w[e] = reinterpret_cast<const uint32_t*>(p)[e];
                else w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
            }
#pragma unroll
        for (int k = 0; k < N / 4; ++k) r.w[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    return r;
}

// A unit of 8 elements of SIZE bytes (N words) to column c of a row that starts
// anywhere.  The whole warp calls it, its lanes with consecutive units; `here`:
// this lane's unit is to be written (its columns below cols).  A lane writes
// the aligned words that end in its unit, with what the lane before has of
// them, and what no lane after it will write.
template <int SIZE, int N>
__device__ __forceinline__ void st_shifted(void* row, int64_t c, int64_t cols, bool here, const uint32_t (&v)[N]) {
    constexpr int G = N < 4 ? N : 4;                           // words of an aligned store
    char* p = static_cast<char*>(row) + c * SIZE;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & (4 * G - 1));
    const int lane = threadIdx.x & 31;
    const bool whole = here && c + 8 <= cols;
    uint32_t w[N + 4];
    if constexpr (G == 2) w[0] = w[1] = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) w[4 - G + i] = __shfl_up_sync(0xFFFFFFFFu, v[N - G + i], 1);
#pragma unroll
    for (int i = 0; i < N; ++i) w[4 + i] = v[i];
    const bool before = __shfl_up_sync(0xFFFFFFFFu, (int)whole, 1) && lane > 0;
    const bool after = __shfl_down_sync(0xFFFFFFFFu, (int)whole, 1) && lane < 31;
    if (!here) return;
    int from = 0, to = (int)(cols - c < 8 ? cols - c : 8);     // elements still to be written one by one
    if (whole && (before || off == 0)) {
        if (off) {
            // words from byte 16 - off of (the lane before's last G words at 4 - G, own words at 4)
            if constexpr (G == 4) {
                shift_words<N>(w, 16 - off);
            } else {
                // 8-byte words: from byte 16 - off, off below 8, so past w[2]
                uint32_t t[N + 4] = {w[2], w[3], w[4], w[5]};
                shift_words<N>(t, 8 - off);
                w[0] = t[0];
                w[1] = t[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = v[i];
        }
        if constexpr (G == 4) {
#pragma unroll
            for (int k = 0; k < N / 4; ++k)
                reinterpret_cast<uint4*>(p - off)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        } else {
            *reinterpret_cast<uint2*>(p - off) = make_uint2(w[0], w[1]);
        }
        from = 8 - off / SIZE;
    }
    if (whole && after) to = 8 - off / SIZE;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= from && e < to) {
            if constexpr (SIZE == 4) reinterpret_cast<uint32_t*>(p)[e] = v[e];
            else if constexpr (SIZE == 2) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
            else reinterpret_cast<uint8_t*>(p)[e] = (uint8_t)(v[e / 4] >> (8 * (e & 3)));
        }
}
template <int DT>
__device__ __forceinline__ void st8_shifted(void* row, int64_t c, int64_t cols, bool here, const Raw8<DT>& r) {
    constexpr int N = DT == ZERO_F32 ? 8 : 4;
    uint32_t v[N];
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
        v[4 * k] = r.w[k].x;
        v[4 * k + 1] = r.w[k].y;
        v[4 * k + 2] = r.w[k].z;
        v[4 * k + 3] = r.w[k].w;
    }
    st_shifted<Elem<DT>::SIZE, N>(row, c, cols, here, v);
}

// ---------------------------------------------------------------- pairs
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// elements 2 q and 2 q + 1 of eight packed ones, as fp32
template <int DT>
__device__ __forceinline__ uint64_t pair8(const Raw8<DT>& r, int q) {
    if constexpr (DT == ZERO_F32) {
        const uint4 w = r.w[q / 2];
        return q % 2 ? pack2(__uint_as_float(w.z), __uint_as_float(w.w)) : pack2(__uint_as_float(w.x), __uint_as_float(w.y));
    } else {
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
        if constexpr (DT == ZERO_BF16) return pack2(__uint_as_float(u[q] << 16), __uint_as_float(u[q] & 0xFFFF0000u));
        else return pack2(Half16<DT>::widen(u[q] & 0xFFFFu), Half16<DT>::widen(u[q] >> 16));
    }
}

// a / b of numbers that are not negative, in 32 bits where both have no more: a
// division in 64 costs about a hundred instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// ---------------------------------------------------------------- reductions
// The largest of three that keeps a NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// |x| as an unsigned integer orders as |x| does, with NaN above infinity: the
// largest of a block keeps a NaN, where fmaxf would drop it.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The block's sum, the same in every thread and every run (a butterfly in
// each warp, then the warps in order).  s: 32 floats of shared memory, 16-byte
// aligned, that no call in flight uses, zero beyond the block's warps; the
// caller alternates two of them between calls.
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    if (blockDim.x <= 32) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int n4 = (blockDim.x + 127) >> 7;
    float t = 0.f;
    for (int w = 0; w < n4; ++w) {
        const float4 p = reinterpret_cast<const float4*>(s)[w];
        t += (p.x + p.y) + (p.z + p.w);
    }
    return t;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* s) {
    v = lanes_max<32>(v);
    if (blockDim.x <= 32) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    uint32_t t = 0;
    for (int w = 0; w < nw; ++w) t = max(t, s[w]);
    return t;
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// ---------------------------------------------------------------- host
// A matrix argument: not NULL, one of the types in `types` (a bit per code),
// rows at least `cols` apart, aligned to its element.
int check_mat(const zero_mat* m, int64_t rows, int64_t cols, unsigned types, const char* call, const char* what);
// Sets the message "call: what" + why and returns code.
int refuse(int code, const char* call, const char* what, const char* why);
constexpr unsigned FLOAT_TYPES = 1u << ZERO_F16 | 1u << ZERO_BF16 | 1u << ZERO_F32;
// Whether every row starts on a 16-byte boundary.
inline bool rows_aligned(const zero_mat& m, int64_t rows) {
    return aligned(m.data, 16) && (rows <= 1 || (m.ld * elem_size(m.dtype)) % 16 == 0);
}
// Raises a kernel's limit of dynamic shared memory on the current device to
// `smem` where it is lower (asked of the driver once).
int raise_smem(const void* f, size_t smem, const char* who);
// SM count of the current device (0 and an error message if it cannot be had).
int sm_count();

}  // namespace zdp
