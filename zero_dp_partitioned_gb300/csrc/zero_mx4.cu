// zero_mx4.cu -- quantising to microscaled 4 bits, the values back, and the
// tiling of scales that were gathered row by row.
//
// A block's scale is 2^(floor(log2 max|x|) - 2), so that its largest value
// lands in [4, 8) and is clipped at e2m1's 6; the values are rounded to
// nearest, ties to even.  Scaling by a power of two is exact, so the result
// does not depend on the order or the precision of the arithmetic.  A block
// that holds an infinity or a NaN gets the scale NaN (255) and stays visible
// to the overflow check of the step that its gradients end in.
//
// Bound: HBM.  Along the rows 8 consecutive elements go to a thread and 4
// lanes share a block.  Along the columns (the operand of a product that sums
// over rows) a warp takes 32 rows by 64 columns, quantises the rows from its
// registers, and the columns from its own piece of shared memory, two to a
// lane: both forms from one read of the matrix.
#include "zero_layer.cuh"
#include "zero_mx4.cuh"

namespace zdp {

constexpr int MX4_THREADS = 256;

struct Mx4Dev {
    uint8_t *data, *scales;
    int64_t ld, blocks, tiles;
    int tiled;
};

struct QuantArgs {
    const void* src;
    int64_t ld, rows, cols;
    int aligned16;
    Mx4Dev q, t;           // along the rows, along the columns (data NULL: not wanted)
};

__device__ __forceinline__ uint32_t mx4_scale(uint32_t top) {
    const int e = (int)(top >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
// 2^-(byte - 127), exact for every byte a scale can have but NaN
__device__ __forceinline__ float mx4_inverse(uint32_t byte) { return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23); }
__device__ __forceinline__ float mx4_value(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Eight scaled values to eight 4-bit codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t to_e2m1(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Two codes of one byte to fp32.
__device__ __forceinline__ float2 from_e2m1(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 b, x, y, z;\n\tmov.b32 {b, x, y, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 8 elements of a row from column c; columns past the end are 0.
template <int DT>
__device__ __forceinline__ void read8(const void* row, int64_t c, int64_t cols, bool vec, float (&v)[8]) {
    if (vec && c + 8 <= cols) {
        widen8<DT>(ld8_stream<DT>(row, c), v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? ld1<DT>(row, c + e) : 0.f;
    }
}

__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = max(t, abs_bits(v[e]));
    return t;
}

// Along the rows.  A warp takes 256 columns of a row (8 blocks, a step of the
// product's tiles); rows and columns of the scales' padding are walked too.
template <int DT>
__global__ void __launch_bounds__(MX4_THREADS) k_mx4_rows(const __grid_constant__ QuantArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int64_t rows = a.q.tiled ? (a.rows + 127) / 128 * 128 : a.rows;
    const int64_t per = (a.cols + 255) / 256, n = rows * per;
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * (MX4_THREADS / 32);
    for (int64_t i = (int64_t)blockIdx.x * (MX4_THREADS / 32) + (threadIdx.x >> 5); i < n; i += stride) {
        const int64_t r = i / per, c = (i - r * per) * 256 + lane * 8, b = c >> 5;
        float v[8];
        if (r < a.rows) {
            read8<DT>(static_cast<const char*>(a.src) + r * a.ld * Elem<DT>::SIZE, c, a.cols, a.aligned16, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        }
        const uint32_t byte = mx4_scale(lanes_max<4>(top8(v)));
        const float inv = mx4_inverse(byte);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= inv;
        if (r < a.rows && b < a.q.blocks)
            *reinterpret_cast<uint32_t*>(a.q.data + r * a.q.ld + c / 2) = to_e2m1(v);
        // the 4 blocks of 16 lanes make one word of a tile
        uint32_t word = byte << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
        if (a.q.tiled) {
            if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(a.q.scales + mx4_tiled_at(r, b, a.q.tiles)) = word;
        } else if ((lane & 3) == 0 && b < a.q.blocks) {
            a.q.scales[r * a.q.blocks + b] = (uint8_t)byte;
        }
    }
}

__device__ __forceinline__ void put_scale(const Mx4Dev& q, int64_t r, int64_t rows, int64_t b, uint32_t byte) {
    if (q.tiled) {
        if (r < (rows + 127) / 128 * 128 && b < q.tiles * 4) q.scales[mx4_tiled_at(r, b, q.tiles)] = (uint8_t)byte;
    } else if (r < rows && b < q.blocks) {
        q.scales[r * q.blocks + b] = (uint8_t)byte;
    }
}

// Along the columns, and along the rows too if they are wanted.
template <int DT>
__global__ void __launch_bounds__(128) k_mx4_both(const __grid_constant__ QuantArgs a) {
    __shared__ __align__(16) float tile[4][DT == ZERO_F32 ? 32 * 64 : 32 * 32];
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a block's 4 warps take 128 rows; both directions are padded to 256 for the scales
    const int64_t nr = (a.rows + 255) / 256 * 2, nc = (a.cols + 255) / 256 * 4;
    for (int64_t i = blockIdx.x; i < nr * nc; i += gridDim.x) {
        const int64_t r0 = (i / nc) * 128 + warp * 32, c0 = (i % nc) * 64;
        float* s = tile[warp];
        const int64_t c = c0 + (lane & 7) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int rr = k * 4 + (lane >> 3);
            const int64_t r = r0 + rr;
            float v[8];
            if (r < a.rows && c < a.cols) {
                read8<DT>(static_cast<const char*>(a.src) + r * a.ld * Elem<DT>::SIZE, c, a.cols, a.aligned16, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0.f;
            }
            if (a.t.data) st8<DT>(s, rr * 64 + (lane & 7) * 8, narrow8<DT>(v));
            if (a.q.data) {
                const uint32_t byte = mx4_scale(lanes_max<4>(top8(v)));
                const float inv = mx4_inverse(byte);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= inv;
                if (r < a.rows && c / 32 < a.q.blocks)
                    *reinterpret_cast<uint32_t*>(a.q.data + r * a.q.ld + c / 2) = to_e2m1(v);
                if ((lane & 3) == 0) put_scale(a.q, r, a.rows, c / 32, byte);
            }
        }
        __syncwarp();
        if (a.t.data) {
            // columns c0 + 2 lane and the next, 32 rows: one block of each
            float v[2][32];
            uint32_t top[2] = {0, 0};
#pragma unroll
            for (int rr = 0; rr < 32; ++rr) {
                if constexpr (DT == ZERO_F32) {
                    const float2 p = reinterpret_cast<const float2*>(s)[rr * 32 + lane];
                    v[0][rr] = p.x;
                    v[1][rr] = p.y;
                } else {
                    const uint32_t p = reinterpret_cast<const uint32_t*>(s)[rr * 32 + lane];
                    v[0][rr] = Half16<DT>::widen(p & 0xFFFFu);
                    v[1][rr] = Half16<DT>::widen(p >> 16);
                }
                top[0] = max(top[0], abs_bits(v[0][rr]));
                top[1] = max(top[1], abs_bits(v[1][rr]));
            }
            const int64_t b = r0 / 32;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t col = c0 + 2 * lane + h;
                const uint32_t byte = mx4_scale(top[h]);
                const float inv = mx4_inverse(byte);
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = v[h][q * 8 + e] * inv;
                    w[q] = to_e2m1(x);
                }
                if (col < a.cols && b < a.t.blocks)
                    *reinterpret_cast<uint4*>(a.t.data + col * a.t.ld + b * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                put_scale(a.t, col, a.cols, b, byte);
            }
        }
        __syncwarp();
    }
}

struct DequantArgs {
    Mx4Dev q;
    void* dst;
    int64_t ld, rows, cols;
    int aligned16;
};

template <int DT>
__global__ void __launch_bounds__(MX4_THREADS) k_mx4_values(const __grid_constant__ DequantArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int64_t per = (a.cols + 7) / 8, n = a.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * MX4_THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * MX4_THREADS) {
        const int64_t r = i / per, c = (i - r * per) * 8, b = c >> 5;
        const uint32_t w = __ldcs(reinterpret_cast<const uint32_t*>(a.q.data + r * a.q.ld + c / 2));
        const float s = mx4_value(a.q.scales[a.q.tiled ? mx4_tiled_at(r, b, a.q.tiles) : r * a.q.blocks + b]);
        float v[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 p = from_e2m1(w >> (8 * q) & 0xFFu);
            v[2 * q] = p.x * s;
            v[2 * q + 1] = p.y * s;
        }
        char* row = static_cast<char*>(a.dst) + r * a.ld * Elem<DT>::SIZE;
        if (a.aligned16 && c + 8 <= a.cols) {
            st8<DT>(row, c, narrow8<DT>(v));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < a.cols) st1<DT>(row, c + e, v[e]);
        }
    }
}

// Scales gathered row by row to the tiles the product reads: a thread makes
// one word, 4 blocks of a row.
__global__ void __launch_bounds__(MX4_THREADS) k_mx4_tile(const uint8_t* src, uint8_t* dst, int64_t rows,
                                                         int64_t blocks, int64_t tiles) {
    pdl_wait();
    pdl_launch_next();
    const int64_t n = (rows + 127) / 128 * 128 * tiles;
    for (int64_t i = (int64_t)blockIdx.x * MX4_THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * MX4_THREADS) {
        const int64_t r = i / tiles, t = i - r * tiles;
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r < rows && t * 4 + k < blocks) w |= (uint32_t)src[r * blocks + t * 4 + k] << (8 * k);
        *reinterpret_cast<uint32_t*>(dst + mx4_tiled_at(r, t * 4, tiles)) = w;
    }
}

int check_mx4(const zero_mx4* m, const char* call, const char* what) {
    if (!m) return refuse(ZERO_EINVAL, call, what, " is NULL");
    if (m->rows < 0 || m->cols < 0) return refuse(ZERO_EINVAL, call, what, ": negative size");
    if (m->layout != ZERO_MX4_ROWS && m->layout != ZERO_MX4_TILES)
        return refuse(ZERO_EINVAL, call, what, ": unknown scale layout");
    if (m->rows == 0 || m->cols == 0) return ZERO_OK;
    if (!m->data || !m->scales) return refuse(ZERO_EINVAL, call, what, ": NULL data or scales");
    if (!aligned(m->data, 16) || (m->layout == ZERO_MX4_TILES && !aligned(m->scales, 16)))
        return refuse(ZERO_EALIGN, call, what, ": data and tiled scales must be 16-byte aligned");
    if (m->ld % 16 != 0 || m->ld < mx4_blocks(m->cols) * 16)
        return refuse(ZERO_EINVAL, call, what, ": ld is a multiple of 16 bytes, at least 16 for every 32 columns");
    return ZERO_OK;
}

static Mx4Dev device_form(const zero_mx4& m) {
    return Mx4Dev{static_cast<uint8_t*>(m.data), static_cast<uint8_t*>(m.scales), m.ld, mx4_blocks(m.cols),
                  mx4_tiles(m.cols), m.layout == ZERO_MX4_TILES};
}

static int blocks_for(int64_t n, int per_sm) {
    const int64_t most = (int64_t)sm_count() * per_sm;
    return (int)(n < most ? (n > 0 ? n : 1) : most);
}

}  // namespace zdp

using namespace zdp;

extern "C" {

int zero_mx4_bytes(int64_t rows, int64_t cols, int layout, int64_t* ld, int64_t* data_bytes, int64_t* scale_bytes) {
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "zero_mx4_bytes: negative size");
    if (layout != ZERO_MX4_ROWS && layout != ZERO_MX4_TILES) return fail(ZERO_EINVAL, "zero_mx4_bytes: unknown scale layout");
    if (!ld || !data_bytes || !scale_bytes) return fail(ZERO_EINVAL, "zero_mx4_bytes: NULL output");
    *ld = mx4_blocks(cols) * 16;
    *data_bytes = rows * *ld;
    *scale_bytes = mx4_scale_bytes(rows, cols, layout);
    return ZERO_OK;
}

int zero_mx4_quantize(const zero_mat* src, int64_t rows, int64_t cols, const zero_mx4* out, const zero_mx4* out_t,
                      void* stream) {
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "zero_mx4_quantize: negative size");
    int rc = check_mat(src, rows, cols, FLOAT_TYPES, "zero_mx4_quantize", "src");
    if (rc == ZERO_OK && out) rc = check_mx4(out, "zero_mx4_quantize", "out");
    if (rc == ZERO_OK && out_t) rc = check_mx4(out_t, "zero_mx4_quantize", "out_t");
    if (rc != ZERO_OK) return rc;
    if (out && (out->rows != rows || out->cols != cols)) return fail(ZERO_EINVAL, "zero_mx4_quantize: out is rows x cols");
    if (out_t && (out_t->rows != cols || out_t->cols != rows))
        return fail(ZERO_EINVAL, "zero_mx4_quantize: out_t is cols x rows");
    if (rows == 0 || cols == 0 || (!out && !out_t)) return ZERO_OK;
    if (!sm_count()) return ZERO_ECUDA;
    QuantArgs a = {};
    a.src = src->data;
    a.ld = src->ld;
    a.rows = rows;
    a.cols = cols;
    a.aligned16 = rows_aligned(*src, rows);
    if (out) a.q = device_form(*out);
    if (out_t) a.t = device_form(*out_t);
    const int dt = src->dtype;
    const void* f;
    int grid, threads;
    if (out_t) {
        f = dt == ZERO_F32 ? (const void*)k_mx4_both<ZERO_F32>
          : dt == ZERO_BF16 ? (const void*)k_mx4_both<ZERO_BF16> : (const void*)k_mx4_both<ZERO_F16>;
        threads = 128;
        grid = blocks_for((rows + 255) / 256 * 2 * ((cols + 255) / 256 * 4), 16);
    } else {
        f = dt == ZERO_F32 ? (const void*)k_mx4_rows<ZERO_F32>
          : dt == ZERO_BF16 ? (const void*)k_mx4_rows<ZERO_BF16> : (const void*)k_mx4_rows<ZERO_F16>;
        threads = MX4_THREADS;
        const int64_t r = a.q.tiled ? (rows + 127) / 128 * 128 : rows;
        grid = blocks_for((r * ((cols + 255) / 256) + 7) / 8, 8);
    }
    void* args[] = {&a};
    return cuda_fail(launch_after_previous(f, grid, threads, args, 0, static_cast<cudaStream_t>(stream)),
                     "zero_mx4_quantize launch");
}

int zero_mx4_dequantize(const zero_mx4* src, const zero_mat* dst, void* stream) {
    int rc = check_mx4(src, "zero_mx4_dequantize", "src");
    if (rc == ZERO_OK) rc = check_mat(dst, src->rows, src->cols, FLOAT_TYPES, "zero_mx4_dequantize", "dst");
    if (rc != ZERO_OK || src->rows == 0 || src->cols == 0) return rc;
    if (!sm_count()) return ZERO_ECUDA;
    DequantArgs a = {};
    a.q = device_form(*src);
    a.dst = dst->data;
    a.ld = dst->ld;
    a.rows = src->rows;
    a.cols = src->cols;
    a.aligned16 = rows_aligned(*dst, a.rows);
    const int dt = dst->dtype;
    const void* f = dt == ZERO_F32 ? (const void*)k_mx4_values<ZERO_F32>
                  : dt == ZERO_BF16 ? (const void*)k_mx4_values<ZERO_BF16> : (const void*)k_mx4_values<ZERO_F16>;
    void* args[] = {&a};
    return cuda_fail(launch_after_previous(f, blocks_for((a.rows * ((a.cols + 7) / 8) + MX4_THREADS - 1) / MX4_THREADS, 16),
                                           MX4_THREADS, args, 0, static_cast<cudaStream_t>(stream)),
                     "zero_mx4_dequantize launch");
}

int zero_mx4_tile_scales(const zero_mx4* src, const zero_mx4* dst, void* stream) {
    int rc = check_mx4(src, "zero_mx4_tile_scales", "src");
    if (rc == ZERO_OK) rc = check_mx4(dst, "zero_mx4_tile_scales", "dst");
    if (rc != ZERO_OK) return rc;
    if (src->layout != ZERO_MX4_ROWS || dst->layout != ZERO_MX4_TILES || src->rows != dst->rows || src->cols != dst->cols)
        return fail(ZERO_EINVAL, "zero_mx4_tile_scales: from ZERO_MX4_ROWS to ZERO_MX4_TILES of the same size");
    if (src->rows == 0 || src->cols == 0) return ZERO_OK;
    if (!sm_count()) return ZERO_ECUDA;
    const uint8_t* s = static_cast<const uint8_t*>(src->scales);
    uint8_t* d = static_cast<uint8_t*>(dst->scales);
    int64_t rows = src->rows, blocks = mx4_blocks(src->cols), tiles = mx4_tiles(src->cols);
    void* args[] = {&s, &d, &rows, &blocks, &tiles};
    return cuda_fail(launch_after_previous((const void*)k_mx4_tile,
                                           blocks_for(((rows + 127) / 128 * 128 * tiles + MX4_THREADS - 1) / MX4_THREADS, 8),
                                           MX4_THREADS, args, 0, static_cast<cudaStream_t>(stream)),
                     "zero_mx4_tile_scales launch");
}

}  // extern "C"
