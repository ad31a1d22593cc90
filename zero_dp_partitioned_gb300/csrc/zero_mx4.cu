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
// over rows) a block takes 128 x 128 elements through shared memory; both forms
// come from one read of the matrix.
//
// Measured (GB300, 14336 x 4096 bf16; the floor is the bytes at the measured
// copy bandwidth): rows 29.5 us (floor 21.9), columns 25.7 (21.9), both 41.0
// (26.5), values back 26.9 (21.9).  Both ways nothing is near full (DRAM 0.42
// of its peak, instruction issue 0.58, a third of the warps): the two passes
// and the stores take turns behind three barriers a tile.  fp32 8192 x 4096:
// rows 27.5 (22.4), both 36.5 (25.0), back 26.5 (22.4).  Rows that start
// anywhere are 2.5 to 3.3 times their floor (8192 x 4097 bf16: 33.6, 49.6 and
// 30.7 us), by the second word of each unit and the shifts.  The tiling of
// gathered scales takes 4.8 us, about a launch (floor 0.5).
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

// A scale tile (128 rows by 4 blocks, as ZERO_MX4_TILES lays it out) from
// shared memory to where q keeps it; i: which of the block's 128 threads.
__device__ __forceinline__ void put_scales(const Mx4Dev& q, const uint8_t* tile, int64_t rows, int64_t tr, int64_t tb, int i) {
    if (q.tiled) {
        if (i < 32 && tr * 128 < rows && tb < q.tiles)
            reinterpret_cast<uint4*>(q.scales + (tr * q.tiles + tb) * 512)[i] = reinterpret_cast<const uint4*>(tile)[i];
    } else if (tr * 128 + i < rows) {
        for (int b = 0; b < 4; ++b)
            if (tb * 4 + b < q.blocks)
                q.scales[(tr * 128 + i) * q.blocks + tb * 4 + b] = tile[(i & 31) * 16 + (i >> 5) * 4 + b];
    }
}

// 8 elements of a row from column c, as they lie; columns past the end are 0.
template <int DT>
__device__ __forceinline__ Raw8<DT> read8(const void* row, int64_t c, int64_t cols, bool vec, const Extent& x) {
    if (vec && c + 8 <= cols) return ld8_stream<DT>(row, c);
    return ld8_shifted<DT>(row, c, cols, x);
}

// The bits of the largest magnitude of 8 elements (ordered as unsigned
// integers, NaN on top): of the fp32 value, or of a 16-bit one, two compared
// at a time.
template <int DT>
__device__ __forceinline__ uint32_t top8(const Raw8<DT>& r) {
    if constexpr (DT == ZERO_F32) {
        uint32_t t = 0;
#pragma unroll
        for (int w = 0; w < 2; ++w)
            t = max(max(t, max(r.w[w].x & 0x7FFFFFFFu, r.w[w].y & 0x7FFFFFFFu)),
                    max(r.w[w].z & 0x7FFFFFFFu, r.w[w].w & 0x7FFFFFFFu));
        return t;
    } else {
        const uint32_t t = __vmaxu2(__vmaxu2(r.w[0].x & 0x7FFF7FFFu, r.w[0].y & 0x7FFF7FFFu),
                                    __vmaxu2(r.w[0].z & 0x7FFF7FFFu, r.w[0].w & 0x7FFF7FFFu));
        return max(t & 0xFFFFu, t >> 16);
    }
}
// The scale byte from such bits.
template <int DT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if constexpr (DT == ZERO_F32) return mx4_scale(top);
    else if constexpr (DT == ZERO_BF16) return mx4_scale(top << 16);
    else return mx4_scale(__float_as_uint(Half16<DT>::widen(top)));
}
// The codes of 8 elements, scaled.
template <int DT>
__device__ __forceinline__ uint32_t codes8(const Raw8<DT>& r, uint64_t inv) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 p = unpack2(mul2(pair8<DT>(r, q), inv));
        v[2 * q] = p.x;
        v[2 * q + 1] = p.y;
    }
    return to_e2m1(v);
}

// i = first, first + step, ... as (row, place) of rows of `per` places: two
// divisions at the start, none on the way (a 64-bit one costs as much as the
// work on 8 elements).
struct Walk {
    int64_t row, at, d_row, d_at, per;
    __device__ __forceinline__ Walk(int64_t first, int64_t step, int64_t per_)
        : row(first / per_), at(first % per_), d_row(step / per_), d_at(step % per_), per(per_) {}
    __device__ __forceinline__ void next() {
        row += d_row;
        at += d_at;
        if (at >= per) {
            at -= per;
            ++row;
        }
    }
};

// Along the rows.  A warp takes up to MX4_SPAN pieces of 256 columns of a row
// (8 blocks each, a step of the product's tiles), their loads issued together;
// rows and columns of the scales' padding are walked too.
constexpr int MX4_SPAN = 4;
template <int DT>
__global__ void __launch_bounds__(MX4_THREADS) k_mx4_rows(const __grid_constant__ QuantArgs a) {
    pdl_wait();
    pdl_launch_next();
    const Extent x = extent_of<DT>(a.src, a.ld, a.rows, a.cols);
    const int64_t rows = a.q.tiled ? (a.rows + 127) / 128 * 128 : a.rows;
    const int64_t pieces = (a.cols + 255) / 256;
    const int lane = threadIdx.x & 31;
    for (Walk i((int64_t)blockIdx.x * (MX4_THREADS / 32) + (threadIdx.x >> 5), (int64_t)gridDim.x * (MX4_THREADS / 32),
                (pieces + MX4_SPAN - 1) / MX4_SPAN);
         i.row < rows; i.next()) {
        const int64_t r = i.row, p0 = i.at * MX4_SPAN;
        const int64_t c0 = p0 * 256 + lane * 8;
        const char* row = static_cast<const char*>(a.src) + r * a.ld * Elem<DT>::SIZE;
        uint8_t* data = a.q.data + r * a.q.ld + c0 / 2;
        uint8_t* scales = a.q.tiled ? a.q.scales + mx4_tiled_at(r, c0 >> 5, a.q.tiles) : a.q.scales + r * a.q.blocks + (c0 >> 5);
        Raw8<DT> v[MX4_SPAN];
#pragma unroll
        for (int k = 0; k < MX4_SPAN; ++k) {
            if (r < a.rows && c0 + k * 256 < a.cols) {
                v[k] = read8<DT>(row, c0 + k * 256, a.cols, a.aligned16, x);
            } else {
#pragma unroll
                for (auto& w : v[k].w) w = make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int k = 0; k < MX4_SPAN; ++k) {
            if (p0 + k >= pieces) break;
            const int64_t b = (c0 >> 5) + k * 8;
            const uint32_t byte = scale_byte<DT>(lanes_max<4>(top8<DT>(v[k])));
            const float inv = mx4_inverse(byte);
            const uint32_t code = codes8<DT>(v[k], pack2(inv, inv));
            if (r < a.rows && b < a.q.blocks) *reinterpret_cast<uint32_t*>(data + k * 128) = code;
            // the 4 blocks of 16 lanes make one word of a tile
            uint32_t word = byte << (8 * ((lane >> 2) & 3));
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
            if (a.q.tiled) {
                if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scales + k * 1024) = word;      // two tiles a piece
            } else if ((lane & 3) == 0 && b < a.q.blocks) {
                scales[k * 8] = (uint8_t)byte;
            }
        }
    }
}

// Along the columns, and along the rows too if they are wanted.  A block takes
// 128 by 128 elements -- one scale tile in each direction.  A warp copies 16
// of its rows to shared memory and quantises those, and then 32 rows by 64
// columns along the columns, two to a lane.  The columns' codes and both scale
// tiles are put together in shared memory, so that they leave in pieces of 64
// and 512 consecutive bytes.
//
// The next tile is on its way to shared memory (cp.async, each lane its own 16
// bytes) while one is worked on; fp32 has room for one tile a block, and two
// blocks cover for each other.
template <int DT>
struct Mx4Both {
    static constexpr int TILE = 128 * 128 * Elem<DT>::SIZE, STAGES = DT == ZERO_F32 ? 1 : 2, SMEM = STAGES * TILE;
    static constexpr int BLOCKS = DT == ZERO_F32 ? 2 : 3;                 // of a multiprocessor
};

constexpr int MX4_BOTH_THREADS = 256;
template <int DT>
__global__ void __launch_bounds__(MX4_BOTH_THREADS) k_mx4_both(const __grid_constant__ QuantArgs a) {
    using B = Mx4Both<DT>;
    extern __shared__ __align__(16) uint8_t tile_raw[];
    __shared__ __align__(16) uint4 codes[128][4];
    __shared__ __align__(16) uint8_t scale_q[512], scale_t[512];
    pdl_wait();
    pdl_launch_next();
    const Extent x = extent_of<DT>(a.src, a.ld, a.rows, a.cols);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // both directions are padded to 256 for the scales
    const int64_t nr = (a.rows + 255) / 256 * 2, nc = (a.cols + 255) / 256 * 2;
    const int lr = lane >> 4, lc = (lane & 15) * 8;  // this lane's rows lr, lr + 2, ... and columns lc .. lc + 7 of the warp's
    auto fetch = [&](const Walk& i, int st) {
        if (i.row < nr) {
            const int64_t r0 = i.row * 128 + warp * 16 + lr, c = i.at * 128 + lc;
            uint8_t* s = tile_raw + st * B::TILE + ((warp * 16 + lr) * 128 + lc) * Elem<DT>::SIZE;
            const char* src = static_cast<const char*>(a.src) + (r0 * a.ld + c) * Elem<DT>::SIZE;
            const bool inside = a.aligned16 && c + 8 <= a.cols;
            const int left = (int)(a.rows - r0 < 16 ? a.rows - r0 : 16);        // rows of the matrix from r0 on
            const int64_t down = 2 * a.ld * Elem<DT>::SIZE;
            const char* from = src;
#pragma unroll
            for (int k = 0; k < 8; ++k, from += down) {
                const int64_t r = r0 + 2 * k;
                uint8_t* to = s + k * 2 * 128 * Elem<DT>::SIZE;
                if (inside && 2 * k < left) {
#pragma unroll
                    for (int w = 0; w < Elem<DT>::SIZE / 2; ++w)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         (uint32_t)__cvta_generic_to_shared(to) + 16 * w),
                                     "l"(from + 16 * w)
                                     : "memory");
                } else {
                    Raw8<DT> v;
                    if (r < a.rows && c < a.cols) {
                        v = read8<DT>(static_cast<const char*>(a.src) + r * a.ld * Elem<DT>::SIZE, c, a.cols, a.aligned16, x);
                    } else {
#pragma unroll
                        for (auto& w : v.w) w = make_uint4(0, 0, 0, 0);
                    }
                    st8<DT>(to, 0, v);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int st = 0;
    Walk i(blockIdx.x, gridDim.x, nc), ahead = i;
    if (B::STAGES == 2) fetch(i, 0);
    for (; i.row < nr; i.next()) {
        ahead.next();
        if (B::STAGES == 2) fetch(ahead, st ^ 1);
        else fetch(i, 0);
        asm volatile("cp.async.wait_group %0;" ::"n"(B::STAGES - 1) : "memory");
        const int64_t tr = i.row, tc = i.at, c0 = tc * 128;
        const uint8_t* s = tile_raw + st * B::TILE;
        if (a.q.data) {
            const int64_t r0 = tr * 128, c = c0 + lc;
            uint8_t* data = a.q.data + (r0 + warp * 16 + lr) * a.q.ld + c / 2;
            const int left = c < a.q.blocks * 32 ? (int)(a.rows - r0 < 128 ? a.rows - r0 : 128) : 0;    // rows to write
#pragma unroll 4
            for (int k = 0; k < 8; ++k, data += 2 * a.q.ld) {
                const int rr = warp * 16 + lr + 2 * k;
                const Raw8<DT> v = ld8<DT>(s, rr * 128 + lc);
                const uint32_t byte = scale_byte<DT>(lanes_max<4>(top8<DT>(v)));
                const float inv = mx4_inverse(byte);
                const uint32_t code = codes8<DT>(v, pack2(inv, inv));
                if (rr < left) *reinterpret_cast<uint32_t*>(data) = code;
                if ((lane & 3) == 0) scale_q[(rr & 31) * 16 + (rr >> 5) * 4 + ((lane & 15) >> 2)] = (uint8_t)byte;
            }
        }
        __syncthreads();
        if (a.t.data) {
            // columns cc and the next, rows 32 rb .. + 31: one block of each
            const int rb = warp >> 1, cc = (warp & 1) * 64 + 2 * lane;
            uint32_t byte0, byte1, w0[4], w1[4];
            if constexpr (DT == ZERO_F32) {
                const float2* p = reinterpret_cast<const float2*>(s) + rb * 32 * 64 + cc / 2;
                float2 v[32];
                uint32_t top0 = 0, top1 = 0;
#pragma unroll
                for (int rr = 0; rr < 32; ++rr) {
                    v[rr] = p[rr * 64];
                    top0 = max(top0, abs_bits(v[rr].x));
                    top1 = max(top1, abs_bits(v[rr].y));
                }
                byte0 = mx4_scale(top0);
                byte1 = mx4_scale(top1);
                const uint64_t inv = pack2(mx4_inverse(byte0), mx4_inverse(byte1));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[8], y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = unpack2(mul2(pack2(v[q * 8 + e].x, v[q * 8 + e].y), inv));
                        x[e] = t.x;
                        y[e] = t.y;
                    }
                    w0[q] = to_e2m1(x);
                    w1[q] = to_e2m1(y);
                }
            } else {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(s) + rb * 32 * 64 + cc / 2;
                uint32_t v[32], t = 0;
#pragma unroll
                for (int rr = 0; rr < 32; ++rr) {
                    v[rr] = p[rr * 64];
                    t = __vmaxu2(t, v[rr] & 0x7FFF7FFFu);
                }
                byte0 = scale_byte<DT>(t & 0xFFFFu);
                byte1 = scale_byte<DT>(t >> 16);
                const uint64_t inv = pack2(mx4_inverse(byte0), mx4_inverse(byte1));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[8], y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t u = v[q * 8 + e];
                        const uint64_t both = DT == ZERO_BF16
                                                  ? pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u))
                                                  : pack2(Half16<DT>::widen(u & 0xFFFFu), Half16<DT>::widen(u >> 16));
                        const float2 f = unpack2(mul2(both, inv));
                        x[e] = f.x;
                        y[e] = f.y;
                    }
                    w0[q] = to_e2m1(x);
                    w1[q] = to_e2m1(y);
                }
            }
            const int at = rb ^ (lane & 3);
            codes[cc][at] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
            codes[cc + 1][at] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
            // rows cc and cc + 1 of the transpose's tile, block rb of its 4
            scale_t[(cc & 31) * 16 + (cc >> 5) * 4 + rb] = (uint8_t)byte0;
            scale_t[((cc + 1) & 31) * 16 + (cc >> 5) * 4 + rb] = (uint8_t)byte1;
        }
        __syncthreads();
        if (a.t.data) {
#pragma unroll
            for (int k = 0; k < 512 / MX4_BOTH_THREADS; ++k) {
                const int id = k * MX4_BOTH_THREADS + threadIdx.x, cc = id >> 2, ch = id & 3;
                const int64_t b = tr * 4 + ch;
                if (c0 + cc < a.cols && b < a.t.blocks)
                    *reinterpret_cast<uint4*>(a.t.data + (c0 + cc) * a.t.ld + b * 16) = codes[cc][ch ^ ((cc >> 1) & 3)];
            }
            if (threadIdx.x < 128) put_scales(a.t, scale_t, a.cols, tc, tr, threadIdx.x);
        }
        if (a.q.data && threadIdx.x >= 128) put_scales(a.q, scale_q, a.rows, tr, tc, threadIdx.x - 128);
        __syncthreads();
        if (B::STAGES == 2) st ^= 1;
    }
}

struct DequantArgs {
    Mx4Dev q;
    void* dst;
    int64_t ld, rows, cols;
    int aligned16, aligned32;
};

// A warp takes up to MX4_SPAN pieces of 256 columns of a row, 8 columns to a
// lane and piece.
template <int DT>
__global__ void __launch_bounds__(MX4_THREADS) k_mx4_values(const __grid_constant__ DequantArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x & 31;
    for (Walk i((int64_t)blockIdx.x * (MX4_THREADS / 32) + (threadIdx.x >> 5), (int64_t)gridDim.x * (MX4_THREADS / 32),
                (a.cols + 256 * MX4_SPAN - 1) / (256 * MX4_SPAN));
         i.row < a.rows; i.next()) {
        const int64_t r = i.row, c0 = i.at * 256 * MX4_SPAN + lane * 8;
        const uint8_t* data = a.q.data + r * a.q.ld + c0 / 2;
        // a piece is two tiles, or 8 blocks of a row
        const uint8_t* scales =
            a.q.tiled ? a.q.scales + mx4_tiled_at(r, c0 >> 5, a.q.tiles) : a.q.scales + r * a.q.blocks + (c0 >> 5);
        const int piece = a.q.tiled ? 1024 : 8;
        uint32_t w[MX4_SPAN] = {}, byte[MX4_SPAN] = {};
#pragma unroll
        for (int k = 0; k < MX4_SPAN; ++k)
            if (c0 + k * 256 < a.cols) {
                w[k] = __ldcs(reinterpret_cast<const uint32_t*>(data + k * 128));
                byte[k] = scales[k * piece];
            }
        char* row = static_cast<char*>(a.dst) + r * a.ld * Elem<DT>::SIZE;
#pragma unroll
        for (int k = 0; k < MX4_SPAN; ++k) {
            const int64_t c = c0 + k * 256;
            if (c - lane * 8 >= a.cols) break;             // the whole warp together
            const float s = mx4_value(byte[k]);
            float v[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 p = from_e2m1(w[k] >> (8 * q) & 0xFFu);
                const float2 f = unpack2(mul2(pack2(p.x, p.y), pack2(s, s)));
                v[2 * q] = f.x;
                v[2 * q + 1] = f.y;
            }
            const Raw8<DT> o = narrow8<DT>(v);
            if (!a.aligned16) {
                st8_shifted<DT>(row, c, a.cols, c < a.cols, o);
            } else if (c + 8 <= a.cols) {
                if constexpr (DT == ZERO_F32) {
                    if (a.aligned32) st32(row + c * 4, o.w[0], o.w[1]);
                    else st8<DT>(row, c, o);
                } else {
                    st8<DT>(row, c, o);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < a.cols) st1<DT>(row, c + e, v[e]);
            }
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
    size_t smem = 0;
    if (out_t) {
        f = dt == ZERO_F32 ? (const void*)k_mx4_both<ZERO_F32>
          : dt == ZERO_BF16 ? (const void*)k_mx4_both<ZERO_BF16> : (const void*)k_mx4_both<ZERO_F16>;
        threads = MX4_BOTH_THREADS;
        smem = dt == ZERO_F32 ? Mx4Both<ZERO_F32>::SMEM : Mx4Both<ZERO_BF16>::SMEM;
        rc = raise_smem(f, smem, "zero_mx4_quantize shared-memory size");
        if (rc != ZERO_OK) return rc;
        grid = blocks_for((rows + 255) / 256 * 2 * ((cols + 255) / 256 * 2), dt == ZERO_F32 ? Mx4Both<ZERO_F32>::BLOCKS : Mx4Both<ZERO_BF16>::BLOCKS);
    } else {
        f = dt == ZERO_F32 ? (const void*)k_mx4_rows<ZERO_F32>
          : dt == ZERO_BF16 ? (const void*)k_mx4_rows<ZERO_BF16> : (const void*)k_mx4_rows<ZERO_F16>;
        threads = MX4_THREADS;
        const int64_t r = a.q.tiled ? (rows + 127) / 128 * 128 : rows;
        grid = blocks_for((r * ((cols + 256 * MX4_SPAN - 1) / (256 * MX4_SPAN)) + 7) / 8, 8);
    }
    void* args[] = {&a};
    return cuda_fail(launch_after_previous(f, grid, threads, args, smem, static_cast<cudaStream_t>(stream)),
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
    a.aligned32 = aligned(dst->data, 32) && (a.rows <= 1 || dst->ld * elem_size(dst->dtype) % 32 == 0);
    const int dt = dst->dtype;
    const void* f = dt == ZERO_F32 ? (const void*)k_mx4_values<ZERO_F32>
                  : dt == ZERO_BF16 ? (const void*)k_mx4_values<ZERO_BF16> : (const void*)k_mx4_values<ZERO_F16>;
    void* args[] = {&a};
    return cuda_fail(launch_after_previous(f, blocks_for((a.rows * ((a.cols + 256 * MX4_SPAN - 1) / (256 * MX4_SPAN)) + 7) / 8, 8),
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
