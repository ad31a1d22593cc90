// zero_dropout.cu -- y = dropout(x) + residual, and with it the gradient:
// dx = dropout(dy) by the same mask (zero_drop.cuh).
//
// Bound: HBM (x and the residual read, y written) where rows start on 16 bytes:
// 32768 x 4096 bf16 in 87 us, 6.2 TB/s (0.91 of the measured copy bandwidth),
// onto a residual in 125 (0.95); fp32 rows that start anywhere too (4095 x 6401
// onto a residual in 49, 0.95).  16-bit rows that start anywhere are bound by
// their instructions, an access an element: 16384 x 4097 bf16 in 74 us (0.53),
// onto a residual in 90 (0.66).
#include "zero_drop.cuh"

namespace zdp {

constexpr int DROP_THREADS = 256;
constexpr int DROP_UNITS = 2;           // units of 8 columns a thread has on their way

struct DropoutArgs {
    const void *x, *r;
    void* y;
    int64_t ldx, ldr, ldy, rows, cols;
    int64_t units, tiles;               // of a row
    DropArgs drop;
};

// Rows that start on 16-byte boundaries, columns a multiple of 8: a unit a
// thread.  A tile is DROP_UNITS * DROP_THREADS units of one row; rows that
// follow one another without gaps come as one.
template <int DT, bool RES>
__global__ void __launch_bounds__(DROP_THREADS) k_dropout(const __grid_constant__ DropoutArgs a) {
    pdl_wait();
    pdl_launch_next();
    const uint32_t step = drop_step(a.drop);
    const int64_t n = a.rows * a.tiles;
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x) {
        const int64_t row = a.rows == 1 ? 0 : quotient(t, a.tiles), u0 = (t - row * a.tiles) * (DROP_UNITS * DROP_THREADS) + threadIdx.x;
        const char* X = static_cast<const char*>(a.x) + row * a.ldx * Elem<DT>::SIZE;
        const char* R = static_cast<const char*>(a.r) + row * a.ldr * Elem<DT>::SIZE;
        char* Y = static_cast<char*>(a.y) + row * a.ldy * Elem<DT>::SIZE;
        Raw8<DT> x[DROP_UNITS], r[DROP_UNITS];
#pragma unroll
        for (int j = 0; j < DROP_UNITS; ++j) {
            const int64_t u = u0 + j * DROP_THREADS;
            if (u < a.units) {
                x[j] = ld8_stream<DT>(X, u * 8);
                if (RES) r[j] = ld8_stream<DT>(R, u * 8);
            }
        }
#pragma unroll
        for (int j = 0; j < DROP_UNITS; ++j) {
            const int64_t u = u0 + j * DROP_THREADS;
            if (u >= a.units) break;
            const uint4 bits = drop_bits(a.drop, step, row * a.units + u);
            float v[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint64_t k = a.drop.on ? drop2(pair8<DT>(x[j], q), bits, q, a.drop.above) : pair8<DT>(x[j], q);
                const float2 p = unpack2(RES ? scaled_onto2(k, a.drop, pair8<DT>(r[j], q)) : mul2(k, pack2(a.drop.scale, a.drop.scale)));
                v[2 * q] = p.x;
                v[2 * q + 1] = p.y;
            }
            st8<DT>(Y, u * 8, narrow8<DT>(v));
        }
    }
}

// Rows that start anywhere: a warp takes 32 units of a row, a lane the bits of
// one; then the lanes take neighbouring elements, 256 in eight turns, and the
// element's bit from the lane that has its unit.
template <int DT, bool RES>
__global__ void __launch_bounds__(DROP_THREADS) k_dropout_any(const __grid_constant__ DropoutArgs a) {
    pdl_wait();
    pdl_launch_next();
    const uint32_t step = drop_step(a.drop);
    const int lane = threadIdx.x & 31;
    const int64_t n = a.rows * a.tiles, warps = (int64_t)gridDim.x * (DROP_THREADS / 32);
    for (int64_t t = (int64_t)blockIdx.x * (DROP_THREADS / 32) + (threadIdx.x >> 5); t < n; t += warps) {
        // a division in 32 bits where it will do, asked of all tiles at once (of each: 84 us for 74, 16384 x 4097 bf16)
        const int64_t row = n <= UINT32_MAX ? (int64_t)((uint32_t)t / (uint32_t)a.tiles) : t / a.tiles;
        const int64_t u0 = (t - row * a.tiles) * 32, c0 = u0 * 8 + lane;
        const int left = (int)min(a.cols - c0, (int64_t)256);            // columns from this lane's first
        const char* X = static_cast<const char*>(a.x) + (row * a.ldx + c0) * Elem<DT>::SIZE;
        const char* R = static_cast<const char*>(a.r) + (RES ? (row * a.ldr + c0) * Elem<DT>::SIZE : 0);
        char* Y = static_cast<char*>(a.y) + (row * a.ldy + c0) * Elem<DT>::SIZE;
        float x[8], r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = 32 * j < left ? ld1<DT>(X, 32 * j) : 0.f;
            if (RES) r[j] = 32 * j < left ? ld1<DT>(R, 32 * j) : 0.f;
        }
        uint32_t keep = 0xFFu;
        if (a.drop.on) {
            const uint4 bits = drop_bits(a.drop, step, row * a.units + u0 + lane);
            keep = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                keep |= (uint32_t)kept_low(word_of(bits, q), a.drop.above) << (2 * q) |
                        (uint32_t)kept_high(word_of(bits, q), a.drop.above) << (2 * q + 1);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool kept = __shfl_sync(0xFFFFFFFFu, keep, 4 * j + (lane >> 3)) >> (lane & 7) & 1u;
            const float v = kept ? x[j] : 0.f;
            if (32 * j < left) st1<DT>(Y, 32 * j, RES ? __fadd_rn(__fmul_rn(v, a.drop.scale), r[j]) : v * a.drop.scale);
        }
    }
}

template <int DT>
static const void* dropout_fn(bool v8, bool res) {
    if (v8) return res ? (const void*)k_dropout<DT, true> : (const void*)k_dropout<DT, false>;
    return res ? (const void*)k_dropout_any<DT, true> : (const void*)k_dropout_any<DT, false>;
}

int check_drop(const zero_drop* d, DropArgs& a, const char* call) {
    a = {};
    a.scale = a.one = 1.f;
    if (!d) return ZERO_OK;
    if (!(d->p >= 0.f) || !(d->p <= 1.f)) return refuse(ZERO_EINVAL, call, "drop", ": p must be in 0 .. 1");
    if (!aligned(d->chain, 8)) return refuse(ZERO_EALIGN, call, "drop", ": chain not 8-byte aligned");
    // p in units of 2^-16, to nearest; exact in fp32 (a scaling) and in fp64 (the addition)
    const uint32_t limit = (uint32_t)((double)d->p * 65536.0 + 0.5);
    if (limit == 0) return ZERO_OK;
    a.on = 1;
    a.k0 = (uint32_t)d->seed;
    a.k1 = (uint32_t)(d->seed >> 32);
    a.site = d->site;
    a.step = (uint32_t)d->step;
    a.chain = d->chain;
    a.above = (uint32_t)(((uint64_t)limit << 16) - 1);      // half << 16 > above where half >= limit; 65536: nothing
    a.scale = limit == 65536 ? 0.f : 65536.f / (float)(65536 - limit);
    return ZERO_OK;
}

}  // namespace zdp

using namespace zdp;

extern "C" int zero_dropout(const zero_mat* x, const zero_mat* residual, int64_t rows, int64_t cols, const zero_drop* drop,
                            const zero_mat* y, void* stream) {
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "zero_dropout: negative rows or cols");
    if (!drop) return fail(ZERO_EINVAL, "zero_dropout: drop is NULL");
    if (rows > 0 && cols > INT64_MAX / 16 / rows) return fail(ZERO_ELIMIT, "zero_dropout: too many elements");
    int rc = check_mat(x, rows, cols, FLOAT_TYPES, "zero_dropout", "x");
    if (rc == ZERO_OK) rc = check_mat(y, rows, cols, FLOAT_TYPES, "zero_dropout", "y");
    if (rc == ZERO_OK && residual) rc = check_mat(residual, rows, cols, FLOAT_TYPES, "zero_dropout", "residual");
    if (rc != ZERO_OK) return rc;
    if (y->dtype != x->dtype || (residual && residual->dtype != x->dtype))
        return fail(ZERO_EINVAL, "zero_dropout: x, residual and y are of one type");
    DropoutArgs a = {};
    rc = check_drop(drop, a.drop, "zero_dropout");
    if (rc != ZERO_OK || rows == 0 || cols == 0) return rc;
    a.x = x->data;
    a.ldx = x->ld;
    a.r = residual ? residual->data : nullptr;
    a.ldr = residual ? residual->ld : 0;
    a.y = y->data;
    a.ldy = y->ld;
    a.rows = rows;
    a.cols = cols;
    const bool v8 = cols % 8 == 0 && rows_aligned(*x, rows) && rows_aligned(*y, rows) && (!residual || rows_aligned(*residual, rows));
    if (v8 && rows > 1 && x->ld == cols && y->ld == cols && (!residual || residual->ld == cols)) {
        a.cols = rows * cols;
        a.rows = 1;
    }
    a.units = (a.cols + 7) / 8;
    const int per_tile = v8 ? DROP_UNITS * DROP_THREADS : 32, per_block = v8 ? 1 : DROP_THREADS / 32;
    a.tiles = (a.units + per_tile - 1) / per_tile;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    const void* f = x->dtype == ZERO_F32    ? dropout_fn<ZERO_F32>(v8, residual != nullptr)
                    : x->dtype == ZERO_BF16 ? dropout_fn<ZERO_BF16>(v8, residual != nullptr)
                                            : dropout_fn<ZERO_F16>(v8, residual != nullptr);
    const int64_t blocks = (a.rows * a.tiles + per_block - 1) / per_block, most = (int64_t)sms * 16;
    void* args[] = {&a};
    return cuda_fail(launch_after_previous(f, (int)(blocks < most ? blocks : most), DROP_THREADS, args, 0,
                                           static_cast<cudaStream_t>(stream)),
                     "zero_dropout launch");
}
