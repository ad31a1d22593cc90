// zero_norm.cu -- the residual RMS norm of a layer, forward and backward.
//
//   h = round(x + r)      (r and h in x's type, or both in fp32)
//   y = h w / sqrt(mean(h^2) + eps)
// and, with xh = h rstd and g = dy w,
//   dx = rstd (g - xh mean(g xh)) + dh        (of x and of r alike)
//   dw = sum over rows of dy xh
//
// Bound: HBM.  Forward reads x and r and writes h and y (8 bytes an element
// in 16 bits, 7 with an e4m3 y); backward reads dy, h and dh and writes dx.
// A row is read once and kept in registers between the sum of squares and the
// output, so one block owns a row and nothing is read again.  Blocks stay and
// walk rows: the next rows are on their way to shared memory meanwhile, and a
// thread's columns, weights and part of dw are the same in every row.
//
// Measured (GB300, bf16): forward 8192 x 4096 in 43 us, 6.3 TB/s (0.92 of the
// measured copy bandwidth); with an e4m3 output and a scale per 128 columns
// 16384 x 4096 in 74 us, 6.4 TB/s (0.94), a scale per row 73; backward 8192 x
// 4096 in 51 us without dw, 5.3 TB/s (0.78; 512 threads a multiprocessor fill
// its registers, and each row waits for the block's sum), 55 us with it.
// Loading a row when its turn comes took 46 and 80 us, rows ahead in registers
// no less (fewer threads fit); one row in threads of 8 columns with fp32
// arithmetic one element at a time was bound by its instructions (29 an element).
//
// Further from the copy bandwidth: fp32 rows (8192 x 4096 in 116 and 138 us,
// 0.68 and 0.57: each lane's 32 bytes are moved as two accesses of 16, half of
// every sector an access touches), widths that are not a multiple of 8 or rows
// that start anywhere (8192 x 4097 bf16 in 109 and 121 us, 0.36 and 0.33: the
// shifts and one more barrier a row), and backward rows of 8193 to 16384
// columns, whose four units a thread do not fit its registers (320 to 568 bytes
// a thread go to local memory; 4096 x 12288 bf16 in 115 us, 0.51).  fp32 rows of
// that length, and all longer ones, are walked twice (4096 x 12288 fp32 in 214
// us, 0.55; 2048 x 20480 bf16 in 163, 0.30).
#include "zero_rows.cuh"

namespace zdp {

// Threads a multiprocessor that the grid and the stages are made for.  Of the
// forward pass registers let 1024 run at once (64 each, 16-bit rows of up to
// 8192 columns) or 512 (101 to 128: fp32, wider rows); with half as many again,
// and twice the blocks that gives, SMs that are done early take the rows of
// others (16384 x 4096 e4m3 73 us, 79 with once as many).  The backward pass,
// whose blocks each leave a partial dw, gains nothing from more than run.
constexpr int NORM_FORWARD_THREADS = 1536, NORM_BACKWARD_THREADS = 512;
constexpr int NORM_FORWARD_OVER = 2;
constexpr float E4M3_MAX = 448.f;
constexpr float SCALE_FLOOR = 7.888609052210118e-31f;   // 2^-100: a zero row still has a usable scale

struct NormArgs {
    const void *x, *r, *w;              // backward: dy, dh, w
    const void* hin;                    // backward: the stored h
    void *h, *y;                        // backward: y is dx
    int64_t ldx, ldr, ldhin, ldh, ldy, rows, n_scale;
    int cols;
    float eps;
    int wdt, w_aligned, y8, block128, stages;
    float *scale, *rstd;
    float* part;                        // backward: [grid][cols] partial dw
    int part16;                         // its rows start on 16-byte boundaries
};

template <bool V8>
__device__ __forceinline__ void store_e4m3(void* row, int u, int cols, const float (&v)[8]) {
    uint32_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        h[q] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * q], v[2 * q + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t w[2] = {h[0] | h[1] << 16, h[2] | h[3] << 16};
    if constexpr (!V8) st_shifted<1, 2>(row, u * 8, cols, u * 8 < cols, w);
    else if (u * 8 < cols) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(row) + u * 8) = make_uint2(w[0], w[1]);
}

// |y|'s largest of a unit, NaN kept (its bits then order above infinity's).
template <int E>
__device__ __forceinline__ float top_of(const float (&y)[E]) {
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) t = max3_nan(t, fabsf(y[e]), fabsf(y[e + 1]));
    return fabsf(t);
}
// A block's scale from its largest magnitude: at least the floor's, NaN kept.
// The product with 1 / 448 may be one unit from the quotient; the scale is what
// is stored, and the values are divided by that.
__device__ __forceinline__ float scale_of(float top) {
    return (top != top ? top : fmaxf(top, SCALE_FLOOR)) * (1.f / E4M3_MAX);
}
// v / scale, correctly rounded before it is rounded to 8 bits: 16-bit rows and
// weights make about one quotient in 10^4 an exact tie of e4m3, which the
// product with a reciprocal moves to either side.  The product is corrected by
// its remainder (P. Markstein, Computation of elementary functions on the IBM
// RISC System/6000 processor, 1990): q = v r, q + r (v - q scale) with the
// correctly rounded reciprocal r, all of -q so that a zero keeps its sign.  Of
// 2 * 10^8 quotients, half of them within two units of a tie, none differed
// from the division, which takes 97 us where this and the bare product take 78
// (16384 x 4096 bf16).  An infinite scale has no remainder: finite values
// become 0.
template <bool V8>
__device__ __forceinline__ void quantised_store(void* row, int u, int cols, float (&v)[Map::E], float scale) {
    const float inv = -__frcp_rn(scale), fin = scale < INFINITY ? scale : 0.f;
    const uint64_t r = pack2(inv, inv), s = pack2(fin, fin);
#pragma unroll
    for (int e = 0; e < Map::E; e += 2) {
        const uint64_t y = pack2(v[e], v[e + 1]), q = mul2(y, r);
        const float2 p = unpack2(fma2(fma2(q, s, y), r, q));
        v[e] = -p.x;
        v[e + 1] = -p.y;
    }
    store_e4m3<V8>(row, u, cols, v);
}

__device__ __forceinline__ void weights(const NormArgs& a, int u, float (&w)[8]) {
    vector8(a.w, a.wdt, a.w_aligned, a.cols, u, 1.f, w);
}

// A thread's columns are the same in every row it walks: their weights stay in registers.
template <int NV>
__device__ __forceinline__ void weight_pairs(const NormArgs& a, uint64_t (&w)[NV][Map::E / 2]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float v[Map::E];
        weights(a, Map::unit(j), v);
#pragma unroll
        for (int q = 0; q < Map::E / 2; ++q) w[j][q] = pack2(v[2 * q], v[2 * q + 1]);
    }
}

// A row in NV units per thread, in registers.
template <int XT, int RT, bool V8, int NV>
__global__ void __launch_bounds__(NORM_THREADS, NV == 2 && RT != ZERO_F32 ? 2 : 1) k_norm_forward(const __grid_constant__ NormArgs a) {
    constexpr int E = Map::E;
    __shared__ __align__(16) float ssum[2][32];
    if (threadIdx.x < 64) ssum[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
    __syncthreads();
    __shared__ uint32_t smax[2][32];
    pdl_wait();
    pdl_launch_next();
    const float inv_n = 1.f / (float)a.cols;
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols);
    extern __shared__ __align__(16) uint4 ring[];
    using X = Slots<XT, NV, V8>;
    using R = Slots<RT, NV, V8>;
    const int S = a.stages, stage_words = X::words() + R::words();
    auto copy = [&](int64_t row, int st) {
        if (row < a.rows) {
            uint4* at = ring + st * stage_words;
            X{at}.copy(row_of<XT>(a.x, a.ldx, row), a.cols, ex);
            if (a.r) R{at + X::words()}.copy(row_of<RT>(a.r, a.ldr, row), a.cols, er);
        }
        copies_commit();
    };
    for (int st = 0; st < S - 1; ++st) copy(blockIdx.x + (int64_t)st * gridDim.x, st);
    uint64_t w[NV][E / 2];
    weight_pairs<NV>(a, w);
    int turn = 0, st = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        Unit<XT, V8> x[NV];
        Unit<RT, V8> r[NV];
        copy(row + (int64_t)(S - 1) * gridDim.x, st == 0 ? S - 1 : st - 1);
        copies_wait_all_but(S - 1);
        if (!V8) __syncthreads();
        uint4* at = ring + st * stage_words;
        X{at}.read(x, row_of<XT>(a.x, a.ldx, row), a.cols);
        if (a.r) R{at + X::words()}.read(r, row_of<RT>(a.r, a.ldr, row), a.cols);
        st = st == S - 1 ? 0 : st + 1;
        // h as it is stored: half the registers of its fp32 values
        uint64_t s2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            r[j] = add_unit<XT, RT, V8>(x[j], r[j], a.r != nullptr);
#pragma unroll
            for (int q = 0; q < E / 2; ++q) s2 = fma2(r[j].pair(q), r[j].pair(q), s2);
            if (a.h) r[j].store(row_of<RT>(a.h, a.ldh, row), Map::unit(j), a.cols);
        }
        const float2 sp = unpack2(s2);
        const float ss = block_sum(sp.x + sp.y, ssum[turn]);
        const float rstd = rsqrtf(fmaf(ss, inv_n, a.eps));
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
        const uint64_t rr = pack2(rstd, rstd);
        auto normed = [&](int j, float (&y)[E]) {
#pragma unroll
            for (int q = 0; q < E / 2; ++q) {
                const float2 v = unpack2(mul2(mul2(r[j].pair(q), rr), w[j][q]));
                y[2 * q] = v.x;
                y[2 * q + 1] = v.y;
            }
        };
        if (!a.y8) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float y[E];
                normed(j, y);
                store_unit<XT, V8>(row_of<XT>(a.y, a.ldy, row), Map::unit(j), a.cols, y);
            }
            continue;
        }
        uint8_t* Y = static_cast<uint8_t*>(a.y) + row * a.ldy;
        float whole = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float y[E];
            normed(j, y);
            const float t = top_of<E>(y);
            if (a.block128) {
                const int u = Map::unit(j);
                const float sc = scale_of(__uint_as_float(lanes_max<Map::LANES>(__float_as_uint(t))));
                if ((u & (Map::LANES - 1)) == 0 && Map::any(u, a.cols))
                    a.scale[row * a.n_scale + u / Map::LANES] = sc;
                quantised_store<V8>(Y, u, a.cols, y, sc);
            }
            whole = max3_nan(whole, t, t);
        }
        if (!a.block128) {
            const float sc = scale_of(__uint_as_float(block_max(__float_as_uint(whole), smax[turn])));
            if (threadIdx.x == 0) a.scale[row * a.n_scale] = sc;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float y[E];
                normed(j, y);
                quantised_store<V8>(Y, Map::unit(j), a.cols, y, sc);
            }
        }
    }
}

// A row too long for the registers: the block walks it once for the sum of
// squares (storing h, if it is wanted) and again for the output, the second
// time from L2.
template <int XT, int RT, bool V8>
__global__ void __launch_bounds__(NORM_THREADS) k_norm_forward_long(const __grid_constant__ NormArgs a) {
    constexpr int E = Map::E;
    __shared__ __align__(16) float ssum[2][32];
    if (threadIdx.x < 64) ssum[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
    __syncthreads();
    __shared__ uint32_t smax[2][32];
    pdl_wait();
    pdl_launch_next();
    const float inv_n = 1.f / (float)a.cols;
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols), eh = extent_of<RT>(a.h, a.ldh, a.rows, a.cols);
    const int steps = ((a.cols + 7) / 8 + (int)blockDim.x - 1) / (int)blockDim.x;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const void* X = row_of<XT>(a.x, a.ldx, row);
        const void* R = a.r ? row_of<RT>(a.r, a.ldr, row) : nullptr;
        void* H = a.h ? row_of<RT>(a.h, a.ldh, row) : nullptr;
        auto value = [&](int u, float (&h)[E]) {      // h again, after it was stored over x or r
            if (H) {
                Unit<RT, V8> s;
                s.load(H, u, a.cols, eh);
                s.values(h);
            } else {
                Unit<XT, V8> x;
                Unit<RT, V8> r;
                x.load(X, u, a.cols, ex);
                if (R) r.load(R, u, a.cols, er);
                add_unit<XT, RT, V8>(x, r, R != nullptr).values(h);
            }
        };
        float ss = 0.f;
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            Unit<XT, V8> x;
            Unit<RT, V8> r;
            x.load(X, u, a.cols, ex);
            if (R) r.load(R, u, a.cols, er);
            const Unit<RT, V8> s = add_unit<XT, RT, V8>(x, r, R != nullptr);
            float h[E];
            s.values(h);
#pragma unroll
            for (int e = 0; e < E; ++e) ss = fmaf(h[e], h[e], ss);
            if (H) s.store(H, u, a.cols);
        }
        ss = block_sum(ss, ssum[turn]);
        const float rstd = rsqrtf(fmaf(ss, inv_n, a.eps));
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
        float whole = 0.f;
        if (a.y8 && !a.block128) {
            uint32_t top = 0;
            for (int j = 0; j < steps; ++j) {
                const int u = threadIdx.x + j * blockDim.x;
                float h[E], w[E];
                value(u, h);
                weights(a, u, w);
#pragma unroll
                for (int e = 0; e < E; ++e) top = max(top, abs_bits(h[e] * rstd * w[e]));
            }
            whole = scale_of(__uint_as_float(block_max(top, smax[turn])));
            if (threadIdx.x == 0) a.scale[row * a.n_scale] = whole;
        }
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            float h[E], w[E];
            value(u, h);
            weights(a, u, w);
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[e] = h[e] * rstd * w[e];
                top = max(top, abs_bits(h[e]));
            }
            if (!a.y8) {
                store_unit<XT, V8>(row_of<XT>(a.y, a.ldy, row), u, a.cols, h);
                continue;
            }
            float mm = whole;
            if (a.block128) {
                mm = scale_of(__uint_as_float(lanes_max<Map::LANES>(top)));
                if ((u & (Map::LANES - 1)) == 0 && Map::any(u, a.cols))
                    a.scale[row * a.n_scale + u / Map::LANES] = mm;
            }
            quantised_store<V8>(static_cast<uint8_t*>(a.y) + row * a.ldy, u, a.cols, h, mm);
        }
    }
}

// Backward: each block walks rows blockIdx.x, + grid, ...; a thread owns the
// same columns of all of them, so its part of dw stays in registers and is
// written once, as one row of `part`.
template <int XT, int RT, bool V8, int NV>
__global__ void __launch_bounds__(NORM_THREADS) k_norm_backward(const __grid_constant__ NormArgs a) {
    constexpr int E = Map::E;
    __shared__ __align__(16) float ssum[2][32];
    if (threadIdx.x < 64) ssum[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
    __syncthreads();
    pdl_wait();
    pdl_launch_next();
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols), eh = extent_of<RT>(a.hin, a.ldhin, a.rows, a.cols);
    uint64_t dw[NV][E / 2] = {};
    const float inv_n = 1.f / (float)a.cols;
    extern __shared__ __align__(16) uint4 ring[];
    using X = Slots<XT, NV, V8>;
    using R = Slots<RT, NV, V8>;
    const int S = a.stages, stage_words = X::words() + 2 * R::words();
    const bool DH = a.r != nullptr;
    auto copy = [&](int64_t row, int st) {
        if (row < a.rows) {
            uint4* at = ring + st * stage_words;
            X{at}.copy(row_of<XT>(a.x, a.ldx, row), a.cols, ex);
            R{at + X::words()}.copy(row_of<RT>(a.hin, a.ldhin, row), a.cols, eh);
            if (DH) R{at + X::words() + R::words()}.copy(row_of<RT>(a.r, a.ldr, row), a.cols, er);
        }
        copies_commit();
    };
    for (int st = 0; st < S - 1; ++st) copy(blockIdx.x + (int64_t)st * gridDim.x, st);
    uint64_t w[NV][E / 2];
    weight_pairs<NV>(a, w);
    int turn = 0, st = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const float rstd = a.rstd[row];
        Unit<XT, V8> dy[NV];
        Unit<RT, V8> h[NV], dh[NV];
        copy(row + (int64_t)(S - 1) * gridDim.x, st == 0 ? S - 1 : st - 1);
        copies_wait_all_but(S - 1);
        if (!V8) __syncthreads();
        uint4* at = ring + st * stage_words;
        X{at}.read(dy, row_of<XT>(a.x, a.ldx, row), a.cols);
        R{at + X::words()}.read(h, row_of<RT>(a.hin, a.ldhin, row), a.cols);
        if (DH) R{at + X::words() + R::words()}.read(dh, row_of<RT>(a.r, a.ldr, row), a.cols);
        st = st == S - 1 ? 0 : st + 1;
        const uint64_t rr = pack2(rstd, rstd);
        uint64_t d2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int q = 0; q < E / 2; ++q) {
                const uint64_t xh = mul2(h[j].pair(q), rr), g = dy[j].pair(q);
                dw[j][q] = fma2(g, xh, dw[j][q]);
                d2 = fma2(mul2(g, w[j][q]), xh, d2);
            }
        const float2 dp = unpack2(d2);
        const float c = block_sum(dp.x + dp.y, ssum[turn]) * inv_n;
        // dx = rstd g w + (dh - xh rstd c), the sum in the brackets first
        const uint64_t rc = pack2(-rstd * c, -rstd * c);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float v[E];
#pragma unroll
            for (int q = 0; q < E / 2; ++q) {
                const uint64_t t = fma2(mul2(h[j].pair(q), rr), rc, DH ? dh[j].pair(q) : 0ull);
                const float2 p = unpack2(fma2(mul2(dy[j].pair(q), w[j][q]), rr, t));
                v[2 * q] = p.x;
                v[2 * q + 1] = p.y;
            }
            store_unit<RT, V8>(row_of<RT>(a.y, a.ldy, row), Map::unit(j), a.cols, v);
        }
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = Map::unit(j) * 8;
        if (a.part16 && c + 8 <= a.cols) {
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                const float2 x = unpack2(dw[j][q]), y = unpack2(dw[j][q + 1]);
                *reinterpret_cast<float4*>(part + c + 2 * q) = make_float4(x.x, x.y, y.x, y.y);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 p = unpack2(dw[j][e / 2]);
                if (c + e < a.cols) part[c + e] = e % 2 ? p.y : p.x;
            }
        }
    }
}

// Rows too long for the registers: dx by walking the row twice, and dw by
// blocks that own 128 columns and a share of the rows (gridDim.y shares).
template <int XT, int RT, bool V8>
__global__ void __launch_bounds__(NORM_THREADS) k_norm_backward_long(const __grid_constant__ NormArgs a) {
    constexpr int E = Map::E;
    __shared__ __align__(16) float ssum[2][32];
    if (threadIdx.x < 64) ssum[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
    __syncthreads();
    pdl_wait();
    pdl_launch_next();
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols), eh = extent_of<RT>(a.hin, a.ldhin, a.rows, a.cols);
    const int steps = ((a.cols + 7) / 8 + (int)blockDim.x - 1) / (int)blockDim.x;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const void* DY = row_of<XT>(a.x, a.ldx, row);
        const void* H = row_of<RT>(a.hin, a.ldhin, row);
        const void* DH = a.r ? row_of<RT>(a.r, a.ldr, row) : nullptr;
        const float rstd = a.rstd[row];
        float dot = 0.f;
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            Unit<XT, V8> dy;
            Unit<RT, V8> h;
            dy.load(DY, u, a.cols, ex);
            h.load(H, u, a.cols, eh);
            float g[E], v[E], w[E];
            dy.values(g);
            h.values(v);
            weights(a, u, w);
#pragma unroll
            for (int e = 0; e < E; ++e) dot = fmaf(g[e] * w[e], v[e] * rstd, dot);
        }
        const float c = block_sum(dot, ssum[turn]) / (float)a.cols;
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            Unit<XT, V8> dy;
            Unit<RT, V8> h, dh;
            dy.load(DY, u, a.cols, ex);
            h.load(H, u, a.cols, eh);
            if (DH) dh.load(DH, u, a.cols, er);
            float g[E], v[E], w[E], up[E];
            dy.values(g);
            h.values(v);
            weights(a, u, w);
            if (DH) dh.values(up);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                g[e] = rstd * (g[e] * w[e] - v[e] * rstd * c);
                if (DH) g[e] += up[e];
            }
            store_unit<RT, V8>(row_of<RT>(a.y, a.ldy, row), u, a.cols, g);
        }
    }
}

// Launched before k_norm_backward_long, whose dx may overwrite dy or dh.
template <int XT, int RT>
__global__ void __launch_bounds__(128) k_norm_dw_long(const __grid_constant__ NormArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (c >= a.cols) return;
    float s = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
        s = fmaf(ld1<XT>(row_of<XT>(a.x, a.ldx, row), c), ld1<RT>(row_of<RT>(a.hin, a.ldhin, row), c) * a.rstd[row], s);
    a.part[(int64_t)blockIdx.y * a.cols + c] = s;
}

// dw[c] = sum of the n partial rows: each of the block's 32 warps adds every
// 32nd of them, a butterfly adds the warps' sums; added to what dw holds if
// accumulate.
__global__ void __launch_bounds__(1024) k_norm_dw(const float* part, int n, int64_t cols, void* dw, int dt,
                                                  int accumulate) {
    __shared__ float s[32][33];
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < cols) {
        const float* p = part + c;
#pragma unroll 8
        for (int i = k; i < n; i += 32) t += p[(int64_t)i * cols];
    }
    s[k][lane] = t;
    __syncthreads();
    // the transpose: warp k has column k of the block's 32
    t = warp_sum(s[lane][k]);
    const int64_t cc = (int64_t)blockIdx.x * 32 + k;
    if (lane || cc >= cols) return;
    if (accumulate) t += ld1_any(dw, cc, dt);
    st1_any(dw, cc, t, dt);
}

// ---------------------------------------------------------------- choice of the launch
template <int XT, int RT, bool V8>
static const void* forward_fn(int nv) {
    switch (nv) {
        case 2: return (const void*)k_norm_forward<XT, RT, V8, 2>;
        case 4: return (const void*)k_norm_forward<XT, RT, V8, 4>;
        default: return (const void*)k_norm_forward_long<XT, RT, V8>;
    }
}
template <int XT, int RT, bool V8>
static const void* backward_fn(int nv) {
    switch (nv) {
        case 2: return (const void*)k_norm_backward<XT, RT, V8, 2>;
        case 4: return (const void*)k_norm_backward<XT, RT, V8, 4>;
        default: return (const void*)k_norm_backward_long<XT, RT, V8>;
    }
}
template <int XT, int RT>
static const void* pick(bool fwd, bool v8, int nv) {
    if (fwd) return v8 ? forward_fn<XT, RT, true>(nv) : forward_fn<XT, RT, false>(nv);
    return v8 ? backward_fn<XT, RT, true>(nv) : backward_fn<XT, RT, false>(nv);
}
static const void* norm_fn(bool fwd, int xt, int rt, bool v8, int nv) {
    if (xt == ZERO_F32) return pick<ZERO_F32, ZERO_F32>(fwd, v8, nv);
    if (xt == ZERO_BF16)
        return rt == ZERO_F32 ? pick<ZERO_BF16, ZERO_F32>(fwd, v8, nv) : pick<ZERO_BF16, ZERO_BF16>(fwd, v8, nv);
    return rt == ZERO_F32 ? pick<ZERO_F16, ZERO_F32>(fwd, v8, nv) : pick<ZERO_F16, ZERO_F16>(fwd, v8, nv);
}

static int check_weight(const zero_mat* w, int64_t cols, NormArgs& a, const char* call) {
    if (!w) return ZERO_OK;
    const int rc = check_mat(w, 1, cols, FLOAT_TYPES, call, "weight");
    if (rc != ZERO_OK || cols == 0) return rc;
    a.w = w->data;
    a.wdt = w->dtype;
    a.w_aligned = aligned(w->data, 16);
    return ZERO_OK;
}

}  // namespace zdp

using namespace zdp;

extern "C" {

int zero_norm_forward(const zero_mat* x, const zero_mat* residual, const zero_mat* weight, int64_t rows, int64_t cols,
                      float eps, const zero_mat* h_out, const zero_mat* y, float* y_scale, int64_t scale_block,
                      float* rstd, void* stream) {
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "zero_norm_forward: negative rows or cols");
    if (cols > NORM_MAX_COLS) return fail(ZERO_ELIMIT, "zero_norm_forward: more than 1048576 columns");
    if (!(eps >= 0.f) || !(eps < INFINITY)) return fail(ZERO_EINVAL, "zero_norm_forward: eps must be finite and >= 0");
    int rc = check_mat(x, rows, cols, FLOAT_TYPES, "zero_norm_forward", "x");
    if (rc == ZERO_OK) rc = check_mat(y, rows, cols, FLOAT_TYPES | 1u << ZERO_E4M3, "zero_norm_forward", "y");
    if (rc == ZERO_OK && residual) rc = check_mat(residual, rows, cols, FLOAT_TYPES, "zero_norm_forward", "residual");
    if (rc == ZERO_OK && h_out) rc = check_mat(h_out, rows, cols, FLOAT_TYPES, "zero_norm_forward", "h_out");
    if (rc != ZERO_OK) return rc;
    const int rt = residual ? residual->dtype : x->dtype;
    if (rt != x->dtype && rt != ZERO_F32)
        return fail(ZERO_EINVAL, "zero_norm_forward: the residual is in x's type or fp32");
    if (h_out && h_out->dtype != rt)
        return fail(ZERO_EINVAL, "zero_norm_forward: h_out is in the residual's type (x's without one)");
    const bool y8 = y->dtype == ZERO_E4M3;
    if (!y8 && y->dtype != x->dtype) return fail(ZERO_EINVAL, "zero_norm_forward: y is in x's type or e4m3");
    if (y8 && (scale_block != 0 && scale_block != 128))
        return fail(ZERO_EINVAL, "zero_norm_forward: scale_block is 0 (a scale per row) or 128");
    if (y8 && rows > 0 && cols > 0 && !y_scale) return fail(ZERO_EINVAL, "zero_norm_forward: e4m3 output needs y_scale");
    if (!aligned(y_scale, 4) || !aligned(rstd, 4)) return fail(ZERO_EALIGN, "zero_norm_forward: y_scale or rstd not 4-byte aligned");
    NormArgs a = {};
    rc = check_weight(weight, cols, a, "zero_norm_forward");
    if (rc != ZERO_OK || rows == 0 || cols == 0) return rc;
    a.x = x->data;
    a.ldx = x->ld;
    a.r = residual ? residual->data : nullptr;
    a.ldr = residual ? residual->ld : 0;
    a.h = h_out ? h_out->data : nullptr;
    a.ldh = h_out ? h_out->ld : 0;
    a.y = y->data;
    a.ldy = y->ld;
    a.rows = rows;
    a.cols = (int)cols;
    a.eps = eps;
    a.y8 = y8;
    a.block128 = y8 && scale_block == 128;
    a.n_scale = a.block128 ? (cols + 127) / 128 : 1;
    a.scale = y_scale;
    a.rstd = rstd;
    const bool y_ok = y8 ? aligned(y->data, 8) && (rows == 1 || y->ld % 8 == 0) : rows_aligned(*y, rows);
    const bool v8 = cols % 8 == 0 && rows_aligned(*x, rows) && y_ok && (!residual || rows_aligned(*residual, rows)) &&
                    (!h_out || rows_aligned(*h_out, rows));
    const NormShape p = shape_of(cols, words_of(x->dtype) + words_of(rt), NORM_FORWARD_THREADS);
    a.stages = p.stages;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    const void* f = norm_fn(true, x->dtype, rt, v8, p.nv);
    rc = raise_smem(f, p.smem, "zero_norm_forward shared-memory size");
    if (rc != ZERO_OK) return rc;
    const int64_t most = (int64_t)sms * p.per_sm * NORM_FORWARD_OVER;
    void* args[] = {&a};
    return cuda_fail(launch_after_previous(f, (int)(rows < most ? rows : most), p.threads, args, p.smem,
                                           static_cast<cudaStream_t>(stream)),
                     "zero_norm_forward launch");
}

size_t zero_norm_workspace_bytes(int64_t cols) {
    return cols > 0 && cols <= NORM_MAX_COLS ? (size_t)NORM_MAX_GRID * (size_t)cols * 4 : 0;
}

int zero_norm_backward(const zero_mat* dy, const zero_mat* h, const zero_mat* weight, int64_t rows, int64_t cols,
                       const float* rstd, const zero_mat* dh, const zero_mat* dx, const zero_mat* dw, int accumulate,
                       void* workspace, size_t workspace_bytes, void* stream) {
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "zero_norm_backward: negative rows or cols");
    if (cols > NORM_MAX_COLS) return fail(ZERO_ELIMIT, "zero_norm_backward: more than 1048576 columns");
    int rc = check_mat(dy, rows, cols, FLOAT_TYPES, "zero_norm_backward", "dy");
    if (rc == ZERO_OK) rc = check_mat(h, rows, cols, FLOAT_TYPES, "zero_norm_backward", "h");
    if (rc == ZERO_OK) rc = check_mat(dx, rows, cols, FLOAT_TYPES, "zero_norm_backward", "dx");
    if (rc == ZERO_OK && dh) rc = check_mat(dh, rows, cols, FLOAT_TYPES, "zero_norm_backward", "dh");
    if (rc == ZERO_OK && dw) rc = check_mat(dw, 1, cols, FLOAT_TYPES, "zero_norm_backward", "dw");
    if (rc != ZERO_OK) return rc;
    const int rt = h->dtype;
    if (rt != dy->dtype && rt != ZERO_F32) return fail(ZERO_EINVAL, "zero_norm_backward: h is in dy's type or fp32");
    if (dx->dtype != rt || (dh && dh->dtype != rt)) return fail(ZERO_EINVAL, "zero_norm_backward: dx and dh are in h's type");
    if (rows > 0 && cols > 0 && (!rstd || !aligned(rstd, 4)))
        return fail(ZERO_EINVAL, "zero_norm_backward: rstd NULL or not 4-byte aligned");
    if (dw && cols > 0 && (!workspace || !aligned(workspace, 4) || workspace_bytes < zero_norm_workspace_bytes(cols)))
        return fail(ZERO_EWORKSPACE, "zero_norm_backward: workspace smaller than zero_norm_workspace_bytes(cols)");
    NormArgs a = {};
    rc = check_weight(weight, cols, a, "zero_norm_backward");
    if (rc != ZERO_OK || cols == 0) return rc;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    a.x = dy->data;
    a.ldx = dy->ld;
    a.hin = h->data;
    a.ldhin = h->ld;
    a.r = dh ? dh->data : nullptr;
    a.ldr = dh ? dh->ld : 0;
    a.y = dx->data;
    a.ldy = dx->ld;
    a.rows = rows;
    a.cols = (int)cols;
    a.rstd = const_cast<float*>(rstd);
    a.part = dw ? static_cast<float*>(workspace) : nullptr;
    a.part16 = cols % 4 == 0 && aligned(workspace, 16);
    const bool v8 = cols % 8 == 0 && rows_aligned(*dy, rows) && rows_aligned(*h, rows) && rows_aligned(*dx, rows) &&
                    (!dh || rows_aligned(*dh, rows));
    const NormShape p = shape_of(cols, words_of(dy->dtype) + 2 * words_of(rt), NORM_BACKWARD_THREADS);
    a.stages = p.stages;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* args[] = {&a};
    int64_t g = (int64_t)p.per_sm * sms;
    if (g > NORM_MAX_GRID) g = NORM_MAX_GRID;
    if (g > rows) g = rows;
    const void* f = norm_fn(false, dy->dtype, rt, v8, p.nv);
    rc = raise_smem(f, p.smem, "zero_norm_backward shared-memory size");
    if (rc != ZERO_OK) return rc;
    int parts = (int)g;
    if (p.nv == 0 && dw && rows > 0) {
        // dw first: dx may be written over dy or dh
        const int64_t chunks = (cols + 127) / 128;
        int64_t shares = (8 * (int64_t)sms + chunks - 1) / chunks;
        if (shares > NORM_MAX_GRID) shares = NORM_MAX_GRID;
        if (shares > rows) shares = rows;
        parts = (int)shares;
        const dim3 grid((unsigned)chunks, (unsigned)shares);
        const void* fw = dy->dtype == ZERO_F32 ? (const void*)k_norm_dw_long<ZERO_F32, ZERO_F32>
                       : dy->dtype == ZERO_BF16 ? (rt == ZERO_F32 ? (const void*)k_norm_dw_long<ZERO_BF16, ZERO_F32>
                                                                  : (const void*)k_norm_dw_long<ZERO_BF16, ZERO_BF16>)
                                                : (rt == ZERO_F32 ? (const void*)k_norm_dw_long<ZERO_F16, ZERO_F32>
                                                                  : (const void*)k_norm_dw_long<ZERO_F16, ZERO_F16>);
        rc = cuda_fail(cudaLaunchKernel(fw, grid, dim3(128), args, 0, s), "zero_norm_backward dw launch");
        if (rc != ZERO_OK) return rc;
    }
    if (rows > 0) {
        if (p.nv == 0) g = rows < 1 << 30 ? rows : 1 << 30;
        rc = cuda_fail(launch_after_previous(f, (int)g, p.threads, args, p.smem, s), "zero_norm_backward launch");
        if (rc != ZERO_OK) return rc;
    }
    if (!dw) return ZERO_OK;
    const float* part = a.part;
    int n = rows > 0 ? parts : 0, dt = dw->dtype;
    int64_t nc = cols;
    void* out = dw->data;
    void* wargs[] = {&part, &n, &nc, &out, &dt, &accumulate};
    return cuda_fail(launch_after_previous((const void*)k_norm_dw, (int)((cols + 31) / 32), 1024, wargs, 0, s),
                     "zero_norm_backward dw reduction launch");
}

}  // extern "C"
