// zero_layernorm_backward.cu -- the layer norm's gradients, with the sums over
// the rows for its weight and bias, and the gradient behind the dropout.
//
// With xh = (h - m) rstd and g = dy w:
//   dr = rstd (g - mean(g) - xh mean(g xh)) + dh     (of h, and so of r)
//   dx = dropout(dr)                                 (of x, by the forward's mask)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound: HBM (dy, h and dh read, dr and dx written).  Rows are shared out as in
// the forward pass (zero_layernorm.cuh); a lane owns the same columns of all its
// rows, so its parts of dw and db stay in registers, a block adds its groups'
// parts and writes one, and k_layernorm_sums adds the blocks' in order.
//
// Measured (GB300, with dw and db; in brackets the share of the measured copy
// bandwidth): 16384 x 3456 bf16 in 84 us (0.80), behind a dropout, with dx too, 117
// (0.72); fp16 with an fp32 stream 120 (0.98); 8192 x 4096 fp32 88 (0.90); 8192 x
// 1600 bf16 28 (0.55: five of them the sums' launch), behind a dropout 37.
// 16-bit rows take 36 instructions an element (with the generator's and dx's 56),
// and narrow ones are bound by latency: 8192 x 1600 fills half of the issue slots.
// Rows that start anywhere: 8192 x 4097 bf16 155 (0.26), fp32 167 (0.47).  Rows past 15360 columns (with a weight
// of another type 13312; onto an fp32 stream 9216 and 9000; fp32 7680) are walked
// twice and their columns' sums taken by a pass of its own: 2048 x 20480 bf16 in 220
// (0.23).
#include "zero_layernorm.cuh"

namespace zdp {

// Sums of two values over the block, the same in every thread and every run.
// s: 32 pairs that no call in flight uses, zero beyond the block's warps.
__device__ __forceinline__ float2 block_sum2(float x, float y, float2* s) {
    x = warp_sum(x);
    y = warp_sum(y);
    if (blockDim.x <= 32) return make_float2(x, y);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    const int n2 = (blockDim.x + 63) >> 6;
    float tx = 0.f, ty = 0.f;
    for (int w = 0; w < n2; ++w) {
        const float4 p = reinterpret_cast<const float4*>(s)[w];
        tx += p.x + p.z;
        ty += p.y + p.w;
    }
    return make_float2(tx, ty);
}

// dropout of a unit's gradient, by the forward's mask
__device__ __forceinline__ void dropped(const DropArgs& d, uint32_t step, int64_t unit, float (&v)[8]) {
    const uint4 bits = drop_bits(d, step, unit);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t w = word_of(bits, q);
        v[2 * q] = kept_low(w, d.above) ? v[2 * q] * d.scale : 0.f;
        v[2 * q + 1] = kept_high(w, d.above) ? v[2 * q + 1] * d.scale : 0.f;
    }
}

// Values are read from shared
// memory for the sums and again for the gradients: registers hold the lane's
// parts of dw and db.  The rows' mean and rstd are read a row ahead; the block's
// G parts of dw and db are added in order, so that a block writes one.
template <int XT, int RT, int WT, int NV, bool SHIFT>
__global__ void __launch_bounds__(LN_THREADS, 1) k_layernorm_backward_rows(const __grid_constant__ LayerNormArgs a) {
    __shared__ __align__(16) float2 ssum[2][32];
    using X = Lane<XT, NV, SHIFT>;
    using R = Lane<RT, NV, SHIFT>;
    using V = Vector<WT>;
    constexpr int XS = 8 * Elem<XT>::SIZE, RS = 8 * Elem<RT>::SIZE;          // bytes of a unit
    const int T = a.T, G = blockDim.x / T, group = threadIdx.x / T, units = a.units;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T >> 5, w0 = group * warps;
    const int uw = (warp - w0) * NV * 32, left = units - uw;                 // the warp's first unit, units from there
    const int n = SHIFT ? (left + 31) >> 5 : (left - lane + 31) >> 5;        // the warp's js, or this lane's (any number above NV: all)
    const int wcols = a.cols - uw * 8, lcols = wcols - lane * 8;             // columns from the warp's first on, from this lane's
    pdl_wait();
    pdl_launch_next();
    const uint32_t step = drop_step(a.drop);
    const float inv_n = 1.f / (float)a.cols;
    extern __shared__ __align__(16) uint4 ring[];
    const int nw = blockDim.x >> 5, S = a.stages, xwords = nw * X::WORDS, rwords = nw * R::WORDS, stage_words = xwords + 2 * rwords;
    const int64_t first = group * (int64_t)gridDim.x + blockIdx.x, every = (int64_t)G * gridDim.x;
    const bool DH = a.r != nullptr;
    uint4 *const gat = ring + warp * X::WORDS, *const hat = ring + xwords + warp * R::WORDS, *const uat = hat + rwords;
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols),
                 eh = extent_of<RT>(a.hin, a.ldhin, a.rows, a.cols);
    const char* cg = static_cast<const char*>(a.x) + first * a.ldx * Elem<XT>::SIZE + (int64_t)uw * XS;
    const char* ch = static_cast<const char*>(a.hin) + first * a.ldhin * Elem<RT>::SIZE + (int64_t)uw * RS;
    const char* cu = static_cast<const char*>(a.r) + (DH ? first * a.ldr * Elem<RT>::SIZE + (int64_t)uw * RS : 0);
    const int64_t dg = every * a.ldx * Elem<XT>::SIZE, dh = every * a.ldhin * Elem<RT>::SIZE, du = every * a.ldr * Elem<RT>::SIZE;
    char* DR = static_cast<char*>(a.y) + (a.y ? first * a.ldy * Elem<RT>::SIZE + (int64_t)uw * RS : 0);
    char* DX = static_cast<char*>(a.h) + (a.h ? first * a.ldh * Elem<XT>::SIZE + (int64_t)uw * XS : 0);
    const int64_t ddr = every * a.ldy * Elem<RT>::SIZE, ddx = every * a.ldh * Elem<XT>::SIZE;
    int64_t crow = first;
    auto copy = [&](int st) {
        if (crow < a.rows) {
            X::copy(gat + st * stage_words, cg, wcols, ex);
            R::copy(hat + st * stage_words, ch, wcols, eh);
            if (DH) R::copy(uat + st * stage_words, cu, wcols, er);
        }
        copies_commit();
        crow += every;
        cg += dg;
        ch += dh;
        cu += du;
    };
    for (int s = 0; s < S - 1; ++s) copy(s);
    uint4* const wat = ring + S * stage_words;
    V::fill(wat, a.w, a.wdt, a.w_aligned, a.cols, units, 1.f);
    __syncthreads();
    uint64_t dw[NV][4] = {}, db[NV][4] = {};
    float mean = 0.f, rstd = 0.f;
    if (first < a.rows) {
        mean = a.mean[first];
        rstd = a.rstd[first];
    }
    int turn = 0, st = 0;
    for (int64_t row = first; row < a.rows; row += every, turn ^= 1) {
        copy(st == 0 ? S - 1 : st - 1);
        float next_mean = 0.f, next_rstd = 0.f;
        if (row + every < a.rows) {
            next_mean = a.mean[row + every];
            next_rstd = a.rstd[row + every];
        }
        copies_wait_all_but(S - 1);
        if (X::SHARED || R::SHARED) __syncwarp();
        const int goff = X::off(cg - S * dg), hoff = R::off(ch - S * dh), uoff = R::off(cu - S * du);
        uint4 *const gs = gat + st * stage_words, *const hs = hat + st * stage_words, *const us = uat + st * stage_words;
        st = st == S - 1 ? 0 : st + 1;
        const uint64_t rr = pack2(rstd, rstd), mm = pack2(-mean, -mean);
        uint64_t g2 = 0, d2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j < n) {
                const int u = SHIFT ? min(uw + lane + 32 * j, units - 1) : uw + lane + 32 * j;
                // past the row's end dy and h are 0 (the next row's may be infinite), and with them every term
                const Raw8<XT> dy = X::read(gs, j, goff, lcols - 256 * j);
                const Raw8<RT> h = R::read(hs, j, hoff, lcols - 256 * j);
                const Raw8<WT> w = V::read(wat, u, units);
                if (SHIFT) {                                 // shifted once, not twice
                    __syncwarp();
                    X::write(gs, j, dy);
                    R::write(hs, j, h);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint64_t xh = mul2(add2(pair8<RT>(h, q), mm), rr), g = pair8<XT>(dy, q), gw = mul2(g, pair8<WT>(w, q));
                    dw[j][q] = fma2(g, xh, dw[j][q]);
                    db[j][q] = add2(g, db[j][q]);
                    g2 = add2(g2, gw);
                    d2 = fma2(gw, xh, d2);
                }
            }
        const float2 gp = unpack2(g2), dp = unpack2(d2);
        float sx = warp_sum(gp.x + gp.y), sy = warp_sum(dp.x + dp.y);
        if (warps > 1) {
            if (lane == 0) ssum[turn][warp] = make_float2(sx, sy);
            row_barrier(group, T);
            sx = sy = 0.f;
#pragma unroll 4
            for (int k = 0; k < warps; ++k) {
                const float2 p = ssum[turn][w0 + k];
                sx += p.x;
                sy += p.y;
            }
        }
        asm volatile("" ::: "memory");                       // the values are read again, not kept
        // dr = rstd g w + (dh - rstd c1 - xh rstd c2), the sum in the brackets first
        const float c1 = -rstd * (sx * inv_n), c2 = -rstd * (sy * inv_n);
        const uint64_t p1 = pack2(c1, c1), p2 = pack2(c2, c2);
        Put<RT, NV, SHIFT> putr;
        Put<XT, NV, SHIFT> putx;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j < n) {
                const int u = SHIFT ? min(uw + lane + 32 * j, units - 1) : uw + lane + 32 * j;
                const Raw8<XT> dy = Lane<XT, NV, false>::read(gs, j, 0, 8);
                const Raw8<RT> h = Lane<RT, NV, false>::read(hs, j, 0, 8);
                const Raw8<WT> w = V::read(wat, u, units);
                Raw8<RT> up;
                if (DH) up = R::read(us, j, uoff, 8);
                float v[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint64_t xh = mul2(add2(pair8<RT>(h, q), mm), rr);
                    const uint64_t t = fma2(xh, p2, DH ? add2(pair8<RT>(up, q), p1) : p1);
                    const float2 p = unpack2(fma2(mul2(pair8<XT>(dy, q), pair8<WT>(w, q)), rr, t));
                    v[2 * q] = p.x;
                    v[2 * q + 1] = p.y;
                }
                if (a.y) putr.put(DR, hs, j, lcols - 256 * j, a.y32, narrow8<RT>(v));
                if (a.h) {
                    if (a.drop.on) dropped(a.drop, step, row * units + u, v);
                    putx.put(DX, gs, j, lcols - 256 * j, a.h32, narrow8<XT>(v));
                }
            }
        if (a.y) putr.end(DR, hs, wcols);
        if (a.h) putx.end(DX, gs, wcols);
        DR += ddr;
        DX += ddx;
        mean = next_mean;
        rstd = next_rstd;
        if (X::SHARED || R::SHARED) __syncwarp();            // the next copies land in words that other lanes read
    }
    if (!a.part) return;
    // the groups' parts by shared memory: 4 words of 4 columns for each unit of dw, then of db, threads side by side
    copies_wait<0>();
    __syncthreads();
    float4* P = reinterpret_cast<float4*>(ring);
    const int all = blockDim.x;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
            const float2 x = unpack2(dw[j][q]), y = unpack2(dw[j][q + 1]), s = unpack2(db[j][q]), t = unpack2(db[j][q + 1]);
            P[(j * 4 + q / 2) * all + threadIdx.x] = make_float4(x.x, x.y, y.x, y.y);
            P[(j * 4 + 2 + q / 2) * all + threadIdx.x] = make_float4(s.x, s.y, t.x, t.y);
        }
    __syncthreads();
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    for (int i = threadIdx.x; i < NV * 4 * T; i += all) {
        const int k = i / T, t = i - k * T, u = (t >> 5) * NV * 32 + (k >> 2) * 32 + (t & 31);
        if (u * 8 + (k & 1) * 4 >= a.cols) continue;
        float4 sum = P[k * all + t];
        for (int g = 1; g < G; ++g) {
            const float4 p = P[k * all + g * T + t];
            sum.x += p.x;
            sum.y += p.y;
            sum.z += p.z;
            sum.w += p.w;
        }
        float* to = part + (k & 2 ? a.cols : 0) + u * 8 + (k & 1) * 4;
        if (a.part16) {
            *reinterpret_cast<float4*>(to) = sum;            // columns a multiple of 4: all of them, or none
        } else {
            const float f[4] = {sum.x, sum.y, sum.z, sum.w};
            for (int e = 0; e < 4; ++e)
                if (u * 8 + (k & 1) * 4 + e < a.cols) to[e] = f[e];
        }
    }
}

// Rows too long for the registers: dr and dx by walking the row twice, dw and db
// by blocks that own 128 columns and a share of the rows (gridDim.y shares).
template <int XT, int RT, bool V8>
__global__ void __launch_bounds__(NORM_THREADS) k_layernorm_backward_long(const __grid_constant__ LayerNormArgs a) {
    constexpr int E = Map::E;
    __shared__ __align__(16) float2 ssum[2][32];
    if (threadIdx.x < 64) ssum[threadIdx.x >> 5][threadIdx.x & 31] = make_float2(0.f, 0.f);
    __syncthreads();
    pdl_wait();
    pdl_launch_next();
    const uint32_t step = drop_step(a.drop);
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols),
                 eh = extent_of<RT>(a.hin, a.ldhin, a.rows, a.cols);
    const int steps = (a.units + (int)blockDim.x - 1) / (int)blockDim.x;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const void* DY = row_of<XT>(a.x, a.ldx, row);
        const void* H = row_of<RT>(a.hin, a.ldhin, row);
        const void* DH = a.r ? row_of<RT>(a.r, a.ldr, row) : nullptr;
        const float rstd = a.rstd[row], mean = a.mean[row];
        float s1 = 0.f, s2 = 0.f;
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            Unit<XT, V8> dy;
            Unit<RT, V8> h;
            dy.load(DY, u, a.cols, ex);
            h.load(H, u, a.cols, eh);
            float g[E], v[E], w[E];
            dy.values(g);
            h.values(v);
            vector8(a.w, a.wdt, a.w_aligned, a.cols, u, 1.f, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s1 = fmaf(g[e], w[e], s1);
                s2 = fmaf(g[e] * w[e], (v[e] - mean) * rstd, s2);
            }
        }
        const float2 c = block_sum2(s1, s2, ssum[turn]);
        const float c1 = c.x / (float)a.cols, c2 = c.y / (float)a.cols;
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
            vector8(a.w, a.wdt, a.w_aligned, a.cols, u, 1.f, w);
            if (DH) dh.values(up);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                g[e] = rstd * (g[e] * w[e] - c1 - (v[e] - mean) * rstd * c2);
                if (DH) g[e] += up[e];
            }
            if (a.y) store_unit<RT, V8>(row_of<RT>(a.y, a.ldy, row), u, a.cols, g);
            if (a.h) {
                if (a.drop.on) dropped(a.drop, step, row * a.units + u, g);
                store_unit<XT, V8>(row_of<XT>(a.h, a.ldh, row), u, a.cols, g);
            }
        }
    }
}

// Launched before k_layernorm_backward_long, whose outputs may overwrite dy or dh.
template <int XT, int RT>
__global__ void __launch_bounds__(128) k_layernorm_sums_long(const __grid_constant__ LayerNormArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (c >= a.cols) return;
    float s = 0.f, t = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float g = ld1<XT>(row_of<XT>(a.x, a.ldx, row), c);
        s = fmaf(g, (ld1<RT>(row_of<RT>(a.hin, a.ldhin, row), c) - a.mean[row]) * a.rstd[row], s);
        t += g;
    }
    float* part = a.part + (int64_t)blockIdx.y * 2 * a.cols;
    part[c] = s;
    part[a.cols + c] = t;
}

// dw (the first half of the blocks) and db from the n partial rows of each: every
// one of the block's 32 warps adds every 32nd of them, a butterfly adds the warps' sums;
// added to what is there if accumulate.
struct SumsArgs {
    const float* part;
    int n, accumulate;
    int64_t cols;
    void* out[2];
    int dt[2];
};
__global__ void __launch_bounds__(1024) k_layernorm_sums(const __grid_constant__ SumsArgs a) {
    __shared__ float s[32][33];
    pdl_wait();
    pdl_launch_next();
    const int chunks = gridDim.x / 2, which = blockIdx.x >= chunks, chunk = blockIdx.x - which * chunks;
    void* out = a.out[which];
    if (!out) return;
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, dt = a.dt[which];
    const int64_t c = (int64_t)chunk * 32 + lane;
    float t = 0.f;
    if (c < a.cols) {
        const float* p = a.part + which * a.cols + c;
#pragma unroll 8
        for (int i = k; i < a.n; i += 32) t += p[(int64_t)i * 2 * a.cols];
    }
    s[k][lane] = t;
    __syncthreads();
    // the transpose: warp k has column k of the block's 32
    t = warp_sum(s[lane][k]);
    const int64_t cc = (int64_t)chunk * 32 + k;
    if (lane || cc >= a.cols) return;
    if (a.accumulate) t += ld1_any(out, cc, dt);
    st1_any(out, cc, t, dt);
}

// Partial rows of dw and db: one of each block, of which an SM has one.  Counted in
// a GB300's 152 SMs, whatever the device, since the workspace's size follows from it.
constexpr int LN_PARTS = 152;
constexpr int64_t LN_ROWS_COLS = (int64_t)LN_THREADS * 4 * 8;            // past these a row is walked, whatever its type
// Shares of the rows where they are walked: eight blocks an SM, of 128 columns each.
static int64_t long_shares(int64_t cols) {
    const int64_t chunks = (cols + 127) / 128;
    return (8 * LN_PARTS + chunks - 1) / chunks;
}
static_assert(8 * LN_PARTS / (7680 / 128) < LN_PARTS, "rows that are walked though shorter than LN_ROWS_COLS have fewer shares than blocks");

// packed: the weight in shared memory in dy's type, not in fp32.
template <int XT, int RT, bool SHIFT>
static const void* rows_of(bool packed, int nv) {
    if constexpr (XT != ZERO_F32)
        if (nv == 4)
            return packed ? (const void*)k_layernorm_backward_rows<XT, RT, XT, 4, SHIFT>
                          : (const void*)k_layernorm_backward_rows<XT, RT, ZERO_F32, 4, SHIFT>;
    return (const void*)k_layernorm_backward_rows<XT, RT, ZERO_F32, 2, SHIFT>;
}
template <int XT, int RT>
static const void* fn_of(bool v8, bool packed, int nv) {
    if (nv) return v8 ? rows_of<XT, RT, false>(packed, nv) : rows_of<XT, RT, true>(packed, nv);
    return v8 ? (const void*)k_layernorm_backward_long<XT, RT, true> : (const void*)k_layernorm_backward_long<XT, RT, false>;
}
// nv 0: rows too long for the registers.
static const void* backward_fn(int xt, int rt, bool v8, bool packed, int nv) {
    if (xt == ZERO_F32) return fn_of<ZERO_F32, ZERO_F32>(v8, packed, nv);
    if (xt == ZERO_BF16) return rt == ZERO_F32 ? fn_of<ZERO_BF16, ZERO_F32>(v8, packed, nv) : fn_of<ZERO_BF16, ZERO_BF16>(v8, packed, nv);
    return rt == ZERO_F32 ? fn_of<ZERO_F16, ZERO_F32>(v8, packed, nv) : fn_of<ZERO_F16, ZERO_F16>(v8, packed, nv);
}
static const void* sums_long_fn(int xt, int rt) {
    if (xt == ZERO_F32) return (const void*)k_layernorm_sums_long<ZERO_F32, ZERO_F32>;
    if (xt == ZERO_BF16)
        return rt == ZERO_F32 ? (const void*)k_layernorm_sums_long<ZERO_BF16, ZERO_F32>
                              : (const void*)k_layernorm_sums_long<ZERO_BF16, ZERO_BF16>;
    return rt == ZERO_F32 ? (const void*)k_layernorm_sums_long<ZERO_F16, ZERO_F32>
                          : (const void*)k_layernorm_sums_long<ZERO_F16, ZERO_F16>;
}

}  // namespace zdp

using namespace zdp;

extern "C" {

size_t zero_layernorm_workspace_bytes(int64_t cols) {
    if (cols <= 0 || cols > NORM_MAX_COLS) return 0;
    return (size_t)(cols > LN_ROWS_COLS ? long_shares(cols) : LN_PARTS) * (size_t)cols * 8;
}

int zero_layernorm_backward(const zero_mat* dy, const zero_mat* h, const zero_mat* weight, int64_t rows, int64_t cols,
                            const float* mean, const float* rstd, const zero_mat* dh, const zero_drop* drop,
                            const zero_mat* dr, const zero_mat* dx, const zero_mat* dw, const zero_mat* db, int accumulate,
                            void* workspace, size_t workspace_bytes, void* stream) {
    const char* me = "zero_layernorm_backward";
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "zero_layernorm_backward: negative rows or cols");
    if (cols > NORM_MAX_COLS) return fail(ZERO_ELIMIT, "zero_layernorm_backward: more than 1048576 columns");
    int rc = check_mat(dy, rows, cols, FLOAT_TYPES, me, "dy");
    if (rc == ZERO_OK) rc = check_mat(h, rows, cols, FLOAT_TYPES, me, "h");
    if (rc == ZERO_OK && weight) rc = check_mat(weight, 1, cols, FLOAT_TYPES, me, "weight");
    if (rc == ZERO_OK && dh) rc = check_mat(dh, rows, cols, FLOAT_TYPES, me, "dh");
    if (rc == ZERO_OK && dr) rc = check_mat(dr, rows, cols, FLOAT_TYPES, me, "dr");
    if (rc == ZERO_OK && dx) rc = check_mat(dx, rows, cols, FLOAT_TYPES, me, "dx");
    if (rc == ZERO_OK && dw) rc = check_mat(dw, 1, cols, FLOAT_TYPES, me, "dw");
    if (rc == ZERO_OK && db) rc = check_mat(db, 1, cols, FLOAT_TYPES, me, "db");
    if (rc != ZERO_OK) return rc;
    if (!dr && !dx) return fail(ZERO_EINVAL, "zero_layernorm_backward: neither dr nor dx");
    const int rt = h->dtype;
    if (rt != dy->dtype && rt != ZERO_F32) return fail(ZERO_EINVAL, "zero_layernorm_backward: h is in dy's type or fp32");
    if ((dr && dr->dtype != rt) || (dh && dh->dtype != rt))
        return fail(ZERO_EINVAL, "zero_layernorm_backward: dr and dh are in h's type");
    if (dx && dx->dtype != dy->dtype) return fail(ZERO_EINVAL, "zero_layernorm_backward: dx is in dy's type");
    if (rows > 0 && cols > 0 && (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)))
        return fail(ZERO_EINVAL, "zero_layernorm_backward: mean or rstd NULL or not 4-byte aligned");
    if ((dw || db) && cols > 0 &&
        (!workspace || !aligned(workspace, 4) || workspace_bytes < zero_layernorm_workspace_bytes(cols)))
        return fail(ZERO_EWORKSPACE, "zero_layernorm_backward: workspace smaller than zero_layernorm_workspace_bytes(cols)");
    LayerNormArgs a = {};
    rc = check_drop(drop, a.drop, me);
    if (rc != ZERO_OK || cols == 0) return rc;
    const int all = sm_count(), sms = all < LN_PARTS ? all : LN_PARTS;
    if (!sms) return ZERO_ECUDA;
    a.x = dy->data;
    a.ldx = dy->ld;
    a.hin = h->data;
    a.ldhin = h->ld;
    a.r = dh ? dh->data : nullptr;
    a.ldr = dh ? dh->ld : 0;
    a.y = dr ? dr->data : nullptr;
    a.ldy = dr ? dr->ld : 0;
    a.h = dx ? dx->data : nullptr;
    a.ldh = dx ? dx->ld : 0;
    if (weight) {
        a.w = weight->data;
        a.wdt = weight->dtype;
        a.w_aligned = aligned(weight->data, 16);
    }
    a.rows = rows;
    a.cols = (int)cols;
    a.units = (int)((cols + 7) / 8);
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = dw || db ? static_cast<float*>(workspace) : nullptr;
    a.part16 = cols % 4 == 0 && aligned(workspace, 16);
    const bool v8 = cols % 8 == 0 && rows_aligned(*dy, rows) && rows_aligned(*h, rows) && (!dr || rows_aligned(*dr, rows)) &&
                    (!dx || rows_aligned(*dx, rows)) && (!dh || rows_aligned(*dh, rows));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* args[] = {&a};
    int parts = 0;
    const int words = words_of(dy->dtype) + 2 * words_of(rt);
    const bool w16 = dy->dtype != ZERO_F32 && (!weight || weight->dtype == dy->dtype);
    RowsShape rs = {};
    int nv = 4;
    bool packed = false;
    if (rows > 0) {
        // of fp32 rows shared memory holds more threads with two units each, whatever the sizes
        rs = dy->dtype == ZERO_F32 ? rows_shape(rows, cols, nv = 2, words, 2, sms) : rows_shape(rows, cols, words, 2, sms, &nv);
        // four units a lane and the shifts beside the sums do not fit the registers: only where two leave the block few threads
        // (8192 x 4097, one row of 288 threads or three of 160)
        if (!v8 && nv == 4) {
            const RowsShape two = rows_shape(rows, cols, 2, words, 2, sms);
            if (two.threads * 5 > rs.threads * 4) {
                rs = two;
                nv = 2;
            }
        }
        packed = !rs.threads && w16;
        if (packed) rs = rows_shape(rows, cols, nv = 4, words, 1, sms);
    }
    if (rs.threads) {
        const void* f = backward_fn(dy->dtype, rt, v8, packed, nv);
        a.stages = rs.stages;
        a.T = rs.T;
        a.y32 = dr && rows_on_32(*dr, rows);
        a.h32 = dx && rows_on_32(*dx, rows);
        parts = rs.grid;
        // at the end the parts of dw and db lie where the stages were
        const size_t ends = (size_t)rs.threads * nv * 64, smem = rs.smem > ends ? rs.smem : ends;
        rc = raise_smem(f, smem, "zero_layernorm_backward shared-memory size");
        if (rc != ZERO_OK) return rc;
        rc = cuda_fail(launch_after_previous(f, rs.grid, rs.threads, args, smem, s), "zero_layernorm_backward launch");
        if (rc != ZERO_OK) return rc;
    } else if (rows > 0) {
        if (a.part) {
            // dw and db first: dr and dx may be written over dy or dh
            const int64_t chunks = (cols + 127) / 128, most = long_shares(cols), shares = rows < most ? rows : most;
            parts = (int)shares;
            const dim3 grid((unsigned)chunks, (unsigned)shares);
            rc = cuda_fail(cudaLaunchKernel(sums_long_fn(dy->dtype, rt), grid, dim3(128), args, 0, s),
                           "zero_layernorm_backward sums launch");
            if (rc != ZERO_OK) return rc;
        }
        const int g = (int)(rows < 1 << 30 ? rows : 1 << 30);
        rc = cuda_fail(launch_after_previous(backward_fn(dy->dtype, rt, v8, false, 0), g, NORM_THREADS, args, 0, s),
                       "zero_layernorm_backward launch");
        if (rc != ZERO_OK) return rc;
    }
    if (!a.part) return ZERO_OK;
    SumsArgs sums = {a.part, parts, accumulate, cols, {dw ? dw->data : nullptr, db ? db->data : nullptr},
                     {dw ? dw->dtype : 0, db ? db->dtype : 0}};
    void* sargs[] = {&sums};
    return cuda_fail(launch_after_previous((const void*)k_layernorm_sums, (int)((cols + 31) / 32) * 2, 1024, sargs, 0, s),
                     "zero_layernorm_backward sums launch");
}

}  // extern "C"
