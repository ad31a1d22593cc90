// zero_layernorm.cu -- the layer norm behind a residual's dropout, forward.
//
//   h = round(dropout(x) + r)      (r and h in x's type, or both in fp32)
//   y = (h - m) rstd w + b,  m = mean(h),  rstd = 1 / sqrt(mean((h - m)^2) + eps)
//
// Bound: HBM (x and r read, h and y written: 8 bytes an element in 16 bits).  A
// row is read once and kept in registers between the statistics and the output;
// how rows are shared out stands in zero_layernorm.cuh.
//
// Measured (GB300; in brackets the share of the measured copy bandwidth): 16384 x
// 3456 bf16 in 81 us (0.83), with dropout 84; fp16 onto an fp32 stream 120
// (0.83); 8192 x 4096 fp32 94 (0.85); 8192 x 1600 bf16 19.8 (0.78: 3 rows a
// group), with dropout 26.0 (the generator's products beside those of the norm);
// 4096 x 12288 bf16 67 (0.89).  Rows that start anywhere: 8192 x 4097 bf16 94
// (0.42), fp32 134 (0.59).  Rows past 16384 columns (with a weight or bias of
// another type 13312; onto an fp32 stream 13312 and 10616; fp32 9104) are walked
// three times: 2048 x 20480 bf16 in 84 (0.59).
//
// The mean and the squares about it come with one barrier: a warp takes the
// mean of its own columns, then the squares about that mean from its registers,
// and the warps' (count, mean, squares) are joined by
//   M2 = sum M2_w + sum n_w (m_w - m)^2
// (T. Chan, G. Golub, R. LeVeque, Algorithms for computing the sample
// variance, 1983), so that a row far off zero loses nothing to cancellation.
#include "zero_layernorm.cuh"

namespace zdp {

// What a block keeps of its warps: the columns of each, and, in two sets used by
// turns, mean and squares.
struct WarpStats {
    float n[32];
    float2 s[2][32];
};

// WT: the type in which weight and bias lie in shared memory.
template <int XT, int RT, int WT, int NV, bool SHIFT>
__global__ void __launch_bounds__(LN_THREADS, 1) k_layernorm_forward_rows(const __grid_constant__ LayerNormArgs a) {
    __shared__ __align__(16) WarpStats st;
    using X = Lane<XT, NV, SHIFT>;
    using R = Lane<RT, NV, SHIFT>;
    using V = Vector<WT>;
    constexpr int XS = 8 * Elem<XT>::SIZE, RS = 8 * Elem<RT>::SIZE;          // bytes of a unit
    const int T = a.T, G = blockDim.x / T, group = threadIdx.x / T, units = a.units;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T >> 5, w0 = group * warps;
    const int uw = (warp - w0) * NV * 32, left = units - uw;                 // the warp's first unit, units from there
    const int n = SHIFT ? (left + 31) >> 5 : (left - lane + 31) >> 5;        // the warp's js, or this lane's (any number above NV: all)
    const int wcols = a.cols - uw * 8, lcols = wcols - lane * 8;             // columns from the warp's first on, from this lane's
    const int mine = max(0, min(NV * 256, wcols));                           // columns of this warp
    const float inv_mine = mine ? 1.f / (float)mine : 0.f, inv_n = 1.f / (float)a.cols;
    if (lane == 0) st.n[warp] = (float)mine;
    pdl_wait();
    pdl_launch_next();
    const uint32_t step = drop_step(a.drop);
    extern __shared__ __align__(16) uint4 ring[];
    const int S = a.stages, xwords = (blockDim.x >> 5) * X::WORDS, stage_words = xwords + (blockDim.x >> 5) * R::WORDS;
    const int64_t first = group * (int64_t)gridDim.x + blockIdx.x, every = (int64_t)G * gridDim.x;
    uint4 *const xat = ring + warp * X::WORDS, *const rat = ring + xwords + warp * R::WORDS;
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols);
    // this warp's part of the row whose copy comes next, and of the row at hand
    const char *cx = static_cast<const char*>(a.x) + first * a.ldx * Elem<XT>::SIZE + (int64_t)uw * XS;
    const char* cr = static_cast<const char*>(a.r) + (a.r ? first * a.ldr * Elem<RT>::SIZE + (int64_t)uw * RS : 0);
    char* H = static_cast<char*>(a.h) + (a.h ? first * a.ldh * Elem<RT>::SIZE + (int64_t)uw * RS : 0);
    char* Y = static_cast<char*>(a.y) + first * a.ldy * Elem<XT>::SIZE + (int64_t)uw * XS;
    const int64_t dx = every * a.ldx * Elem<XT>::SIZE, dr = every * a.ldr * Elem<RT>::SIZE, dh = every * a.ldh * Elem<RT>::SIZE,
                  dy = every * a.ldy * Elem<XT>::SIZE;
    int64_t crow = first, unit = first * units + uw + lane;
    auto copy = [&](int at_stage) {
        if (crow < a.rows) {
            X::copy(xat + at_stage * stage_words, cx, wcols, ex);
            if (a.r) R::copy(rat + at_stage * stage_words, cr, wcols, er);
        }
        copies_commit();
        crow += every;
        cx += dx;
        cr += dr;
    };
    for (int s = 0; s < S - 1; ++s) copy(s);
    uint4* const wat = ring + S * stage_words;
    uint4* const bat = wat + V::W * units;
    V::fill(wat, a.w, a.wdt, a.w_aligned, a.cols, units, 1.f);
    V::fill(bat, a.b, a.bdt, a.b_aligned, a.cols, units, 0.f);
    __syncthreads();
    int turn = 0, at_stage = 0;
    for (int64_t row = first; row < a.rows; row += every, turn ^= 1, unit += every * units, H += dh, Y += dy) {
        Raw8<RT> r[NV];
        copy(at_stage == 0 ? S - 1 : at_stage - 1);
        copies_wait_all_but(S - 1);
        if (X::SHARED || R::SHARED) __syncwarp();
        const int xoff = X::off(cx - S * dx), roff = R::off(cr - S * dr);
        uint4 *const xs = xat + at_stage * stage_words, *const rs = rat + at_stage * stage_words;
        at_stage = at_stage == S - 1 ? 0 : at_stage + 1;
        // h as it is stored
        Put<RT, NV, SHIFT> puth;
        uint64_t s2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j < n) {
                Unit<XT, true> xu;
                Unit<RT, true> ru;
                xu.raw = X::read(xs, j, xoff, lcols - 256 * j);
                if (a.r) ru.raw = R::read(rs, j, roff, lcols - 256 * j);
                r[j] = (a.drop.on ? drop_add_unit<XT, RT, true>(xu, ru, a.r != nullptr, a.drop, step, unit + 32 * j)
                                  : add_unit<XT, RT, true>(xu, ru, a.r != nullptr))
                           .raw;
#pragma unroll
                for (int q = 0; q < 4; ++q) s2 = add2(s2, pair8<RT>(r[j], q));
                if (!SHIFT && a.h) puth.put(H, rs, j, lcols - 256 * j, a.h32, r[j]);
            }
        if (SHIFT && a.h) {
            __syncwarp();                                    // all lanes have read the residual's units
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j < n) puth.put(H, rs, j, lcols - 256 * j, false, r[j]);
            puth.end(H, rs, wcols);
        }
        const float2 sp = unpack2(s2);
        const float mw = warp_sum(sp.x + sp.y) * inv_mine;
        const uint64_t mw2 = pack2(-mw, -mw);
        uint64_t v2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j < n) {
                const int here = lcols - 256 * j;
                if (!SHIFT || here >= 8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint64_t d = add2(pair8<RT>(r[j], q), mw2);
                        v2 = fma2(d, d, v2);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 p = unpack2(add2(pair8<RT>(r[j], q), mw2));
                        const uint64_t d = pack2(2 * q < here ? p.x : 0.f, 2 * q + 1 < here ? p.y : 0.f);
                        v2 = fma2(d, d, v2);
                    }
                }
            }
        const float2 vp = unpack2(v2);
        float m2 = warp_sum(vp.x + vp.y), mean = mw;
        if (warps > 1) {
            if (lane == 0) st.s[turn][warp] = make_float2(mw, m2);
            row_barrier(group, T);
            float sum = 0.f;
#pragma unroll 4
            for (int k = 0; k < warps; ++k) sum = fmaf(st.n[w0 + k], st.s[turn][w0 + k].x, sum);
            mean = sum * inv_n;
            m2 = 0.f;
#pragma unroll 4
            for (int k = 0; k < warps; ++k) {
                const float2 p = st.s[turn][w0 + k];
                const float d = p.x - mean;
                m2 += fmaf(st.n[w0 + k] * d, d, p.y);
            }
        }
        const float rstd = rsqrtf(fmaf(m2, inv_n, a.eps));
        if (warp == w0 && lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const uint64_t mm = pack2(-mean, -mean), rr = pack2(rstd, rstd);
        Put<XT, NV, SHIFT> puty;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j < n) {
                const int u = SHIFT ? min(uw + lane + 32 * j, units - 1) : uw + lane + 32 * j;
                const Raw8<WT> w = V::read(wat, u, units), b = V::read(bat, u, units);
                float y[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 v = unpack2(fma2(mul2(add2(pair8<RT>(r[j], q), mm), rr), pair8<WT>(w, q), pair8<WT>(b, q)));
                    y[2 * q] = v.x;
                    y[2 * q + 1] = v.y;
                }
                puty.put(Y, xs, j, lcols - 256 * j, a.y32, narrow8<XT>(y));
            }
        puty.end(Y, xs, wcols);
        if (SHIFT) __syncwarp();                             // the next copies land in these words
    }
}

// A row too long for the registers: the block walks it for the sum (storing h,
// if it is wanted), for the squares and for the output, after the first time
// from L2.
template <int XT, int RT, bool V8>
__global__ void __launch_bounds__(NORM_THREADS) k_layernorm_forward_long(const __grid_constant__ LayerNormArgs a) {
    constexpr int E = Map::E;
    __shared__ __align__(16) float ssum[2][32];
    if (threadIdx.x < 64) ssum[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
    __syncthreads();
    pdl_wait();
    pdl_launch_next();
    const uint32_t step = drop_step(a.drop);
    const float inv_n = 1.f / (float)a.cols;
    const Extent ex = extent_of<XT>(a.x, a.ldx, a.rows, a.cols), er = extent_of<RT>(a.r, a.ldr, a.rows, a.cols),
                 eh = extent_of<RT>(a.h, a.ldh, a.rows, a.cols);
    const int steps = (a.units + (int)blockDim.x - 1) / (int)blockDim.x;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const void* X = row_of<XT>(a.x, a.ldx, row);
        const void* R = a.r ? row_of<RT>(a.r, a.ldr, row) : nullptr;
        void* H = a.h ? row_of<RT>(a.h, a.ldh, row) : nullptr;
        auto first = [&](int u) {
            Unit<XT, V8> x;
            Unit<RT, V8> r;
            x.load(X, u, a.cols, ex);
            if (R) r.load(R, u, a.cols, er);
            return a.drop.on ? drop_add_unit<XT, RT, V8>(x, r, R != nullptr, a.drop, step, row * a.units + u)
                             : add_unit<XT, RT, V8>(x, r, R != nullptr);
        };
        auto again = [&](int u, float (&h)[E]) {      // after h was stored, over x or r perhaps
            if (H) {
                Unit<RT, V8> s;
                s.load(H, u, a.cols, eh);
                s.values(h);
            } else {
                first(u).values(h);
            }
        };
        float sum = 0.f;
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            const Unit<RT, V8> s = first(u);
            float h[E];
            s.values(h);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (u * 8 + e < a.cols) sum += h[e];
            if (H) s.store(H, u, a.cols);
        }
        const float mean = block_sum(sum, ssum[0]) * inv_n;
        float m2 = 0.f;
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            float h[E];
            again(u, h);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (u * 8 + e < a.cols) m2 = fmaf(h[e] - mean, h[e] - mean, m2);
        }
        const float rstd = rsqrtf(fmaf(block_sum(m2, ssum[1]), inv_n, a.eps));
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int j = 0; j < steps; ++j) {
            const int u = threadIdx.x + j * blockDim.x;
            float h[E], w[E], b[E];
            again(u, h);
            vector8(a.w, a.wdt, a.w_aligned, a.cols, u, 1.f, w);
            vector8(a.b, a.bdt, a.b_aligned, a.cols, u, 0.f, b);
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = fmaf((h[e] - mean) * rstd, w[e], b[e]);
            store_unit<XT, V8>(row_of<XT>(a.y, a.ldy, row), u, a.cols, h);
        }
    }
}

// packed: weight and bias in shared memory in x's type, not in fp32.
template <int XT, int RT, bool SHIFT>
static const void* rows_of(bool packed, int nv) {
    if (nv == 2) return (const void*)k_layernorm_forward_rows<XT, RT, ZERO_F32, 2, SHIFT>;
    return packed ? (const void*)k_layernorm_forward_rows<XT, RT, XT, 4, SHIFT> : (const void*)k_layernorm_forward_rows<XT, RT, ZERO_F32, 4, SHIFT>;
}
template <int XT, int RT>
static const void* fn_of(bool v8, bool packed, int nv) {
    if (nv) return v8 ? rows_of<XT, RT, false>(packed, nv) : rows_of<XT, RT, true>(packed, nv);
    return v8 ? (const void*)k_layernorm_forward_long<XT, RT, true> : (const void*)k_layernorm_forward_long<XT, RT, false>;
}
// nv 0: rows too long for the registers.
static const void* forward_fn(int xt, int rt, bool v8, bool packed, int nv) {
    if (xt == ZERO_F32) return fn_of<ZERO_F32, ZERO_F32>(v8, packed, nv);
    if (xt == ZERO_BF16) return rt == ZERO_F32 ? fn_of<ZERO_BF16, ZERO_F32>(v8, packed, nv) : fn_of<ZERO_BF16, ZERO_BF16>(v8, packed, nv);
    return rt == ZERO_F32 ? fn_of<ZERO_F16, ZERO_F32>(v8, packed, nv) : fn_of<ZERO_F16, ZERO_F16>(v8, packed, nv);
}

}  // namespace zdp

using namespace zdp;

extern "C" int zero_layernorm_forward(const zero_mat* x, const zero_mat* residual, const zero_drop* drop,
                                      const zero_mat* weight, const zero_mat* bias, int64_t rows, int64_t cols, float eps,
                                      const zero_mat* h_out, const zero_mat* y, float* mean, float* rstd, void* stream) {
    const char* me = "zero_layernorm_forward";
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "zero_layernorm_forward: negative rows or cols");
    if (cols > NORM_MAX_COLS) return fail(ZERO_ELIMIT, "zero_layernorm_forward: more than 1048576 columns");
    if (!(eps >= 0.f) || !(eps < INFINITY)) return fail(ZERO_EINVAL, "zero_layernorm_forward: eps must be finite and >= 0");
    int rc = check_mat(x, rows, cols, FLOAT_TYPES, me, "x");
    if (rc == ZERO_OK) rc = check_mat(y, rows, cols, FLOAT_TYPES, me, "y");
    if (rc == ZERO_OK && residual) rc = check_mat(residual, rows, cols, FLOAT_TYPES, me, "residual");
    if (rc == ZERO_OK && h_out) rc = check_mat(h_out, rows, cols, FLOAT_TYPES, me, "h_out");
    if (rc == ZERO_OK && weight) rc = check_mat(weight, 1, cols, FLOAT_TYPES, me, "weight");
    if (rc == ZERO_OK && bias) rc = check_mat(bias, 1, cols, FLOAT_TYPES, me, "bias");
    if (rc != ZERO_OK) return rc;
    const int rt = residual ? residual->dtype : x->dtype;
    if (rt != x->dtype && rt != ZERO_F32)
        return fail(ZERO_EINVAL, "zero_layernorm_forward: the residual is in x's type or fp32");
    if (h_out && h_out->dtype != rt)
        return fail(ZERO_EINVAL, "zero_layernorm_forward: h_out is in the residual's type (x's without one)");
    if (y->dtype != x->dtype) return fail(ZERO_EINVAL, "zero_layernorm_forward: y is in x's type");
    if (!aligned(mean, 4) || !aligned(rstd, 4))
        return fail(ZERO_EALIGN, "zero_layernorm_forward: mean or rstd not 4-byte aligned");
    LayerNormArgs a = {};
    rc = check_drop(drop, a.drop, me);
    if (rc != ZERO_OK || rows == 0 || cols == 0) return rc;
    a.x = x->data;
    a.ldx = x->ld;
    a.r = residual ? residual->data : nullptr;
    a.ldr = residual ? residual->ld : 0;
    a.h = h_out ? h_out->data : nullptr;
    a.ldh = h_out ? h_out->ld : 0;
    a.y = y->data;
    a.ldy = y->ld;
    if (weight) {
        a.w = weight->data;
        a.wdt = weight->dtype;
        a.w_aligned = aligned(weight->data, 16);
    }
    if (bias) {
        a.b = bias->data;
        a.bdt = bias->dtype;
        a.b_aligned = aligned(bias->data, 16);
    }
    a.rows = rows;
    a.cols = (int)cols;
    a.units = (int)((cols + 7) / 8);
    a.eps = eps;
    a.mean = mean;
    a.rstd = rstd;
    const bool v8 = cols % 8 == 0 && rows_aligned(*x, rows) && rows_aligned(*y, rows) &&
                    (!residual || rows_aligned(*residual, rows)) && (!h_out || rows_aligned(*h_out, rows));
    const int sms = sm_count(), words = words_of(x->dtype) + words_of(rt);
    if (!sms) return ZERO_ECUDA;
    void* args[] = {&a};
    const bool w16 = x->dtype != ZERO_F32 && (!weight || weight->dtype == x->dtype) && (!bias || bias->dtype == x->dtype);
    int nv;
    RowsShape p = rows_shape(rows, cols, words, 4, sms, &nv);
    const bool packed = !p.threads && w16;
    if (packed) p = rows_shape(rows, cols, nv = 4, words, 2, sms);
    if (p.threads) {
        a.stages = p.stages;
        a.T = p.T;
        a.h32 = h_out && rows_on_32(*h_out, rows);
        a.y32 = rows_on_32(*y, rows);
    } else {
        nv = 0;
        const int64_t most = (int64_t)sms * 6;
        p = RowsShape{NORM_THREADS, 0, 0, (int)(rows < most ? rows : most), 0};
    }
    const void* f = forward_fn(x->dtype, rt, v8, packed, nv);
    rc = raise_smem(f, p.smem, "zero_layernorm_forward shared-memory size");
    if (rc != ZERO_OK) return rc;
    return cuda_fail(launch_after_previous(f, p.grid, p.threads, args, p.smem, static_cast<cudaStream_t>(stream)),
                     "zero_layernorm_forward launch");
}
