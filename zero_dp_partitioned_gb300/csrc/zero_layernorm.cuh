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

}  // namespace zdp
