// zero_drop.cuh -- the dropout mask that is never stored: which elements are
// kept follows from the seed, the place in the model, the step and the
// element's place in its matrix, so that the backward pass finds it again.
//
// The generator is Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// Parallel random numbers: as easy as 1, 2, 3, SC 2011): ten rounds of two
// 32 x 32 -> 64 bit products on a counter of four words, here (unit's low
// word, unit's high word, site, step), with the seed's two words as the key.
// A unit is 8 consecutive columns of a row, and each takes 16 of the 128 bits,
// so that one counter serves a 16-byte vector of 16-bit elements: ten rounds an
// element or four elements would cost more than the memory traffic (about 60
// instructions a counter; a 16-bit element that is read and written once has
// time for 22).  16 bits give the probability in steps of 2^-16; the kept
// elements are scaled by the inverse of the probability as it is then, so that
// the mean is kept exactly.
#pragma once

#include "zero_layer.cuh"

namespace zdp {

struct DropArgs {
    uint32_t k0, k1, site, step;
    uint32_t above;                 // a half is kept if it, shifted to the word's top, is above this
    float scale;                    // of what is kept
    float one;                      // 1, as a value that the compiler does not know
    int on;
    const zero_chain* chain;
};

// The step that the mask belongs to, read once a thread.
__device__ __forceinline__ uint32_t drop_step(const DropArgs& d) {
    return d.on && d.chain ? (uint32_t)(*reinterpret_cast<const volatile int64_t*>(&d.chain->step)) : d.step;
}

__device__ __forceinline__ uint4 philox4x32(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)0xD2511F53u * c.x, q = (uint64_t)0xCD9E8D57u * c.z;
        c = make_uint4((uint32_t)(q >> 32) ^ c.y ^ k0, (uint32_t)q, (uint32_t)(p >> 32) ^ c.w ^ k1, (uint32_t)p);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}
__device__ __forceinline__ uint4 drop_bits(const DropArgs& d, uint32_t step, int64_t unit) {
    return philox4x32(make_uint4((uint32_t)unit, (uint32_t)((uint64_t)unit >> 32), d.site, step), d.k0, d.k1);
}
// Whether elements 2 q and 2 q + 1 of the unit are kept: the low and the high half of word q.
__device__ __forceinline__ bool kept_low(uint32_t word, uint32_t above) { return word << 16 > above; }
__device__ __forceinline__ bool kept_high(uint32_t word, uint32_t above) { return word > above; }
__device__ __forceinline__ uint32_t word_of(const uint4& w, int q) { return q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w; }

// elements 2 q and 2 q + 1: what is kept, 0 in the others' place (whatever stood there)
__device__ __forceinline__ uint64_t drop2(uint64_t v, const uint4& bits, int q, uint32_t above) {
    const float2 p = unpack2(v);
    const uint32_t w = word_of(bits, q);
    return pack2(kept_low(w, above) ? p.x : 0.f, kept_high(w, above) ? p.y : 0.f);
}

// v scale + r of two elements, the product and the sum each rounded to fp32, as in
// any form that takes them one after the other.  A packed product whose sum is
// packed too comes out as one fma here, .rn and all, with the product unrounded (a
// quarter dropped: 4/3 x, once rounded, often puts the sum on half a step of bf16,
// and unrounded it passed it, always the same way); a product and an fma do not.
// 32768 x 4096 bf16 onto a residual in 125 us, 122 with the one fma.
__device__ __forceinline__ uint64_t scaled_onto2(uint64_t v, const DropArgs& d, uint64_t r) {
    return fma2(mul2(v, pack2(d.scale, d.scale)), pack2(d.one, d.one), r);
}

// ---------------------------------------------------------------- host
// The kernels' form of a zero_drop (NULL, or a probability that rounds to 0: no dropout).
int check_drop(const zero_drop* d, DropArgs& a, const char* call);

}  // namespace zdp
