// zero_distill.cu -- the distillation loss of a student's logits z against a
// teacher's k largest logits t, and its gradient.
//
//   q = softmax(z / T) over the vocabulary;  p = softmax(t / T) over the row's
//   k entries, or exp(t / T - lse_t) with the teacher's own log-sum-exp;  P = sum p
//   loss = w T^2 sum_i p_i (log p_i - log q_i)
//   dz_v = w S c T (P q_v - sum of p_i with id_i = v)
//
// Bound: HBM, 4 bytes a logit in 16 bits (read once, gradient written once).
// A block walks its row twice: once for the maximum and the sum together
// (batches of 8 vectors a thread, the sum brought to a new maximum when there
// is one), once for the gradient.  The second walk finds 8 vectors a thread in
// shared memory and the rest in L2.  Few rows are split over a cluster of up to
// 8 blocks, whose pairs of maximum and sum cross through distributed shared
// memory.
//
// Measured (GB300): 4096 x 128256 bf16 in 358 us, 5.9 TB/s (0.86 of the
// measured copy bandwidth); 1999 x 50257 fp32 in 150 us, 5.4 TB/s (0.79).  The
// loss alone takes 181 and 81 us (0.86 and 0.73), the gradient from a stored
// log-sum-exp 357 and 128 (0.87 and 0.92).  Rows of few vectors are further
// off: 8192 x 16000 bf16 205 us (0.38), 8192 x 8000 fp32 196 (0.39) -- below
// 4096 vectors a thread of 512 has fewer than a batch, and walks them one load
// at a time.
// Without the vectors in shared memory 385 us (a fifth of the second walk
// missed L2); with 12 of them 431 (too little L1 left for the loads in flight);
// with every row in the registers of a cluster of 8 blocks 580 (the work that
// is done once a block came 8 times, and blocks waited for one another); with
// blocks that stay and fetch the next row's vectors into shared memory as they
// write the gradient 400 to 455.
//
// Exponentials are taken in base 2 with one fused multiply-add, 2^(z k - m k)
// with k = log2(e) / T; m k is rounded once and used for the sum, the
// log-sum-exp and the gradient alike, so its rounding cancels.
#include "zero_layer.cuh"

namespace zdp {

constexpr int DISTILL_THREADS = 512;
constexpr int DISTILL_BLOCKS = 2;        // resident blocks of a multiprocessor
constexpr int DISTILL_BATCH = 8;         // vectors a thread has in flight
constexpr int DISTILL_KEEP = 8;          // most vectors a thread keeps in shared memory (a multiple of the batch)
constexpr int DISTILL_CLUSTER = 8;       // most blocks that share a row (the portable cluster size)
constexpr int DISTILL_MAX_K = 1024;
constexpr float DISTILL_EXTREME = 1073741824.f;   // 2^30, of a row's largest z k

struct DistillArgs {
    const void *z, *t, *ids;
    void* dz;
    const float *t_lse, *w, *lse_in;
    float *loss, *lse;
    const zero_chain* chain;
    int64_t ldz, lddz, ldt, ldi, rows, cols;
    int k, t_dt, id64, split, keep;
    float k2, temperature, grad_scale;   // k2 = log2(e) / T
};

// One entry of the row's teacher list, in shared memory: the column (-1: no
// entry), the teacher's logit, the student's logit, and p before it is divided.
struct Entry {
    int id;
    float t, z, p;
};

// Relative error at most 2^-22 by the instruction's specification, and 0 for a
// result below 2^-126, which is nothing beside the row's largest term.  With it
// the outputs of 1999 x 50257 fp32 logits are 9e-8 from 64 bits, as an
// elementwise fp32 form's are.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t exp2_2(uint64_t v) {
    const float2 x = unpack2(v);
    return pack2(exp2_fast(x.x), exp2_fast(x.y));
}

// A row between 16-byte boundaries: `n` whole aligned vectors of W elements
// from element `head`, and fewer than W elements at either end (the edges).
template <int DT>
struct RowVec {
    static constexpr int W = 16 / Elem<DT>::SIZE, PAIRS = W / 2;
    const char *base, *vec;   // element 0, vector 0
    int head, n, cols;
    __device__ __forceinline__ RowVec(const void* p, int cols_) : base(static_cast<const char*>(p)), cols(cols_) {
        const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u) / Elem<DT>::SIZE;
        head = min(off ? W - off : 0, cols);
        n = (cols - head) / W;
        vec = base + (int64_t)head * Elem<DT>::SIZE;
    }
    // the e-th edge element's column, -1 past the last; there are at most 2 (W - 1) <= 14
    __device__ __forceinline__ int edge(int e) const {
        const int c = e < head ? e : e + n * W;
        return c < cols ? c : -1;
    }
    // which of the row's vectors holds column c (-1: an edge)
    __device__ __forceinline__ int vector_of(int c) const {
        const int v = c < head ? -1 : (c - head) / W;
        return v < n ? v : -1;
    }
    // plain loads (the gradient may be in the logits' place): the first walk's lines should stay for the second
    __device__ __forceinline__ uint4 load(int i) const { return reinterpret_cast<const uint4*>(vec)[i]; }
    __device__ __forceinline__ uint4 load_last(int i) const { return __ldcs(reinterpret_cast<const uint4*>(vec) + i); }
    // elements 2 q and 2 q + 1
    static __device__ __forceinline__ uint64_t pair(const uint4& r, int q) {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
        if constexpr (DT == ZERO_F32) return pack2(__uint_as_float(u[2 * q]), __uint_as_float(u[2 * q + 1]));
        else if constexpr (DT == ZERO_BF16) return pack2(__uint_as_float(u[q] << 16), __uint_as_float(u[q] & 0xFFFF0000u));
        else return pack2(Half16<DT>::widen(u[q] & 0xFFFFu), Half16<DT>::widen(u[q] >> 16));
    }
    static __device__ __forceinline__ float top(const uint4& r) {
        if constexpr (DT == ZERO_F32) {
            return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
        } else if constexpr (DT == ZERO_BF16) {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
            const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            const __half2* h = reinterpret_cast<const __half2*>(&r);
            const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__low2float(m), __high2float(m));
        }
    }
    // sum of 2^(z k - m k) of a vector's pairs, added to s
    static __device__ __forceinline__ uint64_t sum(const uint4& r, uint64_t k, uint64_t neg_mk, uint64_t s) {
#pragma unroll
        for (int q = 0; q < PAIRS; ++q) s = add2(s, exp2_2(fma2(pair(r, q), k, neg_mk)));
        return s;
    }
    // g 2^(z k - m k) of a vector, rounded and stored
    static __device__ __forceinline__ void grad(char* dst, bool aligned16, const uint4& r, uint64_t k, uint64_t neg_mk,
                                                uint64_t g) {
        float2 v[PAIRS];
#pragma unroll
        for (int q = 0; q < PAIRS; ++q) v[q] = unpack2(mul2(exp2_2(fma2(pair(r, q), k, neg_mk)), g));
        put(dst, aligned16, v);
    }
    static __device__ __forceinline__ void put(char* dst, bool aligned16, const float2 (&v)[PAIRS]) {
        uint32_t u[4];
#pragma unroll
        for (int q = 0; q < PAIRS; ++q) {
            if constexpr (DT == ZERO_F32) {
                u[2 * q] = __float_as_uint(v[q].x);
                u[2 * q + 1] = __float_as_uint(v[q].y);
            } else {
                u[q] = Half16<DT>::narrow2(v[q].x, v[q].y);
            }
        }
        if (aligned16) {
            __stcs(reinterpret_cast<uint4*>(dst), make_uint4(u[0], u[1], u[2], u[3]));
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                if constexpr (DT == ZERO_F32) reinterpret_cast<uint32_t*>(dst)[e] = u[e];
                else reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
            }
        }
    }
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Store a pair at the same shared-memory address of block `rank` of the cluster.
__device__ __forceinline__ void store_remote(float2* local, int rank, float2 v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(v.x), "f"(v.y) : "memory");
}

// A maximum and the sum of 2^(x - it) of several parts, one a lane and step,
// to those of the whole.  A NaN is kept in the sums (a maximum drops it).
__device__ __forceinline__ float2 merge(const float2* part, int n) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, part[i].x);
    m = warp_max(m);
    float s = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float2 p = part[i];
        s += p.y * exp2f(p.x - m);
    }
    return make_float2(m, warp_sum(s));
}

// A row whose largest |z k| is DISTILL_EXTREME or more (masked with the type's
// lowest value, say): fp32 does not hold its exponents, but different logits are
// then at least 2^6 apart, so that a term is 1 where the logit is the largest
// and below 2^-64 elsewhere.  The row's largest logit (a NaN is kept) and how
// often it comes; the whole block calls it and walks the whole row, off the path
// of every other row.
template <int DT>
__device__ __noinline__ float2 extreme_row(const void* row, int cols) {
    __shared__ float part[DISTILL_THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float m = -INFINITY;
    for (int c = threadIdx.x; c < cols; c += blockDim.x) m = max3_nan(m, m, ld1<DT>(row, c));
    for (int o = 16; o > 0; o >>= 1) {
        const float v = __shfl_xor_sync(0xFFFFFFFFu, m, o);
        m = max3_nan(m, m, v);
    }
    if (lane == 0) part[warp] = m;
    __syncthreads();
    for (int w = 0; w < nw; ++w) m = max3_nan(m, m, part[w]);
    float n = 0.f;
    for (int c = threadIdx.x; c < cols; c += blockDim.x) n += ld1<DT>(row, c) == m ? 1.f : 0.f;
    n = warp_sum(n);
    __syncthreads();
    if (lane == 0) part[warp] = n;
    __syncthreads();
    n = 0.f;
    for (int w = 0; w < nw; ++w) n += part[w];
    return make_float2(m, n);
}
// A power of two that brings such a logit to 2^125, so that its product is exact.
__device__ __forceinline__ float extreme_scale(float top) {
    return __uint_as_float(min(254u, 379u - (__float_as_uint(top) >> 23 & 255u)) << 23);
}

// The teacher's parts, one a lane -- a largest logit and the sum of 2^((t - it) k)
// -- to those of the row; plain sums where the base is given (no softmax of its own).
__device__ __forceinline__ float2 merge_teacher(const float2* part, int n, float k2, bool own) {
    const int lane = threadIdx.x & 31;
    const float2 p = lane < n ? part[lane] : make_float2(-INFINITY, 0.f);
    const float top = warp_max(p.x);
    return make_float2(top, warp_sum(own && p.x != top ? p.y * exp2f((p.x - top) * k2) : p.y));
}

// BWD: the row's log-sum-exp is given (lse_in), so that only the gradient is
// walked and nothing crosses the cluster.
//
// Every warp reduces its own part to a maximum and a sum and sends the pair to
// all blocks of the cluster: one barrier, and each warp merges all pairs.
template <int DT, bool BWD>
__global__ void __launch_bounds__(DISTILL_THREADS, DISTILL_BLOCKS) k_distill(const __grid_constant__ DistillArgs a) {
    using R = RowVec<DT>;
    constexpr int MAX_WARPS = DISTILL_THREADS / 32, U = DISTILL_BATCH;
    extern __shared__ __align__(16) uint8_t dyn[];
    uint4* kept = reinterpret_cast<uint4*>(dyn);            // [keep][T]
    __shared__ float2 zpart[DISTILL_CLUSTER * MAX_WARPS], tpart[MAX_WARPS];
    pdl_wait();
    pdl_launch_next();
    Entry* entry = reinterpret_cast<Entry*>(dyn + (size_t)a.keep * blockDim.x * 16);
    const int C = a.split, T = blockDim.x, rank = C == 1 ? 0 : (int)(blockIdx.x % (unsigned)C);
    const int64_t row = C == 1 ? blockIdx.x : blockIdx.x / (unsigned)C;
    if (!BWD && C > 1) cluster_arrive();          // this block runs: its shared memory may be written
    const R rv(static_cast<const char*>(a.z) + row * a.ldz * Elem<DT>::SIZE, (int)a.cols);
    const int step = C * T, first = rank * T + threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // whether column c is written by this block (the edges are the first block's)
    auto mine = [&](int c) {
        if (C == 1) return true;
        const int v = rv.vector_of(c);
        return (v < 0 ? 0 : v / T % C) == rank;
    };

    // the edges: one element in each of the first lanes of the row's first block
    const int edge = rank == 0 && threadIdx.x < 16 ? rv.edge(threadIdx.x) : -1;
    const float edge_z = edge >= 0 ? ld1<DT>(rv.base, edge) : -INFINITY;
    // the teacher's entries, and the student's logits at them (read before any
    // gradient is written, which may be in their place)
    float tmax = -INFINITY;
    for (int i = threadIdx.x; i < a.k; i += T) {
        const int64_t at = row * a.ldi + i;
        const int64_t id = a.id64 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
        const float t = ld1_any(a.t, row * a.ldt + i, a.t_dt);
        const bool have = id >= 0 && id < a.cols && t != -INFINITY;
        Entry en = {have ? (int)id : -1, t, 0.f, 0.f};
        // the backward pass alone has no barrier between its blocks: it reads what it itself will write
        if (have && (!BWD || mine(en.id))) en.z = ld1<DT>(rv.base, en.id);
        entry[i] = en;
        if (have) tmax = fmaxf(tmax, t != t ? 0.f : t);         // a NaN entry makes the sum NaN, not the row empty
    }
    const float k2 = a.k2;
    uint64_t kk = pack2(k2, k2);
    // log2 of the teacher's p: with its log-sum-exp, or (own) of the difference to the row's largest logit and not yet
    // divided by the sum, so that a common offset of the logits does not matter
    const bool own = !a.t_lse;
    const float tl = own ? 0.f : a.t_lse[row] * 1.4426950408889634f;
    auto log_term = [&](float t, float top) { return fmaf(t - top, k2, -tl); };      // top: 0 with a log-sum-exp
    // This thread's m k and sum.  m k is not below -DISTILL_EXTREME: far below, what it was rounded by would be an
    // exponent of its own (a thread with nothing but the type's lowest value), so such logits count for 0 against it.
    float m = -DISTILL_EXTREME, s = 0.f;
    if constexpr (!BWD) {
        uint64_t s2 = 0;
        auto take = [&](float t) {                // bring the sum to a larger maximum
            if (t > m) {
                const float f = exp2_fast(m - t);
                s2 = mul2(s2, pack2(f, f));
                m = t;
            }
        };
        int i = first, j = 0;
        for (; i + (U - 1) * step < rv.n; i += U * step, j += U) {
            uint4 r[U];
            if (j < a.keep) {
#pragma unroll
                for (int u = 0; u < U; ++u) r[u] = rv.load_last(i + u * step);
#pragma unroll
                for (int u = 0; u < U; ++u) kept[(j + u) * T + threadIdx.x] = r[u];
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) r[u] = rv.load(i + u * step);
            }
            float t = R::top(r[0]);
#pragma unroll
            for (int u = 1; u < U; ++u) t = fmaxf(t, R::top(r[u]));
            take(t * k2);
            const uint64_t nm = pack2(-m, -m);
#pragma unroll
            for (int u = 0; u < U; ++u) s2 = R::sum(r[u], kk, nm, s2);
        }
        for (; i < rv.n; i += step, ++j) {
            const uint4 r = rv.load(i);
            if (j < a.keep) kept[j * T + threadIdx.x] = r;
            take(R::top(r) * k2);
            s2 = R::sum(r, kk, pack2(-m, -m), s2);
        }
        if (edge >= 0) {
            take(edge_z * k2);
            s2 = add2(s2, pack2(exp2_fast(fmaf(edge_z, k2, -m)), 0.f));
        }
        const float2 p = unpack2(s2);
        s = p.x + p.y;
        const float wm = warp_max(m);
        s = warp_sum(s * exp2f(m - wm));
        m = wm;
    }
    {
        const float tm = warp_max(tmax);
        const float top = own ? tm : 0.f;
        float ts = 0.f;
        if (warp * 32 < a.k)
            for (int i = threadIdx.x; i < a.k; i += T)
                if (entry[i].id >= 0) ts += exp2f(log_term(entry[i].t, top));
        ts = warp_sum(ts);
        if (lane == 0) tpart[warp] = make_float2(tm, ts);
    }
    float mk, total;                              // m k and the sum over the whole row
    float kz = k2, ztop = 0.f;                    // an extreme row's k and largest logit
    if constexpr (BWD) {
        __syncthreads();
        mk = a.lse_in[row] * 1.4426950408889634f;
        total = 1.f;
    } else {
        const int nw = T >> 5;
        if (C == 1) {
            if (lane == 0) zpart[warp] = make_float2(m, s);
            __syncthreads();
        } else {
            cluster_wait();                        // every block of the cluster runs
            if (lane < C) store_remote(&zpart[rank * nw + warp], lane, make_float2(m, s));
            __syncwarp();
            cluster_arrive();
            cluster_wait();                        // every pair is here; no block leaves before its last arrives
        }
        const float2 whole = merge(zpart, C * nw);
        mk = whole.x;
        total = whole.y;
        if (fabsf(whole.x) >= DISTILL_EXTREME) {  // the same in every thread of the cluster
            const float2 e = extreme_row<DT>(rv.base, rv.cols);
            if (C > 1) {                          // no block writes a gradient where another still reads
                cluster_arrive();
                cluster_wait();
            }
            if (fabsf(e.x) < INFINITY) {          // infinities and NaN stay what they are
                kz = extreme_scale(e.x);
                kk = pack2(kz, kz);
                ztop = e.x;
                mk = ztop * kz;
                total = e.y;
            }
        }
    }
    const float2 tw = merge_teacher(tpart, T >> 5, k2, own);
    const bool none = tw.x == -INFINITY;          // no teacher entry in the row
    // p_i = 2^(log_term(t_i, tm)) pscale
    const float tm = own ? tw.x : 0.f, pscale = own ? 1.f / tw.y : 1.f, P = none ? 0.f : tw.y * pscale;
    const float w = a.w ? a.w[row] : 1.f;
    const bool dead = none || w == 0.f;
    if constexpr (!BWD) {
        const float lg = log2f(total), zk = ztop == 0.f ? mk : 0.f;       // log2 of q: (z - ztop) k2 - zk - lg
        if (a.lse && rank == 0 && threadIdx.x == 0) a.lse[row] = ztop / a.temperature + (zk + lg) * 0.6931471805599453f;
        if (a.loss && rank == 0 && warp == 0) {
            const float lt = own ? log2f(tw.y) : 0.f;
            float l = 0.f;
            if (!dead)
                for (int i = lane; i < a.k; i += 32) {
                    const Entry en = entry[i];
                    const float lp = log_term(en.t, tm), p = en.id >= 0 ? exp2f(lp) * pscale : 0.f;
                    if (p != 0.f) l += p * ((lp - lt) - (fmaf(en.z - ztop, k2, -zk) - lg));
                }
            l = warp_sum(l);
            if (lane == 0) a.loss[row] = dead ? 0.f : l * 0.6931471805599453f * a.temperature * a.temperature * w;
        }
    }
    if (!a.dz) return;
    float coef = w * a.temperature * a.grad_scale;
    if (a.chain) coef *= (float)a.chain->loss_scale;
    char* drow = static_cast<char*>(a.dz) + row * a.lddz * Elem<DT>::SIZE;
    char* dvec = drow + (int64_t)rv.head * Elem<DT>::SIZE;
    const bool al = (reinterpret_cast<uintptr_t>(dvec) & 15u) == 0;
    if (dead) {
        const float2 zero[R::PAIRS] = {};
        for (int i = first; i < rv.n; i += step) R::put(dvec + (int64_t)i * 16, al, zero);
        if (edge >= 0) st1<DT>(drow, edge, 0.f);
        return;
    }
    for (int j = threadIdx.x; j < a.k; j += T) entry[j].p = exp2f(log_term(entry[j].t, tm));     // read after a barrier
    const float g = coef * P / total;
    const uint64_t gg = pack2(g, g), nm = pack2(-mk, -mk);
    int i = first;
    if constexpr (!BWD)
        for (int j = 0; j < a.keep && i < rv.n; ++j, i += step)
            R::grad(dvec + (int64_t)i * 16, al, kept[j * T + threadIdx.x], kk, nm, gg);
    for (; i + (U - 1) * step < rv.n; i += U * step) {
        uint4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = rv.load_last(i + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u) R::grad(dvec + (int64_t)(i + u * step) * 16, al, r[u], kk, nm, gg);
    }
    for (; i < rv.n; i += step) R::grad(dvec + (int64_t)i * 16, al, rv.load_last(i), kk, nm, gg);
    if (edge >= 0) st1<DT>(drow, edge, g * exp2_fast(fmaf(edge_z, kz, -mk)));
    // the entries that lie in this block's part, written over after it wrote
    // that: the same id twice gives the same value twice
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += T) {
        const Entry en = entry[j];
        if (en.id < 0 || !mine(en.id)) continue;
        float p = 0.f;
        for (int o = 0; o < a.k; ++o)
            if (entry[o].id == en.id) p += entry[o].p;
        st1<DT>(drow, en.id, fmaf(g, exp2_fast(fmaf(en.z, kz, -mk)), -coef * p * pscale));
    }
}

// Rows of no columns: no entries, and a sum of nothing.
__global__ void __launch_bounds__(256) k_distill_empty(float* loss, float* lse, int64_t rows) {
    pdl_wait();
    pdl_launch_next();
    for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < rows; r += (int64_t)gridDim.x * blockDim.x) {
        if (loss) loss[r] = 0.f;
        if (lse) lse[r] = -INFINITY;
    }
}

template <int DT>
static const void* distill_fn(bool bwd) {
    return bwd ? (const void*)k_distill<DT, true> : (const void*)k_distill<DT, false>;
}

static int distill(const char* who, const zero_mat* logits, int64_t rows, int64_t cols, const zero_mat* ids,
                   const zero_mat* teacher, int k, const float* teacher_lse, float temperature, const float* row_weight,
                   float grad_scale, const zero_chain* chain, float* loss, float* lse, const float* lse_in,
                   const zero_mat* dlogits, bool bwd, void* stream) {
    auto bad = [&](int code, const char* what) {
        set_error(std::string(who) + ": " + what);
        return code;
    };
    if (rows < 0 || cols < 0 || k < 0) return bad(ZERO_EINVAL, "negative rows, cols or k");
    if (k > DISTILL_MAX_K) return bad(ZERO_ELIMIT, "more than 1024 teacher entries a row");
    if (cols > INT32_MAX / 2 || rows > INT32_MAX / DISTILL_CLUSTER) return bad(ZERO_ELIMIT, "too many rows or columns");
    if (!(temperature > 0.f) || !(temperature < INFINITY)) return bad(ZERO_EINVAL, "temperature must be finite and > 0");
    if (!(grad_scale - grad_scale == 0.f)) return bad(ZERO_EINVAL, "grad_scale must be finite");
    int rc = check_mat(logits, rows, cols, FLOAT_TYPES, who, "logits");
    if (rc == ZERO_OK) rc = check_mat(ids, rows, k, 1u << ZERO_I32 | 1u << ZERO_I64, who, "ids");
    if (rc == ZERO_OK) rc = check_mat(teacher, rows, k, FLOAT_TYPES, who, "teacher");
    if (rc == ZERO_OK && (dlogits || bwd)) rc = check_mat(dlogits, rows, cols, FLOAT_TYPES, who, "dlogits");
    if (rc != ZERO_OK) return rc;
    if (dlogits && dlogits->dtype != logits->dtype) return bad(ZERO_EINVAL, "dlogits is in the logits' type");
    if (bwd && rows > 0 && cols > 0 && !lse_in) return bad(ZERO_EINVAL, "NULL lse");
    if (!aligned(teacher_lse, 4) || !aligned(row_weight, 4) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(lse_in, 4))
        return bad(ZERO_EALIGN, "a row array is not 4-byte aligned");
    if (!aligned(chain, 8)) return bad(ZERO_EALIGN, "chain not 8-byte aligned");
    if (rows == 0 || (cols == 0 && !loss && !lse)) return ZERO_OK;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;
    if (cols == 0) {
        int64_t n = rows;
        void* args[] = {&loss, &lse, &n};
        return cuda_fail(launch_after_previous((const void*)k_distill_empty, (int)(rows < sms * 256 ? (rows + 255) / 256 : sms),
                                               256, args, 0, static_cast<cudaStream_t>(stream)),
                         who);
    }

    DistillArgs a = {};
    a.z = logits->data;
    a.ldz = logits->ld;
    a.dz = dlogits ? dlogits->data : nullptr;
    a.lddz = dlogits ? dlogits->ld : 0;
    a.t = teacher->data;
    a.ldt = teacher->ld;
    a.t_dt = teacher->dtype;
    a.ids = ids->data;
    a.ldi = ids->ld;
    a.id64 = ids->dtype == ZERO_I64;
    a.t_lse = teacher_lse;
    a.w = row_weight;
    a.lse_in = lse_in;
    a.loss = loss;
    a.lse = lse;
    a.chain = chain;
    a.rows = rows;
    a.cols = cols;
    a.k = k;
    a.k2 = (float)(1.4426950408889634 / (double)temperature);
    a.temperature = temperature;
    a.grad_scale = grad_scale;

    // Threads so that a short row leaves none idle; a block to a row, and a
    // cluster of more while all of them run at once.
    const int W = 16 / elem_size(logits->dtype);
    const int64_t n = cols / W + 1;          // whole vectors of a row, at most
    const int threads = n <= 1024 ? 128 : DISTILL_THREADS;
    int split = 1;
    while (split < DISTILL_CLUSTER && rows * split <= DISTILL_BLOCKS / 2 * (int64_t)sms && split * threads < n) split *= 2;
    a.split = split;
    // what a thread keeps: all its vectors if they are few, in whole batches
    const int64_t own = (n + (int64_t)split * threads - 1) / ((int64_t)split * threads);
    a.keep = bwd || !dlogits ? 0 : own >= DISTILL_KEEP ? DISTILL_KEEP : (int)((own + DISTILL_BATCH - 1) / DISTILL_BATCH * DISTILL_BATCH);

    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * split));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)a.keep * (size_t)threads * 16 + sizeof(Entry) * (size_t)k;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = bwd ? 1 : 2;
    const void* f = logits->dtype == ZERO_F32 ? distill_fn<ZERO_F32>(bwd)
                  : logits->dtype == ZERO_BF16 ? distill_fn<ZERO_BF16>(bwd) : distill_fn<ZERO_F16>(bwd);
    rc = raise_smem(f, cfg.dynamicSmemBytes, who);
    if (rc != ZERO_OK) return rc;
    void* args[] = {&a};
    return cuda_fail(cudaLaunchKernelExC(&cfg, f, args), who);
}

}  // namespace zdp

using namespace zdp;

extern "C" {

int zero_distill_loss(const zero_mat* logits, int64_t rows, int64_t cols, const zero_mat* ids, const zero_mat* teacher,
                      int k, const float* teacher_lse, float temperature, const float* row_weight, float grad_scale,
                      const zero_chain* chain, float* loss, float* lse, const zero_mat* dlogits, void* stream) {
    return distill("zero_distill_loss", logits, rows, cols, ids, teacher, k, teacher_lse, temperature, row_weight,
                   grad_scale, chain, loss, lse, nullptr, dlogits, false, stream);
}

int zero_distill_backward(const zero_mat* logits, int64_t rows, int64_t cols, const zero_mat* ids,
                          const zero_mat* teacher, int k, const float* teacher_lse, float temperature,
                          const float* row_weight, float grad_scale, const zero_chain* chain, const float* lse,
                          const zero_mat* dlogits, void* stream) {
    return distill("zero_distill_backward", logits, rows, cols, ids, teacher, k, teacher_lse, temperature, row_weight,
                   grad_scale, chain, nullptr, nullptr, lse, dlogits, true, stream);
}

}  // extern "C"
