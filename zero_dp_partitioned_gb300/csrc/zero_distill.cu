// zero_distill.cu -- the distillation loss of a student's logits z against a
// teacher's k largest logits t, and its gradient.
//
//   q = softmax(z / T) over the vocabulary;  p = softmax(t / T) over the row's
//   k entries, or exp(t / T - lse_t) with the teacher's own log-sum-exp;  P = sum p
//   loss = w T^2 sum_i p_i (log p_i - log q_i)
//   dz_v = w S c T (P q_v - sum of p_i with id_i = v)
//
// Bound: HBM, 4 bytes a logit in 16 bits (read once, gradient written once).
// A row is split over a cluster of up to 8 blocks so that each block's share
// stays in registers (8 16-byte vectors a thread) from the load to the
// gradient: the row's maximum and sum cross the cluster through distributed
// shared memory, and no logit is read twice.
//
// Exponentials are taken in base 2 with one fused multiply-add, 2^(z k - m k)
// with k = log2(e) / T; m k is rounded once and used for the sum, the
// log-sum-exp and the gradient alike, so its rounding cancels.
#include "zero_layer.cuh"

namespace zdp {

constexpr int DISTILL_THREADS = 512;
constexpr int DISTILL_VECS = 8;          // vectors a thread keeps
constexpr int DISTILL_CLUSTER = 8;       // most blocks that share a row (the portable cluster size)
constexpr int DISTILL_MAX_K = 1024;

struct DistillArgs {
    const void *z, *t, *ids;
    void* dz;
    const float *t_lse, *w, *lse_in;
    float *loss, *lse;
    const zero_chain* chain;
    int64_t ldz, lddz, ldt, ldi, rows, cols;
    int k, t_dt, id64, split;
    float k2, temperature, grad_scale;   // k2 = log2(e) / T
};

// One entry of the row's teacher list, in shared memory.
struct Entry {
    int id;          // -1: no entry
    float p, lp, z;  // p_i (before the division by the sum: e_i), log2 p_i, and the student's logit
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The row as 16-byte vectors: vector i holds elements i W - off .. + W - 1, so
// that every vector but the first and the last is whole and aligned wherever
// the row starts.
template <int DT>
struct RowVec {
    static constexpr int W = 16 / Elem<DT>::SIZE;
    static constexpr uint32_t NEG_INF = DT == ZERO_F32 ? 0xFF800000u : DT == ZERO_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
    const char* base;       // the row's first element
    int off;                // elements between the 16-byte boundary at or before it and it
    int64_t cols, n;
    __device__ __forceinline__ RowVec(const void* p, int64_t cols_)
        : base(static_cast<const char*>(p)), cols(cols_) {
        off = (int)(reinterpret_cast<uintptr_t>(p) & 15u) / Elem<DT>::SIZE;
        n = (cols + off + W - 1) / W;
    }
    __device__ __forceinline__ bool whole(int64_t i) const { return (i > 0 || off == 0) && (i + 1) * W - off <= cols; }
    __device__ __forceinline__ uint4 load(int64_t i) const {
        const int64_t c0 = i * W - off;
        if (whole(i)) return __ldcs(reinterpret_cast<const uint4*>(base + c0 * Elem<DT>::SIZE));
        uint32_t u[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const int64_t c = c0 + e;
            if (c < 0 || c >= cols) continue;
            if constexpr (DT == ZERO_F32) {
                u[e] = reinterpret_cast<const uint32_t*>(base)[c];
            } else {
                const uint32_t h = reinterpret_cast<const uint16_t*>(base)[c];
                u[e / 2] = e % 2 ? (u[e / 2] & 0xFFFFu) | h << 16 : (u[e / 2] & 0xFFFF0000u) | h;
            }
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void store(void* row, bool same_phase, int64_t i, const float (&v)[W]) const {
        const int64_t c0 = i * W - off;
        if (same_phase && whole(i)) {
            uint4 o;
            if constexpr (DT == ZERO_F32)
                o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                               __float_as_uint(v[3]));
            else
                o = make_uint4(Half16<DT>::narrow2(v[0], v[1]), Half16<DT>::narrow2(v[2], v[3]),
                               Half16<DT>::narrow2(v[4], v[5]), Half16<DT>::narrow2(v[6], v[7]));
            __stcs(reinterpret_cast<uint4*>(static_cast<char*>(row) + c0 * Elem<DT>::SIZE), o);
            return;
        }
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (c0 + e >= 0 && c0 + e < cols) st1<DT>(row, c0 + e, v[e]);
    }
};

template <int DT>
__device__ __forceinline__ void widen(const uint4& r, float (&v)[RowVec<DT>::W]) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (DT == ZERO_F32) {
            v[q] = __uint_as_float(u[q]);
        } else {
            v[2 * q] = Half16<DT>::widen(u[q] & 0xFFFFu);
            v[2 * q + 1] = Half16<DT>::widen(u[q] >> 16);
        }
    }
}

// Two values of the block at once: their maxima or sums, in every thread.
template <bool MAX>
__device__ __forceinline__ float2 block_pair(float x, float y, float2* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float a = __shfl_xor_sync(0xFFFFFFFFu, x, o), b = __shfl_xor_sync(0xFFFFFFFFu, y, o);
        x = MAX ? fmaxf(x, a) : x + a;
        y = MAX ? fmaxf(y, b) : y + b;
    }
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    float2 t = s[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) {
        t.x = MAX ? fmaxf(t.x, s[w].x) : t.x + s[w].x;
        t.y = MAX ? fmaxf(t.y, s[w].y) : t.y + s[w].y;
    }
    return t;
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Store a pair at the same shared-memory address of block `rank` of the cluster.
__device__ __forceinline__ void store_remote(float2* local, int rank, float2 v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(v.x), "f"(v.y) : "memory");
}

// RES: the block's share of the row stays in registers (DISTILL_VECS vectors a
// thread); otherwise the row is walked twice.  BWD: the row's log-sum-exp is
// given (lse_in) and nothing crosses the cluster.
template <int DT, bool RES, bool BWD>
__global__ void __launch_bounds__(DISTILL_THREADS, 2) k_distill(const __grid_constant__ DistillArgs a) {
    constexpr int W = RowVec<DT>::W;
    extern __shared__ Entry entry[];
    __shared__ float2 red[2][16], peer[DISTILL_CLUSTER];
    pdl_wait();
    pdl_launch_next();
    const int C = a.split, rank = (int)(blockIdx.x % (unsigned)C);
    const int64_t row = blockIdx.x / (unsigned)C;
    if (!BWD && C > 1) cluster_arrive();          // this block runs: its shared memory may be written
    const RowVec<DT> rv(static_cast<const char*>(a.z) + row * a.ldz * Elem<DT>::SIZE, a.cols);
    const int64_t step = (int64_t)C * blockDim.x, first = (int64_t)rank * blockDim.x + threadIdx.x;

    uint4 raw[RES ? DISTILL_VECS : 1];
    if constexpr (RES && !BWD) {
#pragma unroll
        for (int j = 0; j < DISTILL_VECS; ++j)
            if (first + j * step < rv.n) raw[j] = rv.load(first + j * step);
    }
    // the teacher's entries, and the student's logits at them (read before any
    // gradient is written, which may be in their place)
    float tmax = -INFINITY;
    for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
        const int64_t at = row * a.ldi + i;
        const int64_t id = a.id64 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
        const float t = ld1_any(a.t, row * a.ldt + i, a.t_dt);
        const bool have = id >= 0 && id < a.cols && t != -INFINITY;
        Entry en;
        en.id = have ? (int)id : -1;
        en.lp = have ? t * a.k2 : -INFINITY;
        // the backward pass alone has no barrier between its blocks: it reads what it itself will write
        const bool mine = have && (!BWD || (int)((id + rv.off) / W / blockDim.x % C) == rank);
        en.z = mine ? ld1<DT>(rv.base, id) : 0.f;
        en.p = 0.f;
        entry[i] = en;
        if (have) tmax = fmaxf(tmax, t != t ? 0.f : en.lp);     // a NaN entry makes the sum NaN, not the row empty
    }
    const float k2 = a.k2;
    float zmax = -INFINITY;
    if constexpr (!BWD) {
        if constexpr (RES) {
#pragma unroll
            for (int j = 0; j < DISTILL_VECS; ++j)
                if (first + j * step < rv.n) {
                    float v[W];
                    widen<DT>(raw[j], v);
#pragma unroll
                    for (int e = 0; e < W; ++e) zmax = fmaxf(zmax, v[e]);
                }
        } else {
            for (int64_t i = first; i < rv.n; i += step) {
                float v[W];
                widen<DT>(rv.load(i), v);
#pragma unroll
                for (int e = 0; e < W; ++e) zmax = fmaxf(zmax, v[e]);
            }
        }
    }
    float2 top = block_pair<true>(zmax, tmax, red[0]);
    // a share that holds nothing but -inf adds nothing: its exponents are taken from 0
    const float own_mk = top.x == -INFINITY ? 0.f : top.x * k2;
    float zsum = 0.f, tsum = 0.f;
    if constexpr (!BWD) {
        if constexpr (RES) {
#pragma unroll
            for (int j = 0; j < DISTILL_VECS; ++j)
                if (first + j * step < rv.n) {
                    float v[W];
                    widen<DT>(raw[j], v);
#pragma unroll
                    for (int e = 0; e < W; ++e) zsum += exp2_fast(fmaf(v[e], k2, -own_mk));
                }
        } else {
            for (int64_t i = first; i < rv.n; i += step) {
                float v[W];
                widen<DT>(rv.load(i), v);
#pragma unroll
                for (int e = 0; e < W; ++e) zsum += exp2_fast(fmaf(v[e], k2, -own_mk));
            }
        }
    }
    // with the teacher's own log-sum-exp the entries' exponents are taken from it
    const float tm = a.t_lse ? a.t_lse[row] * 1.4426950408889634f : top.y;
    for (int i = threadIdx.x; i < a.k; i += blockDim.x)
        if (entry[i].id >= 0) tsum += (entry[i].p = exp2f(entry[i].lp - tm));
    float2 sum = block_pair<false>(zsum, tsum, red[1]);
    const bool none = top.y == -INFINITY;           // no teacher entry in the row
    const float pscale = a.t_lse ? 1.f : 1.f / sum.y, P = none ? 0.f : sum.y * pscale;
    const float lpoff = tm + (a.t_lse ? 0.f : log2f(sum.y));

    // m k and the sum of the whole row
    float mk, total;
    if constexpr (BWD) {
        mk = a.lse_in[row] * 1.4426950408889634f;
        total = 1.f;
    } else if (C == 1) {
        mk = own_mk;
        total = sum.x;
    } else {
        cluster_wait();                            // every block of the cluster runs
        if (threadIdx.x < (unsigned)C)
            store_remote(&peer[rank], threadIdx.x, make_float2(top.x == -INFINITY ? -INFINITY : own_mk, sum.x));
        __syncwarp();
        cluster_arrive();
        cluster_wait();                            // every block's pair is here; no block leaves before its last arrives
        mk = -INFINITY;
        for (int c = 0; c < C; ++c) mk = fmaxf(mk, peer[c].x);
        total = 0.f;
        for (int c = 0; c < C; ++c)
            total += peer[c].x == -INFINITY ? 0.f : peer[c].y * exp2f(peer[c].x - mk);
        if (mk == -INFINITY) mk = 0.f;
        for (int c = 0; c < C; ++c)                // a maximum drops NaN; the sums keep it
            if (peer[c].y != peer[c].y) total = peer[c].y;
    }
    const float lg = BWD ? 0.f : log2f(total);
    const float w = a.w ? a.w[row] : 1.f;
    const bool dead = none || w == 0.f;
    if (!BWD && a.lse && rank == 0 && threadIdx.x == 0) a.lse[row] = (mk + lg) * 0.6931471805599453f;
    if (!BWD && a.loss && rank == 0) {
        float l = 0.f;
        if (!dead)
            for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
                const Entry en = entry[i];
                if (en.id >= 0 && en.p != 0.f)
                    l += en.p * pscale * ((en.lp - lpoff) - (fmaf(en.z, k2, -mk) - lg));
            }
        const float2 s = block_pair<false>(l, 0.f, red[0]);
        if (threadIdx.x == 0)
            a.loss[row] = dead ? 0.f : s.x * 0.6931471805599453f * a.temperature * a.temperature * w;
    }
    if (!a.dz) return;
    float coef = w * a.temperature * a.grad_scale;
    if (a.chain) coef *= (float)a.chain->loss_scale;
    const float g = dead ? 0.f : coef * P / total;
    char* drow = static_cast<char*>(a.dz) + row * a.lddz * Elem<DT>::SIZE;
    const bool same = ((reinterpret_cast<uintptr_t>(drow) ^ reinterpret_cast<uintptr_t>(rv.base)) & 15u) == 0;
    if constexpr (RES && !BWD) {
#pragma unroll
        for (int j = 0; j < DISTILL_VECS; ++j)
            if (first + j * step < rv.n) {
                float v[W];
                widen<DT>(raw[j], v);
#pragma unroll
                for (int e = 0; e < W; ++e) v[e] = dead ? 0.f : g * exp2_fast(fmaf(v[e], k2, -mk));
                rv.store(drow, same, first + j * step, v);
            }
    } else {
        for (int64_t i = first; i < rv.n; i += step) {
            float v[W];
            widen<DT>(rv.load(i), v);
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = dead ? 0.f : g * exp2_fast(fmaf(v[e], k2, -mk));
            rv.store(drow, same, i, v);
        }
    }
    if (dead) return;
    // the entries that lie in this block's vectors, written over after it
    // wrote those: the same id twice gives the same value twice
    __syncthreads();
    for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
        const Entry en = entry[i];
        if (en.id < 0) continue;
        const int64_t v = (en.id + rv.off) / W;
        if ((int)(v / blockDim.x % C) != rank) continue;
        float p = 0.f;
        for (int j = 0; j < a.k; ++j) p += entry[j].id == en.id ? entry[j].p : 0.f;
        st1<DT>(drow, en.id, fmaf(g, exp2_fast(fmaf(en.z, k2, -mk)), -coef * p * pscale));
    }
}

template <int DT>
static const void* distill_fn(bool res, bool bwd) {
    if (bwd) return (const void*)k_distill<DT, false, true>;
    return res ? (const void*)k_distill<DT, true, false> : (const void*)k_distill<DT, false, false>;
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
    const std::string w(who);
    int rc = check_mat(logits, rows, cols, FLOAT_TYPES, (w + ": logits").c_str());
    if (rc == ZERO_OK) rc = check_mat(ids, rows, k, 1u << ZERO_I32 | 1u << ZERO_I64, (w + ": ids").c_str());
    if (rc == ZERO_OK) rc = check_mat(teacher, rows, k, FLOAT_TYPES, (w + ": teacher").c_str());
    if (rc == ZERO_OK && (dlogits || bwd)) rc = check_mat(dlogits, rows, cols, FLOAT_TYPES, (w + ": dlogits").c_str());
    if (rc != ZERO_OK) return rc;
    if (dlogits && dlogits->dtype != logits->dtype) return bad(ZERO_EINVAL, "dlogits is in the logits' type");
    if (bwd && rows > 0 && cols > 0 && !lse_in) return bad(ZERO_EINVAL, "NULL lse");
    if (!aligned(teacher_lse, 4) || !aligned(row_weight, 4) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(lse_in, 4))
        return bad(ZERO_EALIGN, "a row array is not 4-byte aligned");
    if (!aligned(chain, 8)) return bad(ZERO_EALIGN, "chain not 8-byte aligned");
    if (rows == 0 || cols == 0) return ZERO_OK;
    const int sms = sm_count();
    if (!sms) return ZERO_ECUDA;

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

    // Vectors of a row, with the one that an unaligned start adds; threads so
    // that a short row leaves none idle; then the fewest blocks that hold a
    // row in registers, and more while the rows alone do not fill the GPU.
    const int W = 16 / elem_size(logits->dtype);
    const int64_t n = (cols + W - 1) / W + 1;
    const int threads = n <= 1024 ? 128 : n <= 2048 ? 256 : DISTILL_THREADS;
    const int64_t per = (int64_t)threads * DISTILL_VECS;
    int split = 1;
    while (split < DISTILL_CLUSTER && split * per < n) split *= 2;
    const bool res = split * per >= n;
    while (split < DISTILL_CLUSTER && rows * split < 2 * (int64_t)sms && split * threads < n) split *= 2;
    a.split = split;

    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * split));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = sizeof(Entry) * (size_t)k;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = bwd ? 1 : 2;
    const void* f = logits->dtype == ZERO_F32 ? distill_fn<ZERO_F32>(res, bwd)
                  : logits->dtype == ZERO_BF16 ? distill_fn<ZERO_BF16>(res, bwd) : distill_fn<ZERO_F16>(res, bwd);
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
