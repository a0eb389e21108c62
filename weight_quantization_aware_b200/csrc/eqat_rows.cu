// Operators over rows of logits [T, V]: log probabilities of given tokens with the
// entropy and the top alternatives of each row, and distillation from a teacher's top
// alternatives (loss and gradient).
//
// Both are HBM-bound: a row is read once from memory, and the gradient written once.
// A CTA owns a row and walks it in 16-byte vectors.  The first walk keeps a running
// maximum m, S = sum 2^y and (for the entropy) A = sum 2^y y per thread, with
// y = (x - m) c and c = log2(e) / temperature; x - m is formed before the product, so
// that a row masked with the type's lowest value, and the largest entries of any row,
// lose nothing.  The second walk (top alternatives, gradient) reads the row again
// while it is in L2.
//
// All sums are fp32 per thread (a few hundred terms of one sign), joined over the
// block in a fixed order; the few values per row (log S, the loss) are fp64.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "eqat_internal.h"
#include "eqat_pdl.cuh"
#include "eqat_qmath.cuh"

namespace eqat {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;         // 16-byte vectors in flight per thread
constexpr int kCandidates = 2048;  // shared-memory candidates of the top-k selection
constexpr uint32_t kNegInfBf16x2 = 0xFF80FF80u;
constexpr uint32_t kNegInfF32 = 0xFF800000u;

// ------------------------------------------------------------------ vectors

__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// A 16-byte vector of a row: N elements, read as N / 2 fp32 pairs.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kFill = kNegInfBf16x2;
    static __device__ __forceinline__ void pairs(const uint4 &r, uint64_t (&p)[4]) {
        p[0] = f2_pack(bf16_lo(r.x), bf16_hi(r.x));
        p[1] = f2_pack(bf16_lo(r.y), bf16_hi(r.y));
        p[2] = f2_pack(bf16_lo(r.z), bf16_hi(r.z));
        p[3] = f2_pack(bf16_lo(r.w), bf16_hi(r.w));
    }
    // the largest element that is not NaN (-inf if there is none)
    static __device__ __forceinline__ float max(const uint4 &r) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ void set(uint4 &r, int j, uint32_t raw) {
        uint32_t *w = reinterpret_cast<uint32_t *>(&r);
        const int sh = 16 * (j & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i == (j >> 1)) w[i] = (w[i] & ~(0xFFFFu << sh)) | ((raw & 0xFFFFu) << sh);
    }
    static __device__ __forceinline__ uint32_t raw(const __nv_bfloat16 *p) {
        return *reinterpret_cast<const unsigned short *>(p);
    }
    static __device__ __forceinline__ float value(const uint4 &r, int j) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
        uint32_t x = w[0];
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i == (j >> 1)) x = w[i];
        return (j & 1) ? bf16_hi(x) : bf16_lo(x);
    }
    static __device__ __forceinline__ uint4 from_pairs(const uint64_t (&p)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(p[i], lo, hi);
            w[i] = pack_bf16x2(lo, hi);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kFill = kNegInfF32;
    static __device__ __forceinline__ void pairs(const uint4 &r, uint64_t (&p)[2]) {
        p[0] = f2_pack(__uint_as_float(r.x), __uint_as_float(r.y));
        p[1] = f2_pack(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ float max(const uint4 &r) {
        return fmaxf(fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                           fmaxf(__uint_as_float(r.z), __uint_as_float(r.w))),
                     -INFINITY);
    }
    static __device__ __forceinline__ void set(uint4 &r, int j, uint32_t raw) {
        uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i == j) w[i] = raw;
    }
    static __device__ __forceinline__ uint32_t raw(const float *p) { return __float_as_uint(*p); }
    static __device__ __forceinline__ float value(const uint4 &r, int j) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
        uint32_t x = w[0];
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i == j) x = w[i];
        return __uint_as_float(x);
    }
    static __device__ __forceinline__ uint4 from_pairs(const uint64_t (&p)[2]) {
        float a, b, c, d;
        f2_unpack(p[0], a, b);
        f2_unpack(p[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
};

// The aligned 16-byte vectors that cover a row: the row starts `mis` elements into the
// first one and ends inside the last.
template <typename T>
struct Row {
    T *base;  // the first vector (at or before the row's first element)
    int64_t V, mis, nv;
    __device__ __forceinline__ Row(T *row, int64_t V_) : V(V_) {
        mis = static_cast<int64_t>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        base = row - mis;
        nv = (mis + V + Vec<T>::N - 1) / Vec<T>::N;
    }
    __device__ __forceinline__ bool full(int64_t v) const {
        return v * Vec<T>::N >= mis && (v + 1) * Vec<T>::N <= mis + V;
    }
    // Vector v; elements outside the row read as -inf and are not touched in memory.
    __device__ __forceinline__ uint4 load(int64_t v) const {
        uint4 r;
        if (full(v)) {
            const T *p = base + v * Vec<T>::N;
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                         : "l"(p)
                         : "memory");
        } else {
            r = make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
            for (int j = 0; j < Vec<T>::N; ++j) {
                const int64_t e = v * Vec<T>::N + j;
                if (e >= mis && e < mis + V) Vec<T>::set(r, j, Vec<T>::raw(base + e));
            }
        }
        return r;
    }
    __device__ __forceinline__ void store(int64_t v, const uint4 &r) const {
        if (full(v)) {
            *reinterpret_cast<uint4 *>(base + v * Vec<T>::N) = r;
        } else {
            for (int j = 0; j < Vec<T>::N; ++j) {
                const int64_t e = v * Vec<T>::N + j;
                if (e >= mis && e < mis + V) Vec<T>::store(base + e, Vec<T>::value(r, j));
            }
        }
    }
};

// ------------------------------------------------------------------ running softmax sums

// m is finite from the start (the type's lowest value), so that x - m is -inf, never
// NaN, for a masked entry.  A NaN or +inf entry makes S NaN and stays.
template <bool ENT>
struct Sums {
    float m = -FLT_MAX;
    uint64_t S = 0, A = 0;  // two partial sums each

    template <typename T, int U>
    __device__ __forceinline__ void add(const uint4 (&r)[U], float c) {
        float mx = Vec<T>::max(r[0]);
#pragma unroll
        for (int u = 1; u < U; ++u) mx = fmaxf(mx, Vec<T>::max(r[u]));
        if (mx > m) {
            const float g = fmaxf((m - mx) * c, -1e4f), f = ex2(g);
            const uint64_t f2 = f2_pack(f, f);
            if (ENT) A = f2_mul(f2_fma(S, f2_pack(g, g), A), f2);
            S = f2_mul(S, f2);
            m = mx;
        }
        const uint64_t nm = f2_pack(-m, -m), c2 = f2_pack(c, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint64_t p[Vec<T>::N / 2];
            Vec<T>::pairs(r[u], p);
#pragma unroll
            for (int i = 0; i < Vec<T>::N / 2; ++i) {
                float a, b;
                f2_unpack(f2_mul(f2_add(p[i], nm), c2), a, b);
                if (ENT) {  // 2^-200 is 0 in fp32, and 0 times -200 is 0
                    a = max_nan(a, -200.0f);
                    b = max_nan(b, -200.0f);
                }
                const uint64_t e = f2_pack(ex2(a), ex2(b));
                S = f2_add(S, e);
                if (ENT) A = f2_fma(e, f2_pack(a, b), A);
            }
        }
    }
};

struct RowSums {
    float m, S, A;
};

__device__ __forceinline__ RowSums join(const RowSums &a, const RowSums &b, float c) {
    RowSums r;
    r.m = fmaxf(a.m, b.m);
    const float ga = fmaxf((a.m - r.m) * c, -1e4f), gb = fmaxf((b.m - r.m) * c, -1e4f);
    const float fa = ex2(ga), fb = ex2(gb);
    r.S = fa * a.S + fb * b.S;
    r.A = fa * fmaf(a.S, ga, a.A) + fb * fmaf(b.S, gb, b.A);
    return r;
}

// The block's sums, in every thread; `buf` holds kWarps entries.  The join over lanes
// is a butterfly (the two sides of a pair differ in operand order only, and join is
// symmetric up to the order of one addition), the join over warps runs in order.
template <bool ENT>
__device__ __forceinline__ RowSums block_join(const Sums<ENT> &s, float c, RowSums *buf) {
    RowSums r;
    float lo, hi;
    r.m = s.m;
    f2_unpack(s.S, lo, hi);
    r.S = lo + hi;
    f2_unpack(s.A, lo, hi);
    r.A = lo + hi;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        RowSums o;
        o.m = __shfl_xor_sync(0xffffffffu, r.m, off);
        o.S = __shfl_xor_sync(0xffffffffu, r.S, off);
        o.A = __shfl_xor_sync(0xffffffffu, r.A, off);
        r = join(r, o, c);
    }
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = r;
    __syncthreads();
    r = buf[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) r = join(r, buf[w], c);
    return r;
}

template <bool ENT, typename T>
__device__ __forceinline__ Sums<ENT> walk_sums(const Row<T> &row, float c) {
    Sums<ENT> s;
    for (int64_t v = threadIdx.x; v < row.nv; v += kThreads * kUnroll) {
        uint4 r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            r[u] = v + u * kThreads < row.nv
                       ? row.load(v + u * kThreads)
                       : make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
        s.template add<T, kUnroll>(r, c);
    }
    return s;
}

// ------------------------------------------------------------------ log probabilities

struct LogprobArgs {
    const void *x;
    int64_t ld, T, V;
    const int64_t *targets;
    float c;         // log2(e) / temperature
    double inv_tau;  // 1 / temperature
    int k;
    float *logprob, *entropy;
    int64_t *top_ids;
    float *top_logprobs;
};

// An order-keeping key of a logit (never NaN here): larger value, larger key; -0 is 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct TopShared {
    uint64_t cand[kCandidates];  // key << 32 | ~index: unique, larger = earlier
    float gmax[kThreads];
    float threshold;
    int count;
    int warp_count[kWarps];
};

// Elements of the row for which pred(key, index) holds, counted over the block.
template <typename T, typename Pred>
__device__ int64_t block_count(const Row<T> &row, TopShared &sh, Pred pred) {
    int n = 0;
    for (int64_t v = threadIdx.x; v < row.nv; v += kThreads) {
        const uint4 r = row.load(v);
#pragma unroll
        for (int j = 0; j < Vec<T>::N; ++j) {
            const float x = Vec<T>::value(r, j);
            n += x > -INFINITY && pred(order_key(x), static_cast<uint32_t>(v * Vec<T>::N + j - row.mis));
        }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.warp_count[threadIdx.x >> 5] = n;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kWarps; ++w) total += sh.warp_count[w];
    return total;
}

// The k largest (value, lowest index first) of a row without NaN or +inf.  The k-th
// largest of at least k thread (or thread-group) maxima is a bound that at least k
// elements reach; what reaches it, usually about 1.4 k elements, is collected in
// shared memory and ranked by counting.  Where ties or an uneven row make that more
// than the buffer, the k-th key and then the last index of its ties are found bit by
// bit with one walk each.
template <typename T>
__device__ void top_k(const Row<T> &row, const LogprobArgs &a, int64_t t, float thread_max, float m, double logS,
                      TopShared &sh) {
    const int tid = threadIdx.x, k = a.k;
    // groups of threads, a power of two at least twice k
    int group = 1;
    while (kThreads / (2 * group) >= 2 * k && group < 32) group *= 2;
    float g = thread_max;
    for (int off = 1; off < group; off *= 2) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, off));
    const int ng = kThreads / group;
    if ((tid & (group - 1)) == 0) sh.gmax[tid / group] = g;
    if (tid == 0) sh.count = 0;
    __syncthreads();
    if (tid < ng) {
        const float mine = sh.gmax[tid];
        int rank = 0;
        for (int j = 0; j < ng; ++j) {
            const float o = sh.gmax[j];
            rank += o > mine || (o == mine && j < tid);
        }
        if (rank == k - 1) sh.threshold = mine;
    }
    __syncthreads();
    const float thr = sh.threshold;
    for (int64_t v = tid; v < row.nv; v += kThreads) {
        const uint4 r = row.load(v);
        if (Vec<T>::max(r) >= thr) {
#pragma unroll
            for (int j = 0; j < Vec<T>::N; ++j) {
                const float x = Vec<T>::value(r, j);
                if (x >= thr && x > -INFINITY) {
                    const int at = atomicAdd(&sh.count, 1);
                    const uint32_t idx = static_cast<uint32_t>(v * Vec<T>::N + j - row.mis);
                    if (at < kCandidates) sh.cand[at] = (static_cast<uint64_t>(order_key(x)) << 32) | ~idx;
                }
            }
        }
    }
    __syncthreads();
    int n = sh.count;
    if (n > kCandidates) {
        uint32_t key = 0;
        for (int b = 31; b >= 0; --b) {
            const uint32_t cand = key | (1u << b);
            if (block_count(row, sh, [=](uint32_t q, uint32_t) { return q >= cand; }) >= k) key = cand;
        }
        const int64_t above = block_count(row, sh, [=](uint32_t q, uint32_t) { return q > key; });
        // the largest index bound that still leaves fewer than the needed ties before it
        const int64_t need = k - above;
        uint32_t last = 0;
        for (int b = 31; b >= 0; --b) {
            const uint32_t cand = last | (1u << b);
            if (cand <= static_cast<uint32_t>(a.V - 1) &&
                block_count(row, sh, [=](uint32_t q, uint32_t i) { return q == key && i < cand; }) < need)
                last = cand;
        }
        __syncthreads();
        if (tid == 0) sh.count = 0;
        __syncthreads();
        for (int64_t v = tid; v < row.nv; v += kThreads) {
            const uint4 r = row.load(v);
#pragma unroll
            for (int j = 0; j < Vec<T>::N; ++j) {
                const float x = Vec<T>::value(r, j);
                const uint32_t q = order_key(x), idx = static_cast<uint32_t>(v * Vec<T>::N + j - row.mis);
                if (x > -INFINITY && (q > key || (q == key && idx <= last)))
                    sh.cand[atomicAdd(&sh.count, 1)] = (static_cast<uint64_t>(q) << 32) | ~idx;
            }
        }
        __syncthreads();
        n = sh.count;  // exactly k
    }
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t mine = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > mine;
        if (rank < k) {
            a.top_ids[t * k + rank] = static_cast<int64_t>(~static_cast<uint32_t>(mine));
            const float x = key_value(static_cast<uint32_t>(mine >> 32));
            a.top_logprobs[t * k + rank] = static_cast<float>((static_cast<double>(x) - m) * a.inv_tau - logS);
        }
    }
    for (int i = n + tid; i < k; i += kThreads) {
        a.top_ids[t * k + i] = -1;
        a.top_logprobs[t * k + i] = -INFINITY;
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_token_logprobs(const LogprobArgs a) {
    __shared__ RowSums buf[kWarps];
    __shared__ TopShared sh;
    pdl_wait();
    pdl_allow_dependents();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        T *p = const_cast<T *>(static_cast<const T *>(a.x)) + t * a.ld;
        const Row<T> row(p, a.V);
        const Sums<true> mine = walk_sums<true>(row, a.c);
        const RowSums s = block_join(mine, a.c, buf);
        const bool none = s.S == 0.0f, bad = !(s.S >= 0.0f) || s.S == INFINITY;
        const double logS = log(static_cast<double>(s.S));
        if (threadIdx.x == 0) {
            const int64_t id = a.targets[t];
            float lp = 0.0f;
            if (id >= a.V)
                lp = NAN;
            else if (id >= 0)
                lp = none ? -INFINITY
                          : static_cast<float>((static_cast<double>(Vec<T>::load(p + id)) - s.m) * a.inv_tau - logS);
            if (bad && id >= 0) lp = NAN;
            a.logprob[t] = lp;
            // H = -sum p ln p = ln S - ln 2 (A / S)
            a.entropy[t] = none ? 0.0f
                                : static_cast<float>(logS - 0.69314718055994530942 * (static_cast<double>(s.A) / s.S));
        }
        if (a.k > 0) {
            if (bad || none) {
                for (int i = threadIdx.x; i < a.k; i += kThreads) {
                    a.top_ids[t * a.k + i] = -1;
                    a.top_logprobs[t * a.k + i] = bad ? NAN : -INFINITY;
                }
            } else {
                top_k(row, a, t, mine.m, s.m, logS, sh);
            }
        }
        __syncthreads();  // buf is written again by the next row
    }
}

// ------------------------------------------------------------------ distillation

struct DistillArgs {
    const void *x;
    int64_t ld, T, V;
    const int64_t *ids;
    const float *tlp;
    int k;
    float c;
    double inv_tau;
    const float *weight;  // nullable: 1
    float *loss;          // nullable
    void *dx;             // nullable; may be x
};

struct Slots {
    int id[kTopMax];  // -1: empty
    float x[kTopMax], tl[kTopMax], q[kTopMax], grad[kTopMax];
    bool first[kTopMax];  // the slot that stands for its id where an id is given twice
    float coef;
    int zero;
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// One warp: the teacher's masses, the loss and the gradient's constants of a row.
// With z = x / temperature, p = softmax(z), q the teacher's masses on the slots:
//   L = sum_i q_i (ln q_i - ln p_i)  [+ q_r (ln q_r - ln p_r)]
//   dL/dz_j = p_j - q_j on a slot, p_j [(1 - q_r / p_r)] elsewhere.
// `s` are the sums over the row (renormalised teacher) or over the entries outside the
// slots (TAIL): p_r is then a sum of its own and not 1 minus the slots' masses, which
// would cancel when nearly all mass is on the slots.
template <bool TAIL>
__device__ void finish_slots(const DistillArgs &a, Slots &sl, const RowSums &s, bool bad_id, bool dup, float w,
                             float *loss) {
    const int lane = threadIdx.x & 31, k = a.k;
    // teacher
    float tm = -INFINITY;
    bool any = false, tnan = false;
    for (int i = lane; i < k; i += 32)
        if (sl.id[i] >= 0) {
            tm = fmaxf(tm, sl.tl[i]);
            any = any || sl.tl[i] > -INFINITY;
            tnan = tnan || isnan(sl.tl[i]);
        }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, off));
    any = __any_sync(0xffffffffu, any);
    tnan = __any_sync(0xffffffffu, tnan);
    const double shift = TAIL || !any ? 0.0 : static_cast<double>(tm);
    double qsum = 0.0;
    for (int i = lane; i < k; i += 32)
        if (sl.id[i] >= 0) qsum += exp(static_cast<double>(sl.tl[i]) - shift);
    qsum = warp_sum(qsum);
    tnan = tnan || !(qsum < INFINITY);
    const double logq0 = TAIL ? 0.0 : shift + log(qsum);  // ln q_i = tl_i - logq0
    // student: the sums over all entries
    RowSums all = s;
    if (TAIL) {
        RowSums mine{-FLT_MAX, 0.0f, 0.0f};
        for (int i = lane; i < k; i += 32)
            if (sl.id[i] >= 0 && sl.first[i]) mine.m = fmaxf(mine.m, sl.x[i]);
        for (int i = lane; i < k; i += 32)
            if (sl.id[i] >= 0 && sl.first[i]) mine.S += ex2((sl.x[i] - mine.m) * a.c);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            RowSums o{__shfl_xor_sync(0xffffffffu, mine.m, off), __shfl_xor_sync(0xffffffffu, mine.S, off), 0.0f};
            mine = join(mine, o, a.c);
        }
        all = join(s, mine, a.c);
    }
    const double lnS = log(static_cast<double>(all.S));
    const double qr = TAIL ? fmax(1.0 - qsum, 0.0) : 0.0;
    const bool live = TAIL && qr > 0.0 && s.S > 0.0f;
    double L = 0.0;
    for (int i = lane; i < k; i += 32) {
        if (sl.id[i] < 0) continue;
        const double lq = static_cast<double>(sl.tl[i]) - logq0;
        const double q = exp(lq);
        sl.q[i] = static_cast<float>(q);
        if (q > 0.0) L += q * (lq - ((static_cast<double>(sl.x[i]) - all.m) * a.inv_tau - lnS));
    }
    L = warp_sum(L);
    if (live)
        L += qr * (log(qr) - (log(static_cast<double>(s.S)) + (static_cast<double>(s.m) - all.m) * a.inv_tau - lnS));
    __syncwarp();
    const double up = static_cast<double>(w) * a.inv_tau;
    for (int i = lane; i < k; i += 32) {
        if (sl.id[i] < 0 || !sl.first[i]) continue;
        double q = sl.q[i];
        if (dup) {  // an id given more than once carries its slots' masses together
            q = 0.0;
            for (int j = 0; j < k; ++j)
                if (sl.id[j] == sl.id[i]) q += sl.q[j];
        }
        const double p = static_cast<double>(ex2((sl.x[i] - all.m) * a.c)) / all.S;
        sl.grad[i] = static_cast<float>(up * (p - q));
    }
    if (lane == 0) {
        // a teacher without an alternative, or a student without an entry: no loss
        const bool zero = !bad_id && !tnan && ((!TAIL && !any) || all.S == 0.0f);
        const bool nan = bad_id || tnan || !(all.S >= 0.0f);
        const double F = static_cast<double>(ex2(fmaxf((s.m - all.m) * a.c, -1e4f)));
        double coef = F / all.S;
        if (live) coef -= qr / s.S;
        sl.zero = zero;
        sl.coef = nan ? NAN : static_cast<float>(up * coef);
        if (loss) *loss = zero ? 0.0f : nan ? NAN : static_cast<float>(w * L);
    }
}

template <typename T, bool TAIL>
__global__ void __launch_bounds__(kThreads, 4) k_distill(const DistillArgs a) {
    extern __shared__ uint32_t bitmap[];  // one bit per element of the row's vectors: it is a slot
    __shared__ RowSums buf[kWarps];
    __shared__ Slots sl;
    const int tid = threadIdx.x;
    const int words = static_cast<int>((a.V + Vec<T>::N + 31) / 32);
    for (int i = tid; i < words; i += kThreads) bitmap[i] = 0;
    pdl_wait();
    pdl_allow_dependents();
    __syncthreads();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        T *p = const_cast<T *>(static_cast<const T *>(a.x)) + t * a.ld;
        const Row<T> row(p, a.V);
        const Row<T> out(a.dx ? static_cast<T *>(a.dx) + t * a.ld : p, a.V);  // same phase as the row
        const float w = a.weight ? a.weight[t] : 1.0f;
        if (w == 0.0f) {  // a token without a loss: nothing of its row is read
            if (a.dx)
                for (int64_t v = tid; v < out.nv; v += kThreads) out.store(v, make_uint4(0, 0, 0, 0));
            if (tid == 0 && a.loss) a.loss[t] = 0.0f;
            continue;
        }
        bool bad = false, twice = false;
        if (tid < a.k) {
            const int64_t id = a.ids[t * a.k + tid];
            bad = id >= a.V;
            const bool use = id >= 0 && !bad;
            sl.id[tid] = use ? static_cast<int>(id) : -1;
            sl.first[tid] = false;
            if (use) {
                const int at = static_cast<int>(id + row.mis);
                const uint32_t bit = 1u << (at & 31);
                const bool first = !(atomicOr(&bitmap[at >> 5], bit) & bit);
                sl.first[tid] = first;
                twice = !first;
                sl.x[tid] = Vec<T>::load(p + id);
                sl.tl[tid] = a.tlp[t * a.k + tid];
            }
        }
        bad = __syncthreads_or(bad);
        twice = __syncthreads_or(twice);
        Sums<false> mine;
        for (int64_t v = tid; v < row.nv; v += kThreads * kUnroll) {
            uint4 r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t vv = v + u * kThreads;
                r[u] = vv < row.nv ? row.load(vv)
                                   : make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
            }
            if (TAIL) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int64_t vv = v + u * kThreads;
                    if (vv < row.nv) {
                        const int at = static_cast<int>(vv * Vec<T>::N);
                        const uint32_t bits = (bitmap[at >> 5] >> (at & 31)) & ((1u << Vec<T>::N) - 1u);
                        if (bits)
                            for (int j = 0; j < Vec<T>::N; ++j)
                                if ((bits >> j) & 1u) Vec<T>::set(r[u], j, Vec<T>::kFill);
                    }
                }
            }
            mine.template add<T, kUnroll>(r, a.c);
        }
        const RowSums s = block_join(mine, a.c, buf);
        if (tid < 32) finish_slots<TAIL>(a, sl, s, bad, twice, w, a.loss ? a.loss + t : nullptr);
        __syncthreads();
        if (a.dx) {
            const float coef = sl.coef;
            const bool zero = sl.zero;
            const uint64_t nm = f2_pack(-s.m, -s.m), c2 = f2_pack(a.c, a.c), k2 = f2_pack(coef, coef);
            for (int64_t v = tid; v < row.nv; v += kThreads * kUnroll) {
                uint4 r[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
                    if (v + u * kThreads < row.nv) r[u] = row.load(v + u * kThreads);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (v + u * kThreads >= row.nv) continue;
                    uint64_t e[Vec<T>::N / 2];
                    Vec<T>::pairs(r[u], e);
#pragma unroll
                    for (int i = 0; i < Vec<T>::N / 2; ++i) {
                        float lo, hi;
                        f2_unpack(f2_mul(f2_add(e[i], nm), c2), lo, hi);
                        e[i] = f2_mul(f2_pack(ex2(lo), ex2(hi)), k2);
                    }
                    out.store(v + u * kThreads, zero ? make_uint4(0, 0, 0, 0) : Vec<T>::from_pairs(e));
                }
            }
        }
        __syncthreads();
        if (tid < a.k && sl.id[tid] >= 0) {
            if (a.dx && !sl.zero && !bad && sl.first[tid])
                Vec<T>::store(out.base + out.mis + sl.id[tid], isnan(sl.coef) ? NAN : sl.grad[tid]);
            bitmap[static_cast<int>(sl.id[tid] + row.mis) >> 5] = 0;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const void *x, bool f32, int64_t ld, int64_t T, int64_t V, const int64_t *targets,
                                  double temperature, int k, float *logprob, float *entropy, int64_t *top_ids,
                                  float *top_logprobs, const DeviceInfo &dev, cudaStream_t st) {
    LogprobArgs a{x, ld, T, V, targets, static_cast<float>(1.44269504088896340736 / temperature), 1.0 / temperature,
                  k, logprob, entropy, top_ids, top_logprobs};
    const int grid = static_cast<int>(std::min<int64_t>(T, static_cast<int64_t>(dev.sm_count) * 4));
    return f32 ? launch_pdl(k_token_logprobs<float>, dim3(grid), dim3(kThreads), 0, st, a)
               : launch_pdl(k_token_logprobs<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, st, a);
}

template <typename T, bool TAIL>
static cudaError_t launch_distill_t(const DistillArgs &a, const DeviceInfo &dev, cudaStream_t st) {
    const size_t smem = static_cast<size_t>((a.V + Vec<T>::N + 31) / 32) * 4;
    cudaError_t e = cudaFuncSetAttribute(k_distill<T, TAIL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kDistillMaxV + 64) / 8);
    if (e != cudaSuccess) return e;
    const int grid = static_cast<int>(std::min<int64_t>(a.T, static_cast<int64_t>(dev.sm_count) * 4));
    return launch_pdl(k_distill<T, TAIL>, dim3(grid), dim3(kThreads), smem, st, a);
}

cudaError_t launch_distill_topk(const void *x, bool f32, int64_t ld, int64_t T, int64_t V, const int64_t *ids,
                                const float *tlp, int k, double temperature, bool tail, const float *weight,
                                float *loss, void *dx, const DeviceInfo &dev, cudaStream_t st) {
    const DistillArgs a{x, ld, T, V, ids, tlp, k, static_cast<float>(1.44269504088896340736 / temperature),
                        1.0 / temperature, weight, loss, dx};
    if (f32) return tail ? launch_distill_t<float, true>(a, dev, st) : launch_distill_t<float, false>(a, dev, st);
    return tail ? launch_distill_t<__nv_bfloat16, true>(a, dev, st) : launch_distill_t<__nv_bfloat16, false>(a, dev, st);
}

}  // namespace eqat
