// Operators over rows of logits [T, V]: log probabilities of given tokens with the
// entropy and the top alternatives of each row, and distillation from a teacher's top
// alternatives (loss and gradient).
//
// Both are HBM-bound: a row is read once from memory, and the gradient written once.
// A CTA owns a row and walks it in 16-byte vectors.  The first walk keeps a running
// maximum m, S = sum 2^y and (for the entropy) A = sum 2^y y per thread, with
// y = (x - m) c and c = log2(e) / temperature.  y is one fma, x c - RN(m c), and what
// the rounding of m c moved all of a thread's terms by is taken out of S and A at the
// end (m c - RN(m c) is exact in one fma).  That form needs |m c| below 2^30, from where
// RN moves it by more than ex2 can say: m starts from a floor of -2^23 / c, which
// also keeps masked entries of any kind (-inf, the type's lowest value, -1e10) from being
// a reference.  A row without an entry above the floor, with one of 2^30 / c or more, or
// whose S is not finite (a NaN, an infinity) is walked again with x - m formed first.  The
// second walk (top alternatives, gradient) reads the row again while it is in L2.
//
// No one unit bounds the first walk: of 2048 x 32000 bf16, ex2 (a quarter of the issue
// rate) is busy half of the time, instructions issue in 61% of the cycles (one packed-fp32
// instruction does two entries of each step), DRAM runs at 47%, and the rest is the latency of
// loads and a last round of rows that is less than half full.
//
// Measured, bf16, calls back to back (a copy runs at 6.55 TB/s): log probabilities of
// 2048 x 32000 29-30 us (4.4 TB/s; fp32 45 us, 5.8 TB/s) and of 1024 x 131072 50 us (5.4
// TB/s), with 64 alternatives 66-68 and 84 us; the distillation step of 2048 x 32000 with
// 64 slots 70-71 us (3.7 TB/s; the block meets at two barriers between a row's walks), its loss
// alone 41 us, and the gradient alone of 2048 x 131072 211-226 us from box to box (4.8-5.1 TB/s).
//
// All sums are fp32 per thread (a few hundred terms of one sign), joined over the
// block in a fixed order; the few values per row (log S, the loss) are fp64.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "eqat_internal.h"
#include "eqat_pdl.cuh"
#include "eqat_ptx.cuh"
#include "eqat_qmath.cuh"

namespace eqat {
namespace {

// W, the template parameter of most functions here, is the number of threads that walk a
// row: 256 with three blocks per SM, or 768 in one block where there are no more long
// rows than SMs.  On 8 rows of 131072 bf16 the wide block takes 17.4 us where the narrow
// one takes 23.8 (distillation step) and 9.0 against 11.1 (log probabilities); on rows of
// 32000 they are even (9.4 and 9.6, 5.2 and 4.5), on shorter ones the narrow one wins.
// With alternatives the block of 256 does: its bound has fewer maxima to rank (22.7
// against 17.3 us on those rows).  64 threads, eight to twelve blocks per SM, walk many
// short rows: what a row costs besides its walk (joins, slots, alternatives) then runs
// for more rows at a time.  4096 rows of 1000 bf16 take 8.1 us (log probabilities) and 20.9
// (distillation step) where blocks of 256 take 20.7 and 49.5; 4096 of 16000 take 28.8 and
// 80.3 against 33.0 and 85.3, and 4096 of 32000 are slower (53.9, 143 against 53.4, 127).
constexpr int kWalkNarrow = 64, kWalk = 256, kWalkWide = 768;
constexpr int kUnroll = 4;  // 16-byte vectors per thread and chunk
constexpr int kStages = 3;  // chunks of the ring
template <int W>
constexpr int kChunk = W * kUnroll;  // vectors of a chunk: 4, 16 or 48 KB
template <int W>
constexpr size_t kRingBytes = static_cast<size_t>(kStages) * kChunk<W> * 16;
template <int W>
constexpr int kCtasPerSm = W == kWalkNarrow ? 8 : W == kWalk ? 3 : 1;
constexpr uint64_t kWaitLimitNs = 4000000000ull;     // far above any legitimate wait
constexpr int kNotes = 256;        // vectors that a warp notes for the top-k selection, in shared memory
constexpr int kKept = 1024;        // entries among them that are ranked
constexpr int64_t kNarrowBytes = 32 * 1024;  // of a row, at most, for the narrow block
constexpr size_t kWideBitBytes = 64 * 1024;  // bitmaps beside the wide ring: V up to 262000
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
    template <int U>
    static __device__ __forceinline__ float max(const uint4 (&r)[U]) {
        __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&r[0]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r[u]);
            m = __hmax2(m, __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        }
        return fmaxf(__low2float(m), __high2float(m));
    }
    // entries below `low` to about it; NaN stays
    static __device__ __forceinline__ uint4 clamp(uint4 r, float low) {
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&r);
        const __nv_bfloat162 f = __float2bfloat162_rn(low);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __hmax2_nan(h[i], f);
        return r;
    }
    static __device__ __forceinline__ void set(uint4 &r, int j, uint32_t raw) {
        const int sh = 16 * (j & 1), i = j >> 1;
        const uint32_t keep = ~(0xFFFFu << sh), put = (raw & 0xFFFFu) << sh;
        r.x = i == 0 ? (r.x & keep) | put : r.x;
        r.y = i == 1 ? (r.y & keep) | put : r.y;
        r.z = i == 2 ? (r.z & keep) | put : r.z;
        r.w = i == 3 ? (r.w & keep) | put : r.w;
    }
    // elements j with bit j set become -inf
    static __device__ __forceinline__ void fill(uint4 &r, uint32_t bits) {
        auto word = [&](uint32_t w, int i) {
            // bits 2 i and 2 i + 1 to the signs of bytes 0 and 1, and from there to halves
            const uint32_t sign = ((bits >> (2 * i)) & 1u) * 0x80u | ((bits >> (2 * i)) & 2u) * 0x4000u;
            uint32_t m;
            asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(m) : "r"(sign));
            return (w & ~m) | (kNegInfBf16x2 & m);
        };
        r = make_uint4(word(r.x, 0), word(r.y, 1), word(r.z, 2), word(r.w, 3));
    }
    static __device__ __forceinline__ uint32_t raw(const __nv_bfloat16 *p) {
        return *reinterpret_cast<const unsigned short *>(p);
    }
    static __device__ __forceinline__ float value(const uint4 &r, int j) {
        const int i = j >> 1;
        const uint32_t x = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
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
    template <int U>
    static __device__ __forceinline__ float max(const uint4 (&r)[U]) {
        float m = max(r[0]);
#pragma unroll
        for (int u = 1; u < U; ++u) m = fmaxf(m, max(r[u]));
        return m;
    }
    static __device__ __forceinline__ uint4 clamp(uint4 r, float low) {
        uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(max_nan(__uint_as_float(w[i]), low));
        return r;
    }
    static __device__ __forceinline__ void set(uint4 &r, int j, uint32_t raw) {
        r.x = j == 0 ? raw : r.x;
        r.y = j == 1 ? raw : r.y;
        r.z = j == 2 ? raw : r.z;
        r.w = j == 3 ? raw : r.w;
    }
    static __device__ __forceinline__ void fill(uint4 &r, uint32_t bits) {
        r.x = bits & 1u ? kFill : r.x;
        r.y = bits & 2u ? kFill : r.y;
        r.z = bits & 4u ? kFill : r.z;
        r.w = bits & 8u ? kFill : r.w;
    }
    static __device__ __forceinline__ uint32_t raw(const float *p) { return __float_as_uint(*p); }
    static __device__ __forceinline__ float value(const uint4 &r, int j) {
        return __uint_as_float(j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w);
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
// first one and ends inside the last.  Vectors b0 .. b1 - 1 lie in it whole.
template <typename T>
struct Row {
    static constexpr int N = Vec<T>::N;
    T *base;  // the first vector (at or before the row's first element)
    int V, mis, b0, b1;
    __device__ __forceinline__ Row(T *row, int V_) : V(V_) {
        mis = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        base = row - mis;
        b0 = mis ? 1 : 0;
        b1 = max(static_cast<int>((static_cast<uint32_t>(mis) + static_cast<uint32_t>(V)) / N), b0);
    }
    __device__ __forceinline__ const uint4 *vec(int v) const { return reinterpret_cast<const uint4 *>(base) + v; }
    // A vector that the row shares with its neighbours: thread 0 has the first, thread 1
    // the last.  False where there is none.
    __device__ __forceinline__ bool edge(int &v) const {
        v = threadIdx.x == 0 ? 0 : b1;
        if (threadIdx.x == 0) return mis != 0;
        return threadIdx.x == 1 && static_cast<int64_t>(b1) * N < static_cast<int64_t>(mis) + V;
    }
    __device__ __forceinline__ bool has(int v, int j) const {
        const int64_t e = static_cast<int64_t>(v) * N + j;
        return e >= mis && e < static_cast<int64_t>(mis) + V;
    }
    // an edge vector; elements outside the row read as -inf and are not touched in memory
    __device__ __forceinline__ uint4 load_edge(int v) const {
        uint4 r = make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
        for (int j = 0; j < N; ++j)
            if (has(v, j)) Vec<T>::set(r, j, Vec<T>::raw(base + static_cast<int64_t>(v) * N + j));
        return r;
    }
    __device__ __forceinline__ void store_edge(int v, const uint4 &r) const {
        for (int j = 0; j < N; ++j)
            if (has(v, j)) Vec<T>::store(base + static_cast<int64_t>(v) * N + j, Vec<T>::value(r, j));
    }
    // index in the row of element j of vector v
    __device__ __forceinline__ uint32_t index(int v, int j) const {
        return static_cast<uint32_t>(v) * N + j - mis;
    }
};

__device__ __forceinline__ uint4 load_vec(const uint4 *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Vectors v, v + W, ... as far as they are in the row (their number is returned); the
// others read as -inf.
template <int W, int U, typename T>
__device__ __forceinline__ int load_some(const Row<T> &row, int v, uint4 (&r)[U]) {
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool in = v + u * W < row.b1;
        n += in;
        r[u] = in ? load_vec(row.vec(v + u * W))
                  : make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
    }
    return n;
}

// Walks the row's whole vectors with W threads, U in flight per thread: f(r, v, n) gets
// vectors v, v + W, ..., of which the first n are in the row (the others read as -inf).
// n is U, known to the compiler, in all batches of a warp but the last.
template <int W, int U, typename T, typename F>
__device__ __forceinline__ void walk_body(const Row<T> &row, F &&f) {
    const int tid = threadIdx.x;
    int v = row.b0 + tid;
    const int last = row.b1 - 1 - (U - 1) * W - (31 - (tid & 31));
    for (; v <= last; v += U * W) {
        uint4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load_vec(row.vec(v + u * W));
        f(r, v, std::integral_constant<int, U>());
    }
    if (v - (tid & 31) < row.b1) {
        uint4 r[U];
        const int n = load_some<W, U>(row, v, r);
        f(r, v, n);
    }
}

// ------------------------------------------------------------------ the ring
// A row's whole vectors come to the walking warps through a ring of chunks in shared
// memory, filled by bulk copies that one thread issues.  The copies run ahead of the
// walk by the whole ring, into the next row too, so that memory stays busy while the
// block joins its sums, ranks alternatives or finishes a loss.
struct RingCtl {
    uint64_t full[kStages], empty[kStages];
    int abort_flag;
};

// Position in the ring; producer and walkers take the same steps.
struct RingPos {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

template <int W>
__device__ __forceinline__ void ring_init(RingCtl &ctl) {
    for (int i = 0; i < kStages; ++i) {
        mbar_init(&ctl.full[i], 1);
        mbar_init(&ctl.empty[i], W / 32);
    }
    ctl.abort_flag = 0;
    fence_mbarrier_init();
}

template <int W, typename T>
__device__ __forceinline__ int chunks_of(const Row<T> &row) {
    return (row.b1 - row.b0 + kChunk<W> - 1) / kChunk<W>;
}

// One thread: the row's chunks, once; `again`: they will be read a second time, so L2 is
// to keep them, and otherwise to let them go first.  A wait that runs out raises the block's abort
// flag, after which every wait returns at once: the block runs to its end on what the
// ring holds, and the device error word tells.
template <int W, typename T>
__device__ __forceinline__ void ring_fill(const Row<T> &row, uint4 *ring, RingCtl &ctl, RingPos &pos, int *err,
                                          bool again) {
    const int chunks = chunks_of<W>(row);
    uint64_t policy;
    if (again)
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
    else
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    for (int c = 0; c < chunks; ++c, pos.next()) {
        if (!mbar_wait_bounded(&ctl.empty[pos.stage], pos.phase ^ 1u, &ctl.abort_flag, err, kWaitLimitNs)) return;
        const int v = row.b0 + c * kChunk<W>;
        const uint32_t bytes = static_cast<uint32_t>(min(kChunk<W>, row.b1 - v)) * 16u;
        mbar_arrive_expect_tx(&ctl.full[pos.stage], bytes);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                smem_u32(ring + pos.stage * kChunk<W>)),
            "l"(row.vec(v)), "r"(bytes), "r"(smem_u32(&ctl.full[pos.stage])), "l"(policy)
            : "memory");
    }
}

// After an abort: copies still in flight land before the block exits (a fixed 2 ms; their
// barriers may not be asked, since the walkers' phases have come apart).
__device__ __forceinline__ void ring_end(RingCtl &ctl) {
    if (*static_cast<volatile int *>(&ctl.abort_flag)) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
}

// The walkers: f(r, v, n) for each chunk, with vectors v, v + W, ... of which the
// first n are in the row (the others read as -inf); n is kUnroll, known to the compiler,
// in whole chunks.
template <int W, typename T, typename F>
__device__ __forceinline__ void ring_walk(const Row<T> &row, const uint4 *ring, RingCtl &ctl, RingPos &pos, int *err,
                                          F &&f) {
    const int tid = threadIdx.x, chunks = chunks_of<W>(row);
#pragma unroll 1
    for (int c = 0; c < chunks; ++c, pos.next()) {
        (void)mbar_wait_bounded(&ctl.full[pos.stage], pos.phase, &ctl.abort_flag, err, kWaitLimitNs);
        const uint4 *src = ring + pos.stage * kChunk<W> + tid;
        const int v = row.b0 + c * kChunk<W> + tid;
        uint4 r[kUnroll];
        if (row.b0 + (c + 1) * kChunk<W> <= row.b1) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) r[u] = src[u * W];
            f(r, v, std::integral_constant<int, kUnroll>());
        } else {
            int n = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const bool in = v + u * W < row.b1;
                n += in;
                r[u] = in ? src[u * W] : make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
            }
            f(r, v, n);
        }
        // The slot is given back when its reads have been performed: arriving right after
        // the load instructions let the next copy overtake them (a few rows in a
        // thousand had entries of a later chunk in their sums).  The fence orders these
        // generic reads before the copy's writes.
        fence_proxy_async_smem();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(&ctl.empty[pos.stage]);
    }
}

// Barriers of the first P threads of the block (the producer warp takes no part).
template <int P>
__device__ __forceinline__ void bar() {
    asm volatile("bar.sync 1, %0;" ::"n"(P) : "memory");
}
template <int P>
__device__ __forceinline__ bool bar_or(bool x) {
    uint32_t r;
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.ne.u32 p, %1, 0;\n"
        "bar.red.or.pred q, 1, %2, p;\n"
        "selp.u32 %0, 1, 0, q;\n"
        "}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x)), "n"(P)
        : "memory");
    return r != 0;
}

// ------------------------------------------------------------------ running softmax sums

// Where the running maximum starts.
__host__ __device__ __forceinline__ float floor_of(float c) { return -8388608.0f / c; }

// A NaN or +inf entry makes S NaN and stays.
template <bool ENT>
struct Sums {
    float m;
    float mu;  // RN(m c), what y is measured from
    float low;  // 0 times -inf would be NaN in A: entries are raised to here, where 2^y is 0
    uint64_t S = 0, A = 0;  // two partial sums each

    __device__ __forceinline__ explicit Sums(float c) : m(floor_of(c)), mu(m * c), low(4.0f * m) {}

    template <typename T, int U>
    __device__ __forceinline__ float add(const uint4 (&r)[U], float c) {
        const float mx = Vec<T>::max(r);
        if (mx > m) {
            const float mu_new = mx * c, g = fmaxf(mu - mu_new, -1e4f), f = ex2(g);
            const uint64_t f2 = f2_pack(f, f);
            if (ENT) A = f2_mul(f2_fma(S, f2_pack(g, g), A), f2);
            S = f2_mul(S, f2);
            m = mx;
            mu = mu_new;
        }
        const uint64_t nmu = f2_pack(-mu, -mu), c2 = f2_pack(c, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint64_t p[Vec<T>::N / 2];
            Vec<T>::pairs(ENT ? Vec<T>::clamp(r[u], low) : r[u], p);
#pragma unroll
            for (int i = 0; i < Vec<T>::N / 2; ++i) {
                const uint64_t y = f2_fma(p[i], c2, nmu);
                float a, b;
                f2_unpack(y, a, b);
                const uint64_t e = f2_pack(ex2(a), ex2(b));
                S = f2_add(S, e);
                if (ENT) A = f2_fma(e, y, A);
            }
        }
        return mx;
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

// Sums of 2 * HALF lanes, in each of them: the maximum first, then one factor per lane,
// then a butterfly of additions (whose order is the same in every lane of a group).
template <int HALF, bool ENT>
__device__ __forceinline__ RowSums lanes_join(RowSums r, float c) {
    float m = r.m;
#pragma unroll
    for (int off = HALF; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float g = fmaxf((r.m - m) * c, -1e4f), f = ex2(g);
    r.m = m;
    if (ENT) r.A = f * fmaf(r.S, g, r.A);
    r.S *= f;
#pragma unroll
    for (int off = HALF; off > 0; off >>= 1) {
        r.S += __shfl_xor_sync(0xffffffffu, r.S, off);
        if (ENT) r.A += __shfl_xor_sync(0xffffffffu, r.A, off);
    }
    return r;
}

// A warp's sums, in all its lanes.
template <bool ENT>
__device__ __forceinline__ RowSums warp_join(const Sums<ENT> &s, float c) {
    RowSums r;
    float lo, hi;
    r.m = s.m;
    const float off_mu = fmaf(s.m, c, -s.mu);  // y is too large by this
    const float f = ex2(-off_mu);
    f2_unpack(s.S, lo, hi);
    const float S = lo + hi;
    f2_unpack(s.A, lo, hi);
    r.S = S * f;
    r.A = (lo + hi - off_mu * S) * f;
    return lanes_join<16, ENT>(r, c);
}

// The sums of W warps (a power of two of entries, of which the first W count), in every thread.
template <int W, bool ENT>
__device__ __forceinline__ RowSums warps_join(const RowSums *buf, float c) {
    constexpr int P = W <= 8 ? 8 : 32;
    static_assert(W <= 32, "at most thirty-two warps");
    const int i = threadIdx.x & (P - 1);
    RowSums r{-FLT_MAX, 0.0f, 0.0f};
    if (i < W) r = buf[i];
    return lanes_join<P / 2, ENT>(r, c);
}

// The sums of a row whose fast walk gave 0 or no finite sum, with the row's own maximum
// taken off first.  `keep(index)` leaves entries out.  The block's first THREADS threads
// call it; the maximum is that of all of them, so that the
// parts are added without another factor.
template <int THREADS, typename T, typename Keep>
__device__ __noinline__ RowSums far_sums(const Row<T> row, float c, RowSums *buf, Keep keep) {
    constexpr int WARPS = THREADS / 32;
    float m = -INFINITY;
    bool nan = false;
    for (int e = threadIdx.x; e < row.V; e += THREADS)
        if (keep(e)) {
            const float x = Vec<T>::load(row.base + row.mis + e);
            nan = nan || isnan(x);
            m = fmaxf(m, x);
        }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    nan = bar_or<THREADS>(nan);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5].m = m;
    bar<THREADS>();
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, buf[w].m);
    bar<THREADS>();
    RowSums r{fmaxf(m, -FLT_MAX), 0.0f, 0.0f};
    if (nan || m == INFINITY) {
        r.S = NAN;
        return r;
    }
    for (int e = threadIdx.x; e < row.V; e += THREADS)
        if (keep(e)) {
            const float x = Vec<T>::load(row.base + row.mis + e);
            if (x > -INFINITY) {
                const float y = fmaxf((x - r.m) * c, -1e4f), t = ex2(y);
                r.S += t;
                r.A = fmaf(t, y, r.A);
            }
        }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        r.S += __shfl_xor_sync(0xffffffffu, r.S, off);
        r.A += __shfl_xor_sync(0xffffffffu, r.A, off);
    }
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = r;
    bar<THREADS>();
    r.S = r.A = 0.0f;
    for (int w = 0; w < WARPS; ++w) {
        r.S += buf[w].S;
        r.A += buf[w].A;
    }
    bar<THREADS>();
    return r;
}

// No entry above the floor, no finite sum, or a maximum whose m c is rounded by so much
// (32 from 2^30 on) that 2^y of the rounding, and y times it, near the ends of fp32.
__device__ __forceinline__ bool is_far(const RowSums &s, float c) {
    return s.m <= floor_of(c) || !(s.S < INFINITY) || s.m * c >= 0x1p30f;
}

// ------------------------------------------------------------------ log probabilities

// Blocks per SM of the log probabilities' kernels: see launch_logprobs_t.
template <bool TOP, int W>
constexpr int kLogprobCtas = W == kWalkNarrow ? (TOP ? 8 : 12) : W == kWalkWide ? 1 : TOP ? 3 : 4;

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
    int *err;
};

// An order-keeping key of a logit (never NaN here): larger value, larger key; -0 is 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

template <int W>
struct TopShared {
    int vecs[W / 32][kNotes];  // each warp's vectors with an entry that reached the walk's bound
    alignas(16) uint64_t kept[kKept];  // entries that reach the row's last bound: key << 32 | ~index
    uint32_t max_key[W];
    double logS;
    float bound;
    int kept_count, overflow;
    int warp_count[W / 32];
};

// Elements of the row for which pred(key, index) holds, counted over the block.
template <int W, typename T, typename Pred>
__device__ __forceinline__ int64_t block_count(const Row<T> &row, TopShared<W> &sh, Pred pred) {
    int n = 0;
    for (int i = threadIdx.x; i < row.V; i += W) {
        const float x = Vec<T>::load(row.base + row.mis + i);
        n += x > -INFINITY && pred(order_key(x), static_cast<uint32_t>(i));
    }
    n = __reduce_add_sync(0xffffffffu, n);
    bar<W>();
    if ((threadIdx.x & 31) == 0) sh.warp_count[threadIdx.x >> 5] = n;
    bar<W>();
    int64_t total = 0;
    for (int w = 0; w < W / 32; ++w) total += sh.warp_count[w];
    return total;
}

// The k first entries of a row with too many that reach any simple bound (ties): the
// k-th key, then the last index of its ties, are found bit by bit with one walk each,
// and exactly k entries collected.
template <int W, typename T>
__device__ __noinline__ void top_k_by_bits(const Row<T> row, int k, TopShared<W> &sh) {
    uint32_t key = 0;
    for (int b = 31; b >= 0; --b) {
        const uint32_t cand = key | (1u << b);
        if (block_count<W>(row, sh, [=](uint32_t q, uint32_t) { return q >= cand; }) >= k) key = cand;
    }
    const int64_t need = k - block_count<W>(row, sh, [=](uint32_t q, uint32_t) { return q > key; });
    // the largest index bound that still leaves fewer than the needed ties before it
    uint32_t last = 0;
    for (int b = 31; b >= 0; --b) {
        const uint32_t cand = last | (1u << b);
        if (cand <= static_cast<uint32_t>(row.V - 1) &&
            block_count<W>(row, sh, [=](uint32_t q, uint32_t i) { return q == key && i < cand; }) < need)
            last = cand;
    }
    bar<W>();
    if (threadIdx.x == 0) sh.kept_count = 0;
    bar<W>();
    for (int i = threadIdx.x; i < row.V; i += W) {
        const float x = Vec<T>::load(row.base + row.mis + i);
        const uint32_t q = order_key(x), idx = static_cast<uint32_t>(i);
        if (x > -INFINITY && (q > key || (q == key && idx <= last)))
            sh.kept[atomicAdd(&sh.kept_count, 1)] = (static_cast<uint64_t>(q) << 32) | ~idx;
    }
    bar<W>();
}

// The k-th largest of 32 Q keys in shared memory, to its upper 16 bits: a search on the
// counts, two bits a step, over the bits in which the keys differ.  One warp.
template <int Q>
__device__ __forceinline__ uint32_t search_bound(const uint32_t *keys, int k) {
    uint32_t q[Q], lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        q[i] = keys[(threadIdx.x & 31) + 32 * i];
        lo = min(lo, q[i]);
        hi = max(hi, q[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    // two-bit digits at 30, 28, .. 16; above `top` all keys agree
    const int top = (31 - __clz(static_cast<int>((lo ^ hi) | 1u))) & ~1;
    uint32_t t = top < 30 ? hi & ~((4u << top) - 1u) : 0u;
#pragma unroll 1
    for (int b = top; b >= 16; b -= 2) {
        uint32_t n = 0;  // how many reach digits 1, 2 and 3, ten bits each (at most 256 do)
#pragma unroll
        for (int i = 0; i < Q; ++i)
            n += (q[i] >= t + (1u << b) ? 1u : 0u) + (q[i] >= t + (2u << b) ? 1u << 10 : 0u) +
                 (q[i] >= t + (3u << b) ? 1u << 20 : 0u);
        n = __reduce_add_sync(0xffffffffu, n);
        const uint32_t need = static_cast<uint32_t>(k);
        t += ((n >> 20) >= need ? 3u : ((n >> 10) & 1023u) >= need ? 2u : (n & 1023u) >= need ? 1u : 0u) << b;
    }
    return t;
}

// A value that at least k entries walked so far reach (-FLT_MAX while there are fewer):
// the k-th largest of the maxima of the threads, or for small k of groups of 2, 4 or 8 of
// them (at least 4 k groups: with 2 k, k = 64 gave more candidates than they saved),
// found by one warp.  `live`: threads that have entries.
template <int W>
__device__ __forceinline__ float refresh_bound(float thread_max, int k, int live, float floor, TopShared<W> &sh) {
    static_assert(W == 64 || W == 256, "32 Q keys");
    const int tid = threadIdx.x;
    int shift = 0;
    while (((min(live, W) >> (shift + 1)) >= 4 * k) && (W >> (shift + 1)) >= 32) ++shift;
    float g = thread_max;
    for (int i = 0; i < shift; ++i) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1 << i));
    if ((tid & ((1 << shift) - 1)) == 0) sh.max_key[tid >> shift] = order_key(g);
    bar<W>();
    if (tid < 32) {
        const int keys = W >> shift;
        uint32_t t;
        if (W == 256 && keys == 256)
            t = search_bound<8>(sh.max_key, k);
        else if (W == 256 && keys == 128)
            t = search_bound<4>(sh.max_key, k);
        else
            t = keys == 64 ? search_bound<2>(sh.max_key, k) : search_bound<1>(sh.max_key, k);
        // a thread without an entry above the floor says the floor: no bound then
        const float v = key_value(t);
        if (tid == 0) sh.bound = v > floor ? v : -FLT_MAX;
    }
    bar<W>();
    return sh.bound;
}

// Notes vector v of the lanes where `hit`, in the warp's list; n is its length.
template <int W>
__device__ __forceinline__ void note(bool hit, int v, int &n, TopShared<W> &sh) {
    const uint32_t hits = __ballot_sync(0xffffffffu, hit);
    if (hits) {
        const int lane = threadIdx.x & 31, at = n + __popc(hits & ((1u << lane) - 1u));
        if (hit && at < kNotes) sh.vecs[threadIdx.x >> 5][at] = v;
        n += __popc(hits);
    }
}

// Entries of vector v that reach the bound, to the kept ones.
template <int W, typename T>
__device__ __forceinline__ void keep(const Row<T> &row, const uint4 &r, int v, float bound, TopShared<W> &sh) {
    uint32_t hits = 0;
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) hits |= Vec<T>::value(r, j) >= bound ? 1u << j : 0u;  // NaN and -inf never do
    int at = hits ? atomicAdd(&sh.kept_count, __popc(hits)) : 0;
    for (; hits; hits &= hits - 1, ++at) {
        const int j = __ffs(static_cast<int>(hits)) - 1;
        if (at < kKept) sh.kept[at] = (static_cast<uint64_t>(order_key(Vec<T>::value(r, j))) << 32) | ~row.index(v, j);
    }
}

// The walk for the sums, which also notes the vectors that may hold alternatives: those
// with an entry that reaches a bound, refreshed when 1, 4, 16, ... chunks are walked and
// after the last.  For a row in random order these are about 4 k log4(chunks) vectors.
template <int W, typename T>
__device__ __forceinline__ Sums<true> walk_candidates(const Row<T> &row, const LogprobArgs &a, const uint4 *ring,
                                                      RingCtl &ctl, RingPos &pos, TopShared<W> &sh, int &notes) {
    Sums<true> s(a.c);
    if (threadIdx.x == 0) sh.kept_count = sh.overflow = 0;
    notes = 0;
    float bound = -FLT_MAX;
    int ve, done = 0, next = 1;
    const int chunks = chunks_of<W>(row);
    const bool edge = row.edge(ve);
    if (edge) {
        uint4 r[1] = {row.load_edge(ve)};
        s.template add<T, 1>(r, a.c);
    }
    ring_walk<W>(row, ring, ctl, pos, a.err, [&](uint4(&r)[kUnroll], int v, int) {
        const float mx = s.template add<T, kUnroll>(r, a.c);
        if (++done == next) {
            bound = refresh_bound<W>(s.m, a.k, row.b1 - row.b0, floor_of(a.c), sh);
            next = min(4 * next, chunks);
        }
        if (__any_sync(0xffffffffu, mx >= bound)) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) note<W>(Vec<T>::max(r[u]) >= bound, v + u * W, notes, sh);
        }
    });
    if (done == 0) bound = refresh_bound<W>(s.m, a.k, row.b1 - row.b0, floor_of(a.c), sh);  // a row within two vectors
    note<W>(edge, ve, notes, sh);
    if (notes > kNotes) sh.overflow = 1;
    return s;
}

// The k largest (value, lowest index first) of a row without NaN or +inf, from the
// vectors noted in its walk: their entries that reach the row's last bound are ranked by
// counting.
template <int W, typename T>
__device__ __forceinline__ void top_k(const Row<T> &row, const LogprobArgs &a, int64_t t, float m, int notes,
                                      TopShared<W> &sh) {
    const int tid = threadIdx.x, k = a.k;
    const float bound = sh.bound;  // the walk's last; the barrier of the sums ended its notes
    if (sh.overflow) {  // a row that rises along the walk: walked again, by the last bound
        walk_body<W, kUnroll>(row, [&](uint4(&r)[kUnroll], int v, int) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (Vec<T>::max(r[u]) >= bound) keep<W>(row, r[u], v + u * W, bound, sh);
        });
        int ve;
        if (row.edge(ve)) keep<W>(row, row.load_edge(ve), ve, bound, sh);
    } else {
        for (int i = tid & 31; i < notes; i += 32) {
            const int v = sh.vecs[tid >> 5][i];
            keep<W>(row, v >= row.b0 && v < row.b1 ? load_vec(row.vec(v)) : row.load_edge(v), v, bound, sh);
        }
    }
    bar<W>();
    if (sh.kept_count > kKept) top_k_by_bits<W>(row, k, sh);
    const int n = sh.kept_count;
    for (int i = tid; i < n; i += W) {
        const uint64_t mine = sh.kept[i];
        int rank = 0;
        int j = 0;
#pragma unroll 4
        for (; j + 2 <= n; j += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(&sh.kept[j]);
            rank += (o.x > mine) + (o.y > mine);
        }
        if (j < n) rank += sh.kept[j] > mine;
        if (rank < k) {
            a.top_ids[t * k + rank] = static_cast<int64_t>(~static_cast<uint32_t>(mine));
            const float x = key_value(static_cast<uint32_t>(mine >> 32));
            a.top_logprobs[t * k + rank] = static_cast<float>((static_cast<double>(x) - m) * a.inv_tau - sh.logS);
        }
    }
    for (int i = n + tid; i < k; i += W) {
        a.top_ids[t * k + i] = -1;
        a.top_logprobs[t * k + i] = -INFINITY;
    }
}

template <typename T, bool TOP, int W>
__global__ void __launch_bounds__(W + 32, kLogprobCtas<TOP, W>) k_token_logprobs(const LogprobArgs a) {
    extern __shared__ __align__(128) uint4 ring[];
    __shared__ RowSums buf[2][W / 32];  // in turn, so that a row's readers need no barrier before the next row
    __shared__ RingCtl ctl;
    __shared__ typename std::conditional<TOP, TopShared<W>, int>::type sh;
    if (threadIdx.x == 0) ring_init<W>(ctl);
    __syncthreads();
    pdl_wait();
    pdl_allow_dependents();
    RingPos pos;
    auto row_of = [&](int64_t t) {
        return Row<T>(const_cast<T *>(static_cast<const T *>(a.x)) + t * a.ld, static_cast<int>(a.V));
    };
    if (threadIdx.x >= W) {
        if (threadIdx.x == W) {
            for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) ring_fill<W>(row_of(t), ring, ctl, pos, a.err, false);
            ring_end(ctl);
        }
        return;
    }
    int turn = 0;
    // the target comes a row ahead, and its logit while the row is walked
    int64_t id = threadIdx.x == 0 ? a.targets[blockIdx.x] : -1, next_id = -1;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1, id = next_id) {
        const Row<T> row = row_of(t);
        float xt = 0.0f;
        if (id >= 0 && id < a.V) xt = Vec<T>::load(row.base + row.mis + id);
        if (threadIdx.x == 0 && t + gridDim.x < a.T) next_id = a.targets[t + gridDim.x];
        int notes = 0;
        const Sums<true> mine = [&] {
            if constexpr (TOP) {
                return walk_candidates<W>(row, a, ring, ctl, pos, sh, notes);
            } else {
                Sums<true> s(a.c);
                ring_walk<W>(row, ring, ctl, pos, a.err,
                          [&](uint4(&r)[kUnroll], int, int) { s.template add<T, kUnroll>(r, a.c); });
                int v;
                if (row.edge(v)) {
                    uint4 r[1] = {row.load_edge(v)};
                    s.template add<T, 1>(r, a.c);
                }
                return s;
            }
        }();
        const RowSums of_warp = warp_join(mine, a.c);
        if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = of_warp;
        bar<W>();
        RowSums s = warps_join<W / 32, true>(buf[turn], a.c);
        if (is_far(s, a.c)) {
            bar<W>();
            s = far_sums<W>(row, a.c, buf[turn], [](int) { return true; });
        }
        const bool none = s.S == 0.0f, bad = !(s.S < INFINITY);
        if (threadIdx.x < 32) {
            const double logS = log(static_cast<double>(s.S));
            if (threadIdx.x == 0) {
                float lp = 0.0f;
                if (id >= 0) {
                    if (bad || id >= a.V)
                        lp = NAN;
                    else
                        lp = none ? -INFINITY : static_cast<float>((static_cast<double>(xt) - s.m) * a.inv_tau - logS);
                }
                a.logprob[t] = lp;
                // H = -sum p ln p = ln S - ln 2 (A / S)
                a.entropy[t] =
                    none ? 0.0f : static_cast<float>(logS - 0.69314718055994530942 * (static_cast<double>(s.A) / s.S));
                if constexpr (TOP) sh.logS = logS;  // before the barriers of top_k
            }
        }
        if constexpr (TOP) {
            if (bad || none) {
                for (int i = threadIdx.x; i < a.k; i += W) {
                    a.top_ids[t * a.k + i] = -1;
                    a.top_logprobs[t * a.k + i] = bad ? NAN : -INFINITY;
                }
            } else {
                top_k<W>(row, a, t, s.m, notes, sh);
            }
            bar<W>();  // the next row's walk clears the counts
        }
    }
}

// ------------------------------------------------------------------ distillation

struct DistillArgs {
    const void *x;
    int64_t ld, ld_dx, T, V;
    const int64_t *ids;
    const float *tlp;
    int k;
    float c;
    double inv_tau;
    const float *weight;  // nullable: 1
    float *loss;          // nullable
    void *dx;             // nullable; may be x; its rows start as x's do, modulo 16 bytes
    int *err;
};

// A row's slots, and what its teacher and its slots alone say.
struct Slots {
    int id[kTopMax];  // -1: empty
    float x[kTopMax], tl[kTopMax], q[kTopMax];
    bool first[kTopMax];  // the slot that stands for its id where an id is given twice
    float w;              // the row's weight
    RowSums own;          // sums over the slots (each id once)
    double logq0;         // ln q_i = tl_i - logq0
    double qr;            // the teacher's mass outside the slots (TAIL)
    bool dup;             // an id is given twice
    bool bad;             // the row's loss and gradient are NaN, by its teacher
    bool empty;           // no teacher: no loss
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// A row's slots as they come from memory, each lane its own, two rows before they are
// used (asynchronous copies, so that no register waits for them).
struct RawSlots {
    int64_t id[kTopMax];
    float tl[kTopMax];
};
constexpr int kSlotsPerLane = kTopMax / 32;

__device__ __forceinline__ float fetch_slots(const DistillArgs &a, int64_t t, RawSlots &raw) {
    const int lane = threadIdx.x & 31;
    if (t >= a.T) return 0.0f;
    for (int j = lane; j < a.k; j += 32) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(&raw.id[j])), "l"(a.ids + t * a.k + j)
                     : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&raw.tl[j])), "l"(a.tlp + t * a.k + j)
                     : "memory");
    }
    return a.weight ? a.weight[t] : 1.0f;  // 0 for no row: nothing of it is read
}

// The logits at a row's slots, asked for a row before they are used.
template <typename T>
__device__ __forceinline__ void gather_slots(const DistillArgs &a, int64_t t, const RawSlots &raw, float w,
                                             float (&x)[kSlotsPerLane]) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    const T *p = static_cast<const T *>(a.x) + t * a.ld;
#pragma unroll
    for (int i = 0; i < kSlotsPerLane; ++i) {
        const int j = (threadIdx.x & 31) + 32 * i;
        const int64_t id = j < a.k && w != 0.0f ? raw.id[j] : -1;
        x[i] = id >= 0 && id < a.V ? Vec<T>::load(p + id) : -INFINITY;
    }
}

// One warp: a row's slots, marked in the bitmap, and the teacher's side of the loss.
template <typename T, bool TAIL>
__device__ void prepare_slots(const DistillArgs &a, int64_t t, const RawSlots &raw, float w,
                              const float (&x)[kSlotsPerLane], Slots &sl, uint32_t *bitmap) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) sl.w = w;
    if (w == 0.0f) return;  // nothing of the row is read
    const T *p = static_cast<const T *>(a.x) + t * a.ld;
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
    constexpr int PER = kSlotsPerLane;
    int id[PER];
    float tl[PER];
    bool first[PER], bad = false, twice = false, any = false;
    float tm = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = lane + 32 * i;
        const int64_t g = j < a.k ? raw.id[j] : -1;
        tl[i] = j < a.k ? raw.tl[j] : -INFINITY;
        bad = bad || g >= a.V;
        id[i] = g < 0 || g >= a.V ? -1 : static_cast<int>(g);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        first[i] = false;
        if (id[i] >= 0) {
            const uint32_t bit = 1u << ((id[i] + mis) & 31);
            first[i] = !(atomicOr(&bitmap[(id[i] + mis) >> 5], bit) & bit);
            twice = twice || !first[i];
            tm = fmaxf(tm, tl[i]);
            any = any || tl[i] > -INFINITY;
            bad = bad || isnan(tl[i]);
        }
    }
    RowSums own{-FLT_MAX, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < PER; ++i) own.m = fmaxf(own.m, first[i] ? x[i] : -FLT_MAX);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, off));
        own.m = fmaxf(own.m, __shfl_xor_sync(0xffffffffu, own.m, off));
    }
    any = __any_sync(0xffffffffu, any);
    // The masses.  What they leave of 1 (TAIL) keeps its relative accuracy only if they
    // are exact beyond fp32; renormalised, expf (within 2 ulp) does.
    const float shift = TAIL || !any ? 0.0f : tm;
    float e[PER];
    double qsum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        e[i] = 0.0f;
        if (32 * i < a.k) {  // the same in all lanes
            const float l = id[i] >= 0 ? tl[i] : -INFINITY;
            const double d = TAIL ? exp(static_cast<double>(l)) : static_cast<double>(expf(l - shift));
            e[i] = static_cast<float>(d);
            qsum += d;
        }
        own.S += first[i] ? ex2((x[i] - own.m) * a.c) : 0.0f;
    }
    qsum = warp_sum(qsum);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) own.S += __shfl_xor_sync(0xffffffffu, own.S, off);
    bad = bad || !(qsum < INFINITY);
    bad = __any_sync(0xffffffffu, bad);
    twice = __any_sync(0xffffffffu, twice);
    const float inv = TAIL ? 1.0f : static_cast<float>(1.0 / qsum);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = lane + 32 * i;
        sl.id[j] = id[i];
        sl.x[j] = x[i];
        sl.tl[j] = tl[i];
        sl.first[j] = first[i];
        sl.q[j] = e[i] * inv;
    }
    if (lane == 0) {
        sl.own = own;
        sl.logq0 = TAIL ? 0.0 : shift + log(qsum);
        sl.qr = TAIL ? fmax(1.0 - qsum, 0.0) : 0.0;
        sl.dup = twice;
        sl.bad = bad;
        sl.empty = !TAIL && !any;
    }
    __syncwarp();
}

// What the walked sums `s` (over the row, or with TAIL over the entries outside the
// slots) make of a row: all its sums, whether it has a loss, and the gradient's factor.
//   L = sum_i q_i (ln q_i - ln p_i)  [+ q_r (ln q_r - ln p_r)],  p = softmax(x / temperature)
//   dL/dz_j = p_j - q_j on a slot, p_j [(1 - q_r / p_r)] elsewhere.
// p_r comes from a sum of its own and not from 1 minus the slots' masses, which would
// cancel when nearly all mass is on the slots.
struct RowState {
    RowSums all;
    bool zero, nan, live;
    float coef;  // dx = coef 2^((x - s.m) c) outside the slots
};

template <bool TAIL>
__device__ __forceinline__ RowState row_state(const DistillArgs &a, const Slots &sl, const RowSums &s) {
    RowState r;
    r.all = TAIL ? join(s, sl.own, a.c) : s;
    r.nan = sl.bad || !(r.all.S >= 0.0f);
    r.zero = !r.nan && (sl.empty || r.all.S == 0.0f);
    r.live = TAIL && sl.qr > 0.0 && s.S > 0.0f;
    const float F = ex2(fmaxf((s.m - r.all.m) * a.c, -1e4f));
    float coef = F / r.all.S;
    if (r.live) coef -= static_cast<float>(sl.qr) / s.S;
    r.coef = r.nan ? NAN : sl.w * static_cast<float>(a.inv_tau) * coef;
    return r;
}

// One warp: the loss of a row, and the gradient at its slots (in sl.x).
template <bool TAIL>
__device__ void finish_slots(const DistillArgs &a, Slots &sl, const RowSums &s, const RowState &r, int64_t t) {
    const int lane = threadIdx.x & 31, k = a.k;
    // ln S, and q_r ln (q_r / p_r) of the masses outside the slots
    const double lnS = log(static_cast<double>(r.all.S));
    const double rest = r.live ? sl.qr * (log(sl.qr * r.all.S / s.S) - (static_cast<double>(s.m) - r.all.m) * a.inv_tau)
                               : 0.0;
    const float up = sl.w * static_cast<float>(a.inv_tau), inv_S = 1.0f / r.all.S;
    double L = 0.0;
#pragma unroll
    for (int i = 0; i < kTopMax / 32; ++i) {
        const int j = lane + 32 * i;
        float q = sl.q[j];
        const float x = sl.x[j], y = x - r.all.m;
        const bool use = sl.id[j] >= 0;
        if (use && q > 0.0f)
            L += static_cast<double>(q) * (static_cast<double>(sl.tl[j]) - sl.logq0 -
                                           ((static_cast<double>(x) - r.all.m) * a.inv_tau - lnS));
        if (use && sl.first[j]) {
            if (sl.dup) {  // an id given more than once carries its slots' masses together
                q = 0.0f;
                for (int m = 0; m < k; ++m)
                    if (sl.id[m] == sl.id[j]) q += sl.q[m];
            }
            sl.x[j] = r.nan ? NAN : up * (ex2(y * a.c) * inv_S - q);
        }
    }
    L = warp_sum(L) + rest;
    if (lane == 0 && a.loss) a.loss[t] = r.zero ? 0.0f : r.nan ? NAN : static_cast<float>(sl.w * L);
    __syncwarp();
}

template <int W, typename T>
__device__ __forceinline__ void zero_row(const Row<T> &out) {
    for (int v = out.b0 + threadIdx.x; v < out.b1; v += W)
        *const_cast<uint4 *>(out.vec(v)) = make_uint4(0, 0, 0, 0);
    int v;
    if (out.edge(v)) out.store_edge(v, make_uint4(0, 0, 0, 0));
}

// The first W threads walk; the next warp looks after the slots: while the others walk a row for its
// sums it prepares the next row's, and while they walk it again for the gradient it works
// out the loss and the gradient at the slots, which it writes when they have passed.
// The last warp fills the ring.
template <typename T, bool TAIL, int W>
__global__ void __launch_bounds__(W + 64, kCtasPerSm<W>) k_distill(const DistillArgs a) {
    extern __shared__ __align__(128) uint4 ring[];
    // two rows': a bit per element of the row's vectors, set on slots
    uint32_t *bitmaps = reinterpret_cast<uint32_t *>(ring + kStages * kChunk<W>);
    constexpr int P = W + 32;  // walkers and slot warp
    __shared__ RowSums buf[2][P / 32];
    __shared__ Slots slots[2];
    __shared__ RawSlots raw[2];  // of odd and even rows
    __shared__ RingCtl ctl;
    const int tid = threadIdx.x;
    const bool walker = tid < W;
    const int words = static_cast<int>((a.V + Vec<T>::N + 31) / 32);
    for (int i = tid; i < 2 * words; i += W + 64) bitmaps[i] = 0;
    if (tid == 0) ring_init<W>(ctl);
    __syncthreads();
    pdl_wait();
    pdl_allow_dependents();
    RingPos pos;
    auto row_of = [&](const void *x, int64_t ld, int64_t t) {
        return Row<T>(const_cast<T *>(static_cast<const T *>(x)) + t * ld, static_cast<int>(a.V));
    };
    if (tid >= P) {
        if (tid == P) {
            for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
                if (a.weight && a.weight[t] == 0.0f) continue;
                ring_fill<W>(row_of(a.x, a.ld, t), ring, ctl, pos, a.err, a.dx != nullptr);
                if (a.dx) ring_fill<W>(row_of(a.x, a.ld, t), ring, ctl, pos, a.err, false);
            }
            ring_end(ctl);
        }
        return;
    }
    int turn = 0;
    // the slot warp: logits at the next row's slots, its weight, and that of the row after it
    float xs[kSlotsPerLane], w_next = 0.0f, w_ahead = 0.0f;
    const int64_t step = gridDim.x;
    if (!walker) {
        const float w0 = fetch_slots(a, blockIdx.x, raw[0]);
        gather_slots<T>(a, blockIdx.x, raw[0], w0, xs);
        w_next = fetch_slots(a, blockIdx.x + step, raw[1]);
        prepare_slots<T, TAIL>(a, blockIdx.x, raw[0], w0, xs, slots[0], bitmaps);
        gather_slots<T>(a, blockIdx.x + step, raw[1], w_next, xs);
        w_ahead = fetch_slots(a, blockIdx.x + 2 * step, raw[0]);
    }
    bar<P>();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        Slots &sl = slots[turn];
        uint32_t *bitmap = bitmaps + turn * words;
        const Row<T> row = row_of(a.x, a.ld, t);
        const Row<T> out = a.dx ? row_of(a.dx, a.ld_dx, t) : row;  // same phase as the row
        const float w = sl.w;
        const bool skip = w == 0.0f;  // a token without a loss: nothing of its row is read
        if (walker && !skip) {
            Sums<false> mine(a.c);
            // slots are left out of the sums (a vector's bits are a byte of the bitmap, or half
            // of one)
            const uint8_t *bytes = reinterpret_cast<const uint8_t *>(bitmap);
            auto mask = [&](uint4 &r, int v) {
                uint32_t bits = bytes[static_cast<uint32_t>(v) * Vec<T>::N / 8];
                if (Vec<T>::N == 4) bits = (v & 1) ? bits >> 4 : bits & 15u;
                if (bits) Vec<T>::fill(r, bits);
            };
            ring_walk<W>(row, ring, ctl, pos, a.err, [&](uint4(&r)[kUnroll], int v, int n) {
                if (TAIL) {
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        if (u < n) mask(r[u], v + u * W);
                }
                mine.template add<T, kUnroll>(r, a.c);
            });
            int ve;
            if (row.edge(ve)) {
                uint4 r[1] = {row.load_edge(ve)};
                if (TAIL) mask(r[0], ve);
                mine.template add<T, 1>(r, a.c);
            }
            const RowSums mine_w = warp_join(mine, a.c);
            if ((tid & 31) == 0) buf[turn][tid >> 5] = mine_w;
        } else if (!walker && t + step < a.T) {
            prepare_slots<T, TAIL>(a, t + step, raw[turn ^ 1], w_next, xs, slots[turn ^ 1], bitmaps + (turn ^ 1) * words);
            gather_slots<T>(a, t + 2 * step, raw[turn], w_ahead, xs);
            w_next = w_ahead;
            w_ahead = fetch_slots(a, t + 3 * step, raw[turn ^ 1]);
        }
        bar<P>();
        RowSums s;
        RowState st;
        if (!skip) {
            s = warps_join<W / 32, false>(buf[turn], a.c);
            if (is_far(s, a.c)) {
                bar<P>();
                s = far_sums<P>(row, a.c, buf[turn], [&](int e) {
                    const int at = e + row.mis;
                    return !TAIL || !((bitmap[at >> 5] >> (at & 31)) & 1u);
                });
            }
            // without a gradient the walkers are done with the row: no barrier keeps its
            // slots from the row after next
            if (a.dx || !walker) st = row_state<TAIL>(a, sl, s);
        }
        if (walker) {
            if (a.dx) {
                if (skip) {
                    zero_row<W>(out);
                } else {
                    const uint64_t nm = f2_pack(-s.m, -s.m), c2 = f2_pack(a.c, a.c), k2 = f2_pack(st.coef, st.coef);
                    auto grad = [&](const uint4 &r) {
                        uint64_t e[Vec<T>::N / 2];
                        Vec<T>::pairs(r, e);
#pragma unroll
                        for (int i = 0; i < Vec<T>::N / 2; ++i) {
                            float lo, hi;
                            f2_unpack(f2_mul(f2_add(e[i], nm), c2), lo, hi);
                            e[i] = f2_mul(f2_pack(ex2(lo), ex2(hi)), k2);
                        }
                        return Vec<T>::from_pairs(e);
                    };
                    const bool zero = st.zero;
                    ring_walk<W>(row, ring, ctl, pos, a.err, [&](uint4(&r)[kUnroll], int v, int n) {
#pragma unroll
                        for (int u = 0; u < kUnroll; ++u)
                            if (u < n)
                                __stcs(const_cast<uint4 *>(out.vec(v + u * W)),
                                       zero ? make_uint4(0, 0, 0, 0) : grad(r[u]));
                    });
                    int ve;
                    if (row.edge(ve)) out.store_edge(ve, zero ? make_uint4(0, 0, 0, 0) : grad(row.load_edge(ve)));
                }
            }
        } else if (skip) {
            if (tid == W && a.loss) a.loss[t] = 0.0f;
        } else {
            finish_slots<TAIL>(a, sl, s, st, t);
        }
        if (a.dx) bar<P>();  // the walkers' stores of the row are done
        if (!walker && !skip) {
            for (int i = tid & 31; i < a.k; i += 32)
                if (sl.id[i] >= 0) {
                    if (a.dx && !st.zero && sl.first[i]) Vec<T>::store(out.base + out.mis + sl.id[i], sl.x[i]);
                    bitmap[(sl.id[i] + row.mis) >> 5] = 0;
                }
            __syncwarp();
        }
    }
}

// Shared memory beyond the default of a kernel: set once per device (setting it twice
// from racing threads is harmless).
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t> &done, const DeviceInfo &dev) {
    const uint64_t bit = 1ull << (dev.device & 63);
    if (done.load() & bit) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

template <typename T, bool TOP, int W>
cudaError_t launch_logprobs_w(const LogprobArgs &a, int per_sm, const DeviceInfo &dev, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    auto kern = k_token_logprobs<T, TOP, W>;
    // fewer blocks per SM than fit are kept apart by shared memory (a smaller grid alone
    // would fill some SMs and leave others)
    constexpr size_t kApart = 72 * 1024;
    const size_t smem = per_sm < kLogprobCtas<TOP, W> ? kApart : kRingBytes<W>;
    cudaError_t e = allow_smem(kern, std::max(kRingBytes<W>, kApart), done, dev);
    if (e != cudaSuccess) return e;
    const int grid = static_cast<int>(std::min<int64_t>(a.T, static_cast<int64_t>(dev.sm_count) * per_sm));
    return launch_pdl(kern, dim3(grid), dim3(W + 32), smem, st, a);
}

// Rows for the wide block: no more than SMs, and long (see kWalkWide).
inline bool few_long_rows(int64_t T, int64_t row_bytes, const DeviceInfo &dev) {
    return T <= dev.sm_count && row_bytes >= 128 * 1024;
}

// Rows for the narrow block: short ones beyond the SMs, longer ones beyond the blocks of
// kWalk (see kWalkNarrow).
inline bool many_short_rows(int64_t T, int64_t row_bytes, const DeviceInfo &dev) {
    return row_bytes <= kNarrowBytes && T > (row_bytes <= 8 * 1024 ? 1 : 3) * static_cast<int64_t>(dev.sm_count);
}

template <typename T>
cudaError_t launch_logprobs_t(const LogprobArgs &a, const DeviceInfo &dev, cudaStream_t st) {
    const int64_t row_bytes = a.V * static_cast<int64_t>(sizeof(T));
    const bool narrow = many_short_rows(a.T, row_bytes, dev);
    if (a.k > 0) {
        // the narrow block has 64 maxima to take a bound from
        return narrow && a.k <= 32 ? launch_logprobs_w<T, true, kWalkNarrow>(a, kLogprobCtas<true, kWalkNarrow>, dev, st)
                                   : launch_logprobs_w<T, true, kWalk>(a, kLogprobCtas<true, kWalk>, dev, st);
    }
    if (few_long_rows(a.T, row_bytes, dev)) return launch_logprobs_w<T, false, kWalkWide>(a, 1, dev, st);
    if (narrow)
        return launch_logprobs_w<T, false, kWalkNarrow>(a, kLogprobCtas<false, kWalkNarrow>, dev, st);
    // Four blocks per SM on short rows (2048 x 32000 bf16: 29.6 us against 32.2 with three),
    // three on long ones (1024 x 131072: 49.9 against 52.6).
    return launch_logprobs_w<T, false, kWalk>(a, row_bytes <= 96 * 1024 ? 4 : 3, dev, st);
}

template <typename T, bool TAIL, int W>
cudaError_t launch_distill_w(const DistillArgs &a, const DeviceInfo &dev, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    auto kern = k_distill<T, TAIL, W>;
    // two bits per vocabulary entry: the wide block's ring leaves room for fewer entries
    const size_t bits = static_cast<size_t>((a.V + Vec<T>::N + 31) / 32) * 8;
    constexpr size_t most = W == kWalk       ? static_cast<size_t>((kDistillMaxV + 64) / 4)
                            : W == kWalkWide ? kWideBitBytes
                                             : static_cast<size_t>(kNarrowBytes);
    cudaError_t e = allow_smem(kern, kRingBytes<W> + most, done, dev);
    if (e != cudaSuccess) return e;
    // The rows that are walked twice at a time have to stay in the 126 MB L2 beside what
    // is written: 2048 rows of 131072 bf16 take 222 us with two blocks per SM, 258 us with
    // three and 296 us with one (in one run, on one box).
    const int64_t row_bytes = a.V * static_cast<int64_t>(sizeof(T)) * dev.sm_count;
    const int64_t per_sm =
        std::max<int64_t>(1, std::min<int64_t>(kCtasPerSm<W>, (80ll << 20) / std::max<int64_t>(row_bytes, 1)));
    const int grid = static_cast<int>(std::min<int64_t>(a.T, dev.sm_count * per_sm));
    return launch_pdl(kern, dim3(grid), dim3(W + 64), kRingBytes<W> + bits, st, a);
}

template <typename T, bool TAIL>
cudaError_t launch_distill_t(const DistillArgs &a, const DeviceInfo &dev, cudaStream_t st) {
    const size_t bits = static_cast<size_t>((a.V + Vec<T>::N + 31) / 32) * 8;
    const int64_t row_bytes = a.V * static_cast<int64_t>(sizeof(T));
    if (many_short_rows(a.T, row_bytes, dev)) return launch_distill_w<T, TAIL, kWalkNarrow>(a, dev, st);
    const bool wide = few_long_rows(a.T, row_bytes, dev) && bits <= kWideBitBytes;
    return wide ? launch_distill_w<T, TAIL, kWalkWide>(a, dev, st) : launch_distill_w<T, TAIL, kWalk>(a, dev, st);
}

}  // namespace

cudaError_t launch_token_logprobs(const void *x, bool f32, int64_t ld, int64_t T, int64_t V, const int64_t *targets,
                                  double temperature, int k, float *logprob, float *entropy, int64_t *top_ids,
                                  float *top_logprobs, const DeviceInfo &dev, cudaStream_t st) {
    LogprobArgs a{x, ld, T, V, targets, static_cast<float>(1.44269504088896340736 / temperature), 1.0 / temperature,
                  k, logprob, entropy, top_ids, top_logprobs, device_error_word()};
    if (!a.err) return cudaErrorInvalidSymbol;
    return f32 ? launch_logprobs_t<float>(a, dev, st) : launch_logprobs_t<__nv_bfloat16>(a, dev, st);
}

cudaError_t launch_distill_topk(const void *x, bool f32, int64_t ld, int64_t T, int64_t V, const int64_t *ids,
                                const float *tlp, int k, double temperature, bool tail, const float *weight,
                                float *loss, void *dx, int64_t ld_dx, const DeviceInfo &dev, cudaStream_t st) {
    const DistillArgs a{x, ld, ld_dx, T, V, ids, tlp, k, static_cast<float>(1.44269504088896340736 / temperature),
                        1.0 / temperature, weight, loss, dx, device_error_word()};
    if (!a.err) return cudaErrorInvalidSymbol;
    if (f32) return tail ? launch_distill_t<float, true>(a, dev, st) : launch_distill_t<float, false>(a, dev, st);
    return tail ? launch_distill_t<__nv_bfloat16, true>(a, dev, st) : launch_distill_t<__nv_bfloat16, false>(a, dev, st);
}

}  // namespace eqat
