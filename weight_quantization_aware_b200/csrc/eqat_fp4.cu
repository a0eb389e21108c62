// Microscaled 4-bit floats: packing, fake quantization, reading back and the tensor scale
// (the formats and their element arithmetic are in eqat_fp4.cuh).
//
// Every kernel here is meant to be HBM-bound: a thread takes 16 values (two 16-byte loads
// of bf16), a warp 512 consecutive values of a row, the next of which are on their way
// while one is encoded.  Measured on 28672 x 8192 bf16 (a copy runs at 6.55 TB/s): tensor
// scale 75 us (6.3 TB/s), pack mx 100 us (5.9) and nv 136 us (4.4), fake quantization mx 164
// and nv 168 us (5.7, 5.6), values from codes 111 us (5.4).  nv packing is bound by its
// instructions, those of the exact division by the block's scale and those that put signs
// back: 67% of the cycles issue, the integer and logic pipe is 62% busy, and of 8 cycles that a
// warp spends on an instruction 0.8 wait for memory (mx: 63%, 66%, 5.3 of 11.7).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "eqat_fp4.cuh"
#include "eqat_internal.h"
#include "eqat_pdl.cuh"
#include "eqat_qmath.cuh"

namespace eqat {
namespace {

using namespace fp4;

constexpr int kThreads = 256;

struct PackArgs {
    const void *x;
    const float *g;  // tensor scale (nv)
    uint8_t *codes, *scales;
    void *values;
    int64_t N, K;
    int64_t rows;     // rows to walk: N, or N rounded up to 128 when scales are written
    int64_t segs;     // 512-value segments of a row, padded blocks included
    int64_t tiles_k;  // scale tiles along a row
};

// Walks the 512-value segments of rows, one warp each, without a division per segment.
struct Segments {
    int64_t row, drow;
    int seg, dseg, segs;
    __device__ __forceinline__ Segments(int64_t segs_) : segs(static_cast<int>(segs_)) {
        const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
        const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * kThreads) >> 5;
        row = warp / segs_;
        seg = static_cast<int>(warp - row * segs_);
        drow = nwarps / segs_;
        dseg = static_cast<int>(nwarps - drow * segs_);
    }
    __device__ __forceinline__ void next() {
        row += drow;
        seg += dseg;
        if (seg >= segs) {
            seg -= segs;
            ++row;
        }
    }
};

// CODES: codes and scale tiles (whose padding, rows past N and blocks past K / block, is
// written as zero); otherwise the values that the codes stand for, rounded to T (V8: they
// are 32-byte aligned).
template <typename T, bool NV, bool CODES, bool V8>
__global__ void __launch_bounds__(kThreads, NV ? 3 : 4) k_encode_fp4(const PackArgs a) {
    pdl_wait();
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31;
    const float g = NV && a.g ? __ldg(a.g) : 1.0f;
    const float inv_g = __fdiv_rn(1.0f, g);
    // the next segment is on its way while one is encoded
    auto fetch = [&](const Segments &u) {
        Raw16<T> r = zero16<T>();
        const int64_t k0 = static_cast<int64_t>(u.seg) * 512 + lane * 16;
        if (u.row < a.N && k0 < a.K) r = load_raw16(static_cast<const T *>(a.x) + u.row * a.K + k0);
        return r;
    };
    Segments u(a.segs);
    Raw16<T> ahead = fetch(u);
    while (u.row < a.rows) {
        const int64_t row = u.row, k0 = static_cast<int64_t>(u.seg) * 512 + lane * 16;
        const bool in = row < a.N && k0 < a.K;
        float x[16];
        unpack16(ahead, x);
        u.next();
        ahead = fetch(u);
        Coded c = encode<NV>(x, g, inv_g);
        if (!in) c.scale = 0;
        if (CODES) {
            if (in) *reinterpret_cast<uint2 *>(a.codes + (row * a.K + k0) / 2) = make_uint2(c.lo, c.hi);
            // four blocks of a row are one aligned word of a scale tile
            constexpr int per = NV ? 1 : 2;  // threads per block
            uint32_t w = c.scale << (8 * ((lane / per) & 3));
#pragma unroll
            for (int off = per; off < 4 * per; off *= 2) w |= __shfl_xor_sync(0xffffffffu, w, off);
            const int64_t block = k0 / (NV ? 16 : 32);
            if (lane % (4 * per) == 0 && block / 4 < a.tiles_k)
                *reinterpret_cast<uint32_t *>(a.scales + scale_at(row, block, a.tiles_k)) = w;
        }
        if (!CODES && in) store_decoded<V8>(static_cast<T *>(a.values) + row * a.K + k0, c.lo, c.hi, c.value);
    }
}

template <typename T, bool NV, bool V8>
__global__ void __launch_bounds__(kThreads) k_dequant_fp4(const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, const float *g_ptr,
                                                          T *__restrict__ out, int64_t N, int64_t K, int64_t segs,
                                                          int64_t tiles_k) {
    pdl_wait();
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31;
    const float g = NV && g_ptr ? __ldg(g_ptr) : 1.0f;
    for (Segments u(segs); u.row < N; u.next()) {
        const int64_t k0 = static_cast<int64_t>(u.seg) * 512 + lane * 16;
        if (k0 >= K) continue;
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes + (u.row * K + k0) / 2));
        const uint32_t b = __ldg(scales + scale_at(u.row, k0 / (NV ? 16 : 32), tiles_k));
        store_decoded<V8>(out + u.row * K + k0, c.x, c.y, NV ? __fmul_rn(e4m3_value(b), g) : e8m0_value(b));
    }
}

// The smallest power of two g with |x| <= 6 * 448 * g, within 2^-100 .. 2^100.
// 6 * 448 = 1.3125 * 2^11.
__device__ __forceinline__ float scale_of_amax(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 11 + ((u & 0x7FFFFFu) > 0x280000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(-100, min(100, e)) + 127) << 23);
}

// amax -> g is monotone, so the largest of the blocks' g is the tensor's: an atomic
// maximum on the bits of positive floats, whose result does not depend on the order.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_tensor_scale_fp4(const T *__restrict__ x, int64_t n16, uint32_t *out) {
    __shared__ float red[kThreads / 32];
    float amax = 0.0f;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n16;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        float v[16];
        load16<T>(x + i * 16, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float m = fabsf(v[j]);
            amax = m <= FLT_MAX ? fmaxf(amax, m) : amax;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) amax = fmaxf(amax, red[w]);
        atomicMax(out, __float_as_uint(scale_of_amax(amax)));
    }
}

inline bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int grid_of(int64_t warps, const DeviceInfo &dev) {
    return static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(cdiv(warps, kThreads / 32), static_cast<int64_t>(dev.sm_count) * 8)));
}

template <typename T, bool NV>
cudaError_t encode_t(const PackArgs &a, const DeviceInfo &dev, cudaStream_t st) {
    const dim3 grid(grid_of(a.rows * a.segs, dev)), block(kThreads);
    if (a.codes) return launch_pdl(k_encode_fp4<T, NV, true, false>, grid, block, 0, st, a);
    return aligned32(a.values) ? launch_pdl(k_encode_fp4<T, NV, false, true>, grid, block, 0, st, a)
                               : launch_pdl(k_encode_fp4<T, NV, false, false>, grid, block, 0, st, a);
}

}  // namespace

cudaError_t launch_encode_fp4(const void *x, bool f32, bool nv, const float *g, int64_t N, int64_t K, uint8_t *codes,
                              uint8_t *scales, void *values, const DeviceInfo &dev, cudaStream_t st) {
    PackArgs a{};
    a.x = x;
    a.g = g;
    a.codes = codes;
    a.scales = scales;
    a.values = values;
    a.N = N;
    a.K = K;
    a.tiles_k = cdiv(K / (nv ? 16 : 32), 4);
    a.rows = codes ? cdiv(N, 128) * 128 : N;
    a.segs = cdiv(a.tiles_k * 4 * (nv ? 16 : 32), 512);
    if (f32) return nv ? encode_t<float, true>(a, dev, st) : encode_t<float, false>(a, dev, st);
    return nv ? encode_t<__nv_bfloat16, true>(a, dev, st) : encode_t<__nv_bfloat16, false>(a, dev, st);
}

cudaError_t launch_dequant_fp4(const uint8_t *codes, const uint8_t *scales, bool nv, const float *g, int64_t N,
                               int64_t K, void *out, bool f32, const DeviceInfo &dev, cudaStream_t st) {
    const int64_t segs = cdiv(K, 512), tiles_k = cdiv(K / (nv ? 16 : 32), 4);
    const dim3 grid(grid_of(N * segs, dev)), block(kThreads);
    auto go = [&](auto kern, auto *o) { return launch_pdl(kern, grid, block, 0, st, codes, scales, g, o, N, K, segs, tiles_k); };
    const bool v8 = aligned32(out);
    if (f32) {
        float *o = static_cast<float *>(out);
        if (nv) return v8 ? go(k_dequant_fp4<float, true, true>, o) : go(k_dequant_fp4<float, true, false>, o);
        return v8 ? go(k_dequant_fp4<float, false, true>, o) : go(k_dequant_fp4<float, false, false>, o);
    }
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out);
    if (nv) return v8 ? go(k_dequant_fp4<__nv_bfloat16, true, true>, o) : go(k_dequant_fp4<__nv_bfloat16, true, false>, o);
    return v8 ? go(k_dequant_fp4<__nv_bfloat16, false, true>, o) : go(k_dequant_fp4<__nv_bfloat16, false, false>, o);
}

cudaError_t launch_tensor_scale_fp4(const void *x, bool f32, int64_t n, float *out, const DeviceInfo &dev,
                                    cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(out, 0, sizeof(float), st);
    if (e != cudaSuccess) return e;
    const int64_t n16 = n / 16;
    const int grid = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(cdiv(n16, kThreads), static_cast<int64_t>(dev.sm_count) * 8)));
    uint32_t *o = reinterpret_cast<uint32_t *>(out);
    if (f32)
        k_tensor_scale_fp4<float><<<grid, kThreads, 0, st>>>(static_cast<const float *>(x), n16, o);
    else
        k_tensor_scale_fp4<__nv_bfloat16><<<grid, kThreads, 0, st>>>(static_cast<const __nv_bfloat16 *>(x), n16, o);
    return cudaGetLastError();
}

}  // namespace eqat
