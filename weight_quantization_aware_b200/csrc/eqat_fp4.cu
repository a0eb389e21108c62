// Microscaled 4-bit floats: blocks of consecutive in-features of a row share one 8-bit
// scale, and each value is an e2m1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign).
//
//   mx: blocks of 32, scale 2^e as an e8m0 byte (e + 127), e = floor(log2 amax) - 2
//       (at least -127); code = RNE_e2m1(x 2^-e), 6 where that would be above 6.
//   nv: blocks of 16, scale s in e4m3 over a scale g of the whole tensor:
//       x' = x (1/g),  s = RNE_e4m3(min(amax' / 6, 448)),  code = RNE_e2m1(x' / s).
//       With g a power of two (as the tensor-scale kernel gives) x' is exact, so every
//       decision is that of exact arithmetic.
//
// A block that holds a NaN or an infinity gets a NaN scale and zero codes; it reads
// back, and multiplies, as NaN.
//
// Kernels here are HBM-bound: a thread takes 16 values (two 16-byte loads of bf16), a
// warp 512 consecutive values of a row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "eqat_internal.h"
#include "eqat_pdl.cuh"
#include "eqat_qmath.cuh"

namespace eqat {
namespace {

constexpr int kThreads = 256;

// Two values -> two codes in a byte (the first in the low half): round to nearest even
// on the e2m1 grid, saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n"
        ".reg .b8 b;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n"
        "cvt.u32.u8 %0, b;\n"
        "}\n"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// x -> e4m3 byte, round to nearest even, 448 beyond it (x >= 0, not NaN).
__device__ __forceinline__ uint32_t e4m3(float x) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
    return r & 0xFFu;
}

__device__ __forceinline__ float e4m3_value(uint32_t b) {
    const uint32_t e = (b >> 3) & 15u, m = b & 7u;
    if ((b & 0x7Fu) == 0x7Fu) return NAN;
    return e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0x1p-9f;
}

__device__ __forceinline__ float e8m0_value(uint32_t b) {
    if (b == 0xFFu) return NAN;
    return b ? __uint_as_float(b << 23) : 0x1p-127f;
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    // bf16 images of 0, .5, 1, 1.5, 2, 3, 4, 6, one byte each (the low bytes are 0x00,
    // 0x80 or 0xC0): looked up in two registers
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, c & 7u) & 0xFFu;
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, c & 7u) & 0xFFu;
    return __uint_as_float(((c & 8u) << 28) | (hi << 24) | (lo << 16));
}

// 16 consecutive values of a row.
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[16]) {
    const Raw8<__nv_bfloat16> a = load_raw8(p), b = load_raw8(p + 8);
    float u[8], v[8];
    unpack8(a, u);
    unpack8(b, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] = u[j];
        x[8 + j] = v[j];
    }
}
template <>
__device__ __forceinline__ void load16<float>(const float *p, float (&x)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + q);
        x[4 * q] = v.x;
        x[4 * q + 1] = v.y;
        x[4 * q + 2] = v.z;
        x[4 * q + 3] = v.w;
    }
}

__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&x)[16]) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
        reinterpret_cast<uint4 *>(p)[q] =
            make_uint4(pack_bf16x2(x[8 * q], x[8 * q + 1]), pack_bf16x2(x[8 * q + 2], x[8 * q + 3]),
                       pack_bf16x2(x[8 * q + 4], x[8 * q + 5]), pack_bf16x2(x[8 * q + 6], x[8 * q + 7]));
}
__device__ __forceinline__ void store16(float *p, const float (&x)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        reinterpret_cast<float4 *>(p)[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
}

// The place of the scale of row r, block j (fp4 scale tiles: 128 rows by 4 blocks).
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t j, int64_t tiles_k) {
    return ((r >> 7) * tiles_k + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
}

// Codes of 16 values and the block's scale byte; `mul` and the returned scale value give
// the values back: code * scale.
struct Coded {
    uint32_t lo, hi;  // codes 0..7, 8..15
    uint32_t scale;   // byte
    float value;      // what a code of 1 stands for
};

template <bool NV>
__device__ __forceinline__ Coded encode(float (&x)[16], float g, float inv_g) {
    Coded c;
    if (NV) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __fmul_rn(x[j], inv_g);
    }
    float amax = 0.0f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        amax = fmaxf(amax, fabsf(x[j]));
        finite = finite && fabsf(x[j]) <= FLT_MAX;
    }
    if (!NV) {  // two threads hold a block of 32
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        finite = __shfl_xor_sync(0xffffffffu, finite, 1) && finite;
    }
    float s;
    if (NV) {
        c.scale = e4m3(__fdiv_rn(amax, 6.0f));
        s = e4m3_value(c.scale);
        c.value = __fmul_rn(s, g);
        // x / s, correctly rounded: with r = RN(1/s) and q = RN(x r), the residual
        // x - q s is exact in one fma and RN(q + residual r) is RN(x / s) (Markstein 1990)
        const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float q = __fmul_rn(x[j], r);
            x[j] = copysignf(__fmaf_rn(__fmaf_rn(-q, s, x[j]), r, q), x[j]);  // -0 stays -0
        }
    } else {
        const uint32_t e = __float_as_uint(amax) >> 23;
        c.scale = e > 2u ? e - 2u : 0u;
        c.value = e8m0_value(c.scale);
        const float r = __uint_as_float((254u - c.scale) << 23);  // 2^(127 - byte)
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __fmul_rn(x[j], r);
    }
    c.lo = 0;
    c.hi = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        c.lo |= e2m1x2(x[2 * j], x[2 * j + 1]) << (8 * j);
        c.hi |= e2m1x2(x[8 + 2 * j], x[9 + 2 * j]) << (8 * j);
    }
    if (!finite) {
        c.scale = NV ? 0x7Fu : 0xFFu;
        c.value = NAN;
        c.lo = 0;
        c.hi = 0;
    }
    return c;
}

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

// One warp per 512-value segment of a row.  CODES: codes and scale tiles (whose padding,
// rows past N and blocks past K / block, is written as zero); VALUES: the values that the
// codes stand for, rounded to T.
template <typename T, bool NV, bool CODES, bool VALUES>
__global__ void __launch_bounds__(kThreads) k_encode_fp4(const PackArgs a) {
    pdl_wait();
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31;
    const float g = NV && a.g ? __ldg(a.g) : 1.0f;
    const float inv_g = __fdiv_rn(1.0f, g);
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * kThreads) >> 5;
    const int64_t units = a.rows * a.segs;
    for (int64_t u = warp; u < units; u += nwarps) {
        const int64_t row = u / a.segs;
        const int64_t k0 = (u - row * a.segs) * 512 + lane * 16;
        const bool in = row < a.N && k0 < a.K;
        float x[16];
        if (in) {
            load16<T>(static_cast<const T *>(a.x) + row * a.K + k0, x);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = 0.0f;
        }
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
        if (VALUES && in) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = __fmul_rn(e2m1_value((c.lo >> (4 * j)) & 15u), c.value);
                x[8 + j] = __fmul_rn(e2m1_value((c.hi >> (4 * j)) & 15u), c.value);
            }
            store16(static_cast<T *>(a.values) + row * a.K + k0, x);
        }
    }
}

template <typename T, bool NV>
__global__ void __launch_bounds__(kThreads) k_dequant_fp4(const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, const float *g_ptr,
                                                          T *__restrict__ out, int64_t N, int64_t K, int64_t segs,
                                                          int64_t tiles_k) {
    pdl_wait();
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31;
    const float g = NV && g_ptr ? __ldg(g_ptr) : 1.0f;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * kThreads) >> 5;
    for (int64_t u = warp; u < N * segs; u += nwarps) {
        const int64_t row = u / segs;
        const int64_t k0 = (u - row * segs) * 512 + lane * 16;
        if (k0 >= K) continue;
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes + (row * K + k0) / 2));
        const uint32_t b = __ldg(scales + scale_at(row, k0 / (NV ? 16 : 32), tiles_k));
        const float s = NV ? __fmul_rn(e4m3_value(b), g) : e8m0_value(b);
        float x[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = __fmul_rn(e2m1_value((c.x >> (4 * j)) & 15u), s);
            x[8 + j] = __fmul_rn(e2m1_value((c.y >> (4 * j)) & 15u), s);
        }
        store16(out + row * K + k0, x);
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

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int grid_of(int64_t warps, const DeviceInfo &dev) {
    return static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(cdiv(warps, kThreads / 32), static_cast<int64_t>(dev.sm_count) * 8)));
}

template <typename T, bool NV>
cudaError_t encode_t(const PackArgs &a, const DeviceInfo &dev, cudaStream_t st) {
    const dim3 grid(grid_of(a.rows * a.segs, dev)), block(kThreads);
    if (a.codes && a.values) return launch_pdl(k_encode_fp4<T, NV, true, true>, grid, block, 0, st, a);
    if (a.codes) return launch_pdl(k_encode_fp4<T, NV, true, false>, grid, block, 0, st, a);
    return launch_pdl(k_encode_fp4<T, NV, false, true>, grid, block, 0, st, a);
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
    if (f32) {
        float *o = static_cast<float *>(out);
        return nv ? launch_pdl(k_dequant_fp4<float, true>, grid, block, 0, st, codes, scales, g, o, N, K, segs, tiles_k)
                  : launch_pdl(k_dequant_fp4<float, false>, grid, block, 0, st, codes, scales, g, o, N, K, segs, tiles_k);
    }
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out);
    return nv ? launch_pdl(k_dequant_fp4<__nv_bfloat16, true>, grid, block, 0, st, codes, scales, g, o, N, K, segs, tiles_k)
              : launch_pdl(k_dequant_fp4<__nv_bfloat16, false>, grid, block, 0, st, codes, scales, g, o, N, K, segs,
                           tiles_k);
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
