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

// Eight values -> eight codes (the first in the low half of the first byte): round to
// nearest even on the e2m1 grid, saturating.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[16], int o) {
    uint32_t r;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}\n"
        : "=r"(r)
        : "f"(x[o]), "f"(x[o + 1]), "f"(x[o + 2]), "f"(x[o + 3]), "f"(x[o + 4]), "f"(x[o + 5]), "f"(x[o + 6]),
          "f"(x[o + 7]));
    return r;
}

// Packed fp32 pairs: each lane is the IEEE operation.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
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
__device__ __forceinline__ float max_nan_abs(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
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

// Eight codes -> eight bf16 pairs-wise in four words.  The bf16 images of 0, .5, 1, 1.5,
// 2, 3, 4, 6 are two tables of bytes; a byte permute looks up four codes at a time, since
// the magnitudes are its selectors.
__device__ __forceinline__ void e2m1_bf16x8(uint32_t c, uint32_t (&w)[4]) {
    const uint32_t mag = c & 0x77777777u;
    const uint32_t even = (c << 4) & 0x80808080u, odd = c & 0x80808080u;  // signs of codes 0 2 4 6 and 1 3 5 7
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sel = mag >> (16 * h);
        const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel) | __byte_perm(even, odd, h ? 0x7362 : 0x5140);
        const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
        w[2 * h] = __byte_perm(lo, hi, 0x5140);
        w[2 * h + 1] = __byte_perm(lo, hi, 0x7362);
    }
}

// The values of eight codes, code * s in fp32 (one rounding).
__device__ __forceinline__ void decode8(uint32_t c, float s, float (&x)[16], int o) {
    uint32_t w[4];
    e2m1_bf16x8(c, w);
    const uint64_t s2 = f2_pack(s, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(f2_pack(bf16_lo(w[i]), bf16_hi(w[i])), s2), x[o + 2 * i], x[o + 2 * i + 1]);
}

// The values of sixteen codes to memory, rounded to the type.  bf16: where s is a bf16
// value (it is whenever the tensor scale is a power of two) the product of two such
// short significands is exact, and half the instructions.
__device__ __forceinline__ void store_decoded(__nv_bfloat16 *p, uint32_t lo, uint32_t hi, float s) {
    uint4 v[2];
    if ((__float_as_uint(s) & 0xFFFFu) == 0) {
        const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t w[4];
            e2m1_bf16x8(q ? hi : lo, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 m = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), s2);
                w[i] = *reinterpret_cast<const uint32_t *>(&m);
            }
            v[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        float x[16];
        decode8(lo, s, x, 0);
        decode8(hi, s, x, 8);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            v[q] = make_uint4(pack_bf16x2(x[8 * q], x[8 * q + 1]), pack_bf16x2(x[8 * q + 2], x[8 * q + 3]),
                              pack_bf16x2(x[8 * q + 4], x[8 * q + 5]), pack_bf16x2(x[8 * q + 6], x[8 * q + 7]));
    }
    reinterpret_cast<uint4 *>(p)[0] = v[0];
    reinterpret_cast<uint4 *>(p)[1] = v[1];
}
__device__ __forceinline__ void store_decoded(float *p, uint32_t lo, uint32_t hi, float s) {
    float x[16];
    decode8(lo, s, x, 0);
    decode8(hi, s, x, 8);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        reinterpret_cast<float4 *>(p)[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
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

// The place of the scale of row r, block j (fp4 scale tiles: 128 rows by 4 blocks).
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t j, int64_t tiles_k) {
    return ((r >> 7) * tiles_k + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
}

// Codes of 16 values and the block's scale byte.
struct Coded {
    uint32_t lo, hi;  // codes 0..7, 8..15
    uint32_t scale;   // byte
    float value;      // what a code of 1 stands for
};

// max |x|, NaN where a value is NaN.
__device__ __forceinline__ float abs_max16(const float (&x)[16]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max_nan_abs(m, x[j]);
    return m;
}

template <bool NV>
__device__ __forceinline__ Coded encode(float (&x)[16], float g, float inv_g) {
    Coded c;
    float amax = abs_max16(x);
    if (NV) {
        // rounding keeps order, so the largest |RN(x inv_g)| is that of the largest |x|
        amax = __fmul_rn(amax, inv_g);
    } else {  // two threads hold a block of 32
        const float o = __shfl_xor_sync(0xffffffffu, amax, 1);
        amax = max_nan_abs(amax, o);
    }
    const bool finite = amax <= FLT_MAX;
    if (NV) {
        c.scale = e4m3(__fdiv_rn(amax, 6.0f));
        const float s = e4m3_value(c.scale);
        c.value = __fmul_rn(s, g);
        // x' = RN(x inv_g), then x' / s correctly rounded: with r = RN(1/s) and q = RN(x' r)
        // the residual x' - q s is exact in one fma, and RN(q + residual r) is RN(x' / s)
        // (Markstein 1990).  The sign is put back for x' = -0.
        const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
        const uint64_t g2 = f2_pack(inv_g, inv_g), r2 = f2_pack(r, r), s2 = f2_pack(-s, -s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t v = f2_mul(f2_pack(x[2 * j], x[2 * j + 1]), g2);
            const uint64_t q = f2_mul(v, r2);
            float lo, hi;
            f2_unpack(f2_fma(f2_fma(q, s2, v), r2, q), lo, hi);
            x[2 * j] = __uint_as_float(__float_as_uint(lo) | (__float_as_uint(x[2 * j]) & 0x80000000u));
            x[2 * j + 1] = __uint_as_float(__float_as_uint(hi) | (__float_as_uint(x[2 * j + 1]) & 0x80000000u));
        }
    } else {
        const uint32_t e = __float_as_uint(amax) >> 23;
        c.scale = e > 2u ? e - 2u : 0u;
        c.value = e8m0_value(c.scale);
        const float r = __uint_as_float((254u - c.scale) << 23);  // 2^(127 - byte)
        const uint64_t r2 = f2_pack(r, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) f2_unpack(f2_mul(f2_pack(x[2 * j], x[2 * j + 1]), r2), x[2 * j], x[2 * j + 1]);
    }
    c.lo = e2m1x8(x, 0);
    c.hi = e2m1x8(x, 8);
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
// written as zero); VALUES: the values that the codes stand for, rounded to T.
template <typename T, bool NV, bool CODES, bool VALUES>
__global__ void __launch_bounds__(kThreads, 5) k_encode_fp4(const PackArgs a) {
    pdl_wait();
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31;
    const float g = NV && a.g ? __ldg(a.g) : 1.0f;
    const float inv_g = __fdiv_rn(1.0f, g);
    for (Segments u(a.segs); u.row < a.rows; u.next()) {
        const int64_t row = u.row, k0 = static_cast<int64_t>(u.seg) * 512 + lane * 16;
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
        if (VALUES && in) store_decoded(static_cast<T *>(a.values) + row * a.K + k0, c.lo, c.hi, c.value);
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
    for (Segments u(segs); u.row < N; u.next()) {
        const int64_t k0 = static_cast<int64_t>(u.seg) * 512 + lane * 16;
        if (k0 >= K) continue;
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes + (u.row * K + k0) / 2));
        const uint32_t b = __ldg(scales + scale_at(u.row, k0 / (NV ? 16 : 32), tiles_k));
        store_decoded(out + u.row * K + k0, c.x, c.y, NV ? __fmul_rn(e4m3_value(b), g) : e8m0_value(b));
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
