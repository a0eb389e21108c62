// Element arithmetic of the microscaled 4-bit floats, shared by the packing kernels and
// the product (which packs few tokens itself): blocks of 16 values per thread to codes
// and a scale byte, and back.
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
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "eqat_qmath.cuh"

namespace eqat {
namespace fp4 {

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

// The values of sixteen codes to memory, rounded to the type; V8: p is 32-byte aligned
// and every store writes whole sectors.  bf16: where s is a bf16 value (it is whenever
// the tensor scale is a power of two) one packed bf16 product rounds once, as fp32 and
// the rounding of its exact product do, in half the instructions.
template <bool V8>
__device__ __forceinline__ void store_decoded(__nv_bfloat16 *p, uint32_t lo, uint32_t hi, float s) {
    uint32_t v[8];
    if ((__float_as_uint(s) & 0xFFFFu) == 0) {
        const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t w[4];
            e2m1_bf16x8(q ? hi : lo, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 m = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), s2);
                v[4 * q + i] = *reinterpret_cast<const uint32_t *>(&m);
            }
        }
    } else {
        float x[16];
        decode8(lo, s, x, 0);
        decode8(hi, s, x, 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
    if (V8) {
        st_global_v8(p, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
template <bool V8>
__device__ __forceinline__ void store_decoded(float *p, uint32_t lo, uint32_t hi, float s) {
    float x[16];
    decode8(lo, s, x, 0);
    decode8(hi, s, x, 8);
    store16<float, V8>(p, x);
}

// 16 consecutive values of a row, as stored and widened.
template <typename T>
struct Raw16 {
    Raw8<T> a, b;
};
template <typename T>
__device__ __forceinline__ Raw16<T> load_raw16(const T *p) {
    return Raw16<T>{load_raw8(p), load_raw8(p + 8)};
}
template <typename T>
__device__ __forceinline__ Raw16<T> zero16();
template <>
__device__ __forceinline__ Raw16<__nv_bfloat16> zero16<__nv_bfloat16>() {
    return Raw16<__nv_bfloat16>{{make_uint4(0, 0, 0, 0)}, {make_uint4(0, 0, 0, 0)}};
}
template <>
__device__ __forceinline__ Raw16<float> zero16<float>() {
    const float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return Raw16<float>{{z, z}, {z, z}};
}
template <typename T>
__device__ __forceinline__ void unpack16(const Raw16<T> &r, float (&x)[16]) {
    float u[8], v[8];
    unpack8(r.a, u);
    unpack8(r.b, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] = u[j];
        x[8 + j] = v[j];
    }
}
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
    unpack16(load_raw16(p), x);
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

}  // namespace fp4
}  // namespace eqat
