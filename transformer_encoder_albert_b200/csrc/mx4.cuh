// mx4.cuh -- microscaled 4-bit values on the device: E2M1 codes with one 8-bit
// scale per block along a row ("mxfp4": blocks of 32, E8M0 scales; "nvfp4":
// blocks of 16, E4M3 scales times one fp32 factor of the tensor).
//
// The decisions (scale byte, code) are taken in fp32 exactly as include/albert.h
// states them, so that two kernels that quantize the same fp32 values agree bit
// for bit:
//   mxfp4: byte = max(biased exponent of amax - 2, 0); q = E2M1(x * 2^(127 - byte)),
//          the power of two exact, so the only rounding is E2M1's;
//   nvfp4: byte = E4M3(fl(amax / fl(6 ts))), d = fl(E4M3 value * ts), q = E2M1(fl(x * fl(1 / d))).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "sm100_ptx.cuh"

namespace albert {

// Storage geometry.  A scale tile holds 128 rows x 4 blocks (512 bytes): byte
// (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 -- the order in which tcgen05.cp
// (32x128b, replicated to the four lane quadrants) brings a 128-row operand's
// scales to tensor memory.  A row's tiles cover a multiple of 256 columns, one
// stage of the products' main loop.
constexpr int kMx4StageCols = 256;
constexpr int kMx4TileBytes = 512;
template <bool NV>
struct Mx4 {
    static constexpr int kBlock = NV ? 16 : 32;
    static constexpr int kTileCols = 4 * kBlock;                   // columns of one scale tile
    static constexpr int kStageTiles = kMx4StageCols / kTileCols;  // 4 (nvfp4) or 2 (mxfp4)
};
__host__ __device__ __forceinline__ int mx4_stages(int cols) { return (cols + kMx4StageCols - 1) / kMx4StageCols; }
__host__ __device__ __forceinline__ int mx4_code_pitch(int cols) { return (cols + 31) / 32 * 16; }  // bytes per row

// Eight fp32 -> eight E2M1 codes, value i in nibble i: nearest, ties to the even
// code, saturating at 6.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    // 2^(byte - 127): byte 0 is below fp32's normals, byte 255 is NaN
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const uint32_t e = (byte >> 3) & 15u, m = byte & 7u;
    if ((byte & 0x7fu) == 0x7fu) return __uint_as_float(0x7fffffffu);
    // (1 + m/8) 2^(e-7), subnormals m/8 2^-6
    const float mag = e == 0 ? (float)m * 0.001953125f : __uint_as_float(((e + 120u) << 23) | (m << 20));
    return (byte & 0x80u) ? -mag : mag;
}
template <bool NV>
__device__ __forceinline__ float mx4_scale_value(uint32_t byte) {
    return NV ? e4m3_value(byte) : e8m0_value(byte);
}

// One block's scale byte, and the factor its values are multiplied by before the
// rounding to E2M1.  amax_bits: the largest |x| of the block as bits (integer
// order puts infinities and NaN above every finite value); a block that holds
// one gets a NaN scale and zero codes (factor 0 with the values replaced by 0).
struct Mx4Scale {
    uint32_t byte;
    float mul;
    bool zero;  // codes are 0 whatever the values
};
// fl(a / b) for a >= 0 from y = fl(1 / b): Markstein's correction (IBM J. Res. Dev. 34,
// 1990) twice -- the first makes the quotient faithful, the second correctly rounded,
// each remainder being exact in an fma.  Quotients from 1024 on all saturate; those
// below fp32's normals all round to an E4M3 zero.
__device__ __forceinline__ float mx4_quotient(float a, float b, float y) {
    const float q0 = a * y;
    const float q1 = fmaf(fmaf(-q0, b, a), y, q0);
    const float q2 = fmaf(fmaf(-q1, b, a), y, q1);
    return q0 < 1024.0f ? q2 : 1024.0f;
}

// The constants of a tensor scale that a block needs.
struct Mx4Ts {
    float ts, six, inv_six;
};
__device__ __forceinline__ Mx4Ts mx4_ts(float ts) { return Mx4Ts{ts, 6.0f * ts, __frcp_rn(6.0f * ts)}; }

template <bool NV>
__device__ __forceinline__ Mx4Scale mx4_block_scale(uint32_t amax_bits, const Mx4Ts &ts) {
    Mx4Scale s;
    const bool bad = amax_bits >= 0x7f800000u;
    if constexpr (!NV) {
        const uint32_t e = amax_bits >> 23;
        s.byte = bad ? 255u : (e > 2u ? e - 2u : 0u);
        s.mul = __uint_as_float((254u - (bad ? 127u : s.byte)) << 23);
        s.zero = bad;
    } else {
        const float t = mx4_quotient(__uint_as_float(bad ? 0u : amax_bits), ts.six, ts.inv_six);
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(t));
        s.byte = bad ? 0x7fu : (uint32_t)(c & 0xffu);
        s.zero = bad || s.byte == 0u;
        const float d = __fmul_rn(e4m3_value(s.byte), ts.ts);
        s.mul = __frcp_rn(s.zero ? 1.0f : d);  // = fl(1 / d); zero: the codes are dropped anyway
    }
    return s;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
    else return __float2bfloat16_rn(x);
}

// Two floats as one 32-bit word of two 16-bit values.
template <typename T>
__device__ __forceinline__ uint32_t pack_x2(float lo, float hi) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
template <typename T>
__device__ __forceinline__ float2 unpack_x2(uint32_t u) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
}

// Eight consecutive values of a row as they are stored: 16 bytes, or 32 for fp32.
template <typename T>
struct Raw8 {
    uint32_t w[sizeof(T) * 2];
};
// From p; only the first `n` (0..8, or more) exist, the rest are 0.  vec: p is
// 16-byte aligned whenever all eight exist.
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T *p, int n, bool vec) {
    Raw8<T> r;
    if (vec && n >= 8) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        if constexpr (sizeof(T) == 4) {
            const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
            r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = i < n ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < n ? __ldg(reinterpret_cast<const unsigned short *>(p) + 2 * i) : 0u;
            const uint32_t hi = 2 * i + 1 < n ? __ldg(reinterpret_cast<const unsigned short *>(p) + 2 * i + 1) : 0u;
            r.w[i] = lo | (hi << 16);
        }
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void raw8_values(const Raw8<T> &r, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f;
            if constexpr (std::is_same<T, __half>::value) f = unpack_x2<T>(r.w[i]);
            else f = make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, bool vec, float (&v)[8]) {
    raw8_values<T>(load_raw8<T>(p, n, vec), v);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int n, bool vec, const float (&v)[8]) {
    if (vec && n >= 8) {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_x2<T>(v[0], v[1]), pack_x2<T>(v[2], v[3]),
                                                       pack_x2<T>(v[4], v[5]), pack_x2<T>(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}

// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float fmax3_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// GELU_tanh of a pair: x / (1 + e), e = exp(-2u), u = sqrt(2/pi) (x + 0.044715 x^3).  The
// two quotients share one reciprocal, 1 / ((1 + e0)(1 + e1)): three special-function
// operations for two values instead of four (they set the pace: 16 lanes per clock and
// SM).  The exponent stops at 63, so that the product stays finite.  Past it (x below -7.61)
// the factor is 0, which is off by at most 7.7 x 2^-63 < 10^-18 and gives -0 however far x
// is, and NaN for -infinity, as the tanh form does.  Above, the relative error is a few 2^-23
// plus 2^-23 |2u| from the exponential's argument.  (18797 x 768 -> 2048 in mxfp4 with a bf16
// result: 30.4 us; 28.7 without the two selections, 31.3 with a reciprocal each and no limit,
// 31.8 where a warp first looks whether it has such a value.)
__device__ __forceinline__ uint64_t gelu_f2(uint64_t x) {
    const float k0 = -2.0f * 0.7978845608028654f * 1.4426950408889634f, k1 = k0 * 0.044715f;
    const float2 t = f2_split(f2_mul(x, f2_fma(f2_mul(x, x), f2_make(k1, k1), f2_make(k0, k0))));
    const uint64_t d = f2_add(f2_make(ex2_approx(fminf(t.x, 63.0f)), ex2_approx(fminf(t.y, 63.0f))), f2_make(1.0f, 1.0f));
    const float2 df = f2_split(d);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(df.x * df.y));
    const float2 f = f2_split(f2_mul(f2_make(df.y, df.x), f2_make(r, r)));  // (1 / d first: x d could overflow)
    return f2_mul(x, f2_make(t.x > 63.0f ? 0.f : f.x, t.y > 63.0f ? 0.f : f.y));
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t umax_x2(uint32_t a, uint32_t b) {  // two 16-bit maxima
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest magnitude of eight values, as bits that order like it (16-bit types:
// their own bits, two at a time), and those bits as fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t raw8_amax(const Raw8<T> &r) {
    if constexpr (sizeof(T) == 4) {
        uint32_t m = r.w[0] & 0x7fffffffu;
#pragma unroll
        for (int i = 1; i < 8; ++i) m = umax(m, r.w[i] & 0x7fffffffu);
        return m;
    } else {
        uint32_t m = r.w[0] & 0x7fff7fffu;
#pragma unroll
        for (int i = 1; i < 4; ++i) m = umax_x2(m, r.w[i] & 0x7fff7fffu);
        return umax(m & 0xffffu, m >> 16);
    }
}
template <typename T>
__device__ __forceinline__ uint32_t amax_f32_bits(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    else if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    else return m << 16;
}

// A warp quantizes 256 consecutive columns of a row, eight per lane: the block's
// lanes (four, or two) share its largest magnitude `m` (of the lane's own eight
// values, fp32 bits) by shuffles.  Returns the lane's codes; `word` becomes the four
// scale bytes of the lane's tile (every lane of the tile holds it).
template <bool NV>
__device__ __forceinline__ uint32_t mx4_warp_quant(const float (&v)[8], uint32_t m, const Mx4Ts &ts, int lane, uint32_t &word) {
    m = umax(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if constexpr (!NV) m = umax(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const Mx4Scale s = mx4_block_scale<NV>(m, ts);
    const uint64_t mul2 = f2_make(s.mul, s.mul);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 f = f2_split(f2_mul(f2_make(v[i], v[i + 1]), mul2));
        y[i] = f.x;
        y[i + 1] = f.y;
    }
    uint32_t q = cvt_e2m1x8(y);
    if (s.zero) q = 0;
    constexpr int kLanes = NV ? 2 : 4;  // lanes of a block
    uint32_t w = s.byte << (8 * ((lane / kLanes) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, kLanes);
    w |= __shfl_xor_sync(0xffffffffu, w, 2 * kLanes);
    word = w;
    return q;
}

// Eight E2M1 codes -> their values.
__device__ __forceinline__ void e2m1x8_values(uint32_t q, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(q >> (8 * i)));
        const float2 f = unpack_x2<__half>(h);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

}  // namespace albert
