// mx.cuh -- microscaled (MX) number formats: blocks of 32 consecutive values
// of a row that share one power-of-two scale.
//
//   e4m3: 1 sign, 4 exponent (bias 7), 3 mantissa bits, largest value 448
//   e2m1: 1 sign, 2 exponent (bias 1), 1 mantissa bit, values 0 .5 1 1.5 2 3 4 6
//   scale: the byte c stands for 2^(c - 127); c = 255 is NaN
// (OCP Microscaling Formats specification v1.0.)  The scale written here is
// the smallest power of two, at least 2^-127, that keeps the block's largest
// magnitude within the format's range, so nothing saturates; codes are
// x / scale rounded to nearest, ties to even.  A block that holds a NaN or an
// infinity gets the scale byte 255 and codes 0: it reads back as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cstdint>

namespace moe {

constexpr int kMxBlock = 32;

// Element types and code formats of the C ABI.
constexpr int kTypeBf16 = 0, kTypeFp16 = 1, kTypeFp32 = 2;
constexpr int kMxE4M3 = 0, kMxE2M1 = 1;

// Bytes of a row of scales: one per block, rows padded to 16 bytes (a tensor
// copy's stride).
__host__ __device__ constexpr int mx_scale_pitch(int cols)
{
    return (cols / kMxBlock + 15) & ~15;
}

// Scale byte for a block whose largest magnitude, finite, has the bits
// `amax` = m 2^(e - 127), 1 <= m < 2: the largest code is 1.75 * 2^8 or
// 1.5 * 2^2, so the byte is e - 8 (e - 2), one more when m is above 1.75 (1.5),
// which the addition carries into the exponent.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_code_finite(uint32_t amax)
{
    const int c = static_cast<int>((amax + (FMT == kMxE4M3 ? 0x1fffffu : 0x3fffffu)) >> 23) -
                  (FMT == kMxE4M3 ? 8 : 2);
    return static_cast<uint32_t>(max(c, 0));
}

// The same for any block: 255 when it holds a NaN or an infinity.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax)
{
    return amax >= 0x7f800000u ? 255u : mx_scale_code_finite<FMT>(amax);
}

// Two e4m3 codes, `lo` in the low byte, rounded to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// 2^(127 - c), exact for every c that mx_scale_code gives; 0 for c = 255,
// which sends every finite value to the code 0.
__device__ __forceinline__ float mx_inv_scale(uint32_t c)
{
    return c == 255u ? 0.0f : __uint_as_float((254u - c) << 23);
}

// 2^(c - 127), NaN for c = 255.
__device__ __forceinline__ float mx_scale(uint32_t c)
{
    return __uint_as_float(c == 255u ? 0x7fffffffu : c == 0u ? 0x00400000u : c << 23);
}

// |x| as bits that order like the magnitudes (NaN above infinity).
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Codes of eight values times `inv`: e4m3 in 8 bytes, e2m1 in 4 (the first
// value in the low half of the first byte).
template <int FMT>
__device__ __forceinline__ uint2 mx_codes8(const float (&v)[8], uint32_t code)
{
    const float inv = mx_inv_scale(code);
    uint32_t w[2] = {0u, 0u};
    if (code != 255u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = make_float2(v[2 * i] * inv, v[2 * i + 1] * inv);
            if constexpr (FMT == kMxE4M3)
                w[i >> 1] |= e4m3x2(p.x, p.y) << (16 * (i & 1));
            else
                w[0] |= static_cast<uint32_t>(
                            __nv_cvt_float2_to_fp4x2(p, __NV_E2M1, cudaRoundNearest))
                        << (8 * i);
        }
    }
    return make_uint2(w[0], w[1]);
}

// The eight values that codes of mx_codes8 and their scale byte stand for.
template <int FMT>
__device__ __forceinline__ void mx_values8(const uint2 &q, uint32_t code, float (&v)[8])
{
    const float s = mx_scale(code);
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2_raw h;
        if constexpr (FMT == kMxE4M3)
            h = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        else
            h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(w[0] >> (8 * i)),
                                           __NV_E2M1);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

// ------------------------------------------------------- rows of 8 elements
// Eight consecutive elements (16-byte aligned) of an array of type TYPE.
template <int TYPE>
struct Vec8 {
    uint4 u[TYPE == kTypeFp32 ? 2 : 1];
};

template <int TYPE>
__host__ __device__ constexpr int type_size() { return TYPE == kTypeFp32 ? 4 : 2; }

template <int TYPE>
__device__ __forceinline__ Vec8<TYPE> load8(const void *p)
{
    Vec8<TYPE> r;
    r.u[0] = static_cast<const uint4 *>(p)[0];
    if constexpr (TYPE == kTypeFp32) r.u[1] = static_cast<const uint4 *>(p)[1];
    return r;
}

template <int TYPE>
__device__ __forceinline__ void unpack8(const Vec8<TYPE> &r, float (&v)[8])
{
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
    if constexpr (TYPE == kTypeFp32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
        v[4] = __uint_as_float(r.u[1].x);
        v[5] = __uint_as_float(r.u[1].y);
        v[6] = __uint_as_float(r.u[1].z);
        v[7] = __uint_as_float(r.u[1].w);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == kTypeBf16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

// Rounded to the nearest value of the type, ties to even.
template <int TYPE>
__device__ __forceinline__ Vec8<TYPE> pack8(const float (&v)[8])
{
    Vec8<TYPE> r;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < (TYPE == kTypeFp32 ? 8 : 4); ++i) {
        if constexpr (TYPE == kTypeFp32) {
            w[i] = __float_as_uint(v[i]);
        } else if constexpr (TYPE == kTypeBf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (TYPE == kTypeFp32) r.u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}

template <int TYPE>
__device__ __forceinline__ void store8(void *p, const Vec8<TYPE> &r)
{
    static_cast<uint4 *>(p)[0] = r.u[0];
    if constexpr (TYPE == kTypeFp32) static_cast<uint4 *>(p)[1] = r.u[1];
}

}  // namespace moe
