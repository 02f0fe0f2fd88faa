// Block-scaled values of the key/value caches: E4M3 or E2M1 elements with an
// E8M0 scale per 32 consecutive features (the OCP microscaling MXFP8 and MXFP4
// layouts), to bf16 and back.
#pragma once

#include "gdn_ops.hpp"

namespace gdnmx {

using namespace gdnops;

constexpr int kBlock = 32;           // features of a scale

// 2^(s - 127) of a scale byte.  255 gives an infinity, which the conversions
// below turn into NaN, as the format has it.
__device__ __forceinline__ float scale_of(uint32_t s) { return __builtin_amdgcn_ldexpf(1.0f, (int)s - 127); }

__device__ __forceinline__ uint32_t bits(bf16x2 x) { return __builtin_bit_cast(uint32_t, x); }

// Formats: two features a byte or one; Raw8 holds eight features as stored.  The
// bf16 values are exact (four significant bits at most; those of a scale below
// 2^-124 may round, where bf16 has no smaller steps).
struct Fp4 {
    static constexpr int kPerByte = 2;
    typedef uint32_t Raw8;
    typedef u32x2 Raw16;
    __device__ static __forceinline__ Raw8 low(Raw16 r) { return r[0]; }
    __device__ static __forceinline__ Raw8 high(Raw16 r) { return r[1]; }
    __device__ static __forceinline__ u32x4 widen(Raw8 r, float s) {
        return u32x4{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 0)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 1)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 2)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 3))};
    }
    __device__ static __forceinline__ void widen(Raw8 r, float s, float* f) {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 1);
        const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 2);
        const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 3);
        f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1], f[4] = c[0], f[5] = c[1], f[6] = d[0], f[7] = d[1];
    }
    // Features 4 i .. 4 i + 3 of eight, as two dwords of bf16.
    __device__ static __forceinline__ u32x2 widen4(const uint8_t* p, float s) {
        const uint32_t r = *reinterpret_cast<const uint16_t*>(p);
        return u32x2{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 0)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 1))};
    }
    // The exponent of the largest element, 6 = 1.5 2^2.
    static constexpr int kTop = 2;
    // Eight values in units of the scale, below 8 in magnitude: to the nearest
    // code (ties to even, 6 at most), with -0 as +0.
    __device__ static __forceinline__ Raw8 narrow(const float* y) {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[0], y[1], 1.0f, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[2], y[3], 1.0f, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[4], y[5], 1.0f, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[6], y[7], 1.0f, 3);
        const uint32_t some = (r | r >> 1 | r >> 2) & 0x11111111u;
        return r & (0x77777777u | some << 3);
    }
};
struct Fp8 {
    static constexpr int kPerByte = 1;
    typedef u32x2 Raw8;
    typedef u32x4 Raw16;
    __device__ static __forceinline__ Raw8 low(Raw16 r) { return u32x2{r[0], r[1]}; }
    __device__ static __forceinline__ Raw8 high(Raw16 r) { return u32x2{r[2], r[3]}; }
    __device__ static __forceinline__ u32x4 widen(Raw8 r, float s) {
        return u32x4{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[0], s, false)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[0], s, true)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[1], s, false)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[1], s, true))};
    }
    __device__ static __forceinline__ void widen(Raw8 r, float s, float* f) {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r[0], s, false);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r[0], s, true);
        const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r[1], s, false);
        const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r[1], s, true);
        f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1], f[4] = c[0], f[5] = c[1], f[6] = d[0], f[7] = d[1];
    }
    __device__ static __forceinline__ u32x2 widen4(const uint8_t* p, float s) {
        const uint32_t r = *reinterpret_cast<const uint32_t*>(p);
        return u32x2{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r, s, false)),
                     bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r, s, true))};
    }
    static constexpr int kTop = 8;   // 448 = 1.75 2^8
    __device__ static __forceinline__ Raw8 narrow(const float* y) {
        float c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = fminf(fmaxf(y[j], -448.f), 448.f);   // beyond 464 the conversion gives NaN
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
        return u32x2{(uint32_t)lo, (uint32_t)hi};
    }
};

}  // namespace gdnmx
