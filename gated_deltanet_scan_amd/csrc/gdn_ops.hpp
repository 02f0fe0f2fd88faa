// Helpers shared by the operators around the scan (layer norm, rotary
// positions, attention): element access, wave sums and the host-side argument
// checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/gdn.h"

namespace gdnops {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// The same vectors at an element's alignment: rows of odd width start
// anywhere, and gfx950 loads and stores such vectors in one instruction.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float bf2f(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ uint16_t f2bf(float x) {
    __bf16 b = (__bf16)x;  // round to nearest even
    return __builtin_bit_cast(uint16_t, b);
}
// Two floats to two bf16 (round to nearest even) in one dword, x in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}

// Eight consecutive elements, held as stored (Raw) and widened on use.
template <typename T> struct Vec8;
template <> struct Vec8<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x4_a2*>(p); }
    __device__ __forceinline__ void zero() { v = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = v[i >> 1];
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<u32x4_a2*>(p) = v; }
};
template <> struct Vec8<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const f32x4_a4*>(p);
        b = *reinterpret_cast<const f32x4_a4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = f[i];
            b[i] = f[i + 4];
        }
    }
    __device__ __forceinline__ void store(float* p) const {
        *reinterpret_cast<f32x4_a4*>(p) = a;
        *reinterpret_cast<f32x4_a4*>(p + 4) = b;
    }
};

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<uint16_t>(uint16_t x) { return bf2f(x); }
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ uint16_t from_f<uint16_t>(float x) { return f2bf(x); }
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// Sum over the 64 lanes, in every lane: DPP swaps inside each 16-lane row, then
// the four rows' sums through scalar registers.  Every lane must be active.
__device__ __forceinline__ float wave_sum(float x) {
    x += dpp_f<0xB1>(x);    // quad_perm [1,0,3,2]
    x += dpp_f<0x4E>(x);    // quad_perm [2,3,0,1]
    x += dpp_f<0x141>(x);   // row_half_mirror
    x += dpp_f<0x140>(x);   // row_mirror
    const int i = __float_as_int(x);
    return (__int_as_float(__builtin_amdgcn_readlane(i, 0)) + __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(i, 32)) + __int_as_float(__builtin_amdgcn_readlane(i, 48)));
}

// ---------------------------------------------------------------- host checks
struct Range {
    uintptr_t lo, hi;
};
inline Range rng(const void* p, size_t n) { return Range{(uintptr_t)p, (uintptr_t)p + (p ? n : 0)}; }
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }
inline bool aligned(const void* p, uintptr_t al) { return ((uintptr_t)p & (al - 1)) == 0; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// GDN_OK on a gfx950 device; *cus its compute units.
inline gdn_status check_device(int* cus) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GDN_ERR_NO_DEVICE;
    // one query per device and process: the answer never changes
    static int cached[64];
    if (dev < 64) {
        const int c = __atomic_load_n(&cached[dev], __ATOMIC_RELAXED);
        if (c > 0) {
            *cus = c;
            return GDN_OK;
        }
    }
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, dev) != hipSuccess) return GDN_ERR_NO_DEVICE;
    if (strncmp(p.gcnArchName, "gfx950", 6) != 0) return GDN_ERR_UNSUPPORTED;
    *cus = p.multiProcessorCount;
    if (dev < 64) __atomic_store_n(&cached[dev], p.multiProcessorCount, __ATOMIC_RELAXED);
    return GDN_OK;
}

}  // namespace gdnops
