// 8-bit floats with an fp32 scale for each group of 128 columns: the C ABI of
// gdn_rms_norm_fwd_fp8 and gdn_quantize_fp8 (declared in include/gdn.h).
//
//     t = x + residual,  y = t (<t^2> + eps)^(-1/2) w      (quantise: y = x)
//     m = max(max |y|, 2^-100) over a group,  scale = m / 448,  code = e4m3(y (448 / m))
//
// Bound by memory: x (and residual) are read once, the codes, their scales and
// the sum written once.  A lane holds eight columns, so a group of 128 is one
// row of 16 lanes and its maximum four lane exchanges inside that row.  The norm is
// formed in fp32 from the unrounded sum of x and residual, and y goes to its code
// unrounded: the code's is the only rounding of y to fewer bits.
#include "gdn_ops.hpp"

#include <algorithm>

namespace {

using namespace gdnops;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kGroup = 128;          // columns of a scale
constexpr int kLanes = kGroup / 8;   // lanes of a group

struct QuantArgs {
    const void *x, *r, *w;
    void* sum;
    uint8_t* y;
    float* scale;                    // [rows][groups]
    int64_t rows;
    int C, groups;
    float eps;
};

typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

// Eight columns from c on; past C they read as zeros and are not stored.
template <typename T>
__device__ __forceinline__ void load8(Vec8<T>& v, const T* row, int c, int C) {
    if (c + 8 <= C) {
        v.load(row + c);
    } else {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = c + j < C ? to_f<T>(row[c + j]) : 0.f;
        v.set(f);                                        // the same values again: exact
    }
}
template <typename T>
__device__ __forceinline__ void store8(const Vec8<T>& v, T* row, int c, int C) {
    if (c + 8 <= C) {
        v.store(row + c);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < C) row[c + j] = from_f<T>(v.get(j));
    }
}

// Maximum over a row of 16 lanes, in each of them.
__device__ __forceinline__ float row16_max(float x) {
    x = fmaxf(x, dpp_f<0xB1>(x));
    x = fmaxf(x, dpp_f<0x4E>(x));
    x = fmaxf(x, dpp_f<0x141>(x));
    return fmaxf(x, dpp_f<0x140>(x));
}

// A lane's eight values of a group to e4m3, which all 16 lanes of the group
// call together.  The products are at most 448 (1 + 2^-23), which rounds to 448.
// A NaN stays one; an infinity makes the scale infinite and its group NaN.
__device__ __forceinline__ void quantise8(const float* f, uint8_t* row, float* scale, int c, int C) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]));
    top = fmaxf(row16_max(top), 0x1p-100f);
    if (c >= C) return;
    const float inv = 448.0f / top;
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inv, f[5] * inv, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inv, f[7] * inv, hi, true);
    if (c + 8 <= C) {
        *reinterpret_cast<u32x2_a1*>(row + c) = u32x2{(uint32_t)lo, (uint32_t)hi};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < C) row[c + j] = (uint8_t)((uint32_t)(j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
    if (c % kGroup == 0) scale[c / kGroup] = top / 448.0f;
}

// Rows of up to 512 NV WPR columns, WPR waves to a row; lane t of a row holds
// the columns 8 (t + 64 WPR i) and the seven after them.  A row stays in registers
// between its norm and its codes, and the next row's loads run meanwhile.  106480 rows
// of 2048 bf16 columns with residual and sum: 290 to 300 us, 5.3 to 5.1 TB/s, what a copy
// reaches (fp32 540 to 543, 5.2 TB/s); 880 rows: 4.3 to 4.6 us, a launch and two trips to
// memory.
template <typename T, typename W, int NV, int WPR>
__global__ __launch_bounds__(kThreads) void rms_quant_kernel(const QuantArgs a) {
    __shared__ float red[2][kWaves];
    constexpr int RPB = kWaves / WPR;                    // rows per workgroup and step
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t = WPR == 1 ? (tid & 63) : tid, C = a.C;
    auto col = [&](int i) { return 8 * (t + 64 * WPR * i); };
    int phase = 0;
    Vec8<W> w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (a.w) load8(w[i], static_cast<const W*>(a.w), col(i), C);
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? wave : 0);
    Vec8<T> nx[NV], nr[NV];
    auto fetch = [&](int64_t rw) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load8(nx[i], static_cast<const T*>(a.x) + rw * C, col(i), C);
            if (a.r) load8(nr[i], static_cast<const T*>(a.r) + rw * C, col(i), C);
        }
    };
    if (row < a.rows) fetch(row);
    for (; row < a.rows; row += step) {
        float f[NV][8];
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = a.r ? nx[i].get(j) + nr[i].get(j) : nx[i].get(j);
#pragma unroll
            for (int j = 0; j < 8; ++j) q += f[i][j] * f[i][j];
        }
        if (row + step < a.rows) fetch(row + step);
        if (a.sum) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                Vec8<T> v;
                v.set(f[i]);
                store8(v, static_cast<T*>(a.sum) + row * C, col(i), C);
            }
        }
        q = wave_sum(q);
        if constexpr (WPR > 1) {
            // two buffers, so one barrier a row is enough
            if ((tid & 63) == 0) red[phase][wave] = q;
            __syncthreads();
            q = (red[phase][0] + red[phase][1]) + (red[phase][2] + red[phase][3]);
            phase ^= 1;
        }
        const float s = 1.0f / sqrtf(q / (float)C + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * s * (a.w ? w[i].get(j) : 1.f);
            quantise8(f[i], a.y + row * C, a.scale + row * a.groups, col(i), C);
        }
    }
}

// Wider rows: a workgroup a row, which reads it twice (the second time from the
// caches).  2000 rows of 12288: 40 us, 4.3 TB/s.
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void rms_quant_wide_kernel(const QuantArgs a) {
    __shared__ float red[2][kWaves];
    const int tid = threadIdx.x, C = a.C;
    int phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T*>(a.x) + row * C, *r = a.r ? static_cast<const T*>(a.r) + row * C : nullptr;
        auto values = [&](int c, float* f) {
            Vec8<T> v, u;
            load8(v, x, c, C);
            if (r) load8(u, r, c, C);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = r ? v.get(j) + u.get(j) : v.get(j);
        };
        float q = 0.f;
        for (int c = 8 * tid; c < C; c += 8 * kThreads) {
            float f[8];
            values(c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) q += f[j] * f[j];
        }
        q = wave_sum(q);
        if ((tid & 63) == 0) red[phase][tid >> 6] = q;
        __syncthreads();
        q = (red[phase][0] + red[phase][1]) + (red[phase][2] + red[phase][3]);
        phase ^= 1;
        const float s = 1.0f / sqrtf(q / (float)C + a.eps);
        // whole groups: all 16 lanes of one take part in its maximum
        for (int c = 8 * tid; c < a.groups * kGroup; c += 8 * kThreads) {
            float f[8];
            values(c, f);
            if (a.sum) {
                Vec8<T> v;
                v.set(f);
                store8(v, static_cast<T*>(a.sum) + row * C, c, C);
            }
            Vec8<W> w;
            if (a.w) load8(w, static_cast<const W*>(a.w), c, C);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * s * (a.w ? w.get(j) : 1.f);
            quantise8(f, a.y + row * C, a.scale + row * a.groups, c, C);
        }
    }
}

// Quantisation alone: 16 lanes a group, groups in their order.  106480 rows of 2048
// bf16 columns: 132 to 136 us, 5.0 to 4.8 TB/s (fp32 224 to 228, 4.9 to 4.8); 880 rows: 2.9
// to 4.0 us.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantise_kernel(const QuantArgs a) {
    const int64_t all = a.rows * a.groups, step = (int64_t)gridDim.x * (kThreads / kLanes);
    for (int64_t g = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; g < all; g += step) {
        const int64_t row = g / a.groups;
        const int c = (int)(g - row * a.groups) * kGroup + 8 * (threadIdx.x % kLanes);
        Vec8<T> v;
        load8(v, static_cast<const T*>(a.x) + row * a.C, c, a.C);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v.get(j);
        quantise8(f, a.y + row * a.C, a.scale + row * a.groups, c, a.C);
    }
}

// ---------------------------------------------------------------- launch
gdn_status done() { return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

// Waves to a row (bf16, residual and sum).  Up to 1024 columns a wave: 880 x 1024 3.6 us
// against 4.1 with four.  Up to 2048 four while a row has a workgroup's time to itself,
// up to 16 rows a CU (8 x 2048 2.8 us against 4.3, 1024 x 2048 4.5 against 5.2, 4096 x
// 2048 11.4 against 12.2), and one for more (50000 x 1280 119 us against 144, 106480 x
// 2048 290 against 300).  Past 8192 the registers of a row leave a CU one workgroup: that
// pays up to a row a CU (8 x 16384 7.0 us against 10.3 for rows read twice; 1024 x 12288
// 35 against 22, 2000 x 16384 54 against 53).
template <typename T, typename W>
gdn_status launch_norm(const QuantArgs& a, int cus, hipStream_t s) {
    if (a.C > 16384 || (a.C > 8192 && a.rows > cus)) {
        hipLaunchKernelGGL((rms_quant_wide_kernel<T, W>), dim3((unsigned)std::min<int64_t>(a.rows, (int64_t)cus * 4)),
                           dim3(kThreads), 0, s, a);
        return done();
    }
    const int wpr = a.C <= 1024 || (a.C <= 2048 && a.rows > (int64_t)cus * 16) ? 1 : 4, rpb = kWaves / wpr;
    const dim3 grid((unsigned)std::min<int64_t>((a.rows + rpb - 1) / rpb, (int64_t)cus * 4));
#define GDN_RMS(NV, WPR) hipLaunchKernelGGL((rms_quant_kernel<T, W, NV, WPR>), grid, dim3(kThreads), 0, s, a)
    if (a.C <= 512)
        GDN_RMS(1, 1);
    else if (a.C <= 1024)
        GDN_RMS(2, 1);
    else if (a.C <= 2048 && wpr == 1)
        GDN_RMS(4, 1);
    else if (a.C <= 2048)
        GDN_RMS(1, 4);
    else if (a.C <= 4096)
        GDN_RMS(2, 4);
    else if (a.C <= 8192)
        GDN_RMS(4, 4);
    else
        GDN_RMS(8, 4);
#undef GDN_RMS
    return done();
}

gdn_status check(const gdn_norm_desc* d, bool norm) {
    if (!d || d->rows < 0 || d->C < 1) return GDN_ERR_INVALID_ARG;
    if (d->io_dtype != GDN_BF16 && d->io_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (norm && (!(d->eps > 0.0f) || !(d->eps < 1e30f))) return GDN_ERR_INVALID_ARG;
    if (norm && d->w_dtype != GDN_F32 && d->w_dtype != d->io_dtype) return GDN_ERR_INVALID_ARG;
    if (d->C > (1 << 20)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status run(const gdn_norm_desc* d, bool norm, const void* x, const void* residual, const void* weight, void* sum,
               void* y, float* y_scale, void* stream) {
    gdn_status st = check(d, norm);
    if (st != GDN_OK) return st;
    if (d->rows == 0) return GDN_OK;
    if (!x || !y || !y_scale) return GDN_ERR_INVALID_ARG;
    const int e = d->io_dtype == GDN_BF16 ? 2 : 4, we = norm && d->w_dtype == GDN_BF16 ? 2 : 4;
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(sum, e) || !aligned(weight, we) || !aligned(y_scale, 4))
        return GDN_ERR_ALIGNMENT;
    QuantArgs a = {};
    a.rows = d->rows, a.C = d->C, a.groups = (d->C + kGroup - 1) / kGroup, a.eps = d->eps;
    const size_t n = (size_t)d->rows * d->C;
    const Range ins[] = {rng(x, n * e), rng(residual, n * e), rng(weight, (size_t)d->C * we)};
    const Range outs[] = {rng(sum, n * e), rng(y, n), rng(y_scale, (size_t)d->rows * a.groups * 4)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j) {
            const bool same = i == 0 && j < 2 && ins[j].lo == outs[0].lo;   // the sum in place of a summand
            if (!same && overlap(outs[i], ins[j])) return GDN_ERR_ALIAS;
        }
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_ALIAS;
    }
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    a.x = x, a.r = residual, a.w = weight, a.sum = sum, a.y = static_cast<uint8_t*>(y), a.scale = y_scale;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f32 = d->io_dtype == GDN_F32;
    if (norm) {
        if (f32) return launch_norm<float, float>(a, cus, s);
        return d->w_dtype == GDN_F32 ? launch_norm<uint16_t, float>(a, cus, s) : launch_norm<uint16_t, uint16_t>(a, cus, s);
    }
    const int64_t per = kThreads / kLanes, all = (a.rows * a.groups + per - 1) / per;
    const dim3 grid((unsigned)std::min<int64_t>(all, (int64_t)cus * 16));
    if (f32)
        hipLaunchKernelGGL(quantise_kernel<float>, grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL(quantise_kernel<uint16_t>, grid, dim3(kThreads), 0, s, a);
    return done();
}

}  // namespace

extern "C" {

gdn_status gdn_rms_norm_fwd_fp8(const gdn_norm_desc* d, const void* x, const void* residual, const void* weight,
                                void* sum, void* y, float* y_scale, void* stream) {
    return run(d, true, x, residual, weight, sum, y, y_scale, stream);
}

gdn_status gdn_quantize_fp8(const gdn_norm_desc* d, const void* x, void* y, float* y_scale, void* stream) {
    return run(d, false, x, nullptr, nullptr, nullptr, y, y_scale, stream);
}

}  // extern "C"
