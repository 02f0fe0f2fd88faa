// Rotary positions over several axes: the C ABI of gdn_rotary (declared in
// include/gdn.h).
//
// Pair j of a head's rotated features belongs to one axis and turns by
// position * theta^(-2i/d) (i its index within the axis, d the axis' features):
//     (a, b) -> (a cos - b sin, a sin + b cos),   the inverse with sin negated.
// The rotation is orthogonal, so the inverse is also the gradient.
//
// Bound by memory: every feature is read and written once.  The angles depend
// on the token and the pair only, so a workgroup computes them once for its
// tokens (in 64 bits up to the reduction to one turn: at position 100,000 a
// 32-bit product would be off by 0.004 radians), keeps the cosines and sines
// in LDS, and all query and key heads use them.
#include "gdn_ops.hpp"

#include <math.h>

#include <algorithm>

namespace {

using namespace gdnops;

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;       // D up to 256
constexpr int kMaxTable = 4096;      // (token, pair) entries of a workgroup: 32 KiB of LDS

struct RotArgs {
    const void* x[2];                // q, k
    void* y[2];
    const void* pos;
    int64_t tokens, pos_rows;
    int heads[2];
    int D, pairs, axes, tb;          // tb: tokens per workgroup
    int pos_f32, inverse;
    int axis_pairs[GDN_ROTARY_MAX_AXES];
    double step[GDN_ROTARY_MAX_AXES];   // theta^(-2/d)
};

// Turns per position of pair j, theta^(-2i/d) / (2 pi), and its axis: a power
// by squaring.  Each squaring doubles what its base is off by, so step^i is off
// by about 2 i half steps of 2^-53 (the rounded step's i, and i of the squarings
// and products), 256 at most.  The angle is off by that share of itself and falls
// faster with i: at theta = 10^4 and positions up to 2^26 by less than the half
// step of 2^-26 turns that fp32 costs next.  (A table in the kernel's arguments
// made them 1.3 KB and the launch 3 us longer.)
__device__ __forceinline__ double turns_of(const RotArgs& a, int j, int& axis) {
    axis = 0;
#pragma unroll
    for (int x = 0; x < GDN_ROTARY_MAX_AXES - 1; ++x)
        if (axis == x && j >= a.axis_pairs[x]) {
            j -= a.axis_pairs[x];
            axis = x + 1;
        }
    double b = axis == 0 ? a.step[0] : axis == 1 ? a.step[1] : axis == 2 ? a.step[2] : a.step[3];
    double r = 0.15915494309189535;     // 1 / (2 pi)
#pragma unroll
    for (int bit = 0; bit < 7; ++bit) {
        if (j >> bit & 1) r *= b;
        b *= b;
    }
    return r;
}

template <typename T, int VW> struct VecN;     // VW consecutive elements, aligned
template <> struct VecN<uint16_t, 8> { using R = u32x4; };
template <> struct VecN<uint16_t, 4> { using R = u32x2; };
template <> struct VecN<uint16_t, 1> { using R = uint16_t; };
template <> struct VecN<float, 4> { using R = f32x4; };
template <> struct VecN<float, 1> { using R = float; };

template <int VW>
__device__ __forceinline__ void widen(u32x4 r, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(r[i] << 16);
        f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
}
template <int VW>
__device__ __forceinline__ void widen(u32x2 r, float* f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[2 * i] = __uint_as_float(r[i] << 16);
        f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
}
template <int VW>
__device__ __forceinline__ void widen(uint16_t r, float* f) { f[0] = bf2f(r); }
template <int VW>
__device__ __forceinline__ void widen(f32x4 r, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = r[i];
}
template <int VW>
__device__ __forceinline__ void widen(float r, float* f) { f[0] = r; }
__device__ __forceinline__ void narrow(const float* f, u32x4& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void narrow(const float* f, u32x2& r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) r[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void narrow(const float* f, uint16_t& r) { r = f2bf(f[0]); }
__device__ __forceinline__ void narrow(const float* f, f32x4& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = f[i];
}
__device__ __forceinline__ void narrow(const float* f, float& r) { r = f[0]; }

// HALVES: pairs (j, j + pairs); a thread turns VW pairs, two vectors of VW
// features.  Otherwise pairs (2j, 2j + 1) and one vector of VW features.
// A thread keeps its place within the head and takes (token, head) items in
// batches of four, loading a batch whole before it stores any of it: the
// outputs may be the inputs, so the compiler may not move a load past a store.
// Measured: 106480 tokens of 16 + 16 heads of 128, bf16, in 317 us (1.74 GB,
// 5.5 TB/s); 880 tokens in 6.9 us, of which the angles and one trip to memory
// are most.  LDS conflicts (table rows read by all heads) stay hidden.
template <typename T, int VW, bool HALVES>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotArgs a) {
    using R = typename VecN<T, VW>::R;
    constexpr int U = 4;
    __shared__ f32x2 table[kMaxTable];
    const int tid = threadIdx.x;
    const int P = a.pairs, D = a.D;
    const int64_t t0 = (int64_t)blockIdx.x * a.tb;
    const int nt = (int)min((int64_t)a.tb, a.tokens - t0);
    for (int i = tid; i < nt * P; i += kThreads) {
        const int tk = i / P, j = i - tk * P;
        int axis;
        const double turns = turns_of(a, j, axis);
        const int64_t at = ((t0 + tk) % a.pos_rows) * a.axes + axis;
        const double p = a.pos_f32 ? (double)static_cast<const float*>(a.pos)[at]
                                   : (double)static_cast<const int32_t*>(a.pos)[at];
        double u = p * turns;
        u -= rint(u);
        float sn, cs;
        sincospif(2.0f * (float)u, &sn, &cs);
        table[i] = f32x2{cs, a.inverse ? -sn : sn};
    }
    __syncthreads();
    // places within a head: the rotated ones first, then (HALVES) the features
    // that stay as they are, a vector each
    const int turned = HALVES ? P / VW : D / VW;
    const int places = HALVES ? turned + (D - 2 * P) / VW : turned;
    const int lanes = kThreads / places;                 // items at a time
    const int place = tid % places, i0 = tid / places;
    if (i0 >= lanes) return;
    const bool turns = place < turned;
    const int at = turns ? place * VW : 2 * P + (place - turned) * VW;
    const int HH = a.heads[0] + a.heads[1], items = nt * HH;
    for (int it = i0; it < items; it += lanes * U) {
        R r0[U], r1[U];
        T* y[U];
        int tk[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = min(it + u * lanes, items - 1);
            tk[u] = n / HH;
            const int h = n - tk[u] * HH, which = h >= a.heads[0];
            const size_t base =
                ((size_t)(t0 + tk[u]) * a.heads[which] + (which ? h - a.heads[0] : h)) * D + at;
            const T* x = static_cast<const T*>(a.x[which]) + base;
            y[u] = static_cast<T*>(a.y[which]) + base;
            r0[u] = *reinterpret_cast<const R*>(x);
            if constexpr (HALVES) r1[u] = *reinterpret_cast<const R*>(turns ? x + P : x);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (it + u * lanes >= items) break;
            const f32x2* cs = table + tk[u] * P;
            if constexpr (HALVES) {
                if (turns) {
                    float p[VW], q[VW], o[VW], v[VW];
                    widen<VW>(r0[u], p);
                    widen<VW>(r1[u], q);
#pragma unroll
                    for (int i = 0; i < VW; ++i) {
                        const f32x2 c = cs[at + i];
                        o[i] = p[i] * c[0] - q[i] * c[1];
                        v[i] = p[i] * c[1] + q[i] * c[0];
                    }
                    narrow(o, r0[u]);
                    narrow(v, r1[u]);
                    *reinterpret_cast<R*>(y[u] + P) = r1[u];
                }
            } else {
                float p[VW];
                widen<VW>(r0[u], p);
#pragma unroll
                for (int i = 0; i < VW / 2; ++i)
                    if (at / 2 + i < P) {
                        const f32x2 c = cs[at / 2 + i];
                        const float e = p[2 * i], o = p[2 * i + 1];
                        p[2 * i] = e * c[0] - o * c[1];
                        p[2 * i + 1] = e * c[1] + o * c[0];
                    }
                narrow(p, r0[u]);
            }
            *reinterpret_cast<R*>(y[u]) = r0[u];
        }
    }
}

gdn_status check_rotary(const gdn_rotary_desc* d, int* pairs) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->pos_rows < 0 || d->Hq < 0 || d->Hk < 0 || d->D < 1) return GDN_ERR_INVALID_ARG;
    if (d->n_axes < 1 || d->n_axes > GDN_ROTARY_MAX_AXES) return GDN_ERR_INVALID_ARG;
    if (d->io_dtype != GDN_BF16 && d->io_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (d->flags & ~(uint32_t)(GDN_FLAG_ROTARY_HALVES | GDN_FLAG_ROTARY_INVERSE | GDN_FLAG_ROTARY_POS_F32))
        return GDN_ERR_INVALID_ARG;
    if (!(d->theta > 0.0) || !(d->theta < 1e300)) return GDN_ERR_INVALID_ARG;
    int64_t r = 0;
    for (int i = 0; i < d->n_axes; ++i) {
        if (d->axis_dim[i] < 0 || d->axis_dim[i] % 2 || d->axis_dim[i] > d->D) return GDN_ERR_INVALID_ARG;
        r += d->axis_dim[i];
    }
    if (r > d->D || r == 0) return GDN_ERR_INVALID_ARG;
    if (d->D % 8 || d->D > 2 * kMaxPairs) return GDN_ERR_UNSUPPORTED;
    if (d->Hq > 65536 || d->Hk > 65536) return GDN_ERR_UNSUPPORTED;
    *pairs = (int)(r / 2);
    return GDN_OK;
}

template <typename T, int VW>
void launch(const RotArgs& a, bool halves, unsigned grid, hipStream_t s) {
    if (halves)
        hipLaunchKernelGGL((rotary_kernel<T, VW, true>), dim3(grid), dim3(kThreads), 0, s, a);
    else if constexpr (VW > 1)
        hipLaunchKernelGGL((rotary_kernel<T, VW, false>), dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace

extern "C" gdn_status gdn_rotary(const gdn_rotary_desc* d, const void* q, const void* k, const void* pos, void* q_out,
                                 void* k_out, void* stream) {
    int pairs;
    gdn_status st = check_rotary(d, &pairs);
    if (st != GDN_OK) return st;
    if (d->tokens == 0 || (d->Hq == 0 && d->Hk == 0)) return GDN_OK;
    if (d->pos_rows < 1) return GDN_ERR_INVALID_ARG;
    if (!pos || (d->Hq > 0 && (!q || !q_out)) || (d->Hk > 0 && (!k || !k_out))) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(pos, 4))
        return GDN_ERR_ALIGNMENT;
    const bool f32 = d->io_dtype == GDN_F32;
    const size_t e = f32 ? 4 : 2;
    const size_t qb = (size_t)d->tokens * d->Hq * d->D * e, kb = (size_t)d->tokens * d->Hk * d->D * e;
    const size_t pb = (size_t)std::min(d->pos_rows, d->tokens) * d->n_axes * 4;
    const Range rq = rng(q, qb), rk = rng(k, kb), rp = rng(pos, pb), oq = rng(q_out, qb), ok = rng(k_out, kb);
    if ((q_out != q && overlap(oq, rq)) || (k_out != k && overlap(ok, rk)) || overlap(oq, rk) || overlap(ok, rq) ||
        overlap(oq, ok) || overlap(oq, rp) || overlap(ok, rp))
        return GDN_ERR_ALIAS;
    const bool halves = (d->flags & GDN_FLAG_ROTARY_HALVES) != 0;
    RotArgs a = {};
    a.x[0] = q, a.x[1] = k, a.y[0] = q_out, a.y[1] = k_out, a.pos = pos;
    a.tokens = d->tokens, a.pos_rows = d->pos_rows;
    a.heads[0] = d->Hq, a.heads[1] = d->Hk;
    a.D = d->D, a.pairs = pairs, a.axes = d->n_axes;
    a.pos_f32 = (d->flags & GDN_FLAG_ROTARY_POS_F32) != 0;
    a.inverse = (d->flags & GDN_FLAG_ROTARY_INVERSE) != 0;
    for (int x = 0; x < d->n_axes; ++x) {
        a.axis_pairs[x] = d->axis_dim[x] / 2;
        a.step[x] = d->axis_dim[x] ? pow(d->theta, -2.0 / d->axis_dim[x]) : 1.0;
    }
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    // Tokens a workgroup: about 16 16-byte vectors a thread, so that the angles
    // are a small part, and fewer where the card would not be filled.
    const int64_t row = (int64_t)(d->Hq + d->Hk) * d->D * e;
    int64_t tb = std::max<int64_t>(1, (int64_t)16 * 16 * kThreads / row);
    tb = std::min<int64_t>(tb, kMaxTable / pairs);
    tb = std::min<int64_t>(tb, std::max<int64_t>(1, d->tokens / (4 * (int64_t)cus)));
    while ((d->tokens + tb - 1) / tb > INT32_MAX && tb < kMaxTable / pairs) tb *= 2;
    if ((d->tokens + tb - 1) / tb > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    a.tb = (int)std::min<int64_t>(tb, kMaxTable / pairs);
    const int64_t blocks = (d->tokens + a.tb - 1) / a.tb;
    if (blocks > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)blocks;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    // The widest vector (16 bytes at most) that the halves' distance allows.
    if (f32) {
        if (!halves || pairs % 4 == 0)
            launch<float, 4>(a, halves, grid, s);
        else
            launch<float, 1>(a, halves, grid, s);
    } else if (!halves || pairs % 8 == 0) {
        launch<uint16_t, 8>(a, halves, grid, s);
    } else if (pairs % 4 == 0) {
        launch<uint16_t, 4>(a, halves, grid, s);
    } else {
        launch<uint16_t, 1>(a, halves, grid, s);
    }
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
