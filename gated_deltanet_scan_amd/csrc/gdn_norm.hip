// Layer norm, forward and backward: the C ABI of gdn_layer_norm_fwd /
// gdn_layer_norm_bwd (declared in include/gdn.h).
//
//     mu = <x>,  r = (<(x - mu)^2> + eps)^(-1/2),  h = (x - mu) r,  y = h w + b
//     g = dy w,  dx = r (g - <g> - h <g h>),  dw = sum_rows dy h,  db = sum_rows dy
//
// Both passes are bound by memory: the forward reads x and writes y, the
// backward reads x and dy and writes dx.  A row stays in registers between its
// statistics and its result, so nothing is read twice; the variance is a second
// sum over the registers, about the mean (no cancellation of <x^2> - mu^2).
// One wave holds a row of up to 2048 elements, so rows of the usual widths need
// no barrier at all; four waves share a row of up to 16384, and wider rows are
// read again from memory (norm_wide_*).
#include "gdn_ops.hpp"

#include <algorithm>

namespace {

using namespace gdnops;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxPartials = 1024;   // workgroups of the backward pass (partial sums of dw and db)

struct NormArgs {
    const void* x;
    const void* dy;
    const void* w;
    const void* b;
    void* y;                         // y or dx
    float* mean;
    float* rstd;
    float* part;                     // [groups][2][C] partial sums of dw and db
    int64_t rows;
    int C;
    float eps, inv_c;
};

// Sum over the WPR waves of a row.  With WPR = 1 the wave's own sum; with four
// the waves add through LDS (two buffers, so one barrier a sum is enough).
template <int WPR>
__device__ __forceinline__ float row_sum(float x, float (*red)[kWaves], int& phase) {
    x = wave_sum(x);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) red[phase][threadIdx.x >> 6] = x;
        __syncthreads();
        x = (red[phase][0] + red[phase][1]) + (red[phase][2] + red[phase][3]);
        phase ^= 1;
    }
    return x;
}

template <int WPR>
__device__ __forceinline__ void row_sum2(float& x, float& y, float (*red)[2 * kWaves], int& phase) {
    x = wave_sum(x);
    y = wave_sum(y);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) {
            red[phase][threadIdx.x >> 6] = x;
            red[phase][kWaves + (threadIdx.x >> 6)] = y;
        }
        __syncthreads();
        x = (red[phase][0] + red[phase][1]) + (red[phase][2] + red[phase][3]);
        y = (red[phase][4] + red[phase][5]) + (red[phase][6] + red[phase][7]);
        phase ^= 1;
    }
}

// A lane's chunk of eight columns from c on.  ODD (C not a multiple of eight):
// the row's last chunk is moved back to end with the row, so that every access
// is a whole vector; its first `off` columns are then the lane before's too.
// They are left out of every sum and stored twice with the same bits.
template <bool ODD>
struct Chunk {
    int at, off;                                         // first column, columns that belong to another lane
    bool in;
    __device__ __forceinline__ Chunk(int c, int C) {
        in = c < C;
        at = ODD ? min(c, C - 8) : c;
        off = ODD ? c - at : 0;
    }
    __device__ __forceinline__ bool own(int j) const { return in && (!ODD || j >= off); }
    template <typename T>
    __device__ __forceinline__ void load(Vec8<T>& v, const T* row) const {
        if (in)
            v.load(row + at);
        else
            v.zero();
    }
    template <typename T>
    __device__ __forceinline__ void store(const Vec8<T>& v, T* row) const {
        if (in) v.store(row + at);
    }
};

// Rows of 8 to 512 * NV * WPR elements; lane t of a row holds the chunks of
// eight at 8 (t + 64 WPR i), i < NV.  Workgroups walk the rows with the
// weights in registers and the next row's loads in flight.
// Measured: 106480 x 2048 bf16 in 150 us (872 MB, 5.8 TB/s, some of x still in
// the caches); 880 x 2048 in 4.4 us, which is one trip to memory and the
// launch; 1777 x 1001 fp32 in 6.6 us.
template <typename T, typename W, int NV, int WPR, bool ODD>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[2][kWaves], red2[2][2 * kWaves];
    constexpr int RPB = kWaves / WPR;                    // rows per workgroup and step
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t = WPR == 1 ? (tid & 63) : tid;
    const int C = a.C;
    int phase = 0, phase2 = 0;
    auto at = [&](int i) { return Chunk<ODD>(8 * (t + 64 * WPR * i), C); };
    Vec8<W> w[NV], b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (a.w) at(i).load(w[i], static_cast<const W*>(a.w));
        if (a.b) at(i).load(b[i], static_cast<const W*>(a.b));
    }
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? wave : 0);
    Vec8<T> nxt[NV];
    if (row < a.rows) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            at(i).load(nxt[i], static_cast<const T*>(a.x) + row * C);
    }
    for (; row < a.rows; row += step) {
        Vec8<T> x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = nxt[i];
        if (row + step < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                at(i).load(nxt[i], static_cast<const T*>(a.x) + (row + step) * C);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += !ODD || at(i).own(j) ? x[i].get(j) : 0.f;   // x is zero past C
        float mu = row_sum<WPR>(s, red, phase) / (float)C;   // divided: rounded once, everywhere the same
        // spread about the rounded mean, and what that mean is off by: its
        // correction makes rows of a large mean exact to their own rounding
        float q = 0.f, e = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = at(i).own(j) ? x[i].get(j) - mu : 0.f;
                q += d * d;
                e += d;
            }
        row_sum2<WPR>(q, e, red2, phase2);
        e /= (float)C;
        mu += e;
        const float var = q * a.inv_c - e * e;
        const float r = 1.0f / sqrtf((var < 0.f ? 0.f : var) + a.eps);   // a NaN stays one
        T* yr = static_cast<T*>(a.y) + row * C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float h = (x[i].get(j) - mu) * r;
                f[j] = h * (a.w ? w[i].get(j) : 1.f) + (a.b ? b[i].get(j) : 0.f);
            }
            Vec8<T> y;
            y.set(f);
            at(i).store(y, yr);
        }
        if (t == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
    }
}

// The same layout for the backward pass.  Every lane adds dy h and dy of its
// columns over the workgroup's rows in fp32 registers; at the end the
// workgroup adds its waves' sums in order through LDS and writes one row of
// partial sums, which norm_colsum_kernel adds up (no atomics).
// Measured: 106480 x 2048 bf16 in 250 us (1.31 GB, 5.2 TB/s); 1777 x 1001 fp32
// in 9.6 us.
template <typename T, typename W, int NV, int WPR, bool ODD>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(const NormArgs a) {
    __shared__ float red[2][2 * kWaves];
    __shared__ float cols[WPR == 1 ? kWaves * 64 * 8 : 1];
    constexpr int RPB = kWaves / WPR;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t = WPR == 1 ? (tid & 63) : tid;
    const int C = a.C;
    int phase = 0;
    auto at = [&](int i) { return Chunk<ODD>(8 * (t + 64 * WPR * i), C); };
    Vec8<W> w[NV];
    float dw[NV][8], db[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (a.w) at(i).load(w[i], static_cast<const W*>(a.w));
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? wave : 0);
    Vec8<T> nx[NV], ny[NV];
    float nmu = 0.f, nr = 0.f;
    auto fetch = [&](int64_t rw) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            at(i).load(nx[i], static_cast<const T*>(a.x) + rw * C);
            at(i).load(ny[i], static_cast<const T*>(a.dy) + rw * C);
        }
        nmu = a.mean[rw];
        nr = a.rstd[rw];
    };
    constexpr bool AHEAD = NV < 8;                       // the widest rows leave no registers for a second one
    if (AHEAD && row < a.rows) fetch(row);
    for (; row < a.rows; row += step) {
        if (!AHEAD) fetch(row);
        Vec8<T> x[NV], dy[NV];
        const float mu = nmu, r = nr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = nx[i];
            dy[i] = ny[i];
        }
        if (AHEAD && row + step < a.rows) fetch(row + step);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = !ODD || at(i).own(j) ? dy[i].get(j) : 0.f, h = (x[i].get(j) - mu) * r;   // zero past C
                const float g = a.w ? d * w[i].get(j) : d;
                s1 += g;
                s2 += g * h;
                dw[i][j] += d * h;
                db[i][j] += d;
            }
        row_sum2<WPR>(s1, s2, red, phase);
        s1 *= a.inv_c;
        s2 *= a.inv_c;
        T* dxr = static_cast<T*>(a.y) + row * C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = dy[i].get(j), h = (x[i].get(j) - mu) * r;
                const float g = a.w ? d * w[i].get(j) : d;
                f[j] = r * ((g - s1) - h * s2);
            }
            Vec8<T> v;
            v.set(f);
            at(i).store(v, dxr);
        }
    }
    if (!a.part) return;
    float* pw = a.part + (size_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float* v = k ? db[i] : dw[i];
            if constexpr (WPR == 1) {
                // the four waves hold the same columns: add them in order
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; ++j) cols[(wave * 8 + j) * 64 + t] = v[j];
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = tid + 256 * e, j = n >> 6, l = n & 63;
                    const Chunk<ODD> c(8 * (l + 64 * i), C);
                    const float s = (cols[j * 64 + l] + cols[(8 + j) * 64 + l]) +
                                    (cols[(16 + j) * 64 + l] + cols[(24 + j) * 64 + l]);
                    if (c.own(j)) pw[(size_t)k * C + c.at + j] = s;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at(i).own(j)) pw[(size_t)k * C + at(i).at + j] = v[j];
            }
        }
}

// Rows wider than a workgroup's registers (V = 8), or narrower than a chunk
// (V = 1): one workgroup a row, which reads it three times (statistics, spread,
// result; the later reads hit the caches).  As in Chunk, the last vector of a
// row moves back to end with it and its first columns count once.
// Measured: 8192 x 32768 bf16 forward in 310 us, dx in 436 (one column a
// thread at a time: 778 and 734).
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float* f) {
    if constexpr (V == 8) {
        Vec8<T> v;
        v.load(p);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v.get(j);
    } else {
        f[0] = to_f<T>(p[0]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* f) {
    if constexpr (V == 8) {
        Vec8<T> v;
        v.set(f);
        v.store(p);
    } else {
        p[0] = from_f<T>(f[0]);
    }
}
// at: first column; own: the first of its V that counts
template <int V, typename F>
__device__ __forceinline__ void each_v(int C, F f) {
    for (int c = V * (int)threadIdx.x; c < C; c += V * kThreads) {
        const int at = min(c, C - V);
        f(at, c - at);
    }
}
template <typename T, typename W, int V>
__global__ __launch_bounds__(kThreads) void norm_wide_fwd_kernel(const NormArgs a) {
    __shared__ float red[2][kWaves], red2[2][2 * kWaves];
    int phase = 0, phase2 = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.C;
        T* y = static_cast<T*>(a.y) + row * a.C;
        float s = 0.f, q = 0.f, e = 0.f;
        each_v<V>(a.C, [&](int at, int own) {
            float f[V];
            load_v<T, V>(x + at, f);
#pragma unroll
            for (int j = 0; j < V; ++j) s += j >= own ? f[j] : 0.f;
        });
        float mu = row_sum<4>(s, red, phase) / (float)a.C;
        each_v<V>(a.C, [&](int at, int own) {
            float f[V];
            load_v<T, V>(x + at, f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = j >= own ? f[j] - mu : 0.f;
                q += d * d;
                e += d;
            }
        });
        row_sum2<4>(q, e, red2, phase2);
        e /= (float)a.C;
        mu += e;
        const float var = q * a.inv_c - e * e;
        const float r = 1.0f / sqrtf((var < 0.f ? 0.f : var) + a.eps);
        each_v<V>(a.C, [&](int at, int) {
            float f[V], w[V], b[V];
            load_v<T, V>(x + at, f);
            if (a.w) load_v<W, V>(static_cast<const W*>(a.w) + at, w);
            if (a.b) load_v<W, V>(static_cast<const W*>(a.b) + at, b);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = (f[j] - mu) * r;
                f[j] = h * (a.w ? w[j] : 1.f) + (a.b ? b[j] : 0.f);
            }
            store_v<T, V>(y + at, f);
        });
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
    }
}
template <typename T, typename W, int V>
__global__ __launch_bounds__(kThreads) void norm_wide_dx_kernel(const NormArgs a) {
    __shared__ float red[2][2 * kWaves];
    int phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.C;
        const T* dy = static_cast<const T*>(a.dy) + row * a.C;
        T* dx = static_cast<T*>(a.y) + row * a.C;
        const float mu = a.mean[row], r = a.rstd[row];
        float s1 = 0.f, s2 = 0.f;
        auto terms = [&](int at, float* g, float* h) {    // dy w and the normalised x
            float w[V];
            load_v<T, V>(dy + at, g);
            load_v<T, V>(x + at, h);
            if (a.w) load_v<W, V>(static_cast<const W*>(a.w) + at, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (a.w) g[j] *= w[j];
                h[j] = (h[j] - mu) * r;
            }
        };
        each_v<V>(a.C, [&](int at, int own) {
            float g[V], h[V];
            terms(at, g, h);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s1 += j >= own ? g[j] : 0.f;
                s2 += j >= own ? g[j] * h[j] : 0.f;
            }
        });
        row_sum2<4>(s1, s2, red, phase);
        s1 *= a.inv_c;
        s2 *= a.inv_c;
        each_v<V>(a.C, [&](int at, int) {
            float g[V], h[V];
            terms(at, g, h);
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = r * ((g[j] - s1) - h[j] * s2);
            store_v<T, V>(dx + at, g);
        });
    }
}
// dw and db of wide rows: one thread a column, workgroup y takes every
// gridDim.y-th row.  8192 x 32768 bf16 in 329 us (1.07 GB, 3.3 TB/s).
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_wide_dw_kernel(const NormArgs a) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.C) return;
    float dw = 0.f, db = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float d = to_f<T>(static_cast<const T*>(a.dy)[row * a.C + c]);
        dw += d * ((to_f<T>(static_cast<const T*>(a.x)[row * a.C + c]) - a.mean[row]) * a.rstd[row]);
        db += d;
    }
    float* pw = a.part + (size_t)blockIdx.y * 2 * a.C;
    pw[c] = dw;
    pw[a.C + c] = db;
}

// dw[c] = sum over the groups' partial rows, 64 columns a workgroup; its 16
// waves take every sixteenth row and add up through LDS in order.  All of it in
// fp32: sums of a few dozen to a few hundred terms one after the other, 1.4e-7 off
// in the Frobenius norm at 1777 rows where 64-bit sums are 0.8e-7.  Bound by the
// latency of those rows: 1024 of 2 x 2048 (16 MiB, in the caches) in 10 us.
constexpr int kColWaves = 16;
template <typename W>
__global__ __launch_bounds__(64 * kColWaves) void norm_colsum_kernel(const float* __restrict__ part, int groups, int C,
                                                                     W* __restrict__ dw, W* __restrict__ db) {
    __shared__ float red[kColWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = blockIdx.x * 64 + lane;                // columns of [2][C]
    float s = 0.f;
    if (n < 2 * C) {
        float u[4] = {0.f, 0.f, 0.f, 0.f};
        int p = wave;
        for (; p + 3 * kColWaves < groups; p += 4 * kColWaves)
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] += part[(size_t)(p + i * kColWaves) * 2 * C + n];
        for (; p < groups; p += kColWaves) u[0] += part[(size_t)p * 2 * C + n];
        s = (u[0] + u[1]) + (u[2] + u[3]);
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && n < 2 * C) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < kColWaves; ++w) s += red[w][lane];
        if (n < C) {
            if (dw) dw[n] = from_f<W>(s);
        } else if (db) {
            db[n - C] = from_f<W>(s);
        }
    }
}

// ---------------------------------------------------------------- launch
gdn_status check_norm(const gdn_norm_desc* d) {
    if (!d || d->rows < 0 || d->C < 1) return GDN_ERR_INVALID_ARG;
    if (!(d->eps > 0.0f) || !(d->eps < 1e30f)) return GDN_ERR_INVALID_ARG;
    if (d->io_dtype != GDN_BF16 && d->io_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (d->w_dtype != GDN_F32 && d->w_dtype != d->io_dtype) return GDN_ERR_INVALID_ARG;
    if (d->C > (1 << 20)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
int elem(int dt) { return dt == GDN_BF16 ? 2 : 4; }

// Waves a row and chunks a lane: the smallest that hold the row.  (Eight chunks
// a lane in one wave leave a SIMD a single wave: 20000 x 4096 forward and
// backward took 195 us so, and takes 179 us.)
bool shape_of(int C, int* nv, int* wpr) {
    if (C < 8) return false;
    for (int w = 1; w <= 4; w *= 4)
        for (int v = 1; v <= (w == 1 ? 4 : 8); v *= 2)
            if (C <= 512 * v * w) {
                *nv = v;
                *wpr = w;
                return true;
            }
    return false;
}
// Workgroups of the backward pass: one a compute unit first, then as many as
// leave each wave a few rows (up to four a unit), since every workgroup writes
// a row of partial sums that is read back (64 MiB of them at most, or 16
// rows).
int bwd_groups(const gdn_norm_desc* d) {
    int nv = 0, wpr = 4;
    shape_of(d->C, &nv, &wpr);
    const int64_t rpb = kWaves / wpr;
    const int64_t g = std::max((d->rows + 4 * rpb - 1) / (4 * rpb),
                               std::min<int64_t>((d->rows + rpb - 1) / rpb, 256));
    const int64_t most = std::min<int64_t>(kMaxPartials, std::max<int64_t>(16, ((int64_t)64 << 20) / (8 * (int64_t)d->C)));
    return (int)std::min(std::max<int64_t>(g, 1), most);
}

template <typename T, typename W>
gdn_status launch_fwd(const NormArgs& a, int cus, hipStream_t s) {
    int nv, wpr;
    if (!shape_of(a.C, &nv, &wpr)) {
        const int64_t grid = std::min<int64_t>(a.rows, (int64_t)cus * 8);
        if (a.C < 8)
            hipLaunchKernelGGL((norm_wide_fwd_kernel<T, W, 1>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
        else
            hipLaunchKernelGGL((norm_wide_fwd_kernel<T, W, 8>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
        return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
    }
    const int rpb = kWaves / wpr;
    const dim3 grid((unsigned)std::min<int64_t>((a.rows + rpb - 1) / rpb, (int64_t)cus * 4));
#define GDN_NORM(NV, WPR)                                                                                       \
    do {                                                                                                        \
        if (a.C % 8)                                                                                            \
            hipLaunchKernelGGL((norm_fwd_kernel<T, W, NV, WPR, true>), grid, dim3(kThreads), 0, s, a);          \
        else                                                                                                    \
            hipLaunchKernelGGL((norm_fwd_kernel<T, W, NV, WPR, false>), grid, dim3(kThreads), 0, s, a);         \
    } while (0)
    if (wpr == 1) {
        if (nv == 1) GDN_NORM(1, 1);
        if (nv == 2) GDN_NORM(2, 1);
        if (nv == 4) GDN_NORM(4, 1);
    } else {
        if (nv == 2) GDN_NORM(2, 4);
        if (nv == 4) GDN_NORM(4, 4);
        if (nv == 8) GDN_NORM(8, 4);
    }
#undef GDN_NORM
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <typename T, typename W>
gdn_status launch_bwd(const NormArgs& a, int groups, void* dw, void* db, int cus, hipStream_t s) {
    int nv, wpr;
    if (a.rows > 0) {
        if (!shape_of(a.C, &nv, &wpr)) {
            const int64_t grid = std::min<int64_t>(a.rows, (int64_t)cus * 8);
            if (a.C < 8)
                hipLaunchKernelGGL((norm_wide_dx_kernel<T, W, 1>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
            else
                hipLaunchKernelGGL((norm_wide_dx_kernel<T, W, 8>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
            if (a.part)
                hipLaunchKernelGGL(norm_wide_dw_kernel<T>, dim3((a.C + kThreads - 1) / kThreads, groups),
                                   dim3(kThreads), 0, s, a);
        } else {
            const dim3 grid(groups);
#define GDN_NORM(NV, WPR)                                                                                       \
    do {                                                                                                        \
        if (a.C % 8)                                                                                            \
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, NV, WPR, true>), grid, dim3(kThreads), 0, s, a);          \
        else                                                                                                    \
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, NV, WPR, false>), grid, dim3(kThreads), 0, s, a);         \
    } while (0)
            if (wpr == 1) {
                if (nv == 1) GDN_NORM(1, 1);
                if (nv == 2) GDN_NORM(2, 1);
                if (nv == 4) GDN_NORM(4, 1);
            } else {
                if (nv == 2) GDN_NORM(2, 4);
                if (nv == 4) GDN_NORM(4, 4);
                if (nv == 8) GDN_NORM(8, 4);
            }
#undef GDN_NORM
        }
        if (hipGetLastError() != hipSuccess) return GDN_ERR_LAUNCH;
    }
    if (dw || db) {
        hipLaunchKernelGGL(norm_colsum_kernel<W>, dim3((2 * a.C + 63) / 64), dim3(64 * kColWaves), 0, s, a.part,
                           a.rows > 0 ? groups : 0, a.C, static_cast<W*>(dw), static_cast<W*>(db));
        if (hipGetLastError() != hipSuccess) return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_layer_norm_fwd(const gdn_norm_desc* d, const void* x, const void* weight, const void* bias, void* y,
                              float* mean, float* rstd, void* stream) {
    gdn_status st = check_norm(d);
    if (st != GDN_OK) return st;
    if (d->rows == 0) return GDN_OK;
    if (!x || !y) return GDN_ERR_INVALID_ARG;
    const int e = elem(d->io_dtype), we = elem(d->w_dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(weight, we) || !aligned(bias, we) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return GDN_ERR_ALIGNMENT;
    const size_t nb = (size_t)d->rows * d->C * e, wb = (size_t)d->C * we, sb = (size_t)d->rows * 4;
    const Range ins[] = {rng(x, nb), rng(weight, wb), rng(bias, wb)};
    const Range outs[] = {rng(y, nb), rng(mean, sb), rng(rstd, sb)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return GDN_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_ALIAS;
    }
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    NormArgs a = {};
    a.x = x, a.w = weight, a.b = bias, a.y = y, a.mean = mean, a.rstd = rstd;
    a.rows = d->rows, a.C = d->C, a.eps = d->eps, a.inv_c = 1.0f / (float)d->C;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (d->io_dtype == GDN_F32) return launch_fwd<float, float>(a, cus, s);
    return d->w_dtype == GDN_F32 ? launch_fwd<uint16_t, float>(a, cus, s) : launch_fwd<uint16_t, uint16_t>(a, cus, s);
}

size_t gdn_layer_norm_workspace_size(const gdn_norm_desc* d) {
    if (check_norm(d) != GDN_OK || d->rows == 0) return 0;
    return round256((size_t)bwd_groups(d) * 2 * d->C * sizeof(float));
}

gdn_status gdn_layer_norm_bwd(const gdn_norm_desc* d, const void* dy, const void* x, const void* weight,
                              const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                              void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status st = check_norm(d);
    if (st != GDN_OK) return st;
    const bool sums = dweight || dbias;
    if (d->rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return GDN_ERR_INVALID_ARG;
    const int e = elem(d->io_dtype), we = elem(d->w_dtype);
    if (!aligned(dy, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(weight, we) || !aligned(dweight, we) ||
        !aligned(dbias, we) || !aligned(mean, 4) || !aligned(rstd, 4))
        return GDN_ERR_ALIGNMENT;
    const size_t need = sums ? gdn_layer_norm_workspace_size(d) : 0;
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
    const size_t nb = (size_t)d->rows * d->C * e, wb = (size_t)d->C * we, sb = (size_t)d->rows * 4;
    const Range ins[] = {rng(dy, nb), rng(x, nb), rng(weight, wb), rng(mean, sb), rng(rstd, sb)};
    const Range outs[] = {rng(dx, nb), rng(dweight, wb), rng(dbias, wb), rng(need ? workspace : nullptr, need)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return GDN_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_ALIAS;
    }
    if (d->rows == 0 && !sums) return GDN_OK;
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    NormArgs a = {};
    a.x = x, a.dy = dy, a.w = weight, a.y = dx, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.part = need ? static_cast<float*>(workspace) : nullptr;
    a.rows = d->rows, a.C = d->C, a.eps = d->eps, a.inv_c = 1.0f / (float)d->C;
    const int groups = d->rows > 0 ? bwd_groups(d) : 0;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (d->io_dtype == GDN_F32) return launch_bwd<float, float>(a, groups, dweight, dbias, cus, s);
    return d->w_dtype == GDN_F32 ? launch_bwd<uint16_t, float>(a, groups, dweight, dbias, cus, s)
                                 : launch_bwd<uint16_t, uint16_t>(a, groups, dweight, dbias, cus, s);
}

}  // extern "C"
