// Softmax attention, forward and backward: the C ABI of gdn_attn_fwd /
// gdn_attn_bwd (declared in include/gdn.h), and the kernels in fp32 matrix
// instructions.
//
//     S = scale q k^T,  P = softmax over the visible keys,  o = P v
//     dP = d_o v^T,  dS = P (dP - <d_o, o>)
//     dq = scale dS k,  dk = scale dS^T q,  dv = P^T d_o
//
// The forward pass keeps a running maximum and sum per row, so P never leaves
// the registers; the backward pass forms P again from the saved logarithm of
// the sum.  dq and (dk, dv) are two kernels, each summing in its own registers
// in a fixed order (no atomics; S and dP are formed twice).
//
// v_mfma_f32_16x16x4_f32: lane l = 16 g + r holds operand A[row r][k = g] and
// B[k = g][column r]; the result sits in lane l as rows 4g..4g+3 of column r.
// Scores are formed transposed (keys as rows, the wave's 16 query rows as
// columns), so the four values that a lane holds are the B operands of the
// next product, key 4g + i for its i-th: P needs no trip through LDS.
// The feature axis is contracted in the order 16 s + 4 g + j, which lets a
// lane read four features at once.
#include "gdn_attn.hpp"

#include <algorithm>

namespace {

using namespace gdnattn;

constexpr int kThreads = 256;
constexpr int kRows = 64;     // query rows (or keys, in the dk/dv kernel) per workgroup: 16 a wave
constexpr int kTile = 32;     // keys (or rows) staged in LDS at a time

__device__ __forceinline__ f32x4 mma(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
    const u32x2 r = *reinterpret_cast<const u32x2*>(p);
    return f32x4{__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u), __uint_as_float(r[1] << 16),
                 __uint_as_float(r[1] & 0xffff0000u)};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
// Over the four lanes that hold one column.
__device__ __forceinline__ float col_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float col_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// Row r of the packed row axis of kv head hk: its global (token, head) row.
__device__ __forceinline__ int64_t packed_row(const AttnArgs& a, const Seq& z, int hk, int r) {
    return (z.q0 + r / a.G) * a.Hq + hk * a.G + r % a.G;
}
template <typename T>
__device__ __forceinline__ const T* q_row(const AttnArgs& a, const Seq& z, int hk, int r) {
    return static_cast<const T*>(a.q) + (z.q0 + r / a.G) * a.ldq + (int64_t)(hk * a.G + r % a.G) * a.D;
}

// The lane's share of one row, features 16 s + 4 g .. + 3 for every s.
template <typename T, int D>
__device__ __forceinline__ void row_frag(f32x4 (&f)[D / 16], const T* row, bool valid, int g) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) f[s] = valid ? load4(row + 16 * s + 4 * g) : f32x4{0.f, 0.f, 0.f, 0.f};
}

// Rows [n0, n0 + kTile) of a key tensor, zeros from hi on: to registers while
// the tile before is computed on, then to LDS as fp32.
template <typename T, int D>
struct Stage {
    static constexpr int C = kTile * D / 4, N = (C + kThreads - 1) / kThreads;
    f32x4 x[N];
    __device__ __forceinline__ void load(const T* base, int64_t ld, int n0, int hi) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (int)threadIdx.x + j * kThreads, n = c / (D / 4), e = c % (D / 4) * 4;
            x[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (n0 + n < hi && c < C) x[j] = load4(base + (int64_t)(n0 + n) * ld + e);
        }
    }
    __device__ __forceinline__ void store(float (*t)[D + 4]) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (int)threadIdx.x + j * kThreads;
            if (c < C) store4(&t[c / (D / 4)][c % (D / 4) * 4], x[j]);
        }
    }
};

// The lane's features of one row times its own, and the sum over the column.
template <typename T, int D>
__device__ __forceinline__ float dot_row(const f32x4 (&f)[D / 16], const T* row, int g) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
        const f32x4 x = load4(row + 16 * e + 4 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j) s += x[j] * f[e][j];
    }
    return col_sum(s);
}

// Bound by the fp32 matrix instructions (154 TFLOP/s in a large product) and,
// of two waves a SIMD, the wait between them: 4096 x 4096, 16 heads of 128, no
// mask: 1326 us, 104 TFLOP/s (D = 64: 102, D = 32: 85).
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_fwd_f32_kernel(const AttnArgs a) {
    __shared__ float kt[kTile][D + 4], vt[kTile][D + 4];
    const Place p = find_place<false>(a, kRows);
    if (p.s < 0) return;
    const Seq z = sequence(a, p.s);
    const int rows = z.lq * a.G, r0 = p.tile * kRows;
    if (r0 >= rows) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int row = r0 + 16 * wave + c;
    const bool valid = row < rows;
    const int n = valid ? visible(a, z, row / a.G) : 0;
    const int upto = visible(a, z, (min(r0 + kRows, rows) - 1) / a.G);
    const int lo = min(p.split * a.chunk, upto), hi = min(lo + a.chunk, upto);
    if (p.split > 0 && p.split * a.chunk >= z.lk) return;     // a shorter sequence has fewer splits
    f32x4 q[D / 16], acc[D / 16];
    row_frag<T, D>(q, valid ? q_row<T>(a, z, p.hk, row) : nullptr, valid, g);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) acc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    const T* kb = static_cast<const T*>(a.k) + z.k0 * a.ldk + (int64_t)p.hk * D;
    const T* vb = static_cast<const T*>(a.v) + z.k0 * a.ldv + (int64_t)p.hk * D;
    const float c2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    Stage<T, D> sk, sv;
    sk.load(kb, a.ldk, lo, hi);
    sv.load(vb, a.ldv, lo, hi);
    for (int n0 = lo; n0 < hi; n0 += kTile) {
        __syncthreads();
        sk.store(kt);
        sv.store(vt);
        __syncthreads();
        sk.load(kb, a.ldk, n0 + kTile, hi);
        sv.load(vb, a.ldv, n0 + kTile, hi);
        f32x4 s[2];
        float mt = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                const f32x4 kf = load4(&kt[16 * t + c][16 * e + 4 * g]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[t] = mma(kf[j], q[e][j], s[t]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (n0 + 16 * t + 4 * g + i >= n) s[t][i] = -INFINITY;
                mt = fmaxf(mt, s[t][i]);
            }
        }
        mt = fmaxf(m, col_max(mt) * c2);
        const float ms = mt == -INFINITY ? 0.f : mt;      // nothing visible so far
        const float al = exp2_f(m - ms);
        m = mt;
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[t][i] = exp2_f(__builtin_fmaf(s[t][i], c2, -ms));
                sum += s[t][i];
            }
        l = l * al + sum;                                 // this lane's keys; joined at the end
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[e] *= al;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < D / 16; ++e) acc[e] = mma(vt[16 * t + 4 * g + i][16 * e + c], s[t][i], acc[e]);
    }
    if (a.causal && !finite(acc)) {                           // see finite()
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int j = lo; j < hi; ++j) {
            const float s = dot_row<T, D>(q, kb + (int64_t)j * a.ldk, g) * c2;
            if (j < n) {
                const float mn = fmaxf(m, s), ms = mn == -INFINITY ? 0.f : mn;
                const float al = exp2_f(m - ms), pj = exp2_f(s - ms);
                m = mn;
                l = l * al + (g == 0 ? pj : 0.f);
#pragma unroll
                for (int e = 0; e < D / 16; ++e)
                    acc[e] = acc[e] * al + pj * load4(vb + (int64_t)j * a.ldv + 16 * e + 4 * g);
            }
        }
    }
    l = col_sum(l);
    if (!valid) return;
    const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
    const float ls = l == 0.f ? -INFINITY : (m + log2_f(l)) * kLn2;
    const int64_t gr = packed_row(a, z, p.hk, row);
    if (a.splits > 1) {
        const int64_t pr = (int64_t)p.split * a.total_q * a.Hq + gr;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) store4(a.part_o + pr * D + 16 * e + 4 * g, acc[e] * inv);
        if (g == 0) a.part_lse[pr] = ls;
        return;
    }
#pragma unroll
    for (int e = 0; e < D / 16; ++e) store4(static_cast<T*>(a.out) + gr * D + 16 * e + 4 * g, acc[e] * inv);
    if (g == 0 && a.lse) a.lse[gr] = ls;
}

// o = sum over the splits of exp(lse_s - lse) o_s, a wave a row.  Every lane
// weighs one split (64 at a time), then each quarter of the wave adds every
// fourth split's row, several loads in flight; the quarters add up in order.
// The rows are the sequences' own, so what lies behind the last is left alone.
// Bound by the latency of a few dependent trips to the partial results: 8
// single queries of 32 heads in 8.5 us, 880 of 16 heads in 9.5.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(const AttnArgs a) {
    constexpr int E = (D + 63) / 64;
    const int per = a.join_rows;
    const int tiles = (int)(((int64_t)a.max_q * a.Hq + per - 1) / per);
    const Seq z = sequence(a, (int)(blockIdx.x / (unsigned)tiles));
    const int lane = threadIdx.x & 63, g = lane >> 4, c = 4 * (lane & 15);
    const int64_t r0 = (int64_t)(blockIdx.x % (unsigned)tiles) * per, end = min(r0 + per, (int64_t)z.lq * a.Hq);
    for (int64_t r = r0 + (threadIdx.x >> 6); r < end; r += kThreads / 64) {
        const int64_t gr = z.q0 * a.Hq + r, all = a.total_q * a.Hq;
        const int splits = max(1, (z.lk + a.chunk - 1) / a.chunk);
        float m = -INFINITY, l = 0.f;
        f32x4 acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < splits; s0 += 64) {
            const float pl = s0 + lane < splits ? a.part_lse[(s0 + lane) * all + gr] : -INFINITY;
            float top = pl;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
            top = fmaxf(top, m);
            const float ms = top == -INFINITY ? 0.f : top;
            const float w = exp2_f((pl - ms) * kLog2e), al = exp2_f((m - ms) * kLog2e);   // 0 for a split that saw nothing
            m = top;
            l = l * al + wave_sum(w);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= al;
            const int n = min(64, splits - s0);
            // every lane takes part in every exchange: a lane that had left the loop
            // early would no longer hand out its split's weight
#pragma unroll 4
            for (int i0 = 0; i0 < n; i0 += 4) {
                const float wi = __shfl(w, i0 + g);           // 0 past the last split
                const int64_t row = (s0 + min(i0 + g, n - 1)) * all + gr;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (64 * e + c < D) acc[e] += wi * load4(a.part_o + row * D + 64 * e + c);
            }
        }
        const float inv = l > 0.f ? 1.0f / l : l;
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[e][j] += __shfl_xor(acc[e][j], 16);
                acc[e][j] += __shfl_xor(acc[e][j], 32);
            }
            if (g == 0 && 64 * e + c < D) store4(static_cast<T*>(a.out) + gr * D + 64 * e + c, acc[e] * inv);
        }
        if (lane == 0 && a.lse) a.lse[gr] = l == 0.f ? -INFINITY : m + log2_f(l) * kLn2;
    }
}

// dq, and <d_o, o> for the dk/dv kernel: query rows as columns, as in the
// forward kernel.  4096 x 4096, 16 heads of 128: 1659 us, 124 TFLOP/s of 6 D
// flops a pair.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_dq_f32_kernel(const AttnArgs a) {
    __shared__ float kt[kTile][D + 4], vt[kTile][D + 4];
    const Place p = find_place<false>(a, kRows);
    if (p.s < 0) return;
    const Seq z = sequence(a, p.s);
    const int rows = z.lq * a.G, r0 = p.tile * kRows;
    if (r0 >= rows) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int row = r0 + 16 * wave + c;
    const bool valid = row < rows;
    const int n = valid ? visible(a, z, row / a.G) : 0;
    const int upto = visible(a, z, (min(r0 + kRows, rows) - 1) / a.G);
    const int64_t gr = packed_row(a, z, p.hk, valid ? row : r0);
    f32x4 q[D / 16], dout[D / 16], acc[D / 16];
    row_frag<T, D>(q, valid ? q_row<T>(a, z, p.hk, row) : nullptr, valid, g);
    row_frag<T, D>(dout, static_cast<const T*>(a.d_o) + gr * D, valid, g);
    float delta = 0.f;
    {
        f32x4 o[D / 16];
        row_frag<T, D>(o, static_cast<const T*>(a.o) + gr * D, valid, g);
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
#pragma unroll
            for (int j = 0; j < 4; ++j) delta += dout[e][j] * o[e][j];
    }
    delta = col_sum(delta);
    if (valid && g == 0) a.delta[gr] = delta;
    const float c2 = a.scale * kLog2e;
    float ls = valid ? a.lse[gr] * kLog2e : -INFINITY;
    const int nn = ls == -INFINITY ? 0 : n;
    if (ls == -INFINITY) ls = 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    const T* kb = static_cast<const T*>(a.k) + z.k0 * a.ldk + (int64_t)p.hk * D;
    const T* vb = static_cast<const T*>(a.v) + z.k0 * a.ldv + (int64_t)p.hk * D;
    Stage<T, D> sk, sv;
    sk.load(kb, a.ldk, 0, upto);
    sv.load(vb, a.ldv, 0, upto);
    for (int n0 = 0; n0 < upto; n0 += kTile) {
        __syncthreads();
        sk.store(kt);
        sv.store(vt);
        __syncthreads();
        sk.load(kb, a.ldk, n0 + kTile, upto);
        sv.load(vb, a.ldv, n0 + kTile, upto);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f}, dp = s;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                const f32x4 kf = load4(&kt[16 * t + c][16 * e + 4 * g]), vf = load4(&vt[16 * t + c][16 * e + 4 * g]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s = mma(kf[j], q[e][j], s);
                    dp = mma(vf[j], dout[e][j], dp);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float pr = exp2_f(__builtin_fmaf(s[i], c2, -ls));
                const float ds = n0 + 16 * t + 4 * g + i < nn ? pr * (dp[i] - delta) : 0.f;
#pragma unroll
                for (int e = 0; e < D / 16; ++e) acc[e] = mma(kt[16 * t + 4 * g + i][16 * e + c], ds, acc[e]);
            }
        }
    }
    if (a.causal && !finite(acc)) {                           // see finite()
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int j = 0; j < upto; ++j) {
            const T* kr = kb + (int64_t)j * a.ldk;
            const float s = dot_row<T, D>(q, kr, g), dp = dot_row<T, D>(dout, vb + (int64_t)j * a.ldv, g);
            if (j < nn) {
                const float ds = exp2_f(__builtin_fmaf(s, c2, -ls)) * (dp - delta);
#pragma unroll
                for (int e = 0; e < D / 16; ++e) acc[e] += ds * load4(kr + 16 * e + 4 * g);
            }
        }
    }
    if (!valid) return;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) store4(static_cast<T*>(a.dq) + gr * D + 16 * e + 4 * g, acc[e] * a.scale);
}

// dk and dv: a wave's 16 keys as columns, the packed query rows staged in LDS.
// 4096 x 4096, 16 heads of 128: 2744 us, 100 TFLOP/s of 8 D flops a pair (one
// wave a SIMD at D = 128: K, V and both sums take 300 registers).
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_dkv_f32_kernel(const AttnArgs a) {
    __shared__ float qt[kTile][D + 4], dt[kTile][D + 4];
    __shared__ float ls[kTile], dl[kTile];
    __shared__ int nv[kTile];
    const Place p = find_place<true>(a, kRows);
    if (p.s < 0) return;
    const Seq z = sequence(a, p.s);
    const int k0 = p.tile * kRows;
    if (k0 >= z.lk) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int key = k0 + 16 * wave + c;
    const bool valid = key < z.lk;
    f32x4 kf[D / 16], vf[D / 16], ak[D / 16], av[D / 16];
    row_frag<T, D>(kf, static_cast<const T*>(a.k) + (z.k0 + key) * a.ldk + (int64_t)p.hk * D, valid, g);
    row_frag<T, D>(vf, static_cast<const T*>(a.v) + (z.k0 + key) * a.ldv + (int64_t)p.hk * D, valid, g);
#pragma unroll
    for (int e = 0; e < D / 16; ++e) ak[e] = av[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float c2 = a.scale * kLog2e;
    const int rows = z.lq * a.G;
    int start = min(first_query(a, z, k0) * a.G, rows), end = rows;
    if (a.k_splits > 1) {
        int lo, hi;
        split_range(rows - start, kTile, a.k_splits, p.split, lo, hi);
        end = start + hi;
        start += lo;
    }
    constexpr int C = kTile * D / 4, N = (C + kThreads - 1) / kThreads;
    f32x4 xq[N], xd[N];
    float xl = 0.f, xs = 0.f;
    int xn = 0;
    auto load = [&](int r0) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int x = (int)threadIdx.x + j * kThreads, r = r0 + x / (D / 4), e = x % (D / 4) * 4;
            xq[j] = xd[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (x < C && r < end) {
                xq[j] = load4(q_row<T>(a, z, p.hk, r) + e);
                xd[j] = load4(static_cast<const T*>(a.d_o) + packed_row(a, z, p.hk, r) * D + e);
            }
        }
        const int r = r0 + (int)threadIdx.x;
        xl = xs = 0.f;
        xn = 0;
        if (threadIdx.x < kTile && r < end) {
            const int64_t gr = packed_row(a, z, p.hk, r);
            xl = a.lse[gr];                                   // used after the tile before
            xs = a.delta[gr];
            xn = visible(a, z, r / a.G);
        }
    };
    load(start);
    for (int r0 = start; r0 < end; r0 += kTile) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int x = (int)threadIdx.x + j * kThreads;
            if (x < C) {
                store4(&qt[x / (D / 4)][x % (D / 4) * 4], xq[j]);
                store4(&dt[x / (D / 4)][x % (D / 4) * 4], xd[j]);
            }
        }
        if (threadIdx.x < kTile) {
            ls[threadIdx.x] = xl == -INFINITY ? 0.f : xl * kLog2e;
            dl[threadIdx.x] = xs;
            nv[threadIdx.x] = xl == -INFINITY ? 0 : xn;
        }
        __syncthreads();
        load(r0 + kTile);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f}, dp = s;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                const f32x4 qf = load4(&qt[16 * t + c][16 * e + 4 * g]), df = load4(&dt[16 * t + c][16 * e + 4 * g]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s = mma(qf[j], kf[e][j], s);
                    dp = mma(df[j], vf[e][j], dp);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * t + 4 * g + i;
                const float pr = key < nv[r] ? exp2_f(__builtin_fmaf(s[i], c2, -ls[r])) : 0.f;
                const float ds = key < nv[r] ? pr * (dp[i] - dl[r]) : 0.f;
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    av[e] = mma(dt[r][16 * e + c], pr, av[e]);
                    ak[e] = mma(qt[r][16 * e + c], ds, ak[e]);
                }
            }
        }
    }
    if (a.causal && (!finite(ak) || !finite(av))) {           // see finite()
#pragma unroll
        for (int e = 0; e < D / 16; ++e) ak[e] = av[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int r = start; r < end; ++r) {
            const int64_t gr = packed_row(a, z, p.hk, r);
            const T *qr = q_row<T>(a, z, p.hk, r), *dr = static_cast<const T*>(a.d_o) + gr * D;
            const float s = dot_row<T, D>(kf, qr, g), dp = dot_row<T, D>(vf, dr, g), lr = a.lse[gr];
            if (lr != -INFINITY && valid && key < visible(a, z, r / a.G)) {
                const float pr = exp2_f(__builtin_fmaf(s, c2, -lr * kLog2e)), ds = pr * (dp - a.delta[gr]);
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    av[e] += pr * load4(dr + 16 * e + 4 * g);
                    ak[e] += ds * load4(qr + 16 * e + 4 * g);
                }
            }
        }
    }
    if (!valid) return;
    if (a.k_splits > 1) {
        const int64_t at = (((int64_t)p.split * a.total_k + z.ko + key) * a.Hk + p.hk) * D;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
            store4(a.part_k + at + 16 * e + 4 * g, ak[e]);
            store4(a.part_v + at + 16 * e + 4 * g, av[e]);
        }
        return;
    }
    const int64_t kr = ((z.ko + key) * a.Hk + p.hk) * D;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
        store4(static_cast<T*>(a.dk) + kr + 16 * e + 4 * g, ak[e] * a.scale);
        store4(static_cast<T*>(a.dv) + kr + 16 * e + 4 * g, av[e]);
    }
}

// dk and dv from the splits' sums, four features a thread.  The keys are the
// sequences' own; what lies outside them is left alone.  Bound by reading the
// sums: 4 splits of 8176 keys, 4 heads of 128 (134 MB, half of it still in the
// caches) in 25 us.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_sum_kernel(const AttnArgs a) {
    const unsigned per = kThreads / (D / 4), groups = ((unsigned)a.max_k * a.Hk + per - 1) / per;
    const Seq z = sequence(a, (int)(blockIdx.x / groups));
    const int64_t r = (int64_t)(blockIdx.x % groups) * per + threadIdx.x / (D / 4);
    if (r >= (int64_t)z.lk * a.Hk) return;
    const int64_t at = (z.ko * a.Hk + r) * D + threadIdx.x % (D / 4) * 4, all = a.total_k * a.Hk * D;
    f32x4 k = {0.f, 0.f, 0.f, 0.f}, v = k;
#pragma unroll 4
    for (int i = 0; i < a.k_splits; ++i) {
        k += *reinterpret_cast<const f32x4*>(a.part_k + i * all + at);
        v += *reinterpret_cast<const f32x4*>(a.part_v + i * all + at);
    }
    k *= a.scale;
    store4(static_cast<T*>(a.dk) + at, k);
    store4(static_cast<T*>(a.dv) + at, v);
}

// ---------------------------------------------------------------- launch
// A token stride that the kernels cannot address: see kMaxStride; 2^40 elements
// in all are more than any tensor has.
bool far(int64_t stride, int most, int64_t tokens) {
    return stride > kMaxStride && (most > 1 || stride > ((int64_t)1 << 40) / std::max<int64_t>(tokens, 1));
}

gdn_status check_attn(const gdn_attn_desc* d) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->n_seq < 0 || d->Hq < 1 || d->Hk < 1 || d->D < 1 || d->total_q < 0 || d->total_k < 0 || d->max_q < 0 ||
        d->max_k < 0)
        return GDN_ERR_INVALID_ARG;
    if (d->Hq % d->Hk) return GDN_ERR_INVALID_ARG;
    if (d->io_dtype != GDN_BF16 && d->io_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (d->flags & ~(uint32_t)GDN_FLAG_ATTN_CAUSAL) return GDN_ERR_INVALID_ARG;
    if ((d->flags & GDN_FLAG_ATTN_CAUSAL) && d->causal_block < 1) return GDN_ERR_INVALID_ARG;
    // below, what a row's maximum may rise by without rescaling is no finite score
    if (!(d->scale >= 1e-30f) || !(d->scale < 1e30f)) return GDN_ERR_INVALID_ARG;
    if (d->k_room && d->k_room < d->max_k) return GDN_ERR_INVALID_ARG;
    const int64_t rq = (int64_t)d->Hq * d->D, rk = (int64_t)d->Hk * d->D;
    if ((d->q_stride && d->q_stride < rq) || (d->k_stride && d->k_stride < rk) || (d->v_stride && d->v_stride < rk))
        return GDN_ERR_INVALID_ARG;
    if (d->D != 16 && d->D != 32 && d->D != 64 && d->D != 128) return GDN_ERR_UNSUPPORTED;
    // row numbers within a sequence are 32-bit, with room for a tile
    if (d->total_q > INT32_MAX || d->total_k > INT32_MAX || (int64_t)d->max_q * d->Hq > (1 << 30) ||
        d->max_k > (1 << 30) || d->k_room > INT32_MAX)
        return GDN_ERR_UNSUPPORTED;
    const int64_t tk = d->k_room ? d->k_room * d->n_seq : d->total_k;
    if (rq > kMaxStride || far(d->q_stride, d->max_q, d->total_q) || far(d->k_stride, d->max_k, tk) ||
        far(d->v_stride, d->max_k, tk))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// The call with its bounds no higher than the tensors allow (whatever lies above
// them is the same call, and would only be more places to launch).
gdn_attn_desc bounded(const gdn_attn_desc* d) {
    gdn_attn_desc b = *d;
    b.max_q = (int32_t)std::min<int64_t>(b.max_q, b.total_q);
    b.max_k = (int32_t)std::min<int64_t>(b.max_k, b.total_k);
    return b;
}

bool fast(const gdn_attn_desc* d) { return d->io_dtype == GDN_BF16 && d->D >= 32; }

int fwd_rows(const gdn_attn_desc* d) {
    return fast(d) ? attn_fwd_bf16_rows(d->max_q, d->Hq / d->Hk, d->D) : kRows;
}

// Keys of a split of the key axis; max_k or more: not split.  Split where the
// row tiles alone would leave compute units idle: as many splits as fill the
// 256 in one round with two waves a SIMD (880 queries against 19360 keys, 16
// heads of 128: 156 us, with twice as many 171).  That is what the D = 128
// kernels hold; for narrower heads, whose registers would let three (D = 64) or
// four waves in, the same count stands and was not measured.  Nor does the rule
// look at the lengths: 540 tiles of a packed batch are not split, and its
// longest sequence's walk (4096 keys, 130 us) is the kernel's whole time, where
// its work spread evenly would take about 92.  A decode step (a few rows a key
// head) is cut eight times finer, because the lengths of its caches differ and
// short work spreads evenly; a split's fp32 partial result is then small
// against its keys, of which it takes 512 at least (128 at the fp32 rate).
int fwd_chunk(const gdn_attn_desc* d) {
    const int64_t rows = (int64_t)d->max_q * (d->Hq / d->Hk);
    int tiles;
    const int64_t units = places(d->total_q * (d->Hq / d->Hk), rows, d->n_seq, fwd_rows(d), true, &tiles) * d->Hk;
    int64_t n = (fwd_rows(d) == 256 ? 256 : 512) / std::max<int64_t>(units, 1);
    if (rows <= 32) n *= 8;
    if (n < 2) return std::max(d->max_k, 1);
    const int64_t chunk = std::max<int64_t>(((d->max_k + n - 1) / n + 63) / 64 * 64, fast(d) ? 512 : 128);
    return (int)std::min<int64_t>(chunk, std::max(d->max_k, 1));
}
int fwd_splits(const gdn_attn_desc* d) {
    const int chunk = fwd_chunk(d);
    return std::max(1, (d->max_k + chunk - 1) / chunk);
}

// Splits of the query rows in the dk/dv kernel.  Its workgroups each walk all
// the rows that see their keys; with few key tiles (grouped heads: few heads
// with many rows each) that leaves compute units idle and the first tiles' long
// walks last, so below two workgroups a unit the rows are split for about four.
// A split's fp32 sums cost 16 D bytes a key, its products 8 D flops a (row,
// key): from 1024 rows a split on (128 at the fp32 rate) the former stay a
// small part.  The sizes do not depend on the lengths on the device, nor on
// whether the sequences are packed (uniform ones count the same tiles).
int bwd_splits(const gdn_attn_desc* d) {
    int tiles;
    const int64_t items = places(d->total_k, d->max_k, d->n_seq, fast(d) ? kBwdTile : kRows, true, &tiles) * d->Hk;
    const int64_t rows = (int64_t)d->max_q * (d->Hq / d->Hk);
    // what 32 MiB of sums allow stays in the caches
    const int64_t near = ((int64_t)32 << 20) / std::max<int64_t>(1, d->total_k * d->Hk * d->D * 8);
    const int64_t most = std::max(rows / (fast(d) ? 1024 : 128), std::min(rows / (fast(d) ? 256 : 64), near));
    if (items < 1 || items >= 512 || most < 2) return 1;
    return (int)std::min<int64_t>(std::min<int64_t>((1024 + items - 1) / items, most), 64);
}

AttnArgs fill(const gdn_attn_desc* d) {
    AttnArgs a = {};
    a.total_q = d->total_q, a.total_k = d->total_k;
    a.n_seq = d->n_seq, a.Hq = d->Hq, a.Hk = d->Hk, a.G = d->Hq / d->Hk, a.D = d->D;
    a.ldq = d->q_stride ? d->q_stride : (int64_t)d->Hq * d->D;
    a.ldk = d->k_stride ? d->k_stride : (int64_t)d->Hk * d->D;
    a.ldv = d->v_stride ? d->v_stride : (int64_t)d->Hk * d->D;
    a.max_q = d->max_q, a.max_k = d->max_k;
    a.k_room = d->k_room ? d->k_room : d->max_k;
    a.causal = (d->flags & GDN_FLAG_ATTN_CAUSAL) ? 1 : 0;
    a.block = a.causal ? d->causal_block : 1;
    a.scale = d->scale;
    a.splits = a.k_splits = 1;
    return a;
}

// Bytes from the first to the last element of a [rows][ld] tensor whose rows
// hold w elements.
size_t span(int64_t rows, int64_t ld, int64_t w, size_t e) { return rows > 0 ? ((size_t)(rows - 1) * ld + w) * e : 0; }

// Key tokens from the first sequence's first to the last one's last.
int64_t key_rows(const gdn_attn_desc* d, bool packed) {
    if (packed || !d->k_room || d->n_seq < 1) return d->total_k;
    return (d->n_seq - 1) * d->k_room + d->max_k;
}

// The launches of a call, all of them sized before the first.
struct FwdGrids {
    Grid main;
    unsigned join;                       // splits > 1
};
bool fwd_grids(AttnArgs& a, int rows, bool f32_kernel, FwdGrids* g) {
    const int64_t n = places(a.total_q * a.G, (int64_t)a.max_q * a.G, a.n_seq, rows, a.cu_q, &g->main.tiles);
    if (!grid_of(n * a.splits * a.Hk, f32_kernel ? kThreads : 2 * rows, &g->main.groups)) return false;
    g->join = 0;
    if (a.splits == 1) return true;
    // A row a wave where they are few (eight single-token requests: 80 us against
    // 95 with four), four where places of shorter sequences stay empty in number.
    const int64_t all = (int64_t)a.max_q * a.Hq;
    a.join_rows = all * a.n_seq > 16384 ? 16 : 4;
    return grid_of((all + a.join_rows - 1) / a.join_rows * a.n_seq, kThreads, &g->join);
}
struct BwdGrids {
    Grid dq, dkv;
    unsigned sum;                        // k_splits > 1
};
bool bwd_grids(const AttnArgs& a, int size, BwdGrids* g) {
    int64_t n = places(a.total_q * a.G, (int64_t)a.max_q * a.G, a.n_seq, size, a.cu_q, &g->dq.tiles);
    if (!grid_of(n * a.Hk, kThreads, &g->dq.groups)) return false;
    n = places(a.total_k, a.max_k, a.n_seq, size, a.cu_k, &g->dkv.tiles);
    if (!grid_of(n * a.Hk * a.k_splits, kThreads, &g->dkv.groups)) return false;
    g->sum = 0;
    const int64_t per = kThreads / (a.D / 4);
    return a.k_splits == 1 || grid_of(((int64_t)a.max_k * a.Hk + per - 1) / per * a.n_seq, kThreads, &g->sum);
}

template <typename T, int D>
gdn_status run_fwd(AttnArgs a, Grid g, hipStream_t s) {
    a.tiles = g.tiles;
    hipLaunchKernelGGL((attn_fwd_f32_kernel<T, D>), dim3(g.groups), dim3(kThreads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
template <typename T, int D>
gdn_status run_join(const AttnArgs& a, unsigned groups, hipStream_t s) {
    hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3(groups), dim3(kThreads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
template <typename T, int D>
gdn_status run_bwd(AttnArgs a, Grid dq, Grid dkv, hipStream_t s) {
    a.tiles = dq.tiles;
    if (dq.groups) hipLaunchKernelGGL((attn_dq_f32_kernel<T, D>), dim3(dq.groups), dim3(kThreads), 0, s, a);
    a.tiles = dkv.tiles;
    if (dkv.groups) hipLaunchKernelGGL((attn_dkv_f32_kernel<T, D>), dim3(dkv.groups), dim3(kThreads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
template <typename T, int D>
gdn_status run_sum(const AttnArgs& a, unsigned groups, hipStream_t s) {
    if (groups) hipLaunchKernelGGL((attn_sum_kernel<T, D>), dim3(groups), dim3(kThreads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

#define GDN_BY_D(FN, T, ...)                                              \
    (a.D == 16 ? FN<T, 16>(__VA_ARGS__) : a.D == 32 ? FN<T, 32>(__VA_ARGS__) \
     : a.D == 64 ? FN<T, 64>(__VA_ARGS__) : FN<T, 128>(__VA_ARGS__))

}  // namespace

extern "C" {

size_t gdn_attn_workspace_size(const gdn_attn_desc* d) {
    if (check_attn(d) != GDN_OK || d->n_seq == 0 || d->total_q == 0 || d->max_q == 0) return 0;
    const gdn_attn_desc b = bounded(d);
    const int64_t n = fwd_splits(&b);
    if (n < 2) return 0;
    return round256((size_t)n * d->total_q * d->Hq * d->D * 4) + round256((size_t)n * d->total_q * d->Hq * 4);
}

gdn_status gdn_attn_fwd(const gdn_attn_desc* d, const void* q, const void* k, const void* v, const int32_t* cu_q,
                        const int32_t* cu_k, const int32_t* k_len, void* o, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK) return st;
    if (!cu_q && (int64_t)d->n_seq * d->max_q != d->total_q) return GDN_ERR_INVALID_ARG;
    if (!cu_k && (int64_t)d->n_seq * d->max_k != d->total_k) return GDN_ERR_INVALID_ARG;
    if (d->n_seq == 0 || d->total_q == 0 || d->max_q == 0) return GDN_OK;
    if (!q || !o || (d->total_k > 0 && (!k || !v))) return GDN_ERR_INVALID_ARG;
    const gdn_attn_desc b = bounded(d);
    AttnArgs a = fill(&b);
    a.cu_q = cu_q, a.cu_k = cu_k, a.k_len = k_len;
    a.splits = fwd_splits(&b);
    a.chunk = fwd_chunk(&b);
    FwdGrids g;
    if (!fwd_grids(a, fwd_rows(&b), !fast(d), &g)) return GDN_ERR_UNSUPPORTED;
    const size_t e = d->io_dtype == GDN_F32 ? 4 : 2;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(k_len, 4))
        return GDN_ERR_ALIGNMENT;
    if (a.ldq * e % 16 || a.ldk * e % 16 || a.ldv * e % 16) return GDN_ERR_ALIGNMENT;
    const size_t need = gdn_attn_workspace_size(d);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
    const int64_t wq = (int64_t)d->Hq * d->D, wk = (int64_t)d->Hk * d->D;
    const Range ins[] = {rng(q, span(d->total_q, a.ldq, wq, e)), rng(k, span(key_rows(d, cu_k), a.ldk, wk, e)),
                         rng(v, span(key_rows(d, cu_k), a.ldv, wk, e)), rng(cu_q, ((size_t)d->n_seq + 1) * 4),
                         rng(cu_k, ((size_t)d->n_seq + 1) * 4), rng(k_len, (size_t)d->n_seq * 4)};
    const Range outs[] = {rng(o, (size_t)d->total_q * wq * e), rng(lse, (size_t)d->total_q * d->Hq * 4),
                          rng(need ? workspace : nullptr, need)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return GDN_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_ALIAS;
    }
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    a.q = q, a.k = k, a.v = v, a.out = o, a.lse = lse;
    if (a.splits > 1) {
        a.part_o = static_cast<float*>(workspace);
        a.part_lse = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                              round256((size_t)a.splits * d->total_q * d->Hq * d->D * 4));
    }
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f32 = d->io_dtype == GDN_F32;
    // bf16 heads of 16 features are narrower than the bf16 tiles and take the fp32 kernels
    st = f32       ? GDN_BY_D(run_fwd, float, a, g.main, s)
         : fast(d) ? attn_fwd_bf16(a, fwd_rows(&b), g.main, s)
                   : run_fwd<uint16_t, 16>(a, g.main, s);
    if (st != GDN_OK || a.splits == 1) return st;
    return f32 ? GDN_BY_D(run_join, float, a, g.join, s) : GDN_BY_D(run_join, uint16_t, a, g.join, s);
}

size_t gdn_attn_workspace_size_bwd(const gdn_attn_desc* d) {
    if (check_attn(d) != GDN_OK || d->n_seq == 0) return 0;
    const gdn_attn_desc b = bounded(d);
    const size_t n = bwd_splits(&b);
    return round256((size_t)d->total_q * d->Hq * 4) + (n > 1 ? 2 * round256(n * d->total_k * d->Hk * d->D * 4) : 0);
}

gdn_status gdn_attn_bwd(const gdn_attn_desc* d, const void* q, const void* k, const void* v, const void* o,
                        const float* lse, const void* dO, const int32_t* cu_q, const int32_t* cu_k, void* dq, void* dk,
                        void* dv, void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK) return st;
    if (!cu_q && (int64_t)d->n_seq * d->max_q != d->total_q) return GDN_ERR_INVALID_ARG;
    if (!cu_k && (int64_t)d->n_seq * d->max_k != d->total_k) return GDN_ERR_INVALID_ARG;
    if (d->n_seq == 0 || (d->total_q == 0 && d->total_k == 0)) return GDN_OK;
    if (d->total_q > 0 && (!q || !o || !lse || !dO || !dq)) return GDN_ERR_INVALID_ARG;
    if (d->total_k > 0 && (!k || !v || !dk || !dv)) return GDN_ERR_INVALID_ARG;
    const gdn_attn_desc b = bounded(d);
    AttnArgs a = fill(&b);
    a.cu_q = cu_q, a.cu_k = cu_k;
    a.k_splits = bwd_splits(&b);
    BwdGrids g;
    if (!bwd_grids(a, fast(d) ? kBwdTile : kRows, &g)) return GDN_ERR_UNSUPPORTED;
    const size_t e = d->io_dtype == GDN_F32 ? 4 : 2;
    for (const void* p : {q, k, v, o, dO, (const void*)dq, (const void*)dk, (const void*)dv})
        if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
    if (!aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return GDN_ERR_ALIGNMENT;
    if (a.ldq * e % 16 || a.ldk * e % 16 || a.ldv * e % 16) return GDN_ERR_ALIGNMENT;
    const size_t need = gdn_attn_workspace_size_bwd(d);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
    const int64_t wq = (int64_t)d->Hq * d->D, wk = (int64_t)d->Hk * d->D;
    const size_t qb = (size_t)d->total_q * wq * e, kb = (size_t)d->total_k * wk * e;
    const Range ins[] = {rng(q, span(d->total_q, a.ldq, wq, e)), rng(k, span(key_rows(d, cu_k), a.ldk, wk, e)),
                         rng(v, span(key_rows(d, cu_k), a.ldv, wk, e)), rng(o, qb), rng(dO, qb),
                         rng(lse, (size_t)d->total_q * d->Hq * 4), rng(cu_q, ((size_t)d->n_seq + 1) * 4),
                         rng(cu_k, ((size_t)d->n_seq + 1) * 4)};
    const Range outs[] = {rng(dq, qb), rng(dk, kb), rng(dv, kb), rng(need ? workspace : nullptr, need)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return GDN_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_ALIAS;
    }
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    a.q = q, a.k = k, a.v = v, a.o = o, a.lse = const_cast<float*>(lse), a.d_o = dO;
    a.dq = dq, a.dk = dk, a.dv = dv;
    a.delta = static_cast<float*>(workspace);
    if (a.k_splits > 1) {
        unsigned char* w = static_cast<unsigned char*>(workspace) + round256((size_t)d->total_q * d->Hq * 4);
        a.part_k = reinterpret_cast<float*>(w);
        a.part_v = reinterpret_cast<float*>(w + round256((size_t)a.k_splits * d->total_k * d->Hk * d->D * 4));
    }
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f32 = d->io_dtype == GDN_F32;
    st = f32       ? GDN_BY_D(run_bwd, float, a, g.dq, g.dkv, s)
         : fast(d) ? attn_bwd_bf16(a, g.dq, g.dkv, s)
                   : run_bwd<uint16_t, 16>(a, g.dq, g.dkv, s);
    if (st != GDN_OK || a.k_splits == 1) return st;
    return f32 ? GDN_BY_D(run_sum, float, a, g.sum, s) : GDN_BY_D(run_sum, uint16_t, a, g.sum, s);
}

}  // extern "C"
