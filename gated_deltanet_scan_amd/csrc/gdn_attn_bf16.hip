// Softmax attention in bf16 matrix instructions (D in {32, 64, 128}): the backward
// kernels, and the launches of both directions.  The mathematics, the mask and the
// entry points are in gdn_attn.hip; the operand layouts and the forward kernel in
// gdn_attn_tile.hpp.
#include "gdn_attn_tile.hpp"

#include <algorithm>
#include <type_traits>

namespace gdnattn {
namespace {

// dq, and <d_o, o> for the dk/dv kernel.  Query rows as columns, as in the
// forward kernel; the key tile is read both ways (S^T = K Q^T, dQ^T += K^T dS^T).
//
// dS is rounded to bf16 for its products, here and in the dk/dv kernel (there P
// as well), half a step each.
//
// <d_o, o> = sum_j p_j dp_j.  From the rounded o it is off by 2^-8 |d_o| |o| at
// most, which matters where a row sees few keys and o is as large as v (a causal
// sequence of 300 tokens: dq off by 2.40e-3 with it and 2.26e-3 without, of
// which 1.68e-3 are dq's own rounding).  Where the workgroup's rows see at most
// kExactKeys keys the sum is formed in fp32 by a first walk over them.  That
// makes 10 D flops of the 6 D a pair there: 8192 packed sequences of 1 to 299
// tokens, 8/2 heads of 64, backward 3452 us with it and 3132 without.
//
// Measured: 4096 x 4096, 16 heads of 128: 227 us, 910 TFLOP/s of 6 D flops a
// pair (783 at D = 64, 603 at 32); two waves a SIMD wait on the products of one
// step before its exponentials, and on those before the next products.
constexpr int kExactKeys = 256;
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attn_dq_kernel(const AttnArgs a) {
    constexpr int NT = 64 * NW, BM = 32 * NW, KS = D / 16, DB = D / 32, TB = kKeys * D * 2;
    __shared__ __attribute__((aligned(16))) unsigned char kt[2][TB], vt[2][TB];
    const Place p = find_place<false>(a, BM);
    if (p.s < 0) return;
    const Seq z = sequence(a, p.s);
    const int rows = z.lq * a.G, r0 = p.tile * BM;
    if (r0 >= rows) return;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w0 = r0 + 32 * wave, row = w0 + r;
    const bool valid = row < rows;
    const int upto = visible(a, z, (min(r0 + BM, rows) - 1) / a.G);
    const int n_first = w0 < rows ? visible(a, z, w0 / a.G) : 0;
    const int n_last = w0 < rows ? visible(a, z, (min(w0 + 32, rows) - 1) / a.G) : 0;
    const int n = valid ? visible(a, z, row / a.G) : 0;
    const int64_t gr = packed_row(a, z, p.hk, valid ? row : r0);
    const u32x4 none = {0u, 0u, 0u, 0u};
    u32x4 q[KS], g[KS];
    float delta = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        q[s] = g[s] = none;
        if (valid) {
            q[s] = *reinterpret_cast<const u32x4*>(q_row(a, z, p.hk, row) + 16 * s + 8 * h);
            g[s] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.d_o) + gr * D + 16 * s + 8 * h);
            const u32x4 o = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.o) + gr * D + 16 * s + 8 * h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                delta += __uint_as_float(g[s][j] << 16) * __uint_as_float(o[j] << 16);
                delta += __uint_as_float(g[s][j] & 0xffff0000u) * __uint_as_float(o[j] & 0xffff0000u);
            }
        }
    }
    delta = half_sum(delta);
    float ls = valid ? a.lse[gr] * kLog2e : INFINITY;
    if (ls == -INFINITY) ls = INFINITY;                       // a row that saw nothing: p = 0
    f32x16 acc[DB];
    const KeysBf16 kb(a.k, nullptr, a.ldk, z.k0, p.hk, a.Hk, D), vb(a.v, nullptr, a.ldv, z.k0, p.hk, a.Hk, D);
    const float c2 = a.scale * kLog2e;
    Addr<D> ad;
    ad.init(lane);
    KeysBf16::Tile<D, NT> sk, sv;
    auto walk = [&](auto first) {
        constexpr bool kFirst = decltype(first)::value;
        float exact = 0.f;
        if (upto > 0) {
            sk.load(kb, 0, upto, tid);
            sv.load(vb, 0, upto, tid);
            sk.store(kt[0], tid);
            sv.store(vt[0], tid);
        }
        __syncthreads();
        int buf = 0;
        for (int n0 = 0; n0 < upto; n0 += kKeys, buf ^= 1) {
            const bool more = n0 + kKeys < upto;
            if (more) {
                sk.load(kb, n0 + kKeys, upto, tid);
                sv.load(vb, n0 + kKeys, upto, tid);
            }
            if (n0 < n_last) {
                const bool mask = n0 + kKeys > n_first;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x16 s = zero16(), dp = zero16();
                    ad.renew();
#pragma unroll
                    for (int e = 0; e < KS; ++e) s = mma(ad.rows(kt[buf], t, e), q[e], s);
#pragma unroll
                    for (int e = 0; e < KS; ++e) dp = mma(ad.rows(vt[buf], t, e), g[e], dp);
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = exp2_f(__builtin_fmaf(s[i], c2, -ls));
                    if (mask) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3) >= n) s[i] = dp[i] = 0.f;
                    }
                    if constexpr (kFirst) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) exact += s[i] * dp[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[i] *= dp[i] - delta;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const u32x4 ds = pack8(s, 8 * u);
#pragma unroll
                            for (int e = 0; e < DB; ++e) acc[e] = mma(ad.cols(kt[buf], e, 2 * t + u), ds, acc[e]);
                        }
                    }
                }
            }
            if (more) {
                sk.store(kt[buf ^ 1], tid);
                sv.store(vt[buf ^ 1], tid);
            }
            __syncthreads();
        }
        if constexpr (kFirst) delta = half_sum(exact);
    };
    if (upto <= kExactKeys) walk(std::true_type());
#pragma unroll
    for (int e = 0; e < DB; ++e) acc[e] = zero16();
    walk(std::false_type());
    if (a.causal && !finite(acc)) {                           // see finite()
#pragma unroll
        for (int e = 0; e < DB; ++e) acc[e] = zero16();
#pragma unroll 1
        for (int j = 0; j < n_last; ++j) {
            const uint16_t* kr = kb.base + (int64_t)j * a.ldk;
            const float s = dot_row(q, kr, h), dp = dot_row(g, vb.base + (int64_t)j * a.ldv, h);
            if (j < n) add_row(acc, exp2_f(__builtin_fmaf(s, c2, -ls)) * (dp - delta), kr, h);
        }
    }
    if (!valid) return;
    if (h == 0) a.delta[gr] = delta;
#pragma unroll
    for (int e = 0; e < DB; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dq) + gr * D + 32 * e + 8 * i + 4 * h) =
                u32x2{pack_bf16x2(acc[e][4 * i] * a.scale, acc[e][4 * i + 1] * a.scale),
                      pack_bf16x2(acc[e][4 * i + 2] * a.scale, acc[e][4 * i + 3] * a.scale)};
}

// Staging of RT packed query rows: q, d_o, and each row's logarithm and
// <d_o, o>.  A row's token, counted from the tile's first, comes from a
// multiplication (place within the tile times 2^32 / G, exact for G <= 2^15);
// tiles that start at the same head share the addresses, which is all of them
// where G divides RT.  Rows past the last lie past the descriptors' ends and
// read as zeros.
template <int D, int NT, int RT>
struct RowStage {
    static constexpr int N = RT * D / 8 / NT;
    static_assert(N >= 1 && RT <= NT, "every thread stages something");
    u32x4 q[N], g[N];
    float ls, dl;
    uint32_t at_q[N], at_g[N], at_l;
    int first = -1;                                       // head of the tile's first row
    __device__ __forceinline__ void load(const AttnArgs& a, const Seq& z, int hk, int r0, uint32_t inv, int tid) {
        const int i0 = r0 / a.G, g0 = r0 - i0 * a.G;
        if (g0 != first) {
            first = g0;
            auto token = [&](int rr, uint32_t& gg) {
                const uint32_t x = (uint32_t)(g0 + rr), tok = a.G == 1 ? x : __umulhi(x, inv);
                gg = x - tok * a.G;
                return tok;
            };
            uint32_t gg;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int i = tid + j * NT, c = i % (D / 8);
                const uint32_t tok = token(i / (D / 8), gg);
                at_q[j] = tok * (tile_stride(a.ldq) * 2) + gg * (2 * D) + c * 16;
                at_g[j] = tok * (uint32_t)(a.Hq * D * 2) + gg * (2 * D) + c * 16;
            }
            const uint32_t tok = token(tid & (RT - 1), gg);
            at_l = (tok * (uint32_t)a.Hq + gg) * 4;
        }
        // the last token's heads end each range
        auto range = [&](const void* p, int64_t tok_bytes, int64_t head_bytes) {
            return make_rsrc(static_cast<const unsigned char*>(p) + (z.q0 + i0) * tok_bytes + hk * a.G * head_bytes,
                             (uint32_t)min((z.lq - i0 - 1) * tok_bytes + a.G * head_bytes, (int64_t)0x7ffffff0));
        };
        const rsrc_t rq = range(a.q, a.ldq * 2, 2 * D), rg = range(a.d_o, (int64_t)a.Hq * D * 2, 2 * D);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            q[j] = __builtin_amdgcn_raw_buffer_load_b128(rq, at_q[j], 0, 0);
            g[j] = __builtin_amdgcn_raw_buffer_load_b128(rg, at_g[j], 0, 0);
        }
        // nothing is computed from the loads here: that would wait for them all
        ls = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(range(a.lse, (int64_t)a.Hq * 4, 4), at_l, 0, 0));
        dl = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(range(a.delta, (int64_t)a.Hq * 4, 4), at_l, 0, 0));
    }
    __device__ __forceinline__ void store(unsigned char* qt, unsigned char* gt, float* ld, int tid) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = tid + j * NT, rr = i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<u32x4*>(qt + chunk_at<D>(rr, c)) = q[j];
            *reinterpret_cast<u32x4*>(gt + chunk_at<D>(rr, c)) = g[j];
        }
        if (tid < RT) {
            ld[tid] = ls == -INFINITY ? INFINITY : ls * kLog2e;   // a row that saw nothing: p = 0
            ld[RT + tid] = dl;
        }
    }
};

// dk and dv.  A wave's 32 keys as columns, with K and V in registers; the
// packed query rows of all heads that share them walk through LDS, read both
// ways (S = Q K^T and dP = dO V^T by rows; dV^T += dO^T P, dK^T += Q^T dS).
// At D = 128 the two accumulators take 128 registers; V then stays in LDS and
// row tiles are half as long, so that two waves fit a SIMD.
// Measured: 4096 x 4096, 16 heads of 128: 359 us, 765 TFLOP/s of 8 D flops a
// pair (759 at D = 64, 565 at 32); bound as dq is, and by V's reads from LDS.
template <int D, int NW, int RT>
__global__ __launch_bounds__(64 * NW, 2) void attn_dkv_kernel(const AttnArgs a) {
    constexpr int NT = 64 * NW, BN = 32 * NW, KS = D / 16, DB = D / 32, TB = RT * D * 2;
    __shared__ __attribute__((aligned(16))) unsigned char qt[2][TB], gt[2][TB];
    __shared__ __attribute__((aligned(16))) float ld[2][2 * RT];   // logarithms, then <d_o, o>
    constexpr bool VL = D == 128;
    __shared__ __attribute__((aligned(16))) unsigned char vl[VL ? BN * D * 2 : 16];
    const Place p = find_place<true>(a, BN);
    if (p.s < 0) return;
    const Seq z = sequence(a, p.s);
    const int k0 = p.tile * BN;
    if (k0 >= z.lk) return;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w0 = k0 + 32 * wave, key = w0 + r;
    const bool valid = key < z.lk;
    const int rows = z.lq * a.G;
    // rows below w_first see none of the wave's keys, rows from w_all on see all 32;
    // no row sees a place past the last key (its score of 0 less a low logarithm
    // would be a probability of infinity, and send the wave to the tail below)
    const int w_first = w0 < z.lk ? first_query(a, z, w0) * a.G : rows;
    const int w_all = w0 + 32 <= z.lk ? first_query(a, z, w0 + 31) * a.G : rows;
    const int from = valid ? first_query(a, z, key) * a.G : rows;
    const u32x4 none = {0u, 0u, 0u, 0u};
    u32x4 kf[KS], vf[VL ? 1 : KS];
    f32x16 ak[DB], av[DB];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int64_t kr = z.k0 + (valid ? key : 0);
        u32x4 vv = none;
        kf[s] = none;
        if (valid) {
            kf[s] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.k) + kr * a.ldk +
                                                    (int64_t)p.hk * D + 16 * s + 8 * h);
            vv = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.v) + kr * a.ldv +
                                                 (int64_t)p.hk * D + 16 * s + 8 * h);
        }
        if constexpr (VL)
            *reinterpret_cast<u32x4*>(vl + chunk_at<D>(32 * wave + r, 2 * s + h)) = vv;   // read by this wave alone
        else
            vf[s] = vv;
    }
#pragma unroll
    for (int e = 0; e < DB; ++e) ak[e] = av[e] = zero16();
    const float c2 = a.scale * kLog2e;
    const uint32_t inv = a.G == 1 ? 0u : (uint32_t)((0x100000000ull + a.G - 1) / a.G);
    Addr<D> ad;
    ad.init(lane);
    RowStage<D, NT, RT> st;
    int start = min(first_query(a, z, k0) * a.G, rows) / RT * RT, end = rows;
    if (a.k_splits > 1) {
        int lo, hi;
        split_range(rows - start, RT, a.k_splits, p.split, lo, hi);
        end = start + hi;
        start += lo;
    }
    if (start < end) {
        st.load(a, z, p.hk, start, inv, tid);
        st.store(qt[0], gt[0], ld[0], tid);
    }
    __syncthreads();
    int buf = 0;
    for (int r0 = start; r0 < end; r0 += RT, buf ^= 1) {
        const bool more = r0 + RT < end;
        if (more) st.load(a, z, p.hk, r0 + RT, inv, tid);
        if (r0 + RT > w_first) {
            const bool mask = r0 < w_all;
#pragma unroll
            for (int t = 0; t < RT / 32; ++t) {
                f32x16 s = zero16(), dp = zero16();
                ad.renew();
#pragma unroll
                for (int e = 0; e < KS; ++e) s = mma(ad.rows(qt[buf], t, e), kf[e], s);
#pragma unroll
                for (int e = 0; e < KS; ++e)
                    dp = mma(ad.rows(gt[buf], t, e), VL ? ad.rows(vl + wave * 64 * D, 0, e) : vf[VL ? 0 : e], dp);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 l4 = *reinterpret_cast<const f32x4*>(&ld[buf][32 * t + 8 * i + 4 * h]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[4 * i + j] = exp2_f(__builtin_fmaf(s[4 * i + j], c2, -l4[j]));
                }
                if (mask) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (r0 + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3) < from) s[i] = 0.f;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const u32x4 pp = pack8(s, 8 * u);
#pragma unroll
                    for (int e = 0; e < DB; ++e) av[e] = mma(ad.cols(gt[buf], e, 2 * t + u), pp, av[e]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 d4 = *reinterpret_cast<const f32x4*>(&ld[buf][RT + 32 * t + 8 * i + 4 * h]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[4 * i + j] *= dp[4 * i + j] - d4[j];
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const u32x4 ds = pack8(s, 8 * u);
#pragma unroll
                    for (int e = 0; e < DB; ++e) ak[e] = mma(ad.cols(qt[buf], e, 2 * t + u), ds, ak[e]);
                }
            }
        }
        if (more) st.store(qt[buf ^ 1], gt[buf ^ 1], ld[buf ^ 1], tid);
        __syncthreads();
    }
    // The lane's place once more, from the lane's number: held over the loop it
    // would take the registers of what the loop needs (4% slower).
    const int lane2 = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)), h2 = lane2 >> 5;
    const int key2 = w0 + (lane2 & 31);
    const bool valid2 = key2 < z.lk;
    // see finite(); a hidden value that spoils dv spoils dS, and so dk, as well.
    // Without a mask only the zeros past the last row are such places, for a key
    // that is infinite (0 times it is a NaN); the wave's other keys keep their sums.
    bool again = false;
    if (a.causal) {
        again = !finite(ak);
    } else if (rows % RT) {
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < KS; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                t = __builtin_fmaf(__uint_as_float(kf[e][i] << 16), 0.f, t);
                t = __builtin_fmaf(__uint_as_float(kf[e][i] & 0xffff0000u), 0.f, t);
            }
        again = half_sum(t) != 0.f;                           // 0, or NaN
    }
    if (__any(again)) {
        if (again) {
#pragma unroll
            for (int e = 0; e < DB; ++e) ak[e] = av[e] = zero16();
        }
        const int from2 = first_query(a, z, min(key2, z.lk - 1)) * a.G;
        u32x4 vr[KS];
#pragma unroll
        for (int e = 0; e < KS; ++e) vr[e] = VL ? ad.rows(vl + wave * 64 * D, 0, e) : vf[VL ? 0 : e];
#pragma unroll 1
        for (int i = max(start, w_first); i < end; ++i) {
            const int64_t gr = packed_row(a, z, p.hk, i);
            const uint16_t *qr = q_row(a, z, p.hk, i), *gi = static_cast<const uint16_t*>(a.d_o) + gr * D;
            const float s = dot_row(kf, qr, h2), dp = dot_row(vr, gi, h2), lr = a.lse[gr];
            if (again && lr != -INFINITY && valid2 && i >= from2) {
                const float pr = exp2_f(__builtin_fmaf(s, c2, -lr * kLog2e));
                add_row(av, pr, gi, h2);
                add_row(ak, pr * (dp - a.delta[gr]), qr, h2);
            }
        }
    }
    if (!valid2) return;
    if (a.k_splits > 1) {
        const int64_t at = (((int64_t)p.split * a.total_k + z.ko + key2) * a.Hk + p.hk) * D;
#pragma unroll
        for (int e = 0; e < DB; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 32 * e + 8 * i + 4 * h2;
                *reinterpret_cast<f32x4*>(a.part_k + at + d) =
                    f32x4{ak[e][4 * i], ak[e][4 * i + 1], ak[e][4 * i + 2], ak[e][4 * i + 3]};
                *reinterpret_cast<f32x4*>(a.part_v + at + d) =
                    f32x4{av[e][4 * i], av[e][4 * i + 1], av[e][4 * i + 2], av[e][4 * i + 3]};
            }
        return;
    }
    const int64_t at = ((z.ko + key2) * a.Hk + p.hk) * D;
#pragma unroll
    for (int e = 0; e < DB; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = 32 * e + 8 * i + 4 * h2;
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dk) + at + d) =
                u32x2{pack_bf16x2(ak[e][4 * i] * a.scale, ak[e][4 * i + 1] * a.scale),
                      pack_bf16x2(ak[e][4 * i + 2] * a.scale, ak[e][4 * i + 3] * a.scale)};
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dv) + at + d) =
                u32x2{pack_bf16x2(av[e][4 * i], av[e][4 * i + 1]), pack_bf16x2(av[e][4 * i + 2], av[e][4 * i + 3])};
        }
}

template <int D, int NW>
gdn_status launch_fwd(AttnArgs a, Grid g, hipStream_t s) {
    a.tiles = g.tiles;
    hipLaunchKernelGGL((attn_fwd_kernel<KeysBf16, D, NW>), dim3(g.groups), dim3(64 * NW), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <int D>
gdn_status launch_bwd(AttnArgs a, Grid dq, Grid dkv, hipStream_t s) {
    constexpr int NW = kBwdTile / 32;
    a.tiles = dq.tiles;
    if (dq.groups) hipLaunchKernelGGL((attn_dq_kernel<D, NW>), dim3(dq.groups), dim3(64 * NW), 0, s, a);
    a.tiles = dkv.tiles;
    if (dkv.groups)
        hipLaunchKernelGGL((attn_dkv_kernel<D, NW, (D == 128 ? 32 : 64)>), dim3(dkv.groups), dim3(64 * NW), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

// Rows of a workgroup.  At D = 128 two waves fill a SIMD's registers: as one
// workgroup of eight they share every key tile, where two of four stage each
// tile twice (frame-causal clip of 18480 tokens, 16 heads: 1440 us against
// 1476).  A decode step, whose rows fill a wave, takes the small one, since its
// other waves only help to stage (eight requests: 80 us against 101).
int attn_fwd_bf16_rows(int max_q, int G, int D) { return D == 128 && (int64_t)max_q * G > 256 ? 256 : 128; }

gdn_status attn_fwd_bf16(const AttnArgs& a, int rows, Grid g, hipStream_t s) {
    if (a.D == 32) return launch_fwd<32, 4>(a, g, s);
    if (a.D == 64) return launch_fwd<64, 4>(a, g, s);
    return rows == 256 ? launch_fwd<128, 8>(a, g, s) : launch_fwd<128, 4>(a, g, s);
}

gdn_status attn_bwd_bf16(const AttnArgs& a, Grid dq, Grid dkv, hipStream_t s) {
    if (a.D == 32) return launch_bwd<32>(a, dq, dkv, s);
    if (a.D == 64) return launch_bwd<64>(a, dq, dkv, s);
    return launch_bwd<128>(a, dq, dkv, s);
}

}  // namespace gdnattn
