// Softmax attention over block-scaled keys and values (MXFP8, MXFP4): the
// launches of gdn_attn_fwd_fp8 and gdn_attn_fwd_fp4, and the kernel for few query
// rows.  More rows take the forward kernel of bf16 keys (gdn_attn_tile.hpp), which
// widens codes to bf16 as it stages them, once for a row tile of up to 256.  It is bound
// by the matrix and vector instructions of two waves a SIMD, as with bf16 keys: 880
// queries against 19360 keys, 16 heads of 128, 154 to 162 us a call in MXFP4; traced, 160
// to 163 and 9 for the join, in MXFP8 154 to 156 and 9, from bf16 caches (of 3.8 times the
// bytes) 159 to 161 and 8.  A prompt of 18480 tokens on its own cache, frame-causal: 1.41
// to 1.48 ms in all three.
//
// Few rows (single tokens, drafts; at most 32 of a key head): a wave takes one key head and a
// chunk of keys, in steps of 32.  v_mfma_f32_16x16x32_bf16: lane l = 16 g + r holds
// eight contraction values of row r (operand A) or column r (operand B); the 16 x 16
// result sits in lane l as rows 4 g .. 4 g + 3 of column r.
//     S^T = K Q^T: a lane reads a quarter g of the features of key r as they are
//     stored, one load; they are contracted in the order 8 e + (0..7) of each quarter.
//     O^T += V^T P^T: the eight scores that a lane holds of query r, keys 4 g .. + 3
//     and 16 + 4 g .. + 3, are its operand as they are; V goes through LDS, a tile of
//     the wave's own (LDS serves a wave in order, so no barrier stands anywhere), and
//     is read transposed.
#include "gdn_attn_tile.hpp"

namespace gdnattn {
namespace {

constexpr int kFewWaves = 4, kStep = 32;

// A lane's share of one row: N / 4 dwords' worth of codes.
template <int DW>
struct Raw {
    uint32_t w[DW];
    __device__ __forceinline__ void load(rsrc_t rs, uint32_t at) {
        if constexpr (DW == 1) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
        } else if constexpr (DW == 2) {
            const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0);
            w[0] = x[0], w[1] = x[1];
        } else {
#pragma unroll
            for (int i = 0; i < DW / 4; ++i) {
                const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rs, at + 16 * i, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
            }
        }
    }
};
template <typename F, int DW>
__device__ __forceinline__ u32x4 eight_of(const Raw<DW>& r, int e, float s) {
    if constexpr (F::kPerByte == 2)
        return F::widen(r.w[e], s);
    else
        return F::widen(u32x2{r.w[2 * e], r.w[2 * e + 1]}, s);
}

__device__ __forceinline__ f32x4 mma16(u32x4 x, u32x4 y, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0,
                                                   0, 0);
}
// Over the four lanes that hold one column.
__device__ __forceinline__ float quarters_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float quarters_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// RT row tiles of 16.  Measured: eight single queries against caches of 40 to 32768 keys
// (96 MB), 32 / 8 heads of 128, MXFP4: 24.5 to 25.1 us, 3.9 TB/s; 31 us a call with the
// join, 62 through the tile kernel.  Bound by the instructions of a step, about 200 of
// which 64 widen codes, in two or three waves a SIMD (with every load taken out the same
// steps take 80% of the time); a load of four bytes a lane for each tile's scales costs
// as much to issue as one of codes, so a step's scales come in one load.  MXFP8 heads of
// 128 are bound by memory: 8 x 11008 keys (186 MB) in 41.5 us a call with two waves a
// SIMD (three spill, 46.9), traced 34 to 35 and 4.5 for the join.  8 x 8192 keys, four
// queries each: 21 and 8 in MXFP4, 29 and 8 in MXFP8.
template <typename F, int D, int RT>
__global__ __launch_bounds__(64 * kFewWaves, RT == 1 && D / F::kPerByte < 128 ? 3 : 2) void attn_few_kernel(const AttnArgs a) {
    constexpr int Q = D / 4, E = D / 32, FT = D / 16, DW = Q / F::kPerByte / 4, TB = kStep * D * 2;
    __shared__ __attribute__((aligned(256))) unsigned char lds[kFewWaves][TB];
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // key heads run fastest: the waves of a workgroup read neighbouring rows of the same keys
    // Workgroups go to the eight XCDs in turn.  Short sequences use their first chunks
    // alone, which would meet the same XCDs every time: each eight are rotated (64 requests
    // with room for 16 chunks, all but one of 300 keys: 41 us against 63).
    const unsigned eight = blockIdx.x / 8;
    const unsigned wg = 8 * eight + 8 <= gridDim.x ? 8 * eight + ((blockIdx.x + (eight * 0x9E3779B1u >> 29)) & 7) : blockIdx.x;
    const unsigned unit = wg * kFewWaves + wave;
    const int hk = (int)(unit % (unsigned)a.Hk), rest = (int)(unit / (unsigned)a.Hk);
    const int split = rest % a.splits, sq = rest / a.splits;
    if (sq >= a.n_seq) return;
    const Seq z = sequence(a, sq);
    const int rows = z.lq * a.G;
    if (rows == 0 || (split > 0 && (int64_t)split * a.chunk >= z.lk)) return;
    const int n_first = visible(a, z, 0), n_last = visible(a, z, z.lq - 1);
    // row 16 u + r of tile u: the query's keys, and its place in the outputs
    int n[RT];
    int64_t row[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        const int x = 16 * u + r;
        n[u] = x < rows ? visible(a, z, x / a.G) : 0;
        row[u] = (z.q0 + x / a.G) * a.Hq + hk * a.G + x % a.G;
    }
    const int lo = min(split * a.chunk, n_last), hi = min(lo + a.chunk, n_last);
    u32x4 q[RT][E];
    f32x4 acc[RT][FT];
    const float c2 = a.scale * kLog2e, slack = kSlack / c2;
    float m[RT], ms[RT], limit[RT], l[RT];                    // as in the tile kernel
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        const int x = 16 * u + r;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[u][e] = u32x4{0u, 0u, 0u, 0u};
            if (x < rows)
                q[u][e] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + (z.q0 + x / a.G) * a.ldq +
                                                          (int64_t)(hk * a.G + x % a.G) * D + g * Q + 8 * e);
        }
#pragma unroll
        for (int t = 0; t < FT; ++t) acc[u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        m[u] = limit[u] = -INFINITY;
        ms[u] = l[u] = 0.f;
    }

    const KeysMx<F> kb(a.k, a.k_scale, 0, z.k0, hk, a.Hk, D), vb(a.v, a.v_scale, 0, z.k0, hk, a.Hk, D);
    // the chunk's codes, and the lane's first place in them; past its end: zeros
    const uint32_t bytes = lo < hi ? (uint32_t)(hi - lo - 1) * kb.ldc + D / F::kPerByte : 0;
    const rsrc_t rk = make_rsrc(kb.codes + (int64_t)lo * kb.ldc, bytes), rv = make_rsrc(vb.codes + (int64_t)lo * vb.ldc, bytes);
    const uint32_t place = r * kb.ldc + g * Q / F::kPerByte;
    struct Keys {
        Raw<DW> x[2];
    };
    // keys [n0, n0 + 32) as two tiles of 16.  Without a condition, since waits count
    // loads: where one may not have been issued, the compiler waits for all.
    auto load = [&](Keys& k, Keys& v, int n0) {
        const uint32_t at = place + (uint32_t)(n0 - lo) * kb.ldc;
#pragma unroll
        for (int t = 0; t < 2; ++t) k.x[t].load(rk, at + t * 16 * kb.ldc);
#pragma unroll
        for (int t = 0; t < 2; ++t) v.x[t].load(rv, at + t * 16 * kb.ldc);
    };
    // The scales of a step in one load: those of a key's row in lane key, of its values in
    // lane 32 + key (both kernels 28.4 us, with a load for each tile of each 33.6).
    const uint8_t* const sp = (lane < 32 ? kb.scales : vb.scales);
    auto load_scales = [&](int n0) {
        const uint8_t* const p = sp + (int64_t)min(n0 + (lane & 31), hi - 1) * kb.lds;
        if constexpr (D == 128)
            return *reinterpret_cast<const uint32_t __attribute__((aligned(1)))*>(p);
        else if constexpr (D == 64)
            return (uint32_t)p[0] | (uint32_t)p[1] << 8;
        else
            return (uint32_t)p[0];
    };
    // tile t's scale of the lane's features
    auto scale_at = [&](uint32_t s, int from) {
        const uint32_t row = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (from + r), (int)s);
        return gdnmx::scale_of(row >> (8 * (g * Q / gdnmx::kBlock)) & 255u);
    };
    unsigned char* tile = lds[wave];
    // a lane's places in the tile: chunk g E + e of row r, and eight bytes of chunk 2 t +
    // of key 4 g + r / 4 (the permutation is an exclusive or, so e and t are as well)
    const uint32_t put = chunk_at<D>(r, g * E), get = chunk_at<D>(4 * g + (r >> 2), (r >> 1) & 1) + (r & 1) * 8;
    constexpr int HALF = 16 * D * 2;                          // bytes of 16 keys
    // keys [n0, n0 + 32); their registers then take those of two steps on
    auto step = [&](Keys& k, Keys& v, uint32_t& scales, int n0) {
        f32x4 s[RT][2];
        float sc[2], vs[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int u = 0; u < RT; ++u) s[u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
            sc[t] = scale_at(scales, 16 * t);
            vs[t] = scale_at(scales, 32 + 16 * t);
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const u32x4 kf = eight_of<F>(k.x[t], e, sc[t]);
#pragma unroll
                for (int u = 0; u < RT; ++u) s[u][t] = mma16(kf, q[u][e], s[u][t]);
            }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < E; ++e)
                *reinterpret_cast<u32x4*>(tile + (put ^ (uint32_t)(16 * e)) + t * HALF) = eight_of<F>(v.x[t], e, vs[t]);
        scales = load_scales(n0 + 2 * kStep);
        load(k, v, n0 + 2 * kStep);
        u32x4 p[RT];
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            if (n0 + kStep > n_first) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n0 + 16 * t + 4 * g + i >= n[u]) s[u][t][i] = -INFINITY;
            }
            float top = s[u][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[u][i >> 2][i & 3]);
            if (__any(top > limit[u])) {
                const float mn = fmaxf(m[u], quarters_max(top) * c2);
                const float al = mn == -INFINITY ? 1.f : exp2_f(m[u] - mn);
                m[u] = mn;
                ms[u] = mn == -INFINITY ? 0.f : mn;
                limit[u] = mn / c2 + slack;
                l[u] *= al;
#pragma unroll
                for (int t = 0; t < FT; ++t) acc[u][t] *= al;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float e = exp2_f(__builtin_fmaf(s[u][i >> 2][i & 3], c2, -ms[u]));
                s[u][i >> 2][i & 3] = e;
                l[u] += e;
            }
            // P in bf16: see the tile kernel
            p[u] = u32x4{pack_bf16x2(s[u][0][0], s[u][0][1]), pack_bf16x2(s[u][0][2], s[u][0][3]),
                         pack_bf16x2(s[u][1][0], s[u][1][1]), pack_bf16x2(s[u][1][2], s[u][1][3])};
        }
#pragma unroll
        for (int t = 0; t < FT; ++t) {
            // features 16 t + r of keys 4 g .. + 3 and 16 + 4 g .. + 3
            const u32x2 x = read_tr(tile + (get ^ (uint32_t)(32 * t)));
            const u32x2 y = read_tr(tile + (get ^ (uint32_t)(32 * t)) + HALF);
#pragma unroll
            for (int u = 0; u < RT; ++u) acc[u][t] = mma16(u32x4{x[0], x[1], y[0], y[1]}, p[u], acc[u][t]);
        }
    };
    if (lo < hi) {
        Keys k0, v0, k1, v1;
        uint32_t s0 = load_scales(lo);
        load(k0, v0, lo);
        uint32_t s1 = load_scales(lo + kStep);
        load(k1, v1, lo + kStep);
        for (int n0 = lo; n0 < hi; n0 += 2 * kStep) {             // chunks are whole pairs; past hi all is masked
            step(k0, v0, s0, n0);
            step(k1, v1, s1, n0 + kStep);
        }
    }
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        if (a.causal && !finite(acc[u])) {                    // see finite()
            m[u] = -INFINITY;
            l[u] = 0.f;
#pragma unroll
            for (int t = 0; t < FT; ++t) acc[u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int j = lo; j < hi; ++j) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) s = dot8(q[u][e], kb.eight(j, g * Q + 8 * e), s);
                s = quarters_sum(s) * c2;
                if (j < n[u]) {
                    const float mn = fmaxf(m[u], s), mj = mn == -INFINITY ? 0.f : mn;
                    const float al = exp2_f(m[u] - mj), pj = exp2_f(s - mj);
                    m[u] = mn;
                    l[u] = l[u] * al + (g == 0 ? pj : 0.f);
#pragma unroll
                    for (int t = 0; t < FT; ++t) {
                        const u32x2 x = vb.four(j, 16 * t + 4 * g);
                        acc[u][t] = acc[u][t] * al + pj * f32x4{__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u),
                                                                __uint_as_float(x[1] << 16), __uint_as_float(x[1] & 0xffff0000u)};
                    }
                }
            }
        }
        const float sum = quarters_sum(l[u]);
        if (16 * u + r >= rows) continue;
        const float inv = sum > 0.f ? 1.0f / sum : sum;
        const float lg = sum == 0.f ? -INFINITY : (m[u] + log2_f(sum)) * kLn2;
        if (a.splits > 1) {
            const int64_t pr = (int64_t)split * a.total_q * a.Hq + row[u];
#pragma unroll
            for (int t = 0; t < FT; ++t)
                *reinterpret_cast<f32x4*>(a.part_o + pr * D + 16 * t + 4 * g) = acc[u][t] * inv;
            if (g == 0) a.part_lse[pr] = lg;
        } else {
#pragma unroll
            for (int t = 0; t < FT; ++t)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + row[u] * D + 16 * t + 4 * g) =
                    u32x2{pack_bf16x2(acc[u][t][0] * inv, acc[u][t][1] * inv),
                          pack_bf16x2(acc[u][t][2] * inv, acc[u][t][3] * inv)};
            if (g == 0 && a.lse) a.lse[row[u]] = lg;
        }
    }
}

// o = sum over the splits of exp(lse_s - lse) o_s, a workgroup a row.  Its groups of
// D / 4 lanes take the splits in turn, 128 at once, each with a maximum of its own,
// so that nothing waits for a first look at all of them; the groups are joined in order
// through LDS.  Bound by a launch and two trips to memory: 256 rows of 128, up to 128
// splits, in 5 us.
template <int D>
__global__ __launch_bounds__(256) void attn_few_join_kernel(const AttnArgs a) {
    constexpr int L = D / 4, NG = 256 / L, U = 128 / NG;
    __shared__ f32x4 sums[NG][L];
    __shared__ float tops[NG], weights[NG];
    const int per = a.max_q * a.Hq;
    const Seq z = sequence(a, (int)(blockIdx.x / (unsigned)per));
    const int64_t rr = blockIdx.x % (unsigned)per;
    if (rr >= (int64_t)z.lq * a.Hq) return;
    const int64_t row = z.q0 * a.Hq + rr, all = a.total_q * a.Hq;
    const int splits = max(1, (z.lk + a.chunk - 1) / a.chunk);
    const int group = threadIdx.x / L, c = threadIdx.x % L;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    for (int s0 = group; s0 < splits; s0 += U * NG) {
        float ls[U];
        f32x4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = min(s0 + u * NG, splits - 1) * all + row;
            ls[u] = a.part_lse[at] * kLog2e;
            o[u] = *reinterpret_cast<const f32x4*>(a.part_o + at * D + 4 * c);
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, ls[u]);
        const float base = top == -INFINITY ? 0.f : top, al = exp2_f(m - base);
        m = top;
        acc *= al;
        l *= al;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u * NG < splits) {
                const float w = exp2_f(ls[u] - base);             // 0 for a split that saw nothing
                acc += w * o[u];
                l += w;
            }
    }
    sums[group][c] = acc;
    if (c == 0) {
        tops[group] = m;
        weights[group] = l;
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int i = 1; i < NG; ++i) m = fmaxf(m, tops[i]);
    const float base = m == -INFINITY ? 0.f : m;
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
    l = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const float w = exp2_f(tops[i] - base);
        acc += w * sums[i][c];
        l += w * weights[i];
    }
    const float inv = l > 0.f ? 1.0f / l : l;
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + row * D + 4 * c) =
        u32x2{pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv)};
    if (c == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2_f(l)) * kLn2;
}

gdn_status done() { return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

template <typename F, int D>
gdn_status launch_few(const AttnArgs& a, FewGrids g, hipStream_t s) {
    if (a.max_q * a.G <= 16)
        hipLaunchKernelGGL((attn_few_kernel<F, D, 1>), dim3(g.main), dim3(64 * kFewWaves), 0, s, a);
    else
        hipLaunchKernelGGL((attn_few_kernel<F, D, 2>), dim3(g.main), dim3(64 * kFewWaves), 0, s, a);
    if (a.splits > 1) hipLaunchKernelGGL((attn_few_join_kernel<D>), dim3(g.join), dim3(256), 0, s, a);
    return done();
}
template <typename F>
gdn_status few_by_size(const AttnArgs& a, FewGrids g, hipStream_t s) {
    return a.D == 32 ? launch_few<F, 32>(a, g, s) : a.D == 64 ? launch_few<F, 64>(a, g, s) : launch_few<F, 128>(a, g, s);
}

template <typename F, int D, int NW>
gdn_status launch(AttnArgs a, Grid g, hipStream_t s) {
    a.tiles = g.tiles;
    hipLaunchKernelGGL((attn_fwd_kernel<KeysMx<F>, D, NW>), dim3(g.groups), dim3(64 * NW), 0, s, a);
    return done();
}
template <typename F>
gdn_status by_size(const AttnArgs& a, int rows, Grid g, hipStream_t s) {
    if (a.D == 32) return launch<F, 32, 4>(a, g, s);
    if (a.D == 64) return launch<F, 64, 4>(a, g, s);
    return rows == 256 ? launch<F, 128, 8>(a, g, s) : launch<F, 128, 4>(a, g, s);
}

}  // namespace

gdn_status attn_fwd_mx(const AttnArgs& a, bool fp4, int rows, Grid g, hipStream_t s) {
    return fp4 ? by_size<gdnmx::Fp4>(a, rows, g, s) : by_size<gdnmx::Fp8>(a, rows, g, s);
}

// Keys of a chunk: for about 8192 waves if every sequence were as long as it may be
// (three fit a SIMD, a little over 3000 the card; lengths differ, and short work spreads
// evenly).  Eight single queries of 40 to 32768 keys, 8 key heads of 128, so 256 keys a
// chunk: 28.3 us in both kernels, with 128 keys 34.7, with 512 38.9.
//   - Past 2048 a quarter, so that the longest of many requests is no long tail: one of
//     32768 keys beside 255 of 40 71 us against 204 with 8192, 256 of 8192 keys 555
//     against 560.
//   - 128 at least, and up to 256 where so many waves are left (32 of 2048 keys 23.3 us
//     against 26.6 with 128; 4 of 1500 keys 11.3 with 128, 13.6 with 256) or where the
//     join would take more than 128 splits, its one step (one of 20000 13.7 against 16.4).
//   - More than 16 rows: 256 at least, and up to 512 where there are many, since a chunk's
//     fp32 results grow with the rows: 8 requests of 8 queries and 40 to 32768 keys, 4
//     heads on each of 8, 43.0 us against 53.2; 4 queries, 8 heads on each of 4, 31.9 with
//     256 and 38.7 with 512.
int attn_few_chunk(int rows, int n_seq, int Hk, int D, int max_k) {
    const int64_t all = std::min((int64_t)max_k * n_seq, (int64_t)1 << 45) * Hk;      // Hk is below 2^16
    const int64_t even = (all + 8191) / 8192, keys = std::max(std::min<int64_t>(even, 2048), even / 4);
    // a chunk and the steps behind it within 32-bit offsets
    const int64_t most = ((int64_t)1 << 31) / ((int64_t)Hk * D) - 4 * kStep;
    const int64_t least = rows > 16 ? std::min<int64_t>(std::max<int64_t>(all / 4096 * D / 128, 256), 512)
                                    : std::min<int64_t>(std::max<int64_t>({(all + 2047) / 2048, (max_k + 127) / 128, 128}), 256);
    const int64_t chunk = std::min(std::max(keys, least), most);
    return (int)std::min<int64_t>((chunk + 2 * kStep - 1) / (2 * kStep) * (2 * kStep), std::max(max_k, 1));
}
bool attn_few_grids(const AttnArgs& a, FewGrids* g) {
    if ((int64_t)a.n_seq * a.Hk >= INT32_MAX) return false;
    const int64_t units = (int64_t)a.n_seq * a.Hk * a.splits;
    if (!grid_of((units + kFewWaves - 1) / kFewWaves, 64 * kFewWaves, &g->main)) return false;
    g->join = 0;
    return units < INT32_MAX && (a.splits == 1 || grid_of((int64_t)a.n_seq * a.max_q * a.Hq, 256, &g->join));
}
gdn_status attn_fwd_few(const AttnArgs& a, bool fp4, FewGrids g, hipStream_t s) {
    return fp4 ? few_by_size<gdnmx::Fp4>(a, g, s) : few_by_size<gdnmx::Fp8>(a, g, s);
}

}  // namespace gdnattn
