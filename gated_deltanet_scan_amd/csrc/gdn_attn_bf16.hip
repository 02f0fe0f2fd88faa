// Softmax attention in bf16 matrix instructions (D in {32, 64, 128}); the
// mathematics, the mask and the entry points are in gdn_attn.hip.
//
// v_mfma_f32_32x32x16_bf16: lane l = 32 h + r holds eight contraction values of
// row r (operand A) or column r (operand B); the 32 x 32 result sits in lane l
// as column r, value i at row 8 (i / 4) + 4 h + i % 4.  As in the fp32 kernels
// the scores are formed transposed, S^T = K Q^T with a wave's query rows as
// columns, so the exponentials of one lane are already the B operand of
// O^T += V^T P^T: a lane's eight values of a 16-key step are keys 4 h + 0..3 and
// 8 + 4 h + 0..3, and V^T is read from LDS in that same order by the transpose
// read (four keys of one feature at a time).
#include "gdn_attn.hpp"

#include <algorithm>
#include <type_traits>

namespace gdnattn {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef short i16x4 __attribute__((ext_vector_type(4)));

// The base must be the same in all lanes and known to be (a descriptor in vector
// registers turns every load into a loop over its values).
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, uint32_t bytes) {
    p = reinterpret_cast<const void*>(uniform((int64_t)p));
    bytes = (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ f32x16 mma(u32x4 x, u32x4 y, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
    return f32x16{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}
// The other half's value (lane l ^ 32), by exchanging halves of two registers.
__device__ __forceinline__ float half_max(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// LDS tiles hold rows of D features in 16-byte chunks whose place within the
// row is permuted by the row.  LDS serves 256 bytes a cycle: sixteen lanes of a
// row-wise fragment (one chunk column of sixteen rows) and 32 lanes of a
// transposed one (64 bytes of four rows).  The permutation sends each of these
// to different banks: the row's lowest two bits move groups of four chunks, the
// next two permute within a group (a row of D = 64 is half of the 256 bytes and
// one of D = 32 a quarter, so they need one bit and two bits less).  With a
// permutation made for 128 bytes a cycle both reads took twice the cycles.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
    const int f = (D == 128 ? (row & 3) << 2 : D == 64 ? (row & 2) << 1 : 0) + ((row >> 2) & 3);
    return (uint32_t)(row * 2 * D) + (uint32_t)((c ^ f) << 4);
}
__device__ __forceinline__ u32x2 read_tr(const unsigned char* p) {
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p));
}
// A lane's addresses in a tile.  The permutation is an exclusive or within the
// bits that the chunk alone sets, so all of them follow from three.  renew()
// keeps the compiler from holding the rest (16 registers at D = 128) across the
// whole loop, where the backward kernels have none to spare.
template <int D>
struct Addr {
    uint32_t row, lo, hi;
    __device__ __forceinline__ void init(int lane) {
        const int h = lane >> 5, r = lane & 31, j = lane >> 4, q = lane & 15;
        const int k = 4 * (j >> 1) + (q >> 2), c = 2 * (j & 1) + ((q >> 1) & 1);
        row = chunk_at<D>(r, h);
        lo = chunk_at<D>(k, c) + (q & 1) * 8;
        hi = chunk_at<D>(k + 8, c) + (q & 1) * 8;
    }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(row), "+v"(lo), "+v"(hi)); }
    // rows 32 t + r, features 16 e + 8 h .. + 7
    __device__ __forceinline__ u32x4 rows(const unsigned char* tile, int t, int e) const {
        return *reinterpret_cast<const u32x4*>(tile + (row ^ (uint32_t)(32 * e)) + t * 64 * D);
    }
    // features 32 e + r, rows 16 s + 4 h + 0..3 and 16 s + 8 + 4 h + 0..3
    __device__ __forceinline__ u32x4 cols(const unsigned char* tile, int e, int s) const {
        const u32x2 a = read_tr(tile + (lo ^ (uint32_t)(64 * e)) + s * 32 * D);
        const u32x2 b = read_tr(tile + (hi ^ (uint32_t)(64 * e)) + s * 32 * D);
        return u32x4{a[0], a[1], b[0], b[1]};
    }
};

// Eight values as one bf16 operand.
__device__ __forceinline__ u32x4 pack8(const f32x16& x, int at) {
    return u32x4{pack_bf16x2(x[at], x[at + 1]), pack_bf16x2(x[at + 2], x[at + 3]),
                 pack_bf16x2(x[at + 4], x[at + 5]), pack_bf16x2(x[at + 6], x[at + 7])};
}

// Row r of the packed row axis of kv head hk: its global (token, head) row.
__device__ __forceinline__ int64_t packed_row(const AttnArgs& a, const Seq& z, int hk, int r) {
    return (z.q0 + r / a.G) * a.Hq + hk * a.G + r % a.G;
}
__device__ __forceinline__ const uint16_t* q_row(const AttnArgs& a, const Seq& z, int hk, int r) {
    return static_cast<const uint16_t*>(a.q) + (z.q0 + r / a.G) * a.ldq + (int64_t)(hk * a.G + r % a.G) * a.D;
}

// For the sums formed again element by element: a lane's half of the features
// of one row (16 s + 8 h .. + 7) times its own, summed over both halves, and
// w times the features that its result registers stand for (32 e + 8 i + 4 h ..).
template <int KS>
__device__ __forceinline__ float dot_row(const u32x4 (&f)[KS], const uint16_t* row, int h) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < KS; ++e) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(row + 16 * e + 8 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s += __uint_as_float(f[e][j] << 16) * __uint_as_float(x[j] << 16);
            s += __uint_as_float(f[e][j] & 0xffff0000u) * __uint_as_float(x[j] & 0xffff0000u);
        }
    }
    return half_sum(s);
}
template <int DB>
__device__ __forceinline__ void add_row(f32x16 (&acc)[DB], float w, const uint16_t* row, int h) {
#pragma unroll
    for (int e = 0; e < DB; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(row + 32 * e + 8 * i + 4 * h);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                acc[e][4 * i + 2 * j] += w * __uint_as_float(x[j] << 16);
                acc[e][4 * i + 2 * j + 1] += w * __uint_as_float(x[j] & 0xffff0000u);
            }
        }
}

constexpr int kKeys = 64;       // keys per tile
// The running maximum is raised only when a row's scores pass it by this many
// powers of two (the exponentials then reach 2^8, which costs no precision in
// bf16 or fp32), so most tiles skip the rescaling of the outputs.
constexpr float kSlack = 8.0f;

// Staging of one tile of keys: global memory to registers to LDS.  Rows past the
// range read as zeros.
template <int D, int NT>
struct Tile {
    static constexpr int N = kKeys * D / 8 / NT;         // 16-byte chunks a thread
    static_assert(N >= 1, "every thread stages something");
    u32x4 x[N];
    __device__ __forceinline__ void load(const uint16_t* base, int64_t ld, int n0, int hi, int tid) {
        const int rows = min(kKeys, hi - n0);
        const rsrc_t rs = make_rsrc(base + (int64_t)n0 * ld, (uint32_t)(((rows - 1) * ld + D) * 2));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = tid + j * NT, row = i / (D / 8), c = i % (D / 8);
            x[j] = __builtin_amdgcn_raw_buffer_load_b128(rs, (uint32_t)row * tile_stride(ld) * 2 + c * 16, 0, 0);
        }
    }
    __device__ __forceinline__ void store(unsigned char* t, int tid) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = tid + j * NT, row = i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<u32x4*>(t + chunk_at<D>(row, c)) = x[j];
        }
    }
};

// One workgroup: NW waves of 32 packed query rows each, all walking the same
// key tiles, double-buffered in LDS.
//
// A wave walks the keys in steps of 32 and keeps three of them in flight: the
// scores of the next step and the output products of the last one (16 matrix
// instructions, 512 cycles) stand beside the exponentials of this one (about
// 450 cycles of vector instructions), with no dependence between them, so both
// pipes of a SIMD work at once.  K of a tile is therefore in LDS half a tile
// before V of it.
//
// Measured: frame-causal clip of 18480 tokens, 16 heads of 128: 2.88 million
// cycles, 1.39 to 1.48 ms a call at the 2.07 to 1.95 GHz that cards hold with
// calls in a row (the first calls after a pause run at 1.6 to 1.8 GHz), which is
// 1060 to 1000 TFLOP/s; the matrix pipes are busy half the time, two waves a SIMD
// leave the rest to dependences within a step.  Sequences of unequal lengths leave
// waves idle as well: the longest walk, not the sum of them, sets the time.
// 4096 x 4096, 16 heads, no mask: 908 TFLOP/s at D = 128 (256 workgroups, one
// round), 655 at 64 and 473 at 32, where exponentials (16 a lane and step
// whatever D is) bound it.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attn_fwd_kernel(const AttnArgs a) {
    constexpr int NT = 64 * NW, BM = 32 * NW, KS = D / 16, DB = D / 32, TB = kKeys * D * 2, HB = TB / 2;
    __shared__ __attribute__((aligned(16))) unsigned char kt[2][TB], vt[2][TB];
    const Place p = find_place<false>(a, BM);
    if (p.s < 0) return;
    const Seq z = sequence(a, p.s);
    const int rows = z.lq * a.G, r0 = p.tile * BM;
    if (r0 >= rows) return;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w0 = r0 + 32 * wave, row = w0 + r;              // the wave's first row, the lane's
    const bool valid = row < rows;
    const int upto = visible(a, z, (min(r0 + BM, rows) - 1) / a.G);
    const int lo = min(p.split * a.chunk, upto), hi = min(lo + a.chunk, upto);
    if (p.split > 0 && p.split * a.chunk >= z.lk) return;     // a shorter sequence has fewer splits
    // the wave's rows see the keys below n_first all, and none from n_last on
    const int n_first = w0 < rows ? visible(a, z, w0 / a.G) : 0;
    const int n_last = w0 < rows ? visible(a, z, (min(w0 + 32, rows) - 1) / a.G) : 0;
    const int n = valid ? visible(a, z, row / a.G) : 0;

    u32x4 q[KS];
    f32x16 acc[DB];
    const u32x4 none = {0u, 0u, 0u, 0u};
    {
        const uint16_t* src = valid ? q_row(a, z, p.hk, row) : nullptr;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[s] = valid ? *reinterpret_cast<const u32x4*>(src + 16 * s + 8 * h) : none;
    }
#pragma unroll
    for (int e = 0; e < DB; ++e) acc[e] = zero16();
    const float c2 = a.scale * kLog2e, slack = kSlack / c2;
    // running maximum (powers of two), the same with 0 before any key, the raw
    // score from which it has to be raised, and the lane's part of the sum
    float m = -INFINITY, ms = 0.f, limit = -INFINITY, l = 0.f;

    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + z.k0 * a.ldk + (int64_t)p.hk * D;
    const uint16_t* vb = static_cast<const uint16_t*>(a.v) + z.k0 * a.ldv + (int64_t)p.hk * D;
    Addr<D> ad;
    ad.init(lane);
    Tile<D, NT> sk, sv;                                       // on their way: K of the next tile, V of this one

    // keys [base, base + 32): scores in `cur`; `nxt` takes the next scores, `last`
    // holds the step before, `now` takes this one's exponentials
    auto step = [&](f32x16& cur, f32x16& nxt, u32x4(&last)[2], u32x4(&now)[2], const unsigned char* k_next,
                    const unsigned char* v_last, int base) {
        if (base + 32 > n_first) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (base + 8 * (i >> 2) + 4 * h + (i & 3) >= n) cur[i] = -INFINITY;
        }
        float top = cur[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, cur[i]);
        if (__any(top > limit)) {
            // a row's two lanes share one maximum; what they hold is scaled to it
            const float mn = fmaxf(m, half_max(top) * c2);
            const float al = mn == -INFINITY ? 1.f : exp2_f(m - mn);
            m = mn;
            ms = mn == -INFINITY ? 0.f : mn;
            limit = mn / c2 + slack;
            l *= al;
#pragma unroll
            for (int e = 0; e < DB; ++e) acc[e] *= al;
            // the step still pending, rounded to bf16 once more: in fp32 it would take
            // 8 registers more, and a row comes here a few times at most
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    last[u][i] = pack_bf16x2(__uint_as_float(last[u][i] << 16) * al,
                                             __uint_as_float(last[u][i] & 0xffff0000u) * al);
        }
        __builtin_amdgcn_s_setprio(1);                        // over a wave that stages or masks: 1.3% faster
        nxt = zero16();
#pragma unroll
        for (int e = 0; e < KS; ++e) nxt = mma(ad.rows(k_next, 0, e), q[e], nxt);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < DB; ++e) acc[e] = mma(ad.cols(v_last, e, u), last[u], acc[e]);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            cur[i] = exp2_f(__builtin_fmaf(cur[i], c2, -ms));
            sum += cur[i];
        }
        l += sum;                                             // this lane's keys; joined at the end
        // P in bf16, which the products take: off by half a step (2^-8 at most,
        // 1.7e-3 in the mean square), as much as o's own rounding
        now[0] = pack8(cur, 0);
        now[1] = pack8(cur, 8);
        __builtin_amdgcn_s_setprio(0);
    };

    if (lo < hi) {
        sk.load(kb, a.ldk, lo, hi, tid);
        sk.store(kt[0], tid);
        if (lo + kKeys < hi) sk.load(kb, a.ldk, lo + kKeys, hi, tid);
        sv.load(vb, a.ldv, lo, hi, tid);
        for (int i = tid; i < HB / 16; i += NT) *reinterpret_cast<u32x4*>(vt[1] + HB + 16 * i) = none;
        __syncthreads();
        f32x16 s0 = zero16(), s1;
        u32x4 p0[2], p1[2] = {none, none};                    // no step before the first
#pragma unroll
        for (int e = 0; e < KS; ++e) s0 = mma(ad.rows(kt[0], 0, e), q[e], s0);
        int buf = 0;
        for (int n0 = lo; n0 < hi; n0 += kKeys, buf ^= 1) {
            // a step past the wave's last key still adds the step before it
            if (n0 < n_last + 32) step(s0, s1, p1, p0, kt[buf] + HB, vt[buf ^ 1] + HB, n0);
            sk.store(kt[buf ^ 1], tid);                       // past the last tile: never used
            sv.store(vt[buf], tid);
            __syncthreads();
            if (n0 + kKeys < hi) {
                if (n0 + 2 * kKeys < hi) sk.load(kb, a.ldk, n0 + 2 * kKeys, hi, tid);
                sv.load(vb, a.ldv, n0 + kKeys, hi, tid);
            }
            if (n0 + 32 < n_last + 32) step(s1, s0, p0, p1, kt[buf ^ 1], vt[buf], n0 + 32);
        }
        if ((hi - 1 - lo) / kKeys * kKeys + lo + 32 < n_last) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < DB; ++e) acc[e] = mma(ad.cols(vt[buf ^ 1] + HB, e, u), p1[u], acc[e]);
        }
    }
    if (a.causal && !finite(acc)) {                           // see finite()
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < DB; ++e) acc[e] = zero16();
        const int end = min(hi, n_last);
#pragma unroll 1
        for (int j = lo; j < end; ++j) {
            const float s = dot_row(q, kb + (int64_t)j * a.ldk, h) * c2;
            if (j < n) {
                const float mn = fmaxf(m, s), mj = mn == -INFINITY ? 0.f : mn;
                const float al = exp2_f(m - mj), pj = exp2_f(s - mj);
                m = mn;
                l = l * al + (h == 0 ? pj : 0.f);
#pragma unroll
                for (int e = 0; e < DB; ++e) acc[e] *= al;
                add_row(acc, pj, vb + (int64_t)j * a.ldv, h);
            }
        }
    }
    l = half_sum(l);
    if (!valid) return;
    const float inv = l > 0.f ? 1.0f / l : l;
    const float lg = l == 0.f ? -INFINITY : (m + log2_f(l)) * kLn2;
    const int64_t gr = packed_row(a, z, p.hk, row);
    if (a.splits > 1) {
        const int64_t pr = (int64_t)p.split * a.total_q * a.Hq + gr;
#pragma unroll
        for (int e = 0; e < DB; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4*>(a.part_o + pr * D + 32 * e + 8 * i + 4 * h) =
                    f32x4{acc[e][4 * i] * inv, acc[e][4 * i + 1] * inv, acc[e][4 * i + 2] * inv,
                          acc[e][4 * i + 3] * inv};
        if (h == 0) a.part_lse[pr] = lg;
    } else {
#pragma unroll
        for (int e = 0; e < DB; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + gr * D + 32 * e + 8 * i + 4 * h) =
                    u32x2{pack_bf16x2(acc[e][4 * i] * inv, acc[e][4 * i + 1] * inv),
                          pack_bf16x2(acc[e][4 * i + 2] * inv, acc[e][4 * i + 3] * inv)};
        if (h == 0 && a.lse) a.lse[gr] = lg;
    }
}

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
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + z.k0 * a.ldk + (int64_t)p.hk * D;
    const uint16_t* vb = static_cast<const uint16_t*>(a.v) + z.k0 * a.ldv + (int64_t)p.hk * D;
    const float c2 = a.scale * kLog2e;
    Addr<D> ad;
    ad.init(lane);
    Tile<D, NT> sk, sv;
    auto walk = [&](auto first) {
        constexpr bool kFirst = decltype(first)::value;
        float exact = 0.f;
        if (upto > 0) {
            sk.load(kb, a.ldk, 0, upto, tid);
            sv.load(vb, a.ldv, 0, upto, tid);
            sk.store(kt[0], tid);
            sv.store(vt[0], tid);
        }
        __syncthreads();
        int buf = 0;
        for (int n0 = 0; n0 < upto; n0 += kKeys, buf ^= 1) {
            const bool more = n0 + kKeys < upto;
            if (more) {
                sk.load(kb, a.ldk, n0 + kKeys, upto, tid);
                sv.load(vb, a.ldv, n0 + kKeys, upto, tid);
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
            const uint16_t* kr = kb + (int64_t)j * a.ldk;
            const float s = dot_row(q, kr, h), dp = dot_row(g, vb + (int64_t)j * a.ldv, h);
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
    hipLaunchKernelGGL((attn_fwd_kernel<D, NW>), dim3(g.groups), dim3(64 * NW), 0, s, a);
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
