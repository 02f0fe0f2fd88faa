// Softmax attention in bf16 matrix instructions: what its kernels share (operand
// layouts, LDS tiles, the staging of keys), and the forward kernel, which takes
// keys and values as bf16 or as block-scaled codes.
//
// v_mfma_f32_32x32x16_bf16: lane l = 32 h + r holds eight contraction values of
// row r (operand A) or column r (operand B); the 32 x 32 result sits in lane l
// as column r, value i at row 8 (i / 4) + 4 h + i % 4.  As in the fp32 kernels
// the scores are formed transposed, S^T = K Q^T with a wave's query rows as
// columns, so the exponentials of one lane are already the B operand of
// O^T += V^T P^T: a lane's eight values of a 16-key step are keys 4 h + 0..3 and
// 8 + 4 h + 0..3, and V^T is read from LDS in that same order by the transpose
// read (four keys of one feature at a time).
#pragma once

#include "gdn_attn.hpp"
#include "gdn_mx.hpp"

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
__device__ __forceinline__ float dot8(u32x4 f, u32x4 x, float s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s += __uint_as_float(f[j] << 16) * __uint_as_float(x[j] << 16);
        s += __uint_as_float(f[j] & 0xffff0000u) * __uint_as_float(x[j] & 0xffff0000u);
    }
    return s;
}
__device__ __forceinline__ void add4(f32x16& acc, int at, float w, u32x2 x) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        acc[at + 2 * j] += w * __uint_as_float(x[j] << 16);
        acc[at + 2 * j + 1] += w * __uint_as_float(x[j] & 0xffff0000u);
    }
}
template <int KS>
__device__ __forceinline__ float dot_row(const u32x4 (&f)[KS], const uint16_t* row, int h) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < KS; ++e) s = dot8(f[e], *reinterpret_cast<const u32x4*>(row + 16 * e + 8 * h), s);
    return half_sum(s);
}
template <int DB>
__device__ __forceinline__ void add_row(f32x16 (&acc)[DB], float w, const uint16_t* row, int h) {
#pragma unroll
    for (int e = 0; e < DB; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            add4(acc[e], 4 * i, w, *reinterpret_cast<const u32x2*>(row + 32 * e + 8 * i + 4 * h));
}

constexpr int kKeys = 64;       // keys per tile
// The running maximum is raised only when a row's scores pass it by this many
// powers of two (the exponentials then reach 2^8, which costs no precision in
// bf16 or fp32), so most tiles skip the rescaling of the outputs.
constexpr float kSlack = 8.0f;

// Keys (or values) of one sequence and head, as the forward kernel reads them:
// where they are, their staging of one tile (global memory to registers to LDS;
// rows past the range read as zeros), and a row of them for the sums formed again.
struct KeysBf16 {
    const uint16_t* base;
    int64_t ld;
    __device__ __forceinline__ KeysBf16(const void* p, const uint8_t*, int64_t ld_, int64_t first, int hk, int, int D)
        : base(static_cast<const uint16_t*>(p) + first * ld_ + (int64_t)hk * D), ld(ld_) {}
    template <int D, int NT>
    struct Tile {
        static constexpr int N = kKeys * D / 8 / NT;         // 16-byte chunks a thread
        static_assert(N >= 1, "every thread stages something");
        u32x4 x[N];
        __device__ __forceinline__ void load(const KeysBf16& k, int n0, int hi, int tid) {
            const int rows = min(kKeys, hi - n0);
            const rsrc_t rs = make_rsrc(k.base + (int64_t)n0 * k.ld, (uint32_t)(((rows - 1) * k.ld + D) * 2));
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int i = tid + j * NT, row = i / (D / 8), c = i % (D / 8);
                x[j] = __builtin_amdgcn_raw_buffer_load_b128(rs, (uint32_t)row * tile_stride(k.ld) * 2 + c * 16, 0, 0);
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
    template <int KS>
    __device__ __forceinline__ float dot(const u32x4 (&f)[KS], int64_t j, int h) const {
        return dot_row(f, base + j * ld, h);
    }
    template <int DB>
    __device__ __forceinline__ void add(f32x16 (&acc)[DB], float w, int64_t j, int h) const {
        add_row(acc, w, base + j * ld, h);
    }
};

// Block-scaled keys: codes and scales of packed tokens.  A thread stages 16
// features, half a scale's block: 8 or 16 bytes and the block's scale, widened to
// bf16 on the way to LDS (exact).
template <typename F>
struct KeysMx {
    const uint8_t *codes, *scales;
    uint32_t ldc, lds;                                    // bytes from one token to the next
    __device__ __forceinline__ KeysMx(const void* p, const uint8_t* s, int64_t, int64_t first, int hk, int Hk, int D) {
        ldc = (uint32_t)(Hk * D / F::kPerByte);
        lds = (uint32_t)(Hk * D / gdnmx::kBlock);
        codes = static_cast<const uint8_t*>(p) + first * ldc + hk * D / F::kPerByte;
        scales = s + first * lds + hk * D / gdnmx::kBlock;
    }
    template <int D, int NT>
    struct Tile {
        static constexpr int U = kKeys * D / 16, N = (U + NT - 1) / NT, B = 16 / F::kPerByte;
        typename F::Raw16 x[N];
        uint32_t s[N];
        __device__ __forceinline__ void load(const KeysMx& k, int n0, int hi, int tid) {
            const uint32_t last = (uint32_t)(min(kKeys, hi - n0) - 1);
            const rsrc_t rc = make_rsrc(k.codes + (int64_t)n0 * k.ldc, last * k.ldc + D / F::kPerByte);
            const rsrc_t rs = make_rsrc(k.scales + (int64_t)n0 * k.lds, last * k.lds + D / gdnmx::kBlock);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t i = tid + j * NT, row = i / (D / 16), c = i % (D / 16);
                if constexpr (F::kPerByte == 2)
                    x[j] = __builtin_amdgcn_raw_buffer_load_b64(rc, row * k.ldc + c * B, 0, 0);
                else
                    x[j] = __builtin_amdgcn_raw_buffer_load_b128(rc, row * k.ldc + c * B, 0, 0);
                s[j] = __builtin_amdgcn_raw_buffer_load_b8(rs, row * k.lds + c / 2, 0, 0);
            }
        }
        __device__ __forceinline__ void store(unsigned char* t, int tid) const {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int i = tid + j * NT, row = i / (D / 16), c = i % (D / 16);
                if (U % NT && i >= U) continue;
                const float sc = gdnmx::scale_of(s[j]);
                // neighbouring rows (pairs of them at 64) begin with different halves, so that
                // a store meets all banks alike (880 queries, 19360 MXFP8 keys, 16 heads of
                // 128, calls in turn: 170 us against 174)
                const int odd = D == 128 ? row & 1 : D == 64 ? (row >> 1) & 1 : 0;
                *reinterpret_cast<u32x4*>(t + chunk_at<D>(row, 2 * c + odd)) = F::widen(odd ? F::high(x[j]) : F::low(x[j]), sc);
                *reinterpret_cast<u32x4*>(t + chunk_at<D>(row, 2 * c + 1 - odd)) = F::widen(odd ? F::low(x[j]) : F::high(x[j]), sc);
            }
        }
    };
    // Features [at, at + 8) of key j, and four of them, as bf16.
    __device__ __forceinline__ u32x4 eight(int64_t j, int at) const {
        return F::widen(*reinterpret_cast<const typename F::Raw8*>(codes + j * ldc + at / F::kPerByte),
                        gdnmx::scale_of(scales[j * lds + at / gdnmx::kBlock]));
    }
    __device__ __forceinline__ u32x2 four(int64_t j, int at) const {
        return F::widen4(codes + j * ldc + at / F::kPerByte, gdnmx::scale_of(scales[j * lds + at / gdnmx::kBlock]));
    }
    template <int KS>
    __device__ __forceinline__ float dot(const u32x4 (&f)[KS], int64_t j, int h) const {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < KS; ++e) s = dot8(f[e], eight(j, 16 * e + 8 * h), s);
        return half_sum(s);
    }
    template <int DB>
    __device__ __forceinline__ void add(f32x16 (&acc)[DB], float w, int64_t j, int h) const {
#pragma unroll
        for (int e = 0; e < DB; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) add4(acc[e], 4 * i, w, four(j, 32 * e + 8 * i + 4 * h));
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
template <typename KV, int D, int NW>
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

    const KV kb(a.k, a.k_scale, a.ldk, z.k0, p.hk, a.Hk, D), vb(a.v, a.v_scale, a.ldv, z.k0, p.hk, a.Hk, D);
    Addr<D> ad;
    ad.init(lane);
    typename KV::template Tile<D, NT> sk, sv;                                       // on their way: K of the next tile, V of this one

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
        sk.load(kb, lo, hi, tid);
        sk.store(kt[0], tid);
        if (lo + kKeys < hi) sk.load(kb, lo + kKeys, hi, tid);
        sv.load(vb, lo, hi, tid);
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
                if (n0 + 2 * kKeys < hi) sk.load(kb, n0 + 2 * kKeys, hi, tid);
                sv.load(vb, n0 + kKeys, hi, tid);
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
            const float s = kb.dot(q, j, h) * c2;
            if (j < n) {
                const float mn = fmaxf(m, s), mj = mn == -INFINITY ? 0.f : mn;
                const float al = exp2_f(m - mj), pj = exp2_f(s - mj);
                m = mn;
                l = l * al + (h == 0 ? pj : 0.f);
#pragma unroll
                for (int e = 0; e < DB; ++e) acc[e] *= al;
                vb.add(acc, pj, j, h);
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

}  // namespace
}  // namespace gdnattn
