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

namespace gdnattn {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef short i16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, uint32_t bytes) {
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
// row is permuted by the row, so that neither read meets bank conflicts.
// Row-wise fragments (eight lanes read one chunk column of eight rows):
template <int D>
__device__ __forceinline__ uint32_t row_chunk(int row, int c) {
    return (uint32_t)(row * 2 * D) + (uint32_t)((D >= 64 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
}
// Transposed fragments (sixteen lanes read 32 bytes of four rows):
template <int D>
__device__ __forceinline__ uint32_t col_chunk(int row, int c) {
    return (uint32_t)(row * 2 * D) + (uint32_t)((D >= 64 ? c ^ (2 * (row & 3)) : c ^ (row & 2)) << 4);
}
__device__ __forceinline__ u32x4 read_row(const unsigned char* t, uint32_t off) {
    return *reinterpret_cast<const u32x4*>(t + off);
}
__device__ __forceinline__ u32x2 read_tr(const unsigned char* p) {
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p));
}
// Operand A of a transposed tile: features 32 db + r, rows 16 s + 4 h + 0..3 and
// 16 s + 8 + 4 h + 0..3.
template <int D>
__device__ __forceinline__ u32x4 read_col(const unsigned char* t, int db, int s, int lane) {
    const int j = lane >> 4, q = lane & 15;
    const int row = 16 * s + 4 * (j >> 1) + (q >> 2);
    const int c = 4 * db + 2 * (j & 1) + ((q >> 1) & 1);
    const uint32_t sub = (q & 1) * 8;
    const u32x2 lo = read_tr(t + col_chunk<D>(row, c) + sub), hi = read_tr(t + col_chunk<D>(row + 8, c) + sub);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

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

// (kv head, sequence, split, tile) of a workgroup, the head fastest: workgroups
// go round the eight XCDs in turn, so with eight heads or a multiple each
// XCD's L2 holds the keys of its own heads only.  Tiles run slowest, from the
// last (under a causal mask the longest) to the first.
struct Place {
    int s, hk, tile, split;
};
__device__ __forceinline__ Place place(const AttnArgs& a) {
    unsigned b = blockIdx.x;
    Place p;
    p.hk = (int)(b % (unsigned)a.Hk);
    b /= (unsigned)a.Hk;
    p.s = (int)(b % (unsigned)a.n_seq);
    b /= (unsigned)a.n_seq;
    p.split = (int)(b % (unsigned)a.splits);
    p.tile = a.tiles - 1 - (int)(b / (unsigned)a.splits);
    return p;
}

constexpr int kKeys = 64;       // keys per tile
// The running maximum is raised only when a row's scores pass it by this many
// powers of two (the exponentials then reach 2^8, which costs no precision in
// bf16 or fp32), so most tiles skip the rescaling of the outputs.
constexpr float kSlack = 8.0f;

// Staging of one tile of K and V: global memory to registers to LDS.
template <int D, int NT>
struct Stage {
    static constexpr int N = kKeys * D / 8 / NT;         // 16-byte chunks a thread and tensor
    static_assert(N >= 1, "every thread stages something");
    u32x4 k[N], v[N];
    __device__ __forceinline__ void load(const uint16_t* kb, const uint16_t* vb, int64_t ldk, int64_t ldv, int n0,
                                         int hi, int tid) {
        const int rows = min(kKeys, hi - n0);
        // rows past the range read as zeros
        const rsrc_t rk = make_rsrc(kb + (int64_t)n0 * ldk, (uint32_t)(((rows - 1) * ldk + D) * 2));
        const rsrc_t rv = make_rsrc(vb + (int64_t)n0 * ldv, (uint32_t)(((rows - 1) * ldv + D) * 2));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = tid + j * NT, row = i / (D / 8), c = i % (D / 8);
            k[j] = __builtin_amdgcn_raw_buffer_load_b128(rk, (uint32_t)(row * (int)ldk * 2 + c * 16), 0, 0);
            v[j] = __builtin_amdgcn_raw_buffer_load_b128(rv, (uint32_t)(row * (int)ldv * 2 + c * 16), 0, 0);
        }
    }
    __device__ __forceinline__ void store(unsigned char* kt, unsigned char* vt, int tid) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = tid + j * NT, row = i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<u32x4*>(kt + row_chunk<D>(row, c)) = k[j];
            *reinterpret_cast<u32x4*>(vt + col_chunk<D>(row, c)) = v[j];
        }
    }
};

// One workgroup: NW waves of 32 QB packed query rows each, all walking the same
// key tiles, double-buffered in LDS.
template <int D, int QB, int NW>
__global__ __launch_bounds__(64 * NW, NW * QB <= 8 && QB == 1 ? 2 : 1) void attn_fwd_kernel(const AttnArgs a) {
    constexpr int NT = 64 * NW, BM = 32 * QB * NW, KS = D / 16, DB = D / 32, TB = kKeys * D * 2;
    __shared__ __attribute__((aligned(16))) unsigned char kt[2][TB], vt[2][TB];
    const Place p = place(a);
    const Seq z = sequence(a, p.s);
    const int rows = z.lq * a.G, r0 = p.tile * BM;
    if (r0 >= rows) return;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w0 = r0 + 32 * QB * wave;                       // the wave's first row
    const int upto = visible(a, z, (min(r0 + BM, rows) - 1) / a.G);
    int lo, hi;
    split_range(upto, kKeys, a.splits, p.split, lo, hi);
    // the wave's rows see the keys below n_first all, and none from n_last on
    const int n_first = w0 < rows ? visible(a, z, w0 / a.G) : 0;
    const int n_last = w0 < rows ? visible(a, z, (min(w0 + 32 * QB, rows) - 1) / a.G) : 0;

    u32x4 q[QB][KS];
    f32x16 acc[QB][DB];
    float m[QB], l[QB];
    int n[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        const int row = w0 + 32 * b + r;
        const bool valid = row < rows;
        n[b] = valid ? visible(a, z, row / a.G) : 0;
        const uint16_t* src = valid ? q_row(a, z, p.hk, row) : nullptr;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[b][s] = valid ? *reinterpret_cast<const u32x4*>(src + 16 * s + 8 * h) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < DB; ++e) acc[b][e] = zero16();
        m[b] = -INFINITY;
        l[b] = 0.f;
    }
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + z.k0 * a.ldk + (int64_t)p.hk * D;
    const uint16_t* vb = static_cast<const uint16_t*>(a.v) + z.k0 * a.ldv + (int64_t)p.hk * D;
    const float c2 = a.scale * kLog2e;
    Stage<D, NT> st;
    if (lo < hi) {
        st.load(kb, vb, a.ldk, a.ldv, lo, hi, tid);
        st.store(kt[0], vt[0], tid);
    }
    __syncthreads();
    int buf = 0;
    for (int n0 = lo; n0 < hi; n0 += kKeys, buf ^= 1) {
        const bool more = n0 + kKeys < hi;
        if (more) st.load(kb, vb, a.ldk, a.ldv, n0 + kKeys, hi, tid);
        if (n0 < n_last) {
            f32x16 s[2][QB];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int b = 0; b < QB; ++b) s[t][b] = zero16();
#pragma unroll
            for (int e = 0; e < KS; ++e)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const u32x4 kf = read_row(kt[buf], row_chunk<D>(32 * t + r, 2 * e + h));
#pragma unroll
                    for (int b = 0; b < QB; ++b) s[t][b] = mma(kf, q[b][e], s[t][b]);
                }
            if (n0 + kKeys > n_first) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int b = 0; b < QB; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3) >= n[b]) s[t][b][i] = -INFINITY;
            }
            float mt[QB];
            bool raise = false;
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                float x = s[0][b][0];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x = fmaxf(x, s[t][b][i]);
                mt[b] = half_max(x) * c2;
                raise = raise || mt[b] > m[b] + kSlack;
            }
            if (__any(raise)) {
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    const float mn = fmaxf(m[b], mt[b]);
                    const float al = mn == -INFINITY ? 1.f : exp2_f(m[b] - mn);
                    m[b] = mn;
                    l[b] *= al;
#pragma unroll
                    for (int e = 0; e < DB; ++e) acc[b][e] *= al;
                }
            }
            u32x4 pf[2][QB][2];
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                const float ms = m[b] == -INFINITY ? 0.f : m[b];      // nothing visible so far
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        s[t][b][i] = exp2_f(__builtin_fmaf(s[t][b][i], c2, -ms));
                        sum += s[t][b][i];
                    }
                    pf[t][b][0] = pack8(s[t][b], 0);
                    pf[t][b][1] = pack8(s[t][b], 8);
                }
                l[b] += sum;                                          // this lane's keys; joined at the end
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < DB; ++e) {
                        const u32x4 vf = read_col<D>(vt[buf], e, 2 * t + u, lane);
#pragma unroll
                        for (int b = 0; b < QB; ++b) acc[b][e] = mma(vf, pf[t][b][u], acc[b][e]);
                    }
        }
        if (more) st.store(kt[buf ^ 1], vt[buf ^ 1], tid);
        __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        const float ls = half_sum(l[b]);
        const int row = w0 + 32 * b + r;
        if (row >= rows) continue;
        const float inv = ls > 0.f ? 1.0f / ls : ls;
        const float lg = ls == 0.f ? -INFINITY : (m[b] + log2_f(ls)) * kLn2;
        const int64_t gr = packed_row(a, z, p.hk, row);
        if (a.splits > 1) {
            const int64_t pr = (int64_t)p.split * a.total_q * a.Hq + gr;
#pragma unroll
            for (int e = 0; e < DB; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<f32x4*>(a.part_o + pr * D + 32 * e + 8 * i + 4 * h) =
                        f32x4{acc[b][e][4 * i] * inv, acc[b][e][4 * i + 1] * inv, acc[b][e][4 * i + 2] * inv,
                              acc[b][e][4 * i + 3] * inv};
            if (h == 0) a.part_lse[pr] = lg;
        } else {
#pragma unroll
            for (int e = 0; e < DB; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + gr * D + 32 * e + 8 * i + 4 * h) =
                        u32x2{pack_bf16x2(acc[b][e][4 * i] * inv, acc[b][e][4 * i + 1] * inv),
                              pack_bf16x2(acc[b][e][4 * i + 2] * inv, acc[b][e][4 * i + 3] * inv)};
            if (h == 0 && a.lse) a.lse[gr] = lg;
        }
    }
}

bool grid_of(int64_t n, unsigned* g) {
    if (n > INT32_MAX) return false;
    *g = (unsigned)n;
    return true;
}

template <int D, int QB, int NW>
gdn_status launch_fwd(AttnArgs a, hipStream_t s) {
    unsigned grid;
    a.tiles = (int)(((int64_t)a.max_q * a.G + 32 * QB * NW - 1) / (32 * QB * NW));
    if (!grid_of((int64_t)a.tiles * a.splits * a.Hk * a.n_seq, &grid)) return GDN_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((attn_fwd_kernel<D, QB, NW>), dim3(grid), dim3(64 * NW), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

int attn_fwd_bf16_rows(int max_q, int G, int D) { return 128; }

gdn_status attn_fwd_bf16(const AttnArgs& a, hipStream_t s) {
    if (a.D == 32) return launch_fwd<32, 1, 4>(a, s);
    if (a.D == 64) return launch_fwd<64, 1, 4>(a, s);
    return launch_fwd<128, 1, 4>(a, s);
}

}  // namespace gdnattn
