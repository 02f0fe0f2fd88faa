// Products of 8-bit floats with a scale for each block of 128: the C ABI of
// gdn_matmul_fp8 (declared in include/gdn.h).
//
//     y[m][n] = sum over blocks b of 128 columns of
//               x_scale[m][b] w_scale[n / 128][b] sum_{k in b} x[m][k] w[n][k]
//
// v_mfma_f32_16x16x128_f8f6f4: lane l = 16 g + r holds 32 contraction values of
// row r (operand A) or column r (operand B); the 16 x 16 result sits in lane l
// as rows 4 g .. 4 g + 3 of column r.  Both operands take the same 32 places of a
// row, so their order within the block does not matter.  The products are formed
// transposed, rows of w as operand A: a lane then holds four outputs of one token,
// which needs one scale of x, and its store is four values wide.  One instruction
// contracts exactly one scale's block; its result starts from zero and is added to
// the fp32 sum with the block's scale.
#include "gdn_matmul_rule.hpp"
#include "gdn_ops.hpp"

#include <algorithm>

namespace {

using namespace gdnops;
using namespace gdnmatmul;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;

struct MatmulArgs {
    const uint8_t *x, *w;
    const float *xs, *ws;
    uint16_t* y;
    int64_t M;
    int N, K, kb, part;              // part: columns of one of the outputs
    int tiles_n, tiles_m;
};

typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ f32x4 mma(i32x8 a, i32x8 b) {
    // without the instruction's own (power of two) scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// ---------------------------------------------------------------- tiles
// Rows of tiles that an XCD walks together: 1220 us for 106480 x 6144, K = 2048, as with
// four; with two 1252, with sixteen 1249.
constexpr unsigned kTileRows = 8;

// Memory to LDS, 16 or 4 bytes a lane, one run of a wave's lanes at `to` (a
// wave-uniform LDS address); places past the descriptor's end are written as zeros.
// Written as assembly because the compiler, which cannot tell the stages apart, waits
// for every such load before the next read of LDS.  It has no output register;
// wait_loads orders it.
__device__ __forceinline__ void load_lds16(u32x4 rsrc, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(offset), "s"(rsrc)
                 : "m0");
}
__device__ __forceinline__ void load_lds4(u32x4 rsrc, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(offset), "s"(rsrc)
                 : "m0");
}
// All but the wave's N youngest loads and stores are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ u32x4 descriptor(const void* p, int64_t bytes) {
    const uint64_t at = (uint64_t)uniform((int64_t)p);
    return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform((int64_t)p)), 0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
constexpr uint32_t kNowhere = 0x80000000u;    // past the end of every descriptor, with room for a tile's steps

// Tiles of TN columns of y and TM tokens, S stages of one block each.
//
// A workgroup walks tiles without a pause: loads run S - 1 blocks ahead across the ends
// of tiles, one beside each of a block's first products (all at its start, they kept
// both waves of a SIMD from their products: 1325 us against 1250).  A block has one
// barrier, before its last row of products: by then its fragments are read, and the
// next block's first ones are read beside those products.  Sums stand two products
// behind, so a wave waits for none of them.
//
// Bound by power: 106480 x 6144, K = 2048, takes 1.19 to 1.56 ms from card to card and
// launch to launch, 2250 to 1720 TFLOP/s (calls in a row 1.24 to 1.34, traced launches
// 1.28 to 1.43).  Its 2.36 million cycles (1.28 of them of matrix instructions on every
// SIMD) pass at 1.5 to 2.0 GHz, with operands of zeros at 2.4; a library product with one
// scale for everything takes 1.00 ms on the faster cards.  Of the cycles 0.3 million are
// the ends of tiles.
template <int TN, int TM, int WN, int WM, int S>
__global__ __launch_bounds__(64 * WN * WM, 2) void matmul_kernel(const MatmulArgs a) {
    constexpr int WAVES = WN * WM, FN = TN / WN, FM = TM / WM, NI = FN / 16, NT = FM / 16;
    constexpr int JN = TN / 8 / WAVES, JM = TM / 8 / WAVES, LOADS = JN + JM + 2;
    constexpr int XS = (TN + TM) * kBlock, WS = XS + TM * 4, STAGE = WS + 256;    // bytes: operands, scales of x, of w
    // the loads of a block stand between the first products of another, all of them
    // before its last row of products, where the wait counts them
    constexpr int BEFORE = LOADS < (NI - 1) * NT ? LOADS : (NI - 1) * NT;
    static_assert(kBlock % FN == 0 && FN % 64 == 0 && FM % 16 == 0 && WAVES % 4 == 0 && JN >= 1 && JM >= 1 && TM % 64 == 0 && S >= 2, "");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S * STAGE];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15, K = a.K;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave % WN, wm = wave / WN;
    // The eight XCDs, which take workgroups in turn, each walk a range of tiles, eight
    // rows of tiles at a time: what its workgroups read at once is shared in its L2.
    const unsigned tiles = a.tiles_n * a.tiles_m, xcd = blockIdx.x % 8, per = tiles / 8, rem = tiles % 8;
    const unsigned first = xcd * per + min(xcd, rem), end = first + per + (xcd < rem), step = (gridDim.x + 7 - xcd) / 8;
    auto tile_at = [&](unsigned id, int& n0, int64_t& m0) {
        const unsigned gm = kTileRows, group = id / (gm * a.tiles_n), in = id % (gm * a.tiles_n), rows = min(gm, a.tiles_m - group * gm);
        m0 = (int64_t)(group * gm + in % rows) * TM;
        n0 = (int)(in / rows) * TN;
    };
    const unsigned id0 = first + blockIdx.x / 8;
    if (id0 >= end) return;
    // ---- loads, S blocks ahead of their use
    // Rows of 128 bytes in eight chunks, chunk c of row r at place c ^ f(r): the sixteen
    // rows of a fragment, in the two chunk columns that a read takes, meet all banks
    // alike.  f(r) is (r / 2) % 8 for x; for w, whose fragments take runs of four rows
    // eight apart, bit 1 of r and then bits 3 and 4.
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds;
    const uint32_t row = 8 * wave + (lane >> 3);
    const uint32_t cw = (lane & 7) ^ (((lane >> 4) & 1) | (wave & 3) << 1), cx = (lane & 7) ^ ((lane >> 4) | (wave & 1) << 2);
    const uint32_t ow = row * K + cw * 16, ox = row * K + cx * 16, down = 8 * WAVES * K;
    const uint32_t osx = (64 * (wave % (TM / 64)) + lane) * a.kb * 4, osw = (lane % (TN > kBlock ? TN / kBlock : 1)) * a.kb * 4;
    unsigned next = id0;                                      // tile and block of the next load
    int nb = 0, stage = 0;
    u32x4 rw, rx, rsw, rsx;
    auto open = [&]() {
        int n0 = 0;
        int64_t m0 = 0;
        const bool some = next < end;
        if (some) tile_at(next, n0, m0);
        const int64_t nr = some ? min(TN, a.N - n0) : 0, mr = some ? min((int64_t)TM, a.M - m0) : 0;
        const int sb = n0 / kBlock, sr = some ? min((TN + kBlock - 1) / kBlock, (a.N + kBlock - 1) / kBlock - sb) : 0;
        rw = descriptor(a.w + (int64_t)n0 * K, nr * K);
        rx = descriptor(a.x + m0 * K, mr * K);
        rsw = descriptor(a.ws + (int64_t)sb * a.kb, (int64_t)sr * a.kb * 4);
        rsx = descriptor(a.xs + m0 * a.kb, mr * a.kb * 4);
    };
    open();
    // load j of a block's LOADS
    auto fetch = [&](int j) {
        const int k = nb * kBlock;
        const uint32_t to = base + stage * STAGE;
        if (j < JN)
            load_lds16(rw, (k + (int)cw * 16 < K ? ow + k : kNowhere) + j * down, to + (wave + j * WAVES) * 1024);
        else if (j < JN + JM)
            load_lds16(rx, (k + (int)cx * 16 < K ? ox + k : kNowhere) + (j - JN) * down,
                       to + TN * kBlock + (wave + (j - JN) * WAVES) * 1024);
        else if (j == JN + JM)
            load_lds4(rsx, osx + nb * 4, to + XS + (wave % (TM / 64)) * 256);
        else
            load_lds4(rsw, osw + nb * 4, to + WS);
        if (j == LOADS - 1) {
            stage = stage == S - 1 ? 0 : stage + 1;
            ++nb;
        }
    };
    // to the next tile once the last block of one is loaded
    auto advance = [&]() {
        if (nb == a.kb) {
            nb = 0;
            next += step;
            open();
        }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        advance();
#pragma unroll
        for (int j = 0; j < LOADS; ++j) fetch(j);
    }
    // ---- fragments
    const uint32_t rowx = r * kBlock, roww = (8 * (r >> 2) + (r & 3)) * kBlock;
    const uint32_t fx = (r >> 1) & 7, fw = ((r >> 1) & 1) | (r >> 2) << 1;
    const uint32_t x0 = TN * kBlock + wm * FM * kBlock + rowx + (g ^ fx) * 16, x1 = x0 ^ 64;
    const uint32_t w0 = wn * FN * kBlock + roww + (g ^ fw) * 16, w1 = w0 ^ 64;
    auto pair = [&](const unsigned char* p, const unsigned char* q) {
        const i32x4 u = *reinterpret_cast<const i32x4*>(p), v = *reinterpret_cast<const i32x4*>(q);
        return i32x8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
    };
    auto x_frag = [&](const unsigned char* s, int t) { return pair(s + x0 + t * 16 * kBlock, s + x1 + t * 16 * kBlock); };
    // fragment i of w: rows 32 (i / 2) + 8 (r / 4) + 4 (i % 2) + r % 4, so that two of them give a lane eight outputs in a row
    auto w_frag = [&](const unsigned char* s, int i) {
        const int at = (32 * (i >> 1) + 4 * (i & 1)) * kBlock;
        return pair(s + w0 + at, s + w1 + at);
    };
    auto x_scale = [&](const unsigned char* s, int t) {
        return *reinterpret_cast<const float*>(s + XS + (wm * FM + 16 * t + r) * 4);
    };
    auto w_scale = [&](const unsigned char* s) {
        return *reinterpret_cast<const float*>(s + WS + (wn * FN / kBlock) * 4);
    };
    i32x8 xf[NT], wf[2];
    float sc[NT];
    wait_loads<LOADS*(S - 2)>();
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        xf[t] = x_frag(lds, t);
        sc[t] = x_scale(lds, t) * w_scale(lds);
    }
    wf[0] = w_frag(lds, 0);
    int cur = 0;
    for (unsigned id = id0; id < end; id += step) {
        f32x4 acc[NI][NT];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int b = 0; b < a.kb; ++b) {
            advance();
            const unsigned char* s = lds + cur * STAGE;
            cur = cur == S - 1 ? 0 : cur + 1;
            const unsigned char* sn = lds + cur * STAGE;
            f32x4 p[3];
            float ns[NT], nw = 0.f;
            // product n = i NT + t is added two products later, when it is there
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                if (i + 1 < NI) {
                    wf[(i + 1) & 1] = w_frag(s, i + 1);
                } else {
                    // Every fragment of this block is read.  The next block has arrived, its first
                    // fragments are read beside the last products, and loads go on into this stage.
                    wait_loads<LOADS*(S - 2)>();
                    __syncthreads();
                    wf[(i + 1) & 1] = w_frag(sn, 0);
                    nw = w_scale(sn);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int n = i * NT + t;
                    p[n % 3] = mma(wf[i & 1], xf[t]);
#pragma unroll
                    for (int j = n * LOADS / BEFORE; j < (n + 1) * LOADS / BEFORE && j < LOADS; ++j) fetch(j);
                    if (i == NI - 1) {
                        xf[t] = x_frag(sn, t);
                        ns[t] = x_scale(sn, t);
                    }
                    if (n >= 2) acc[(n - 2) / NT][(n - 2) % NT] += p[(n - 2) % 3] * sc[(n - 2) % NT];
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int n = NI * NT - 2; n < NI * NT; ++n) acc[n / NT][n % NT] += p[n % 3] * sc[n % NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t] = ns[t] * nw;
        }
        int n0;
        int64_t m0;
        tile_at(id, n0, m0);
        const int last = min(n0 + TN, a.N) - 1, part = n0 / a.part;
        const bool whole = part == last / a.part && a.part % 8 == 0;   // the tile lies in one of the outputs
        uint16_t* y = a.y + (int64_t)part * (a.M - 1) * a.part;        // of column n: y + m part + n
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t mt = m0 + wm * FM + 16 * t;
#pragma unroll
            for (int i = 0; i < NI; i += 4) {
                // Two runs of eight outputs, 32 columns apart, of token r.  Lanes r and r + 8 swap
                // one, so that a store covers whole lines: 64 columns of eight tokens.
                u32x4 own[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const f32x4 u = acc[i + 2 * e][t], v = acc[i + 2 * e + 1][t];
                    own[e] = u32x4{pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(v[0], v[1]),
                                   pack_bf16x2(v[2], v[3])};
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t give = r < 8 ? own[1][j] : own[0][j];
                    const uint32_t take = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xF, 0xF, false);
                    own[0][j] = r < 8 ? own[0][j] : take;
                    own[1][j] = r < 8 ? take : own[1][j];
                }
                // own[e]: token 8 e + r % 8, columns of half r / 8
                const int n = n0 + wn * FN + 16 * i + 32 * (r >> 3) + 8 * g;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t m = mt + 8 * e + (r & 7);
                    if (m >= a.M) continue;
                    if (whole) {
                        if (n <= last) __builtin_nontemporal_store(own[e], reinterpret_cast<u32x4*>(y + m * a.part + n));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (n + j <= last) {
                                const int q = (n + j) / a.part;
                                a.y[((int64_t)q * a.M + m) * a.part + (n + j - q * a.part)] =
                                    (uint16_t)(own[e][j / 2] >> (16 * (j & 1)));
                            }
                    }
                }
            }
        }
    }
    // the loads behind the last tile (of nothing, zeros) still write this workgroup's LDS
    wait_loads<0>();
}

// ---------------------------------------------------------------- few tokens
// Up to 16 T tokens a workgroup, 16 columns of y: the eight waves take every eighth
// block, operands straight from memory (each byte of w is read once for its tokens),
// and add their sums in order through LDS.  Bound by memory where w is large (one token,
// N = K = 8192: 13.5 us, 5.0 TB/s) and by a launch and two trips to memory where not (7
// tokens, N = 6144, K = 2048: 5.4 to 6.0 us; two trips' worth of blocks at once, 6.5
// beside 5.4).
constexpr int kFewWaves = 8;
template <int T>
__global__ __launch_bounds__(64 * kFewWaves) void matmul_few_kernel(const MatmulArgs a) {
    __shared__ f32x4 red[kFewWaves][T][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
    const int n0 = (int)(blockIdx.x % (unsigned)a.tiles_n) * 16;
    const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)a.tiles_n) * (16 * T);
    const int K = a.K;
    const int64_t mr = min((int64_t)16 * T, a.M - m0);
    const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * K, (int64_t)min(16, a.N - n0) * K);
    const rsrc_t rx = make_rsrc(a.x + m0 * K, mr * K), rs = make_rsrc(a.xs + m0 * a.kb, mr * a.kb * 4);
    const rsrc_t rws = make_rsrc(a.ws + (int64_t)(n0 / kBlock) * a.kb, (int64_t)a.kb * 4);
    // the lane's 32 places of a row's block from k on; zeros past the row's end and past
    // the last row (the loads stand without conditions, so all of them are under way at once)
    auto frag = [&](rsrc_t rsrc, uint32_t row, int k) {
        const u32x4 u = __builtin_amdgcn_raw_buffer_load_b128(rsrc, k < K ? row * K + k : kNowhere, 0, 0);
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, k + 16 < K ? row * K + k + 16 : kNowhere, 0, 0);
        return i32x8{(int)u[0], (int)u[1], (int)u[2], (int)u[3], (int)v[0], (int)v[1], (int)v[2], (int)v[3]};
    };
    f32x4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // several blocks at a time; past the last one operands and scales are zeros
    constexpr int U = 2;
    for (int b0 = wave; b0 < a.kb; b0 += U * kFewWaves) {
        i32x8 wf[U], xf[U][T];
        float ws[U], xs[U][T];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kFewWaves, k = b * kBlock + 32 * g;
            const uint32_t at = b < a.kb ? b * 4 : kNowhere;
            wf[u] = frag(rw, r, k);
            ws[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rws, at, 0, 0));
#pragma unroll
            for (int t = 0; t < T; ++t) {
                xf[u][t] = frag(rx, 16 * t + r, k);
                xs[u][t] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (16 * t + r) * a.kb * 4 + at, 0, 0));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < T; ++t) acc[t] += mma(wf[u], xf[u][t]) * (ws[u] * xs[u][t]);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) red[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave >= T) return;
    f32x4 s = red[0][wave][lane];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) s += red[i][wave][lane];
    const int64_t m = m0 + 16 * wave + r;
    const int n = n0 + 4 * g;
    if (m >= a.M) return;
    if (a.part % 4 == 0) {
        if (n >= a.N) return;
        const int q = n / a.part;
        *reinterpret_cast<u32x2*>(a.y + ((int64_t)q * a.M + m) * a.part + (n - q * a.part)) =
            u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < a.N) {
                const int q = (n + j) / a.part;
                a.y[((int64_t)q * a.M + m) * a.part + (n + j - q * a.part)] = f2bf(s[j]);
            }
    }
}

template <int TN, int TM, int WN, int WM, int S>
gdn_status run_tiles(MatmulArgs a, int cus, hipStream_t s) {
    a.tiles_n = (a.N + TN - 1) / TN;
    a.tiles_m = (int)((a.M + TM - 1) / TM);
    const int64_t tiles = (int64_t)a.tiles_n * a.tiles_m;
    hipLaunchKernelGGL((matmul_kernel<TN, TM, WN, WM, S>), dim3((unsigned)std::min<int64_t>(tiles, cus)),
                       dim3(64 * WN * WM), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
template <int T>
gdn_status run_few(MatmulArgs a, hipStream_t s) {
    a.tiles_n = (a.N + 15) / 16;
    const int64_t tiles = a.tiles_n * ((a.M + 16 * T - 1) / (16 * T));
    hipLaunchKernelGGL(matmul_few_kernel<T>, dim3((unsigned)tiles), dim3(64 * kFewWaves), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" gdn_status gdn_matmul_fp8(const gdn_matmul_desc* d, const void* x, const float* x_scale, const void* w,
                                     const float* w_scale, void* y, void* stream) {
    if (!d || d->M < 0 || d->N < 1 || d->K < 1 || d->parts < 1 || d->N % d->parts) return GDN_ERR_INVALID_ARG;
    if (d->K % 16 || d->N > (1 << 20) || d->K > (1 << 20) || d->M > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    if (d->M == 0) return GDN_OK;
    if (!x || !x_scale || !w || !w_scale || !y) return GDN_ERR_INVALID_ARG;
    if ((d->M / 64 + 1) * (d->N / 128 + 1) > INT32_MAX) return GDN_ERR_UNSUPPORTED;   // tiles are counted in 32 bits
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4))
        return GDN_ERR_ALIGNMENT;
    const int kb = (d->K + kBlock - 1) / kBlock, nb = (d->N + kBlock - 1) / kBlock;
    const Range out = rng(y, (size_t)d->M * d->N * 2);
    const Range ins[] = {rng(x, (size_t)d->M * d->K), rng(x_scale, (size_t)d->M * kb * 4),
                         rng(w, (size_t)d->N * d->K), rng(w_scale, (size_t)nb * kb * 4)};
    for (const Range& r : ins)
        if (overlap(out, r)) return GDN_ERR_ALIAS;
    int cus;
    const gdn_status st = check_device(&cus);
    if (st != GDN_OK) return st;
    MatmulArgs a = {};
    a.x = static_cast<const uint8_t*>(x), a.w = static_cast<const uint8_t*>(w), a.xs = x_scale, a.ws = w_scale;
    a.y = static_cast<uint16_t*>(y);
    a.M = d->M, a.N = d->N, a.K = d->K, a.kb = kb, a.part = d->N / d->parts;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    switch (choose(a.M, a.N, cus)) {
        case kFew16: return run_few<1>(a, s);
        case kFew32: return run_few<2>(a, s);
        case k128x64: return run_tiles<128, 64, 2, 2, 3>(a, 2 * cus, s);
        case k128x128: return run_tiles<128, 128, 2, 4, 4>(a, cus, s);
        case k256x128: return run_tiles<256, 128, 2, 4, 3>(a, cus, s);
        default: return run_tiles<256, 256, 2, 4, 2>(a, cus, s);
    }
}
