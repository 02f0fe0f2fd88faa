// Softmax attention: what its kernels share (arguments, the geometry of packed
// sequences and of the mask, and the split of a long key axis).
//
// For every sequence and key/value head the G = Hq / Hk query heads that share
// it are packed into one axis of rows, row r = query r / G of head G hk + r % G:
// a key tile is then read once for all of them, and a single query still fills
// G rows of a matrix tile.  The mask is a number of visible keys per query,
//     n(i) = lk,   or causal:  min(lk, (floor(p / block) + 1) block),  p = i + lk - lq  (0 where p < 0)
// which does not fall with i: whole key tiles past a row tile's last n are
// skipped and tiles below its first n need no mask.
#pragma once

#include "gdn_ops.hpp"

namespace gdnattn {

using namespace gdnops;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The widest token stride of sequences of several tokens, so that offsets
// within a tile fit 32 bits.  Single tokens may lie further apart: they are
// addressed in 64 bits as the first of their sequence, and the places of a tile
// past them need no address but one past its end, which this stride gives too.
constexpr int64_t kMaxStride = 1 << 20;
__device__ __forceinline__ uint32_t tile_stride(int64_t ld) { return (uint32_t)min(ld, kMaxStride); }

struct AttnArgs {
    const void *q, *k, *v, *o, *d_o;
    void *out, *dq, *dk, *dv;            // out: o of the forward call
    float* lse;                          // [total_q][Hq], natural logarithm (forward: may be NULL)
    float* delta;                        // [total_q][Hq] <d_o, o> (backward)
    float *part_o, *part_lse;            // splits > 1: [splits][total_q Hq][D], [splits][total_q Hq]
    float *part_k, *part_v;              // k_splits > 1: [k_splits][total_k Hk][D] each (backward)
    const int32_t *cu_q, *cu_k, *k_len;
    int64_t total_q, total_k, ldq, ldk, ldv, k_room;
    int n_seq, Hq, Hk, G, D;
    int max_q, max_k;
    int tiles;                           // row (or key) tiles of the longest sequence
    int splits, k_splits;                // of the key axis (forward), of the row axis (dk, dv)
    int chunk;                           // keys of a split (the longest sequence's fill them all)
    int join_rows;                       // rows of a workgroup of the join
    int causal, block;
    float scale;
};

// Rows [start, start + len) of sequence s.  Whatever the device arrays hold,
// the range lies within the tensor and is no longer than `most`.
__device__ __forceinline__ void seq_range(const int32_t* cu, int s, int64_t total, int most, int64_t& start, int& len) {
    if (cu) {
        const int64_t a = min(max((int64_t)cu[s], (int64_t)0), total);
        const int64_t b = min(max((int64_t)cu[s + 1], a), total);
        start = a;
        len = (int)min(b - a, (int64_t)most);
    } else {
        start = (int64_t)s * most;
        len = most;
    }
}
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
struct Seq {
    int64_t q0, k0, ko;                  // first query, first key, and its place in dk and dv
    int lq, lk;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int s) {
    Seq z;
    seq_range(a.cu_q, s, a.total_q, a.max_q, z.q0, z.lq);
    seq_range(a.cu_k, s, a.total_k, a.max_k, z.ko, z.lk);
    z.k0 = a.cu_k ? z.ko : (int64_t)s * a.k_room;
    if (a.k_len) z.lk = min(z.lk, max(a.k_len[s], 0));
    // one sequence a workgroup: scalar registers
    z.q0 = uniform(z.q0), z.k0 = uniform(z.k0), z.ko = uniform(z.ko);
    z.lq = __builtin_amdgcn_readfirstlane(z.lq), z.lk = __builtin_amdgcn_readfirstlane(z.lk);
    return z;
}
// Keys that query i sees.
__device__ __forceinline__ int visible(const AttnArgs& a, const Seq& z, int i) {
    if (!a.causal) return z.lk;
    const int p = i + (z.lk - z.lq);
    if (p < 0) return 0;
    if (a.block == 1) return p + 1 < z.lk ? p + 1 : z.lk;
    return (int)min((int64_t)z.lk, ((int64_t)(p / a.block) + 1) * a.block);
}
// The first query that sees key j (causal: the start of j's block, as a query).
__device__ __forceinline__ int first_query(const AttnArgs& a, const Seq& z, int j) {
    if (!a.causal) return 0;
    return max(0, j / a.block * a.block - (z.lk - z.lq));
}
// Part sp of n of [0, upto), in whole tiles.
__device__ __forceinline__ void split_range(int upto, int tile, int n, int sp, int& lo, int& hi) {
    const int t = (upto + tile - 1) / tile, per = (t + n - 1) / n;
    lo = min(sp * per * tile, upto);
    hi = min(lo + per * tile, upto);
}

// What a workgroup computes: one tile of rows (queries) or of keys of one
// sequence and key head, one split of it.  s < 0: nothing.
struct Place {
    int s, hk, split, tile;
};
__device__ __forceinline__ int wave_sum_i(int x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    return __builtin_amdgcn_readfirstlane(x);
}
// Tiles of `size` of sequence s, along its packed query rows or its keys.
template <bool KEYS>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int s, int size) {
    int64_t at;
    int len;
    if (KEYS)
        seq_range(a.cu_k, s, a.total_k, a.max_k, at, len);
    else
        seq_range(a.cu_q, s, a.total_q, a.max_q, at, len);
    return KEYS ? (len + size - 1) / size : (len * a.G + size - 1) / size;
}
// The key head runs fastest: workgroups go round the eight XCDs in turn, so
// with eight key heads or a multiple of eight each XCD's L2 holds the keys of
// its own heads only.  Then the splits, then the tiles: level by level across
// the sequences, the longest sequences' last tiles first (under a causal mask
// tile L of any sequence costs about L, so long work starts early), and only
// tiles that exist.  (A grid over (level, sequence) with its empty places left
// in put all the long sequences of one packed batch on four of the XCDs.)
// Key tiles run the other way, since the first keys are seen by the most rows.
template <bool KEYS>
__device__ __forceinline__ Place find_place(const AttnArgs& a, int size) {
    unsigned b = blockIdx.x;
    Place p;
    p.hk = (int)(b % (unsigned)a.Hk);
    b /= (unsigned)a.Hk;
    const unsigned splits = KEYS ? a.k_splits : a.splits;
    p.split = (int)(b % splits);
    const int w = (int)(b / splits);
    const int32_t* cu = KEYS ? a.cu_k : a.cu_q;
    int count, level;                                     // tiles of the sequence, and ours
    if (!cu || a.tiles == 1) {
        p.s = w % a.n_seq;
        count = a.tiles;
        level = a.tiles - 1 - w / a.n_seq;
    } else if (a.n_seq <= 64) {
        const int lane = threadIdx.x & 63;
        const int t = lane < a.n_seq ? tiles_of<KEYS>(a, lane, size) : 0;
        // the highest level with more than w tiles at it or above
        int lo = 0, hi = a.tiles, above = 0;              // count(hi) <= w, `above` of it
        if (wave_sum_i(t) <= w) {
            p.s = -1;
            return p;
        }
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            const int n = wave_sum_i(max(0, t - mid));
            if (n > w) {
                lo = mid;
            } else {
                hi = mid;
                above = n;
            }
        }
        level = lo;
        const uint64_t at = __ballot(t > level);
        const int before = __popcll(at & ((1ull << lane) - 1));
        p.s = __builtin_amdgcn_readfirstlane(
            __ffsll((unsigned long long)__ballot(t > level && before == w - above)) - 1);
        count = __builtin_amdgcn_readlane(t, p.s);
    } else {
        // Many sequences: in their order, which by itself spreads the work.
        // Sequence s has the places from floor(rows before it / size) + s on, which
        // are never fewer than its tiles, so a search of 64 places at a time finds
        // it without adding up the tiles of all before it (8192 sequences of 1 to
        // 299 tokens, forward and backward: 4670 us against 13900 with the sum).
        const int lane = threadIdx.x & 63;
        auto start = [&](int s) {
            const uint64_t at = (uint64_t)min(max((int64_t)cu[s], (int64_t)0), KEYS ? a.total_k : a.total_q);
            return (int64_t)((KEYS ? at : at * (unsigned)a.G) / (unsigned)size) + s;
        };
        int lo = 0, hi = a.n_seq;                             // start(lo) <= w < start(hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) / 64, s = lo + step * lane;
            const uint64_t at = __ballot(s < hi && (lane == 0 || start(s) <= w));
            lo += step * (63 - __clzll((long long)at));
            hi = min(hi, lo + step);
        }
        p.s = __builtin_amdgcn_readfirstlane(lo);
        count = tiles_of<KEYS>(a, p.s, size);
        level = count - 1 - (int)(w - start(p.s));
        if (level < 0 || level >= count) p.s = -1;
        if (p.s < 0) return p;
    }
    p.s = __builtin_amdgcn_readfirstlane(p.s);
    p.tile = __builtin_amdgcn_readfirstlane(KEYS ? count - 1 - level : level);
    return p;
}
// Workgroups of one split and key head that find_place hands out: no more than
// every sequence's share of the tensor, rounded up (all of them where the places
// are found by search).
inline int64_t places(int64_t rows, int64_t most, int n_seq, int size, bool packed, int* tiles) {
    *tiles = (int)((most + size - 1) / size);
    const int64_t all = (int64_t)*tiles * n_seq;
    if (!packed || *tiles <= 1) return all;
    const int64_t share = rows / size + n_seq;
    return n_seq > 64 || share < all ? share : all;
}

// One launch over tiles of rows or keys; a launch takes fewer than 2^32 work items.
struct Grid {
    unsigned groups;
    int tiles;                           // of the longest sequence
};
inline bool grid_of(int64_t groups, int threads, unsigned* g) {
    if (groups > (int64_t)(UINT32_MAX / (unsigned)threads)) return false;
    *g = (unsigned)groups;
    return true;
}

// Hidden places and values that are not finite.  A matrix product multiplies a
// hidden place by an exact 0, which for an infinity or a NaN there gives NaN in
// rows that must not see it.  Nothing in the loops guards against it: where a
// mask is in force, a wave whose sums are not all finite at its end forms them
// again element by element, over the places that each row sees alone; so does
// the bf16 dk/dv kernel, mask or not, for an infinite key whose last row tile
// ends in zeros.
// Rows that do see such a value come out as the sums give it.  Costs one
// product with 0 per result (bf16 training cases 0.2% slower at most, the
// smallest fp32 one 72.3 us against 71.2).
template <int N, typename V>
__device__ __forceinline__ bool finite(const V (&x)[N], float t = 0.f) {
#pragma unroll
    for (int e = 0; e < N; ++e)
#pragma unroll
        for (int i = 0; i < (int)(sizeof(V) / 4); ++i) t = __builtin_fmaf(x[e][i], 0.f, t);
    return !__any(t != 0.f);                                  // 0, or NaN
}

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_f(float x) { return __builtin_amdgcn_logf(x); }

// Kernels in bf16 matrix instructions (gdn_attn_bf16.hip), D in {32, 64, 128}.
// `rows` is attn_fwd_bf16_rows(): two threads a row; the backward kernels have
// tiles of kBwdTile rows or keys.
constexpr int kBwdTile = 128;
gdn_status attn_fwd_bf16(const AttnArgs& a, int rows, Grid g, hipStream_t s);
gdn_status attn_bwd_bf16(const AttnArgs& a, Grid dq, Grid dkv, hipStream_t s);
// Row tile of the forward kernel that these arguments select.
int attn_fwd_bf16_rows(int max_q, int G, int D);

}  // namespace gdnattn
