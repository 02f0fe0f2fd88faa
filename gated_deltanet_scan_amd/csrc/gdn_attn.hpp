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

struct AttnArgs {
    const void *q, *k, *v, *o, *d_o;
    void *out, *dq, *dk, *dv;            // out: o of the forward call
    float* lse;                          // [total_q][Hq], natural logarithm (forward: may be NULL)
    float* delta;                        // [total_q][Hq] <d_o, o> (backward)
    float *part_o, *part_lse;            // splits > 1: [splits][total_q Hq][D], [splits][total_q Hq]
    const int32_t *cu_q, *cu_k, *k_len;
    int64_t total_q, total_k, ldq, ldk, ldv, k_room;
    int n_seq, Hq, Hk, G, D;
    int max_q, max_k;
    int tiles;                           // row (or key) tiles of the longest sequence
    int splits;
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
// Keys [lo, hi) of split sp of n, of the first `upto` keys, in whole tiles.
__device__ __forceinline__ void split_range(int upto, int tile, int n, int sp, int& lo, int& hi) {
    const int t = (upto + tile - 1) / tile, per = (t + n - 1) / n;
    lo = min(sp * per * tile, upto);
    hi = min(lo + per * tile, upto);
}

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_f(float x) { return __builtin_amdgcn_logf(x); }

// Kernels in bf16 matrix instructions (gdn_attn_bf16.hip), D in {32, 64, 128}.
gdn_status attn_fwd_bf16(const AttnArgs& a, hipStream_t s);
gdn_status attn_bwd_bf16(const AttnArgs& a, hipStream_t s);
// Row tile of the forward kernel that these arguments select.
int attn_fwd_bf16_rows(int max_q, int G, int D);

}  // namespace gdnattn
