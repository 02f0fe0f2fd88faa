// Key/value caches in MXFP8 and MXFP4: the C ABI of gdn_cache_write and
// gdn_cache_read (declared in include/gdn.h).
//
// For a block of 32 features with largest magnitude m, e = floor(log2 m) less the
// format's largest exponent, scale byte e + 127 (0 at least; 127 for m = 0; 255
// where a value is not finite: the block reads as NaN), and codes are x / 2^e to
// the nearest representable value, ties to the even code, saturated.
// m's exponent field gives e, and x / 2^e is exact, so the codes are the format's
// to the bit.
//
// Bound by memory.  Four lanes hold a block, eight features each, so a block's
// maximum is two exchanges within a quad, and a lane's codes are one store.  16 heads of
// 128, bf16, both caches: 106480 tokens are written in 223 to 229 us (MXFP4) and 265 to 271
// (MXFP8) and read in 221 to 226 and 265 to 266, 4.8 to 5.0 TB/s; 880 tokens in 3.6 to 4.3;
// eight in 2.4 to 3.0, a launch.  From fp32 412 and 446 (4.8 and 4.9 TB/s), to fp32 563
// and 610 (3.5 and 3.6).
#include "gdn_attn.hpp"
#include "gdn_mx.hpp"

#include <algorithm>

namespace {

using namespace gdnattn;
using namespace gdnmx;

constexpr int kThreads = 256;

struct CacheArgs {
    const void *k, *v;               // write: the new tokens
    void *k_out, *v_out;             // read
    uint8_t *kc, *ks, *vc, *vs;
    const int32_t *cu_new, *cu_k, *k_len;
    int64_t total_new, total_k, ldk, ldv, k_room;
    int n_seq, H, D, max_new, max_k;
    int groups;                      // workgroups of a sequence
};

// A sequence's slot of the cache: first token, tokens, and those in use.
struct Slot {
    int64_t at, out;                 // in the cache, and in the tensors that it is read to
    int size, used;
    int64_t want;                    // keys in use as the caller has it
};
__device__ __forceinline__ Slot slot_of(const CacheArgs& a, int s) {
    Slot z;
    seq_range(a.cu_k, s, a.total_k, a.max_k, z.out, z.size);
    z.at = a.cu_k ? z.out : (int64_t)s * a.k_room;
    z.want = a.k_len ? a.k_len[s] : z.size;
    z.used = a.k_len ? min(z.size, max(a.k_len[s], 0)) : z.size;
    return z;
}

// Eight features of a block (four lanes) to codes and the block's scale.
template <typename F, typename T>
__device__ __forceinline__ void encode(const Vec8<T>& x, uint8_t* codes, uint8_t* scale, bool first) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x.get(j)) & 0x7fffffffu);   // NaN above infinity
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, false));
    const int ex = (int)(top >> 23);
    const int s = ex == 255 ? 255 : top == 0 ? 127 : max(ex - F::kTop, 0);
    const float inv = __uint_as_float((uint32_t)(254 - s) << 23);      // 2^(127 - s); s is 254 - kTop at most
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = ex == 255 ? 0.f : x.get(j) * inv;
    *reinterpret_cast<typename F::Raw8*>(codes) = F::narrow(y);
    if (first) *scale = (uint8_t)s;
}

template <typename F, typename T>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(const CacheArgs a) {
    const int s = (int)(blockIdx.x / (unsigned)a.groups), w = (int)(blockIdx.x % (unsigned)a.groups);
    int64_t n0;
    int n;
    seq_range(a.cu_new, s, a.total_new, a.max_new, n0, n);
    const Slot z = slot_of(a, s);
    const int per = a.H * (a.D / 8);                     // chunks of eight features a token
    const int64_t all = (int64_t)n * per;
    for (int64_t i = (int64_t)w * kThreads + threadIdx.x; i < all; i += (int64_t)a.groups * kThreads) {
        const int64_t t = i / per;
        const int c = (int)(i - t * per) * 8;            // feature within the token's row
        const int64_t p = z.want - n + t;                // the token's place in its slot
        if (p < 0 || p >= z.size) continue;              // for the whole row, so for whole blocks
        Vec8<T> k, v;
        k.load(static_cast<const T*>(a.k) + (n0 + t) * a.ldk + c);
        v.load(static_cast<const T*>(a.v) + (n0 + t) * a.ldv + c);
        const int64_t at = (z.at + p) * a.H * a.D + c;
        encode<F, T>(k, a.kc + at / F::kPerByte, a.ks + at / kBlock, (c & 31) == 0);
        encode<F, T>(v, a.vc + at / F::kPerByte, a.vs + at / kBlock, (c & 31) == 0);
    }
}

template <typename F, typename T>
__device__ __forceinline__ void decode(const uint8_t* codes, uint8_t scale, T* out) {
    const typename F::Raw8 r = *reinterpret_cast<const typename F::Raw8*>(codes);
    Vec8<T> y;
    if constexpr (sizeof(T) == 2) {
        y.v = F::widen(r, scale_of(scale));
    } else {
        float f[8];
        F::widen(r, scale_of(scale), f);
        y.set(f);
    }
    y.store(out);
}

template <typename F, typename T>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(const CacheArgs a) {
    const int s = (int)(blockIdx.x / (unsigned)a.groups), w = (int)(blockIdx.x % (unsigned)a.groups);
    const Slot z = slot_of(a, s);
    const int64_t row = (int64_t)a.H * a.D, all = z.used * (row / 8);
    for (int64_t i = (int64_t)w * kThreads + threadIdx.x; i < all; i += (int64_t)a.groups * kThreads) {
        const int64_t at = z.at * row + i * 8, to = z.out * row + i * 8;
        decode<F, T>(a.kc + at / F::kPerByte, a.ks[at / kBlock], static_cast<T*>(a.k_out) + to);
        decode<F, T>(a.vc + at / F::kPerByte, a.vs[at / kBlock], static_cast<T*>(a.v_out) + to);
    }
}

// ---------------------------------------------------------------- launch
gdn_status check(const gdn_cache_desc* d) {
    if (!d || d->n_seq < 0 || d->H < 1 || d->D < 1 || d->total_new < 0 || d->total_k < 0 || d->max_new < 0 ||
        d->max_k < 0 || d->k_stride < 0 || d->v_stride < 0 || d->k_room < 0)
        return GDN_ERR_INVALID_ARG;
    if (d->io_dtype != GDN_BF16 && d->io_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (d->cache_dtype != GDN_FP8_E4M3 && d->cache_dtype != GDN_FP4_E2M1) return GDN_ERR_INVALID_ARG;
    if (d->k_room && d->k_room < d->max_k) return GDN_ERR_INVALID_ARG;
    const int64_t row = (int64_t)d->H * d->D;
    if ((d->k_stride && d->k_stride < row) || (d->v_stride && d->v_stride < row)) return GDN_ERR_INVALID_ARG;
    if (d->D != 32 && d->D != 64 && d->D != 128) return GDN_ERR_UNSUPPORTED;
    if (row > (1 << 20) || d->total_new > INT32_MAX || d->total_k > INT32_MAX || d->k_room > INT32_MAX ||
        d->k_stride > ((int64_t)1 << 31) || d->v_stride > ((int64_t)1 << 31))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
CacheArgs fill(const gdn_cache_desc* d) {
    CacheArgs a = {};
    a.total_new = d->total_new, a.total_k = d->total_k;
    const int64_t row = (int64_t)d->H * d->D;
    a.ldk = d->k_stride ? d->k_stride : row, a.ldv = d->v_stride ? d->v_stride : row;
    a.k_room = d->k_room ? d->k_room : d->max_k;
    a.n_seq = d->n_seq, a.H = d->H, a.D = d->D;
    a.max_new = (int)std::min<int64_t>(d->max_new, d->total_new);
    a.max_k = (int)std::min<int64_t>(d->max_k, d->total_k);
    return a;
}
// Tokens from the first slot's first to the last one's last.
int64_t cache_rows(const gdn_cache_desc* d, bool packed) {
    if (packed || !d->k_room || d->n_seq < 1) return d->total_k;
    return (d->n_seq - 1) * d->k_room + d->max_k;
}
size_t span(int64_t rows, int64_t ld, int64_t w, size_t e) { return rows > 0 ? ((size_t)(rows - 1) * ld + w) * e : 0; }

// Workgroups of a sequence: its longest possible walk, or fewer that go round.  The
// sequences share 2^18, beyond what the card holds at once, since packed ones are shorter
// than the longest may be and a workgroup with nothing to do costs its start.
bool size_grid(CacheArgs& a, int64_t tokens, unsigned* grid) {
    const int64_t one = (tokens * a.H * (a.D / 8) + kThreads - 1) / kThreads;
    a.groups = (int)std::max<int64_t>(1, std::min<int64_t>({one, 4096, (1 << 18) / a.n_seq}));
    const int64_t g = (int64_t)a.groups * a.n_seq;
    if (g > (int64_t)(UINT32_MAX / kThreads)) return false;
    *grid = (unsigned)g;
    return true;
}

template <typename F, typename T>
gdn_status run_write(const CacheArgs& a, unsigned grid, hipStream_t s) {
    hipLaunchKernelGGL((cache_write_kernel<F, T>), dim3(grid), dim3(kThreads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
template <typename F, typename T>
gdn_status run_read(const CacheArgs& a, unsigned grid, hipStream_t s) {
    hipLaunchKernelGGL((cache_read_kernel<F, T>), dim3(grid), dim3(kThreads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
#define GDN_BY_FORMAT(FN, ...)                                                                      \
    (d->cache_dtype == GDN_FP4_E2M1                                                                 \
         ? (d->io_dtype == GDN_F32 ? FN<Fp4, float>(__VA_ARGS__) : FN<Fp4, uint16_t>(__VA_ARGS__))  \
         : (d->io_dtype == GDN_F32 ? FN<Fp8, float>(__VA_ARGS__) : FN<Fp8, uint16_t>(__VA_ARGS__)))

}  // namespace

extern "C" {

gdn_status gdn_cache_write(const gdn_cache_desc* d, const void* k, const void* v, const int32_t* cu_new,
                           const int32_t* cu_k, const int32_t* k_len, void* k_codes, uint8_t* k_scale, void* v_codes,
                           uint8_t* v_scale, void* stream) {
    gdn_status st = check(d);
    if (st != GDN_OK) return st;
    if (!cu_new && (int64_t)d->n_seq * d->max_new != d->total_new) return GDN_ERR_INVALID_ARG;
    if (!cu_k && (int64_t)d->n_seq * d->max_k != d->total_k) return GDN_ERR_INVALID_ARG;
    if (d->n_seq == 0 || d->total_new == 0 || d->max_new == 0 || d->total_k == 0 || d->max_k == 0) return GDN_OK;
    if (!k || !v || !k_codes || !k_scale || !v_codes || !v_scale) return GDN_ERR_INVALID_ARG;
    CacheArgs a = fill(d);
    unsigned grid;
    if (!size_grid(a, a.max_new, &grid)) return GDN_ERR_UNSUPPORTED;
    const size_t e = d->io_dtype == GDN_F32 ? 4 : 2;
    for (const void* p : {k, v, (const void*)k_codes, (const void*)v_codes})
        if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
    if (!aligned(cu_new, 4) || !aligned(cu_k, 4) || !aligned(k_len, 4) || a.ldk * e % 16 || a.ldv * e % 16)
        return GDN_ERR_ALIGNMENT;
    const int64_t row = (int64_t)d->H * d->D;
    const size_t n = (size_t)cache_rows(d, cu_k) * row, cb = d->cache_dtype == GDN_FP4_E2M1 ? n / 2 : n, sb = n / kBlock;
    const Range ins[] = {rng(k, span(d->total_new, a.ldk, row, e)), rng(v, span(d->total_new, a.ldv, row, e)),
                         rng(cu_new, ((size_t)d->n_seq + 1) * 4), rng(cu_k, ((size_t)d->n_seq + 1) * 4),
                         rng(k_len, (size_t)d->n_seq * 4)};
    const Range outs[] = {rng(k_codes, cb), rng(k_scale, sb), rng(v_codes, cb), rng(v_scale, sb)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return GDN_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_ALIAS;
    }
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    a.k = k, a.v = v, a.cu_new = cu_new, a.cu_k = cu_k, a.k_len = k_len;
    a.kc = static_cast<uint8_t*>(k_codes), a.ks = k_scale, a.vc = static_cast<uint8_t*>(v_codes), a.vs = v_scale;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return GDN_BY_FORMAT(run_write, a, grid, s);
}

gdn_status gdn_cache_read(const gdn_cache_desc* d, const void* k_codes, const uint8_t* k_scale, const void* v_codes,
                          const uint8_t* v_scale, const int32_t* cu_k, const int32_t* k_len, void* k, void* v,
                          void* stream) {
    gdn_status st = check(d);
    if (st != GDN_OK) return st;
    if (!cu_k && (int64_t)d->n_seq * d->max_k != d->total_k) return GDN_ERR_INVALID_ARG;
    if (d->n_seq == 0 || d->total_k == 0 || d->max_k == 0) return GDN_OK;
    if (!k || !v || !k_codes || !k_scale || !v_codes || !v_scale) return GDN_ERR_INVALID_ARG;
    CacheArgs a = fill(d);
    unsigned grid;
    if (!size_grid(a, a.max_k, &grid)) return GDN_ERR_UNSUPPORTED;
    const size_t e = d->io_dtype == GDN_F32 ? 4 : 2;
    for (const void* p : {(const void*)k, (const void*)v, k_codes, v_codes})
        if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
    if (!aligned(cu_k, 4) || !aligned(k_len, 4)) return GDN_ERR_ALIGNMENT;
    const int64_t row = (int64_t)d->H * d->D;
    const size_t n = (size_t)cache_rows(d, cu_k) * row, cb = d->cache_dtype == GDN_FP4_E2M1 ? n / 2 : n, sb = n / kBlock;
    const Range ins[] = {rng(k_codes, cb), rng(k_scale, sb), rng(v_codes, cb), rng(v_scale, sb),
                         rng(cu_k, ((size_t)d->n_seq + 1) * 4), rng(k_len, (size_t)d->n_seq * 4)};
    const size_t ob = (size_t)d->total_k * row * e;
    const Range outs[] = {rng(k, ob), rng(v, ob)};
    for (const Range& r : ins)
        if (overlap(outs[0], r) || overlap(outs[1], r)) return GDN_ERR_ALIAS;
    if (overlap(outs[0], outs[1])) return GDN_ERR_ALIAS;
    int cus;
    if ((st = check_device(&cus)) != GDN_OK) return st;
    a.cu_k = cu_k, a.k_len = k_len, a.k_out = k, a.v_out = v;
    a.kc = static_cast<uint8_t*>(const_cast<void*>(k_codes)), a.ks = const_cast<uint8_t*>(k_scale);
    a.vc = static_cast<uint8_t*>(const_cast<void*>(v_codes)), a.vs = const_cast<uint8_t*>(v_scale);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return GDN_BY_FORMAT(run_read, a, grid, s);
}

}  // extern "C"
