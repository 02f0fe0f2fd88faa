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
#include "gdn_ops.hpp"

#include <algorithm>

namespace {

using namespace gdnops;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;

struct MatmulArgs {
    const uint8_t *x, *w;
    const float *xs, *ws;
    uint16_t* y;
    int64_t M;
    int N, K, kb, part;              // part: columns of one of the outputs
};

__device__ __forceinline__ f32x4 mma(i32x8 a, i32x8 b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                            0x7f7f7f7f);
}
// The lane's 32 places of a row's block from k on; zeros past the row's end (K is
// a multiple of 16).
__device__ __forceinline__ i32x8 frag(const uint8_t* row, int k, int K) {
    i32x4 a = {0, 0, 0, 0}, b = a;
    if (k < K) a = *reinterpret_cast<const i32x4*>(row + k);
    if (k + 16 < K) b = *reinterpret_cast<const i32x4*>(row + k + 16);
    return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Output column n of token m.
__device__ __forceinline__ uint16_t* place(const MatmulArgs& a, int64_t m, int n) {
    const int p = n / a.part;
    return a.y + ((int64_t)p * a.M + m) * a.part + (n - p * a.part);
}

// Four waves, 64 columns of y (16 a wave) of 64 tokens; operands straight from
// memory.
__global__ __launch_bounds__(256) void matmul_kernel(const MatmulArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
    const int tiles = (a.N + 63) / 64;
    const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)tiles) * 64;
    const int n0 = (int)(blockIdx.x % (unsigned)tiles) * 64 + 16 * wave;
    if (n0 >= a.N) return;
    const uint8_t* w = a.w + (int64_t)min(n0 + r, a.N - 1) * a.K;
    f32x4 acc[4];
    for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < a.kb; ++b) {
        const int k = b * kBlock + 32 * g;
        const i32x8 wf = frag(w, k, a.K);
        const float ws = a.ws[(int64_t)(n0 / kBlock) * a.kb + b];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t m = min(m0 + 16 * t + r, a.M - 1);
            const f32x4 p = mma(wf, frag(a.x + m * a.K, k, a.K));
            acc[t] += p * (ws * a.xs[m * a.kb + b]);
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t m = m0 + 16 * t + r;
        if (m >= a.M) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 4 * g + i;
            if (n < a.N) *place(a, m, n) = f2bf(acc[t][i]);
        }
    }
}

}  // namespace

extern "C" gdn_status gdn_matmul_fp8(const gdn_matmul_desc* d, const void* x, const float* x_scale, const void* w,
                                     const float* w_scale, void* y, void* stream) {
    if (!d || d->M < 0 || d->N < 1 || d->K < 1 || d->parts < 1 || d->N % d->parts) return GDN_ERR_INVALID_ARG;
    if (d->K % 16 || d->N > (1 << 20) || d->K > (1 << 20) || d->M > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    if (d->M == 0) return GDN_OK;
    if (!x || !x_scale || !w || !w_scale || !y) return GDN_ERR_INVALID_ARG;
    const int64_t tiles = ((int64_t)d->N + 63) / 64 * ((d->M + 63) / 64);
    if (tiles > UINT32_MAX / 256) return GDN_ERR_UNSUPPORTED;
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
    hipLaunchKernelGGL(matmul_kernel, dim3((unsigned)tiles), dim3(256), 0, reinterpret_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
