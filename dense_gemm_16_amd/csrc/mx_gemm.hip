// mx_gemm.hip -- the product of two MXFP4 matrices (format: mx.hip) on the
// gfx950 matrix cores, FP32 sums.
//
// C = alpha A B + beta C with A (M x K) and B given transposed (N x K), both
// quantised along k.  v_mfma_scale_f32_16x16x128_f8f6f4 with both formats FP4
// takes, in lane (r + 16 g), the 32 elements k = 32 g .. 32 g + 31 of row r of a
// 16-row block: 16 bytes, one MXFP4 block, and that block's scale byte.  Every
// product of two elements is exact and the scales are powers of two, so the
// only roundings are those of the FP32 sums.
//
// k is counted in 16-byte chunks (blocks) below.  Rows past M or N are clamped
// to the last one (their outputs are never stored); chunks past K read as zero
// elements with scale byte 0, so whatever lies in a scale row's padding is
// not used.
#include "mfma_gemm.hpp"

namespace migemm {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

// c += A B for one 16 x 16 x 128 block: 16 bytes of elements and one scale byte
// per lane and operand (the low byte of sa and sb).
__device__ __forceinline__ void mfma_mx(f32x4& c, u32x4 a, u32x4 b, uint32_t sa, uint32_t sb) {
    const i32x4 ai = __builtin_bit_cast(i32x4, a), bi = __builtin_bit_cast(i32x4, b);
    const i32x8 a8 = __builtin_shufflevector(ai, ai, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 b8 = __builtin_shufflevector(bi, bi, 0, 1, 2, 3, -1, -1, -1, -1);
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, static_cast<int>(sa),
                                                         0, static_cast<int>(sb));
}

// The plain kernel: fragments straight from global memory.  Four waves, each
// TM x TN blocks of 16 x 16.
template <int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * kWave) void mx_plain_kernel(MxArgs p) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int r = lane % 16, g = lane / 16;
    const int64_t tiles_n = ceil_div(p.N, 16 * TN * WN);
    const int64_t m0 = (blockIdx.x / tiles_n * WM + wave / WN) * (16 * TM);
    const int64_t n0 = (blockIdx.x % tiles_n * WN + wave % WN) * (16 * TN);
    const int64_t chunks = p.K / 32;
    f32x4 acc[TM][TN] = {};
    for (int64_t c0 = 0; c0 < chunks; c0 += 4) {
        const int64_t c = c0 + g;
        u32x4 a[TM], b[TN];
        uint32_t sa[TM], sb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t row = min(m0 + 16 * i + r, p.M - 1);
            a[i] = u32x4{0u, 0u, 0u, 0u};
            sa[i] = 0;
            if (c < chunks) {
                a[i] = *reinterpret_cast<const u32x4*>(p.A + row * p.lda + 16 * c);
                sa[i] = p.sa[row * p.ldsa + c];
            }
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t row = min(n0 + 16 * j + r, p.N - 1);
            b[j] = u32x4{0u, 0u, 0u, 0u};
            sb[j] = 0;
            if (c < chunks) {
                b[j] = *reinterpret_cast<const u32x4*>(p.B + row * p.ldb + 16 * c);
                sb[j] = p.sb[row * p.ldsb + c];
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) mfma_mx(acc[i][j], a[i], b[j], sa[i], sb[j]);
    }
    using L = AccLayout<16>;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t row = m0 + 16 * i + L::row(lane, e), col = n0 + 16 * j + L::col(lane);
                if (row < p.M && col < p.N)
                    store_out<true>(p.out, row * p.out.ldc + col, acc[i][j][e]);
            }
}

}  // namespace

hipError_t launch_gemm_mx(const MxArgs& p) {
    const int64_t grid = ceil_div(p.M, 64) * ceil_div(p.N, 64);
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    mx_plain_kernel<2, 2, 2, 2><<<dim3(static_cast<unsigned>(grid)), dim3(256), 0, p.stream>>>(p);
    return hipGetLastError();
}

}  // namespace migemm
