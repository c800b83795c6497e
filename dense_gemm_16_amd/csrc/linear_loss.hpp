// linear_loss.hpp -- the losses of an output layer's rows (softmax cross entropy
// and distillation from a teacher's top logits) and what their kernels share.
//
// z = X W^T (X: T tokens x D, W: V vocabulary rows x D) is never stored.  The
// forward pass runs the product with an output step that keeps, per row and
// wave-wide chunk of columns, the largest value m and the sum of exp(z - m)
// (LseOut); a row kernel joins the chunks into the row's log-sum-exp and forms the few
// logits the loss names as the product forms them, bit for bit.  The backward pass
// walks the vocabulary in pieces: it recomputes a piece of z with an output step
// that writes the derivative of the loss to it,
//     dz[t][v] = c_t (exp(z[t][v] / tau - lse_t) - p[t][v]),  c_t = tau g_t
// (tau = 1 and p one-hot for cross entropy), in the operands' type (DzOut), then
// adds dz W to dX and writes dz^T X to the piece's rows of dW.
//
// 16-bit dz holds a factor f = 2^14 / max |c_t|, taken out of the gradients in
// FP32.  FP16 derivatives far below the largest stay normal, and where all rows
// weigh the same (a mean) c f is a power of two: rounding c (q - 1) then costs a
// target half a step just below 2^14, where steps are finest, instead of giving
// every row of small q the same rounding of c (BF16, 8192 rows: dW off by 0.0031
// without it, of which 0.0017 are the final rounding).  Rows of other weights are rounded
// as those would be (BF16, 512 x 8192 x 256: both gradients off by 0.0020 with equal
// weights, 0.0023 with weights of 0.25 to 1.25, 0.0027 with 0.6 beside a single 1).
//
// Exponents are kept in base 2: with s = log2(e) / tau, exp(z / tau - lse) =
// 2^(s z - l), l = lse log2(e), one fused multiply-add and one hardware exp2.
// Statistics are FP32, except that lse is kept in 64 bits (an FP32 one of 8 to 16 is off
// by up to 2^-21, and with it every q of the row, and a distillation's loss by tau^2
// times that).
//
// Up to kTwin rows of 16-bit dz are kept as two terms, dz and what its rounding left:
// row t + kTwin of x is row t again, and the tile of 64 rows has the room.  dw's sum
// over rows and dx's over a row and its twin then hold dz to 16 (FP16: 22) bits.  With
// few rows the roundings of dz do not average out (5 tokens, distillation, BF16: dx
// and dw off by 0.0026 without, of which 0.0017 are the final rounding).
#pragma once

#include "mfma16_direct.hpp"

namespace migemm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;

// What the derivative of a row needs: l, c_t (0: a row without a loss, whose
// derivative is 0 whatever its logits), the target's column (-1: none), and what l lacks
// of its 64-bit value (l of 16 to 32 in FP32 is off by up to 2^-20, which is all there is
// to 1 - q of a nearly certain row).
struct LossRow {
    float lse2, coef;
    int32_t target;
    float extra;
};
constexpr int64_t kTwin = 32;

// A float2-like pair of one row's statistics over one chunk of columns: the
// largest s z, and the sum of 2^(s z - largest).
struct RowStat {
    float largest, sum;
};

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum and sum over the 16 lanes of a DPP row, left in every lane.
template <int CTRL> __device__ __forceinline__ float dpp_ror(float v) {
    return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(__float_as_uint(v)), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float max16(float v) {
    v = fmaxf(v, dpp_ror<0x128>(v));
    v = fmaxf(v, dpp_ror<0x124>(v));
    v = fmaxf(v, dpp_ror<0x122>(v));
    return fmaxf(v, dpp_ror<0x121>(v));
}
__device__ __forceinline__ float sum16(float v) {
    v += dpp_ror<0x128>(v);
    v += dpp_ror<0x124>(v);
    v += dpp_ror<0x122>(v);
    return v + dpp_ror<0x121>(v);
}

// Output step of the forward product: statistics of each row over the wave's
// columns, to part[row * chunks + column / WTN].  A lane holds column lane % 16
// of rows 4 g .. 4 g + 3 of every 16 x 16 block, so a row's columns lie in the
// lane's TN registers and 16 lanes of one DPP row: no LDS and no barrier.  4096 x 65536
// x 4096 BF16 on the ping-pong tile: 1463 us, 1.50 PFLOPS, matrix units 83% busy; 8 x
// 131072 x 4096: 170 us, W read at 6.3 TB/s.
struct LseOut : Epi {
    RowStat* part;
    int64_t chunks;
    float scale;  // s
    template <class Cfg, class Acc>
    __device__ __forceinline__ void store(const Acc (&acc)[Cfg::TM][Cfg::TN], MIGEMM_LDS char*,
                                          int64_t m, int64_t n, int, int lane, int64_t M,
                                          int64_t N) const {
        constexpr int TM = Cfg::TM, TN = Cfg::TN;
        static_assert(Cfg::MF == 16, "16 x 16 blocks");
        const int g = lane >> 4, lj = lane & 15;
        const bool inside = n + Cfg::WTN <= N;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            float largest = 0.0f, sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    v[j] = inside || n + 16 * j + lj < N ? acc[i][j][e] : -INFINITY;
                float mx = v[0];
#pragma unroll
                for (int j = 1; j < TN; ++j) mx = fmaxf(mx, v[j]);
                mx = max16(mx) * scale;
                // an infinite maximum is left out of the exponents: the sum is
                // then 0 (nothing but -infinity) or +infinity
                const float shift = fabsf(mx) < INFINITY ? mx : 0.0f;
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < TN; ++j) s += exp2_of(fmaf(v[j], scale, -shift));
                s = sum16(s);
                // lane lj = 0..3 of each group keeps row 4 g + lj
                if (lj == e) {
                    largest = mx;
                    sum = s;
                }
            }
            const int64_t row = m + 16 * i + 4 * g + lj;
            if (lj < 4 && row < M) part[row * chunks + n / Cfg::WTN] = RowStat{largest, sum};
        }
    }
};

// FP32 to the storage of a 16-bit or FP32 element.
template <typename E> __device__ __forceinline__ E narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ _Float16 narrow<_Float16>(float x) {
    return static_cast<_Float16>(x);
}
template <> __device__ __forceinline__ bf16_t narrow<bf16_t>(float x) {
    return bf16_t{f32_to_bf16_bits(x)};
}

// Output step of the backward product: dz, rounded once into the operands' type
// because the two products that follow run on the matrix cores in that type;
// the rounding is half a step of each dz, independent of the others (a twin row
// holds it).  Columns
// from N to the end of the last tile (at most ldz, the piece's width rounded up to
// 64) become 0, so that the products may read whole 16-byte chunks past N, and so do
// rows from M to `rows` (rounded up to 64), so that dw's product runs whole k-tiles.
// Each 16-row block of the wave's tile goes through the wave's own LDS to be
// written 16 bytes per lane in whole row pieces.  4096 x 65536 x 4096 BF16: 1545 us, 1.42
// PFLOPS, matrix units 77% busy.
template <typename E>
struct DzOut : Epi {
    E* dz;
    int64_t ldz, rows, v0;
    const LossRow* info;  // padded to whole tiles of rows
    const float* factor;  // f, or NULL
    float scale;          // s
    int64_t twin;         // rows from here on hold what their twins' rounding left
    template <class Cfg, class Acc>
    __device__ __forceinline__ void store(const Acc (&acc)[Cfg::TM][Cfg::TN],
                                          MIGEMM_LDS char* smem, int64_t m, int64_t n, int wave,
                                          int lane, int64_t, int64_t N) const {
        constexpr int TM = Cfg::TM, TN = Cfg::TN, WTM = Cfg::WTM, WTN = Cfg::WTN;
        constexpr int ES = sizeof(E), VE = 16 / ES, PIECES = WTN / VE;
        using Bits = std::conditional_t<ES == 4, uint32_t, uint16_t>;
        constexpr int kBytes = WTM * 16 + 16 * WTN * ES;
        static_assert(Cfg::MF == 16 && Cfg::NW * kBytes <= Cfg::LDS_BYTES, "scratch fits");
        static_assert((PIECES & (PIECES - 1)) == 0, "the swizzle permutes a row's pieces");
        MIGEMM_LDS f32x4* const ri = (MIGEMM_LDS f32x4*)(smem + wave * kBytes);
        MIGEMM_LDS char* const scr = smem + wave * kBytes + WTM * 16;
        const float f = factor ? *factor : 1.0f;
        for (int i = lane; i < WTM; i += kWave) {
            f32x4 r = reinterpret_cast<const f32x4*>(info)[m + i];
            r[1] *= f;
            ri[i] = r;
        }
        const int g = lane >> 4, lj = lane & 15;
        asm volatile("" : : : "memory");
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * g + e;
                const LossRow row = __builtin_bit_cast(LossRow, f32x4(ri[16 * i + r]));
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int64_t col = n + 16 * j + lj;
                    const float l = fmaf(acc[i][j][e], scale, -row.lse2);
                    float v = row.coef * exp2_of(l - row.extra);
                    if (v0 + col == row.target) v -= row.coef;
                    if (row.coef == 0.0f || col >= N) v = 0.0f;
                    if (ES != 4 && Cfg::BM == 64 && m + 16 * i + r >= twin)  // (64-row tiles)
                        v -= to_f32(narrow<E>(v));
                    const int c = 16 * j + lj;
                    const int piece = (c / VE) ^ ((g << 1) & (PIECES - 1));
                    *(MIGEMM_LDS Bits*)(scr + (r * WTN + piece * VE + c % VE) * ES) =
                        __builtin_bit_cast(Bits, narrow<E>(v));
                }
            }
            asm volatile("" : : : "memory");
#pragma unroll
            for (int q = 0; q < (16 * PIECES + kWave - 1) / kWave; ++q) {
                const int p = lane + q * kWave, r = p / PIECES, c = p % PIECES;
                if (16 * PIECES % kWave != 0 && p >= 16 * PIECES) continue;
                const int phys = c ^ (((r >> 2) << 1) & (PIECES - 1));
                const u32x4 w = *(const MIGEMM_LDS u32x4*)(scr + (r * WTN + phys * VE) * ES);
                const int64_t grow = m + 16 * i + r, gcol = n + c * VE;
                if (grow < rows && gcol < ldz)
                    *reinterpret_cast<u32x4*>(dz + grow * ldz + gcol) = w;
            }
            asm volatile("" : : : "memory");
        }
    }
};

// Output step of dw = dz^T x where the products' own does not do: the sums times
// *factor (1 / f), rounded into the operands' type, columns below `cols` only (x
// is a copy padded to whole chunks).
// As DzOut, through LDS into 16-byte row pieces, non-temporal where rows are whole
// 128-byte lines (dz and dw of 64 x 32000 x 4096 BF16 112 us against 158, with an
// optimizer's pass over dw behind it 246 against 265).  65536 x 4096 x 4096 BF16: 1673
// us, 1.31 PFLOPS, matrix units 72% busy; both operands have k as their row index.
template <typename E>
struct GradOut : Epi {
    E* grad;
    int64_t ldg, cols;
    const float* factor;
    bool nt;
    template <class Cfg, class Acc>
    __device__ __forceinline__ void store(const Acc (&acc)[Cfg::TM][Cfg::TN],
                                          MIGEMM_LDS char* smem, int64_t m, int64_t n, int wave,
                                          int lane, int64_t M, int64_t) const {
        constexpr int TM = Cfg::TM, TN = Cfg::TN, WTN = Cfg::WTN;
        constexpr int ES = sizeof(E), VE = 16 / ES, PIECES = WTN / VE;
        using Bits = std::conditional_t<ES == 4, uint32_t, uint16_t>;
        constexpr int kBytes = 16 * WTN * ES;
        static_assert(Cfg::MF == 16 && Cfg::NW * kBytes <= Cfg::LDS_BYTES, "scratch fits");
        MIGEMM_LDS char* const scr = smem + wave * kBytes;
        const float f = factor ? *factor : 1.0f;
        const int g = lane >> 4, lj = lane & 15;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int r = 4 * g + e, c = 16 * j + lj;
                    const int piece = (c / VE) ^ ((g << 1) & (PIECES - 1));
                    *(MIGEMM_LDS Bits*)(scr + (r * WTN + piece * VE + c % VE) * ES) =
                        __builtin_bit_cast(Bits, narrow<E>(acc[i][j][e] * f));
                }
            asm volatile("" : : : "memory");
#pragma unroll
            for (int q = 0; q < (16 * PIECES + kWave - 1) / kWave; ++q) {
                const int p = lane + q * kWave, r = p / PIECES, c = p % PIECES;
                if (16 * PIECES % kWave != 0 && p >= 16 * PIECES) continue;
                const int phys = c ^ (((r >> 2) << 1) & (PIECES - 1));
                const MIGEMM_LDS char* const from = scr + (r * WTN + phys * VE) * ES;
                const int64_t grow = m + 16 * i + r, gcol = n + c * VE;
                if (grow >= M || gcol >= cols) continue;
                E* const to = grad + grow * ldg + gcol;
                if (gcol + VE <= cols) {
                    const u32x4 w = *(const MIGEMM_LDS u32x4*)from;
                    if (nt)
                        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(to));
                    else
                        __builtin_memcpy(to, &w, 16);  // one store, whatever the alignment
                } else {
#pragma nounroll
                    for (int e = 0; e < VE; ++e)
                        if (gcol + e < cols)
                            reinterpret_cast<Bits*>(to)[e] =
                                *(const MIGEMM_LDS Bits*)(from + e * ES);
                }
            }
            asm volatile("" : : : "memory");
        }
    }
};

// One product with one of the output steps: X W^T (M x N, K deep) with lse or dz,
// dz^T X (A stored K x M, zero-filled to whole chunks, B stored K x N) with grad, or
// the sums of `slices` slices of dz W's k (A M x K, zero-filled to whole chunks, B
// stored K x N), M x N of FP32 each, one after another at `sums`.  A and B are
// 16-byte aligned with leading dimensions in whole 16-byte chunks, and so are K (lse,
// dz) or N (grad, sums).
struct LossTile {
    int64_t M, N, K;
    int dtype;
    const void* A;
    int64_t lda;
    const void* B;
    int64_t ldb;
    hipStream_t stream;
    const LseOut* lse;
    const void* dz;    // DzOut of the type
    const void* grad;  // GradOut of the type
    float* sums = nullptr;
    int slices = 0;
};

// The tile configuration for a product of these sizes, its chunk width (columns
// per wave) and its columns per tile; the launcher of configuration C for
// element type E (linear_loss_part.hip).
struct LossShape {
    int config, chunk, bn;
};
LossShape loss_shape(int dtype, int64_t M, int64_t N, int64_t K);
template <typename E, int C>
hipError_t launch_loss_tile(const LossTile& t);
hipError_t launch_loss(const LossTile& t, int config);

// The arguments of one call, as the row kernels take them.
struct LossArgs {
    int64_t T, V, D;
    int dtype;
    const void* X;
    int64_t ldx;
    const void* W;
    int64_t ldw;
    // cross entropy (top == 0)
    const int64_t* target;
    int64_t ignore;
    // distillation: `top` teacher logits and vocabulary indices per row
    int64_t top;
    int t_dtype;
    const void* t_logits;
    int64_t ldt;
    const int64_t* t_index;
    int64_t ldi;
    float tau;
    float* student;  // the student's logits at the indices (written forward, read backward)
    int64_t lds;
    hipStream_t stream;
};

// Row kernels (linear_loss.hip).  X and W: 16-byte aligned rows, `depth` elements
// (whole chunks) of them read.  head: how many elements before k = 0 the logits' product
// starts its first slab of k.
hipError_t launch_loss_rows(const LossArgs& a, const void* X, int64_t ldx, const void* W,
                            int64_t ldw, int64_t depth, int head, const RowStat* part,
                            int64_t chunks, float* loss, double* lse);
// info for `rows_info` rows, X's rows as a zero-padded copy (rows x ldc; rows
// without a loss become 0), for distillation tp[t][j] = c_t p_j, and for cross
// entropy the factor (NULL: none).  twin: kTwin, or 0.
hipError_t launch_loss_prepare(const LossArgs& a, const double* lse, const float* grad,
                               LossRow* info, int64_t rows_info, void* copy, int64_t rows,
                               int64_t ldc, float* tp, float* factor, int64_t twin);
// factor[0] = what brings the largest |coef| to 2^14, factor[1] its inverse.
hipError_t launch_loss_factor(const LossRow* info, int64_t rows, float* factor, hipStream_t s);
// Overwrites the entries of dz that distillation's indices name.
hipError_t launch_loss_scatter(const LossArgs& a, const LossRow* info, const float* tp,
                               const float* factor, void* dz, int64_t ldz, int64_t v0, int64_t v1,
                               int64_t twin);
// dst (rows_out x ldd, zero-padded) = src (rows x cols).
hipError_t launch_pad_copy(int dtype, int64_t rows, int64_t cols, const void* src, int64_t lds,
                           void* dst, int64_t rows_out, int64_t ldd, hipStream_t s);
// dst (rows x cols, dtype) = the sum of `slices` FP32 matrices (leading dimension lds,
// whole 16-byte chunks, each `slab` elements after the one before), times (factor ?
// *factor : 1).
hipError_t launch_join(int dtype, int64_t rows, int64_t cols, const float* src, int64_t lds,
                       int64_t slab, int slices, const float* factor, void* dst, int64_t ldd,
                       hipStream_t s);

}  // namespace migemm
