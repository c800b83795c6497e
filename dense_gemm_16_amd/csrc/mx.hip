// mx.hip -- quantisation of FP32, FP16 and BF16 matrices to microscaled 4-bit
// floating point (MXFP4), and its decoding.
//
// The format.  A row is cut into blocks of 32 elements along k.  A block has
// one scale byte b, the power of two 2^(b - 127) (255: the block is NaN), and
// 32 four-bit elements: sign, two exponent bits, one mantissa bit, the values
// 0, 0.5, 1, 1.5, 2, 3, 4 and 6 and their negatives (codes 0 to 7, sign 8).  Two
// elements share a byte, the even one in the low half; a block is 16 bytes.
//
// The rule.  With m the largest magnitude of a block, the scale is 2^e with
// e = floor(log2 m) - 2 (the largest element, 6 = 1.5 x 2^2, then covers m up to
// a quarter of a step), at least -127; every element is x 2^-e rounded to the
// nearest of the values above, midpoints to the even code, magnitudes past 6 to
// 6.  In bits: for FP32 m with biased exponent field E, b = max(E - 2, 0), and
// x 2^-e = x 2^(127 - b) is a product by a normal FP32 power of two, exact.  A
// block that holds an infinity or a NaN has no such scale and becomes NaN
// (b = 255, all codes 0); an all-zero one has b = 0.
#include "common.hpp"

namespace migemm {
namespace {

constexpr int kThreads = 256;

// The larger of m and |x|, NaN if either is (v_maximum3_f32 takes two elements).
__device__ __forceinline__ float largest_of(float m, float x) {
    return __builtin_elementwise_maximum(m, fabsf(x));
}

// The scale byte of a block whose largest magnitude is m.
__device__ __forceinline__ uint32_t scale_byte(float m) {
    const int e = static_cast<int>(__float_as_uint(m) >> 23);  // sign 0
    return e >= 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}

// 2^(127 - b), the factor that brings a block of scale byte b to element units;
// 0 for a NaN block, whose codes are dropped by the caller.
__device__ __forceinline__ float unscale(uint32_t b) {
    return b == 255u ? 0.0f : __uint_as_float((254u - b) << 23);
}

// The codes of eight values in element units: the hardware rounds to the nearest
// code, midpoints to the even one, larger magnitudes to 6 (its own scale operand
// stays 1: a block's 2^e may be subnormal).  Spelled out in integer arithmetic the
// rounding took 12 instructions an element and bounded the kernel.
__device__ __forceinline__ uint32_t fp4_codes(const float (&y)[8]) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
}

// Eight consecutive elements from column c of a row, zeros past cols.
template <typename T>
__device__ __forceinline__ void load8(const T* __restrict__ row, int64_t c, int64_t cols,
                                      float (&v)[8]) {
    if (c + 8 <= cols) {
        T e[8];
        __builtin_memcpy(e, row + c, sizeof(e));  // 16 bytes at a time, whatever the alignment
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_f32(row[c + i]) : 0.0f;
    }
}

// Rows along k (OP_N).  Four lanes share a block, eight elements each, so loads
// are 16 bytes per lane and contiguous over a wavefront.  A workgroup takes
// kThreads / lpr rows (lpr lanes each, a power of two) of one segment of columns.
// Bound by memory: 8192 x 8192 FP32 48 us (6.3 TB/s), BF16 32 (5.3).
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(
    int64_t rows, int64_t cols, const T* __restrict__ src, int64_t lds, uint8_t* __restrict__ data,
    int64_t ldd, uint8_t* __restrict__ scales, int64_t ldsc, int lpr, int64_t segs) {
    const int64_t group = blockIdx.x / segs, seg = blockIdx.x % segs;
    const int64_t row = group * (kThreads / lpr) + threadIdx.x / lpr;
    const int64_t piece = seg * lpr + threadIdx.x % lpr;  // of eight elements
    const int64_t blocks = ceil_div(cols, 32);
    // whole groups of four lanes leave together
    if (row >= rows || piece / 4 >= blocks) return;
    float v[8];
    load8<T>(src + row * lds, piece * 8, cols, v);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = largest_of(m, v[i]);
    m = largest_of(m, __shfl_xor(m, 1));
    m = largest_of(m, __shfl_xor(m, 2));
    const uint32_t b = scale_byte(m);
    const float f = unscale(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= f;
    const uint32_t w = b == 255u ? 0u : fp4_codes(v);
    *reinterpret_cast<uint32_t*>(data + row * ldd + piece * 4) = w;
    if (piece % 4 == 0) scales[row * ldsc + piece / 4] = static_cast<uint8_t>(b);
}

// k as the row index of the source (OP_T): a lane owns a few neighbouring rows of
// the result (8 bytes of a source row) and one block at a time, so that a
// wavefront's loads are 512 bytes of one source row; a workgroup takes its rows by
// 8 blocks, and the packed blocks go through LDS (the 16-byte slot XORed by the
// lane, which spreads a wavefront's writes over the banks) to be written 128 bytes
// to a row.
//
// ONCE: non-temporal loads, for a source on 8-byte boundaries that the 256 MB
// last-level cache cannot hold beside the result (8192 x 8192 FP32, 268 MB: 53.7 us,
// 5.7 TB/s, against 65.0 for plain ones; one that still lies in the cache is read
// faster with those, BF16 of that size 34.2 us against 37.2).  One row per lane, 256
// bytes of an FP32 source row, took 102.
constexpr int kBlocks = 8;
template <typename T> constexpr int kPerLane = 8 / sizeof(T);

template <typename T, bool ONCE>
__global__ __launch_bounds__(kBlocks * kWave) void quantize_cols_kernel(
    int64_t rows, int64_t cols, const T* __restrict__ src, int64_t lds, uint8_t* __restrict__ data,
    int64_t ldd, uint8_t* __restrict__ scales, int64_t ldsc, int64_t tiles_k) {
    constexpr int P = kPerLane<T>, kRows = kWave * P;
    __shared__ __attribute__((aligned(16))) u32x4 out[kRows][kBlocks];
    __shared__ uint8_t sc[kRows][kBlocks];
    const int64_t r0 = blockIdx.x / tiles_k * kRows, b0 = blockIdx.x % tiles_k * kBlocks;
    const int64_t blocks = ceil_div(cols, 32);
    const int lane = threadIdx.x % kWave;
    const int64_t row = r0 + lane * P;
    const int blk = threadIdx.x / kWave;
    const int64_t k0 = (b0 + blk) * 32;
    if (k0 < cols) {
        T v[32][P];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const T* const p = src + (k0 + i) * lds + row;
            if (k0 + i < cols && row + P <= rows) {
                u32x2 w;
                if constexpr (ONCE)
                    w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
                else
                    __builtin_memcpy(&w, p, sizeof(w));
                __builtin_memcpy(v[i], &w, sizeof(v[i]));
            } else {
#pragma unroll
                for (int c = 0; c < P; ++c)
                    v[i][c] = k0 + i < cols && row + c < rows ? p[c] : ZeroOf<T>::get();
            }
        }
#pragma unroll
        for (int c = 0; c < P; ++c) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) m = largest_of(m, to_f32(v[i][c]));
            const uint32_t b = scale_byte(m);
            const float f = unscale(b);
            u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = to_f32(v[8 * q + i][c]) * f;
                w[q] = b == 255u ? 0u : fp4_codes(y);
            }
            out[lane * P + c][blk ^ (lane & 7)] = w;
            sc[lane * P + c][blk] = static_cast<uint8_t>(b);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kBlocks; i += kBlocks * kWave) {
        const int r = i / kBlocks, blk = i % kBlocks;
        if (r0 + r >= rows || b0 + blk >= blocks) continue;
        *reinterpret_cast<u32x4*>(data + (r0 + r) * ldd + (b0 + blk) * 16) =
            out[r][blk ^ ((r / P) & 7)];
        scales[(r0 + r) * ldsc + b0 + blk] = sc[r][blk];
    }
}

// The value of a four-bit code.
__device__ __forceinline__ float fp4_value(uint32_t code) {
    // codes 0 and 1 are 0 and 0.5; from 2 on, exponent field code / 2 over 1 / 2,
    // mantissa bit code % 2: the code placed at FP32 bit 22, bias 126
    const uint32_t mag = code & 7u;
    const float a = mag < 2u ? 0.5f * static_cast<float>(mag)
                             : __uint_as_float((mag << 22) + (126u << 23));
    return code & 8u ? -a : a;
}

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ _Float16 from_f32<_Float16>(float x) {
    return static_cast<_Float16>(x);
}
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float x) {
    return bf16_t{f32_to_bf16_bits(x)};
}

// 16 bytes of the result per lane and store, so that each store of a wavefront is
// contiguous (32 bytes of an FP32 row per lane, as two stores: 8192 x 8192 102 us).  A
// result that the 32 MiB of the L2 caches hold is written piece by piece: a reader
// that follows finds it there (4096 x 4096 BF16 and then a negation 23.9 us, 25.9 in the
// other form).  A larger one four pieces a lane, with non-temporal stores where it is
// aligned: 8192 x 8192 FP32 44.6 us (6.8 TB/s, part of it into the last-level cache)
// against 81, 67.8 with plain stores; and a negation 156 against 175.  BF16 27 us (6.2 TB/s).
template <typename T, int U>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(
    int64_t rows, int64_t cols, const uint8_t* __restrict__ data, int64_t ldd,
    const uint8_t* __restrict__ scales, int64_t ldsc, T* __restrict__ dst, int64_t ld, int lpr,
    int64_t segs, bool once) {
    constexpr int VE = 16 / sizeof(T);
    using Codes = std::conditional_t<VE == 8, uint32_t, uint16_t>;
    const int64_t group = blockIdx.x / segs, seg = blockIdx.x % segs;
    const int64_t row = group * (kThreads / lpr) + threadIdx.x / lpr;
    const int64_t first = seg * lpr * U + threadIdx.x % lpr;
    if (row >= rows) return;
    uint32_t w[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t piece = first + u * lpr;
        if (piece * VE >= cols) continue;
        w[u] = *reinterpret_cast<const Codes*>(data + row * ldd + piece * (VE / 2));
        b[u] = scales[row * ldsc + piece * VE / 32];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = (first + u * lpr) * VE;
        if (c >= cols) continue;
        const float s = b[u] == 255u ? __uint_as_float(0x7fc00000u)
                                     : __uint_as_float(b[u] == 0u ? 0x00400000u : b[u] << 23);
        T v[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = from_f32<T>(fp4_value((w[u] >> (4 * i)) & 15u) * s);
        T* const p = dst + row * ld + c;
        if (c + VE <= cols) {
            u32x4 raw;
            __builtin_memcpy(&raw, v, 16);
            if (once)
                __builtin_nontemporal_store(raw, reinterpret_cast<u32x4*>(p));
            else
                __builtin_memcpy(p, &raw, 16);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (c + i < cols) p[i] = v[i];
        }
    }
}

// Lanes per row (a power of two, 4 to 256) and column segments for rows of
// `pieces` eight-element pieces.
void row_shape(int64_t pieces, int& lpr, int64_t& segs) {
    lpr = 4;
    while (lpr < kThreads && lpr < pieces) lpr *= 2;
    segs = ceil_div(pieces, lpr);
}

// Calls launch(first row, rows, workgroups) for parts of the rows, kThreads / lpr rows and
// `segs` workgroups a group, that one launch holds.
template <typename F>
hipError_t by_rows(int64_t rows, int lpr, int64_t segs, F launch) {
    const int64_t per = kThreads / lpr, step = launch_groups(kThreads) / segs * per;
    for (int64_t r = 0; r < rows; r += step) {
        const int64_t n = rows - r < step ? rows - r : step;
        launch(r, n, static_cast<unsigned>(ceil_div(n, per) * segs));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T>
hipError_t quantize_typed(bool trans, int64_t rows, int64_t cols, const void* src, int64_t lds,
                          uint8_t* data, int64_t ldd, uint8_t* scales, int64_t ldsc,
                          hipStream_t s) {
    const T* p = static_cast<const T*>(src);
    if (trans) {
        const bool vec = reinterpret_cast<uintptr_t>(src) % 8 == 0 &&
                         lds % kPerLane<T> == 0;
        const bool large =
            static_cast<double>(cols) * static_cast<double>(lds) * sizeof(T) > 201326592.0;
        auto* const fn =
            vec && large ? quantize_cols_kernel<T, true> : quantize_cols_kernel<T, false>;
        // whole tiles of k and of rows, as many as one launch holds
        constexpr int64_t kRows = kWave * kPerLane<T>, kCols = 32 * kBlocks;
        constexpr int64_t most = launch_groups(kBlocks * kWave), kMostK = int64_t(1) << 20;
        for (int64_t k = 0; k < cols; k += kMostK * kCols) {
            const int64_t nk = cols - k < kMostK * kCols ? cols - k : kMostK * kCols;
            const int64_t tiles_k = ceil_div(nk, kCols), step = most / tiles_k * kRows;
            for (int64_t r = 0; r < rows; r += step) {
                const int64_t nr = rows - r < step ? rows - r : step;
                fn<<<dim3(static_cast<unsigned>(ceil_div(nr, kRows) * tiles_k)),
                     dim3(kBlocks * kWave), 0, s>>>(nr, nk, p + k * lds + r, lds,
                                                    data + r * ldd + k / 2, ldd,
                                                    scales + r * ldsc + k / 32, ldsc, tiles_k);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
        }
        return hipSuccess;
    }
    int lpr;
    int64_t segs;
    row_shape(4 * ceil_div(cols, 32), lpr, segs);
    return by_rows(rows, lpr, segs, [&](int64_t r, int64_t n, unsigned grid) {
        quantize_rows_kernel<T><<<dim3(grid), dim3(kThreads), 0, s>>>(
            n, cols, p + r * lds, lds, data + r * ldd, ldd, scales + r * ldsc, ldsc, lpr, segs);
    });
}

template <typename T>
hipError_t dequantize_typed(int64_t rows, int64_t cols, const uint8_t* data, int64_t ldd,
                            const uint8_t* scales, int64_t ldsc, void* dst, int64_t ld,
                            hipStream_t s) {
    const int64_t pieces = ceil_div(cols, 16 / static_cast<int64_t>(sizeof(T)));
    int lpr;
    int64_t segs;
    row_shape(pieces, lpr, segs);
    const bool large =
        static_cast<double>(rows) * static_cast<double>(cols) * sizeof(T) > 33554432.0;
    const bool wide = segs > 1 && large;
    if (wide) segs = ceil_div(segs, 4);
    const bool once = large && aligned16(dst) && (ld * static_cast<int64_t>(sizeof(T))) % 16 == 0;
    auto* const fn = wide ? dequantize_kernel<T, 4> : dequantize_kernel<T, 1>;
    return by_rows(rows, lpr, segs, [&](int64_t r, int64_t n, unsigned grid) {
        fn<<<dim3(grid), dim3(kThreads), 0, s>>>(n, cols, data + r * ldd, ldd, scales + r * ldsc,
                                                 ldsc, static_cast<T*>(dst) + r * ld, ld, lpr, segs,
                                                 once);
    });
}

}  // namespace

hipError_t launch_quantize_mx(int dtype, bool trans, int64_t rows, int64_t cols, const void* src,
                              int64_t lds, uint8_t* data, int64_t ldd, uint8_t* scales,
                              int64_t ldsc, hipStream_t s) {
    if (dtype == 0)
        return quantize_typed<float>(trans, rows, cols, src, lds, data, ldd, scales, ldsc, s);
    if (dtype == 1)
        return quantize_typed<_Float16>(trans, rows, cols, src, lds, data, ldd, scales, ldsc, s);
    return quantize_typed<bf16_t>(trans, rows, cols, src, lds, data, ldd, scales, ldsc, s);
}

hipError_t launch_dequantize_mx(int dtype, int64_t rows, int64_t cols, const uint8_t* data,
                                int64_t ldd, const uint8_t* scales, int64_t ldsc, void* dst,
                                int64_t ld, hipStream_t s) {
    if (dtype == 0) return dequantize_typed<float>(rows, cols, data, ldd, scales, ldsc, dst, ld, s);
    if (dtype == 1)
        return dequantize_typed<_Float16>(rows, cols, data, ldd, scales, ldsc, dst, ld, s);
    return dequantize_typed<bf16_t>(rows, cols, data, ldd, scales, ldsc, dst, ld, s);
}

}  // namespace migemm
