// mx_api.cpp -- the MXFP4 entry points of the C ABI: argument checks, then the
// launchers in mx.hip and mx_gemm.hip.
#include "common.hpp"
#include "migemm.h"

namespace migemm {
namespace {

// A rows x cols MXFP4 matrix in two byte arrays: sizes, alignment and ranges
// (rows and cols at least 1 where need_ptrs is set).
struct MxRange {
    uintptr_t d0 = 0, d1 = 0, s0 = 0, s1 = 0;
};

bool mx_shape_ok(int64_t rows, int64_t cols, int64_t ldd, int64_t ldsc) {
    const int64_t blocks = ceil_div(cols, 32);
    return rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxDim && ldd >= 16 * blocks &&
           ldsc >= blocks && ldd >= 0 && ldsc >= 0 && ldd < kMaxLd && ldsc < kMaxLd &&
           ldd % 16 == 0 && ldsc % 16 == 0;
}

bool mx_range(const void* data, int64_t ldd, const void* scales, int64_t ldsc, int64_t rows,
              MxRange& r) {
    return data && scales && aligned16(data) && aligned16(scales) &&
           extent(data, rows, ldd, ldd, 1, r.d0, r.d1) &&
           extent(scales, rows, ldsc, ldsc, 1, r.s0, r.s1);
}

bool meets(const MxRange& r, uintptr_t lo, uintptr_t hi) {
    return overlaps(r.d0, r.d1, lo, hi) || overlaps(r.s0, r.s1, lo, hi);
}

}  // namespace
}  // namespace migemm

using namespace migemm;

extern "C" {

int migemm_quantize_mx(int src_dtype, int op, int64_t rows, int64_t cols, const void* src,
                       int64_t lds, void* data, int64_t ldd, void* scales, int64_t ldsc,
                       void* stream) {
    if (!known_dtype(src_dtype) || (op != MIGEMM_OP_N && op != MIGEMM_OP_T))
        return MIGEMM_ERR_INVALID_ARG;
    if (!mx_shape_ok(rows, cols, ldd, ldsc)) return MIGEMM_ERR_INVALID_ARG;
    const bool trans = op == MIGEMM_OP_T;
    const int64_t srows = trans ? cols : rows, scols = trans ? rows : cols;
    if (lds < (scols > 1 ? scols : 1) || lds >= kMaxLd) return MIGEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MIGEMM_OK;
    MxRange r;
    uintptr_t s0, s1;
    if (!src || !mx_range(data, ldd, scales, ldsc, rows, r) ||
        !extent(src, srows, scols, lds, elem_size(src_dtype), s0, s1) || meets(r, s0, s1) ||
        overlaps(r.d0, r.d1, r.s0, r.s1))
        return MIGEMM_ERR_INVALID_ARG;
    return hip_status(launch_quantize_mx(src_dtype, trans, rows, cols, src, lds,
                                         static_cast<uint8_t*>(data), ldd,
                                         static_cast<uint8_t*>(scales), ldsc,
                                         static_cast<hipStream_t>(stream)));
}

int migemm_dequantize_mx(int dst_dtype, int64_t rows, int64_t cols, const void* data, int64_t ldd,
                         const void* scales, int64_t ldsc, void* dst, int64_t ld, void* stream) {
    if (!known_dtype(dst_dtype) || !mx_shape_ok(rows, cols, ldd, ldsc))
        return MIGEMM_ERR_INVALID_ARG;
    if (ld < (cols > 1 ? cols : 1) || ld >= kMaxLd) return MIGEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MIGEMM_OK;
    MxRange r;
    uintptr_t s0, s1;
    if (!dst || !mx_range(data, ldd, scales, ldsc, rows, r) ||
        !extent(dst, rows, cols, ld, elem_size(dst_dtype), s0, s1) || meets(r, s0, s1))
        return MIGEMM_ERR_INVALID_ARG;
    return hip_status(launch_dequantize_mx(dst_dtype, rows, cols,
                                           static_cast<const uint8_t*>(data), ldd,
                                           static_cast<const uint8_t*>(scales), ldsc, dst, ld,
                                           static_cast<hipStream_t>(stream)));
}

int migemm_gemm_mx(int config, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                   const void* a_scales, int64_t ldas, const void* B, int64_t ldb,
                   const void* b_scales, int64_t ldbs, float alpha, float beta, int c_dtype,
                   void* C, int64_t ldc, void* stream) {
    if (!known_dtype(c_dtype) || !mx_shape_ok(M, K, lda, ldas) || !mx_shape_ok(N, K, ldb, ldbs) ||
        K % 32 != 0 || config < -1 || config >= mx_config_count())
        return MIGEMM_ERR_INVALID_ARG;
    if (ldc < (N > 1 ? N : 1) || ldc >= kMaxLd) return MIGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MIGEMM_OK;
    uintptr_t c0, c1;
    if (!C || !extent(C, M, N, ldc, elem_size(c_dtype), c0, c1)) return MIGEMM_ERR_INVALID_ARG;
    if (K > 0) {
        MxRange a, b;
        if (!mx_range(A, lda, a_scales, ldas, M, a) || !mx_range(B, ldb, b_scales, ldbs, N, b) ||
            meets(a, c0, c1) || meets(b, c0, c1))
            return MIGEMM_ERR_INVALID_ARG;
    }
    MxArgs p{M, N, K,
             static_cast<const uint8_t*>(A), lda, static_cast<const uint8_t*>(a_scales), ldas,
             static_cast<const uint8_t*>(B), ldb, static_cast<const uint8_t*>(b_scales), ldbs,
             Epi{C, ldc, alpha, beta, c_dtype}, static_cast<hipStream_t>(stream), false};
    p.whole_lines = c_whole_lines(p.out);
    return hip_status(launch_gemm_mx(p, config));
}

int migemm_mx_config_count(void) { return mx_config_count(); }

const char* migemm_mx_config_name(int config) { return mx_config_name(config); }

}  // extern "C"
