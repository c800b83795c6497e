// linear_loss.hip -- the row kernels of the output-layer losses
// (linear_loss.hpp): joining the forward statistics, the logits that a loss
// names, the losses; and the backward pass's row data, its scattered entries and
// its conversions.
#include "linear_loss.hpp"

namespace migemm {
namespace {

constexpr int kThreads = 256, kRowWaves = kThreads / kWave;
constexpr int kMaxTop = 1024;

// Joins two pairs (largest, sum) of base-2 statistics.  An empty pair has sum 0.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    if (s2 == 0.0f) return;
    if (s == 0.0f) {
        m = m2;
        s = s2;
        return;
    }
    const float hi = fmaxf(m, m2);
    // equal maxima (infinite ones too) keep their sums as they are
    s = s * (m == hi ? 1.0f : exp2_of(m - hi)) + s2 * (m2 == hi ? 1.0f : exp2_of(m2 - hi));
    m = hi;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// The dot products of a row x with U rows w[u], of `depth` elements each (whole
// 16-byte chunks), over a wavefront, in FP32.
template <int U, typename E>
__device__ __forceinline__ void row_dots(const E* __restrict__ x, const E* const (&w)[U],
                                         int64_t depth, int lane, float (&sum)[U]) {
    constexpr int EPC = 16 / sizeof(E);
#pragma unroll
    for (int u = 0; u < U; ++u) sum[u] = 0.0f;
#pragma unroll(U == 1 ? 4 : 2)
    for (int64_t c = static_cast<int64_t>(lane) * EPC; c < depth; c += kWave * EPC) {
        E xe[EPC], we[U][EPC];
        __builtin_memcpy(xe, __builtin_assume_aligned(x + c, 16), 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
            __builtin_memcpy(we[u], __builtin_assume_aligned(w[u] + c, 16), 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < EPC; ++e) sum[u] = fmaf(to_f32(xe[e]), to_f32(we[u][e]), sum[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) sum[u] = wave_sum(sum[u]);
}

// Teacher logit j of a row, in the teacher's type.
__device__ __forceinline__ float teacher_logit(const LossArgs& a, int64_t row, int64_t j) {
    const int64_t i = row * a.ldt + j;
    if (a.t_dtype == 0) return static_cast<const float*>(a.t_logits)[i];
    if (a.t_dtype == 1) return to_f32(static_cast<const _Float16*>(a.t_logits)[i]);
    return to_f32(static_cast<const bf16_t*>(a.t_logits)[i]);
}

// The teacher's distribution over a row's held entries (index >= 0), by one
// wavefront: p_j = 2^(scale (t_j - largest)) / sum.  held: a held entry with a
// logit above -infinity exists; bad: an index at or past V.
struct Teacher {
    float largest, sum;
    bool held, bad;
};
__device__ __forceinline__ Teacher teacher_row(const LossArgs& a, int64_t row, int lane) {
    const float scale = kLog2e / a.tau;
    Teacher t{-INFINITY, 0.0f, false, false};
    int bad = 0, nan = 0;
    for (int64_t j = lane; j < a.top; j += kWave) {
        const int64_t v = a.t_index[row * a.ldi + j];
        if (v < 0) continue;
        if (v >= a.V) bad = 1;
        const float x = teacher_logit(a, row, j);
        if (x != x) nan = 1;
        t.largest = fmaxf(t.largest, x);
    }
    t.largest = wave_max(t.largest);
    t.bad = __any(bad);
    // a NaN beside nothing else must not look like an empty row
    t.held = t.largest > -INFINITY || __any(nan);
    float s = 0.0f;
    for (int64_t j = lane; j < a.top; j += kWave)
        if (a.t_index[row * a.ldi + j] >= 0)
            s += exp2_of(scale * (teacher_logit(a, row, j) - t.largest));
    t.sum = wave_sum(s);
    return t;
}

// One workgroup per row: its log-sum-exp from the chunks' statistics, the logits
// at its target or at the teacher's indices, and its loss.  Bound by reading the rows
// of W that are named, from memory and caches: 4096 rows of 64 entries, D 4096 BF16, 269
// us (8 TB/s; 328 with one entry at a time).
// KD: distillation (cross entropy keeps fewer registers).
template <typename E, bool KD>
__global__ __launch_bounds__(kThreads) void loss_rows_kernel(LossArgs a, const E* __restrict__ X,
                                                             int64_t ldx, const E* __restrict__ W,
                                                             int64_t ldw, int64_t depth,
                                                             const RowStat* __restrict__ part,
                                                             int64_t chunks,
                                                             float* __restrict__ loss,
                                                             double* __restrict__ lse_out) {
    __shared__ RowStat stat[kRowWaves];
    __shared__ float logit[KD ? kMaxTop : 1];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    float m = -INFINITY, s = 0.0f;
    // eight chunks at a time, their loads in flight together (a row of 8192 chunks
    // joined one by one took 25 us)
    constexpr int kAhead = 8;
    const RowStat* const stats = part + row * chunks;
    for (int64_t c = threadIdx.x; c < chunks; c += kAhead * kThreads) {
        RowStat r[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t at = c + i * kThreads;
            r[i] = stats[at < chunks ? at : c];
            if (at >= chunks) r[i].sum = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) join(m, s, r[i].largest, r[i].sum);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const float m2 = __shfl_xor(m, d), s2 = __shfl_xor(s, d);
        join(m, s, m2, s2);
    }
    if (lane == 0) stat[wave] = RowStat{m, s};
    const E* const x = X + row * ldx;
    if constexpr (!KD) {
        const int64_t y = a.target[row];
        if (wave == 0 && y >= 0 && y < a.V && y != a.ignore) {
            const E* const w[1] = {W + y * ldw};
            float z[1];
            row_dots(x, w, depth, lane, z);
            if (lane == 0) logit[0] = z[0];
        }
    } else {
        // four entries of a wavefront at a time, their loads in flight together; one
        // that is not held reads row 0 and counts as 0
        constexpr int kEntries = 4;
        for (int64_t j0 = wave; j0 < a.top; j0 += kEntries * kRowWaves) {
            const E* w[kEntries];
            bool held[kEntries];
            float z[kEntries];
#pragma unroll
            for (int u = 0; u < kEntries; ++u) {
                const int64_t j = j0 + u * kRowWaves;
                const int64_t v = a.t_index[row * a.ldi + (j < a.top ? j : j0)];
                held[u] = v >= 0 && v < a.V;
                w[u] = W + (held[u] ? v : 0) * ldw;
            }
            row_dots(x, w, depth, lane, z);
#pragma unroll
            for (int u = 0; u < kEntries; ++u) {
                const int64_t j = j0 + u * kRowWaves;
                if (lane != 0 || j >= a.top) continue;
                logit[j] = held[u] ? z[u] : 0.0f;
                a.student[row * a.lds + j] = logit[j];
            }
        }
    }
    __syncthreads();
    if (wave != 0) return;
    m = stat[0].largest;
    s = stat[0].sum;
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) join(m, s, stat[w].largest, stat[w].sum);
    const double lse = (static_cast<double>(m) + log2(static_cast<double>(s))) * kLn2;
    float out = 0.0f;
    if constexpr (!KD) {
        const int64_t y = a.target[row];
        if (y != a.ignore) out = y >= 0 && y < a.V ? static_cast<float>(lse - logit[0]) : NAN;
    } else {
        const Teacher t = teacher_row(a, row, lane);
        if (t.held) {
            const double log_sum = log2(static_cast<double>(t.sum)) * kLn2;
            const double inv = 1.0 / a.tau;
            float terms = 0.0f;
            for (int64_t j = lane; j < a.top; j += kWave) {
                if (a.t_index[row * a.ldi + j] < 0) continue;
                const double log_p = (teacher_logit(a, row, j) - t.largest) * inv - log_sum;
                const float p = exp2_of(static_cast<float>(log_p * kLog2e));
                // no weight, no term: log p may be -infinity there
                if (p != 0.0f)
                    terms = fmaf(p, static_cast<float>(log_p - logit[j] * inv + lse), terms);
            }
            out = a.tau * a.tau * wave_sum(terms);
        }
        if (t.bad) out = NAN;
    }
    if (lane == 0) {
        loss[row] = out;
        lse_out[row] = lse;
    }
}

// factor[0] = f = 2^14 / m, within 2^+-100, and its inverse.
__device__ __forceinline__ void write_factor(float m, float* factor) {
    const float f = fminf(fmaxf(m > 0.0f ? 16384.0f / m : 1.0f, 0x1p-100f), 0x1p100f);
    factor[0] = f;
    factor[1] = 1.0f / f;
}

// A cross-entropy row's coefficient: 0 without a loss, NaN for a target outside
// the vocabulary.
__device__ __forceinline__ float ce_coef(const LossArgs& a, int64_t row,
                                         const float* __restrict__ grad) {
    const int64_t y = a.target[row];
    const float g = grad[row];  // (loaded whatever y is: both loads go out together)
    return y == a.ignore ? 0.0f : y >= 0 && y < a.V ? g : NAN;
}

// Row data of the backward pass, and X's row into the padded copy; rows from `twin` on
// (if not 0) are those of `twin` before.  factor (cross
// entropy only): written by the first workgroup, from all rows' coefficients;
// non-finite ones do not count.
template <typename E>
__global__ __launch_bounds__(kThreads) void loss_prepare_kernel(
    LossArgs a, const double* __restrict__ lse, const float* __restrict__ grad,
    LossRow* __restrict__ info, E* __restrict__ copy, int64_t rows, int64_t ldc,
    float* __restrict__ tp, float* __restrict__ factor, int64_t twin) {
    constexpr int EPC = 16 / sizeof(E);
    __shared__ float shared_coef, part[kRowWaves];
    if (factor != nullptr && blockIdx.x == 0) {
        float m = 0.0f;
        // eight rows at a time, their loads in flight together (one by one, 5888 rows
        // took 12 us)
        constexpr int kAhead = 8;
        for (int64_t i = threadIdx.x; i < a.T; i += kAhead * kThreads) {
            float c[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t at = i + j * kThreads;
                c[j] = fabsf(ce_coef(a, at < a.T ? at : i, grad));
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (c[j] < INFINITY) m = fmaxf(m, c[j]);
        }
        m = wave_max(m);
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kRowWaves; ++w) m = fmaxf(m, part[w]);
            write_factor(m, factor);
        }
    }
    const bool second = twin > 0 && blockIdx.x >= twin;
    const int64_t row = blockIdx.x - (second ? twin : 0);  // of the arguments
    const int64_t to = blockIdx.x;                         // of info and the copy
    const int lane = threadIdx.x % kWave;
    if (threadIdx.x < kWave) {
        LossRow r{0.0f, 0.0f, -1, 0.0f};
        if (row < a.T) {
            const double l = lse[row] * 1.4426950408889634;
            r.lse2 = static_cast<float>(l);
            if constexpr (sizeof(E) == 4)
                r.extra = fabsf(r.lse2) < INFINITY ? static_cast<float>(l - r.lse2) : 0.0f;
            else
                r.extra = second ? 1.0f : 0.0f;
            if (a.top == 0) {
                const int64_t y = a.target[row];
                r.coef = ce_coef(a, row, grad);
                if (y != a.ignore && y >= 0 && y < a.V) r.target = static_cast<int32_t>(y);
            } else {
                const Teacher t = teacher_row(a, row, lane);
                if (t.held) r.coef = a.tau * grad[row];
                if (t.bad) r.coef = NAN;
                const float scale = kLog2e / a.tau;
                for (int64_t j = lane; j < a.top; j += kWave) {
                    float p = 0.0f;
                    if (r.coef != 0.0f && a.t_index[row * a.ldi + j] >= 0)
                        p = exp2_of(scale * (teacher_logit(a, row, j) - t.largest)) / t.sum;
                    if (!second) tp[row * a.top + j] = r.coef * p;
                }
            }
        }
        if (lane == 0) {
            info[to] = r;
            shared_coef = r.coef;
        }
    }
    __syncthreads();
    if (to >= rows) return;
    const bool live = row < a.T && shared_coef != 0.0f;
    const E* const x = static_cast<const E*>(a.X) + row * a.ldx;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * EPC; c < ldc; c += kThreads * EPC) {
        u32x4 w = {0u, 0u, 0u, 0u};
        if (live && c + EPC <= a.D) {
            __builtin_memcpy(&w, x + c, 16);
        } else if (live) {
            E v[EPC];
            __builtin_memcpy(v, &w, 16);
#pragma unroll
            for (int e = 0; e < EPC; ++e)
                if (c + e < a.D) v[e] = x[c + e];
            __builtin_memcpy(&w, v, 16);
        }
        *reinterpret_cast<u32x4*>(copy + to * ldc + c) = w;
    }
}

// One workgroup.  Non-finite coefficients do not count.
__global__ __launch_bounds__(1024) void loss_factor_kernel(const LossRow* __restrict__ info,
                                                           int64_t rows,
                                                           float* __restrict__ factor) {
    __shared__ float part[16];
    float m = 0.0f;
    for (int64_t i = threadIdx.x; i < rows; i += 1024) {
        const float c = fabsf(info[i].coef);
        if (c < INFINITY) m = fmaxf(m, c);
    }
    m = wave_max(m);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = m;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 16; ++w) m = fmaxf(m, part[w]);
    write_factor(m, factor);
}

// A wavefront per row: dz at the indices inside [v0, v1).  An index that a row
// names more than once gets the sum of its weights, written by each of them.
template <typename E>
__global__ __launch_bounds__(kThreads) void loss_scatter_kernel(
    LossArgs a, const LossRow* __restrict__ info, const float* __restrict__ tp,
    const float* __restrict__ factor, E* __restrict__ dz, int64_t ldz, int64_t v0, int64_t v1,
    int64_t twin) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWaves + threadIdx.x / kWave;
    const int lane = threadIdx.x % kWave;
    if (row >= a.T) return;
    const LossRow r = info[row];
    if (r.coef == 0.0f) return;  // the whole row is 0 already
    const float f = factor ? *factor : 1.0f, scale = kLog2e / a.tau;
    const int64_t* const index = a.t_index + row * a.ldi;
    for (int64_t j = lane; j < a.top; j += kWave) {
        const int64_t v = index[j];
        if (v < v0 || v >= v1) continue;
        float weight = 0.0f;
        for (int64_t i = 0; i < a.top; ++i)
            if (index[i] == v) weight += tp[row * a.top + i];
        const float l = fmaf(a.student[row * a.lds + j], scale, -r.lse2);
        const float q = exp2_of(sizeof(E) == 4 ? l - r.extra : l);
        const float d = (r.coef * q - weight) * f;
        const E first = narrow<E>(d);
        dz[row * ldz + (v - v0)] = first;
        if (twin > 0) dz[(row + twin) * ldz + (v - v0)] = narrow<E>(d - to_f32(first));
    }
}

// 16 bytes of dst per lane.  65890 x 471 FP16: 27 us, 4.7 TB/s (40 an element at a time).
template <typename E>
__global__ __launch_bounds__(kThreads) void pad_copy_kernel(int64_t rows, int64_t cols,
                                                            const E* __restrict__ src, int64_t lds,
                                                            E* __restrict__ dst, int64_t pieces,
                                                            int64_t ldd) {
    constexpr int EPC = 16 / sizeof(E);
    for (int64_t p = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; p < pieces;
         p += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = p / (ldd / EPC), c = p % (ldd / EPC) * EPC;
        const E* const from = src + r * lds + c;
        u32x4 w = {0u, 0u, 0u, 0u};
        if (r < rows && c + EPC <= cols) {
            __builtin_memcpy(&w, from, 16);  // one load, whatever the alignment
        } else if (r < rows) {
            E v[EPC];
            __builtin_memcpy(v, &w, 16);
#pragma unroll
            for (int e = 0; e < EPC; ++e)
                if (c + e < cols) v[e] = from[e];
            __builtin_memcpy(&w, v, 16);
        }
        *reinterpret_cast<u32x4*>(dst + r * ldd + c) = w;
    }
}

// The sum over slices, scaled, four columns at a time.  LANES lanes share a piece of
// four columns, each adding every LANES-th slice with its loads in flight together;
// their sums join in a fixed order.  4096 x 4096, one slice into BF16: 20.5 us, 4.9 TB/s.
template <typename E, int LANES>
__global__ __launch_bounds__(kThreads) void join_kernel(int64_t rows, int64_t cols,
                                                        const float* __restrict__ src, int64_t lds,
                                                        int64_t slab, int slices,
                                                        const float* __restrict__ factor,
                                                        E* __restrict__ dst, int64_t ldd) {
    constexpr int kPieces = kWave / LANES;  // per wavefront
    const int lane = threadIdx.x % kWave, sub = lane / kPieces;
    const float f = factor ? *factor : 1.0f;
    const int64_t per = ceil_div(cols, 4), pieces = rows * per;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kRowWaves + threadIdx.x / kWave;
    for (int64_t p0 = wave * kPieces; p0 < pieces;
         p0 += static_cast<int64_t>(gridDim.x) * kRowWaves * kPieces) {
        const int64_t p = p0 + lane % kPieces;
        const int64_t r = (p < pieces ? p : p0) / per, c = (p < pieces ? p : p0) % per * 4;
        const float* const from = src + r * lds + c;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int s = sub; s < slices; s += LANES) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(from + s * slab);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += x[e];
        }
#pragma unroll
        for (int d = kPieces; d < kWave; d *= 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], d);
        if (sub != 0 || p >= pieces) continue;
        E out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = narrow<E>(v[e] * f);
        E* const to = dst + r * ldd + c;
        if (c + 4 <= cols) {
            __builtin_memcpy(to, out, sizeof(out));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < cols) to[e] = out[e];
        }
    }
}

unsigned grid_for(int64_t items) {
    const int64_t g = ceil_div(items, kThreads);
    return static_cast<unsigned>(g < 16384 ? g : 16384);
}

template <typename F>
hipError_t by_type(int dtype, F f) {
    if (dtype == 0) return f(float{});
    if (dtype == 1) return f(_Float16{});
    return f(bf16_t{});
}

}  // namespace

hipError_t launch_loss_rows(const LossArgs& a, const void* X, int64_t ldx, const void* W,
                            int64_t ldw, int64_t depth, const RowStat* part, int64_t chunks,
                            float* loss, double* lse) {
    return by_type(a.dtype, [&](auto tag) {
        using E = decltype(tag);
        auto* const fn = a.top ? loss_rows_kernel<E, true> : loss_rows_kernel<E, false>;
        fn<<<dim3(static_cast<unsigned>(a.T)), dim3(kThreads), 0, a.stream>>>(
            a, static_cast<const E*>(X), ldx, static_cast<const E*>(W), ldw, depth, part, chunks,
            loss, lse);
        return hipGetLastError();
    });
}

hipError_t launch_loss_prepare(const LossArgs& a, const double* lse, const float* grad,
                               LossRow* info, int64_t rows_info, void* copy, int64_t rows,
                               int64_t ldc, float* tp, float* factor, int64_t twin) {
    return by_type(a.dtype, [&](auto tag) {
        using E = decltype(tag);
        loss_prepare_kernel<E>
            <<<dim3(static_cast<unsigned>(rows_info)), dim3(kThreads), 0, a.stream>>>(
                a, lse, grad, info, static_cast<E*>(copy), rows, ldc, tp, factor, twin);
        return hipGetLastError();
    });
}

hipError_t launch_loss_factor(const LossRow* info, int64_t rows, float* factor, hipStream_t s) {
    loss_factor_kernel<<<dim3(1), dim3(1024), 0, s>>>(info, rows, factor);
    return hipGetLastError();
}

hipError_t launch_loss_scatter(const LossArgs& a, const LossRow* info, const float* tp,
                               const float* factor, void* dz, int64_t ldz, int64_t v0, int64_t v1,
                               int64_t twin) {
    return by_type(a.dtype, [&](auto tag) {
        using E = decltype(tag);
        const unsigned grid = static_cast<unsigned>(ceil_div(a.T, kRowWaves));
        loss_scatter_kernel<E><<<dim3(grid), dim3(kThreads), 0, a.stream>>>(
            a, info, tp, factor, static_cast<E*>(dz), ldz, v0, v1, twin);
        return hipGetLastError();
    });
}

hipError_t launch_pad_copy(int dtype, int64_t rows, int64_t cols, const void* src, int64_t lds,
                           void* dst, int64_t rows_out, int64_t ldd, hipStream_t s) {
    return by_type(dtype, [&](auto tag) {
        using E = decltype(tag);
        const int64_t pieces = rows_out * (ldd * static_cast<int64_t>(sizeof(E)) / 16);
        pad_copy_kernel<E><<<dim3(grid_for(pieces)), dim3(kThreads), 0, s>>>(
            rows, cols, static_cast<const E*>(src), lds, static_cast<E*>(dst), pieces, ldd);
        return hipGetLastError();
    });
}

hipError_t launch_join(int dtype, int64_t rows, int64_t cols, const float* src, int64_t lds,
                       int64_t slab, int slices, const float* factor, void* dst, int64_t ldd,
                       hipStream_t s) {
    return by_type(dtype, [&](auto tag) {
        using E = decltype(tag);
        const int lanes = slices >= 16 ? 8 : 1;
        auto* const fn = lanes == 8 ? join_kernel<E, 8> : join_kernel<E, 1>;
        fn<<<dim3(grid_for(rows * ceil_div(cols, 4) * lanes)), dim3(kThreads), 0, s>>>(
            rows, cols, src, lds, slab, slices, factor, static_cast<E*>(dst), ldd);
        return hipGetLastError();
    });
}

}  // namespace migemm
