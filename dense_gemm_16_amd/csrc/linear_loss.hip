// linear_loss.hip -- the row kernels of the output-layer losses
// (linear_loss.hpp): joining the forward statistics, the logits that a loss
// names, the losses; and the backward pass's row data, its scattered entries and
// its conversions.
#include <utility>

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

// Each lane i of a 16-lane row gets lane (i + N) % 16's value, in the groups of four lanes
// that BANKS names; the others keep `old`.
template <int N, int BANKS = 0xf>
__device__ __forceinline__ u32x4 rotated(u32x4 v, u32x4 old = u32x4{0u, 0u, 0u, 0u}) {
    if constexpr (N % 16 == 0) return v;
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        r[e] = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
            static_cast<int>(old[e]), static_cast<int>(v[e]), 0x120 + (16 - N % 16) % 16, 0xf,
            BANKS, false));
    return r;
}

template <int... N, class F>
__device__ __forceinline__ void for_each_slab(std::integer_sequence<int, N...>, F f) {
    (f(std::integral_constant<int, N>{}), ...);
}

// Logits of row x and PER rows w (w[h]: that of this lane's entry, lane % PER, or 8 h +
// lane % 8 of 16), in lanes 0 to PER - 1, in the bits that the product's accumulators
// hold: the same matrix instructions over the same slabs of k (a slab is one 16-byte chunk
// per lane group, DirectOperand's row images) in the same order, zeros before and past the
// ends.  lse is a sum over those accumulators, so their roundings cancel in lse - z; an
// FP32 dot product of another order is off by 1e-4 at logits of 200, which the loss and
// the derivative of a nearly certain row then consisted of.  head: elements before k = 0
// in the first slab (a partial first k-tile of the 256x256 product).  `depth` elements,
// whole chunks.
//
// The instruction's block is row x sixteen times by 16 entries.  With fewer than 16 the
// other lanes of a group load the slabs that follow, and the registers rotate by PER lanes
// from one slab to the next; 16 entries come as two loads of eight rows by two slabs (whole
// 128-byte lines), exchanged by halves.  The next U loads are in flight while U run.
// XS: x lies in LDS (x_slabs), read a slab at a time, which leaves registers for more of
// w's loads (2048 rows of 32 entries, D 2048 FP16: 56 us against 62).
template <int PER, bool XS, typename E>
__device__ __forceinline__ float named_logits(const E* __restrict__ x, const u32x4* xs,
                                              const E* const (&w)[PER == 16 ? 2 : 1],
                                              int64_t depth, int head, int lane) {
    constexpr int EPC = 16 / sizeof(E), kSlab = 4 * EPC;
    constexpr int H = PER == 16 ? 2 : 1, S = PER == 16 ? 2 : 16 / PER;  // rows, slabs of a load
    constexpr int U = (XS ? 8 : 4) / H, kLoad = S * kSlab, kStep = U * kLoad;
    const int64_t k0 = (lane / 16) * EPC + (lane % 16 / (16 / S)) * kSlab - head;
    const int64_t end = depth + head;
    struct Batch {
        u32x4 a[XS ? 1 : U], b[H][U];
    };
    auto load = [&](int64_t s, Batch& t) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + s + u * kLoad;
            const bool in = k >= 0 && k < depth;
            if constexpr (!XS) {
                t.a[u] = u32x4{0u, 0u, 0u, 0u};
                if (in) t.a[u] = *reinterpret_cast<const u32x4*>(x + k);
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                t.b[h][u] = u32x4{0u, 0u, 0u, 0u};
                if (in) t.b[h][u] = *reinterpret_cast<const u32x4*>(w[h] + k);
            }
        }
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    // slab n of load u, which starts at slab `slab`
    auto one = [&](int64_t slab, int u, const Batch& t, auto n_tag) __attribute__((always_inline)) {
        constexpr int N = decltype(n_tag)::value;
        u32x4 a, b;
        if constexpr (XS)
            a = xs[(slab + N) * 4 + lane / 16];
        else
            a = rotated<N * (16 / S)>(t.a[u]);
        if constexpr (PER != 16)
            b = rotated<N * PER>(t.b[0][u]);
        else if constexpr (N == 0)
            b = rotated<8, 0xc>(t.b[1][u], t.b[0][u]);
        else
            b = rotated<8, 0x3>(t.b[0][u], t.b[1][u]);
        MfmaOp<E, 16>::run(acc, a, b);
    };
    auto run = [&](int64_t s, const Batch& t) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u * kLoad >= end) break;
            for_each_slab(std::make_integer_sequence<int, S>{},
                          [&](auto n) __attribute__((always_inline)) {
                              one(s / kSlab + u * S, u, t, n);
                          });
        }
    };
    Batch t0, t1;
    load(0, t0);
    for (int64_t s = 0; s < end; s += 2 * kStep) {
        load(s + kStep, t1);
        run(s, t0);
        load(s + 2 * kStep, t0);
        run(s + kStep, t1);
    }
    return acc[0];
}

// Row x as named_logits reads it from LDS: `head` zeros, x, zeros to the end of the last
// load.  Up to kSlabBytes of x.
constexpr int kSlabBytes = 16384, kSlabRoom = kSlabBytes + 2048;
template <typename E>
__device__ __forceinline__ void x_slabs(const E* __restrict__ x, int64_t depth, int head,
                                        u32x4* xs) {
    constexpr int EPC = 16 / sizeof(E), kMost = 16 * 4;  // chunks of sixteen slabs
    const int last = static_cast<int>(depth + head) / EPC, first = head / EPC;
    for (int c = threadIdx.x; c < (last + kMost - 1) / kMost * kMost; c += kThreads) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (c >= first && c < last) v = *reinterpret_cast<const u32x4*>(x + (c - first) * EPC);
        xs[c] = v;
    }
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
// of W that are named, from memory and caches: 4096 rows of 64 entries, D 4096 BF16, 280
// us (7.7 TB/s); few rows by the chain of matrix instructions (33 rows of 8 entries, D 520
// FP32, 130 of them: 11 us).
// KD: distillation (cross entropy keeps fewer registers).  PER: entries of a wavefront at
// a time, a power of two up to 16: the fewest that the four need once, or 16.
template <typename E, bool KD, int PER, bool XS>
__global__ __launch_bounds__(kThreads) void loss_rows_kernel(LossArgs a, const E* __restrict__ X,
                                                             int64_t ldx, const E* __restrict__ W,
                                                             int64_t ldw, int64_t depth, int head,
                                                             float scale,
                                                             const RowStat* __restrict__ part,
                                                             int64_t chunks,
                                                             float* __restrict__ loss,
                                                             double* __restrict__ lse_out) {
    __shared__ RowStat stat[kRowWaves];
    __shared__ float logit[KD ? kMaxTop : 1];
    __shared__ u32x4 xs[XS ? kSlabRoom / 16 : 1];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    float m = -INFINITY, s = 0.0f;
    // eight chunks at a time, their loads in flight together (a row of 8192 chunks
    // joined one by one took 25 us); the target's logit is wave 0's meanwhile
    constexpr int kAhead = 8, kFirst = KD ? 0 : kWave, kOver = kThreads - kFirst;
    const RowStat* const stats = part + row * chunks;
    const E* const x = X + row * ldx;
    if constexpr (XS) x_slabs(x, depth, head, xs);
    if (!KD && wave == 0) {
        const int64_t y = a.target[row];
        if (y >= 0 && y < a.V && y != a.ignore) {
            const E* const w[1] = {W + y * ldw};
            const float z = named_logits<1, false>(x, xs, w, depth, head, lane);
            if (lane == 0) logit[0] = z;
        }
    } else {
        for (int64_t c = static_cast<int>(threadIdx.x) - kFirst; c < chunks; c += kAhead * kOver) {
            RowStat r[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int64_t at = c + i * kOver;
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
    }
    if (lane == 0) stat[wave] = RowStat{m, s};
    if constexpr (KD) {
        if constexpr (XS) __syncthreads();
        // one that is not held reads row 0 and counts as 0
        for (int64_t j0 = wave * PER; j0 < a.top; j0 += PER * kRowWaves) {
            constexpr int H = PER == 16 ? 2 : 1, kRows = PER / H;
            const E* w[H];
            bool held = false;
            const int64_t j = j0 + lane % PER;  // the entry whose logit this lane gets
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int64_t i = j0 + h * kRows + lane % kRows;
                const int64_t v = a.t_index[row * a.ldi + (i < a.top ? i : j0)];
                const bool in = v >= 0 && v < a.V;
                if (i == j) held = in;
                w[h] = W + (in ? v : 0) * ldw;
            }
            const float z = named_logits<PER, XS>(x, xs, w, depth, head, lane);
            if (lane < PER && j < a.top) {
                logit[j] = held ? z : 0.0f;
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
    // in base 2, as the statistics are: s z of a named logit is subtracted from it exactly
    const double lse2 = static_cast<double>(m) + log2(static_cast<double>(s));
    float out = 0.0f;
    if constexpr (!KD) {
        const int64_t y = a.target[row];
        if (y != a.ignore)
            out = y >= 0 && y < a.V
                      ? static_cast<float>((lse2 - static_cast<double>(scale) * logit[0]) * kLn2)
                      : NAN;
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
                    terms = fmaf(p, static_cast<float>(log_p + (lse2 - static_cast<double>(scale) *
                                                                          logit[j]) * kLn2),
                                 terms);
            }
            out = a.tau * a.tau * wave_sum(terms);
        }
        if (t.bad) out = NAN;
    }
    if (lane == 0) {
        loss[row] = out < 0.0f ? 0.0f : out;  // (neither loss is negative but for rounding)
        lse_out[row] = lse2 * kLn2;
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
            r.extra = fabsf(r.lse2) < INFINITY ? static_cast<float>(l - r.lse2) : 0.0f;
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
        const float q = exp2_of(fmaf(a.student[row * a.lds + j], scale, -r.lse2) - r.extra);
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
                            int64_t ldw, int64_t depth, int head, const RowStat* part,
                            int64_t chunks, float* loss, double* lse) {
    return by_type(a.dtype, [&](auto tag) {
        using E = decltype(tag);
        const bool xs = depth * static_cast<int64_t>(sizeof(E)) <= kSlabBytes;
#define MIGEMM_ROWS(PER) \
    (xs ? loss_rows_kernel<E, true, PER, true> : loss_rows_kernel<E, true, PER, false>)
        auto* const fn = a.top == 0                ? loss_rows_kernel<E, false, 1, false>
                         : a.top <= kRowWaves     ? MIGEMM_ROWS(1)
                         : a.top <= 2 * kRowWaves ? MIGEMM_ROWS(2)
                         : a.top <= 4 * kRowWaves ? MIGEMM_ROWS(4)
                         : a.top <= 8 * kRowWaves ? MIGEMM_ROWS(8)
                                                  : MIGEMM_ROWS(16);
#undef MIGEMM_ROWS
        fn<<<dim3(static_cast<unsigned>(a.T)), dim3(kThreads), 0, a.stream>>>(
            a, static_cast<const E*>(X), ldx, static_cast<const E*>(W), ldw, depth, head,
            kLog2e / a.tau, part, chunks, loss, lse);
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
