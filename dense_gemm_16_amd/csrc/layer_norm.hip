// layer_norm.hip -- layer norm over rows, forwards and backwards, with the sums over rows
// that are the gradients of its weight and bias.
//
// With mu and var the mean and variance of a row of D, r = 1 / sqrt(var + eps) and
// h = (x - mu) r:  y = h w + b.  Backwards, with g = dy w:
//     dx = r (g - mean(g) - h mean(g h)),   dw = sum over rows of dy h,   db = ... of dy.
// Everything is FP32 from the loads to the one rounding into the result's type.  The
// variance is the mean of (x - mu)^2 over the row's registers, not a difference of
// squares: a row far from zero keeps its digits.
//
// Bound by memory: x is read and y written once; backwards dy and x are read and dx
// written once.  A row lives in the registers of LANES lanes (16 to 1024), E elements
// each.
#include "rows.hpp"
#include "training.hpp"

namespace migemm {
namespace {

constexpr int kLongThreads = 1024;  // a row that no register form holds
constexpr int kColumns = 8;         // its columns per work-item, backwards

template <int LANES> constexpr int kThreads = LANES <= kWave ? 256 : LANES;
template <int LANES> constexpr int kRows = kThreads<LANES> / LANES;
template <int LANES> constexpr int kWaves = LANES <= kWave ? 1 : LANES / kWave;

// Sums of N values over a row's lanes, in every one of them.  `lds` is free again once
// the row's work-items have passed the barrier of the call after this one.
template <int LANES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (&lds)[N][kWaves<LANES>]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = sum_lanes<LANES <= kWave ? LANES : kWave>(v[i]);
    if constexpr (LANES > kWave) {
        if (threadIdx.x % kWave == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds[i][threadIdx.x / kWave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = lds[i][0];
#pragma unroll
            for (int w = 1; w < kWaves<LANES>; ++w) v[i] += lds[i][w];
        }
    }
}

// A lane's pieces of a row of D: CH chunks of 16 bytes (of T), LANES chunks apart.
template <typename T, int LANES, int CH> struct Pieces {
    static constexpr int C = kChunk<T>;
    static __device__ __forceinline__ int column(int c, int lane) { return (c * LANES + lane) * C; }
    template <typename E>
    static __device__ __forceinline__ void load(const E* row, int D, int lane, E (&e)[CH][C]) {
#pragma unroll
        for (int c = 0; c < CH; ++c) load_part(row + column(c, lane), D - column(c, lane), e[c]);
    }
    template <typename E>
    static __device__ __forceinline__ void store(E* row, int D, int lane, const E (&e)[CH][C]) {
#pragma unroll
        for (int c = 0; c < CH; ++c) store_part(row + column(c, lane), D - column(c, lane), e[c]);
    }
};

template <typename T, typename W, int LANES, int CH>
__global__ __launch_bounds__(kThreads<LANES>) void norm_kernel(
    int64_t rows, int D, const T* __restrict__ X, int64_t ldx, const W* __restrict__ weight,
    const W* __restrict__ bias, float eps, T* __restrict__ Y, int64_t ldy,
    float* __restrict__ means, float* __restrict__ rstds) {
    using P = Pieces<T, LANES, CH>;
    constexpr int C = P::C;
    __shared__ float lds[2][1][kWaves<LANES>];
    const int lane = threadIdx.x % LANES;
    const float d = static_cast<float>(D);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows<LANES> + threadIdx.x / LANES;
         row < rows; row += static_cast<int64_t>(gridDim.x) * kRows<LANES>) {
        T x[CH][C];
        W w[CH][C], b[CH][C];
        P::load(X + row * ldx, D, lane, x);
        if (weight) P::load(weight, D, lane, w);
        if (bias) P::load(bias, D, lane, b);
        float v[CH][C], sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[c][i] = to_f32(x[c][i]);
                sum[0] += v[c][i];
            }
        row_sums<LANES>(sum, lds[0]);
        const float mean = sum[0] / d;
        sum[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[c][i] -= mean;
                if (P::column(c, lane) + i < D) sum[0] += v[c][i] * v[c][i];
            }
        row_sums<LANES>(sum, lds[1]);
        const float rstd = 1.0f / sqrtf(sum[0] / d + eps);
        T y[CH][C];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float o = v[c][i] * rstd;
                if (weight) o *= to_f32(w[c][i]);
                if (bias) o += to_f32(b[c][i]);
                y[c][i] = narrow<T>(o);
            }
        P::store(Y + row * ldy, D, lane, y);
        if (lane == 0) {
            if (means) means[row] = mean;
            if (rstds) rstds[row] = rstd;
        }
    }
}

// The same for rows of any length: three passes, the later ones from the caches.
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(
    int64_t rows, int64_t D, const T* __restrict__ X, int64_t ldx, const W* __restrict__ weight,
    const W* __restrict__ bias, float eps, T* __restrict__ Y, int64_t ldy,
    float* __restrict__ means, float* __restrict__ rstds) {
    constexpr int C = kChunk<T>;
    __shared__ float lds[2][1][kWaves<kLongThreads>];
    const float d = static_cast<float>(D);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* const x = X + row * ldx;
        float sum[1] = {0.0f};
        for (int64_t k = threadIdx.x * C; k < D; k += kLongThreads * C) {
            T e[C];
            load_part(x + k, D - k, e);
#pragma unroll
            for (int i = 0; i < C; ++i) sum[0] += to_f32(e[i]);
        }
        row_sums<kLongThreads>(sum, lds[0]);
        const float mean = sum[0] / d;
        sum[0] = 0.0f;
        for (int64_t k = threadIdx.x * C; k < D; k += kLongThreads * C) {
            T e[C];
            load_part(x + k, D - k, e);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float v = to_f32(e[i]) - mean;
                if (k + i < D) sum[0] += v * v;
            }
        }
        row_sums<kLongThreads>(sum, lds[1]);
        const float rstd = 1.0f / sqrtf(sum[0] / d + eps);
        for (int64_t k = threadIdx.x * C; k < D; k += kLongThreads * C) {
            T e[C];
            W w[C], b[C];
            load_part(x + k, D - k, e);
            if (weight) load_part(weight + k, D - k, w);
            if (bias) load_part(bias + k, D - k, b);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float o = (to_f32(e[i]) - mean) * rstd;
                if (weight) o *= to_f32(w[i]);
                if (bias) o += to_f32(b[i]);
                e[i] = narrow<T>(o);
            }
            store_part(Y + row * ldy + k, D - k, e);
        }
        if (threadIdx.x == 0) {
            if (means) means[row] = mean;
            if (rstds) rstds[row] = rstd;
        }
    }
}

// Backwards.  A workgroup walks rows a grid apart, the next row's loads in flight while a
// row is summed; each lane keeps dw and db of its columns in registers, and the workgroup
// writes one partial sum of each, which norm_join_kernel adds.  SUMS: dw or db is wanted.
template <typename T, typename W, int LANES, int CH, bool SUMS>
__global__ __launch_bounds__(kThreads<LANES>) void norm_backward_kernel(
    int64_t rows, int D, const T* __restrict__ dY, int64_t lddy, const T* __restrict__ X,
    int64_t ldx, const W* __restrict__ weight, const float* __restrict__ means,
    const float* __restrict__ rstds, T* __restrict__ dX, int64_t lddx,
    float* __restrict__ partial, int64_t pitch) {
    using P = Pieces<T, LANES, CH>;
    constexpr int C = P::C, R = kRows<LANES>;
    __shared__ float lds[2][2][kWaves<LANES>];
    const int lane = threadIdx.x % LANES, part = threadIdx.x / LANES;
    const float d = static_cast<float>(D);
    float w[CH][C], dw[CH][C], db[CH][C];
    {
        W e[CH][C];
        if (weight) P::load(weight, D, lane, e);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                w[c][i] = weight ? to_f32(e[c][i]) : 1.0f;
                dw[c][i] = db[c][i] = 0.0f;
            }
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * R;
    int64_t row = static_cast<int64_t>(blockIdx.x) * R + part;
    T x[CH][C], dy[CH][C];
    float mean = 0.0f, rstd = 0.0f;
    if (row < rows) {
        P::load(X + row * ldx, D, lane, x);
        P::load(dY + row * lddy, D, lane, dy);
        mean = means[row];
        rstd = rstds[row];
    }
    for (int turn = 0; row < rows; row += step, turn ^= 1) {
        float h[CH][C], g[CH][C], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float o = to_f32(dy[c][i]);
                h[c][i] = (to_f32(x[c][i]) - mean) * rstd;
                g[c][i] = o * w[c][i];
                if (P::column(c, lane) + i < D) {
                    sum[0] += g[c][i];
                    sum[1] += g[c][i] * h[c][i];
                }
                if constexpr (SUMS) {
                    dw[c][i] += o * h[c][i];
                    db[c][i] += o;
                }
            }
        const float r = rstd;
        if (row + step < rows) {
            P::load(X + (row + step) * ldx, D, lane, x);
            P::load(dY + (row + step) * lddy, D, lane, dy);
            mean = means[row + step];
            rstd = rstds[row + step];
        }
        if (dX) {
            row_sums<LANES>(sum, lds[turn]);
            const float a = sum[0] / d, b = sum[1] / d;
            T o[CH][C];
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < C; ++i) o[c][i] = narrow<T>(r * (g[c][i] - a - h[c][i] * b));
            P::store(dX + row * lddx, D, lane, o);
        }
    }
    if constexpr (SUMS) {
        float* const out = partial + static_cast<int64_t>(blockIdx.x) * 2 * pitch;
        if constexpr (R == 1) {
            P::store(out, D, lane, dw);
            P::store(out + pitch, D, lane, db);
        } else {
            // the workgroup's rows are joined in order, dw first
            constexpr int kWidth = LANES * CH * C;
            __shared__ __attribute__((aligned(16))) float rows_of[R][kWidth];
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                if (which) __syncthreads();
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    store_whole(&rows_of[part][P::column(c, lane)], which ? db[c] : dw[c]);
                __syncthreads();
                for (int k = threadIdx.x; k < kWidth && k < D; k += kThreads<LANES>) {
                    float s = rows_of[0][k];
#pragma unroll
                    for (int i = 1; i < R; ++i) s += rows_of[i][k];
                    out[which * pitch + k] = s;
                }
            }
        }
    }
}

// Rows too long for registers, backwards: first the two sums of each row,
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_long_sums_kernel(
    int64_t rows, int64_t D, const T* __restrict__ dY, int64_t lddy, const T* __restrict__ X,
    int64_t ldx, const W* __restrict__ weight, const float* __restrict__ means,
    const float* __restrict__ rstds, float* __restrict__ sums) {
    constexpr int C = kChunk<T>;
    __shared__ float lds[2][2][kWaves<kLongThreads>];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        const float mean = means[row], rstd = rstds[row];
        float sum[2] = {0.0f, 0.0f};
        for (int64_t k = threadIdx.x * C; k < D; k += kLongThreads * C) {
            T x[C], dy[C];
            W w[C];
            load_part(X + row * ldx + k, D - k, x);
            load_part(dY + row * lddy + k, D - k, dy);
            if (weight) load_part(weight + k, D - k, w);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float g = to_f32(dy[i]);
                if (weight) g *= to_f32(w[i]);
                if (k + i < D) {
                    sum[0] += g;
                    sum[1] += g * ((to_f32(x[i]) - mean) * rstd);
                }
            }
        }
        row_sums<kLongThreads>(sum, lds[turn]);
        if (threadIdx.x == 0) {
            sums[2 * row] = sum[0];
            sums[2 * row + 1] = sum[1];
        }
    }
}

// then dx and the partial sums of a slab of rows by a band of columns.
template <typename T, typename W>
__global__ __launch_bounds__(256) void norm_long_backward_kernel(
    int64_t rows, int64_t D, int64_t slab, int64_t bands, const T* __restrict__ dY, int64_t lddy,
    const T* __restrict__ X, int64_t ldx, const W* __restrict__ weight,
    const float* __restrict__ means, const float* __restrict__ rstds,
    const float* __restrict__ sums, T* __restrict__ dX, int64_t lddx,
    float* __restrict__ partial, int64_t pitch) {
    constexpr int N = kColumns;
    const int64_t p = blockIdx.x / bands;
    const int64_t k = ((blockIdx.x % bands) * 256 + threadIdx.x) * N;
    if (k >= D) return;
    const float d = static_cast<float>(D);
    float w[N], dw[N], db[N];
    {
        W e[N];
        if (weight) load_part(weight + k, D - k, e);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = weight ? to_f32(e[i]) : 1.0f;
            dw[i] = db[i] = 0.0f;
        }
    }
    const int64_t end = (p + 1) * slab < rows ? (p + 1) * slab : rows;
#pragma unroll 2
    for (int64_t row = p * slab; row < end; ++row) {
        T x[N], dy[N];
        load_part(X + row * ldx + k, D - k, x);
        load_part(dY + row * lddy + k, D - k, dy);
        const float mean = means[row], rstd = rstds[row];
        const float a = sums[2 * row] / d, b = sums[2 * row + 1] / d;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float o = to_f32(dy[i]), h = (to_f32(x[i]) - mean) * rstd;
            dw[i] += o * h;
            db[i] += o;
            x[i] = narrow<T>(rstd * (o * w[i] - a - h * b));
        }
        if (dX) store_part(dX + row * lddx + k, D - k, x);
    }
    float* const out = partial + p * 2 * pitch + k;
    store_part(out, D - k, dw);
    store_part(out + pitch, D - k, db);
}

// dw (blockIdx.y 0) and db (1): the partial sums of 64 columns, every sixteenth of them by
// one wavefront, joined in order.
constexpr int kJoin = 16;
template <typename W>
__global__ __launch_bounds__(kJoin * kWave) void norm_join_kernel(
    int64_t parts, int64_t D, const float* __restrict__ partial, int64_t pitch,
    W* __restrict__ dW, W* __restrict__ dB) {
    __shared__ float lds[kJoin][kWave];
    W* const out = blockIdx.y ? dB : dW;
    if (!out) return;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * kWave + lane;
    float s = 0.0f;
    if (k < D) {
        const float* const from = partial + blockIdx.y * pitch + k;
#pragma unroll 8
        for (int64_t p = wave; p < parts; p += kJoin) s += from[p * 2 * pitch];
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && k < D) {
#pragma unroll
        for (int i = 1; i < kJoin; ++i) s += lds[i][lane];
        out[k] = narrow<W>(s);
    }
}

// How a row of D lies in registers: lanes, and elements of each.  Two elements a lane more
// than a row needs cost nothing; more than 16 leave too few wavefronts in flight
// backwards, where five values a column are held.
constexpr int64_t kMaxInRegisters = 16384;

template <typename T, typename F> hipError_t with_form(int64_t D, F f) {
    constexpr int C = kChunk<T>;
    using std::integral_constant;
    auto form = [&](auto lanes, auto elements) {
        return f(lanes, integral_constant<int, decltype(elements)::value / C>{});
    };
    using e8 = integral_constant<int, 8>;
    using e16 = integral_constant<int, 16>;
    if (D <= 128) return form(integral_constant<int, 16>{}, e8{});
    if (D <= 512) return form(integral_constant<int, 64>{}, e8{});
    if (D <= 1024) return form(integral_constant<int, 64>{}, e16{});
    if (D <= 2048) return form(integral_constant<int, 128>{}, e16{});
    if (D <= 4096) return form(integral_constant<int, 256>{}, e16{});
    if (D <= 8192) return form(integral_constant<int, 512>{}, e16{});
    return form(integral_constant<int, 1024>{}, e16{});
}

int rows_of_form(int64_t D) { return D <= 128 ? 16 : D <= 1024 ? 4 : 1; }

template <typename T, typename W> hipError_t forward(const NormArgs& a) {
    const T* const x = static_cast<const T*>(a.X);
    const W *const w = static_cast<const W*>(a.W), *const b = static_cast<const W*>(a.B);
    T* const y = static_cast<T*>(a.Y);
    const int64_t most = int64_t(1) << 20;  // workgroups; they stride over the rest
    if (a.D > kMaxInRegisters) {
        norm_long_kernel<T, W><<<dim3(static_cast<unsigned>(a.T < most ? a.T : most)),
                                 dim3(kLongThreads), 0, a.stream>>>(
            a.T, a.D, x, a.ldx, w, b, a.eps, y, a.ldy, a.mean, a.rstd);
        return hipGetLastError();
    }
    return with_form<T>(a.D, [&](auto lanes, auto chunks) {
        constexpr int L = decltype(lanes)::value, CH = decltype(chunks)::value;
        int64_t blocks = ceil_div(a.T, kRows<L>);
        if (blocks > most) blocks = most;
        norm_kernel<T, W, L, CH><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads<L>), 0,
                                   a.stream>>>(a.T, static_cast<int>(a.D), x, a.ldx, w, b, a.eps,
                                               y, a.ldy, a.mean, a.rstd);
        return hipGetLastError();
    });
}

// Workgroups of the backward pass, each of which writes partial sums.
int64_t backward_parts(int64_t T, int64_t D) {
    const int64_t groups = ceil_div(T, 4 * rows_of_form(D));
    return groups < 512 ? groups : 512;
}
int64_t long_slab(int64_t T) { return ceil_div(T, T < 64 * 32 ? ceil_div(T, 32) : 64); }
int64_t pitch_of(int64_t D) { return ceil_div(D, 64) * 64; }

template <typename T, typename W> hipError_t backward(const NormArgs& a, void* ws) {
    const T *const x = static_cast<const T*>(a.X), *const dy = static_cast<const T*>(a.dY);
    const W* const w = static_cast<const W*>(a.W);
    T* const dx = static_cast<T*>(a.Y);
    float* partial = static_cast<float*>(ws);
    const int64_t pitch = pitch_of(a.D);
    int64_t parts = 0;
    hipError_t err;
    if (a.D > kMaxInRegisters) {
        const int64_t slab = long_slab(a.T), bands = ceil_div(a.D, 256 * kColumns);
        parts = ceil_div(a.T, slab);
        float* const sums = partial + parts * 2 * pitch;
        const int64_t most = int64_t(1) << 20;
        norm_long_sums_kernel<T, W><<<dim3(static_cast<unsigned>(a.T < most ? a.T : most)),
                                      dim3(kLongThreads), 0, a.stream>>>(
            a.T, a.D, dy, a.lddy, x, a.ldx, w, a.mean, a.rstd, sums);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
        norm_long_backward_kernel<T, W><<<dim3(static_cast<unsigned>(parts * bands)), dim3(256), 0,
                                          a.stream>>>(a.T, a.D, slab, bands, dy, a.lddy, x, a.ldx,
                                                      w, a.mean, a.rstd, sums, dx, a.ldy, partial,
                                                      pitch);
        err = hipGetLastError();
    } else {
        const bool sums = a.dW || a.dB;
        err = with_form<T>(a.D, [&](auto lanes, auto chunks) {
            constexpr int L = decltype(lanes)::value, CH = decltype(chunks)::value;
            auto go = [&](auto want) {
                norm_backward_kernel<T, W, L, CH, decltype(want)::value>
                    <<<dim3(static_cast<unsigned>(parts)), dim3(kThreads<L>), 0, a.stream>>>(
                        a.T, static_cast<int>(a.D), dy, a.lddy, x, a.ldx, w, a.mean, a.rstd, dx,
                        a.ldy, partial, pitch);
                return hipGetLastError();
            };
            if (sums) {
                parts = backward_parts(a.T, a.D);
                return go(std::true_type{});
            }
            const int64_t most = int64_t(1) << 20;
            parts = ceil_div(a.T, kRows<L>);
            if (parts > most) parts = most;
            return go(std::false_type{});
        });
    }
    if (err != hipSuccess || (!a.dW && !a.dB)) return err;
    norm_join_kernel<W><<<dim3(static_cast<unsigned>(ceil_div(a.D, kWave)), 2), dim3(kJoin * kWave),
                          0, a.stream>>>(parts, a.D, partial, pitch, static_cast<W*>(a.dW),
                                         static_cast<W*>(a.dB));
    return hipGetLastError();
}

template <typename F> hipError_t with_types(int dtype, int w_dtype, F f) {
    switch (dtype) {
        case 0: return f(float{}, float{});
        case 1: return w_dtype == 0 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
        default: return w_dtype == 0 ? f(bf16_t{}, float{}) : f(bf16_t{}, bf16_t{});
    }
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a) {
    return with_types(a.dtype, a.w_dtype, [&](auto t, auto w) {
        return forward<decltype(t), decltype(w)>(a);
    });
}

int64_t layer_norm_workspace(int64_t T, int64_t D, bool vectors) {
    if (T == 0) return 0;
    if (D <= kMaxInRegisters) return vectors ? backward_parts(T, D) * 2 * pitch_of(D) * 4 : 0;
    return (ceil_div(T, long_slab(T)) * 2 * pitch_of(D) + 2 * T) * 4;
}

hipError_t launch_layer_norm_backward(const NormArgs& a, void* ws) {
    return with_types(a.dtype, a.w_dtype, [&](auto t, auto w) {
        if (a.T > 0) return backward<decltype(t), decltype(w)>(a, ws);
        // no rows: dw = db = 0
        using W = decltype(w);
        norm_join_kernel<W><<<dim3(static_cast<unsigned>(ceil_div(a.D, kWave)), 2),
                              dim3(kJoin * kWave), 0, a.stream>>>(
            0, a.D, nullptr, 0, static_cast<W*>(a.dW), static_cast<W*>(a.dB));
        return hipGetLastError();
    });
}

}  // namespace migemm
