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
// written once.  A row lives in the registers of LANES lanes (16 to 1024), 16 elements each.
// 16384 x 8192 BF16: 97 to 119 us forwards (5.5 to 4.5 TB/s), 136 to 149 backwards and 7 for the
// join of 512 partial sums (5.7 to 5.2 TB/s); 8191 x 771 FP32, which the last-level cache holds,
// 10, 14 and 4.  Forms are 512, 1024, 2048 ... columns wide, and the lanes past a row's end load
// and store its last chunk again: 2468 x 2624 FP32, in 4096, takes 12, 16 and 5 us, 1.6 times its
// bytes' time.
#include "rows.hpp"
#include "training.hpp"

namespace migemm {
namespace {

constexpr int kLongThreads = 1024;  // a row that no register form holds
constexpr int kColumns = 8;         // its columns per work-item, backwards
constexpr int64_t kMaxInRegisters = 16384;  // (and longer ones are those)
// Work-items of the workgroups that are given rows to walk: four or five wavefronts a SIMD
// are what the registers leave room for.
constexpr int64_t kResident = 256 * 1024;
// Past this many bytes of x, dy and dx, backwards, x and dy are read past the caches, whose
// last level (256 MiB) holds too little of them for the next reader.
constexpr double kOnceBytes = 256 << 20;

template <int LANES> constexpr int kThreads = LANES <= kWave ? 256 : LANES;
template <int LANES> constexpr int kRows = kThreads<LANES> / LANES;
template <int LANES> constexpr int kWaves = LANES <= kWave ? 1 : LANES / kWave;

// Sums of N values over a row's lanes (the workgroup, or LANES of it with an `lds` of their
// own), in every one of them.  `lds` is free again once
// the row's work-items have passed the barrier of the call after this one.
template <int LANES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (&lds)[N][kWaves<LANES>]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = sum_lanes<LANES <= kWave ? LANES : kWave>(v[i]);
    if constexpr (LANES > kWave) {
        if (threadIdx.x % kWave == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds[i][threadIdx.x % LANES / kWave] = v[i];
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

// A lane's pieces of a row of D: CH chunks of C elements, LANES chunks apart.
template <int C, int LANES, int CH> struct Pieces {
    int at[CH], skip[CH];
    __device__ __forceinline__ Pieces(int D, int lane) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const Span<C> s((c * LANES + lane) * C, D);
            at[c] = static_cast<int>(s.at);
            skip[c] = s.skip;
        }
    }
    template <bool ONCE = false, typename E>
    __device__ __forceinline__ void load(const E* row, E (&e)[CH][C]) const {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if constexpr (ONCE)
                load_once(row + at[c], e[c]);
            else
                load_whole(row + at[c], e[c]);
        }
    }
    template <typename E>
    __device__ __forceinline__ void store(E* row, const E (&e)[CH][C]) const {
#pragma unroll
        for (int c = 0; c < CH; ++c) store_whole(row + at[c], e[c]);
    }
};

// Forwards.  A workgroup walks rows a grid apart, the next row's loads in flight while one
// is summed; weight and bias stay in registers.  (The last row is loaded once more in place
// of one past it: loads and the result's stores are under no branch, or the compiler would
// wait for all stores before the next row.)
template <typename T, typename W, int C, int LANES, int CH>
__global__ __launch_bounds__(kThreads<LANES>) void norm_kernel(
    int64_t rows, int D, const T* __restrict__ X, int64_t ldx, const W* __restrict__ weight,
    const W* __restrict__ bias, float eps, T* __restrict__ Y, int64_t ldy,
    float* __restrict__ means, float* __restrict__ rstds) {
    __shared__ float lds[2][1][kWaves<LANES>];
    const int lane = threadIdx.x % LANES;
    const Pieces<C, LANES, CH> piece(D, lane);
    const float d = static_cast<float>(D);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows<LANES>;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows<LANES> + threadIdx.x / LANES;
    T x[CH][C];
    W w[CH][C], b[CH][C];
    piece.load(X + (row < rows ? row : 0) * ldx, x);
    if (weight) piece.load(weight, w);
    if (bias) piece.load(bias, b);
    for (; row < rows; row += step) {
        const int64_t next = row + step < rows ? row + step : row;
        float v[CH][C], sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[c][i] = to_f32(x[c][i]);
                sum[0] += i >= piece.skip[c] ? v[c][i] : 0.0f;
            }
        piece.load(X + next * ldx, x);
        row_sums<LANES>(sum, lds[0]);
        const float mean = sum[0] / d;
        sum[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[c][i] -= mean;
                sum[0] += i >= piece.skip[c] ? v[c][i] * v[c][i] : 0.0f;
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
        if (lane == 0) {
            if (means) means[row] = mean;
            if (rstds) rstds[row] = rstd;
        }
        piece.store(Y + row * ldy, y);
    }
}

// The same for rows of any length: three passes, the later ones from the caches (1024 x
// 60000 BF16 84 to 91 us, 2.9 to 2.7 TB/s; its bytes alone take 48).
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
        for (int64_t k = 0; k < D; k += kLongThreads * C) {
            const Span<C> piece(k + threadIdx.x * C, D);
            T e[C];
            piece.load(x, e);
#pragma unroll
            for (int i = 0; i < C; ++i) sum[0] += i >= piece.skip ? to_f32(e[i]) : 0.0f;
        }
        row_sums<kLongThreads>(sum, lds[0]);
        const float mean = sum[0] / d;
        sum[0] = 0.0f;
        for (int64_t k = 0; k < D; k += kLongThreads * C) {
            const Span<C> piece(k + threadIdx.x * C, D);
            T e[C];
            piece.load(x, e);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float v = to_f32(e[i]) - mean;
                sum[0] += i >= piece.skip ? v * v : 0.0f;
            }
        }
        row_sums<kLongThreads>(sum, lds[1]);
        const float rstd = 1.0f / sqrtf(sum[0] / d + eps);
        for (int64_t k = 0; k < D; k += kLongThreads * C) {
            const Span<C> piece(k + threadIdx.x * C, D);
            T e[C];
            W w[C], b[C];
            piece.load(x, e);
            if (weight) piece.load(weight, w);
            if (bias) piece.load(bias, b);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float o = (to_f32(e[i]) - mean) * rstd;
                if (weight) o *= to_f32(w[i]);
                if (bias) o += to_f32(b[i]);
                e[i] = narrow<T>(o);
            }
            piece.store(Y + row * ldy, e);
        }
        if (threadIdx.x == 0) {
            if (means) means[row] = mean;
            if (rstds) rstds[row] = rstd;
        }
    }
}

// Backwards.  A workgroup walks rows a grid apart, the next row's loads in flight while a
// row is summed; each lane keeps dw and db of its columns in registers, and the workgroup
// writes one partial sum of each, which norm_join_kernel adds.  Rows stay in registers as
// they were loaded, and h and g are formed twice: kept in FP32 they left one workgroup less
// to a CU.  The form of 1024 lanes has 128 registers a lane: FP32 rows leave no room there for
// the next one's, and 16-bit ones with sums and dx spill 2 to 4 (17, 48 bytes of scratch a
// lane, with BF16 weights past the caches; 8192 x 12000 BF16 140 us, 4.2 TB/s).  The last
// row's loads are repeated in place of one past it: with ONCE from memory, a row of x and dy
// for each workgroup (16384 x 8192 BF16 17 MB beside 537).  SUMS: dw or db is wanted; ROWS:
// dx is; ONCE: x and dy are read past the caches.
template <typename T, typename W, int C, int LANES, int CH, bool SUMS, bool ROWS, bool ONCE>
__global__ __launch_bounds__(kThreads<LANES>) void norm_backward_kernel(
    int64_t rows, int D, const T* __restrict__ dY, int64_t lddy, const T* __restrict__ X,
    int64_t ldx, const W* __restrict__ weight, const float* __restrict__ means,
    const float* __restrict__ rstds, T* __restrict__ dX, int64_t lddx,
    float* __restrict__ partial, int64_t pitch) {
    constexpr int R = kRows<LANES>;
    constexpr bool AHEAD = !(LANES == 1024 && sizeof(T) == 4);
    __shared__ float lds[2][2][kWaves<LANES>];
    const int lane = threadIdx.x % LANES, part = threadIdx.x / LANES;
    const Pieces<C, LANES, CH> piece(D, lane);
    const float d = static_cast<float>(D);
    const int64_t step = static_cast<int64_t>(gridDim.x) * R;
    int64_t row = static_cast<int64_t>(blockIdx.x) * R + part;
    struct Row {
        T x[CH][C], dy[CH][C];
        float mean, rstd;
    };
    auto load = [&](int64_t r, Row& t) __attribute__((always_inline)) {
        piece.template load<ONCE>(X + r * ldx, t.x);
        piece.template load<ONCE>(dY + r * lddy, t.dy);
        t.mean = means[r];
        t.rstd = rstds[r];
    };
    Row now;
    if constexpr (AHEAD) load(row < rows ? row : 0, now);
    W w[CH][C];
    if (weight) {
        piece.load(weight, w);
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) w[c][i] = narrow<W>(1.0f);
    }
    float dw[CH][C], db[CH][C];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < C; ++i) dw[c][i] = db[c][i] = 0.0f;
    for (int turn = 0; row < rows; row += step, turn ^= 1) {
        Row next;
        if constexpr (AHEAD)
            load(row + step < rows ? row + step : row, next);
        else
            load(row, now);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float o = to_f32(now.dy[c][i]);
                const float h = (to_f32(now.x[c][i]) - now.mean) * now.rstd;
                const float g = o * to_f32(w[c][i]);
                if (i >= piece.skip[c]) {
                    sum[0] += g;
                    sum[1] += g * h;
                }
                if constexpr (SUMS) {
                    dw[c][i] += o * h;
                    db[c][i] += o;
                }
            }
        if constexpr (ROWS) {
            row_sums<LANES>(sum, lds[turn]);
            const float a = sum[0] / d, b = sum[1] / d;
            T o[CH][C];
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const float h = (to_f32(now.x[c][i]) - now.mean) * now.rstd;
                    const float g = to_f32(now.dy[c][i]) * to_f32(w[c][i]);
                    o[c][i] = narrow<T>(now.rstd * (g - a - h * b));
                }
            piece.store(dX + row * lddx, o);
        }
        if constexpr (AHEAD) now = next;
    }
    if constexpr (SUMS) {
        float* const out = partial + static_cast<int64_t>(blockIdx.x) * 2 * pitch;
        if constexpr (R == 1) {
            piece.store(out, dw);
            piece.store(out + pitch, db);
        } else {
            // the workgroup's rows are joined in order, dw first
            constexpr int kWidth = LANES * CH * C;
            __shared__ __attribute__((aligned(16))) float rows_of[R][kWidth];
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                if (which) __syncthreads();
                if (which)
                    piece.store(rows_of[part], db);
                else
                    piece.store(rows_of[part], dw);
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

// Few rows, backwards, in one launch: dw and db need no sums over a row, only what the forward
// pass left.  The first workgroups take rows, one to LANES lanes; those behind them a band of
// 128 bytes of columns each, eight lanes to a row, and join their rows' sums in order.  x and
// dy are read twice, the second time from the caches.  On the same rows over and over, against
// partial sums and their join: 76 x 1032 FP16 3.5 us instead of 6.4, 1003 7.5 instead of 10.5,
// 512 x 8192 BF16 8.2 instead of 15.1 (1003 x 1032 after the forward pass 8.8, 512 x 8192
// 8.9); past kFewRows rows a band's workgroup is at work too long (2048 x 1032 14.9 instead of
// 12.8), past kFewBytes of x the second reading costs more than a launch (1024 x 3000 FP32 13.7
// instead of 11.4).
constexpr int64_t kFewRows = 1024, kFewBytes = 8 << 20;
bool few_rows(int64_t T, int64_t D, int bytes) {
    return T <= kFewRows && D <= kMaxInRegisters && T * D * bytes <= kFewBytes;
}
template <int LANES> constexpr int kFewThreads = LANES <= 512 ? 512 : LANES;
constexpr int kBandLanes = 8;
// Rows in flight in a band.  What decides is how many rows there are, 512 work-items having 64
// lane groups: FP16, with 8 and with 4, 1003 x 1032 7.5 and 8.7 us, 512 x 1032 4.6 and 5.0, 256
// x 1032 4.0 and 3.7, 100 x 1032 3.7 and 3.3.  The rule goes by the row's form instead, since
// one kernel holds both: it is right for the forms of 1024 lanes (256 x 16384 10.1 and 8.1) and
// 512 (512 x 8192 9.6 and 9.6, 512 x 6144 7.9 and 8.8, 100 x 8192 3.9 and 3.5) and for rows up to
// 2048 columns past 400 of them; in the form of 256 lanes it gains 0.3 us on few rows (100 x
// 4096 3.4 instead of 3.8) and loses up to 2.3 on many (1024 x 4096 12.8 instead of 10.5).
template <int LANES> constexpr int kBandAhead = LANES <= 128 ? 8 : 4;
template <typename T, typename W, int C, int LANES, int CH>
__global__ __launch_bounds__(kFewThreads<LANES>) void norm_few_kernel(
    int rows, int D, const T* __restrict__ dY, int64_t lddy, const T* __restrict__ X, int64_t ldx,
    const W* __restrict__ weight, const float* __restrict__ means,
    const float* __restrict__ rstds, T* __restrict__ dX, int64_t lddx, W* __restrict__ dW,
    W* __restrict__ dB, int row_groups) {
    constexpr int THREADS = kFewThreads<LANES>;
    if (static_cast<int>(blockIdx.x) < row_groups) {
        constexpr int R = THREADS / LANES;
        __shared__ float lds[R][2][kWaves<LANES>];
        const int lane = threadIdx.x % LANES, part = threadIdx.x / LANES;
        const Pieces<C, LANES, CH> piece(D, lane);
        // (past the last row that one again, whose result comes out as the same bits)
        const int64_t at = static_cast<int64_t>(blockIdx.x) * R + part;
        const int64_t row = at < rows ? at : rows - 1;
        T x[CH][C], dy[CH][C];
        W w[CH][C];
        piece.load(X + row * ldx, x);
        piece.load(dY + row * lddy, dy);
        if (weight) piece.load(weight, w);
        const float mean = means[row], rstd = rstds[row], d = static_cast<float>(D);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (!weight) w[c][i] = narrow<W>(1.0f);
                const float h = (to_f32(x[c][i]) - mean) * rstd;
                const float g = to_f32(dy[c][i]) * to_f32(w[c][i]);
                if (i >= piece.skip[c]) {
                    sum[0] += g;
                    sum[1] += g * h;
                }
            }
        row_sums<LANES>(sum, lds[part]);
        const float a = sum[0] / d, b = sum[1] / d;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float h = (to_f32(x[c][i]) - mean) * rstd;
                const float g = to_f32(dy[c][i]) * to_f32(w[c][i]);
                x[c][i] = narrow<T>(rstd * (g - a - h * b));
            }
        piece.store(dX + row * lddx, x);
        return;
    }
    constexpr int kBand = kBandLanes * C, kGroups = THREADS / kBandLanes;
    constexpr int AHEAD = kBandAhead<LANES>;
    __shared__ float lds[2][kGroups / 2][kBand + 1];
    const int first = (blockIdx.x - row_groups) * kBand, lane = threadIdx.x % kBandLanes;
    const Span<C> piece(first + lane * C, D);
    float dw[C], db[C];
#pragma unroll
    for (int i = 0; i < C; ++i) dw[i] = db[i] = 0.0f;
    for (int row = threadIdx.x / kBandLanes; row < rows; row += kGroups * AHEAD) {
        T x[AHEAD][C], dy[AHEAD][C];
        float mean[AHEAD], rstd[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t r = row + u * kGroups < rows ? row + u * kGroups : rows - 1;
            piece.load(X + r * ldx, x[u]);
            piece.load(dY + r * lddy, dy[u]);
            mean[u] = means[r];
            rstd[u] = rstds[r];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (row + u * kGroups < rows) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const float o = to_f32(dy[u][i]);
                    dw[i] += o * ((to_f32(x[u][i]) - mean[u]) * rstd[u]);
                    db[i] += o;
                }
            }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        dw[i] += row_rotated<8>(dw[i]);  // (the other row of the 16 lanes)
        db[i] += row_rotated<8>(db[i]);
        if (threadIdx.x % 16 < kBandLanes && i >= piece.skip) {
            lds[0][threadIdx.x / 16][piece.at + i - first] = dw[i];
            lds[1][threadIdx.x / 16][piece.at + i - first] = db[i];
        }
    }
    __syncthreads();
    const int which = threadIdx.x / kBand, k = threadIdx.x % kBand;
    W* const out = which ? dB : dW;
    if (which > 1 || first + k >= D || !out) return;
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups / 2; ++g) s += lds[which][g][k];
    out[first + k] = narrow<W>(s);
}

// Rows too long for registers, backwards (1024 x 60000 BF16 117 to 127 us: 43, 67 and 7 for
// the join; its bytes alone take 72): first the two sums of each row,
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
        for (int64_t k = 0; k < D; k += kLongThreads * C) {
            const Span<C> piece(k + threadIdx.x * C, D);
            T x[C], dy[C];
            W w[C];
            piece.load(X + row * ldx, x);
            piece.load(dY + row * lddy, dy);
            if (weight) piece.load(weight, w);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float g = to_f32(dy[i]);
                if (weight) g *= to_f32(w[i]);
                if (i >= piece.skip) {
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
    const Span<N> piece(k, D);
    const float d = static_cast<float>(D);
    W w[N];
    float dw[N], db[N];
    if (weight) piece.load(weight, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (!weight) w[i] = narrow<W>(1.0f);
        dw[i] = db[i] = 0.0f;
    }
    const int64_t end = (p + 1) * slab < rows ? (p + 1) * slab : rows;
#pragma unroll 2
    for (int64_t row = p * slab; row < end; ++row) {
        T x[N], dy[N];
        piece.load(X + row * ldx, x);
        piece.load(dY + row * lddy, dy);
        const float mean = means[row], rstd = rstds[row];
        const float a = sums[2 * row] / d, b = sums[2 * row + 1] / d;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float o = to_f32(dy[i]), h = (to_f32(x[i]) - mean) * rstd;
            dw[i] += o * h;
            db[i] += o;
            x[i] = narrow<T>(rstd * (o * to_f32(w[i]) - a - h * b));
        }
        if (dX) piece.store(dX + row * lddx, x);
    }
    float* const out = partial + p * 2 * pitch;
    piece.store(out, dw);
    piece.store(out + pitch, db);
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

// How a row of D lies in registers: C elements a chunk, lanes, and chunks of each.  16
// elements a lane: more leave too few wavefronts in flight backwards, where five values a
// column are held.  Rows shorter than a chunk take one element a lane.
template <typename T, typename F> hipError_t with_form(int64_t D, F f) {
    using std::integral_constant;
    auto form = [&](auto lanes, auto elements) {
        constexpr int C = kChunk<T>;
        return f(integral_constant<int, C>{}, lanes,
                 integral_constant<int, decltype(elements)::value / C>{});
    };
    using e8 = integral_constant<int, 8>;
    using e16 = integral_constant<int, 16>;
    if (D < kChunk<T>)
        return f(integral_constant<int, 1>{}, integral_constant<int, 16>{},
                 integral_constant<int, 1>{});
    if (D <= 128) return form(integral_constant<int, 16>{}, e8{});
    if (D <= 512) return form(integral_constant<int, 64>{}, e8{});
    if (D <= 1024) return form(integral_constant<int, 64>{}, e16{});
    if (D <= 2048) return form(integral_constant<int, 128>{}, e16{});
    if (D <= 4096) return form(integral_constant<int, 256>{}, e16{});
    if (D <= 8192) return form(integral_constant<int, 512>{}, e16{});
    return form(integral_constant<int, 1024>{}, e16{});
}

// Rows, and work-items, of a workgroup of that form.
int rows_of_form(int64_t D) { return D <= 128 ? 16 : D <= 1024 ? 4 : 1; }
int threads_of_form(int64_t D) {
    return D <= 1024 ? 256 : D <= 2048 ? 128 : D <= 4096 ? 256 : D <= 8192 ? 512 : 1024;
}

// Workgroups for `groups` of rows, `most` at a time, each with as many as the others.
int64_t even_groups(int64_t groups, int64_t most) {
    return ceil_div(groups, ceil_div(groups, most));
}

template <typename T, typename W> hipError_t forward(const NormArgs& a) {
    const T* const x = static_cast<const T*>(a.X);
    const W *const w = static_cast<const W*>(a.W), *const b = static_cast<const W*>(a.B);
    T* const y = static_cast<T*>(a.Y);
    if (a.D > kMaxInRegisters) {
        const int64_t most = int64_t(1) << 20;  // workgroups; they stride over the rest
        norm_long_kernel<T, W><<<dim3(static_cast<unsigned>(a.T < most ? a.T : most)),
                                 dim3(kLongThreads), 0, a.stream>>>(
            a.T, a.D, x, a.ldx, w, b, a.eps, y, a.ldy, a.mean, a.rstd);
        return hipGetLastError();
    }
    return with_form<T>(a.D, [&](auto chunk, auto lanes, auto chunks) {
        constexpr int C = decltype(chunk)::value, L = decltype(lanes)::value,
                      CH = decltype(chunks)::value;
        const int64_t blocks = even_groups(ceil_div(a.T, kRows<L>), kResident / kThreads<L>);
        norm_kernel<T, W, C, L, CH><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads<L>), 0,
                                      a.stream>>>(a.T, static_cast<int>(a.D), x, a.ldx, w, b,
                                                  a.eps, y, a.ldy, a.mean, a.rstd);
        return hipGetLastError();
    });
}

// Workgroups of the backward pass, each of which writes partial sums.
int64_t backward_parts(int64_t T, int64_t D) {
    const int64_t groups = ceil_div(T, rows_of_form(D));
    int64_t most = kResident / threads_of_form(D);
    if (most > 512) most = 512;
    // four rows to a partial sum at least, two where there are few
    const int64_t parts = ceil_div(groups, groups <= 256 ? 2 : 4);
    return even_groups(groups, parts < most ? parts : most);
}
int64_t long_slab(int64_t T) { return ceil_div(T, T < 64 * 32 ? ceil_div(T, 32) : 64); }
int64_t pitch_of(int64_t D) { return ceil_div(D, 64) * 64; }

template <typename T, typename W> hipError_t backward(const NormArgs& a, void* ws) {
    const T *const x = static_cast<const T*>(a.X), *const dy = static_cast<const T*>(a.dY);
    const W* const w = static_cast<const W*>(a.W);
    T* const dx = static_cast<T*>(a.Y);
    float* partial = static_cast<float*>(ws);
    const int64_t pitch = pitch_of(a.D);
    const bool few = (a.dW || a.dB) && few_rows(a.T, a.D, sizeof(T));
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
        const bool once = 3.0 * sizeof(T) * a.T * a.D > kOnceBytes;
        using yes = std::true_type;
        using no = std::false_type;
        err = with_form<T>(a.D, [&](auto chunk, auto lanes, auto chunks) {
            constexpr int C = decltype(chunk)::value, L = decltype(lanes)::value,
                          CH = decltype(chunks)::value;
            auto go = [&](auto want, auto to_x, auto past) {
                norm_backward_kernel<T, W, C, L, CH, decltype(want)::value, decltype(to_x)::value,
                                     decltype(past)::value>
                    <<<dim3(static_cast<unsigned>(parts)), dim3(kThreads<L>), 0, a.stream>>>(
                        a.T, static_cast<int>(a.D), dy, a.lddy, x, a.ldx, w, a.mean, a.rstd, dx,
                        a.ldy, partial, pitch);
                return hipGetLastError();
            };
            if (few) {
                constexpr int R = kFewThreads<L> / L, B = kBandLanes * C;
                const int groups = dx ? static_cast<int>(ceil_div(a.T, R)) : 0;
                norm_few_kernel<T, W, C, L, CH>
                    <<<dim3(static_cast<unsigned>(groups + ceil_div(a.D, B))),
                       dim3(kFewThreads<L>), 0, a.stream>>>(
                        static_cast<int>(a.T), static_cast<int>(a.D), dy, a.lddy, x, a.ldx, w,
                        a.mean, a.rstd, dx, a.ldy, static_cast<W*>(a.dW), static_cast<W*>(a.dB),
                        groups);
                return hipGetLastError();
            }
            if (sums) {
                parts = backward_parts(a.T, a.D);
                if (!dx) return go(yes{}, no{}, no{});
                return once ? go(yes{}, yes{}, yes{}) : go(yes{}, yes{}, no{});
            }
            parts = even_groups(ceil_div(a.T, kRows<L>), kResident / kThreads<L>);
            return go(no{}, yes{}, no{});
        });
    }
    if (err != hipSuccess || (!a.dW && !a.dB) || few) return err;
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
    // (enough for every type: FP32 rows are few sooner)
    if (T == 0 || few_rows(T, D, 4)) return 0;
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
