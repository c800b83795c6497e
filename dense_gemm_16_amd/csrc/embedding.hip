// embedding.hip -- rows of a table by token, and the table's gradient.
//
// Forwards y[t] = scale w[index[t]]; a token of the ignored index has a row of zeros,
// one outside the table NaN.  Backwards dw[v] = scale sum of dy[t] over the tokens t of
// entry v (+ what was there).
//
// The gradient's sums are FP32, in the order of the tokens, with no atomics.  The tokens
// are sorted by entry (stable, so that each entry's tokens keep their order); the sorted
// list is cut into stretches of equal length, whatever entries they hold, so that an entry
// that a tenth of all tokens name is summed by as many wavefronts as its tokens need;
// what a stretch holds of an entry that it shares with its neighbours goes to the
// workspace as one FP32 row, and a last kernel adds those.
//
// Bound by memory: dy is read once, a row of dw written once (read too where it is added
// to).  Rows of dw that no token names are zeroed by workgroups of the same launch, and
// not touched where the gradient is added.
#include "rows.hpp"
#include "training.hpp"

namespace migemm {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- forwards

// `lpr` lanes (a power of two) take a segment of kUnroll chunks a lane of one row; the
// loads of all of them are in flight together.
constexpr int kUnroll = 4;
template <typename T>
__global__ __launch_bounds__(kThreads) void gather_kernel(
    int64_t T_, int64_t V, int64_t D, const T* __restrict__ W, int64_t ldw,
    const int64_t* __restrict__ index, int64_t ignore, float scale, T* __restrict__ Y,
    int64_t ldy, int lpr, int64_t segs, int64_t groups) {
    constexpr int C = kChunk<T>;
    const int rows = kThreads / lpr, lane = threadIdx.x % lpr;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        const int64_t t = g / segs * rows + threadIdx.x / lpr;
        if (t >= T_) continue;
        const int64_t k0 = (g % segs * kUnroll * lpr + lane) * C, v = index[t];
        T* const to = Y + t * ldy;
        if (v != ignore && v >= 0 && v < V) {
            const T* const from = W + v * ldw;
            T e[kUnroll][C];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t k = k0 + static_cast<int64_t>(u) * lpr * C;
                load_part(from + k, D - k, e[u]);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t k = k0 + static_cast<int64_t>(u) * lpr * C;
#pragma unroll
                for (int i = 0; i < C; ++i) e[u][i] = narrow<T>(scale * to_f32(e[u][i]));
                store_part(to + k, D - k, e[u]);
            }
        } else {
            T e[C];
#pragma unroll
            for (int i = 0; i < C; ++i)
                e[i] = narrow<T>(v == ignore ? 0.0f : __builtin_nanf(""));
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t k = k0 + static_cast<int64_t>(u) * lpr * C;
                store_part(to + k, D - k, e);
            }
        }
    }
}

// -------------------------------------------------------------------- sorting

// A stable sort of (entry, token) pairs by entry, kDigit bits at a time, the lowest first.
// Tokens without an entry (ignored, or outside the table) sort last, as entry V.
constexpr int kDigit = 9, kBins = 1 << kDigit;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kTile = 4096;            // pairs of a workgroup where several share a pass
constexpr int kTileEach = kTile / kSortThreads;

__device__ __forceinline__ uint32_t entry_of(const int64_t* index, int64_t t, int64_t ignore,
                                             int64_t V) {
    const int64_t v = index[t];
    return static_cast<uint32_t>(v != ignore && v >= 0 && v < V ? v : V);
}

// The lanes of the wavefront whose digit equals this lane's, among those that hold one.
__device__ __forceinline__ uint64_t peers(uint32_t digit, bool held) {
    uint64_t same = __ballot(held);
#pragma unroll
    for (int b = 0; b < kDigit; ++b) {
        const uint64_t ones = __ballot((digit >> b) & 1u);
        same &= (digit >> b) & 1u ? ones : ~ones;
    }
    return same;
}

// Ranks within one wavefront's consecutive 64 pairs after `count[digit]` earlier ones, and
// the count brought up to date.  Wavefronts have counts of their own.
template <typename N>
__device__ __forceinline__ uint32_t rank_of(uint32_t digit, bool held, N* count) {
    const uint64_t same = peers(digit, held);
    const int lane = threadIdx.x % kWave;
    const uint64_t below = same & ((uint64_t(1) << lane) - 1);
    uint32_t before = 0;
    if (held) before = count[digit];
    // the lanes' reads come before the write, and that before the next call's reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (held && below == 0) count[digit] = static_cast<N>(before + __popcll(same));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return before + static_cast<uint32_t>(__popcll(below));
}

// Exclusive sums, in place, over count[wave][digit] in the order digit by digit, wavefront
// by wavefront within a digit.
__device__ __forceinline__ void scan_counts(uint16_t (&count)[kSortWaves][kBins],
                                            uint32_t* wave_sum) {
    // work-item i < kBins owns digit i
    const int i = threadIdx.x;
    uint32_t mine = 0;
    if (i < kBins) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = count[w][i];
            count[w][i] = static_cast<uint16_t>(mine);
            mine += c;
        }
    }
    uint32_t up = mine;
    const int lane = i % kWave;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = __shfl_up(up, d);
        if (lane >= d) up += o;
    }
    if (lane == kWave - 1) wave_sum[i / kWave] = up;
    __syncthreads();
    if (i < kBins) {
        uint32_t before = up - mine;
        for (int w = 0; w < i / kWave; ++w) before += wave_sum[w];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w)
            count[w][i] = static_cast<uint16_t>(count[w][i] + before);
    }
    __syncthreads();
}

// Up to kSortOne pairs by one workgroup, in LDS: a pair is its token and what is left of
// its entry after the digits sorted so far.  The first digit comes straight from the
// index, so 16 bits of token and 32 - 16 further bits of entry make up a word: V below 2^25.
constexpr int kOneEach = 32, kSortOne = kOneEach * kSortThreads;
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(
    int T_, int64_t V, const int64_t* __restrict__ index, int64_t ignore, int passes,
    uint32_t* __restrict__ keys, uint32_t* __restrict__ tokens) {
    __shared__ uint32_t held[kSortOne];
    __shared__ uint16_t count[kSortWaves][kBins];  // (32-bit ones would not fit beside `held`)
    __shared__ uint32_t wave_sum[kSortWaves];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    // a wavefront owns `each` consecutive groups of 64 pairs
    const int each = (T_ + kSortThreads - 1) / kSortThreads;
    const int first = wave * each * kWave + lane;
    for (int pass = 0; pass < passes; ++pass) {
        for (int i = threadIdx.x; i < kSortWaves * kBins; i += kSortThreads)
            (&count[0][0])[i] = 0;
        __syncthreads();
        uint32_t word[kOneEach];
        uint32_t rank[kOneEach];  // the digit above 16 bits of rank
#pragma unroll
        for (int i = 0; i < kOneEach; ++i) {
            const int at = first + i * kWave;
            if (i >= each) break;
            const bool in = at < T_;
            uint32_t digit = 0;
            word[i] = 0;
            if (in) {
                if (pass == 0) {
                    const uint32_t e = entry_of(index, at, ignore, V);
                    digit = e & (kBins - 1);
                    word[i] = (e >> kDigit) << 16 | static_cast<uint32_t>(at);
                } else {
                    const uint32_t w = held[at];
                    digit = (w >> 16) & (kBins - 1);
                    word[i] = (w >> 16 >> kDigit) << 16 | (w & 0xffffu);
                }
            }
            rank[i] = digit << 16 | rank_of(digit, in, count[wave]);
        }
        __syncthreads();
        scan_counts(count, wave_sum);
#pragma unroll
        for (int i = 0; i < kOneEach; ++i) {
            const int at = first + i * kWave;
            if (i >= each) break;
            if (at >= T_) continue;
            const uint32_t to = count[wave][rank[i] >> 16] + (rank[i] & 0xffffu);
            if (pass + 1 < passes) {
                held[to] = word[i];
            } else {
                const uint32_t t = word[i] & 0xffffu;
                tokens[to] = t;
                keys[to] = entry_of(index, t, ignore, V);
            }
        }
        __syncthreads();
    }
}

// More pairs: each pass counts the digits of every tile, sums the counts over digits and
// tiles, and moves the pairs.  The first pass reads the index.
struct Pairs {
    const int64_t* index;  // the first pass's source, NULL afterwards
    int64_t ignore, V;
    const uint32_t *keys, *tokens;
    __device__ __forceinline__ uint32_t key(int64_t i) const {
        return index ? entry_of(index, i, ignore, V) : keys[i];
    }
    __device__ __forceinline__ uint32_t token(int64_t i) const {
        return index ? static_cast<uint32_t>(i) : tokens[i];
    }
};

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(int64_t T_, Pairs from,
                                                                  int shift, int64_t tiles,
                                                                  uint32_t* __restrict__ counts) {
    __shared__ uint32_t bins[kBins];
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        if (threadIdx.x < kBins) bins[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTileEach; ++i) {
            const int64_t at = tile * kTile + i * kSortThreads + threadIdx.x;
            // counts alone: their order does not matter
            if (at < T_) atomicAdd(&bins[(from.key(at) >> shift) & (kBins - 1)], 1u);
        }
        __syncthreads();
        if (threadIdx.x < kBins) counts[threadIdx.x * tiles + tile] = bins[threadIdx.x];
        __syncthreads();
    }
}

// Exclusive sums of n values in place, by one workgroup.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(int64_t n,
                                                                 uint32_t* __restrict__ counts) {
    constexpr int kEach = 8;
    __shared__ uint32_t wave_sum[2][kSortWaves];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    uint32_t before = 0;
    int turn = 0;
    for (int64_t base = 0; base < n; base += kSortThreads * kEach, turn ^= 1) {
        const int64_t at = base + threadIdx.x * kEach;
        uint32_t c[kEach], mine = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const uint32_t v = at + i < n ? counts[at + i] : 0;
            c[i] = mine;
            mine += v;
        }
        uint32_t up = mine;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const uint32_t o = __shfl_up(up, d);
            if (lane >= d) up += o;
        }
        if (lane == kWave - 1) wave_sum[turn][wave] = up;
        __syncthreads();
        uint32_t mybase = before + up - mine;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) mybase += wave_sum[turn][w];
            before += wave_sum[turn][w];
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (at + i < n) counts[at + i] = mybase + c[i];
    }
}

__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(
    int64_t T_, Pairs from, int shift, int64_t tiles, const uint32_t* __restrict__ offsets,
    uint32_t* __restrict__ keys, uint32_t* __restrict__ tokens) {
    __shared__ uint32_t count[kSortWaves][kBins];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        for (int i = threadIdx.x; i < kSortWaves * kBins; i += kSortThreads)
            (&count[0][0])[i] = 0;
        __syncthreads();
        const int64_t first = tile * kTile + wave * kTileEach * kWave + lane;
        uint32_t key[kTileEach], rank[kTileEach];
#pragma unroll
        for (int i = 0; i < kTileEach; ++i) {
            const int64_t at = first + i * kWave;
            key[i] = at < T_ ? from.key(at) : 0;
            rank[i] = rank_of((key[i] >> shift) & (kBins - 1), at < T_, count[wave]);
        }
        __syncthreads();
        // each digit's place in the whole list, then wavefront by wavefront
        if (threadIdx.x < kBins) {
            uint32_t at = offsets[threadIdx.x * tiles + tile];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = count[w][threadIdx.x];
                count[w][threadIdx.x] = at;
                at += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTileEach; ++i) {
            const int64_t at = first + i * kWave;
            if (at >= T_) continue;
            const uint32_t to = count[wave][(key[i] >> shift) & (kBins - 1)] + rank[i];
            keys[to] = key[i];
            tokens[to] = from.token(at);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------- sums

struct GradArgs {
    int64_t T, V, D;
    const uint32_t *keys, *tokens;  // sorted
    int64_t ldy, ldw;
    float scale;
    bool accumulate;
    int stretch;        // pairs of a stretch
    int64_t stretches, pitch;
    float* shared_rows;  // two rows of `pitch` a stretch: of an entry begun before it, of
                         // one that goes on after it
    int lpr;             // lanes of a segment of a row, a power of two up to 64
    int64_t segs;        // segments of a row: 16 bytes of dy a lane each
    int64_t zero_groups; // workgroups that zero rows
};

// Adds scale times a sum to, or puts it into, a piece of dw.
template <typename W, int C>
__device__ __forceinline__ void put(W* to, int64_t held, const float (&sum)[C], float scale,
                                    bool accumulate) {
    W e[C];
    if (accumulate) {
        load_part(to, held, e);
#pragma unroll
        for (int i = 0; i < C; ++i) e[i] = narrow<W>(fmaf(scale, sum[i], to_f32(e[i])));
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) e[i] = narrow<W>(scale * sum[i]);
    }
    store_part(to, held, e);
}

// Zeros the rows of entries v0 .. v0 + kZeroRows - 1 that no token names, by one
// wavefront: its lanes look for one entry each in the sorted list.
constexpr int kZeroRows = 16;
template <typename W>
__device__ __forceinline__ void zero_rows(const GradArgs& a, int64_t v0, W* __restrict__ dW) {
    const int lane = threadIdx.x % kWave;
    const int64_t v = v0 + lane;
    bool absent = false;
    if (lane < kZeroRows && v < a.V) {
        int64_t lo = 0, hi = a.T;
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (a.keys[mid] < v)
                lo = mid + 1;
            else
                hi = mid;
        }
        absent = lo == a.T || a.keys[lo] != v;
    }
    constexpr int C = kChunk<W>;
    W zero[C];
#pragma unroll
    for (int i = 0; i < C; ++i) zero[i] = narrow<W>(0.0f);
    for (uint64_t todo = __ballot(absent); todo; todo &= todo - 1) {
        W* const row = dW + (v0 + __builtin_ctzll(todo)) * a.ldw;
        for (int64_t k = lane * C; k < a.D; k += kWave * C) store_part(row + k, a.D - k, zero);
    }
}

constexpr int kAhead = 8;  // rows of dy in flight
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void scatter_kernel(GradArgs a, const T* __restrict__ dY,
                                                           W* __restrict__ dW) {
    constexpr int C = kChunk<T>;
    if (blockIdx.x < a.zero_groups) {
        const int64_t v0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / kWave) +
                            threadIdx.x / kWave) * kZeroRows;
        if (v0 < a.V) zero_rows(a, v0, dW);
        return;
    }
    const int64_t group = (blockIdx.x - a.zero_groups) * (kThreads / a.lpr) + threadIdx.x / a.lpr;
    const int64_t s = group / a.segs;
    if (s >= a.stretches) return;
    const int64_t k = (group % a.segs * a.lpr + threadIdx.x % a.lpr) * C;
    if (k >= a.D) return;
    const int64_t first = s * a.stretch;
    const int64_t end = first + a.stretch < a.T ? first + a.stretch : a.T;
    const uint32_t none = static_cast<uint32_t>(a.V);
    // the entry that the stretch before ends with: its sum is begun there
    const uint32_t before = first > 0 ? a.keys[first - 1] : none;
    const uint32_t after = end < a.T ? a.keys[end] : none;
    float sum[C];
#pragma unroll
    for (int i = 0; i < C; ++i) sum[i] = 0.0f;
    uint32_t now = a.keys[first];
    bool begun = now == before;
    auto finish = [&](uint32_t v, bool here, bool on) {
        if (v == none) return;
        if (here && !on) {
            put(dW + v * a.ldw + k, a.D - k, sum, a.scale, a.accumulate);
        } else {
            // rows of the workspace have room for whole chunks
            float* const row = a.shared_rows + (2 * s + (here ? 1 : 0)) * a.pitch + k;
            store_whole(row, sum);
        }
    };
    for (int64_t i = first; i < end; i += kAhead) {
        uint32_t key[kAhead];
        T e[kAhead][C];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const bool in = i + u < end;
            key[u] = in ? a.keys[i + u] : none;
            if (in && key[u] != none)
                load_part(dY + a.tokens[i + u] * a.ldy + k, a.D - k, e[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i + u >= end) break;
            if (key[u] != now) {
                finish(now, !begun, false);
                now = key[u];
                begun = false;
#pragma unroll
                for (int c = 0; c < C; ++c) sum[c] = 0.0f;
            }
            if (key[u] != none) {
#pragma unroll
                for (int c = 0; c < C; ++c) sum[c] += to_f32(e[u][c]);
            }
        }
    }
    finish(now, !begun, now == after);
}

// Entries that several stretches share: the stretch where one begins adds up the rows
// that they left.
constexpr int kJoinWaves = 8, kJoinThreads = kJoinWaves * kWave;
template <typename T, typename W>
__global__ __launch_bounds__(kJoinThreads) void scatter_join_kernel(GradArgs a,
                                                                    W* __restrict__ dW) {
    constexpr int C = kChunk<T>;
    __shared__ float lds[kJoinWaves][kWave][C + 1];
    const int64_t s = blockIdx.x;  // (the last stretch shares nothing with a later one)
    const int64_t end = (s + 1) * a.stretch;
    const uint32_t v = a.keys[end - 1];
    // it goes on after this stretch, and begins inside it
    if (v == static_cast<uint32_t>(a.V) || a.keys[end] != v) return;
    const int64_t first = s * a.stretch;
    if (first > 0 && a.keys[first - 1] == v) return;
    // the last stretch that holds it: the entries are sorted
    int64_t lo = s + 1, hi = a.stretches;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (a.keys[mid * a.stretch] == v)
            lo = mid + 1;
        else
            hi = mid;
    }
    const int64_t last = lo - 1;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (int64_t k0 = 0; k0 < a.D; k0 += kWave * C) {
        const int64_t k = k0 + lane * C;
        float sum[C];
#pragma unroll
        for (int c = 0; c < C; ++c) sum[c] = 0.0f;
        if (k < a.D) {
            if (wave == 0) load_whole(a.shared_rows + (2 * s + 1) * a.pitch + k, sum);
#pragma unroll 4
            for (int64_t i = s + 1 + wave; i <= last; i += kJoinWaves) {
                float e[C];
                load_whole(a.shared_rows + 2 * i * a.pitch + k, e);
#pragma unroll
                for (int c = 0; c < C; ++c) sum[c] += e[c];
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) lds[wave][lane][c] = sum[c];
        __syncthreads();
        if (wave == 0 && k < a.D) {
#pragma unroll
            for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
                for (int c = 0; c < C; ++c) sum[c] += lds[w][lane][c];
            put(dW + v * a.ldw + k, a.D - k, sum, a.scale, a.accumulate);
        }
        __syncthreads();
    }
}

// dw of no tokens: zeros.
template <typename W>
__global__ __launch_bounds__(kThreads) void zero_kernel(int64_t V, int64_t D, W* __restrict__ dW,
                                                        int64_t ldw) {
    constexpr int C = kChunk<W>;
    W zero[C];
#pragma unroll
    for (int i = 0; i < C; ++i) zero[i] = narrow<W>(0.0f);
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x)
        for (int64_t k = threadIdx.x * C; k < D; k += kThreads * C)
            store_part(dW + v * ldw + k, D - k, zero);
}

// The workspace: sorted entries and tokens, the other copy of them and the counts where
// the sort takes several workgroups, and the stretches' shared rows.
struct Plan {
    bool one;      // one workgroup sorts
    int passes;
    int64_t tiles, stretches, pitch;
    int stretch;
    int64_t keys, tokens, keys2, tokens2, counts, rows, bytes;  // offsets
};

int64_t aligned(int64_t n) { return ceil_div(n, kWorkspaceAlign) * kWorkspaceAlign; }

Plan make_plan(int64_t T, int64_t V, int64_t D) {
    Plan p{};
    int bits = 1;
    while ((V >> bits) != 0) ++bits;  // the largest key is V
    p.passes = static_cast<int>(ceil_div(bits, kDigit));
    p.one = T <= kSortOne && V < (int64_t(1) << 25);
    p.tiles = ceil_div(T, kTile);
    p.pitch = ceil_div(D, 64) * 64;
    // stretches of 8 to 32 pairs, longer ones past 2048 of them: an entry named by every
    // token leaves a row in each, which one workgroup adds
    int64_t stretch = ceil_div(T, 2048);
    stretch = stretch < 32 ? (T >= 8192 ? 32 : T >= 2048 ? 16 : 8) : ceil_div(stretch, kAhead) * kAhead;
    p.stretch = static_cast<int>(stretch);
    p.stretches = ceil_div(T, stretch);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += aligned(bytes);
        return here;
    };
    p.keys = take(T * 4);
    p.tokens = take(T * 4);
    if (!p.one) {
        p.keys2 = take(T * 4);
        p.tokens2 = take(T * 4);
        p.counts = take(p.tiles * kBins * 4);
    }
    p.rows = take(p.stretches * 2 * p.pitch * 4);
    p.bytes = at;
    return p;
}

unsigned grid_of(int64_t groups) {
    const int64_t most = int64_t(1) << 20;  // the kernels stride over the rest
    return static_cast<unsigned>(groups < most ? groups : most);
}

template <typename T> hipError_t gather(const EmbedArgs& a) {
    const int64_t chunks = ceil_div(a.D, kChunk<T>);
    int lpr = 1;
    while (lpr < kThreads && lpr < chunks) lpr *= 2;
    const int64_t segs = ceil_div(chunks, static_cast<int64_t>(lpr) * kUnroll);
    const int64_t groups = ceil_div(a.T, kThreads / lpr) * segs;
    gather_kernel<T><<<dim3(grid_of(groups)), dim3(kThreads), 0, a.stream>>>(
        a.T, a.V, a.D, static_cast<const T*>(a.W), a.ldw, a.index, a.ignore, a.scale,
        static_cast<T*>(a.Y), a.ldy, lpr, segs, groups);
    return hipGetLastError();
}

// Sorts the tokens; *keys and *tokens are where the result lies.
hipError_t sort(const EmbedArgs& a, const Plan& p, uint8_t* ws, uint32_t** keys,
                uint32_t** tokens) {
    auto at = [&](int64_t offset) { return reinterpret_cast<uint32_t*>(ws + offset); };
    *keys = at(p.keys);
    *tokens = at(p.tokens);
    if (p.one) {
        sort_one_kernel<<<dim3(1), dim3(kSortThreads), 0, a.stream>>>(
            static_cast<int>(a.T), a.V, a.index, a.ignore, p.passes, *keys, *tokens);
        return hipGetLastError();
    }
    Pairs from{a.index, a.ignore, a.V, nullptr, nullptr};
    const unsigned grid = grid_of(p.tiles);
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * kDigit;
        // the last pass ends in keys and tokens
        const bool last = (p.passes - 1 - pass) % 2 == 0;
        uint32_t *const k = at(last ? p.keys : p.keys2), *const t = at(last ? p.tokens : p.tokens2);
        sort_count_kernel<<<dim3(grid), dim3(kSortThreads), 0, a.stream>>>(a.T, from, shift,
                                                                           p.tiles, at(p.counts));
        sort_scan_kernel<<<dim3(1), dim3(kSortThreads), 0, a.stream>>>(p.tiles * kBins,
                                                                       at(p.counts));
        sort_move_kernel<<<dim3(grid), dim3(kSortThreads), 0, a.stream>>>(
            a.T, from, shift, p.tiles, at(p.counts), k, t);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        from = Pairs{nullptr, 0, 0, k, t};
    }
    return hipSuccess;
}

template <typename T, typename W> hipError_t scatter(const EmbedArgs& a, void* ws) {
    W* const dw = static_cast<W*>(a.dW);
    if (a.T == 0) {
        if (a.accumulate) return hipSuccess;
        zero_kernel<W><<<dim3(grid_of(a.V)), dim3(kThreads), 0, a.stream>>>(a.V, a.D, dw, a.ldw);
        return hipGetLastError();
    }
    const Plan p = make_plan(a.T, a.V, a.D);
    uint8_t* const base = static_cast<uint8_t*>(ws);
    uint32_t *keys, *tokens;
    hipError_t err = sort(a, p, base, &keys, &tokens);
    if (err != hipSuccess) return err;
    GradArgs g{};
    g.T = a.T;
    g.V = a.V;
    g.D = a.D;
    g.keys = keys;
    g.tokens = tokens;
    g.ldy = a.ldy;
    g.ldw = a.ldw;
    g.scale = a.scale;
    g.accumulate = a.accumulate;
    g.stretch = p.stretch;
    g.stretches = p.stretches;
    g.pitch = p.pitch;
    g.shared_rows = reinterpret_cast<float*>(base + p.rows);
    const int64_t chunks = ceil_div(a.D, kChunk<T>);
    g.lpr = 1;
    while (g.lpr < kWave && g.lpr < chunks) g.lpr *= 2;
    g.segs = ceil_div(chunks, g.lpr);
    g.zero_groups = a.accumulate ? 0 : ceil_div(a.V, kZeroRows * (kThreads / kWave));
    const int64_t groups = g.zero_groups + ceil_div(g.stretches * g.segs, kThreads / g.lpr);
    scatter_kernel<T, W><<<dim3(static_cast<unsigned>(groups)), dim3(kThreads), 0, a.stream>>>(
        g, static_cast<const T*>(a.dY), dw);
    err = hipGetLastError();
    if (err != hipSuccess || g.stretches < 2) return err;
    scatter_join_kernel<T, W><<<dim3(static_cast<unsigned>(g.stretches - 1)), dim3(kJoinThreads), 0,
                                a.stream>>>(g, dw);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding(const EmbedArgs& a) {
    switch (a.dtype) {
        case 0: return gather<float>(a);
        case 1: return gather<_Float16>(a);
        default: return gather<bf16_t>(a);
    }
}

int64_t embedding_workspace(int64_t T, int64_t V, int64_t D) {
    return T == 0 ? 0 : make_plan(T, V, D).bytes;
}

hipError_t launch_embedding_backward(const EmbedArgs& a, void* ws) {
    switch (a.dtype) {
        case 0: return scatter<float, float>(a, ws);
        case 1: return a.w_dtype == 0 ? scatter<_Float16, float>(a, ws)
                                      : scatter<_Float16, _Float16>(a, ws);
        default: return a.w_dtype == 0 ? scatter<bf16_t, float>(a, ws)
                                       : scatter<bf16_t, bf16_t>(a, ws);
    }
}

}  // namespace migemm
