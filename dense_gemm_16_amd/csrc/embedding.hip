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
// workspace as one FP32 row, and a last kernel adds those.  Up to 2048 tokens take one launch
// and no sort: each token's workgroup looks for the others of its entry.
//
// Bound by memory: dy is read once, a row of dw written once (read too where it is added
// to).  Rows of dw that no token names are zeroed by workgroups of the same launch, and
// not touched where the gradient is added.  32768 tokens, 11000 entries of 131072 x 4096
// BF16: 64 to 72 us forwards (171 MB read, an entry once by each L2 cache, and 268 written);
// backwards, added, 21 for the sort, 105 for the sums (432 MB, 4.1 TB/s), 12 for the join.
// 65536 of 50001 x 2048 FP32: 190 us for the sums and zeros (907 MB, 4.8 TB/s).
#include "rows.hpp"
#include "training.hpp"

namespace migemm {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- forwards

// `lpr` lanes (a power of two) take a segment of `unroll` chunks a lane of one row, all of
// whose loads are in flight together.
constexpr int kUnroll = 4;
constexpr int64_t kFewChunks = 65536;
template <typename T, int C, int U>
__global__ __launch_bounds__(kThreads) void gather_kernel(
    int64_t tokens, int64_t V, int64_t D, const T* __restrict__ W, int64_t ldw,
    const int64_t* __restrict__ index, int64_t ignore, float scale, T* __restrict__ Y,
    int64_t ldy, int lpr, int64_t segs) {
    const int rows = kThreads / lpr, lane = threadIdx.x % lpr;
    const int64_t k0 = (blockIdx.x % segs * U * lpr + lane) * C;
    for (int64_t t = blockIdx.x / segs * rows + threadIdx.x / lpr; t < tokens;
         t += gridDim.x / segs * rows) {
        const int64_t v = index[t];
        const bool inside = v != ignore && v >= 0 && v < V;
        const T* const from = W + (inside ? v : 0) * ldw;  // (row 0 is read, and dropped)
        T e[U][C];
#pragma unroll
        for (int u = 0; u < U; ++u)
            Span<C>(k0 + static_cast<int64_t>(u) * lpr * C, D).load(from, e[u]);
        const T fill = narrow<T>(v == ignore ? 0.0f : __builtin_nanf(""));
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const T o = narrow<T>(scale * to_f32(e[u][i]));
                e[u][i] = inside ? o : fill;
            }
            Span<C>(k0 + static_cast<int64_t>(u) * lpr * C, D).store(Y + t * ldy, e[u]);
        }
    }
}

// -------------------------------------------------------------------- sorting

// A stable sort of (entry, token) pairs by entry, kDigit bits at a time, the lowest first.
// Tokens without an entry (ignored, or outside the table) sort last, as entry V.
constexpr int kDigit = 9, kBins = 1 << kDigit;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
// Pairs of a work-item: one up to 65536 pairs, where there are few workgroups, two in
// longer lists (2^18 pairs 33 us against 36 with one, 2^20 60 against 69).
constexpr int kEachFew = 1, kEachMany = 2;
constexpr int64_t kManyPairs = 65536;

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
__device__ __forceinline__ uint32_t rank_of(uint32_t digit, bool held, uint32_t* count) {
    const uint64_t same = peers(digit, held);
    const int lane = threadIdx.x % kWave;
    const uint64_t below = same & ((uint64_t(1) << lane) - 1);
    uint32_t before = 0;
    if (held) before = count[digit];
    // the lanes' reads come before the write, and that before the next call's reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (held && below == 0) count[digit] = before + static_cast<uint32_t>(__popcll(same));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return before + static_cast<uint32_t>(__popcll(below));
}

// Up to kRankMost pairs: each workgroup finds the places of kRankKeys of them by counting
// those that come before, all against all: 64 slices of the list, a work-item to a slice
// and a pair.  T^2 comparisons, but one short launch over many CUs: 4096 pairs 5.2 us and 8192
// 11, against 17 and 20 by the launches of the radix sort below; 16384 take four times as long
// as 8192, and 18 there.
constexpr int kRankMost = 8192, kRankKeys = 16, kRankSlices = kSortThreads / kRankKeys;
__global__ __launch_bounds__(kSortThreads) void sort_rank_kernel(
    int total, int64_t V, const int64_t* __restrict__ index, int64_t ignore,
    uint32_t* __restrict__ keys, uint32_t* __restrict__ tokens) {
    __shared__ __attribute__((aligned(16))) uint32_t all[kRankMost];
    __shared__ uint32_t place[kRankKeys];
    // whole slices of 16-byte reads; what is past the list comes after everything
    const int slice = (total + 4 * kRankSlices - 1) / (4 * kRankSlices) * 4;
    for (int i = threadIdx.x; i < slice * kRankSlices; i += kSortThreads)
        all[i] = i < total ? entry_of(index, i, ignore, V) : 0xffffffffu;
    if (threadIdx.x < kRankKeys) place[threadIdx.x] = 0;
    __syncthreads();
    const int mine = threadIdx.x % kRankKeys, s = threadIdx.x / kRankKeys;
    const int begin = blockIdx.x * kRankKeys, end = begin + kRankKeys, at = begin + mine;
    const uint32_t key = all[at];
    uint32_t before = 0;
    // those of [from, to) that come before it; `bound(j)`: how far up the entry of pair j may
    // go.  Both ends are multiples of 4.
    auto count = [&](int from, int to, auto bound) __attribute__((always_inline)) {
#pragma unroll 4
        for (int j = from; j < to; j += 4) {
            const u32x4 k = *reinterpret_cast<const u32x4*>(&all[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) before += k[e] < bound(j + e);
        }
    };
    const int lo = s * slice, hi = lo + slice;
    // earlier tokens of the same entry come first
    count(lo, hi < begin ? hi : begin, [&](int) { return key + 1; });
    count(lo > end ? lo : end, hi, [&](int) { return key; });
    if (s == 0) count(begin, end, [&](int j) { return key + (j < at); });
    atomicAdd(&place[mine], before);  // (a count: its order does not matter)
    __syncthreads();
    if (threadIdx.x < kRankKeys && at < total) {
        keys[place[mine]] = key;
        tokens[place[mine]] = static_cast<uint32_t>(at);
    }
}

// More pairs: each pass counts the digits of every tile, sums the counts over digits and
// tiles, and moves the pairs.  The first pass reads the index.  Up to kFewTiles tiles, the
// workgroups that move the pairs sum all counts themselves, which saves a launch; the
// counts then lie tile by tile.  Otherwise they lie digit by digit, a workgroup to a digit
// sums them over the tiles, and the digits' totals follow them.
constexpr int64_t kFewTiles = 128;
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

// The sum of the lanes up to this one.
__device__ __forceinline__ uint32_t sum_up(uint32_t v) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

template <int EACH>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(int64_t total, Pairs from,
                                                                  int shift, int64_t tiles,
                                                                  uint32_t* __restrict__ counts) {
    constexpr int kTile = EACH * kSortThreads;
    const bool few = tiles <= kFewTiles;
    __shared__ uint32_t bins[kBins];
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        if (threadIdx.x < kBins) bins[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int64_t at = tile * kTile + i * kSortThreads + threadIdx.x;
            // counts alone: their order does not matter
            if (at < total) atomicAdd(&bins[(from.key(at) >> shift) & (kBins - 1)], 1u);
        }
        __syncthreads();
        if (threadIdx.x < kBins)
            counts[few ? tile * kBins + threadIdx.x : threadIdx.x * tiles + tile] =
                bins[threadIdx.x];
        __syncthreads();
    }
}

// Exclusive sums over the tiles, in place, of the digit blockIdx.x, and its total.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(int64_t tiles,
                                                                 uint32_t* __restrict__ counts) {
    constexpr int kEach = 4;
    __shared__ uint32_t wave_sum[2][kSortWaves];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    uint32_t* const mine = counts + blockIdx.x * tiles;
    uint32_t before = 0;
    int turn = 0;
    for (int64_t base = 0; base < tiles; base += kSortThreads * kEach, turn ^= 1) {
        const int64_t at = base + threadIdx.x * kEach;
        uint32_t c[kEach], sum = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const uint32_t v = at + i < tiles ? mine[at + i] : 0;
            c[i] = sum;
            sum += v;
        }
        const uint32_t up = sum_up(sum);
        if (lane == kWave - 1) wave_sum[turn][wave] = up;
        __syncthreads();
        uint32_t here = before + up - sum;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) here += wave_sum[turn][w];
            before += wave_sum[turn][w];
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (at + i < tiles) mine[at + i] = here + c[i];
    }
    if (threadIdx.x == 0) counts[kBins * tiles + blockIdx.x] = before;
}

template <int EACH>
__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(
    int64_t total, Pairs from, int shift, int64_t tiles, const uint32_t* __restrict__ offsets,
    uint32_t* __restrict__ keys, uint32_t* __restrict__ tokens) {
    constexpr int kTile = EACH * kSortThreads;
    __shared__ uint32_t count[kSortWaves][kBins];
    __shared__ uint32_t early[2][kBins], wave_sum[kSortWaves];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const bool few = tiles <= kFewTiles;  // (then a workgroup has one tile)
    // `place`: of the first pair of digit threadIdx.x, in the tile (few) or in the list
    const int digit = threadIdx.x % kBins, half = threadIdx.x / kBins;
    uint32_t place = 0, all = 0;
    if (few) {
        // each digit's pairs in the tiles before this one, and in all; even tiles by one half
        // of the workgroup, odd ones by the other
#pragma unroll 8
        for (int t = half; t < static_cast<int>(tiles); t += 2) {
            const uint32_t c = offsets[t * kBins + digit];
            all += c;
            place += t < static_cast<int>(blockIdx.x) ? c : 0;
        }
        if (half) {
            early[0][digit] = place;
            early[1][digit] = all;
        }
        __syncthreads();
        place += early[0][digit];
        all += early[1][digit];
    } else {
        all = offsets[kBins * tiles + digit];
    }
    // (the second half of the workgroup drops what it sums up)
    const uint32_t up = sum_up(all);
    if (lane == kWave - 1) wave_sum[wave] = up;
    __syncthreads();
    place += up - all;
    for (int w = 0; w < wave; ++w) place += wave_sum[w];
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        for (int i = threadIdx.x; i < kSortWaves * kBins; i += kSortThreads)
            (&count[0][0])[i] = 0;
        __syncthreads();
        const int64_t first = tile * kTile + wave * EACH * kWave + lane;
        uint32_t key[EACH], rank[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int64_t at = first + i * kWave;
            key[i] = at < total ? from.key(at) : 0;
            rank[i] = rank_of((key[i] >> shift) & (kBins - 1), at < total, count[wave]);
        }
        __syncthreads();
        // each digit's place in the whole list, then wavefront by wavefront
        if (threadIdx.x < kBins) {
            uint32_t at = place + (few ? 0 : offsets[digit * tiles + tile]);
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = count[w][threadIdx.x];
                count[w][threadIdx.x] = at;
                at += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int64_t at = first + i * kWave;
            if (at >= total) continue;
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
    int stretch;  // pairs of a stretch
    int64_t stretches, pitch;
    float* shared_rows;  // two rows of `pitch` a stretch: of an entry begun before it, of
                         // one that goes on after it
    int lpr;             // lanes of a segment of a row, a power of two up to 64
    int64_t segs;        // segments of a row: a chunk of dy a lane each
    int64_t sum_groups;  // workgroups that add; those after them zero rows
    int64_t few_parts;   // of few tokens: workgroups of a token
    bool once;           // of few tokens: zeros go past the caches
};

// The first pair of an entry of v or more, by a whole wavefront: 64 places at a time, so
// three loads one after the other for 2^18 pairs.
__device__ __forceinline__ int64_t first_of(const GradArgs& a, int64_t v) {
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, n = a.T;
    while (n > 0) {
        const int64_t step = ceil_div(n, kWave), at = lo + (lane + 1) * step - 1, end = lo + n;
        lo += step * __popcll(__ballot(at < end && a.keys[at < end ? at : lo] < v));
        n = lo < end ? (end - lo < step - 1 ? end - lo : step - 1) : 0;
    }
    return lo < a.T ? lo : a.T;
}

// Zeros rows of entries v0 .. v0 + kZeroRows - 1, those that no bit of `named` stands for,
// by one wavefront.
constexpr int kZeroRows = 16;
template <typename W, int C, bool ONCE>
__device__ __forceinline__ void zero_rows(const GradArgs& a, int64_t v0, uint64_t named,
                                          W* __restrict__ dW) {
    const int lane = threadIdx.x % kWave;
    const int64_t rows = v0 + kZeroRows < a.V ? kZeroRows : a.V - v0;
    W zero[C];
#pragma unroll
    for (int i = 0; i < C; ++i) zero[i] = narrow<W>(0.0f);
    for (uint64_t todo = ((uint64_t(1) << rows) - 1) & ~named; todo; todo &= todo - 1) {
        W* const row = dW + (v0 + __builtin_ctzll(todo)) * a.ldw;
        for (int64_t k = lane * C; k < a.D; k += kWave * C) {
            const Span<C> piece(k, a.D);
            if constexpr (ONCE)
                store_once(row + piece.at, zero);
            else
                store_whole(row + piece.at, zero);
        }
    }
}

// Those of the entries v0 .. v0 + kZeroRows - 1 that sorted tokens name.
__device__ __forceinline__ uint64_t named_rows(const GradArgs& a, int64_t v0) {
    const int lane = threadIdx.x % kWave;
    const int64_t v1 = v0 + kZeroRows < a.V ? v0 + kZeroRows : a.V;
    uint64_t named = 0;
    for (int64_t v = v0; v < v1;) {
        // 64 pairs from the first of an entry not seen yet
        const int64_t at = first_of(a, v) + lane;
        const int64_t key = at < a.T ? a.keys[at] : a.V;
#pragma unroll
        for (int i = 0; i < kZeroRows; ++i)
            if (__ballot(key == v0 + i)) named |= uint64_t(1) << i;
        v = __builtin_amdgcn_readlane(static_cast<uint32_t>(key), kWave - 1) + int64_t(1);
    }
    return named;
}

// A group of a.lpr lanes sums a segment of columns over one stretch.  An entry that begins
// in it and ends in the next one is finished here, and left out there: where every other
// stretch ended inside an entry, the sums left to join took 37 us beside 90 (32768 tokens
// of 4096 columns).  The group's lanes load the entries and tokens of as many pairs at
// once; then kAhead rows of dy are in flight together, and, where the gradient is added
// (ADD), the rows of dw whose entries end among them.  WAVE: the group is a wavefront
// (pairs come by readlane, and branches are uniform).  ONCE: dy is read, and zeros are
// written, past the caches.
constexpr int kAhead = 8;
template <typename T, typename W, int C, bool WAVE, bool ADD, bool ONCE>
__global__ __launch_bounds__(kThreads) void scatter_kernel(GradArgs a, const T* __restrict__ dY,
                                                           W* __restrict__ dW) {
    if (blockIdx.x >= a.sum_groups) {
        const int64_t v0 = (static_cast<int64_t>(blockIdx.x - a.sum_groups) * (kThreads / kWave) +
                            threadIdx.x / kWave) * kZeroRows;
        if (v0 < a.V) zero_rows<W, C, ONCE>(a, v0, named_rows(a, v0), dW);
        return;
    }
    const int lpr = WAVE ? kWave : a.lpr;
    const int64_t group = static_cast<int64_t>(blockIdx.x) * (kThreads / lpr) + threadIdx.x / lpr;
    const int64_t s = group / a.segs;
    if (s >= a.stretches) return;
    const int lane = threadIdx.x % lpr;
    const Span<C> piece((group % a.segs * lpr + lane) * C, a.D);
    int64_t first = s * a.stretch;
    const int64_t end = first + a.stretch < a.T ? first + a.stretch : a.T;
    const uint32_t none = static_cast<uint32_t>(a.V);
    // the entry at i, or one past all of them where the list has ended or not begun
    auto entry = [&](int64_t i) { return i >= 0 && i < a.T ? a.keys[i] : none + 1; };
    const uint32_t before = entry(first - 1), head = entry(first), tail = entry(end - 1);
    const uint32_t after = entry(end), earlier = entry(first - a.stretch - 1);
    const uint32_t later = entry(end + a.stretch);
    // pairs of [from, from + stretch) that go on with entry v
    auto run = [&](int64_t from, uint32_t v) {
        const int shift = static_cast<int>(threadIdx.x) % kWave / lpr * lpr;
        int64_t n = 0;
        while (n < a.stretch) {
            const uint64_t same = __ballot(n + lane < a.stretch && entry(from + n + lane) == v);
            const uint64_t mine = same >> shift & (~uint64_t(0) >> (kWave - lpr));
            n += __popcll(mine);
            if (static_cast<int>(__popcll(mine)) < lpr) break;
        }
        return n;
    };
    // whether the sum of its first entry is begun in a stretch before
    bool begun = before == head && head != none;
    if (begun && earlier != head && after != head) {  // begun in the last one and ended here
        first += run(first, head);
        begun = false;
    }
    int64_t stop = end;
    if (tail != none && after == tail && before != tail && later != tail) stop += run(end, tail);
    float sum[C];
#pragma unroll
    for (int c = 0; c < C; ++c) sum[c] = 0.0f;
    for (int64_t base = first; base < stop; base += lpr) {
        // pair base + lane, and the entry after it
        const int64_t mine = base + lane < a.T ? base + lane : a.T - 1;
        const uint32_t my_key = a.keys[mine], my_token = a.tokens[mine];
        const uint32_t my_next = mine + 1 < a.T ? a.keys[mine + 1] : none;
        const int pairs = static_cast<int>(stop - base < lpr ? stop - base : lpr);
        for (int i = 0; i < pairs; i += kAhead) {
            uint32_t key[kAhead], next[kAhead];
            T e[kAhead][C];
            W old[ADD ? kAhead : 1][C];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int from = i + u < pairs ? i + u : pairs - 1;
                uint32_t token;
                if constexpr (WAVE) {
                    key[u] = __builtin_amdgcn_readlane(my_key, from);
                    next[u] = __builtin_amdgcn_readlane(my_next, from);
                    token = __builtin_amdgcn_readlane(my_token, from);
                } else {
                    key[u] = __shfl(my_key, from, lpr);
                    next[u] = __shfl(my_next, from, lpr);
                    token = __shfl(my_token, from, lpr);
                }
                // (the row of a token without an entry is read, and dropped)
                if constexpr (ONCE)
                    load_once(dY + token * a.ldy + piece.at, e[u]);
                else
                    piece.load(dY + token * a.ldy, e[u]);
                if constexpr (ADD) {
                    // the last row stands in for those that are not needed
                    const uint32_t row = key[u] != next[u] && key[u] != none ? key[u] : key[0];
                    piece.load(dW + (row != none ? row : 0) * a.ldw, old[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (i + u >= pairs || key[u] == none) break;
#pragma unroll
                for (int c = 0; c < C; ++c) sum[c] += to_f32(e[u][c]);
                const bool last = key[u] != next[u];
                if (last && !begun) {
                    W o[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        if constexpr (ADD)
                            o[c] = narrow<W>(fmaf(a.scale, sum[c], to_f32(old[u][c])));
                        else
                            o[c] = narrow<W>(a.scale * sum[c]);
                    }
                    piece.store_own(dW + key[u] * a.ldw, o);
                } else if (last || base + i + u + 1 == stop) {
                    piece.store(a.shared_rows + (2 * s + (begun ? 0 : 1)) * a.pitch, sum);
                }
                if (last) {
                    begun = false;
#pragma unroll
                    for (int c = 0; c < C; ++c) sum[c] = 0.0f;
                }
            }
        }
    }
}

// Entries that several stretches share: the stretch where one begins adds up the rows
// that they left.  A workgroup looks at kJoinEach stretches, one lane at each (one to a
// workgroup, most of which then end at once, took 14 us for 1024 stretches of 4096
// columns), and adds up to them one after the other, 64 C columns.
constexpr int kJoinWaves = 8, kJoinThreads = kJoinWaves * kWave, kJoinEach = 8;
template <typename W, int C, bool ADD>
__global__ __launch_bounds__(kJoinThreads) void scatter_join_kernel(GradArgs a,
                                                                   W* __restrict__ dW) {
    __shared__ float lds[kJoinWaves][kWave][C + 1];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kJoinEach;
    bool open = false;
    if (lane < kJoinEach && base + lane + 1 < a.stretches) {
        const int64_t first = (base + lane) * a.stretch, end = first + a.stretch;
        const uint32_t v = a.keys[end - 1];
        const uint32_t before = a.keys[first > 0 ? first - 1 : 0];
        const int64_t far = end + a.stretch < a.T ? end + a.stretch : a.T - 1;
        // its last entry begins inside it, and goes on past the next one
        open = v != static_cast<uint32_t>(a.V) && (first == 0 || before != v) &&
               end + a.stretch < a.T && a.keys[far] == v;
    }
    const Span<C> piece((static_cast<int64_t>(blockIdx.y) * kWave + lane) * C, a.D);
    for (uint64_t todo = __ballot(open); todo; todo &= todo - 1) {
        const int64_t s = base + __builtin_ctzll(todo);
        const uint32_t v = a.keys[(s + 1) * a.stretch];
        // the last stretch that holds it: 64 of them are looked at together, ever closer ones
        int64_t lo = s + 1;
        for (int64_t by = kWave * kWave; by > 0; by /= kWave) {
            const int64_t at = lo + lane * by;
            const bool holds = at < a.stretches && a.keys[at * a.stretch] == v;
            lo += (__popcll(__ballot(holds)) - 1) * by;
        }
        ++lo;
        float sum[C];
#pragma unroll
        for (int c = 0; c < C; ++c) sum[c] = 0.0f;
        if (wave == 0) piece.load(a.shared_rows + (2 * s + 1) * a.pitch, sum);
        for (int64_t i = s + 1 + wave; i < lo; i += kJoinWaves * kAhead) {
            float e[kAhead][C];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t j = i + u * kJoinWaves < lo ? i + u * kJoinWaves : lo - 1;
                piece.load(a.shared_rows + 2 * j * a.pitch, e[u]);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c) sum[c] += i + u * kJoinWaves < lo ? e[u][c] : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) lds[wave][lane][c] = sum[c];
        __syncthreads();
        if (wave == 0) {
            W o[C];
            if constexpr (ADD) piece.load(dW + v * a.ldw, o);
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int w = 1; w < kJoinWaves; ++w) sum[c] += lds[w][lane][c];
                o[c] = narrow<W>(ADD ? fmaf(a.scale, sum[c], to_f32(o[c])) : a.scale * sum[c]);
            }
            piece.store_own(dW + v * a.ldw, o);
        }
        __syncthreads();
    }
}

// Up to kFewTokens tokens, in one launch and without a sort.  A workgroup stands for a token
// and kFewWaves segments of columns.  It looks at all tokens, KEYS a lane, and lists those of
// its token's entry, in order; the workgroup of the first of them sums them, a wavefront to a
// segment.  Where the list is long, those of the first kFewGroups tokens sum a quarter of a
// segment each, 16 lanes to a part of the list, joined in order.  Workgroups behind all these
// zero the rows that no token names.
//
// Each token's workgroups read the whole list, so the work grows with its square, and wide
// rows take more workgroups: kFewWide of them at most (of 16-bit rows; FP32 rows take twice as
// many).  Against the sort, sums and join of longer lists, added: 16 tokens of 4096 BF16
// columns 3.3 us instead of 8.5, 256 3.9 instead of 10.5, 2048 14.5 instead of 21.8 (16.8 after
// the lookup of other tokens), all of one entry 17.8 instead of 18.0; 512 of 16384 FP32 columns 21.7 instead of 24.7.  2048 of 8192
// BF16 columns would take 31.6 instead of 26.6, 4096 of 4096 30.7 instead of 25.2.
constexpr int64_t kFewTokens = 2048, kFewWide = 4096;
bool few_tokens(int64_t T, int64_t D) {
    return T <= kFewTokens && T * ceil_div(D, 2048) <= kFewWide;
}
constexpr int kFewAhead = 8, kFewWaves = 4, kFewMany = 16;
constexpr int kFewLanes = 16, kFewQuarters = kWave / kFewLanes;
constexpr int kFewGroups = kFewWaves * kFewQuarters;  // (kFewMany or fewer)
template <typename T, typename W, int C, int KEYS, bool ADD>
__global__ __launch_bounds__(kFewWaves * kWave) void scatter_few_kernel(
    GradArgs a, const int64_t* __restrict__ index, int64_t ignore, const T* __restrict__ dY,
    W* __restrict__ dW) {
    __shared__ int list[kFewWaves * KEYS * kWave];
    __shared__ float lds[kFewGroups][kFewLanes][C + 1];
    __shared__ int found[kFewWaves], earlier[kFewWaves];
    __shared__ uint32_t rows[kFewWaves * kZeroRows / 32];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int tokens = static_cast<int>(a.T), first = wave * KEYS * kWave + lane;
    const uint32_t none = static_cast<uint32_t>(a.V);
    uint32_t key[KEYS];
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
        const int t = first + k * kWave;
        const uint32_t v = entry_of(index, t < tokens ? t : tokens - 1, ignore, a.V);
        key[k] = t < tokens ? v : none;
    }
    if (blockIdx.x >= a.sum_groups) {
        const int64_t v0 = static_cast<int64_t>(blockIdx.x - a.sum_groups) * kFewWaves * kZeroRows;
        if (threadIdx.x < kFewWaves * kZeroRows / 32) rows[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KEYS; ++k) {
            const uint32_t row = key[k] - static_cast<uint32_t>(v0);  // (2^31 and more: before v0)
            if (row < kFewWaves * kZeroRows) atomicOr(&rows[row / 32], 1u << row % 32);
        }
        __syncthreads();
        const int mine = wave * kZeroRows;
        if (v0 + mine >= a.V) return;
        const uint32_t named = rows[mine / 32] >> mine % 32;
        if (a.once)
            zero_rows<W, C, true>(a, v0 + mine, named, dW);
        else
            zero_rows<W, C, false>(a, v0 + mine, named, dW);
        return;
    }
    const int token = static_cast<int>(blockIdx.x / a.few_parts);
    const uint32_t v = entry_of(index, token, ignore, a.V);
    if (v == none) return;
    int held = 0, before = 0;
    uint64_t same[KEYS];
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
        same[k] = __ballot(key[k] == v);
        held += static_cast<int>(__popcll(same[k]));
        before += static_cast<int>(__popcll(__ballot(key[k] == v && first + k * kWave < token)));
    }
    if (lane == 0) {
        found[wave] = held;
        earlier[wave] = before;
    }
    __syncthreads();
    int count = 0, rank = 0, at = 0;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
        at += w < wave ? found[w] : 0;
        count += found[w];
        rank += earlier[w];
    }
    const bool many = count > kFewMany;
    if (rank >= (many ? kFewGroups : 1)) return;  // (all of the workgroup)
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
        if (key[k] == v)
            list[at + __popcll(same[k] & ((uint64_t(1) << lane) - 1))] = first + k * kWave;
        at += static_cast<int>(__popcll(same[k]));
    }
    __syncthreads();
    const int64_t seg = static_cast<int64_t>(blockIdx.x % a.few_parts) * kFewWaves +
                        (many ? rank / kFewQuarters : wave);
    if (seg >= a.segs) return;  // (many: all of the workgroup)
    const int chunk = many ? rank % kFewQuarters * kFewLanes + lane % kFewLanes : lane;
    const Span<C> piece((seg * kWave + chunk) * C, a.D);
    const int each = many ? (count + kFewGroups - 1) / kFewGroups : count;
    const int from = many ? threadIdx.x / kFewLanes * each : 0;
    const int to = from + each < count ? from + each : count;
    W o[C];
    if constexpr (ADD) piece.load(dW + v * a.ldw, o);
    float sum[C];
#pragma unroll
    for (int c = 0; c < C; ++c) sum[c] = 0.0f;
    for (int i = from; i < to; i += kFewAhead) {
        T e[kFewAhead][C];
#pragma unroll
        for (int u = 0; u < kFewAhead; ++u) {
            const int t = list[i + u < to ? i + u : to - 1];
            piece.load(dY + static_cast<int64_t>(t) * a.ldy, e[u]);
        }
#pragma unroll
        for (int u = 0; u < kFewAhead; ++u)
#pragma unroll
            for (int c = 0; c < C; ++c) sum[c] += i + u < to ? to_f32(e[u][c]) : 0.0f;
    }
    if (many) {
#pragma unroll
        for (int c = 0; c < C; ++c) lds[threadIdx.x / kFewLanes][lane % kFewLanes][c] = sum[c];
        __syncthreads();
        if (threadIdx.x >= kFewLanes) return;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int g = 1; g < kFewGroups; ++g) sum[c] += lds[g][lane][c];
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        o[c] = narrow<W>(ADD ? fmaf(a.scale, sum[c], to_f32(o[c])) : a.scale * sum[c]);
    piece.store_own(dW + v * a.ldw, o);
}

// dw of no tokens: zeros.
template <typename W>
__global__ __launch_bounds__(kThreads) void zero_kernel(int64_t V, int64_t D, W* __restrict__ dW,
                                                        int64_t ldw) {
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x)
        for (int64_t k = threadIdx.x; k < D; k += kThreads) dW[v * ldw + k] = narrow<W>(0.0f);
}

// The workspace: sorted entries and tokens, the other copy of them and the counts where
// the sort takes several passes, and the stretches' shared rows.
struct Plan {
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
    p.tiles = ceil_div(T, (T <= kManyPairs ? kEachFew : kEachMany) * kSortThreads);
    p.pitch = ceil_div(D, 64) * 64;
    // stretches of 8 to 32 pairs (16384 tokens of 1024 columns: 12.6 us with 16, 15.4 with
    // 32), longer ones past some number of them: an entry named by every token leaves a row
    // in each, which one workgroup adds.  The narrower the rows, the more of them: 2^22
    // tokens of 128 columns 570 us with 8192, 1520 with 2048; with 32768 475, but 920
    // instead of 460 where all tokens name one entry
    int64_t most = (int64_t(1) << 22) / D;
    most = most < 2048 ? 2048 : most > 8192 ? 8192 : most;
    const int64_t stretch = T < 2048    ? 8
                            : T < 32768 ? 16
                                        : ceil_div(ceil_div(T, most), 32) * 32;
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
    if (T > kRankMost) {
        p.keys2 = take(T * 4);
        p.tokens2 = take(T * 4);
        p.counts = take((p.tiles + 1) * kBins * 4);
    }
    p.rows = take(p.stretches * 2 * p.pitch * 4);
    p.bytes = at;
    return p;
}

unsigned grid_of(int64_t groups) {
    const int64_t most = int64_t(1) << 20;  // the kernels stride over the rest
    return static_cast<unsigned>(groups < most ? groups : most);
}

// Rows shorter than a chunk are taken one element a lane.
template <typename T, int C> hipError_t gather(const EmbedArgs& a) {
    const int64_t chunks = ceil_div(a.D, C);
    // few tokens: a chunk a lane, so that many lanes share the latency; else kUnroll
    const bool few = a.T * chunks <= kFewChunks;
    const int unroll = few ? 1 : kUnroll;
    int lpr = 1;
    while (lpr < kThreads && lpr * unroll < chunks) lpr *= 2;
    const int64_t segs = ceil_div(chunks, static_cast<int64_t>(lpr) * unroll);
    int64_t rows = ceil_div(a.T, kThreads / lpr);
    const int64_t most = launch_groups(kThreads) / segs;  // the kernel strides over the rest
    if (rows > most) rows = most;
    const auto fn = few ? gather_kernel<T, C, 1> : gather_kernel<T, C, kUnroll>;
    fn<<<dim3(static_cast<unsigned>(rows * segs)), dim3(kThreads), 0, a.stream>>>(
        a.T, a.V, a.D, static_cast<const T*>(a.W), a.ldw, a.index, a.ignore, a.scale,
        static_cast<T*>(a.Y), a.ldy, lpr, segs);
    return hipGetLastError();
}

// Sorts the tokens; *keys and *tokens are where the result lies.
hipError_t sort(const EmbedArgs& a, const Plan& p, uint8_t* ws, uint32_t** keys,
                uint32_t** tokens) {
    auto at = [&](int64_t offset) { return reinterpret_cast<uint32_t*>(ws + offset); };
    *keys = at(p.keys);
    *tokens = at(p.tokens);
    const int n = static_cast<int>(a.T);
    if (a.T <= kRankMost) {
        sort_rank_kernel<<<dim3(static_cast<unsigned>(ceil_div(a.T, kRankKeys))),
                           dim3(kSortThreads), 0, a.stream>>>(n, a.V, a.index, a.ignore, *keys,
                                                              *tokens);
        return hipGetLastError();
    }
    Pairs from{a.index, a.ignore, a.V, nullptr, nullptr};
    uint32_t* const counts = at(p.counts);
    const dim3 grid(grid_of(p.tiles)), block(kSortThreads);
    const bool many = a.T > kManyPairs;
    const auto count = many ? sort_count_kernel<kEachMany> : sort_count_kernel<kEachFew>;
    const auto move = many ? sort_move_kernel<kEachMany> : sort_move_kernel<kEachFew>;
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * kDigit;
        // the last pass ends in keys and tokens
        const bool last = (p.passes - 1 - pass) % 2 == 0;
        uint32_t *const k = at(last ? p.keys : p.keys2), *const t = at(last ? p.tokens : p.tokens2);
        count<<<grid, block, 0, a.stream>>>(a.T, from, shift, p.tiles, counts);
        if (p.tiles > kFewTiles)
            sort_scan_kernel<<<dim3(kBins), block, 0, a.stream>>>(p.tiles, counts);
        move<<<grid, block, 0, a.stream>>>(a.T, from, shift, p.tiles, counts, k, t);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        from = Pairs{nullptr, 0, 0, k, t};
    }
    return hipSuccess;
}

// From this many bytes of dy and of rows to zero, both go past the caches, whose last level
// (256 MiB) holds too little of them for the next reader: 65536 tokens of 50001 x 2048 FP32
// 192 us instead of 207, 32768 of 131072 x 4096 BF16, added, 99 instead of 105; 8192 of
// those 35 instead of 32.
constexpr double kOnceBytes = 256 << 20;

template <typename T, typename W, int C>
hipError_t scatter_few(const EmbedArgs& a) {
    const int64_t zero_groups = a.accumulate ? 0 : ceil_div(a.V, kZeroRows * kFewWaves);
    GradArgs g{};
    g.T = a.T;
    g.V = a.V;
    g.D = a.D;
    g.ldy = a.ldy;
    g.ldw = a.ldw;
    g.scale = a.scale;
    g.segs = ceil_div(ceil_div(a.D, C), kWave);
    g.few_parts = ceil_div(g.segs, kFewWaves);
    g.sum_groups = a.T * g.few_parts;
    g.once = static_cast<double>(sizeof(W)) * a.V * a.D >= kOnceBytes;
    auto go = [&](auto keys, auto add) {
        scatter_few_kernel<T, W, C, decltype(keys)::value, decltype(add)::value>
            <<<dim3(static_cast<unsigned>(g.sum_groups + zero_groups)), dim3(kFewWaves * kWave), 0,
               a.stream>>>(g, a.index, a.ignore, static_cast<const T*>(a.dY),
                           static_cast<W*>(a.dW));
        return hipGetLastError();
    };
    auto by_keys = [&](auto add) {
        if (a.T <= kFewWaves * kWave) return go(std::integral_constant<int, 1>{}, add);
        if (a.T <= 2 * kFewWaves * kWave) return go(std::integral_constant<int, 2>{}, add);
        if (a.T <= 4 * kFewWaves * kWave) return go(std::integral_constant<int, 4>{}, add);
        static_assert(kFewTokens == 8 * kFewWaves * kWave, "the longest list fits");
        return go(std::integral_constant<int, 8>{}, add);
    };
    return a.accumulate ? by_keys(std::true_type{}) : by_keys(std::false_type{});
}

template <typename T, typename W, int C> hipError_t scatter(const EmbedArgs& a, void* ws) {
    W* const dw = static_cast<W*>(a.dW);
    if (a.T == 0) {
        if (a.accumulate) return hipSuccess;
        zero_kernel<W><<<dim3(grid_of(a.V)), dim3(kThreads), 0, a.stream>>>(a.V, a.D, dw, a.ldw);
        return hipGetLastError();
    }
    if (few_tokens(a.T, a.D)) return scatter_few<T, W, C>(a);
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
    g.stretch = p.stretch;
    g.stretches = p.stretches;
    g.pitch = p.pitch;
    g.shared_rows = reinterpret_cast<float*>(base + p.rows);
    const int64_t chunks = ceil_div(a.D, C);
    g.lpr = kAhead;
    while (g.lpr < kWave && g.lpr < chunks) g.lpr *= 2;
    g.segs = ceil_div(chunks, g.lpr);
    g.sum_groups = ceil_div(g.stretches * g.segs, kThreads / g.lpr);
    const int64_t zero_groups = a.accumulate ? 0 : ceil_div(a.V, kZeroRows * (kThreads / kWave));
    const dim3 groups(static_cast<unsigned>(g.sum_groups + zero_groups)), threads(kThreads);
    const dim3 joins(static_cast<unsigned>(ceil_div(g.stretches - 1, kJoinEach)),
                     static_cast<unsigned>(ceil_div(chunks, kWave)));
    auto go = [&](auto wave, auto add, auto past) {
        constexpr bool WAVE = decltype(wave)::value, ADD = decltype(add)::value,
                       ONCE = decltype(past)::value;
        scatter_kernel<T, W, C, WAVE, ADD, ONCE>
            <<<groups, threads, 0, a.stream>>>(g, static_cast<const T*>(a.dY), dw);
        const hipError_t e = hipGetLastError();
        // (one stretch, of up to 8 pairs of rows past a million columns, shares no entry)
        if (e != hipSuccess || g.stretches < 2) return e;
        scatter_join_kernel<W, C, ADD><<<joins, dim3(kJoinThreads), 0, a.stream>>>(g, dw);
        return hipGetLastError();
    };
    using yes = std::true_type;
    using no = std::false_type;
    const double bytes = static_cast<double>(sizeof(T)) * a.T * a.D +
                         (a.accumulate ? 0.0 : static_cast<double>(sizeof(W)) * a.V * a.D);
    const bool once = bytes >= kOnceBytes;
    if (g.lpr < kWave) return a.accumulate ? go(no{}, yes{}, no{}) : go(no{}, no{}, no{});
    if (once) return a.accumulate ? go(yes{}, yes{}, yes{}) : go(yes{}, no{}, yes{});
    return a.accumulate ? go(yes{}, yes{}, no{}) : go(yes{}, no{}, no{});
}

template <typename T> hipError_t gather_any(const EmbedArgs& a) {
    return a.D < kChunk<T> ? gather<T, 1>(a) : gather<T, kChunk<T>>(a);
}
template <typename T, typename W> hipError_t scatter_any(const EmbedArgs& a, void* ws) {
    return a.D < kChunk<T> ? scatter<T, W, 1>(a, ws) : scatter<T, W, kChunk<T>>(a, ws);
}

}  // namespace

hipError_t launch_embedding(const EmbedArgs& a) {
    switch (a.dtype) {
        case 0: return gather_any<float>(a);
        case 1: return gather_any<_Float16>(a);
        default: return gather_any<bf16_t>(a);
    }
}

int64_t embedding_workspace(int64_t T, int64_t V, int64_t D) {
    return few_tokens(T, D) ? 0 : make_plan(T, V, D).bytes;
}

hipError_t launch_embedding_backward(const EmbedArgs& a, void* ws) {
    switch (a.dtype) {
        case 0: return scatter_any<float, float>(a, ws);
        case 1: return a.w_dtype == 0 ? scatter_any<_Float16, float>(a, ws)
                                      : scatter_any<_Float16, _Float16>(a, ws);
        default: return a.w_dtype == 0 ? scatter_any<bf16_t, float>(a, ws)
                                       : scatter_any<bf16_t, bf16_t>(a, ws);
    }
}

}  // namespace migemm
