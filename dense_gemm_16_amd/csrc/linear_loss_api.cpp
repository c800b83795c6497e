// linear_loss_api.cpp -- the output-layer losses' entry points: argument checks,
// the plan of a call (what is copied, the pieces of the vocabulary, where each
// scratch array lies in the lent workspace) and its launches.
#include <math.h>

#include "linear_loss.hpp"
#include "migemm.h"

namespace migemm {

// 256x256 tiles from half a round of them on, else 128x128 from half a round,
// else 64x64; the ping-pong schedule where every tile and k-tile is whole.  Forward
// pass, us on 64 / 128 / 256 (BF16): 64 x 32000 x 1024 18 / 19 / 34, 200 x 50000 x 2048
// 89 / 78 / 61, 4096 x 1000 x 1024 31 / 25 / 41; FP32 100 x 4000 x 512 16 / 38, 500 x 8000
// x 512 46 / 42.  At 128 to 160 tiles of 256x256 neither side is always the better:
// forward and backward pass on 128 / 256, 1000 x 8000 x 512 21 + 55 / 25 + 61, 2048 x 4096 x
// 2048 50 + 135 / 52 + 134, 200 x 33000 x 1024 36 + 105 / 33 + 98, 500 x 17000 x 1024 37 +
// 99 / 33 + 98, 1024 x 8192 x 4096 77 + 241 / 77 + 214; 128 where the 256-high tiles stand
// half empty, 300 x 20000 x 2048 41 + 128 / 54 + 134.
// FP32, which the matrix cores' rate bounds, takes 64x64 tiles (two to a CU) where a
// last round of 128x128 ones would stand mostly empty (723 x 5489 x 804: 82 against
// 108), 64x32 ones on at most half a round, whose k-tile is half as long (33 x 4099 x
// 520: 10.1 against 13.7), and 32x64 ones for up to 32 rows (5 x 21566 x 1920: 43
// against 68).  2^23 tiles of 64x64 are more than one launch holds (2^32 threads): so many
// are always 128x128, where a last round no longer counts.
LossShape loss_shape(int dtype, int64_t M, int64_t N, int64_t K) {
    auto tiles = [&](int64_t b) { return ceil_div(M, b) * ceil_div(N, b); };
    const bool f32 = dtype == MIGEMM_F32;
    if (!f32 && M > 128 && tiles(256) >= 128)
        return {M % 256 == 0 && N % 256 == 0 && K % 64 == 0 ? 3 : 2, 64, 256};
    if (f32 && M > 64 && tiles(128) >= 128) {
        const int64_t t = tiles(64) % 512;
        const double c64 =
            static_cast<double>(tiles(64) / 512) + (t > 256 ? 1.0 : t > 0 ? 0.63 : 0.0);
        if (tiles(64) >= int64_t(1) << 23 ||
            2.0 * static_cast<double>(ceil_div(tiles(128), 256)) <= c64)
            return {1, 32, 128};
        return {0, 16, 64};
    }
    if (M > 64 && tiles(128) >= 128) return {1, 32, 128};
    if (f32 && M <= 32) return {3, 16, 64};
    if (f32 && tiles(64) <= 128) return {2, 16, 32};
    return {0, 16, 64};
}

hipError_t launch_loss(const LossTile& t, int config) {
    if (t.dtype == MIGEMM_F32)
        return config == 3   ? launch_loss_tile<float, 3>(t)
               : config == 2 ? launch_loss_tile<float, 2>(t)
               : config == 1 ? launch_loss_tile<float, 1>(t)
                             : launch_loss_tile<float, 0>(t);
#define MIGEMM_LOSS(E)                                        \
    switch (config) {                                         \
        case 0: return launch_loss_tile<E, 0>(t);             \
        case 1: return launch_loss_tile<E, 1>(t);             \
        case 2: return launch_loss_tile<E, 2>(t);             \
        default: return launch_loss_tile<E, 3>(t);            \
    }
    if (t.dtype == MIGEMM_F16) {
        MIGEMM_LOSS(_Float16)
    }
    MIGEMM_LOSS(bf16_t)
#undef MIGEMM_LOSS
}

namespace {

constexpr int64_t kMaxTop = 1024;
// Entries of dz in one piece of the vocabulary: 2^28, 512 MiB in 16 bits.
constexpr int64_t kPieceEntries = int64_t(1) << 28;
// Widest piece: dz's rows stay within the direct kernels' offset limit (2^21).
constexpr int64_t kPieceMax = int64_t(1) << 20;
// Multiply-adds below which a launch more costs more than it saves.
constexpr double kSmallWork = 2147483648.0;  // 2^31
// Multiply-adds of one product from which whole tiles pay (whole_tiles).
constexpr double kWholeWork = 68719476736.0;  // 2^36

int64_t round_up(int64_t x, int64_t to) { return ceil_div(x, to) * to; }

// How dx = dz W (T x cols, k deep) is summed where one piece holds the whole
// vocabulary: slices of k on `config`'s tiles, or (slices 0) the library's product.
struct LossSlices {
    int config = 0, slices = 0;
};
// Each tile takes as many slices as make 256 workgroups; the tile is the one whose
// k-tiles (0.27, 0.62, 1.78 us on 64x64, 128x128, 256x256; 0.19 where two workgroups
// of 64x64 share a CU), prologue and output step, and slices' sums written and read
// cost least, and the library's product is taken where that one has a single slice.
// us for dz and then dx, BF16, 64 / 128 / 256, and the library's product (at most 16
// slices, and a launch more to convert its sums): 1 x 96923 x 256 30 / 34 / - / 67, 64
// x 8000 x 1024 20 / 25 / - / 27, 200 x 20000 x 2048 78 / 70 / 84 / 74, 3000 x 32000 x
// 2048 - / - / 725 / 889, 800 x 600 x 4096 - / - / 54 / 40; FP32 15 x 20986 x 320 34 /
// 44 / - / 49.  256x256 slices run the ping-pong schedule where sizes are whole tiles
// and k-tiles (1000 x 128255 x 4096, dx alone: 755 against 854).
LossSlices dx_slices(int dtype, int64_t T, int64_t cols, int64_t k) {
    const bool whole = T % 256 == 0 && cols % 256 == 0 && k % 64 == 0;
    const double step[] = {0.27, 0.62, whole ? 1.6 : 1.78}, once[] = {2.0, 5.0, 10.0};
    LossSlices best;
    double least = 1e30;
    for (int c = 0; c < (dtype == MIGEMM_F32 ? 2 : 3); ++c) {
        if (c == 2 && k % 8 != 0) break;  // (its partial k-tile takes whole chunks)
        const int64_t b = int64_t(64) << c, tiles = ceil_div(T, b) * ceil_div(cols, b);
        const int64_t ks = splitk_slice(k, tiles <= 128 ? 256 / tiles : 1);
        const int64_t slices = ceil_div(k, ks), rounds = ceil_div(tiles, 256);
        const double rate = c == 0 && rounds > 1 ? 0.19 : step[c];
        const double cost = static_cast<double>(rounds * (ks / 64)) * rate + once[c] +
                            (slices < 2 ? 0.0 : static_cast<double>(slices * T * cols) * 8.0 / 3e6);
        if (cost < least) {
            least = cost;
            best.config = c == 0 && dtype == MIGEMM_F32 && T <= 32 ? 3 : c == 2 && whole ? 3 : c;
            best.slices = slices < 2 ? 0 : static_cast<int>(slices);
        }
    }
    return best;
}

// What one call copies and where its scratch arrays lie (byte offsets into the
// workspace, 256-byte aligned).
struct Plan {
    bool copy_x = false, copy_w = false, wide = false, small_w = false;
    int64_t depth = 0;   // k of the logits' product
    int64_t ld_copy = 0; // leading dimension of copies
    int64_t bytes = 0;
    int64_t x = 0, w = 0;
    // rows of the products whose other side is the vocabulary: T, or whole tiles of it
    int64_t rows = 0;
    bool band = false;  // the vocabulary past whole tiles is a step of its own
    int64_t twin = 0;   // kTwin where dz is kept as two terms
    // forward
    int64_t part = 0, chunks = 0;
    // backward
    int64_t t_pad = 0, x_rows = 0, piece = 0, pieces = 0, ldz = 0, cols = 0;
    bool dx_acc = false;
    LossSlices dx;
    int dx_slabs = 0;  // dx.slices, and one for the band
    int64_t info = 0, factor = 0, dz = 0, acc_x = 0, tp = 0, gemm = 0, gemm_bytes = 0;
    int64_t take(int64_t n) {
        const int64_t at = bytes;
        bytes += round_up(n, 256);
        return at;
    }
};

// Rows that the direct kernels read in place: 16-byte aligned, in whole chunks,
// within their offset limit.
bool rows_ok(const void* p, int64_t ld, int64_t epc) {
    return aligned16(p) && ld % epc == 0 && ld < (int64_t(1) << 21);
}

// The variant and configuration of dx's product (T x cols, k deep) where the vocabulary
// takes several pieces, -1 the selection's.  Where 128x128 tiles just make a round of 256
// workgroups the selection walks all of k on them; a long k is better cut into slices on
// the 256x256 tile (dz and dx of 2048 x 200000 x 2048 BF16: 2752 us against 3176; 8192 x
// 40001 x 512: 868 against 914).
struct Choice {
    int variant, config;
};
Choice dx_choice(int dtype, int64_t T, int64_t cols, int64_t k) {
    auto tiles = [&](int64_t b) { return ceil_div(T, b) * ceil_div(cols, b); };
    if (dtype != MIGEMM_F32 && k % 8 == 0 && k >= 16384 && tiles(256) <= 64 && tiles(128) >= 256)
        return {MIGEMM_MFMA16, 17};
    return {-1, -1};
}

// The forward statistics' chunks of n columns.
int64_t chunks_of(const LossShape& s, int64_t n) { return ceil_div(n, s.bn) * (s.bn / s.chunk); }

// Whether ragged sizes are brought to whole 256x256 tiles, for the ping-pong schedule:
// x copied to whole tiles of rows, the vocabulary past whole tiles as a band of its
// own, which costs a copy of x and a small launch or three.  Forward and backward
// pass, us, without and with (BF16): 8190 x 32003 x 4096 1722 / 1495, 5170 / 4544; 2040 x
// 32001 x 2048 246 / 217, 747 / 687; 500 x 128255 x 2048 260 / 237, 923 / 835; 8000 x
// 8001 x 1024 149 / 151, 443 / 457; 1500 x 20000 x 768 60 / 65, 168 / 185.
bool whole_tiles(const LossArgs& a, int64_t depth) {
    return loss_shape(a.dtype, a.T, a.V, depth).bn == 256 && depth % 64 == 0 && a.V >= 512 &&
           static_cast<double>(a.T * a.V) * static_cast<double>(a.D) >= kWholeWork;
}

// Columns [v0, end) of the vocabulary that a step takes: up to `piece`, and whole
// tiles and what is left past them as steps of their own where `band` is set.
int64_t step_of(int64_t v0, int64_t end, int64_t piece, bool band) {
    const int64_t n = end - v0 < piece ? end - v0 : piece;
    return band && n > 256 ? n - n % 256 : n;
}

// The tiles of a product with n columns of the vocabulary, and the rows they run
// over: p.rows where they are 256 high.
struct Tiling {
    int64_t rows;
    LossShape shape;
};
// All passes have to form the same bits of a logit.  Every tile adds k in the same order,
// except that 256x256 ones take a partial k-tile first (head_of): where k ends inside a
// k-tile, all steps follow the whole vocabulary's choice.
Tiling tiling(const LossArgs& a, const Plan& p, int64_t n) {
    if (a.dtype != MIGEMM_F32 && p.depth % 64 != 0) n = a.V;
    const LossShape s = loss_shape(a.dtype, p.rows, n, p.depth);
    return s.bn == 256 || p.twin ? Tiling{p.rows, s} : Tiling{a.T, loss_shape(a.dtype, a.T, n, p.depth)};
}

// Elements before k = 0 in the first 32-deep slab of the logits' product.
int head_of(const LossArgs& a, int64_t depth) {
    const bool head = a.dtype != MIGEMM_F32 && depth % 64 != 0 &&
                      loss_shape(a.dtype, a.T, a.V, depth).config == 2;
    return head ? static_cast<int>((32 - depth % 32) % 32) : 0;
}

Plan make_plan(const LossArgs& a, bool backward) {
    Plan p;
    const int64_t es = elem_size(a.dtype), epc = 16 / es;
    const bool whole = a.D % epc == 0;
    p.ld_copy = round_up(a.D, 64);
    p.copy_w = !whole || !rows_ok(a.W, a.ldw, epc);
    // the backward pass always copies x: its rows without a loss become 0, so
    // that whatever they hold (NaN from a masked position) stays out of dw; where w is
    // copied x is in either pass, so that both see one depth
    p.copy_x = backward || p.copy_w || !rows_ok(a.X, a.ldx, epc);
    p.depth = p.copy_w ? p.ld_copy : a.D;
    p.rows = a.T;
    if (whole_tiles(a, p.depth)) {
        p.rows = round_up(a.T, 256);
        p.copy_x = p.copy_x || p.rows != a.T;
        p.band = a.V % 256 != 0;
    }
    if (p.copy_w) p.w = p.take(round_up(a.V, 64) * p.ld_copy * es);
    if (!backward) {
        if (p.copy_x) p.x = p.take(p.rows * p.ld_copy * es);
        for (int64_t v0 = 0, n; v0 < a.V; v0 += n) {
            n = step_of(v0, a.V, a.V, p.band);
            p.chunks += chunks_of(tiling(a, p, n).shape, n);
        }
        p.part = p.take(p.rows * p.chunks * static_cast<int64_t>(sizeof(RowStat)));
        return p;
    }
    if (a.dtype != MIGEMM_F32 && a.T <= kTwin) {
        p.twin = kTwin;
        p.rows = 2 * kTwin;
    }
    p.t_pad = round_up(a.T, a.dtype == MIGEMM_F32 ? 32 : 64);  // whole k-tiles of dw
    p.x_rows = p.rows > p.t_pad ? p.rows : p.t_pad;
    p.x = p.take(p.x_rows * p.ld_copy * es);
    const int64_t fit = kPieceEntries / p.x_rows / 256 * 256;
    p.piece = fit < 2048 ? 2048 : fit > kPieceMax ? kPieceMax : fit;
    if (p.piece > a.V) p.piece = a.V;
    p.pieces = ceil_div(a.V, p.piece);
    p.ldz = round_up(p.piece, 64);
    // 16-bit dz holds a factor that the gradients' output steps take out again; and
    // rows that end inside a chunk are computed as whole ones
    p.wide = a.dtype != MIGEMM_F32 || !whole;
    p.cols = whole ? a.D : p.ld_copy;
    // A small dw takes one launch (launch_grad): the products' own selection splits
    // ragged bands off, which costs up to two launches more and pays only where the
    // product outweighs them.
    p.small_w = static_cast<double>(p.piece) * static_cast<double>(p.cols) *
                    static_cast<double>(p.t_pad) < kSmallWork;
    if (p.pieces == 1) {
        p.dx = dx_slices(a.dtype, p.rows, p.cols, step_of(0, a.V, p.piece, p.band));
        p.dx_slabs = p.dx.slices > 0 ? p.dx.slices + p.band : 0;
    }
    p.dx_acc = p.wide || p.dx.slices > 0;
    p.info = p.take(round_up(a.T, 256) * static_cast<int64_t>(sizeof(LossRow)));
    p.factor = p.take(256);
    p.dz = p.take(p.x_rows * p.ldz * es);
    if (p.dx_acc) p.acc_x = p.take((p.dx_slabs > 0 ? p.dx_slabs : 1) * p.rows * p.cols * 4);
    if (a.top) p.tp = p.take(a.T * a.top * 4);
    // what the two products ask for, for a full piece and the last one (their
    // operands are aligned; NULL stands for that)
    const int64_t dx_rows = p.dx_acc ? p.rows : a.T;
    for (int64_t v0 = 0, n; v0 < a.V; v0 += n) {
        n = step_of(v0, a.V, p.piece, p.band);
        int64_t b = 0;
        const Choice c = dx_choice(a.dtype, dx_rows, p.cols, n);
        if (p.dx.slices == 0 &&
            workspace_bytes(c.variant, c.config, MIGEMM_OP_N, MIGEMM_OP_N, dx_rows, p.cols, n,
                            a.dtype, nullptr, p.ldz, nullptr, p.copy_w ? p.ld_copy : a.ldw, &b,
                            true) == MIGEMM_OK &&
            b > p.gemm_bytes)
            p.gemm_bytes = b;
        if (!p.wide && !p.small_w &&
            workspace_bytes(-1, -1, MIGEMM_OP_T, MIGEMM_OP_N, n, p.cols, p.t_pad, a.dtype, nullptr,
                            p.ldz, nullptr, p.ld_copy, &b, true) == MIGEMM_OK &&
            b > p.gemm_bytes)
            p.gemm_bytes = b;
    }
    p.gemm = p.take(p.gemm_bytes);
    return p;
}

char* at(void* ws, int64_t offset) { return static_cast<char*>(ws) + offset; }

// X or W as the products read them: in place, or the copy made here.
hipError_t operand(const LossArgs& a, bool copy, const void* src, int64_t lds, int64_t rows,
                   int64_t rows_out, const Plan& p, void* to, const void** out, int64_t* ld) {
    *out = copy ? to : src;
    *ld = copy ? p.ld_copy : lds;
    if (!copy) return hipSuccess;
    return launch_pad_copy(a.dtype, rows, a.D, src, lds, to, rows_out, p.ld_copy, a.stream);
}

int forward(const LossArgs& a, float* loss, double* lse, void* ws) {
    const Plan p = make_plan(a, false);
    const int64_t es = elem_size(a.dtype);
    const void *x, *w;
    int64_t ldx, ldw;
    int st = hip_status(operand(a, p.copy_x, a.X, a.ldx, a.T, p.rows, p, at(ws, p.x), &x,
                                &ldx));
    if (st != MIGEMM_OK) return st;
    st = hip_status(operand(a, p.copy_w, a.W, a.ldw, a.V, round_up(a.V, 64), p, at(ws, p.w), &w,
                            &ldw));
    if (st != MIGEMM_OK) return st;
    RowStat* const part = reinterpret_cast<RowStat*>(at(ws, p.part));
    LseOut out{};
    out.part = part;
    out.chunks = p.chunks;
    out.scale = kLog2e / a.tau;
    for (int64_t v0 = 0, n; v0 < a.V; v0 += n) {
        n = step_of(v0, a.V, a.V, p.band);
        const Tiling tl = tiling(a, p, n);
        const LossTile t{tl.rows, n, p.depth, a.dtype, x, ldx,
                         static_cast<const char*>(w) + v0 * ldw * es, ldw, a.stream, &out,
                         nullptr, nullptr};
        st = hip_status(launch_loss(t, tl.shape.config));
        if (st != MIGEMM_OK) return st;
        out.part += chunks_of(tl.shape, n);
    }
    return hip_status(launch_loss_rows(a, x, ldx, w, ldw, p.depth, head_of(a, p.depth), part,
                                       p.chunks, loss, lse));
}

template <typename E>
hipError_t launch_dz(const LossArgs& a, const Plan& p, const void* x, const void* w, int64_t ldw,
                     int64_t v0, int64_t n, void* ws, const float* factor) {
    DzOut<E> out{};
    out.dz = reinterpret_cast<E*>(at(ws, p.dz));
    out.ldz = round_up(n, 64);
    out.rows = p.x_rows;
    out.v0 = v0;
    out.info = reinterpret_cast<const LossRow*>(at(ws, p.info));
    out.factor = factor;
    out.scale = kLog2e / a.tau;
    out.twin = p.twin ? p.twin : kMaxDim;
    const Tiling tl = tiling(a, p, n);
    const LossTile t{tl.rows, n, p.depth, a.dtype, x, p.ld_copy, w, ldw, a.stream, nullptr, &out,
                     nullptr};
    return launch_loss(t, tl.shape.config);
}

// dw's rows of one piece, through the factor and the column limit.  Columns past
// whole 256-wide tiles, where few, take narrow tiles of their own: a 256-wide one
// for eight columns would cost as much as one for 256.
template <typename E>
hipError_t launch_grad(const LossArgs& a, const Plan& p, const void* dz, int64_t ldz,
                       const void* x, int64_t n, const float* factor, void* dw, int64_t lddw) {
    GradOut<E> out{};
    out.grad = static_cast<E*>(dw);
    out.ldg = lddw;
    out.cols = a.D;
    out.factor = factor;
    out.nt = (lddw * sizeof(E)) % 128 == 0 && (reinterpret_cast<uintptr_t>(dw) & 127) == 0;
    LossTile t{n, p.cols, p.t_pad, a.dtype, dz, ldz, x, p.ld_copy, a.stream, nullptr, nullptr,
               &out};
    LossShape s = loss_shape(a.dtype, n, p.cols, p.t_pad);
    if (a.dtype == MIGEMM_F32 && s.config > 1) s = {0, 16, 64};  // (k is their row index)
    const int64_t rest = p.cols % 256;
    if (s.bn != 256 || p.cols < 256 || rest == 0 || rest > 64) return launch_loss(t, s.config);
    t.N -= rest;
    const hipError_t e = launch_loss(t, loss_shape(a.dtype, n, t.N, p.t_pad).config);
    if (e != hipSuccess) return e;
    t.B = static_cast<const E*>(x) + t.N;
    out.grad += t.N;
    out.cols -= t.N;
    t.N = rest;
    return launch_loss(t, 0);
}

int backward(const LossArgs& a, const double* lse, const float* grad, void* dx, int64_t lddx,
             void* dw, int64_t lddw, void* ws) {
    const Plan p = make_plan(a, true);
    const int64_t es = elem_size(a.dtype);
    LossRow* const info = reinterpret_cast<LossRow*>(at(ws, p.info));
    float* const tp = a.top ? reinterpret_cast<float*>(at(ws, p.tp)) : nullptr;
    void* const x = at(ws, p.x);
    void* const dz = at(ws, p.dz);
    void* const gws = p.gemm_bytes ? at(ws, p.gemm) : nullptr;
    const void* w;
    int64_t ldw;
#define MIGEMM_TRY(call)                                       \
    do {                                                       \
        const int st_ = (call);                                \
        if (st_ != MIGEMM_OK) return st_;                      \
    } while (0)
    MIGEMM_TRY(hip_status(operand(a, p.copy_w, a.W, a.ldw, a.V, round_up(a.V, 64), p, at(ws, p.w),
                                  &w, &ldw)));
    float* const factor =
        a.dtype == MIGEMM_F32 ? nullptr : reinterpret_cast<float*>(at(ws, p.factor));
    MIGEMM_TRY(hip_status(launch_loss_prepare(a, lse, grad, info, round_up(a.T, 256), x, p.x_rows,
                                              p.ld_copy, tp, a.top ? nullptr : factor, p.twin)));
    if (factor && a.top) MIGEMM_TRY(hip_status(launch_loss_factor(info, a.T, factor, a.stream)));
    const float* const inverse = factor ? factor + 1 : nullptr;
    const int64_t dx_rows = p.dx_acc ? p.rows : a.T;
    for (int64_t v0 = 0, n; v0 < a.V; v0 += n) {
        n = step_of(v0, a.V, p.piece, p.band);
        const int64_t ldz = round_up(n, 64);
        const char* const wp = static_cast<const char*>(w) + v0 * ldw * es;
        hipError_t e;
        if (a.dtype == MIGEMM_F32)
            e = launch_dz<float>(a, p, x, wp, ldw, v0, n, ws, factor);
        else if (a.dtype == MIGEMM_F16)
            e = launch_dz<_Float16>(a, p, x, wp, ldw, v0, n, ws, factor);
        else
            e = launch_dz<bf16_t>(a, p, x, wp, ldw, v0, n, ws, factor);
        MIGEMM_TRY(hip_status(e));
        if (a.top)
            MIGEMM_TRY(
                hip_status(launch_loss_scatter(a, info, tp, factor, dz, ldz, v0, v0 + n, p.twin)));
        if (dx && p.dx.slices > 0) {
            LossTile t{p.rows, p.cols, n, a.dtype, dz, ldz, wp, ldw, a.stream, nullptr, nullptr,
                       nullptr};
            t.sums = reinterpret_cast<float*>(at(ws, p.acc_x));
            t.slices = p.dx.slices;
            if (v0 > 0) {  // the band: the last slab
                t.sums += p.dx.slices * p.rows * p.cols;
                t.slices = 1;
            }
            MIGEMM_TRY(hip_status(launch_loss(t, v0 > 0 ? 1 : p.dx.config)));
        } else if (dx) {
            void* const c = p.dx_acc ? at(ws, p.acc_x) : dx;
            const int ct = p.dx_acc ? MIGEMM_F32 : a.dtype;
            const Choice ch = dx_choice(a.dtype, dx_rows, p.cols, n);
            MIGEMM_TRY(run_gemm(ch.variant, ch.config, MIGEMM_OP_N, MIGEMM_OP_N, dx_rows, p.cols,
                                n, a.dtype, dz, ldz, wp, ldw, 1.0f, v0 ? 1.0f : 0.0f, ct, c,
                                p.dx_acc ? p.cols : lddx, gws, p.gemm_bytes, a.stream, true));
        }
        if (dw) {
            char* const to = static_cast<char*>(dw) + v0 * lddw * es;
            if (!p.wide && !p.small_w)
                MIGEMM_TRY(run_gemm(-1, -1, MIGEMM_OP_T, MIGEMM_OP_N, n, p.cols, p.t_pad, a.dtype,
                                    dz, ldz, x, p.ld_copy, 1.0f, 0.0f, a.dtype, to, lddw, gws,
                                    p.gemm_bytes, a.stream, true));
            else if (a.dtype == MIGEMM_F32)
                MIGEMM_TRY(hip_status(launch_grad<float>(a, p, dz, ldz, x, n, inverse, to, lddw)));
            else if (a.dtype == MIGEMM_F16)
                MIGEMM_TRY(
                    hip_status(launch_grad<_Float16>(a, p, dz, ldz, x, n, inverse, to, lddw)));
            else
                MIGEMM_TRY(
                    hip_status(launch_grad<bf16_t>(a, p, dz, ldz, x, n, inverse, to, lddw)));
        }
    }
    if (dx && p.dx_acc)
        MIGEMM_TRY(hip_status(launch_join(a.dtype, a.T, a.D,
                                          reinterpret_cast<float*>(at(ws, p.acc_x)), p.cols,
                                          (p.twin ? p.twin : p.rows) * p.cols,
                                          (p.dx_slabs > 0 ? p.dx_slabs : 1) * (p.twin ? 2 : 1),
                                          inverse, dx, lddx, a.stream)));
#undef MIGEMM_TRY
    return MIGEMM_OK;
}

bool ld_ok(int64_t ld, int64_t cols) { return ld >= (cols > 1 ? cols : 1) && ld < kMaxLd; }

// Sizes and leading dimensions that both passes share.
bool shape_ok(const LossArgs& a, bool kd) {
    if (!known_dtype(a.dtype) || a.T < 0 || a.V < 1 || a.D < 1 || a.T > kMaxDim || a.V > kMaxDim ||
        a.D > kMaxDim || !ld_ok(a.ldx, a.D) || !ld_ok(a.ldw, a.D))
        return false;
    // copies and the products' offsets: rows of fewer than 2^21 - 64 elements
    if (a.D > (int64_t(1) << 21) - 64) return false;
    // a launch holds fewer than 2^32 threads: 256 for each row, 512 for each tile of
    // the logits, which are 256x256 (FP32: 128x128) unless T is at most 128 (64 for
    // 64x64) or they are few (fewer than 2^23, loss_shape)
    if (a.T > (int64_t(1) << 23) - 256 || a.V > int64_t(1) << 28 ||
        a.T * a.V > int64_t(1) << (a.dtype == MIGEMM_F32 ? 36 : 38))
        return false;
    return !kd || (a.top >= 1 && a.top <= kMaxTop);
}

bool kd_ok(const LossArgs& a) {
    return known_dtype(a.t_dtype) && ld_ok(a.ldt, a.top) && ld_ok(a.ldi, a.top) &&
           ld_ok(a.lds, a.top) && a.tau >= 0x1p-60f && a.tau <= 0x1p60f;  // tau^2 is finite
}

struct Range {
    uintptr_t lo, hi;
};

// Adds the range of a rows x cols array; false for NULL or one past the address space.
bool add(Range* list, int& count, const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
    Range r;
    if (!p || !extent(p, rows, cols, ld, es, r.lo, r.hi)) return false;
    list[count++] = r;
    return true;
}

// No output meets an input or another output.
bool disjoint(const Range* in, int n_in, const Range* out, int n_out) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i].lo, out[i].hi, in[j].lo, in[j].hi)) return false;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].lo, out[i].hi, out[j].lo, out[j].hi)) return false;
    }
    return true;
}

int check_workspace(const Plan& p, const void* ws, int64_t ws_bytes) {
    if (ws_bytes < 0) return MIGEMM_ERR_INVALID_ARG;
    if (p.bytes == 0) return MIGEMM_OK;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % kWorkspaceAlign != 0 || ws_bytes < p.bytes)
        return MIGEMM_ERR_WORKSPACE;
    return MIGEMM_OK;
}

// The inputs of a pass (T >= 1): x, w and what names the targets.
bool add_inputs(const LossArgs& a, Range* in, int& n) {
    const int es = elem_size(a.dtype);
    if (!add(in, n, a.X, a.T, a.D, a.ldx, es) || !add(in, n, a.W, a.V, a.D, a.ldw, es))
        return false;
    if (a.top == 0) return add(in, n, a.target, 1, a.T, a.T, 8);
    return add(in, n, a.t_logits, a.T, a.top, a.ldt, elem_size(a.t_dtype)) &&
           add(in, n, a.t_index, a.T, a.top, a.ldi, 8);
}

int run_forward(const LossArgs& a, float* loss, double* lse, void* ws, int64_t ws_bytes) {
    if (a.T == 0) return ws_bytes < 0 ? MIGEMM_ERR_INVALID_ARG : MIGEMM_OK;
    Range in[8], out[8];
    int n_in = 0, n_out = 0;
    if (!add_inputs(a, in, n_in) || !add(out, n_out, loss, 1, a.T, a.T, 4) ||
        !add(out, n_out, lse, 1, a.T, a.T, 8))
        return MIGEMM_ERR_INVALID_ARG;
    if (a.top && !add(out, n_out, a.student, a.T, a.top, a.lds, 4)) return MIGEMM_ERR_INVALID_ARG;
    const Plan p = make_plan(a, false);
    const int st = check_workspace(p, ws, ws_bytes);
    if (st != MIGEMM_OK) return st;
    if (p.bytes > 0 && !add(out, n_out, ws, 1, p.bytes, p.bytes, 1)) return MIGEMM_ERR_INVALID_ARG;
    if (!disjoint(in, n_in, out, n_out)) return MIGEMM_ERR_INVALID_ARG;
    return forward(a, loss, lse, ws);
}

int run_backward(const LossArgs& a, const double* lse, const float* grad, void* dx, int64_t lddx,
                 void* dw, int64_t lddw, void* ws, int64_t ws_bytes) {
    if ((dx && !ld_ok(lddx, a.D)) || (dw && !ld_ok(lddw, a.D)) || ws_bytes < 0)
        return MIGEMM_ERR_INVALID_ARG;
    const int es = elem_size(a.dtype);
    if (a.T == 0) {
        // no rows: dw = 0
        if (!dw) return MIGEMM_OK;
        uintptr_t lo, hi;
        if (!extent(dw, a.V, a.D, lddw, es, lo, hi)) return MIGEMM_ERR_INVALID_ARG;
        return run_gemm(-1, -1, MIGEMM_OP_N, MIGEMM_OP_N, a.V, a.D, 0, a.dtype, nullptr, 1,
                        nullptr, a.D, 1.0f, 0.0f, a.dtype, dw, lddw, nullptr, 0, a.stream);
    }
    Range in[8], out[8];
    int n_in = 0, n_out = 0;
    if (!add_inputs(a, in, n_in) || !add(in, n_in, lse, 1, a.T, a.T, 8) ||
        !add(in, n_in, grad, 1, a.T, a.T, 4))
        return MIGEMM_ERR_INVALID_ARG;
    if (a.top && !add(in, n_in, a.student, a.T, a.top, a.lds, 4)) return MIGEMM_ERR_INVALID_ARG;
    if (dx && !add(out, n_out, dx, a.T, a.D, lddx, es)) return MIGEMM_ERR_INVALID_ARG;
    if (dw && !add(out, n_out, dw, a.V, a.D, lddw, es)) return MIGEMM_ERR_INVALID_ARG;
    const Plan p = make_plan(a, true);
    const int st = check_workspace(p, ws, ws_bytes);
    if (st != MIGEMM_OK) return st;
    if (!add(out, n_out, ws, 1, p.bytes, p.bytes, 1)) return MIGEMM_ERR_INVALID_ARG;
    if (!disjoint(in, n_in, out, n_out)) return MIGEMM_ERR_INVALID_ARG;
    if (!dx && !dw) return MIGEMM_OK;
    return backward(a, lse, grad, dx, lddx, dw, lddw, ws);
}

LossArgs layer(int64_t T, int64_t V, int64_t D, int dtype, const void* X, int64_t ldx,
               const void* W, int64_t ldw, void* stream) {
    LossArgs a{};
    a.T = T;
    a.V = V;
    a.D = D;
    a.dtype = dtype;
    a.X = X;
    a.ldx = ldx;
    a.W = W;
    a.ldw = ldw;
    a.tau = 1.0f;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

}  // namespace
}  // namespace migemm

using namespace migemm;

extern "C" {

int migemm_linear_loss_workspace_size(int backward, int64_t T, int64_t V, int64_t D, int64_t top,
                                      int dtype, const void* X, int64_t ldx, const void* W,
                                      int64_t ldw, int64_t* bytes) {
    LossArgs a = layer(T, V, D, dtype, X, ldx, W, ldw, nullptr);
    a.top = top;
    if (!bytes || !shape_ok(a, top != 0)) return MIGEMM_ERR_INVALID_ARG;
    *bytes = T == 0 ? 0 : make_plan(a, backward != 0).bytes;
    return MIGEMM_OK;
}

int migemm_linear_ce_forward(int64_t T, int64_t V, int64_t D, int dtype, const void* X,
                             int64_t ldx, const void* W, int64_t ldw, const int64_t* target,
                             int64_t ignore_index, float* loss, double* lse, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    LossArgs a = layer(T, V, D, dtype, X, ldx, W, ldw, stream);
    a.target = target;
    a.ignore = ignore_index;
    if (!shape_ok(a, false)) return MIGEMM_ERR_INVALID_ARG;
    return run_forward(a, loss, lse, workspace, workspace_bytes);
}

int migemm_linear_ce_backward(int64_t T, int64_t V, int64_t D, int dtype, const void* X,
                              int64_t ldx, const void* W, int64_t ldw, const int64_t* target,
                              int64_t ignore_index, const double* lse, const float* grad, void* dX,
                              int64_t lddx, void* dW, int64_t lddw, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    LossArgs a = layer(T, V, D, dtype, X, ldx, W, ldw, stream);
    a.target = target;
    a.ignore = ignore_index;
    if (!shape_ok(a, false)) return MIGEMM_ERR_INVALID_ARG;
    return run_backward(a, lse, grad, dX, lddx, dW, lddw, workspace, workspace_bytes);
}

int migemm_linear_kd_forward(int64_t T, int64_t V, int64_t D, int64_t top, int dtype,
                             const void* X, int64_t ldx, const void* W, int64_t ldw,
                             int teacher_dtype, const void* teacher, int64_t ldt,
                             const int64_t* index, int64_t ldi, float temperature, float* loss,
                             double* lse, float* student, int64_t lds, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    LossArgs a = layer(T, V, D, dtype, X, ldx, W, ldw, stream);
    a.top = top;
    a.t_dtype = teacher_dtype;
    a.t_logits = teacher;
    a.ldt = ldt;
    a.t_index = index;
    a.ldi = ldi;
    a.tau = temperature;
    a.student = student;
    a.lds = lds;
    if (!shape_ok(a, true) || !kd_ok(a)) return MIGEMM_ERR_INVALID_ARG;
    return run_forward(a, loss, lse, workspace, workspace_bytes);
}

int migemm_linear_kd_backward(int64_t T, int64_t V, int64_t D, int64_t top, int dtype,
                              const void* X, int64_t ldx, const void* W, int64_t ldw,
                              int teacher_dtype, const void* teacher, int64_t ldt,
                              const int64_t* index, int64_t ldi, float temperature,
                              const double* lse, const float* student, int64_t lds,
                              const float* grad, void* dX, int64_t lddx, void* dW, int64_t lddw,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    LossArgs a = layer(T, V, D, dtype, X, ldx, W, ldw, stream);
    a.top = top;
    a.t_dtype = teacher_dtype;
    a.t_logits = teacher;
    a.ldt = ldt;
    a.t_index = index;
    a.ldi = ldi;
    a.tau = temperature;
    a.student = const_cast<float*>(student);
    a.lds = lds;
    if (!shape_ok(a, true) || !kd_ok(a)) return MIGEMM_ERR_INVALID_ARG;
    return run_backward(a, lse, grad, dX, lddx, dW, lddw, workspace, workspace_bytes);
}

}  // extern "C"
