// linear_loss_part.hip -- the products of the output-layer losses: the direct
// kernels of mfma16_direct.hpp with the output steps of linear_loss.hpp.  Built
// once per (element type, configuration): the build passes MIGEMM_PART_E and
// MIGEMM_PART_C, the configuration's index as loss_shape names it.
#include "linear_loss.hpp"

namespace migemm {
namespace {

// <E, BM, BN, WM, WN, MF, STAGES, BK, GM, SCHED, FLAGS>, the tiles of the products'
// own tables (mfma16_part.hip, regtile_mfma_part.hip)
template <typename E, int C> struct Tile;
template <typename E> struct Tile<E, 0> {  // 64x64, K in whole chunks
    using Cfg = DirectCfg<E, 64, 64, 2, 4, 16, 4, 64, 8, 0, 56>;
};
template <typename E> struct Tile<E, 1> {  // 128x128, K in whole chunks
    using Cfg = DirectCfg<E, 128, 128, 2, 4, 16, 4, 64, 4, 2, 48>;
};
template <typename E> struct Tile<E, 2> {  // 256x256, K in whole chunks
    using Cfg = DirectCfg<E, 256, 256, 2, 4, 16, 2, 64, 4, 2, 92>;
};
template <typename E> struct Tile<E, 3> {  // 256x256 ping-pong: whole tiles and k-tiles
    using Cfg = DirectCfg<E, 256, 256, 2, 4, 16, 2, 64, 4, 4, 20>;
};
template <> struct Tile<float, 0> {
    using Cfg = DirectCfg<float, 64, 64, 2, 4, 16, 4, 32, 8, 2, 48>;
};
template <> struct Tile<float, 1> {
    using Cfg = DirectCfg<float, 128, 128, 2, 4, 16, 4, 32, 4, 2, 48>;
};
template <> struct Tile<float, 2> {  // 64x32 on four waves: twice the workgroups
    using Cfg = DirectCfg<float, 64, 32, 2, 2, 16, 4, 32, 8, 2, 48>;
};

template <> struct Tile<float, 3> {  // 32x64 on four waves, for up to 32 rows
    using Cfg = DirectCfg<float, 32, 64, 1, 4, 16, 4, 32, 8, 2, 48>;
};

template <class Cfg, bool TRANS, class Out>
hipError_t launch_with(const LossTile& t, const Out& out) {
    using E = typename Cfg::E;
    GemmArgs g{};
    g.ta = g.pad_a = TRANS;
    g.M = t.M;
    g.N = t.N;
    g.K = t.K;
    g.tb = !TRANS;
    g.A = t.A;
    g.lda = t.lda;
    g.B = t.B;
    g.ldb = t.ldb;
    g.stream = t.stream;
    if (!direct_fits<Cfg>(g)) return hipErrorInvalidValue;
    const int64_t tm = ceil_div(g.M, Cfg::BM), tn = ceil_div(g.N, Cfg::BN);
    // (a launch holds fewer than 2^32 threads; loss_shape keeps within it)
    if (tm * tn > 0xffffffff / Cfg::NT) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(tm * tn)), block(Cfg::NT);
    const E* A = static_cast<const E*>(g.A);
    const E* B = static_cast<const E*>(g.B);
    const int itm = static_cast<int>(tm), itn = static_cast<int>(tn);
    if constexpr (TRANS) {
        if (g.K % Cfg::BK != 0) return hipErrorInvalidValue;  // K is padded to whole k-tiles
    } else {
        constexpr bool kTail = (Cfg::FLAGS & 32) != 0, kHead = (Cfg::FLAGS & 64) != 0;
        if ((kTail || kHead) && g.K % Cfg::BK != 0)
            return launch_kernel(
                g, mfma16_direct_kernel<Cfg, false, false, true, kTail, kHead, false, Out>, grid,
                block, g.M, g.N, g.K, A, g.lda, B, g.ldb, out, itm, itn);
    }
    return launch_kernel(
        g, mfma16_direct_kernel<Cfg, false, TRANS, !TRANS, false, false, false, Out>, grid, block,
        g.M, g.N, g.K, A, g.lda, B, g.ldb, out, itm, itn);
}

// Slices of dz W's k: workgroups of one tile and slice each (SPLITK of
// mfma16_direct.hpp), plain FP32 sums.
template <class Cfg>
hipError_t launch_slices(const LossTile& t) {
    using E = typename Cfg::E;
    GemmArgs g{};
    g.pad_a = true;
    g.M = t.M;
    g.N = t.N;
    g.K = t.K;
    g.A = t.A;
    g.lda = t.lda;
    g.B = t.B;
    g.ldb = t.ldb;
    g.stream = t.stream;
    constexpr bool kTail = (Cfg::FLAGS & 32) != 0, kHead = (Cfg::FLAGS & 64) != 0;
    const bool ragged = g.K % Cfg::BK != 0;
    if (!direct_fits<Cfg>(g) || (ragged && !kTail && (!kHead || g.K % (16 / sizeof(E)) != 0)))
        return hipErrorInvalidValue;
    if (Cfg::SCHED == 4 && (ragged || g.M % Cfg::BM != 0 || g.N % Cfg::BN != 0))
        return hipErrorInvalidValue;
    const int64_t tm = ceil_div(g.M, Cfg::BM), tn = ceil_div(g.N, Cfg::BN);
    if (tm * tn * t.slices > 0x7fffffff / Cfg::NT) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(tm * tn * t.slices)), block(Cfg::NT);
    const E* A = static_cast<const E*>(g.A);
    const E* B = static_cast<const E*>(g.B);
    const int itm = static_cast<int>(tm), itn = static_cast<int>(tn);
    const Epi out{t.sums, t.N, 1.0f, 0.0f, 0};
    if constexpr (kTail || kHead)
        if (ragged)
            return launch_kernel(
                g, mfma16_direct_kernel<Cfg, false, false, false, kTail, kHead, true>, grid,
                block, g.M, g.N, g.K, A, g.lda, B, g.ldb, out, itm, itn);
    return launch_kernel(g, mfma16_direct_kernel<Cfg, false, false, false, false, false, true>,
                         grid, block, g.M, g.N, g.K, A, g.lda, B, g.ldb, out, itm, itn);
}

}  // namespace

template <typename E, int C>
hipError_t launch_loss_tile(const LossTile& t) {
    using Cfg = typename Tile<E, C>::Cfg;
    if (t.lse) return launch_with<Cfg, false>(t, *t.lse);
    if (t.dz) return launch_with<Cfg, false>(t, *static_cast<const DzOut<E>*>(t.dz));
    // (a k-row image is at least 64 FP32 columns wide)
    if constexpr (Cfg::BM >= 64 && Cfg::BN >= 64)
        if (t.grad) return launch_with<Cfg, true>(t, *static_cast<const GradOut<E>*>(t.grad));
    if constexpr (Cfg::BN >= 64)
        if (t.slices > 0) return launch_slices<Cfg>(t);
    return hipErrorInvalidValue;
}

#if defined(MIGEMM_PART_E) && defined(MIGEMM_PART_C)
template hipError_t launch_loss_tile<MIGEMM_PART_E, MIGEMM_PART_C>(const LossTile&);
#else
#error "linear_loss_part.hip is built with MIGEMM_PART_E and MIGEMM_PART_C defined"
#endif

}  // namespace migemm
