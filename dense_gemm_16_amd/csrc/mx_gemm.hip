// mx_gemm.hip -- the product of two MXFP4 matrices (format: mx.hip) on the
// gfx950 matrix cores, FP32 sums.
//
// C = alpha A B + beta C with A (M x K) and B given transposed (N x K), both
// quantised along k.  v_mfma_scale_f32_16x16x128_f8f6f4 with both formats FP4
// takes, in lane (r + 16 g), the 32 elements k = 32 g .. 32 g + 31 of row r of a
// 16-row block: 16 bytes, one MXFP4 block, and that block's scale byte.  Every
// product of two elements is exact and the scales are powers of two, so the
// only roundings are those of the FP32 sums.
//
// k is counted in 16-byte chunks (blocks) below.  Rows past M or N are clamped
// to the last one (their outputs are never stored); chunks past K read as zero
// elements with scale byte 0, so whatever lies in a scale row's padding is
// not used.
//
// Three kernels:
// * mx_tile_kernel: tiles of C through LDS, ping-pong wave groups, for many tiles;
// * mx_deep_kernel: the same without turns and with more loads in flight, for few;
// * mx_rows_kernel: few rows of A, bound by reading B once.
#include "mfma16_direct.hpp"

namespace migemm {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

// c += A B for one 16 x 16 x 128 block: 16 bytes of elements per lane and
// operand, and one scale byte, byte SEL of sa and sb.
template <int SEL>
__device__ __forceinline__ void mfma_mx(f32x4& c, u32x4 a, u32x4 b, uint32_t sa, uint32_t sb) {
    const i32x4 ai = __builtin_bit_cast(i32x4, a), bi = __builtin_bit_cast(i32x4, b);
    const i32x8 a8 = __builtin_shufflevector(ai, ai, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 b8 = __builtin_shufflevector(bi, bi, 0, 1, 2, 3, -1, -1, -1, -1);
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        a8, b8, c, 4, 4, SEL, static_cast<int>(sa), SEL, static_cast<int>(sb));
}

// ------------------------------------------------------------------ tiles of C
//
// The ping-pong schedule of mfma16_direct.hpp (two groups of four waves take
// turns on each SIMD, one running a k-tile of matrix instructions while the other
// reads its next k-tile of fragments), for operands with k contiguous on both
// sides.  A k-tile is 128 bytes per row, 256 elements, 8 blocks.  What differs:
//
// * Scales.  Two k-tiles' scales of a row are 16 bytes, so every second k-tile a
//   direct load per 64 rows brings them into LDS as they lie in memory.  The
//   order of k within a sum is free as long as A and B agree, so lane group g
//   takes blocks 2 g and 2 g + 1 of the k-tile (in its first and second slab)
//   rather than g and 4 + g: its two scale bytes are then neighbours, one 2-byte
//   LDS read per fragment and k-tile, and the two instructions select the byte.
//   (Reading eight bytes and permuting g and 4 + g together costs twice the LDS
//   time and waits between reads.)
// * LDS.  Two stages of A, two and a half of B and two pairs of scales fill the 160
//   KiB of the 256 x 256 tile.  B moves in halves of the tile's columns, half h of
//   k-tile kt in slot (2 kt + h) mod 5.  While Y reads k-tile kt, four slots hold
//   k-tiles kt and kt + 1 and Y fills the fifth with the first half of kt + 2; once
//   it has read, X fills kt's first slot with the second half, and A's stage, in
//   its own reading turn: twelve loads of X's waves and four of Y's.  (With the
//   second half between Y's matrix instructions instead, or the scales first copied
//   into the order that the lanes read them in, 8192^3 took 260 to 263 us against
//   260 to 265.)
// * Ragged sizes run on the same kernel: every load's row is clamped on the
//   spot (the address arithmetic hides in the reading turn), and a last k-tile
//   that K ends inside (TAIL) has A's chunks past K and both operands' scales
//   past K zeroed in LDS once it has landed.
template <int B_> struct MxTile {
    static constexpr int BX = B_;                        // the tile is BX x BX
    static constexpr int WTM = BX / 2, WTN = BX / 4;     // a wave's part
    static constexpr int TM = WTM / 16, TN = WTN / 16;
    static constexpr int STAGE = BX * 128;               // one operand's k-tile
    static constexpr int HALF = STAGE / 2;
    static constexpr int A0 = 0, B0 = 2 * STAGE, S0 = B0 + 5 * HALF;
    static constexpr int SCALES = 2 * BX * 16;           // a pair of k-tiles, A's rows then B's
    static constexpr int LDS_BYTES = S0 + 2 * SCALES;
    static constexpr int PA = BX / 8 / 4;                // A's loads per X wave and k-tile
    static constexpr int PB = PA / 2;                    // loads per wave and half of B
    static constexpr int NS = 2 * BX / 64;               // scale loads per pair, over the X waves
    static constexpr int GM = 4;
    static_assert(LDS_BYTES <= 160 * 1024 && PB >= 1, "stages and scales fit");
};

// The output step of the tile kernels.  Every fragment read of the workgroup is
// done; each wave sends its accumulators (the tile's part at row mw, column nw),
// one 16-row block at a time, through LDS of its own, so that C is read (beta) and
// written 16 bytes per lane in whole row pieces.  The 16-byte chunk index of the
// block's rows is XORed by 4 (row >> 2), which spreads the accumulator writes over
// the banks.  CT: C's type; RD: beta != 0.  One branch picks the form, so the code
// that runs is short and straight.
template <class T>
__device__ __forceinline__ void mx_store(const MxArgs& p, const f32x4 (&acc)[T::TM][T::TN],
                                         MIGEMM_LDS char* lds, int wave, int lane, int64_t mw,
                                         int64_t nw) {
    constexpr int WTN = T::WTN, TM = T::TM, TN = T::TN;
    MIGEMM_LDS float* const scr = (MIGEMM_LDS float*)(lds + wave * (16 * WTN * 4));
    const Epi out = p.out;
    const int ar = lane % 16, ag = lane / 16;
    auto store = [&](auto ct_tag, auto rd_tag) __attribute__((always_inline)) {
        constexpr int CT = decltype(ct_tag)::value;
        constexpr bool RD = decltype(rd_tag)::value, HALF = CT != 0;
        constexpr int VE = HALF ? 8 : 4, ES = HALF ? 2 : 4, PIECES = WTN / VE;
        constexpr int kXor = (WTN / 4 - 1) & 12;  // chunks of FP32 in a row: move by whole blocks
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int c = 16 * j + ar;
                    scr[(4 * ag + r) * WTN + ((((c >> 2) ^ ((ag << 2) & kXor)) << 2) | (c & 3))] =
                        acc[i][j][r];
                }
            asm volatile("" : : : "memory");
#pragma unroll
            for (int q = 0; q < (16 * PIECES + kWave - 1) / kWave; ++q) {
                const int piece = lane + q * kWave, row = piece / PIECES, c0 = piece % PIECES * VE;
                if (16 * PIECES % kWave != 0 && piece >= 16 * PIECES) continue;
                const int64_t grow = mw + 16 * i + row, gcol = nw + c0;
                const int x4 = row & kXor;  // (row >> 2) << 2
                if (grow >= p.M || gcol >= p.N) continue;
                const int64_t idx = grow * out.ldc + gcol;
                if (gcol + VE <= p.N) {
                    char* const dst = static_cast<char*>(out.C) + idx * ES;
                    u32x4 old = {0u, 0u, 0u, 0u}, w = {0u, 0u, 0u, 0u};
                    if constexpr (RD) __builtin_memcpy(&old, dst, 16);
#pragma unroll
                    for (int h = 0; h < VE / 4; ++h) {
                        const f32x4 x = *(const MIGEMM_LDS f32x4*)(scr + row * WTN +
                                                                   4 * (((c0 >> 2) + h) ^ x4));
#pragma unroll
                        for (int e4 = 0; e4 < 4; ++e4) {
                            const int e = 4 * h + e4;
                            float prev = 0.0f;
                            if constexpr (RD && HALF) {
                                const uint32_t bits = (old[e / 2] >> (16 * (e % 2))) & 0xffffu;
                                prev = CT == 1 ? static_cast<float>(__builtin_bit_cast(
                                                     _Float16, static_cast<uint16_t>(bits)))
                                               : __uint_as_float(bits << 16);
                            } else if constexpr (RD) {
                                prev = __uint_as_float(old[e]);
                            }
                            const float res = RD ? fmaf(out.alpha, x[e4], out.beta * prev)
                                                 : out.alpha * x[e4];
                            if constexpr (HALF) {
                                const uint32_t b =
                                    CT == 1 ? static_cast<uint32_t>(__builtin_bit_cast(
                                                  uint16_t, static_cast<_Float16>(res)))
                                            : static_cast<uint32_t>(f32_to_bf16_bits(res));
                                w[e / 2] |= b << (16 * (e % 2));
                            } else {
                                w[e] = __float_as_uint(res);
                            }
                        }
                    }
                    if (p.whole_lines)
                        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(dst));
                    else
                        __builtin_memcpy(dst, &w, 16);  // one store, whatever the alignment
                } else {
                    // the last columns, an element at a time (a rolled loop keeps
                    // this small)
#pragma nounroll
                    for (int e = 0; e < VE; ++e)
                        if (gcol + e < p.N)
                            store_update<false>(
                                out, idx + e,
                                scr[row * WTN + 4 * (((c0 + e) >> 2) ^ x4) + ((c0 + e) & 3)],
                                RD ? load_prev(out, idx + e) : 0.0f);
                }
            }
            asm volatile("" : : : "memory");
        }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    using F32 = std::integral_constant<int, 0>;
    using F16 = std::integral_constant<int, 1>;
    using BF16 = std::integral_constant<int, 2>;
    if (out.beta != 0.0f) {
        if (out.c_dtype == 0)
            store(F32{}, Yes{});
        else if (out.c_dtype == 1)
            store(F16{}, Yes{});
        else
            store(BF16{}, Yes{});
    } else if (out.c_dtype == 0) {
        store(F32{}, No{});
    } else if (out.c_dtype == 1) {
        store(F16{}, No{});
    } else {
        store(BF16{}, No{});
    }
}

template <int BX, bool TAIL>
__global__ __launch_bounds__(512) void mx_tile_kernel(MxArgs p, int tiles_m, int tiles_n) {
    using T = MxTile<BX>;
    constexpr int TM = T::TM, TN = T::TN, PA = T::PA, PB = T::PB;
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];
    MIGEMM_LDS char* const lds = (MIGEMM_LDS char*)smem;
    const uint32_t lds_addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wx = wave & 3;
    const bool gx = wave < 4;
    const int wm0 = (wave >> 2) * T::WTM;

    int pm, pn;
    tile_coords<T::GM>(blockIdx.x, tiles_m, tiles_n, pm, pn);
    const int64_t m0 = static_cast<int64_t>(pm) * BX, n0 = static_cast<int64_t>(pn) * BX;
    const int chunks = static_cast<int>(p.K / 32), KT = (chunks + 7) / 8;
    const int left = TAIL ? chunks % 8 : 8;  // chunks in the last k-tile (TAIL: 1 to 7)

    // Element loads.  One covers eight rows; load q of wave wx rows 8 (wx + 4 q) +
    // lane / 8 of the image.  Block 2 g + s of a row lies at chunk (4 s + g) ^
    // swizzle: neighbouring lane groups, which share a cycle of a 16-byte LDS read,
    // then differ in the lowest chunk bit, as the swizzle needs (with the blocks in
    // order they differ in the next one and meet on the same banks).  The swizzle
    // depends on the row modulo 16, so a lane's block is the same in all its loads.
    const int r0 = 8 * wx + lane / 8;
    const int at_chunk = (lane % 8) ^ swz_a<8>(r0);
    const int logical = (at_chunk & 3) * 2 + (at_chunk >> 2);
    const uint32_t c16 = 16 * logical, c16_last = 16 * min(logical, left - 1);
    const int last_m = static_cast<int>(min(p.M - m0, int64_t(BX))) - 1;
    const int last_n = static_cast<int>(min(p.N - n0, int64_t(BX))) - 1;
    const uint32_t lda = static_cast<uint32_t>(p.lda), ldb = static_cast<uint32_t>(p.ldb);
    const uint8_t* const a_tile = p.A + m0 * p.lda;
    const uint8_t* const b_tile = p.B + n0 * p.ldb;
    // r: r0, made opaque once per k-tile, or the compiler keeps all of a wave's
    // row offsets in registers for the whole loop and spills others to memory
    auto load_a = [&](int kt, int q, int r) __attribute__((always_inline)) {
        const uint32_t row = min(r + 32 * q, last_m);
        dma16(lds_addr + T::A0 + (kt & 1) * T::STAGE + (wx + 4 * q) * 1024,
              a_tile + static_cast<int64_t>(kt) * 128,
              __umul24(row, lda) + (TAIL && kt == KT - 1 ? c16_last : c16));
    };
    // Load q of half h of B's k-tile kt, into slot `slot`.
    auto load_b = [&](int kt, int h, int slot, int q, int r) __attribute__((always_inline)) {
        const uint32_t row = min(r + 32 * q + h * (BX / 2), last_n);
        dma16(lds_addr + T::B0 + slot * T::HALF + (wx + 4 * q) * 1024,
              b_tile + static_cast<int64_t>(kt) * 128,
              __umul24(row, ldb) + (TAIL && kt == KT - 1 ? c16_last : c16));
    };
    // Scale load j (0 .. NS - 1) of pair `pair`: 64 rows of A, or of B.
    auto load_scales = [&](int pair, int j) __attribute__((always_inline)) {
        const bool of_a = j < T::NS / 2;
        int row = 64 * (of_a ? j : j - T::NS / 2) + lane;
        asm volatile("" : "+v"(row));
        const uint8_t* const base = of_a ? p.sa + m0 * p.ldsa : p.sb + n0 * p.ldsb;
        const uint32_t ld = static_cast<uint32_t>(of_a ? p.ldsa : p.ldsb);
        dma16(lds_addr + T::S0 + (pair & 1) * T::SCALES + j * 1024,
              base + static_cast<int64_t>(pair) * 16,
              __umul24(static_cast<uint32_t>(min(row, of_a ? last_m : last_n)), ld));
    };
    auto load_pair = [&](int pair) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < T::NS; j += 4)
            if (j + wx < T::NS) load_scales(pair, j + wx);
    };
    // Zeroes what the last k-tile's loads of this wave (group X) brought from past
    // K (each lane its own LDS slots), once they have landed: A's elements, so
    // that B's do not matter, and both operands' scales, so that no NaN one does.
    auto zero_tail = [&]() __attribute__((always_inline)) {
        if constexpr (TAIL) {
            if (logical >= left) {
#pragma unroll
                for (int q = 0; q < PA; ++q)
                    *(MIGEMM_LDS u32x4*)(lds + T::A0 + ((KT - 1) & 1) * T::STAGE +
                                         (wx + 4 * q) * 1024 + 16 * lane) = u32x4{0u, 0u, 0u, 0u};
            }
            const int pair = (KT - 1) / 2, valid = chunks - 16 * pair;  // 1 .. 15 bytes
#pragma unroll
            for (int j = 0; j < T::NS; j += 4)
                if (j + wx < T::NS) {
                    MIGEMM_LDS u32x4* const s = (MIGEMM_LDS u32x4*)(lds + T::S0 +
                        (pair & 1) * T::SCALES + (j + wx) * 1024 + 16 * lane);
                    u32x4 v = *s;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int n = valid - 4 * d;  // valid bytes of this word
                        v[d] &= n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                    }
                    *s = v;
                }
        }
    };

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // accumulators in AGPRs (see mfma16_direct.hpp)
    float agpr_hint = 0.0f;
    asm volatile("" : "+a"(agpr_hint));

    const int ar = lane % 16, ag = lane / 16;
    // this wave's columns: rows wb0 .. of half wh of B's image
    const int wh = wx >> 1, wb0 = (wx & 1) * T::WTN;
    u32x4 fa[2][TM], fb[2][TN];
    uint32_t sa[TM], sb[TN];
    auto wrap = [](int slot) { return slot >= 5 ? slot - 5 : slot; };
    // A k-tile of fragments and scales, its B half in slot `slot` + wh (mod 5),
    // interleaved with direct loads of k-tile kt + ahead: LOADS 1 (X) A, the second
    // half of B and, for an even k-tile, the scales; 2 (Y) the first half of B.
    auto read_ktile = [&](int kt, int slot, auto loads, int kt_load)
        __attribute__((always_inline)) {
        constexpr int LOADS = decltype(loads)::value;
        constexpr int kLoads = LOADS == 1 ? PA + PB : LOADS == 2 ? PB : 0;
        constexpr int kReads = 2 * (TM + TN);
        constexpr int EVERY = kLoads && kReads / kLoads > 0 ? kReads / kLoads : 1;
        int r = 0, q = 0;
        if (LOADS == 1 && (kt_load & 1) == 0) load_pair(kt_load >> 1);
        int r_now = r0;
        asm volatile("" : "+v"(r_now));
        auto one_load = [&]() __attribute__((always_inline)) {
            if constexpr (LOADS == 1) {
                // kt_load = kt + 1: its second half goes where the first half of
                // k-tile kt_load - 2 was
                if (q % 3 == 2)
                    load_b(kt_load, 1, wrap(slot + 3), q / 3, r_now);
                else
                    load_a(kt_load, q - q / 3, r_now);
            }
            if constexpr (LOADS == 2) load_b(kt_load, 0, wrap(slot + 4), q, r_now);
            ++q;
        };
        auto after_read = [&]() __attribute__((always_inline)) {
            ++r;
            if (LOADS && r % EVERY == 0 && q < kLoads) one_load();
        };
        int st = (kt & 1) * T::STAGE, sh = wrap(slot + wh) * T::HALF;
        int sc = T::S0 + ((kt >> 1) & 1) * T::SCALES + (kt & 1) * 8;
        asm("" : "+s"(st), "+s"(sc), "+s"(sh));
        const MIGEMM_LDS char* const ia = lds + T::A0 + st;
        const MIGEMM_LDS char* const ib = lds + T::B0 + sh;
        const MIGEMM_LDS char* const is = lds + sc;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int chunk = (4 * s + ag) ^ swz_a<8>(ar);
            auto read_a = [&](int i) __attribute__((always_inline)) {
                fa[s][i] = *(const MIGEMM_LDS u32x4*)(ia + (wm0 + ar) * 128 + chunk * 16 + i * 2048);
                if (s == 0)
                    sa[i] = *(const MIGEMM_LDS uint16_t*)(is + (wm0 + ar + 16 * i) * 16 + 2 * ag);
                after_read();
            };
            auto read_b = [&](int j) __attribute__((always_inline)) {
                fb[s][j] = *(const MIGEMM_LDS u32x4*)(ib + (wb0 + ar) * 128 + chunk * 16 + j * 2048);
                if (s == 0)
                    sb[j] = *(const MIGEMM_LDS uint16_t*)(
                        is + (BX + wx * T::WTN + ar + 16 * j) * 16 + 2 * ag);
                after_read();
            };
            read_a(0);
#pragma unroll
            for (int j = 0; j < TN; ++j) read_b(j);
#pragma unroll
            for (int i = 1; i < TM; ++i) read_a(i);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i >= q) one_load();
    };
    // A k-tile of matrix instructions; BAR 1 (X: its loads have landed, then the
    // barrier; 2: also zeroing what lies past K) or 3 (Y: the barrier), met a few
    // instructions before the last one as in mfma16_direct.hpp.
    constexpr int kMfma = 2 * TM * TN, kEarly = kMfma > 16 ? 8 : kMfma / 2;
    auto run_ktile = [&](auto bar) __attribute__((always_inline)) {
        constexpr int BAR = decltype(bar)::value;
        __builtin_amdgcn_sched_barrier(0);
        int n = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if (s == 0)
                        mfma_mx<0>(acc[i][j], fa[0][i], fb[0][j], sa[i], sb[j]);
                    else
                        mfma_mx<1>(acc[i][j], fa[1][i], fb[1][j], sa[i], sb[j]);
                    if (BAR && n == kMfma - 1 - kEarly) {
                        __builtin_amdgcn_sched_barrier(0);
                        __builtin_amdgcn_s_setprio(1);
                        if constexpr (BAR == 1) wait_then_barrier<0>();
                        if constexpr (BAR == 2) {
                            vm_wait<0>();
                            zero_tail();
                            lds_wait_then_barrier();
                        }
                        if constexpr (BAR == 3) lds_wait_then_barrier();
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    ++n;
                }
        __builtin_amdgcn_sched_barrier(0);
        if (BAR) __builtin_amdgcn_s_setprio(0);
    };
    using NoBarrier = std::integral_constant<int, 0>;
    using XBarrier = std::integral_constant<int, 1>;
    using XTail = std::integral_constant<int, TAIL ? 2 : 1>;
    using YBarrier = std::integral_constant<int, 3>;
    using NoLoads = std::integral_constant<int, 0>;
    using XLoads = std::integral_constant<int, 1>;
    using YLoads = std::integral_constant<int, 2>;

    // Prologue: k-tiles 0 and 1 (X loads A and the first scales, Y loads B).
    if (gx) {
        load_pair(0);
#pragma unroll
        for (int q = 0; q < PA; ++q) load_a(0, q, r0);
        if (KT > 1)
#pragma unroll
            for (int q = 0; q < PA; ++q) load_a(1, q, r0);
    } else {
#pragma unroll
        for (int q = 0; q < 2 * PB; ++q) load_b(0, q / PB, q / PB, q % PB, r0);
        if (KT > 1)
#pragma unroll
            for (int q = 0; q < 2 * PB; ++q) load_b(1, q / PB, 2 + q / PB, q % PB, r0);
    }
    if (KT > 1) {
        vm_wait<PA>();
    } else {
        vm_wait<0>();
        if (gx) zero_tail();
    }
    lds_wait_then_barrier();
    // slot of B's first half of the k-tile being read: 2 kt mod 5
    int slot = 0;
    if (gx) {
        read_ktile(0, 0, NoLoads{}, 0);
        lds_wait_then_barrier();
        for (int kt = 0; kt + 2 < KT; ++kt) {
            run_ktile(XBarrier{});
            slot = wrap(slot + 2);
            read_ktile(kt + 1, slot, XLoads{}, kt + 2);
            lds_wait_then_barrier();
        }
        if (KT >= 2) {
            run_ktile(XTail{});
            slot = wrap(slot + 2);
            read_ktile(KT - 1, slot, NoLoads{}, 0);
            lds_wait_then_barrier();
        }
        run_ktile(XBarrier{});
    } else {
        lds_wait_then_barrier();
        for (int kt = 0; kt + 2 < KT; ++kt) {
            read_ktile(kt, slot, YLoads{}, kt + 2);
            // the B half of k-tile kt + 1 has landed; that of kt + 2 may still fly
            wait_then_barrier<PB>();
            run_ktile(YBarrier{});
            slot = wrap(slot + 2);
        }
        if (KT >= 2) {
            read_ktile(KT - 2, slot, NoLoads{}, 0);
            wait_then_barrier<0>();
            run_ktile(YBarrier{});
            slot = wrap(slot + 2);
        }
        read_ktile(KT - 1, slot, NoLoads{}, 0);
        wait_then_barrier<0>();
        run_ktile(NoBarrier{});
    }

    mx_store<T>(p, acc, lds, wave, lane, m0 + wm0, n0 + wx * T::WTN);
}

// ---------------------------------------------------------- few tiles, deep loads
//
// Where the tiles do not fill the CUs, a k-tile of the ping-pong schedule costs the
// latency of its parts (loads, barriers, LDS reads, dependent instructions),
// about 0.4 us however small the tile.  Here a step is a pair of k-tiles (512
// elements, and the 16 scale bytes of a row that go with them), one barrier per
// step, no turns, and S stages keep S - 1 steps of loads in flight.  Every wave
// issues the same number of loads for every step (the scales at 4 bytes per lane),
// so the wait can count them.
template <int B_, int S_> struct MxDeep {
    static constexpr int BX = B_, S = S_;
    static constexpr int WTM = BX / 2, WTN = BX / 4, TM = WTM / 16, TN = WTN / 16;
    static constexpr int IMAGE = BX * 128;            // one operand's k-tile
    static constexpr int SCALES = 2 * BX * 16;        // both operands
    static constexpr int STAGE = 4 * IMAGE + SCALES;  // A's two images, B's two, scales
    static constexpr int PE = BX / 64, PS = BX / 64;  // loads per wave: an image; the scales
    static constexpr int L = 4 * PE + PS;             // per wave and step
    static constexpr int LDS_BYTES = S * STAGE;
    static_assert(LDS_BYTES <= 160 * 1024 && (S - 2) * L < 64, "fits LDS and the wait counter");
};

// 4 bytes per lane straight into LDS at lds_base + 4 * lane (see dma16).
__device__ __forceinline__ void dma4(uint32_t lds_base, const void* sbase, uint32_t voff) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, %1"
                 :
                 : "v"(voff), "s"(uniform_ptr(sbase)), "{m0}"(lds_base)
                 : "memory");
}

template <int BX, int S, bool TAIL>
__global__ __launch_bounds__(512) void mx_deep_kernel(MxArgs p, int tiles_m, int tiles_n) {
    using T = MxDeep<BX, S>;
    constexpr int TM = T::TM, TN = T::TN;
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];
    MIGEMM_LDS char* const lds = (MIGEMM_LDS char*)smem;
    const uint32_t lds_addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm0 = (wave >> 2) * T::WTM, wn0 = (wave & 3) * T::WTN;
    int pm, pn;
    tile_coords<8>(blockIdx.x, tiles_m, tiles_n, pm, pn);
    const int64_t m0 = static_cast<int64_t>(pm) * BX, n0 = static_cast<int64_t>(pn) * BX;
    const int chunks = static_cast<int>(p.K / 32), steps = (chunks + 15) / 16;
    const int left = TAIL ? chunks % 16 : 16;  // blocks in the last step (TAIL: 1 to 15)

    // element load q of a wave: rows 8 (wave + 8 q) + lane / 8, blocks placed and
    // swizzled as in mx_tile_kernel; scale load q: rows 16 (wave + 8 q) + lane / 4 of
    // A's rows and then B's
    const int r0 = 8 * wave + lane / 8;
    const int at_chunk = (lane % 8) ^ swz_a<8>(r0);
    const int logical = (at_chunk & 3) * 2 + (at_chunk >> 2);  // and 8 more in the second image
    const int last_m = static_cast<int>(min(p.M - m0, int64_t(BX))) - 1;
    const int last_n = static_cast<int>(min(p.N - n0, int64_t(BX))) - 1;
    const uint8_t* const a_tile = p.A + m0 * p.lda;
    const uint8_t* const b_tile = p.B + n0 * p.ldb;
    uint32_t va[T::PE], vb[T::PE], vs[T::PS];
#pragma unroll
    for (int q = 0; q < T::PE; ++q) {
        va[q] = static_cast<uint32_t>(min(r0 + 64 * q, last_m)) * static_cast<uint32_t>(p.lda);
        vb[q] = static_cast<uint32_t>(min(r0 + 64 * q, last_n)) * static_cast<uint32_t>(p.ldb);
    }
    const uint8_t* s_tile[T::PS];
#pragma unroll
    for (int q = 0; q < T::PS; ++q) {
        const int first = 16 * (wave + 8 * q);  // uniform: wholly in A's rows or in B's
        const bool of_a = first < BX;
        const int row = (of_a ? first : first - BX) + lane / 4;
        s_tile[q] = of_a ? p.sa + m0 * p.ldsa : p.sb + n0 * p.ldsb;
        vs[q] = static_cast<uint32_t>(min(row, of_a ? last_m : last_n)) *
                    static_cast<uint32_t>(of_a ? p.ldsa : p.ldsb) + 4 * (lane % 4);
    }
    auto issue = [&](int step, int stage) __attribute__((always_inline)) {
        const uint32_t st = lds_addr + stage * T::STAGE;
        const int64_t k = static_cast<int64_t>(step) * 256;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int block = logical + 8 * h;
            const uint32_t c = 16 * (TAIL && step == steps - 1 ? min(block, left - 1) : block);
#pragma unroll
            for (int q = 0; q < T::PE; ++q)
                dma16(st + h * T::IMAGE + (wave + 8 * q) * 1024, a_tile + k, va[q] + c);
#pragma unroll
            for (int q = 0; q < T::PE; ++q)
                dma16(st + (2 + h) * T::IMAGE + (wave + 8 * q) * 1024, b_tile + k, vb[q] + c);
        }
#pragma unroll
        for (int q = 0; q < T::PS; ++q)
            dma4(st + 4 * T::IMAGE + (wave + 8 * q) * 256,
                 s_tile[q] + static_cast<int64_t>(step) * 16, vs[q]);
    };
    // as mx_tile_kernel's: what this wave's loads of the last step brought from past
    // K becomes 0 (A's elements, both operands' scales)
    auto zero_tail = [&](int stage) __attribute__((always_inline)) {
        MIGEMM_LDS char* const st = lds + stage * T::STAGE;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (logical + 8 * h >= left) {
#pragma unroll
                for (int q = 0; q < T::PE; ++q)
                    *(MIGEMM_LDS u32x4*)(st + h * T::IMAGE + (wave + 8 * q) * 1024 + 16 * lane) =
                        u32x4{0u, 0u, 0u, 0u};
            }
        const int n = left - 4 * (lane % 4);  // valid bytes of the word
        const uint32_t mask = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
#pragma unroll
        for (int q = 0; q < T::PS; ++q) {
            MIGEMM_LDS uint32_t* const w =
                (MIGEMM_LDS uint32_t*)(st + 4 * T::IMAGE + (wave + 8 * q) * 256 + 4 * lane);
            *w = *w & mask;
        }
    };

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int ar = lane % 16, ag = lane / 16;
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
        if (t < steps) issue(t, t);
    int stage = 0;
    for (int step = 0; step < steps; ++step) {
        // this step has landed; the S - 2 after it may still fly
        if (step + S - 2 < steps)
            vm_wait<(S - 2) * T::L>();
        else
            vm_wait<0>();
        if (TAIL && step == steps - 1) zero_tail(stage);
        lds_wait_then_barrier();
        // every wave has read the step before: its stage takes step + S - 1
        if (step + S - 1 < steps) issue(step + S - 1, stage == 0 ? S - 1 : stage - 1);
        const MIGEMM_LDS char* const ia = lds + stage * T::STAGE;
        const MIGEMM_LDS char* const ib = ia + 2 * T::IMAGE;
        const MIGEMM_LDS char* const is = ia + 4 * T::IMAGE + 2 * ag;
        u32x4 fa[4][TM], fb[4][TN];
        uint32_t sa[2][TM], sb[2][TN];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                sa[h][i] = *(const MIGEMM_LDS uint16_t*)(is + (wm0 + 16 * i + ar) * 16 + 8 * h);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                sb[h][j] =
                    *(const MIGEMM_LDS uint16_t*)(is + (BX + wn0 + 16 * j + ar) * 16 + 8 * h);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int off = h * T::IMAGE + ((4 * s + ag) ^ swz_a<8>(ar)) * 16;
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    fa[2 * h + s][i] =
                        *(const MIGEMM_LDS u32x4*)(ia + (wm0 + 16 * i + ar) * 128 + off);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    fb[2 * h + s][j] =
                        *(const MIGEMM_LDS u32x4*)(ib + (wn0 + 16 * j + ar) * 128 + off);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    mfma_mx<0>(acc[i][j], fa[2 * h][i], fb[2 * h][j], sa[h][i], sb[h][j]);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    mfma_mx<1>(acc[i][j], fa[2 * h + 1][i], fb[2 * h + 1][j], sa[h][i], sb[h][j]);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    lds_wait_then_barrier();  // the last step's stage becomes the output step's scratch
    mx_store<T>(p, acc, lds, wave, lane, m0 + wm0, n0 + wn0);
}

// ------------------------------------------------------------------ few rows of A
//
// M of at most 16 TM rows: nothing is reused but A, which the caches hold, so the
// time is that of reading B once.  A workgroup takes 16 TN rows of B (columns of
// C); its waves split k in groups of 16 blocks (512 elements: four matrix
// instructions per fragment pair, and the 16 scale bytes of a row in one load),
// taken in turn, and add their sums through LDS in wave order, so the result does
// not depend on timing.
template <int TM, int TN, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void mx_rows_kernel(MxArgs p) {
    __shared__ f32x4 part[WAVES][TM * TN][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int r = lane % 16, g = lane / 16;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * TN);
    const int64_t chunks = p.K / 32, groups = ceil_div(chunks, 16);
    const uint8_t *b_row[TN], *sb_row[TN], *a_row[TM], *sa_row[TM];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int64_t row = min(n0 + 16 * j + r, p.N - 1);
        b_row[j] = p.B + row * p.ldb + 16 * g;
        sb_row[j] = p.sb + row * p.ldsb;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t row = min(int64_t(16 * i + r), p.M - 1);
        a_row[i] = p.A + row * p.lda + 16 * g;
        sa_row[i] = p.sa + row * p.ldsa;
    }
    f32x4 acc[TM][TN] = {};
    for (int64_t k = wave; k < groups; k += WAVES) {
        // step s of the group takes block 16 k + 4 s + g in this lane
        const int left = static_cast<int>(min(chunks - 16 * k, int64_t(16))) - g;
        u32x4 b[TN][4], a[TM][4], wb[TN], wa[TM];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            wb[j] = *reinterpret_cast<const u32x4*>(sb_row[j] + 16 * k);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                b[j][s] = u32x4{0u, 0u, 0u, 0u};
                if (4 * s < left)
                    b[j][s] = *reinterpret_cast<const u32x4*>(b_row[j] + 256 * k + 64 * s);
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            wa[i] = *reinterpret_cast<const u32x4*>(sa_row[i] + 16 * k);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                a[i][s] = u32x4{0u, 0u, 0u, 0u};
                if (4 * s < left)
                    a[i][s] = *reinterpret_cast<const u32x4*>(a_row[i] + 256 * k + 64 * s);
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            // byte g of the step's four scales; 0 past K, whatever the padding holds
            const bool in = 4 * s < left;
            uint32_t ea[TM], eb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) ea[i] = in ? wa[i][s] >> (8 * g) : 0u;
#pragma unroll
            for (int j = 0; j < TN; ++j) eb[j] = in ? wb[j][s] >> (8 * g) : 0u;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) mfma_mx<0>(acc[i][j], a[i][s], b[j][s], ea[i], eb[j]);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) part[wave][i * TN + j][lane] = acc[i][j];
    __syncthreads();
    using L = AccLayout<16>;
    for (int q = wave; q < TM * TN; q += WAVES) {
        f32x4 sum = part[0][q][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            const f32x4 x = part[w][q][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += x[e];
        }
        const int64_t col = n0 + 16 * (q % TN) + L::col(lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t row = 16 * (q / TN) + L::row(lane, e);
            if (row < p.M && col < p.N)
                store_out<true>(p.out, row * p.out.ldc + col, sum[e]);
        }
    }
}

template <int BX>
hipError_t launch_tile(const MxArgs& p) {
    const int64_t tm = ceil_div(p.M, BX), tn = ceil_div(p.N, BX);
    if (tm * tn > launch_groups(512)) return hipErrorInvalidValue;
    auto* const fn =
        p.K % 256 != 0 ? mx_tile_kernel<BX, true> : mx_tile_kernel<BX, false>;
    fn<<<dim3(static_cast<unsigned>(tm * tn)), dim3(512), 0, p.stream>>>(
        p, static_cast<int>(tm), static_cast<int>(tn));
    return hipGetLastError();
}

template <int BX, int S>
hipError_t launch_deep(const MxArgs& p) {
    const int64_t tm = ceil_div(p.M, BX), tn = ceil_div(p.N, BX);
    if (tm * tn > launch_groups(512)) return hipErrorInvalidValue;
    auto* const fn =
        p.K % 512 != 0 ? mx_deep_kernel<BX, S, true> : mx_deep_kernel<BX, S, false>;
    fn<<<dim3(static_cast<unsigned>(tm * tn)), dim3(512), 0, p.stream>>>(
        p, static_cast<int>(tm), static_cast<int>(tn));
    return hipGetLastError();
}

template <int TM, int TN>
hipError_t launch_rows(const MxArgs& p) {
    mx_rows_kernel<TM, TN, 8><<<dim3(static_cast<unsigned>(ceil_div(p.N, 16 * TN))),
                                dim3(8 * kWave), 0, p.stream>>>(p);
    return hipGetLastError();
}

// Rows of A 64 at a time through the few-rows kernel: any leading dimension.  32
// columns per workgroup, which read A half as often, where that still makes 256
// workgroups (us at K = 8192, N = 8192, 32 against 16 columns: M = 1 8.1 / 8.4, 16
// 10.0 / 12.3, 64 17.6 / 27.3; N = 1024, M = 16 9.2 / 7.1, 64 16.5 / 13.9).
hipError_t launch_rows_any(const MxArgs& p) {
    const bool two = p.N > 32 * 255;
    for (int64_t m = 0; m < p.M; m += 64) {
        MxArgs q = p;
        q.M = p.M - m < 64 ? p.M - m : 64;
        q.A = p.A + m * p.lda;
        q.sa = p.sa + m * p.ldsa;
        q.out.C = static_cast<char*>(p.out.C) + m * p.out.ldc * (p.out.c_dtype == 0 ? 4 : 2);
        const hipError_t e = q.M <= 16   ? (two ? launch_rows<1, 2>(q) : launch_rows<1, 1>(q))
                             : q.M <= 32 ? (two ? launch_rows<2, 2>(q) : launch_rows<2, 1>(q))
                                         : (two ? launch_rows<4, 2>(q) : launch_rows<4, 1>(q));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

const char* const kNames[] = {"rows: 16 or 32 columns per workgroup, k over 8 waves",
                              "64x64x512 deep s4", "64x64x512 deep s2", "128x128x512 deep s2",
                              "128x128x256 pingpong", "256x256x256 pingpong"};
constexpr int kCount = sizeof(kNames) / sizeof(kNames[0]);

// The kernel for these sizes.  Up to 32 rows go to the rows kernel (M = 32 / 48 / 64
// by N = K = 8192: 12.5 / 16.3 / 17.6 us, 64x64 tiles 12.0 / 12.2 / 12.3; 32 x 1024 x
// 4096 6.1 against 7.1).  Of the tiles, the one whose workgroups cost least: `slots` of
// them fit the 256 CUs together, a full set takes `full` and a lone one `lone` (us
// at K = 8192, BF16 C, and about in proportion to K), in between in proportion.
// Measured, us for configurations 1 to 5, N = K = 8192:
//   M = 128   13.0   16.1  24.0   27.0  47.4      M = 1024  87   72   50.6  46.9  51.3
//   M = 192   23.2   18.4  24.3   26.9  46.9      M = 2048 171  143  100    90    67.6
//   M = 512   46.0   36.7  26.7   30.0  49.0
// and 2048^3 17.9 12.9 9.5 10.9 18.8, 3000 x 3000 x 3008 54 39 35 32 27.
int choose(const MxArgs& p) {
    if (p.M <= 32) return 0;
    auto cost = [&](int64_t b, int64_t slots, double lone, double full) {
        const int64_t t = ceil_div(p.M, b) * ceil_div(p.N, b), part = t % slots;
        return static_cast<double>(t / slots) * full +
               (part ? lone + (full - lone) * static_cast<double>(part) / slots : 0.0);
    };
    const double c[] = {cost(64, 256, 12.0, 13.0), cost(64, 512, 13.0, 19.5),
                        cost(128, 256, 21.5, 26.0), cost(128, 512, 25.0, 46.5),
                        cost(256, 256, 46.0, 67.0)};
    int best = 0;
    for (int i = 1; i < 5; ++i)
        if (c[i] < c[best]) best = i;
    return best + 1;
}

hipError_t launch_part(const MxArgs& p, int config) {
    switch (config) {
        case 0: return launch_rows_any(p);
        case 1: return launch_deep<64, 4>(p);
        case 2: return launch_deep<64, 2>(p);
        case 3: return launch_deep<128, 2>(p);
        case 4: return launch_tile<128>(p);
        default: return launch_tile<256>(p);
    }
}

}  // namespace

int mx_config_count() { return kCount; }
const char* mx_config_name(int c) { return c >= 0 && c < kCount ? kNames[c] : nullptr; }

hipError_t launch_gemm_mx(const MxArgs& p, int config) {
    if (p.K == 0) {
        GemmArgs g{};
        g.M = p.M;
        g.N = p.N;
        g.out = p.out;
        g.stream = p.stream;
        return launch_empty_product(g);
    }
    if (config < 0) config = choose(p);
    // the tile kernel's load offsets are 32 bits, over 255 rows
    const int64_t far = int64_t(1) << 23;
    if (p.lda >= far || p.ldb >= far || p.ldsa >= far || p.ldsb >= far) config = 0;
    // one launch where it holds the workgroups (of 512 threads); else parts of C that do
    const int64_t b = config == 0 ? 16 : config <= 2 ? 64 : config <= 4 ? 128 : 256;
    const int64_t tm = config == 0 ? 1 : ceil_div(p.M, b), most = launch_groups(512);
    if (ceil_div(p.N, b) <= most / tm) return launch_part(p, config);
    const int64_t part_m = tm < 4096 ? tm : 4096, rows = config == 0 ? p.M : part_m * b;
    const int64_t cols = most / part_m * b;
    for (int64_t m = 0; m < p.M; m += rows)
        for (int64_t n = 0; n < p.N; n += cols) {
            MxArgs q = p;
            q.M = p.M - m < rows ? p.M - m : rows;
            q.N = p.N - n < cols ? p.N - n : cols;
            q.A = p.A + m * p.lda;
            q.sa = p.sa + m * p.ldsa;
            q.B = p.B + n * p.ldb;
            q.sb = p.sb + n * p.ldsb;
            q.out.C = static_cast<char*>(p.out.C) +
                      (m * p.out.ldc + n) * (p.out.c_dtype == 0 ? 4 : 2);
            const hipError_t e = launch_part(q, config);
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

}  // namespace migemm
