// rows.hpp -- pieces of rows in registers: what the layer norm, embedding and AdamW
// kernels share.
#pragma once

#include "common.hpp"

namespace migemm {

// Elements of type T in one 16-byte access.
template <typename T> constexpr int kChunk = 16 / static_cast<int>(sizeof(T));

template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ _Float16 narrow<_Float16>(float x) {
    return static_cast<_Float16>(x);
}
template <> __device__ __forceinline__ bf16_t narrow<bf16_t>(float x) {
    return bf16_t{f32_to_bf16_bits(x)};
}

// N consecutive elements, 16 bytes at a time, whatever the alignment.
template <typename T, int N>
__device__ __forceinline__ void load_whole(const T* __restrict__ p, T (&e)[N]) {
    __builtin_memcpy(e, p, sizeof(e));
}
template <typename T, int N>
__device__ __forceinline__ void store_whole(T* __restrict__ p, const T (&e)[N]) {
    __builtin_memcpy(p, e, sizeof(e));
}

// 16- and 8-byte accesses past the caches, at any alignment; wider pieces do not fill whole
// lines with one access of a wavefront, and go through them.
template <typename T, int N> __device__ __forceinline__ void load_once(const T* p, T (&e)[N]) {
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(1)));
    typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(1)));
    if constexpr (sizeof(e) == 16) {
        const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const v4*>(p));
        __builtin_memcpy(e, &w, sizeof(e));
    } else if constexpr (sizeof(e) == 8) {
        const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const v2*>(p));
        __builtin_memcpy(e, &w, sizeof(e));
    } else {
        load_whole(p, e);
    }
}
template <typename T, int N> __device__ __forceinline__ void store_once(T* p, const T (&e)[N]) {
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(1)));
    typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(1)));
    if constexpr (sizeof(e) == 16) {
        u32x4 w;
        __builtin_memcpy(&w, e, sizeof(e));
        __builtin_nontemporal_store(w, reinterpret_cast<v4*>(p));
    } else if constexpr (sizeof(e) == 8) {
        u32x2 w;
        __builtin_memcpy(&w, e, sizeof(e));
        __builtin_nontemporal_store(w, reinterpret_cast<v2*>(p));
    } else {
        store_whole(p, e);
    }
}

// Where a lane reads its N elements from `column` on, in a row of `length` (N at least): at
// the column itself, or, where the row ends sooner, N elements before its end.  So every
// load is one whole access without a branch, whatever the length; with a branch around the
// last elements the compiler waits for each load before the next.  The first `skip` of the
// elements are then another lane's (all of them where the column is past the row): they
// stay out of sums, and store_own leaves them to that lane.  store writes them too, for
// values that come out as the same bits in both lanes: a store under no branch can stay in
// flight while the next loads are waited for.
template <int N> struct Span {
    int64_t at;
    int skip;
    __device__ __forceinline__ Span(int64_t column, int64_t length) {
        at = column < length - N ? column : length - N;
        skip = static_cast<int>(column - at < N ? column - at : N);
    }
    template <typename T> __device__ __forceinline__ void load(const T* row, T (&e)[N]) const {
        load_whole(row + at, e);
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const T (&e)[N]) const {
        store_whole(row + at, e);
    }
    template <typename T>
    __device__ __forceinline__ void store_own(T* row, const T (&e)[N]) const {
        if (skip == 0) {
            store_whole(row + at, e);
        } else {
#pragma unroll
            for (int i = 1; i < N; ++i)
                if (i >= skip) row[at + i] = e[i];
        }
    }
};

// N elements of an array's last ones, `held` of them (zeros for the others).
template <typename T, int N>
__device__ __forceinline__ void load_part(const T* __restrict__ p, int64_t held, T (&e)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = i < held ? p[i] : ZeroOf<T>::get();
}
template <typename T, int N>
__device__ __forceinline__ void store_part(T* __restrict__ p, int64_t held, const T (&e)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < held) p[i] = e[i];
}

// The sum, or largest, over the 16 lanes of a DPP row, in every one of them: rotations by
// 8, 4, 2 and 1 lanes inside the instruction that adds.
template <int N> __device__ __forceinline__ float row_rotated(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                                 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum16(float v) {
    v += row_rotated<8>(v);
    v += row_rotated<4>(v);
    v += row_rotated<2>(v);
    return v + row_rotated<1>(v);
}

// The sum over LANES lanes (16 or 64, aligned), in every one of them.
template <int LANES> __device__ __forceinline__ float sum_lanes(float v) {
    static_assert(LANES == 16 || LANES == kWave, "a DPP row or a wavefront");
    v = sum16(v);
    if constexpr (LANES == kWave) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}

}  // namespace migemm
