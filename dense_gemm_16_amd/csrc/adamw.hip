// adamw.hip -- one AdamW step over many tensors.
//
// Per element, with g the gradient (times its scale), in FP32:
//     m = b1 m + (1 - b1) g,     v = b2 v + (1 - b2) g^2,
//     p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps).
// The factors are rounded once, on the host, from 64 bits.  Products and sums are not
// contracted, so that the states are the same bits as those of the formulas taken one
// operation at a time; of 8-bit ones a last bit may move a whole code.
//
// 8-bit states.  m and r = sqrt(v) are E4M3 codes times one FP32 scale for each block of
// 256 consecutive elements: the block's largest magnitude / 448 (E4M3's largest), so that
// the largest element comes back as it was and a block whose gradients stop decays as it should,
// which it would not under a power of two.  The root is kept instead of v because its
// range is the square root of v's.  A positive root never becomes code 0: the element's
// next step would be divided by little more than eps.  The update uses m and r as they
// were before rounding to codes.
//
// Bound by memory: 28 bytes an element with FP32 parameters and states (5.5 TB/s), 10.06
// with 16-bit parameters and 8-bit states (738 million elements 1240 to 1310 us on four
// boards, 6.0 to 5.7 TB/s).  A
// workgroup takes a piece of 4096 elements of one tensor, found in a table of tensors that
// the launch carries in its arguments: no copy of it to the device, and a captured launch
// keeps it.
#include <math.h>

#include "rows.hpp"
#include "training.hpp"

namespace migemm {
namespace {

constexpr int kThreads = 256, kPiece = 4096;
constexpr int kBlock = 256;          // elements of one scale
constexpr int kTensors = 48;         // of one launch: its arguments stay below 4 KiB (a last
                                     // launch of three tensors takes 5 to 6.5 us)
constexpr int64_t kPieces = int64_t(1) << 23;  // of one launch: fewer than 2^32 threads

struct Table {
    AdamNumbers n;
    double lr, beta1, beta2, decay;
    const float* lr_device;
    const int64_t* step_device;
    const float* grad_scale;
    int64_t step;
    int tensors;
    uint32_t first[kTensors];  // each tensor's first piece
    migemm_adamw_tensor t[kTensors];
};
static_assert(sizeof(Table) <= 4096, "kernel arguments");

// The numbers that depend on the rate and the step, rounded to FP32.
__host__ __device__ inline void set_rate(AdamNumbers& n, double lr, double decay, double beta1,
                                         double beta2, int64_t step) {
    const double t = static_cast<double>(step);
    n.decay = static_cast<float>(1.0 - lr * decay);
    n.rate = static_cast<float>(lr / (1.0 - pow(beta1, t)));
    n.unbias = static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, t)));
}

__device__ __forceinline__ float largest_of(float m, float x) {
    return __builtin_elementwise_maximum(m, fabsf(x));  // NaN if either is
}

// One element's moments.
__device__ __forceinline__ void moments(const AdamNumbers& n, float g, float& m, float& v) {
#pragma clang fp contract(off)
    m = m * n.beta1 + g * n.rest1;
    v = v * n.beta2 + (g * g) * n.rest2;
}
// Its parameter's step: r is the root of v.
__device__ __forceinline__ float stepped(const AdamNumbers& n, float p, float m, float r) {
#pragma clang fp contract(off)
    return p * n.decay - (m / (r * n.unbias + n.eps)) * n.rate;
}

// The scale of a block whose largest magnitude is m: NaN where that is NaN or infinite, and
// 0 (the block is held as zeros) below 2^-100, where 448 over it would leave FP32.
__device__ __forceinline__ float block_scale(float m) {
    if (!(m <= 3.402823466e38f)) return __builtin_nanf("");
    return m < 0x1p-100f ? 0.0f : m * (1.0f / 448.0f);
}

__device__ __forceinline__ float largest16(float v) {
    v = __builtin_elementwise_maximum(v, row_rotated<8>(v));
    v = __builtin_elementwise_maximum(v, row_rotated<4>(v));
    v = __builtin_elementwise_maximum(v, row_rotated<2>(v));
    return __builtin_elementwise_maximum(v, row_rotated<1>(v));
}

// The values of eight codes under a scale.
__device__ __forceinline__ void decode(const uint8_t (&codes)[8], float scale, float (&v)[8]) {
    uint32_t w[2];
    __builtin_memcpy(w, codes, sizeof(w));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
        v[4 * i] = lo[0] * scale;
        v[4 * i + 1] = lo[1] * scale;
        v[4 * i + 2] = hi[0] * scale;
        v[4 * i + 3] = hi[1] * scale;
    }
}

// The codes of eight values in units of the scale; the hardware rounds to the nearest,
// ties to even.
__device__ __forceinline__ void encode(const float (&x)[8], uint8_t (&codes)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
        w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], c, true);
    }
    __builtin_memcpy(codes, w, sizeof(w));
}

// How a lane's E elements lie in a tensor: all of them in it (WHOLE); in a tensor's last
// piece, E elements before its end, of which those past `skip` are the lane's (LAST, no
// branch around the loads: element by element they took 9 us); or, in a tensor of fewer
// than E, the `held` first (SHORT).  ONCE is WHOLE with accesses past the caches.
enum class Lie { WHOLE, ONCE, LAST, SHORT };
template <Lie L, int E> struct Piece {
    int64_t at;
    int skip, held;
    __device__ __forceinline__ Piece(int64_t i, int64_t count) : at(i), skip(0), held(E) {
        if constexpr (L == Lie::LAST) {
            const Span<E> s(i, count);
            at = s.at;
            skip = s.skip;
        }
        if constexpr (L == Lie::SHORT) {
            held = i < count ? static_cast<int>(count - i) : 0;
            at = i < count ? i : 0;
        }
    }
    __device__ __forceinline__ bool own(int e) const { return e >= skip && e < held; }
    template <typename T> __device__ __forceinline__ void load(const T* p, T (&e)[E]) const {
        if constexpr (L == Lie::SHORT)
            load_part(p + at, held, e);
        else if constexpr (L == Lie::ONCE)
            load_once(p + at, e);
        else
            load_whole(p + at, e);
    }
    template <typename T> __device__ __forceinline__ void store(T* p, const T (&e)[E]) const {
        if constexpr (L == Lie::WHOLE) {
            store_whole(p + at, e);
        } else if constexpr (L == Lie::ONCE) {
            store_once(p + at, e);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (own(i)) p[at + i] = e[i];
        }
    }
};

// 32-bit states: four elements a lane at a time, so that every access of a wavefront is
// contiguous.
constexpr int kEach32 = 4;
template <typename P, typename G, bool MASTER, Lie L>
__device__ __forceinline__ void step32(const AdamNumbers& n, const migemm_adamw_tensor& t,
                                       int64_t at, float scale) {
    constexpr int E = kEach32, U = kPiece / (kThreads * E);
    P* const param = static_cast<P*>(t.param);
    const G* const grad = static_cast<const G*>(t.grad);
    float *const avg = static_cast<float*>(t.avg), *const sq = static_cast<float*>(t.sq);
    float p[U][E], m[U][E], v[U][E];
    G g[U][E];
    P narrow_p[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Piece<L, E> piece(at + (u * kThreads + threadIdx.x) * E, t.count);
        piece.load(grad, g[u]);
        piece.load(avg, m[u]);
        piece.load(sq, v[u]);
        if constexpr (MASTER)
            piece.load(t.master, p[u]);
        else
            piece.load(param, narrow_p[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Piece<L, E> piece(at + (u * kThreads + threadIdx.x) * E, t.count);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (!MASTER) p[u][e] = to_f32(narrow_p[u][e]);
            moments(n, to_f32(g[u][e]) * scale, m[u][e], v[u][e]);
            p[u][e] = stepped(n, p[u][e], m[u][e], sqrtf(v[u][e]));
            narrow_p[u][e] = narrow<P>(p[u][e]);
        }
        piece.store(avg, m[u]);
        piece.store(sq, v[u]);
        if constexpr (MASTER) piece.store(t.master, p[u]);
        piece.store(param, narrow_p[u]);
    }
}

// 8-bit states: the 16 lanes of a DPP row hold one block, as two halves of eight elements
// a lane, so that every access to 16-bit elements and to codes covers whole lines.
constexpr int kEach8 = 8;
template <typename P, typename G, bool MASTER, Lie L>
__device__ __forceinline__ void step8(const AdamNumbers& n, const migemm_adamw_tensor& t,
                                      int64_t at, float scale) {
    constexpr int E = kEach8, H = 2;
    static_assert(kThreads * E * H == kPiece && E * H * 16 == kBlock, "one block to a DPP row");
    constexpr bool whole = L == Lie::WHOLE || L == Lie::ONCE;
    const int64_t start = at + threadIdx.x / 16 * kBlock;  // of the lane's block
    const bool any = whole || t.count > start;
    const int64_t block = any ? start / kBlock : 0, i = start + threadIdx.x % 16 * E;
    P* const param = static_cast<P*>(t.param);
    const G* const grad = static_cast<const G*>(t.grad);
    uint8_t *const avg = static_cast<uint8_t*>(t.avg), *const sq = static_cast<uint8_t*>(t.sq);
    const Piece<L, E> piece[H] = {{i, t.count}, {i + kBlock / H, t.count}};
    G g[H][E];
    P narrow_p[H][E];
    float p[H][E], m[H][E], r[H][E];
    uint8_t cm[H][E], cr[H][E];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        piece[h].load(grad, g[h]);
        piece[h].load(avg, cm[h]);
        piece[h].load(sq, cr[h]);
        if constexpr (MASTER)
            piece[h].load(t.master, p[h]);
        else
            piece[h].load(param, narrow_p[h]);
    }
    const float sm = t.avg_scales[block], sr = t.sq_scales[block];
    float lm = 0.0f, lr = 0.0f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        // (elements that are not the lane's may belong to another block: they are dropped)
        decode(cm[h], sm, m[h]);
        decode(cr[h], sr, r[h]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (!MASTER) p[h][e] = to_f32(narrow_p[h][e]);
            float v = r[h][e] * r[h][e];
            moments(n, to_f32(g[h][e]) * scale, m[h][e], v);
            r[h][e] = sqrtf(v);
            p[h][e] = stepped(n, p[h][e], m[h][e], r[h][e]);
            narrow_p[h][e] = narrow<P>(p[h][e]);
            if (whole || piece[h].own(e)) {
                lm = largest_of(lm, m[h][e]);
                lr = largest_of(lr, r[h][e]);
            }
        }
        if constexpr (MASTER) piece[h].store(t.master, p[h]);
        piece[h].store(param, narrow_p[h]);
    }
    const float nm = block_scale(largest16(lm)), nr = block_scale(largest16(lr));
    const float im = nm > 0.0f ? 1.0f / nm : 0.0f, ir = nr > 0.0f ? 1.0f / nr : 0.0f;
    const float least = nr > 0.0f ? 0x1p-9f : 0.0f;  // E4M3's smallest
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            m[h][e] *= im;
            const float x = r[h][e] * ir;
            r[h][e] = r[h][e] > 0.0f ? fmaxf(x, least) : x;
        }
        encode(m[h], cm[h]);
        encode(r[h], cr[h]);
        piece[h].store(avg, cm[h]);
        piece[h].store(sq, cr[h]);
    }
    if (any && threadIdx.x % 16 == 0) {
        t.avg_scales[block] = nm;
        t.sq_scales[block] = nr;
    }
}

template <typename P, typename G, bool EIGHT, bool MASTER, bool ONCE>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Table a) {
    float scale = 1.0f;
    if (a.grad_scale) {
        scale = *a.grad_scale;
        if (!(fabsf(scale) <= 3.402823466e38f)) return;  // the step is skipped
    }
    AdamNumbers n = a.n;
    if (a.lr_device || a.step_device) {
        // read where the kernel runs, so that a captured step goes on counting
        __shared__ AdamNumbers now;
        if (threadIdx.x == 0) {
            now = n;
            const int64_t step = a.step_device ? *a.step_device : a.step;
            set_rate(now, a.lr_device ? static_cast<double>(*a.lr_device) : a.lr, a.decay, a.beta1,
                     a.beta2, step < 1 ? 1 : step);
        }
        __syncthreads();
        n = now;
    }
    // the tensor whose pieces hold this workgroup's
    int lo = 0, hi = a.tensors;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.first[mid] <= blockIdx.x)
            lo = mid;
        else
            hi = mid;
    }
    const migemm_adamw_tensor& t = a.t[lo];
    const int64_t at = static_cast<int64_t>(blockIdx.x - a.first[lo]) * kPiece;
    auto run = [&](auto lie) __attribute__((always_inline)) {
        constexpr Lie L = decltype(lie)::value;
        if constexpr (EIGHT)
            step8<P, G, MASTER, L>(n, t, at, scale);
        else
            step32<P, G, MASTER, L>(n, t, at, scale);
    };
    if (at + kPiece <= t.count)
        run(std::integral_constant<Lie, ONCE ? Lie::ONCE : Lie::WHOLE>{});
    else if (t.count >= (EIGHT ? kEach8 : kEach32))
        run(std::integral_constant<Lie, Lie::LAST>{});
    else
        run(std::integral_constant<Lie, Lie::SHORT>{});
}

using Kernel = void (*)(Table);

template <typename P, typename G, bool ONCE> Kernel kernel_of(bool eight, bool master) {
    if constexpr (!std::is_same<P, float>::value) {
        if (master)
            return eight ? adamw_kernel<P, G, true, true, ONCE>
                         : adamw_kernel<P, G, false, true, ONCE>;
    }
    return eight ? adamw_kernel<P, G, true, false, ONCE> : adamw_kernel<P, G, false, false, ONCE>;
}
template <typename P, typename G> Kernel kernel_of(const AdamArgs& a, bool once) {
    return once ? kernel_of<P, G, true>(a.eight, a.master)
                : kernel_of<P, G, false>(a.eight, a.master);
}

// Past this many bytes a step's tensors go past the caches: the last-level one (256 MiB)
// holds too little of them for the next reader.  On one board, 738 million BF16 elements with
// 8-bit states (7.4 GB) 1240 us, 1425 through the caches; 133 million with FP32 states and master
// copies (3.7 GB) 675 and 708; 40 million with 8-bit states (0.4 GB) 69 and 64.
constexpr int64_t kOnceBytes = int64_t(512) << 20;

float* moved(float* p, int64_t elements) { return p ? p + elements : p; }
void* moved(void* p, int64_t bytes) { return static_cast<char*>(p) + bytes; }

}  // namespace

hipError_t launch_adamw(const AdamArgs& a) {
    const int pb = elem_size(a.param_dtype), gb = elem_size(a.grad_dtype), sb = a.eight ? 1 : 4;
    double bytes = 0.0;
    for (int64_t k = 0; k < a.tensors; ++k)
        bytes += static_cast<double>(a.list[k].count) * (2 * pb + gb + 4 * sb + (a.master ? 8 : 0));
    const bool once = bytes > static_cast<double>(kOnceBytes);
    Kernel fn;
    switch (a.param_dtype) {
        case 0: fn = kernel_of<float, float>(a, once); break;
        case 1:
            fn = a.grad_dtype == 0 ? kernel_of<_Float16, float>(a, once)
                                   : kernel_of<_Float16, _Float16>(a, once);
            break;
        default:
            fn = a.grad_dtype == 0 ? kernel_of<bf16_t, float>(a, once)
                                   : kernel_of<bf16_t, bf16_t>(a, once);
    }
    const migemm_adamw_options& o = a.o;
    Table t{};
    t.n.beta1 = static_cast<float>(o.beta1);
    t.n.rest1 = static_cast<float>(1.0 - o.beta1);
    t.n.beta2 = static_cast<float>(o.beta2);
    t.n.rest2 = static_cast<float>(1.0 - o.beta2);
    t.n.eps = static_cast<float>(o.eps);
    set_rate(t.n, o.lr, o.weight_decay, o.beta1, o.beta2, o.step < 1 ? 1 : o.step);
    t.lr = o.lr;
    t.beta1 = o.beta1;
    t.beta2 = o.beta2;
    t.decay = o.weight_decay;
    t.step = o.step;
    t.lr_device = o.lr_device;
    t.step_device = o.step_device;
    t.grad_scale = o.grad_scale;
    int64_t pieces = 0;
    auto flush = [&]() {
        if (pieces == 0) return hipSuccess;
        fn<<<dim3(static_cast<unsigned>(pieces)), dim3(kThreads), 0, a.stream>>>(t);
        t.tensors = 0;
        pieces = 0;
        return hipGetLastError();
    };
    for (int64_t k = 0; k < a.tensors; ++k) {
        const migemm_adamw_tensor& s = a.list[k];
        int64_t done = 0;
        while (done < s.count) {
            if (t.tensors == kTensors || pieces == kPieces) {
                const hipError_t err = flush();
                if (err != hipSuccess) return err;
            }
            const int64_t left = s.count - done, room = (kPieces - pieces) * kPiece;
            const int64_t take = left < room ? left : room;
            migemm_adamw_tensor& e = t.t[t.tensors];
            e.count = take;
            e.param = moved(s.param, done * pb);
            e.grad = static_cast<const char*>(s.grad) + done * gb;
            e.master = moved(s.master, done);
            e.avg = moved(s.avg, done * sb);
            e.sq = moved(s.sq, done * sb);
            e.avg_scales = moved(s.avg_scales, done / kBlock);
            e.sq_scales = moved(s.sq_scales, done / kBlock);
            t.first[t.tensors++] = static_cast<uint32_t>(pieces);
            pieces += ceil_div(take, kPiece);
            done += take;
        }
    }
    return flush();
}

}  // namespace migemm
