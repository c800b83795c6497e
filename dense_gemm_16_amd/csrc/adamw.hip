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
// the largest element is exact and a block whose gradients stop decays as it should,
// which it would not under a power of two.  The root is kept instead of v because its
// range is the square root of v's.  A positive root never becomes code 0: the element's
// next step would be divided by little more than eps.  The update uses m and r as they
// were before rounding to codes.
//
// Bound by memory: 28 bytes an element with FP32 parameters and states, 10.06 with 16-bit
// parameters and 8-bit states.  A workgroup takes a piece of 4096 elements of one tensor,
// found in a table of tensors that the launch carries in its arguments: no copy of it to
// the device, and a captured launch keeps it.
#include <math.h>

#include "rows.hpp"
#include "training.hpp"

namespace migemm {
namespace {

constexpr int kThreads = 256, kPiece = 4096;
constexpr int kBlock = 256;          // elements of one scale
constexpr int kTensors = 48;         // of one launch: its arguments stay below 4 KiB
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

// The values of 16 codes under a scale.
__device__ __forceinline__ void decode(const uint8_t (&codes)[16], float scale, float (&v)[16]) {
    uint32_t w[4];
    __builtin_memcpy(w, codes, sizeof(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
        v[4 * i] = lo[0] * scale;
        v[4 * i + 1] = lo[1] * scale;
        v[4 * i + 2] = hi[0] * scale;
        v[4 * i + 3] = hi[1] * scale;
    }
}

// The codes of 16 values in units of the scale; the hardware rounds to the nearest, ties
// to even.
__device__ __forceinline__ void encode(const float (&x)[16], uint8_t (&codes)[16]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
        w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], c, true);
    }
    __builtin_memcpy(codes, w, sizeof(w));
}

// 32-bit states: four elements a lane at a time, so that every access of a wavefront is
// contiguous.
template <typename P, typename G, bool MASTER>
__device__ __forceinline__ void step32(const AdamNumbers& n, const migemm_adamw_tensor& t,
                                       int64_t at, float scale) {
    constexpr int E = 4, U = kPiece / (kThreads * E);
    P* const param = static_cast<P*>(t.param);
    const G* const grad = static_cast<const G*>(t.grad);
    float *const avg = static_cast<float*>(t.avg), *const sq = static_cast<float*>(t.sq);
    float p[U][E], m[U][E], v[U][E];
    G g[U][E];
    P narrow_p[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = at + (u * kThreads + threadIdx.x) * E, held = t.count - i;
        load_part(grad + i, held, g[u]);
        load_part(avg + i, held, m[u]);
        load_part(sq + i, held, v[u]);
        if constexpr (MASTER)
            load_part(t.master + i, held, p[u]);
        else
            load_part(param + i, held, narrow_p[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = at + (u * kThreads + threadIdx.x) * E, held = t.count - i;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (!MASTER) p[u][e] = to_f32(narrow_p[u][e]);
            moments(n, to_f32(g[u][e]) * scale, m[u][e], v[u][e]);
            p[u][e] = stepped(n, p[u][e], m[u][e], sqrtf(v[u][e]));
            narrow_p[u][e] = narrow<P>(p[u][e]);
        }
        store_part(avg + i, held, m[u]);
        store_part(sq + i, held, v[u]);
        if constexpr (MASTER) store_part(t.master + i, held, p[u]);
        store_part(param + i, held, narrow_p[u]);
    }
}

// 8-bit states: 16 elements a lane, so that the 16 lanes of a DPP row hold one block.
template <typename P, typename G, bool MASTER>
__device__ __forceinline__ void step8(const AdamNumbers& n, const migemm_adamw_tensor& t,
                                      int64_t at, float scale) {
    constexpr int E = 16;
    static_assert(kThreads * E == kPiece && E * 16 == kBlock, "one block to a DPP row");
    const int64_t i = at + threadIdx.x * E, held = t.count - i, block = i / kBlock;
    P* const param = static_cast<P*>(t.param) + i;
    uint8_t *const avg = static_cast<uint8_t*>(t.avg) + i, *const sq = static_cast<uint8_t*>(t.sq) + i;
    const bool any = t.count > block * kBlock;
    G g[E];
    P narrow_p[E];
    float p[E], m[E], r[E];
    uint8_t cm[E], cr[E];
    load_part(static_cast<const G*>(t.grad) + i, held, g);
    load_part(avg, held, cm);
    load_part(sq, held, cr);
    if constexpr (MASTER)
        load_part(t.master + i, held, p);
    else
        load_part(param, held, narrow_p);
    const float sm = any ? t.avg_scales[block] : 0.0f, sr = any ? t.sq_scales[block] : 0.0f;
    decode(cm, sm, m);
    decode(cr, sr, r);
    float lm = 0.0f, lr = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if constexpr (!MASTER) p[e] = to_f32(narrow_p[e]);
        float v = r[e] * r[e];
        moments(n, to_f32(g[e]) * scale, m[e], v);
        r[e] = sqrtf(v);
        p[e] = stepped(n, p[e], m[e], r[e]);
        narrow_p[e] = narrow<P>(p[e]);
        lm = largest_of(lm, m[e]);
        lr = largest_of(lr, r[e]);
    }
    if constexpr (MASTER) store_part(t.master + i, held, p);
    store_part(param, held, narrow_p);
    const float nm = block_scale(largest16(lm)), nr = block_scale(largest16(lr));
    const float im = nm > 0.0f ? 1.0f / nm : 0.0f, ir = nr > 0.0f ? 1.0f / nr : 0.0f;
    const float least = nr > 0.0f ? 0x1p-9f : 0.0f;  // E4M3's smallest
#pragma unroll
    for (int e = 0; e < E; ++e) {
        m[e] *= im;
        const float x = r[e] * ir;
        r[e] = r[e] > 0.0f ? fmaxf(x, least) : x;
    }
    encode(m, cm);
    encode(r, cr);
    store_part(avg, held, cm);
    store_part(sq, held, cr);
    if (any && threadIdx.x % 16 == 0) {
        t.avg_scales[block] = nm;
        t.sq_scales[block] = nr;
    }
}

template <typename P, typename G, bool EIGHT, bool MASTER>
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
    if constexpr (EIGHT)
        step8<P, G, MASTER>(n, t, at, scale);
    else
        step32<P, G, MASTER>(n, t, at, scale);
}

using Kernel = void (*)(Table);

template <typename P, typename G> Kernel kernel_of(bool eight, bool master) {
    if constexpr (std::is_same<P, float>::value) {
        return eight ? adamw_kernel<P, G, true, false> : adamw_kernel<P, G, false, false>;
    } else {
        if (eight) return master ? adamw_kernel<P, G, true, true> : adamw_kernel<P, G, true, false>;
        return master ? adamw_kernel<P, G, false, true> : adamw_kernel<P, G, false, false>;
    }
}

float* moved(float* p, int64_t elements) { return p ? p + elements : p; }
void* moved(void* p, int64_t bytes) { return static_cast<char*>(p) + bytes; }

}  // namespace

hipError_t launch_adamw(const AdamArgs& a) {
    Kernel fn;
    switch (a.param_dtype) {
        case 0: fn = kernel_of<float, float>(a.eight, a.master); break;
        case 1:
            fn = a.grad_dtype == 0 ? kernel_of<_Float16, float>(a.eight, a.master)
                                   : kernel_of<_Float16, _Float16>(a.eight, a.master);
            break;
        default:
            fn = a.grad_dtype == 0 ? kernel_of<bf16_t, float>(a.eight, a.master)
                                   : kernel_of<bf16_t, bf16_t>(a.eight, a.master);
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
    const int pb = elem_size(a.param_dtype), gb = elem_size(a.grad_dtype), sb = a.eight ? 1 : 4;
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
