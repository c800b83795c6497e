// training_api.cpp -- the entry points of layer norm, embeddings and AdamW: argument
// checks, then the launchers in layer_norm.hip, embedding.hip and adamw.hip.
#include <math.h>

#include <algorithm>
#include <new>

#include "training.hpp"

namespace migemm {
namespace {

constexpr int64_t kMaxNormDim = int64_t(1) << 24;
constexpr int64_t kMaxEntries = int64_t(1) << 28, kMaxEmbedDim = int64_t(1) << 21;
constexpr int64_t kMaxCount = int64_t(1) << 40, kMaxTensors = int64_t(1) << 24;

bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld < kMaxLd; }
bool second_type_ok(int t, int dtype) { return t == dtype || t == MIGEMM_F32; }

struct Range {
    uintptr_t lo, hi;
};

// The byte ranges that a call reads and writes.
struct Ranges {
    static constexpr int kMax = 12;
    Range in[kMax], out[kMax];
    int n_in = 0, n_out = 0;
    bool fits = true;  // none is NULL or passes the address space
    void add(bool writes, const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
        Range r;
        if (!p || !extent(p, rows, cols, ld, es, r.lo, r.hi)) {
            fits = false;
        } else if (writes) {
            out[n_out++] = r;
        } else {
            in[n_in++] = r;
        }
    }
    void reads(const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
        add(false, p, rows, cols, ld, es);
    }
    void writes(const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
        add(true, p, rows, cols, ld, es);
    }
    // All are there, and nothing written meets anything else.
    bool ok() const {
        if (!fits) return false;
        for (int i = 0; i < n_out; ++i) {
            for (int j = 0; j < n_in; ++j)
                if (overlaps(out[i].lo, out[i].hi, in[j].lo, in[j].hi)) return false;
            for (int j = 0; j < i; ++j)
                if (overlaps(out[i].lo, out[i].hi, out[j].lo, out[j].hi)) return false;
        }
        return true;
    }
};

// Kernels read a row's statistics and a token's index by scalar loads, which drop an
// address's lowest bits: those lie on their elements' boundaries.  (Elements of matrices
// and vectors are read by vector loads, at any address.)
bool on_elements(const void* p, int es) { return reinterpret_cast<uintptr_t>(p) % es == 0; }

// The workspace lent is `need` bytes or more, and aligned.
int check_workspace(int64_t need, const void* ws, int64_t ws_bytes) {
    if (need == 0) return MIGEMM_OK;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % kWorkspaceAlign != 0 || ws_bytes < need)
        return MIGEMM_ERR_WORKSPACE;
    return MIGEMM_OK;
}

bool norm_shape_ok(int64_t T, int64_t D) {
    return T >= 0 && T <= kMaxDim && D >= 1 && D <= kMaxNormDim;
}

bool embed_shape_ok(int64_t T, int64_t V, int64_t D) {
    return T >= 0 && T <= kMaxDim && V >= 1 && V <= kMaxEntries && D >= 1 && D <= kMaxEmbedDim;
}

bool is_finite(double x) { return x - x == 0.0; }

bool options_ok(const migemm_adamw_options& o) {
    return is_finite(o.lr) && is_finite(o.weight_decay) && is_finite(o.eps) && o.eps >= 0.0 &&
           o.beta1 >= 0.0 && o.beta1 < 1.0 && o.beta2 >= 0.0 && o.beta2 < 1.0 &&
           (o.step >= 1 || o.step_device);
}

// One range among all that a step names, for sorting by where it begins.
struct Named {
    uintptr_t lo, hi;
    bool written;
};

// The ranges of a tensor's arrays; false where one is missing, misaligned to its elements
// or passes the address space, or one is given that the call has no use for.
bool name_tensor(const migemm_adamw_tensor& t, int pb, int gb, bool eight, bool master, Named* at,
                 int& n) {
    auto add = [&](const void* p, int64_t count, int es, bool written) {
        Named r{0, 0, written};
        if (!p || !on_elements(p, es) || !extent(p, 1, count, count, es, r.lo, r.hi))
            return false;
        at[n++] = r;
        return true;
    };
    const int sb = eight ? 1 : 4;
    const int64_t blocks = ceil_div(t.count, 256);
    if (!add(t.param, t.count, pb, true) || !add(t.grad, t.count, gb, false) ||
        !add(t.avg, t.count, sb, true) || !add(t.sq, t.count, sb, true))
        return false;
    if (master != (t.master != nullptr)) return false;
    if (master && !add(t.master, t.count, 4, true)) return false;
    if (!eight) return !t.avg_scales && !t.sq_scales;
    return add(t.avg_scales, blocks, 4, true) && add(t.sq_scales, blocks, 4, true);
}

// Whether any written range meets another one.
bool some_meet(Named* r, int64_t n) {
    std::sort(r, r + n, [](const Named& a, const Named& b) { return a.lo < b.lo; });
    uintptr_t end = 0, written_end = 0;  // of all before, and of the written ones
    for (int64_t i = 0; i < n; ++i) {
        if (r[i].lo < (r[i].written ? end : written_end)) return true;
        end = std::max(end, r[i].hi);
        if (r[i].written) written_end = std::max(written_end, r[i].hi);
    }
    return false;
}

}  // namespace
}  // namespace migemm

using namespace migemm;

extern "C" {

int migemm_layer_norm_forward(int64_t T, int64_t D, int dtype, const void* X, int64_t ldx,
                              int w_dtype, const void* W, const void* B, float eps, void* Y,
                              int64_t ldy, float* mean, float* rstd, void* stream) {
    if (!known_dtype(dtype) || !second_type_ok(w_dtype, dtype) || !norm_shape_ok(T, D) ||
        !ld_ok(ldx, D) || !ld_ok(ldy, D) || !(eps >= 0.0f) || !is_finite(eps))
        return MIGEMM_ERR_INVALID_ARG;
    if (T == 0) return MIGEMM_OK;
    const int es = elem_size(dtype), ws = elem_size(w_dtype);
    Ranges r;
    r.reads(X, T, D, ldx, es);
    if (W) r.reads(W, 1, D, D, ws);
    if (B) r.reads(B, 1, D, D, ws);
    r.writes(Y, T, D, ldy, es);
    if (mean) r.writes(mean, 1, T, T, 4);
    if (rstd) r.writes(rstd, 1, T, T, 4);
    if (!r.ok()) return MIGEMM_ERR_INVALID_ARG;
    NormArgs a{};
    a.T = T;
    a.D = D;
    a.dtype = dtype;
    a.w_dtype = w_dtype;
    a.X = X;
    a.ldx = ldx;
    a.W = W;
    a.B = B;
    a.eps = eps;
    a.Y = Y;
    a.ldy = ldy;
    a.mean = mean;
    a.rstd = rstd;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(launch_layer_norm(a));
}

int migemm_layer_norm_workspace_size(int64_t T, int64_t D, int vectors, int64_t* bytes) {
    if (!bytes || !norm_shape_ok(T, D)) return MIGEMM_ERR_INVALID_ARG;
    *bytes = layer_norm_workspace(T, D, vectors != 0);
    return MIGEMM_OK;
}

int migemm_layer_norm_backward(int64_t T, int64_t D, int dtype, const void* dY, int64_t lddy,
                               const void* X, int64_t ldx, int w_dtype, const void* W,
                               const float* mean, const float* rstd, void* dX, int64_t lddx,
                               void* dW, void* dB, void* workspace, int64_t workspace_bytes,
                               void* stream) {
    if (!known_dtype(dtype) || !second_type_ok(w_dtype, dtype) || !norm_shape_ok(T, D) ||
        !ld_ok(lddy, D) || !ld_ok(ldx, D) || (dX && !ld_ok(lddx, D)) || workspace_bytes < 0)
        return MIGEMM_ERR_INVALID_ARG;
    const int es = elem_size(dtype), vs = elem_size(w_dtype);
    Ranges r;
    if (T > 0) {
        r.reads(dY, T, D, lddy, es);
        r.reads(X, T, D, ldx, es);
        if (W) r.reads(W, 1, D, D, vs);
        r.reads(mean, 1, T, T, 4);
        r.reads(rstd, 1, T, T, 4);
        if (dX) r.writes(dX, T, D, lddx, es);
        if (!on_elements(mean, 4) || !on_elements(rstd, 4)) return MIGEMM_ERR_INVALID_ARG;
    }
    if (dW) r.writes(dW, 1, D, D, vs);
    if (dB) r.writes(dB, 1, D, D, vs);
    if (!r.ok()) return MIGEMM_ERR_INVALID_ARG;
    if (!dW && !dB && (!dX || T == 0)) return MIGEMM_OK;
    const int64_t need = layer_norm_workspace(T, D, dW || dB);
    const int st = check_workspace(need, workspace, workspace_bytes);
    if (st != MIGEMM_OK) return st;
    if (need > 0) r.writes(workspace, 1, need, need, 1);
    if (!r.ok()) return MIGEMM_ERR_INVALID_ARG;
    NormArgs a{};
    a.T = T;
    a.D = D;
    a.dtype = dtype;
    a.w_dtype = w_dtype;
    a.X = X;
    a.ldx = ldx;
    a.W = W;
    a.Y = dX;
    a.ldy = lddx;
    a.dY = dY;
    a.lddy = lddy;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dW = dW;
    a.dB = dB;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(launch_layer_norm_backward(a, workspace));
}

int migemm_embedding_forward(int64_t T, int64_t V, int64_t D, int dtype, const void* W,
                             int64_t ldw, const int64_t* index, int64_t ignore_index, float scale,
                             void* Y, int64_t ldy, void* stream) {
    if (!known_dtype(dtype) || !embed_shape_ok(T, V, D) || !ld_ok(ldw, D) || !ld_ok(ldy, D))
        return MIGEMM_ERR_INVALID_ARG;
    if (T == 0) return MIGEMM_OK;
    const int es = elem_size(dtype);
    Ranges r;
    r.reads(W, V, D, ldw, es);
    r.reads(index, 1, T, T, 8);
    r.writes(Y, T, D, ldy, es);
    if (!r.ok()) return MIGEMM_ERR_INVALID_ARG;
    EmbedArgs a{};
    a.T = T;
    a.V = V;
    a.D = D;
    a.dtype = dtype;
    a.W = W;
    a.ldw = ldw;
    a.index = index;
    a.ignore = ignore_index;
    a.scale = scale;
    a.Y = Y;
    a.ldy = ldy;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(launch_embedding(a));
}

int migemm_embedding_workspace_size(int64_t T, int64_t V, int64_t D, int64_t* bytes) {
    if (!bytes || !embed_shape_ok(T, V, D)) return MIGEMM_ERR_INVALID_ARG;
    *bytes = embedding_workspace(T, V, D);
    return MIGEMM_OK;
}

int migemm_embedding_backward(int64_t T, int64_t V, int64_t D, int dtype, const void* dY,
                              int64_t lddy, const int64_t* index, int64_t ignore_index,
                              float scale, int accumulate, int dw_dtype, void* dW, int64_t lddw,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    if (!known_dtype(dtype) || !second_type_ok(dw_dtype, dtype) || !embed_shape_ok(T, V, D) ||
        !ld_ok(lddy, D) || !ld_ok(lddw, D) || (accumulate != 0 && accumulate != 1) ||
        workspace_bytes < 0)
        return MIGEMM_ERR_INVALID_ARG;
    Ranges r;
    if (T > 0) {
        r.reads(dY, T, D, lddy, elem_size(dtype));
        r.reads(index, 1, T, T, 8);
        if (!on_elements(index, 8)) return MIGEMM_ERR_INVALID_ARG;
    }
    r.writes(dW, V, D, lddw, elem_size(dw_dtype));
    if (!r.ok()) return MIGEMM_ERR_INVALID_ARG;
    const int64_t need = embedding_workspace(T, V, D);
    const int st = check_workspace(need, workspace, workspace_bytes);
    if (st != MIGEMM_OK) return st;
    if (need > 0) r.writes(workspace, 1, need, need, 1);
    if (!r.ok()) return MIGEMM_ERR_INVALID_ARG;
    EmbedArgs a{};
    a.T = T;
    a.V = V;
    a.D = D;
    a.dtype = dtype;
    a.w_dtype = dw_dtype;
    a.dW = dW;
    a.ldw = lddw;
    a.index = index;
    a.ignore = ignore_index;
    a.scale = scale;
    a.accumulate = accumulate != 0;
    a.dY = dY;
    a.ldy = lddy;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(launch_embedding_backward(a, workspace));
}

int migemm_adamw(int64_t tensors, const migemm_adamw_tensor* list, int param_dtype,
                 int grad_dtype, int state_bits, const migemm_adamw_options* options,
                 void* stream) {
    if (tensors < 0 || tensors > kMaxTensors || (tensors > 0 && !list) || !options ||
        !known_dtype(param_dtype) || !second_type_ok(grad_dtype, param_dtype) ||
        (state_bits != 32 && state_bits != 8) || !options_ok(*options))
        return MIGEMM_ERR_INVALID_ARG;
    const bool eight = state_bits == 8;
    const int pb = elem_size(param_dtype), gb = elem_size(grad_dtype);
    // up to seven arrays a tensor, and the three numbers on the device
    constexpr int kHere = 64;
    Named here[kHere * 7 + 3];
    Named* named = here;
    if (tensors > kHere) {
        named = new (std::nothrow) Named[static_cast<size_t>(tensors) * 7 + 3];
        if (!named) return MIGEMM_ERR_INVALID_ARG;
    }
    int64_t n = 0;
    bool ok = true, master = false, first = true;
    for (int64_t k = 0; ok && k < tensors; ++k) {
        const migemm_adamw_tensor& t = list[k];
        if (t.count == 0) continue;
        if (first) master = t.master != nullptr;
        first = false;
        int added = 0;
        ok = t.count > 0 && t.count < kMaxCount && !(master && param_dtype == MIGEMM_F32) &&
             name_tensor(t, pb, gb, eight, master, named + n, added);
        n += added;
    }
    const struct {
        const void* p;
        int es;
    } numbers[] = {{options->lr_device, 4}, {options->step_device, 8}, {options->grad_scale, 4}};
    for (const auto& q : numbers) {
        if (!ok || !q.p) continue;
        Named r{0, 0, false};
        ok = on_elements(q.p, q.es) && extent(q.p, 1, 1, 1, q.es, r.lo, r.hi);
        named[n++] = r;
    }
    ok = ok && !some_meet(named, n);
    if (named != here) delete[] named;
    if (!ok) return MIGEMM_ERR_INVALID_ARG;
    AdamArgs a{};
    a.list = list;
    a.tensors = tensors;
    a.param_dtype = param_dtype;
    a.grad_dtype = grad_dtype;
    a.eight = eight;
    a.master = master;
    a.o = *options;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(launch_adamw(a));
}

}  // extern "C"
