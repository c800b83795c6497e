// training.hpp -- layer norm, embeddings and AdamW: what their entry points
// (training_api.cpp) and kernels (layer_norm.hip, embedding.hip, adamw.hip) share.
#pragma once

#include "common.hpp"
#include "migemm.h"

namespace migemm {

struct NormArgs {
    int64_t T, D;
    int dtype, w_dtype;
    const void* X;
    int64_t ldx;
    const void* W;  // NULL: ones
    const void* B;  // NULL: zeros (forward only)
    float eps;
    void* Y;  // forward: the result; backward: dX, NULL where not wanted
    int64_t ldy;
    const void* dY;
    int64_t lddy;
    float* mean;
    float* rstd;
    void* dW;  // NULL where not wanted
    void* dB;
    hipStream_t stream;
};
hipError_t launch_layer_norm(const NormArgs& a);
// The workspace of a backward pass: partial sums of dW and dB, and for rows too long for
// registers two sums a row.
int64_t layer_norm_workspace(int64_t T, int64_t D, bool vectors);
hipError_t launch_layer_norm_backward(const NormArgs& a, void* ws);

struct EmbedArgs {
    int64_t T, V, D;
    int dtype, w_dtype;  // w_dtype: the gradient's
    const void* W;       // forward: the table
    void* dW;            // backward: its gradient
    int64_t ldw;
    const int64_t* index;
    int64_t ignore;
    float scale;
    bool accumulate;
    void* Y;         // forward: the result
    const void* dY;  // backward: its gradient
    int64_t ldy;
    hipStream_t stream;
};
hipError_t launch_embedding(const EmbedArgs& a);
int64_t embedding_workspace(int64_t T, int64_t V, int64_t D);
hipError_t launch_embedding_backward(const EmbedArgs& a, void* ws);

// The step's numbers, rounded once to FP32.
struct AdamNumbers {
    float beta1, rest1, beta2, rest2;  // rest: 1 - beta
    float decay;                       // 1 - lr weight_decay
    float rate;                        // lr / (1 - beta1^step)
    float unbias;                      // 1 / sqrt(1 - beta2^step)
    float eps;
};
struct AdamArgs {
    const migemm_adamw_tensor* list;
    int64_t tensors;
    int param_dtype, grad_dtype;
    bool eight, master;
    migemm_adamw_options o;
    hipStream_t stream;
};
hipError_t launch_adamw(const AdamArgs& a);

}  // namespace migemm
