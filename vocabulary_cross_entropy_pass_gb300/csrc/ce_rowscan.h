// ce_rowscan.h -- launchers of the passes over rows of logits: their statistics and
// largest logits (ce_logprobs.cu), the gradient from them (ce_softgrad.cu).  Needs
// ce_rowscan.cuh's row types.
#pragma once

#include "ce_list_table.h"
#include "ce_rowscan.cuh"

namespace gbce {

// A pass over the rows: statistics, and with top_k the largest logits.
struct ScanArgs {
    const char* x;
    RowAddr row;
    int64_t N, V;
    float L;               // log2(e) / temperature
    int segs;              // segments of a row, `per` vectors of its body in each
    int64_t per;
    int places, heads;     // of the queue; groups' maxima of each
    RowTokens tokens;
    float4* part;          // [N][segs] {m, d, s, candidates}, or NULL: one segment, finished in place
    uint64_t* cand;        // [N][segs][top_k]
    int top_k;
    float* logprobs;       // [N][tokens.n]
    float* entropy;
    int64_t* top_tokens;   // [N][top_k]
    float* top_logprobs;
    float4* stats;         // [N] {m, log d, entropy, 0}
    uint32_t* claim;       // rows taken beyond each CTA's first two, or NULL: every gridDim.x-th item
    uint32_t* err;
};
// The gradient p_j (a + b lp_j) of every row, and what its listed tokens get.
struct SoftGradArgs {
    const char* x;
    char* out;
    RowAddr row, orow;
    int64_t N, V;
    float L, scale;
    RowTokens tokens;
    const float4* stats;
    const float* grad_logprobs;  // [N][tokens.n] or NULL (log-probabilities)
    const float* grad_entropy;   // [N] or NULL
    const void* teacher;         // distillation: logits of the listed tokens
    int teacher_dtype;
    RowAddr trow;
    int64_t tstep;
    float tau;
    int normalize;
    const float* dloss;
    const int64_t* n_dev;        // the mean's kept rows, or NULL
    int64_t cols;                // columns of a CTA's run
    int64_t runs;
};
cudaError_t launch_softgrad(SoftGradArgs a, int dtype, cudaStream_t s);

// Argument checks and marshalling that the entry points share.
ce_status check_rows(const void* logits, int dtype, int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides);
ce_status check_tokens(const int64_t* tokens, const int64_t* strides, int64_t n, int64_t rows);
RowTokens row_tokens(const int64_t* tokens, const int64_t* strides, int64_t n, int64_t dim0, int64_t dim1,
                     int64_t ignore_idx);
ce_status check_grad(const void* logits, int dtype, int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides,
                     const void* grad, const int64_t* grad_strides);

// What list_enter changes a slot with.
__device__ __forceinline__ uint32_t slot_cas(uint16_t* slot, uint32_t expected, uint32_t value) {
    return atomicCAS(reinterpret_cast<unsigned short*>(slot), (unsigned short)expected, (unsigned short)value);
}

__device__ __forceinline__ float teacher_at(const void* z, int dtype, int64_t k) {
    if (dtype == CE_F32) return __ldg(static_cast<const float*>(z) + k);
    if (dtype == CE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(z)[k]);
    return __half2float(static_cast<const __half*>(z)[k]);
}

}  // namespace gbce
