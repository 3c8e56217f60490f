// ce_distill.cu -- the divergence of a row's softmax from a teacher that is known by
// its top logits, and its C entry points.
//
// With s = 1 / temperature, z_k the teacher's logit of its token t_k:
//   q_k = exp(s z_k) / sum exp(s z)   (normalize; else exp(s z_k), the rest left out)
//   p_j = exp(s x_j) / sum exp(s x)
//   loss = temperature^2 sum_k q_k (log q_k - log p_{t_k})
//   grad_j = dloss temperature (Q p_j - sum_k q_k [t_k = j]),   Q = sum_k q_k
// The statistics of x come from ce_scan_kernel, a CTA per row here adds the teacher's
// and the loss, ce_softgrad_kernel writes the gradient.
#include <math.h>

#include "ce_rowscan.h"

namespace gbce {
namespace {

struct DistillArgs {
    const char* x;
    RowAddr row;
    int64_t N, V;
    float L, scale, tau;
    RowTokens tokens;
    const void* teacher;
    int teacher_dtype;
    RowAddr trow;
    int64_t tstep;
    int normalize;
    int segs;
    const float4* part;   // [N][segs]
    float* loss;          // [N]
    float4* stats;        // [N] {m, log d, the teacher's maximum, log of its sum}
    uint32_t* err;
};

// A row's loss and statistics.
template <typename T>
__global__ void __launch_bounds__(kScanThreads) ce_distill_row_kernel(const __grid_constant__ DistillArgs p) {
    __shared__ float4 red4[kScanThreads / 32];
    __shared__ float red[3][kScanThreads / 32];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    if (p.tokens.at(r, 0) == p.tokens.ignore_idx) {
        if (tid == 0) {
            p.loss[r] = 0.f;
            p.stats[r] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        }
        return;
    }
    const char* x = p.x + p.row.at(r) * sizeof(T);
    constexpr int EACH = kMaxListed / kScanThreads;
    float z[EACH], xv[EACH];
    bool bad = false;
    float zm = -INFINITY;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int k = tid + i * kScanThreads;
        z[i] = -INFINITY;
        xv[i] = 0.f;
        if (k < p.tokens.n) {
            const int64_t y = p.tokens.at(r, k);
            if (y != p.tokens.ignore_idx) {
                if (y < 0 || y >= p.V) {
                    bad = true;
                } else {
                    z[i] = teacher_at(p.teacher, p.teacher_dtype, p.trow.at(r) + k * p.tstep);
                    xv[i] = Vec<T>::load1(x + y * sizeof(T));
                }
            }
        }
        zm = fmaxf(zm, z[i]);
    }
    Stat st = stat_identity();
    if (tid < p.segs) {
        const float4 v = p.part[r * p.segs + tid];
        st = Stat{v.x, v.y, v.z};
    }
    st = stat_block(st, p.L, red4);
    const bool none = stat_none(st.m, st.d);
    const float logd = none ? 0.f : logf(st.d);
    zm = scan_max(zm, red[0]);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (z[i] != -INFINITY) sum += ex2_approx((z[i] - zm) * p.L);
    sum = scan_sum(sum, red[1]);
    const bool nothing = zm == -INFINITY && sum == 0.f;  // no token has any probability
    const float logs = nothing ? 0.f : logf(sum);
    float loss = 0.f;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (z[i] == -INFINITY) continue;
        const float lq = p.normalize ? (z[i] - zm) * p.scale - logs : z[i] * p.scale;
        const float lp = none ? -INFINITY : (xv[i] - st.m) * p.scale - logd;
        const float q = ex2_approx(lq * kLog2e);
        loss += q == 0.f ? 0.f : q * (lq - lp);
    }
    loss = scan_sum(loss, red[2]);
    const bool wrong = scan_count(bad) > 0;
    if (tid == 0) {
        if (wrong) atomicOr(p.err, CE_DEVERR_TARGET_RANGE);
        p.loss[r] = wrong ? NAN : p.tau * p.tau * loss;
        p.stats[r] = make_float4(st.m, logd, zm, logs);
    }
}

struct Layout {
    ScanPlan plan;
    size_t loss, stats, part, bytes;
};
Layout layout(int64_t N, int64_t V, int es) {
    Layout l;
    l.plan = plan_scan(N, V, es);
    l.loss = kWsHeaderBytes;
    l.stats = l.loss + align_up((size_t)N * 4, 256);
    l.part = l.stats + align_up((size_t)N * 16, 256);
    l.bytes = l.part + align_up((size_t)N * l.plan.segs * 16, 256);
    return l;
}

struct Teacher {
    const int64_t* tokens;
    const int64_t* token_strides;
    const void* logits;
    ce_dtype dtype;
    const int64_t* strides;
    int64_t n;
    float tau;
    int normalize;
    int64_t ignore_idx;
};

ce_status check_teacher(const Teacher& t, int64_t rows) {
    const ce_status st = check_tokens(t.tokens, t.token_strides, t.n, rows);
    if (st != CE_OK) return st;
    if (t.n < 1 || !t.strides) return CE_ERR_INVALID_ARG;
    if (t.dtype < CE_F32 || t.dtype > CE_F16) return CE_ERR_UNSUPPORTED_DTYPE;
    if ((rows > 0 && !t.logits) || reinterpret_cast<uintptr_t>(t.logits) % elem_size(t.dtype))
        return CE_ERR_INVALID_ARG;
    for (int k = 0; k < 3; ++k)
        if (t.strides[k] < 0) return CE_ERR_BAD_STRIDE;
    // beyond these a difference of logits over the temperature leaves float32
    if (!(t.tau >= 1e-4f && t.tau <= 1e4f)) return CE_ERR_INVALID_ARG;
    return CE_OK;
}

SoftGradArgs grad_args(const void* logits, int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides,
                       const Teacher& t, const float4* stats, const float* dloss, const int64_t* n_dev, void* grad,
                       const int64_t* grad_strides) {
    SoftGradArgs a = {};
    a.x = static_cast<const char*>(logits);
    a.out = static_cast<char*>(grad);
    a.row = row_addr(strides[0], strides[1], dim0, dim1);
    a.orow = row_addr(grad_strides[0], grad_strides[1], dim0, dim1);
    a.N = dim0 * dim1;
    a.V = V;
    a.scale = 1.f / t.tau;
    a.L = kLog2e / t.tau;
    a.tokens = row_tokens(t.tokens, t.token_strides, t.n, dim0, dim1, t.ignore_idx);
    a.stats = stats;
    a.teacher = t.logits;
    a.teacher_dtype = t.dtype;
    a.trow = row_addr(t.strides[0], t.strides[1], dim0, dim1);
    a.tstep = t.strides[2];
    a.tau = t.tau;
    a.normalize = t.normalize;
    a.dloss = dloss;
    a.n_dev = n_dev;
    return a;
}

// Forward, and with grad the gradient behind it.
ce_status distill(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides,
                  const Teacher& t, int reduce, const float* dloss, float* loss_out, float* stats_out, void* grad,
                  const int64_t* grad_strides, int64_t* n_out, void* workspace, size_t workspace_bytes,
                  cudaStream_t s) {
    const int64_t N = dim0 * dim1;
    if (reinterpret_cast<uintptr_t>(loss_out) % 4 || reinterpret_cast<uintptr_t>(dloss) % 4 ||
        reinterpret_cast<uintptr_t>(stats_out) % 16 || reinterpret_cast<uintptr_t>(n_out) % 8 || !workspace ||
        reinterpret_cast<uintptr_t>(workspace) % 16)
        return CE_ERR_INVALID_ARG;
    if (!loss_out && (N > 0 || reduce)) return CE_ERR_INVALID_ARG;
    const Layout l = layout(N, V, elem_size(dtype));
    if (workspace_bytes < l.bytes) return CE_ERR_WORKSPACE_TOO_SMALL;
    char* ws = static_cast<char*>(workspace);
    // the first token of each row says whether the row counts
    const int64_t ts[2] = {t.token_strides[0], t.token_strides[1]};
    Problem pb;
    problem_init(pb, logits, dtype, dim0, dim1, V, strides, t.tokens, ts, 0.f, t.ignore_idx, reduce);
    pb.err = reinterpret_cast<uint32_t*>(ws + kWsErrOffset);
    pb.n_dev = reinterpret_cast<int64_t*>(ws + kWsCountOffset);
    pb.ticket = reinterpret_cast<uint32_t*>(ws + kWsTicketOffset);
    pb.loss_rows = reduce ? reinterpret_cast<float*>(ws + l.loss) : loss_out;
    cudaError_t e = launch_count(pb, n_out, s);
    if (e != cudaSuccess) return launch_failed();
    if (N > 0) {
        ScanArgs a = {};
        a.x = static_cast<const char*>(logits);
        a.row = row_addr(strides[0], strides[1], dim0, dim1);
        a.N = N;
        a.V = V;
        a.scale = 1.f / t.tau;
        a.L = kLog2e / t.tau;
        a.segs = l.plan.segs;
        a.per = l.plan.per;
        a.tokens = row_tokens(t.tokens, t.token_strides, t.n, dim0, dim1, t.ignore_idx);
        a.skip_first = 1;
        a.part = reinterpret_cast<float4*>(ws + l.part);
        e = launch_scan(a, dtype, false, s);
        if (e != cudaSuccess) return launch_failed();
        DistillArgs d = {};
        d.x = a.x;
        d.row = a.row;
        d.N = N;
        d.V = V;
        d.L = a.L;
        d.scale = a.scale;
        d.tau = t.tau;
        d.tokens = a.tokens;
        d.teacher = t.logits;
        d.teacher_dtype = t.dtype;
        d.trow = row_addr(t.strides[0], t.strides[1], dim0, dim1);
        d.tstep = t.strides[2];
        d.normalize = t.normalize;
        d.segs = a.segs;
        d.part = a.part;
        d.loss = pb.loss_rows;
        d.stats = stats_out ? reinterpret_cast<float4*>(stats_out) : reinterpret_cast<float4*>(ws + l.stats);
        d.err = pb.err;
        if (dtype == CE_F32) ce_distill_row_kernel<float><<<(unsigned)N, kScanThreads, 0, s>>>(d);
        else if (dtype == CE_BF16) ce_distill_row_kernel<__nv_bfloat16><<<(unsigned)N, kScanThreads, 0, s>>>(d);
        else ce_distill_row_kernel<__half><<<(unsigned)N, kScanThreads, 0, s>>>(d);
        if (cudaGetLastError() != cudaSuccess) return CE_ERR_LAUNCH;
        if (grad) {
            e = launch_softgrad(grad_args(logits, dim0, dim1, V, strides, t, d.stats, dloss,
                                          reduce ? pb.n_dev : nullptr, grad, grad_strides),
                                dtype, s);
            if (e != cudaSuccess) return launch_failed();
        }
    }
    if (reduce && launch_reduce_mean(pb, loss_out, s) != cudaSuccess) return launch_failed();
    return CE_OK;
}

}  // namespace
}  // namespace gbce

extern "C" size_t ce_distill_workspace_bytes(int64_t N, int64_t V, ce_dtype dtype) {
    using namespace gbce;
    if (dtype < CE_F32 || dtype > CE_F16 || N < 0 || N > 0x7fffffffLL || V < 1 || V > 0x7fffffffLL) return 0;
    return layout(N, V, elem_size(dtype)).bytes;
}

extern "C" ce_status ce_distill_fwd_bwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                        const int64_t strides[3], const int64_t* teacher_tokens,
                                        const int64_t teacher_token_strides[3], const void* teacher_logits,
                                        ce_dtype teacher_dtype, const int64_t teacher_strides[3], int64_t K,
                                        float temperature, int normalize, int64_t ignore_idx, int reduce_loss,
                                        const float* dloss, float* loss_out, void* grad,
                                        const int64_t grad_strides[3], int64_t* n_non_ignore_out, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    using namespace gbce;
    ce_status st = check_rows(logits, dtype, dim0, dim1, V, strides);
    if (st != CE_OK) return st;
    const Teacher t{teacher_tokens, teacher_token_strides, teacher_logits, teacher_dtype, teacher_strides, K,
                    temperature, normalize, ignore_idx};
    if ((st = check_teacher(t, dim0 * dim1)) != CE_OK) return st;
    if ((st = check_grad(logits, dtype, dim0, dim1, V, strides, grad, grad_strides)) != CE_OK) return st;
    return distill(logits, dtype, dim0, dim1, V, strides, t, reduce_loss, dloss, loss_out, nullptr, grad,
                   grad_strides, n_non_ignore_out, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" ce_status ce_distill_fwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                    const int64_t strides[3], const int64_t* teacher_tokens,
                                    const int64_t teacher_token_strides[3], const void* teacher_logits,
                                    ce_dtype teacher_dtype, const int64_t teacher_strides[3], int64_t K,
                                    float temperature, int normalize, int64_t ignore_idx, int reduce_loss,
                                    float* loss_out, float* stats, int64_t* n_non_ignore_out, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    using namespace gbce;
    ce_status st = check_rows(logits, dtype, dim0, dim1, V, strides);
    if (st != CE_OK) return st;
    const Teacher t{teacher_tokens, teacher_token_strides, teacher_logits, teacher_dtype, teacher_strides, K,
                    temperature, normalize, ignore_idx};
    if ((st = check_teacher(t, dim0 * dim1)) != CE_OK) return st;
    return distill(logits, dtype, dim0, dim1, V, strides, t, reduce_loss, nullptr, loss_out, stats, nullptr, nullptr,
                   n_non_ignore_out, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" ce_status ce_distill_bwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                    const int64_t strides[3], const int64_t* teacher_tokens,
                                    const int64_t teacher_token_strides[3], const void* teacher_logits,
                                    ce_dtype teacher_dtype, const int64_t teacher_strides[3], int64_t K,
                                    float temperature, int normalize, int64_t ignore_idx, int reduce_loss,
                                    const float* stats, const float* dloss, const int64_t* n_non_ignore, void* grad,
                                    const int64_t grad_strides[3], void* stream) {
    using namespace gbce;
    ce_status st = check_rows(logits, dtype, dim0, dim1, V, strides);
    if (st != CE_OK) return st;
    const Teacher t{teacher_tokens, teacher_token_strides, teacher_logits, teacher_dtype, teacher_strides, K,
                    temperature, normalize, ignore_idx};
    if ((st = check_teacher(t, dim0 * dim1)) != CE_OK) return st;
    if ((st = check_grad(logits, dtype, dim0, dim1, V, strides, grad, grad_strides)) != CE_OK) return st;
    if (reinterpret_cast<uintptr_t>(stats) % 16 || reinterpret_cast<uintptr_t>(dloss) % 4 ||
        reinterpret_cast<uintptr_t>(n_non_ignore) % 8)
        return CE_ERR_INVALID_ARG;
    if (dim0 * dim1 > 0 && (!stats || (reduce_loss && !n_non_ignore))) return CE_ERR_INVALID_ARG;
    if (dim0 * dim1 == 0) return CE_OK;
    const SoftGradArgs a = grad_args(logits, dim0, dim1, V, strides, t, reinterpret_cast<const float4*>(stats), dloss,
                                     reduce_loss ? n_non_ignore : nullptr, grad, grad_strides);
    return launch_softgrad(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CE_OK : launch_failed();
}
