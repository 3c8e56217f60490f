// ce_softgrad.cu -- gradients through a row's log-probabilities, from the statistics
// {m, log d, ...} that the forward pass has saved (the exponentials' maximum and the
// log of their sum).
//
// With lp_j = (x_j - m) / temperature - log d and p_j = exp(lp_j):
//   log-probabilities g_k of listed tokens t_k and the entropy's h:
//     grad_j = sum_k g_k [t_k = j] - p_j sum_k g_k - h p_j (lp_j + H)
//   distillation, q_k the teacher's probabilities of its tokens t_k, Q their sum:
//     grad_j = g temperature (Q p_j - sum_k q_k [t_k = j])
// Both are p_j (a + b lp_j) with two numbers a row, and something more at the few
// listed columns.  Bound by HBM: a logit read, a gradient written.  A CTA streams a
// run of a row's columns, by the output's 16-byte vectors, and then writes the run's
// listed columns again; their logits are read before the stream, which may replace
// them.  A token listed twice gets the sum of its entries.
// Measured: 4096 x 128000 bf16, one token a row, 308 us (6.8 TB/s, the copy rate); 2048 x
// 65536, 128 tokens, 101 us (5.1 TB/s), where every CTA's list comes before its stream.
#include <math.h>

#include "ce_rowscan.h"

namespace gbce {
namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;

// The CTA's sum of v, in a fixed order.
__device__ __forceinline__ float cta_sum(float v, float* red) {
    v = warp_allsum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += red[w];
    return t;
}

struct Listed {
    int col[kMaxListed];
    float coef[kMaxListed], x[kMaxListed];
    uint16_t slot[2 * kMaxListed];  // of the table that finds tokens listed twice (ce_list_table.h)
};

template <typename T, bool SECOND>  // SECOND: b is not zero
__global__ void __launch_bounds__(kThreads) ce_softgrad_kernel(const __grid_constant__ SoftGradArgs p) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems, ES = sizeof(T), PP = VEC / 2, U = 4;
    __shared__ Listed ls;
    __shared__ float red[kThreads / 32];
    __shared__ int wn[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r = blockIdx.x / p.runs, run = blockIdx.x - r * p.runs;
    const int64_t c0 = run * p.cols;
    const int n = (int)min(p.cols, p.V - c0);
    const char* x = p.x + (p.row.at(r) + c0) * ES;
    char* out = p.out + (p.orow.at(r) + c0) * ES;
    const float4 st = __ldg(p.stats + r);

    // the row's scale, and the run's listed columns in list order
    const bool distill = p.teacher != nullptr;
    float gt = 1.f, total = 0.f;
    if (distill) {
        const float g = p.n_dev ? (p.dloss ? __ldg(p.dloss) : 1.f) / (float)(*p.n_dev)
                                : (p.dloss ? __ldg(p.dloss + r) : 1.f);
        gt = g * p.tau;
    }
    bool keep = p.tokens.n == 0, bad = false;
    int listed = 0;
    for (int k0 = 0; k0 < p.tokens.n; k0 += kThreads) {
        const int k = k0 + tid;
        bool in = false;
        int col = 0;
        float c = 0.f;
        if (k < p.tokens.n) {
            const int64_t y = p.tokens.at(r, k);
            if (y != p.tokens.ignore_idx) {
                keep = true;
                if (y < 0 || y >= p.V) {
                    bad = true;
                } else {
                    if (distill) {
                        const float z = teacher_at(p.teacher, p.teacher_dtype, p.trow.at(r) + k * p.tstep);
                        const float lq = p.normalize ? (z - st.z) * p.scale - st.w : z * p.scale;
                        c = z == -INFINITY ? 0.f : -gt * ex2_approx(lq * kLog2e);
                    } else if (p.grad_logprobs) {
                        c = __ldg(p.grad_logprobs + r * p.tokens.n + k);
                        total += c;
                    }
                    in = y >= c0 && y < c0 + n;
                    col = (int)(y - c0);
                }
            }
        }
        const unsigned m = __ballot_sync(kFull, in);
        if (lane == 0) wn[warp] = __popc(m);
        __syncthreads();
        int at = listed, all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += wn[w];
            all += wn[w];
        }
        if (in) {
            at += __popc(m & ((1u << lane) - 1u));
            ls.col[at] = col;
            ls.coef[at] = c;
            ls.x[at] = VT::load1(x + (int64_t)col * ES);
        }
        listed += all;
        __syncthreads();
    }
    bool zero = stat_none(st.x, st.y);
    float a, b = 0.f;
    if (distill) {
        zero |= p.tokens.at(r, 0) == p.tokens.ignore_idx;
        zero |= __syncthreads_or(bad) != 0;
        // Q: 0 where the teacher gives no token any probability, NaN where its logits are no numbers
        const float Q = st.w != st.w         ? st.w
                        : st.z == -INFINITY  ? 0.f
                        : p.normalize        ? 1.f
                                             : ex2_approx((st.z * p.scale + st.w) * kLog2e);
        a = gt * Q;
    } else {
        if (p.tokens.n > 0) {
            zero |= __syncthreads_or(keep) == 0;
            total = cta_sum(total, red);
        }
        b = SECOND ? -__ldg(p.grad_entropy + r) : 0.f;
        a = SECOND ? fmaf(b, st.z, -total) : -total;
        b *= kLn2;
    }
    const float shift = -st.y * kLog2e, nm = -st.x;
    auto grad = [&](float v) -> float {
        float y = fmaf(v + nm, p.L, shift);
        const float e = ex2_approx(y);
        return SECOND ? e * fmaf(b, fmaxf(y, kFarBelow), a) : e * a;
    };

    const Span16 sp = span16<ES>(out, 0, n);
    const int nv = (int)sp.nv, off = (int)sp.h1;
    uint4* to = reinterpret_cast<uint4*>(out + off * ES);
    const int edge = (int)span16_edge(sp, 0, n, tid);
    if (zero) {
        for (int v = tid; v < nv; v += kThreads) stg128_stream(to + v, make_uint4(0, 0, 0, 0));
        if (edge >= 0) VT::store1(out + edge * ES, 0.f);
        return;
    }
    if (edge >= 0) VT::store1(out + edge * ES, grad(VT::load1(x + edge * ES)));
    // inputs at another offset from 16 bytes than the outputs are cut out of two vectors
    // that both lie inside the row
    const uint32_t ph = (uint32_t)(reinterpret_cast<uintptr_t>(x + off * ES) & 15u);
    const uint4* in = reinterpret_cast<const uint4*>(x + off * ES - ph);
    const int safe0 = ph && c0 + off < (int64_t)(ph / ES) ? 1 : 0;
    const int64_t room = ((p.V - c0 - off) * ES + ph) / 16 - 1;
    const int safe1 = (int)min(room, (int64_t)nv);
    auto load = [&](int v) -> uint4 {
        if (ph == 0) return __ldcs(in + v);
        if (v >= safe0 && v < safe1) return shift_bytes(__ldg(in + v), __ldg(in + v + 1), ph);
        float f[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = VT::load1(x + (off + v * VEC + k) * ES);
        return VT::pack(f);
    };
    const float2 NM = make_float2(nm, nm), LL = make_float2(p.L, p.L), SH = make_float2(shift, shift);
    const float2 A = make_float2(a, a), B = make_float2(b, b);
    for (int v0 = tid; v0 < nv; v0 += kThreads * U) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + u * kThreads < nv) raw[u] = load(v0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v0 + u * kThreads >= nv) continue;
            float2 f[PP];
            VT::unpack2(raw[u], f);
#pragma unroll
            for (int k = 0; k < PP; ++k) {
                float2 y = __ffma2_rn(__fadd2_rn(f[k], NM), LL, SH);
                const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                if (SECOND) {
                    y.x = fmaxf(y.x, kFarBelow);
                    y.y = fmaxf(y.y, kFarBelow);
                    f[k] = __fmul2_rn(e, __ffma2_rn(B, y, A));
                } else {
                    f[k] = __fmul2_rn(e, A);
                }
            }
            stg128_stream(to + v0 + u * kThreads, VT::pack2(f));
        }
    }
    if (listed == 0) return;
    // Of a token's entries one writes for all.  Up to 64 are looked at by each other; of more, the
    // first to find a slot of a hash table writes, and a warp sums what belongs to it, in an
    // order fixed by the list (4096 x 32000, bf16, drawn with replacement, 64 tokens: 98 us, with the
    // table 105; 256: 143 and 118; 1024: 1110 and 212).
    if (listed <= 64) {
        __syncthreads();
        if (tid >= listed) return;
        const int col = ls.col[tid];
        float c = 0.f;
        bool first = true;
        for (int j = 0; j < listed; ++j) {
            if (ls.col[j] != col) continue;
            if (j < tid) first = false;
            c += ls.coef[j];
        }
        if (first) VT::store1(out + (int64_t)col * ES, grad(ls.x[tid]) + c);
        return;
    }
    int slots = 64;
    while (slots < 2 * listed) slots *= 2;
    for (int h = tid; h < slots; h += kThreads) ls.slot[h] = kSlotFree;
    __syncthreads();
    for (int k = tid; k < listed; k += kThreads) {
        const int col = ls.col[k];
        if (list_enter(ls.slot, (uint32_t)slots, k, col, [&](int j) { return ls.col[j]; }, slot_cas)) ls.col[k] = -2 - col;
    }
    __syncthreads();
    for (int h = warp * 32; h < slots; h += kThreads) {
        const unsigned mine = ls.slot[h + lane];
        for (unsigned m = __ballot_sync(kFull, slot_twice(mine)); m; m &= m - 1u) {
            const int k = slot_entry(__shfl_sync(kFull, mine, __ffs(m) - 1)), col = ls.col[k];
            float c = 0.f;
            for (int j = lane; j < listed; j += 32)
                if (ls.col[j] == col || ls.col[j] == -2 - col) c += ls.coef[j];
            c = warp_allsum(c);
            __syncwarp();
            if (lane == 0) ls.coef[k] = c;
        }
    }
    __syncthreads();
    for (int k = tid; k < listed; k += kThreads) {
        const int col = ls.col[k];
        if (col >= 0) VT::store1(out + (int64_t)col * ES, grad(ls.x[k]) + ls.coef[k]);
    }
}

template <typename T>
cudaError_t launch_softgrad_t(const SoftGradArgs& a, cudaStream_t s) {
    const int64_t grid = a.N * a.runs;
    if (a.grad_entropy)
        ce_softgrad_kernel<T, true><<<(unsigned)grid, kThreads, 0, s>>>(a);
    else
        ce_softgrad_kernel<T, false><<<(unsigned)grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Runs of 32 KB; longer ones under lists of more than 4, which every CTA of a row walks
// through, while that leaves the SMs several rounds (20 tokens of 4096 x 128000 bf16: 326 us,
// in runs of 32 KB 364), and where the grid would not hold them;
// shorter ones (down to 4 KB) where few rows leave SMs without.
cudaError_t launch_softgrad(SoftGradArgs a, int dtype, cudaStream_t s) {
    const int vec = 16 / elem_size(dtype);
    a.cols = (int64_t)kThreads * 8 * vec;
    while (a.cols > kThreads * vec && a.N * ((a.V + a.cols - 1) / a.cols) < 2 * kScanSlots) a.cols /= 2;
    while (a.tokens.n > 4 && a.cols < a.V && a.N * ((a.V + 2 * a.cols - 1) / (2 * a.cols)) >= 4096) a.cols *= 2;
    while (a.N * ((a.V + a.cols - 1) / a.cols) > 0x7fffffffLL) a.cols *= 2;
    a.runs = (a.V + a.cols - 1) / a.cols;
    if (dtype == CE_F32) return launch_softgrad_t<float>(a, s);
    if (dtype == CE_BF16) return launch_softgrad_t<__nv_bfloat16>(a, s);
    return launch_softgrad_t<__half>(a, s);
}

ce_status check_grad(const void* logits, int dtype, int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides,
                     const void* grad, const int64_t* grad_strides) {
    if (!grad_strides || (dim0 * dim1 > 0 && !grad) || reinterpret_cast<uintptr_t>(grad) % elem_size(dtype))
        return CE_ERR_INVALID_ARG;
    if (grad_strides[2] != 1 || grad_strides[0] < 0 || grad_strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (!rows_apart(dim0, dim1, V, grad_strides)) return CE_ERR_BAD_STRIDE;
    if (grad == logits && (grad_strides[0] != strides[0] || grad_strides[1] != strides[1]))
        return CE_ERR_BAD_STRIDE;  // in place means the same strides
    return CE_OK;
}

}  // namespace gbce

extern "C" ce_status ce_logprobs_bwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                     const int64_t strides[3], const int64_t* tokens, const int64_t token_strides[3],
                                     int64_t given, int64_t ignore_idx, const float* stats,
                                     const float* grad_logprobs, const float* grad_entropy, void* grad,
                                     const int64_t grad_strides[3], void* stream) {
    using namespace gbce;
    ce_status st = check_rows(logits, dtype, dim0, dim1, V, strides);
    if (st != CE_OK) return st;
    const int64_t N = dim0 * dim1;
    if ((st = check_tokens(tokens, token_strides, given, N)) != CE_OK) return st;
    if ((st = check_grad(logits, dtype, dim0, dim1, V, strides, grad, grad_strides)) != CE_OK) return st;
    if (reinterpret_cast<uintptr_t>(stats) % 16 || reinterpret_cast<uintptr_t>(grad_logprobs) % 4 ||
        reinterpret_cast<uintptr_t>(grad_entropy) % 4)
        return CE_ERR_INVALID_ARG;
    if (N > 0 && (!stats || (grad_logprobs && given == 0))) return CE_ERR_INVALID_ARG;
    if (N == 0) return CE_OK;
    SoftGradArgs a = {};
    a.x = static_cast<const char*>(logits);
    a.out = static_cast<char*>(grad);
    a.row = row_addr(strides[0], strides[1], dim0, dim1);
    a.orow = row_addr(grad_strides[0], grad_strides[1], dim0, dim1);
    a.N = N;
    a.V = V;
    a.L = kLog2e;
    a.scale = 1.f;
    a.tokens = row_tokens(tokens, token_strides, given, dim0, dim1, ignore_idx);
    a.stats = reinterpret_cast<const float4*>(stats);
    a.grad_logprobs = grad_logprobs;
    a.grad_entropy = grad_entropy;
    return launch_softgrad(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CE_OK : launch_failed();
}
