// ce_logits.cu -- penalties, biases, a grammar's bit mask and the temperature
// on the logits, and the gradient through them.
//
// Per row, with c_j the number of times token j occurs in the answer so far
// (the history past its first prompt_length tokens), s_j whether it occurs in
// the history at all, b_j the summed biases given for it:
//   z_j = s_j ? (x_j > 0 ? x_j / rep : x_j rep) : x_j
//   y_j = (z_j - freq c_j - pres [c_j > 0] + b_j) / temp
//   out_j = allowed_j ? y_j : mask_value
// Backward: dx_j = allowed_j ? dy_j / temp * (s_j ? (x_j > 0 ? 1/rep : rep) : 1) : 0.
//
// Bound by HBM: each allowed logit is read once and each output written once.
// A CTA takes one row's run of columns.  The few columns that the history or
// the biases touch are counted in shared memory first (integer atomics, so any
// order gives the same counts; the biases of one column are added in list
// order by one warp).
#include "ce_device.cuh"
#include "ce_internal.h"
#include "ce_pack.cuh"
#include "ce_span.cuh"

namespace gbce {
namespace {

constexpr int kLogitThreads = 256;
constexpr int kLogitCols = 4096;       // columns of a CTA, a multiple of 32
constexpr uint32_t kSeen = 0x80000000u;  // the token occurs; the low bits count its occurrences in the answer

struct LogitArgs {
    const char* x;         // logits (backward: read where the history touches them)
    const char* g;         // backward: the gradient of the outputs, else NULL
    char* out;
    int64_t xs0, xs1, gs0, gs1, os0, os1;  // in elements
    int64_t dim1, N, V;
    int chunks;            // runs of kLogitCols columns per row
    const int64_t* hist;
    int64_t hist_stride, hist_max;
    const int64_t* hist_len;
    const int64_t* prompt_len;
    const float* rep;
    const float* freq;
    const float* pres;
    const int64_t* btok;
    const float* bval;
    int64_t btok_stride, bval_stride, bias_max;
    const uint32_t* mask;
    int64_t mask_stride;
    const float* temp;
    float mask_value;
};

// One column's value (or gradient).
struct RowScalars {
    float rep, inv_rep, freq, pres, inv_temp;
};

template <bool BWD>
__device__ __forceinline__ float special(float v, float x, uint32_t word, float bias, const RowScalars& r) {
    if (BWD) return word ? (x > 0.f ? v * r.inv_rep : v * r.rep) : v;
    float z = word ? (x > 0.f ? x * r.inv_rep : x * r.rep) : x;
    const uint32_t c = word & ~kSeen;
    if (c) z = fmaf(-r.freq, (float)c, z) - r.pres;
    return z + bias;
}

template <typename T, bool BWD>
__global__ void __launch_bounds__(kLogitThreads) ce_logits_kernel(const __grid_constant__ LogitArgs p) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems;
    constexpr int ES = sizeof(T);
    __shared__ uint32_t word[kLogitCols];
    __shared__ float bias[kLogitCols];
    const int64_t row = blockIdx.x / p.chunks;
    const int64_t c0 = (int64_t)(blockIdx.x - row * p.chunks) * kLogitCols;
    const int64_t c1 = min(p.V, c0 + kLogitCols);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t i = row / p.dim1, j = row - i * p.dim1;
    const char* x = p.x + (i * p.xs0 + j * p.xs1) * ES;
    const char* src = BWD ? p.g + (i * p.gs0 + j * p.gs1) * ES : x;
    char* out = p.out + (i * p.os0 + j * p.os1) * ES;
    const bool listed = p.hist_max > 0 || p.bias_max > 0;

    RowScalars rs;
    rs.rep = p.rep ? __ldg(p.rep + row) : 1.f;
    rs.inv_rep = 1.f / rs.rep;
    rs.freq = p.freq ? __ldg(p.freq + row) : 0.f;
    rs.pres = p.pres ? __ldg(p.pres + row) : 0.f;
    rs.inv_temp = p.temp ? 1.f / __ldg(p.temp + row) : 1.f;

    if (listed) {
        for (int k = tid; k < (int)(c1 - c0); k += kLogitThreads) {
            word[k] = 0u;
            bias[k] = 0.f;
        }
        __syncthreads();
        if (p.hist_max > 0) {
            int64_t len = p.hist_len ? __ldg(p.hist_len + row) : p.hist_max;
            len = len < 0 ? 0 : (len > p.hist_max ? p.hist_max : len);
            const int64_t prompt = p.prompt_len ? __ldg(p.prompt_len + row) : 0;
            const int64_t* h = p.hist + row * p.hist_stride;
            for (int64_t k = tid; k < len; k += kLogitThreads) {
                const int64_t t = __ldg(h + k);
                if (t >= c0 && t < c1) {
                    if (k < prompt) atomicOr(&word[t - c0], kSeen);
                    else atomicAdd(&word[t - c0], 1u);
                }
            }
        }
        if (!BWD && p.bias_max > 0 && warp == 0) {
            const int64_t* bt = p.btok + row * p.btok_stride;
            const float* bv = p.bval + row * p.bval_stride;
            for (int64_t k0 = 0; k0 < p.bias_max; k0 += 32) {
                const int64_t k = k0 + lane;
                int64_t t = k < p.bias_max ? __ldg(bt + k) : -1;
                const float b = k < p.bias_max ? __ldg(bv + k) : 0.f;
                const bool in = t >= c0 && t < c1;
                const uint32_t key = in ? (uint32_t)(t - c0) : 0xffffffffu;
                unsigned peers = __match_any_sync(kFull, key);
                const bool lead = in && lane == __ffs(peers) - 1;
                // the leader adds its column's biases in list order
                unsigned todo = lead ? peers : 0u;
                float sum = lead ? bias[key] : 0.f;
                while (__any_sync(kFull, todo != 0u)) {
                    const int from = todo ? __ffs(todo) - 1 : 0;
                    const float v = __shfl_sync(kFull, b, from);
                    if (todo) {
                        sum += v;
                        todo &= todo - 1;
                    }
                }
                if (lead) bias[key] = sum;
                __syncwarp();
            }
        }
        __syncthreads();
    }

    const uint32_t* mask = p.mask ? p.mask + row * p.mask_stride : nullptr;
    const float blocked = BWD ? 0.f : p.mask_value;
    auto one = [&](int64_t c) {
        float o = blocked;
        if (!mask || ((__ldg(mask + (c >> 5)) >> (c & 31)) & 1u)) {
            float v = VT::load1(src + c * ES);
            if (listed) {
                const int k = (int)(c - c0);
                const uint32_t w = word[k];
                const float b = bias[k];
                if (BWD) {
                    if (w) v = special<BWD>(v, VT::load1(x + c * ES), w, 0.f, rs);
                } else {
                    v = special<BWD>(v, v, w, b, rs);
                }
            }
            o = v * rs.inv_temp;
        }
        VT::store1(out + c * ES, o);
    };
    const bool vec_ok = ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    if (!vec_ok) {
        for (int64_t c = c0 + tid; c < c1; c += kLogitThreads) one(c);
        return;
    }
    const Span16 sp = span16<ES>(src, c0, c1);
    const int64_t e = span16_edge(sp, c0, c1, tid);
    if (e >= 0) one(e);
    for (int64_t v = tid; v < sp.nv; v += kLogitThreads) {
        const int64_t c = sp.h1 + v * VEC;
        uint32_t bits = 0xffffffffu;
        if (mask) {
            const int64_t w = c >> 5;
            const int sh = (int)(c & 31);
            const uint32_t lo = __ldg(mask + w);
            // the vector's bits may run into the next word
            const uint32_t hi = sh > 32 - VEC ? __ldg(mask + w + 1) : 0u;
            bits = __funnelshift_r(lo, hi, sh);
        }
        float f[VEC];
        VT::unpack(__ldcs(reinterpret_cast<const uint4*>(src + c * ES)), f);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            if (listed) {
                const int k = (int)(c - c0) + q;
                const uint32_t w = word[k];
                const float b = bias[k];
                if (BWD) {
                    if (w) f[q] = special<BWD>(f[q], VT::load1(x + (c + q) * ES), w, 0.f, rs);
                } else {
                    f[q] = special<BWD>(f[q], f[q], w, b, rs);
                }
            }
            f[q] = (bits >> q) & 1u ? f[q] * rs.inv_temp : blocked;
        }
        stg128_stream(out + c * ES, VT::pack(f));
    }
}

template <bool BWD>
cudaError_t launch_logits(const LogitArgs& a, int dtype, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.N * a.chunks);
    if (dtype == CE_F32) ce_logits_kernel<float, BWD><<<grid, kLogitThreads, 0, s>>>(a);
    else if (dtype == CE_BF16) ce_logits_kernel<__nv_bfloat16, BWD><<<grid, kLogitThreads, 0, s>>>(a);
    else ce_logits_kernel<__half, BWD><<<grid, kLogitThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// Rows at (i * s0 + j * s1) that share no element.
bool rows_apart(int64_t d0, int64_t d1, int64_t V, const int64_t* s) {
    int64_t in_s = s[1], in_n = d1, out_s = s[0], out_n = d0;
    if (in_n <= 1 || (out_n > 1 && s[0] < s[1])) {
        in_s = s[0]; in_n = d0; out_s = s[1]; out_n = d1;
    }
    if (in_n > 1 && in_s < V) return false;
    if (out_n > 1 && out_s < (in_n > 1 ? in_s * in_n : V)) return false;
    return true;
}

ce_status logits_common(const void* grad, const int64_t* grad_strides, const void* logits, ce_dtype dtype,
                        int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides,
                        const ce_logits_params* q, void* out, const int64_t* out_strides, bool bwd, cudaStream_t s) {
    if (dtype < CE_F32 || dtype > CE_F16) return CE_ERR_UNSUPPORTED_DTYPE;
    if (!strides || !out_strides || !q || (bwd && !grad_strides)) return CE_ERR_INVALID_ARG;
    if (dim0 < 0 || dim1 < 0 || dim0 > 0x7fffffffLL || dim1 > 0x7fffffffLL || V < 1 || V > 0x7fffffffLL)
        return CE_ERR_INVALID_ARG;
    const int64_t N = dim0 * dim1;
    for (int k = 0; k < 2; ++k)
        if (q->reserved[k] != 0) return CE_ERR_INVALID_ARG;
    if (q->history_max < 0 || q->bias_max < 0) return CE_ERR_INVALID_ARG;
    if (N > 0) {
        if (!logits || !out || (bwd && !grad)) return CE_ERR_INVALID_ARG;
        const uintptr_t all = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out) |
                              reinterpret_cast<uintptr_t>(bwd ? grad : out);
        if (all % elem_size(dtype)) return CE_ERR_INVALID_ARG;
        if (q->history_max > 0 && !q->history) return CE_ERR_INVALID_ARG;
        if (q->bias_max > 0 && (!q->bias_tokens || !q->bias_values)) return CE_ERR_INVALID_ARG;
        if (strides[2] != 1 || strides[0] < 0 || strides[1] < 0) return CE_ERR_BAD_STRIDE;
        if (bwd && (grad_strides[2] != 1 || grad_strides[0] < 0 || grad_strides[1] < 0)) return CE_ERR_BAD_STRIDE;
        if (out_strides[2] != 1 || out_strides[0] < 0 || out_strides[1] < 0) return CE_ERR_BAD_STRIDE;
        if (!rows_apart(dim0, dim1, V, out_strides)) return CE_ERR_BAD_STRIDE;
        if (q->history_stride < 0 || q->bias_tokens_stride < 0 || q->bias_values_stride < 0 || q->mask_stride < 0)
            return CE_ERR_BAD_STRIDE;
        if (q->mask && q->mask_stride != 0 && q->mask_stride < (V + 31) / 32) return CE_ERR_BAD_STRIDE;
        const int64_t* in_s = bwd ? grad_strides : strides;
        if (out == (bwd ? grad : logits) && (out_strides[0] != in_s[0] || out_strides[1] != in_s[1]))
            return CE_ERR_BAD_STRIDE;  // in place means the same strides
        if (bwd && out == logits) return CE_ERR_INVALID_ARG;
    }
    if (N == 0) return CE_OK;
    LogitArgs a;
    a.x = static_cast<const char*>(logits);
    a.g = static_cast<const char*>(grad);
    a.out = static_cast<char*>(out);
    a.xs0 = strides[0];
    a.xs1 = strides[1];
    a.gs0 = bwd ? grad_strides[0] : 0;
    a.gs1 = bwd ? grad_strides[1] : 0;
    a.os0 = out_strides[0];
    a.os1 = out_strides[1];
    a.dim1 = dim1;
    a.N = N;
    a.V = V;
    a.chunks = (int)((V + kLogitCols - 1) / kLogitCols);
    if (N > 0x7fffffffLL / a.chunks) return CE_ERR_INVALID_ARG;
    a.hist = q->history;
    a.hist_stride = q->history_stride;
    a.hist_max = q->history_max;
    a.hist_len = q->history_lengths;
    a.prompt_len = q->prompt_lengths;
    a.rep = q->repetition_penalty;
    a.freq = q->frequency_penalty;
    a.pres = q->presence_penalty;
    a.btok = q->bias_tokens;
    a.bval = q->bias_values;
    a.btok_stride = q->bias_tokens_stride;
    a.bval_stride = q->bias_values_stride;
    a.bias_max = bwd ? 0 : q->bias_max;
    a.mask = reinterpret_cast<const uint32_t*>(q->mask);
    a.mask_stride = q->mask_stride;
    a.temp = q->temperature;
    a.mask_value = q->mask_value;
    if (bwd && !a.rep) a.hist_max = 0;  // only the repetition penalty scales the gradient
    cudaError_t e = bwd ? launch_logits<true>(a, dtype, s) : launch_logits<false>(a, dtype, s);
    return e == cudaSuccess ? CE_OK : CE_ERR_LAUNCH;
}

}  // namespace
}  // namespace gbce

extern "C" ce_status ce_logits_process(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                       const int64_t strides[3], const ce_logits_params* params, void* out,
                                       const int64_t out_strides[3], void* stream) {
    return gbce::logits_common(nullptr, nullptr, logits, dtype, dim0, dim1, V, strides, params, out, out_strides,
                               false, static_cast<cudaStream_t>(stream));
}

extern "C" ce_status ce_logits_process_bwd(const void* grad_out, const int64_t grad_out_strides[3],
                                           const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                           const int64_t strides[3], const ce_logits_params* params, void* grad,
                                           const int64_t grad_strides[3], void* stream) {
    return gbce::logits_common(grad_out, grad_out_strides, logits, dtype, dim0, dim1, V, strides, params, grad,
                               grad_strides, true, static_cast<cudaStream_t>(stream));
}
