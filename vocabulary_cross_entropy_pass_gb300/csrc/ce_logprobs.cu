// ce_logprobs.cu -- log-probabilities of given tokens, the entropy and the largest
// logits of each row, and their C entry points.
//
//   lp_j = x_j - logsumexp(x),   H = -sum_j exp(lp_j) lp_j,
//   top: the K largest x in falling order (ties: the lower column first), with lp
//
// Bound by HBM: every logit is read once.  ce_scan_kernel reads a segment of a row in
// tiles of 16 KB, sums its statistics and selects its candidates (ce_rowscan.cuh);
// a row in one piece is finished by the CTA that read it, a row in segments by
// ce_join_kernel from their partial results.
#include <math.h>

#include "ce_rowscan.h"

namespace gbce {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Whether row r is left out.  All scanning threads; a barrier where a row has several tokens.
__device__ __forceinline__ bool row_skipped(const RowTokens& t, int64_t r, bool first) {
    if (t.n == 0) return false;
    if (first || t.n == 1) return t.at(r, 0) == t.ignore_idx;
    bool keep = false;
    for (int k = threadIdx.x; k < t.n; k += kScanThreads) keep |= t.at(r, k) != t.ignore_idx;
    return scan_count(keep) == 0;
}

__device__ __forceinline__ void write_skipped(const ScanArgs& p, int64_t r) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        if (p.entropy) p.entropy[r] = 0.f;
        if (p.stats) p.stats[r] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    }
    for (int k = tid; k < p.tokens.n; k += kScanThreads) p.logprobs[r * p.tokens.n + k] = 0.f;
    for (int k = tid; k < p.top_k; k += kScanThreads) {
        p.top_tokens[r * p.top_k + k] = p.tokens.ignore_idx;
        p.top_logprobs[r * p.top_k + k] = 0.f;
    }
}

// A row's outputs from its statistics and its candidates in falling order (c of them).
template <typename T>
__device__ __forceinline__ void finish_row(const ScanArgs& p, int64_t r, const Stat& t, const uint64_t* top, int c) {
    const int tid = threadIdx.x;
    const bool none = stat_none(t.m, t.d);
    const float logd = none ? 0.f : logf(t.d);
    if (tid == 0) {
        const float h = none ? 0.f : logd - kLn2 * t.s / t.d;
        if (p.entropy) p.entropy[r] = h;
        if (p.stats) p.stats[r] = make_float4(t.m, logd, h, 0.f);
    }
    const char* x = p.x + p.row.at(r) * sizeof(T);
    for (int k = tid; k < p.tokens.n; k += kScanThreads) {
        const int64_t y = p.tokens.at(r, k);
        float lp = 0.f;
        if (y != p.tokens.ignore_idx) {
            if (y < 0 || y >= p.V) {
                lp = NAN;
                atomicOr(p.err, CE_DEVERR_TARGET_RANGE);
            } else {
                lp = none ? -INFINITY : (Vec<T>::load1(x + y * sizeof(T)) - t.m) - logd;
            }
        }
        p.logprobs[r * p.tokens.n + k] = lp;
    }
    for (int k = tid; k < p.top_k; k += kScanThreads) {
        int64_t token = -1;  // NaN is no alternative: a row of fewer than K others ends so
        float lp = NAN;
        if (k < c) {
            token = key_column(top[k]);
            lp = none ? -INFINITY : (key_value(top[k]) - t.m) - logd;
        }
        p.top_tokens[r * p.top_k + k] = token;
        p.top_logprobs[r * p.top_k + k] = lp;
    }
}

template <typename T, bool TOP, bool ENT>
__global__ void __launch_bounds__(kScanThreads) ce_scan_kernel(const __grid_constant__ ScanArgs p) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems, ES = sizeof(T);
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float4 red[kScanThreads / 32];
    TopSmem& top = *reinterpret_cast<TopSmem*>(sm);
    const int tid = threadIdx.x;
    for (int64_t item = blockIdx.x; item < p.N * p.segs; item += gridDim.x) {
        const int64_t r = item / p.segs;
        const int seg = (int)(item - r * p.segs);
        if (row_skipped(p.tokens, r, p.skip_first)) {
            if (!p.part) write_skipped(p, r);
            continue;
        }
        const char* x = p.x + p.row.at(r) * ES;
        const Span16 sp = span16<ES>(x, 0, p.V);
        const int64_t v0 = min(sp.nv, seg * p.per), v1 = seg == p.segs - 1 ? sp.nv : min(sp.nv, v0 + p.per);
        const T* body = reinterpret_cast<const T*>(x + sp.h1 * ES);
        // the elements before the body go with the first segment, those after it with the last
        const bool head = seg == 0 && tid < sp.h1;
        const bool tail = seg == p.segs - 1 && sp.t0 + tid < p.V;
        const float xh = head ? VT::load1(x + tid * ES) : -INFINITY;
        const float xt = tail ? VT::load1(x + (sp.t0 + tid) * ES) : -INFINITY;
        Stat st = stat_identity();
        if (head) stat_add(st, xh, p.L);
        if (tail) stat_add(st, xt, p.L);
        TopState ts = {};
        const int64_t ntiles = (v1 - v0 + kScanTileVecs - 1) / kScanTileVecs;
        for (int64_t t = 0; t < ntiles || t == 0; ++t) {
            const int64_t f = v0 + t * kScanTileVecs;
            const int n = (int)min((int64_t)kScanTileVecs, v1 - f);
            const T* tile = body + f * VEC;
            uint4 raw[kScanVecs];
            bool have[kScanVecs];
#pragma unroll
            for (int i = 0; i < kScanVecs; ++i) {
                have[i] = tid + i * kScanThreads < n;
                if (have[i]) raw[i] = __ldg(reinterpret_cast<const uint4*>(tile) + tid + i * kScanThreads);
            }
            float mx = stat_tile<T, kScanVecs, ENT>(st, raw, have, p.L);
            if constexpr (TOP) {
                const bool edge = t == 0 && head;
                if (edge) mx = fmaxf(mx, xh);
                if (t == 0) ts = top_start(top, p.top_k, have[0] || edge, mx);
                top_tile<T>(top, ts, have[0] || edge, mx, tile, n, (uint32_t)(sp.h1 + f * VEC), edge, xh, tid);
                if (t == 0 && !ts.all) ts.strict = true;
            }
        }
        int c = 0;
        if constexpr (TOP) {
            const bool more = tail && ts.takes(xt);
            if (scan_count(more) > 0) {
                if (ts.bound + VEC > kTopCap) ts.compact(top);
                if (more && ts.takes(xt)) top_push_one(top, xt, (uint32_t)(sp.t0 + tid));
            }
            ts.compact(top);
            c = ts.bound;
        }
        st = stat_block(st, p.L, red);
        if (p.part) {
            if (tid == 0) p.part[item] = make_float4(st.m, st.d, st.s, __int_as_float(c));
            for (int k = tid; k < c; k += kScanThreads) p.cand[item * p.top_k + k] = top.buf[k];
        } else {
            finish_row<T>(p, r, st, top.buf, c);
        }
        scan_sync();
    }
}

// A row's segments put together.
template <typename T>
__global__ void __launch_bounds__(kScanThreads) ce_join_kernel(const __grid_constant__ ScanArgs p) {
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float4 red[kScanThreads / 32];
    TopSmem& top = *reinterpret_cast<TopSmem*>(sm);
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    if (row_skipped(p.tokens, r, p.skip_first)) {
        write_skipped(p, r);
        return;
    }
    Stat st = stat_identity();
    if (tid < p.segs) {
        const float4 v = p.part[r * p.segs + tid];
        st = Stat{v.x, v.y, v.z};
    }
    st = stat_block(st, p.L, red);
    int c = 0;
    if (p.top_k > 0) {
        TopState ts = {};
        ts.K = p.top_k;
        ts.all = true;
        ts.T = -INFINITY;
        if (tid == 0) top.count = 0;
        scan_sync();
        for (int g = 0; g < p.segs; ++g) {
            const int n = __float_as_int(p.part[r * p.segs + g].w);
            if (ts.bound + n > kTopCap) ts.compact(top);
            const int base = ts.bound;
            for (int k = tid; k < n; k += kScanThreads) top.buf[base + k] = p.cand[(r * p.segs + g) * p.top_k + k];
            ts.bound += n;
            if (tid == 0) top.count = ts.bound;
        }
        ts.compact(top);
        c = ts.bound;
    }
    finish_row<T>(p, r, st, top.buf, c);
}

template <typename T, bool TOP, bool ENT>
cudaError_t launch_scan_t(const ScanArgs& a, cudaStream_t s) {
    const size_t smem = TOP ? sizeof(TopSmem) : 0;
    auto* k = ce_scan_kernel<T, TOP, ENT>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    const int64_t items = a.N * a.segs;
    k<<<(unsigned)(items < (1 << 30) ? items : (1 << 30)), kScanThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scan_type(const ScanArgs& a, bool entropy, cudaStream_t s) {
    if (a.top_k > 0) return entropy ? launch_scan_t<T, true, true>(a, s) : launch_scan_t<T, true, false>(a, s);
    return entropy ? launch_scan_t<T, false, true>(a, s) : launch_scan_t<T, false, false>(a, s);
}

template <typename T>
cudaError_t launch_join(const ScanArgs& a, cudaStream_t s) {
    const size_t smem = a.top_k > 0 ? sizeof(TopSmem) : 0;
    auto* k = ce_join_kernel<T>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)a.N, kScanThreads, smem, s>>>(a);
    return cudaGetLastError();
}

size_t part_bytes(int64_t N, int segs) { return align_up((size_t)N * segs * sizeof(float4), 256); }

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, int dtype, bool entropy, cudaStream_t s) {
    if (dtype == CE_F32) return launch_scan_type<float>(a, entropy, s);
    if (dtype == CE_BF16) return launch_scan_type<__nv_bfloat16>(a, entropy, s);
    return launch_scan_type<__half>(a, entropy, s);
}

// What every entry over rows of logits refuses (sizes, types, strides).
ce_status check_rows(const void* logits, int dtype, int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides) {
    if (dtype < CE_F32 || dtype > CE_F16) return CE_ERR_UNSUPPORTED_DTYPE;
    if (!strides) return CE_ERR_INVALID_ARG;
    if (dim0 < 0 || dim1 < 0 || dim0 > 0x7fffffffLL || dim1 > 0x7fffffffLL || V < 1 || V > 0x7fffffffLL ||
        dim0 * dim1 > 0x7fffffffLL)
        return CE_ERR_INVALID_ARG;
    if (dim0 * dim1 > 0 && !logits) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % elem_size(dtype)) return CE_ERR_INVALID_ARG;
    if (strides[2] != 1 || strides[0] < 0 || strides[1] < 0) return CE_ERR_BAD_STRIDE;
    return CE_OK;
}

ce_status check_tokens(const int64_t* tokens, const int64_t* strides, int64_t n, int64_t rows) {
    if (n < 0 || n > kMaxListed) return CE_ERR_INVALID_ARG;
    if (n == 0) return CE_OK;
    if (!strides || (rows > 0 && !tokens) || reinterpret_cast<uintptr_t>(tokens) % 8) return CE_ERR_INVALID_ARG;
    for (int k = 0; k < 3; ++k)
        if (strides[k] < 0) return CE_ERR_BAD_STRIDE;
    return CE_OK;
}

RowTokens row_tokens(const int64_t* tokens, const int64_t* strides, int64_t n, int64_t dim0, int64_t dim1,
                     int64_t ignore_idx) {
    RowTokens t = {};
    t.n = (int)n;
    t.ignore_idx = ignore_idx;
    if (n == 0) return t;
    t.t = tokens;
    t.row = row_addr(strides[0], strides[1], dim0, dim1);
    t.step = strides[2];
    return t;
}

}  // namespace gbce

extern "C" size_t ce_logprobs_workspace_bytes(int64_t N, int64_t V, ce_dtype dtype, int top_k) {
    using namespace gbce;
    if (dtype < CE_F32 || dtype > CE_F16 || N < 0 || N > 0x7fffffffLL || V < 1 || V > 0x7fffffffLL || top_k < 0 ||
        top_k > kMaxTop)
        return 0;
    const ScanPlan pl = plan_scan(N, V, elem_size(dtype));
    if (pl.segs == 1) return kWsHeaderBytes;
    return kWsHeaderBytes + part_bytes(N, pl.segs) + align_up((size_t)N * pl.segs * top_k * 8, 256);
}

extern "C" ce_status ce_logprobs_fwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                     const int64_t strides[3], const int64_t* tokens, const int64_t token_strides[3],
                                     int64_t given, int64_t ignore_idx, float* logprobs, float* entropy, int top_k,
                                     int64_t* top_tokens, float* top_logprobs, float* stats, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    using namespace gbce;
    ce_status st = check_rows(logits, dtype, dim0, dim1, V, strides);
    if (st != CE_OK) return st;
    const int64_t N = dim0 * dim1;
    if ((st = check_tokens(tokens, token_strides, given, N)) != CE_OK) return st;
    if (top_k < 0 || top_k > kMaxTop || top_k > V) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logprobs) % 4 || reinterpret_cast<uintptr_t>(entropy) % 4 ||
        reinterpret_cast<uintptr_t>(top_tokens) % 8 || reinterpret_cast<uintptr_t>(top_logprobs) % 4 ||
        reinterpret_cast<uintptr_t>(stats) % 16 || reinterpret_cast<uintptr_t>(workspace) % 16)
        return CE_ERR_INVALID_ARG;
    if (N > 0) {
        if ((given > 0 && !logprobs) || (top_k > 0 && (!top_tokens || !top_logprobs)) || !workspace)
            return CE_ERR_INVALID_ARG;
        if (given == 0 && top_k == 0 && !entropy && !stats) return CE_ERR_INVALID_ARG;
        if (workspace_bytes < ce_logprobs_workspace_bytes(N, V, dtype, top_k)) return CE_ERR_WORKSPACE_TOO_SMALL;
    }
    if (N == 0) return CE_OK;
    const ScanPlan pl = plan_scan(N, V, elem_size(dtype));
    char* ws = static_cast<char*>(workspace);
    ScanArgs a = {};
    a.x = static_cast<const char*>(logits);
    a.row = row_addr(strides[0], strides[1], dim0, dim1);
    a.N = N;
    a.V = V;
    a.L = kLog2e;
    a.scale = 1.f;
    a.segs = pl.segs;
    a.per = pl.per;
    a.tokens = row_tokens(tokens, token_strides, given, dim0, dim1, ignore_idx);
    a.top_k = top_k;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.top_tokens = top_tokens;
    a.top_logprobs = top_logprobs;
    a.stats = reinterpret_cast<float4*>(stats);
    a.err = reinterpret_cast<uint32_t*>(ws + kWsErrOffset);
    if (pl.segs > 1) {
        a.part = reinterpret_cast<float4*>(ws + kWsHeaderBytes);
        a.cand = reinterpret_cast<uint64_t*>(ws + kWsHeaderBytes + part_bytes(N, pl.segs));
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(a.err, 0, 4, s);
    if (e == cudaSuccess) e = launch_scan(a, dtype, entropy || stats, s);
    if (e == cudaSuccess && a.part) {
        if (dtype == CE_F32) e = launch_join<float>(a, s);
        else if (dtype == CE_BF16) e = launch_join<__nv_bfloat16>(a, s);
        else e = launch_join<__half>(a, s);
    }
    return e == cudaSuccess ? CE_OK : launch_failed();
}
