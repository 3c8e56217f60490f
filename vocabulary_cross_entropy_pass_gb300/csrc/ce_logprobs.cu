// ce_logprobs.cu -- log-probabilities of given tokens, the entropy and the largest
// logits of each row, and their C entry points.
//
//   lp_j = x_j - logsumexp(x),   H = -sum_j exp(lp_j) lp_j,
//   top: the K largest x in falling order (ties: the lower column first), with lp
//
// Bound by HBM: every logit is read once.  ce_scan_kernel is a persistent grid, two CTAs
// per SM; a warp of each keeps a ring of 16 KB tiles filled with bulk copies, segment
// after segment and row after row, and eight warps take them out, sum the statistics and
// select candidates (ce_rowscan.cuh), so the copies go on while a row is finished.  A
// row in one piece is finished by the CTA that read it, a row in segments by
// ce_join_kernel from their partial results.
#include <math.h>

#include "ce_rowscan.h"

namespace gbce {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Whether row r is left out.  All scanning threads; a barrier where a row has several tokens.
__device__ __forceinline__ bool row_skipped(const RowTokens& t, int64_t r) {
    if (t.n == 0) return false;
    if (t.n == 1) return t.at(r, 0) == t.ignore_idx;
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

// Shared memory: the ring, its barriers, the candidates.
constexpr int kTileBytes = kScanTileVecs * 16;
constexpr int scan_stages(bool top) { return top ? 4 : 6; }  // two CTAs of 228 KB
constexpr size_t scan_smem(bool top) {
    return (size_t)scan_stages(top) * kTileBytes + (top ? sizeof(TopSmem) : 0);
}

struct Segment {
    const char* x;     // the row
    Span16 sp;
    int64_t v0, v1;    // its vectors of the body
    bool first, last;
};
template <int ES>
__device__ __forceinline__ Segment segment(const ScanArgs& p, int64_t r, int seg) {
    Segment g;
    g.x = p.x + p.row.at(r) * ES;
    g.sp = span16<ES>(g.x, 0, p.V);
    g.first = seg == 0;
    g.last = seg == p.segs - 1;
    g.v0 = min(g.sp.nv, seg * p.per);
    g.v1 = g.last ? g.sp.nv : min(g.sp.nv, g.v0 + p.per);
    return g;
}

template <typename T, bool TOP, bool ENT>
__global__ void __launch_bounds__(kScanThreads + 32, 2) ce_scan_kernel(const __grid_constant__ ScanArgs p) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems, ES = sizeof(T), STAGES = scan_stages(TOP);
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ RingBars bars;
    __shared__ float4 red[kScanThreads / 32];
    unsigned char* ring = sm;
    TopSmem& top = *reinterpret_cast<TopSmem*>(sm + (size_t)STAGES * kTileBytes);
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) ring_init(bars, STAGES);
    __syncthreads();
    const int64_t items = p.N * p.segs;
    auto row_of = [&](int64_t item) { return p.segs == 1 ? item : item / p.segs; };

    if (tid >= kScanThreads) {  // the copying warp
        const uint64_t policy = l2_evict_first_policy();
        RingAt at;
        uint32_t issued = 0;
        const bool lists = p.tokens.n > 1;
        int64_t y = p.tokens.n == 1 && blockIdx.x < items ? p.tokens.at(row_of(blockIdx.x), 0) : 0;
        for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
            const int64_t r = row_of(item), next = item + gridDim.x;
            bool skip = p.tokens.n == 1 && y == p.tokens.ignore_idx;
            if (p.tokens.n == 1 && next < items) y = p.tokens.at(row_of(next), 0);
            if (lists) {
                bool keep = false;
                for (int k = lane; k < p.tokens.n; k += 32) keep |= p.tokens.at(r, k) != p.tokens.ignore_idx;
                skip = !__any_sync(kFull, keep);
            }
            if (skip) continue;
            bool ok = true;
            if (lane == 0) {
                const Segment g = segment<ES>(p, r, (int)(item - r * p.segs));
                const char* body = g.x + g.sp.h1 * ES;
                for (int64_t f = g.v0; ok && f < g.v1; f += kScanTileVecs)
                    ok = ring_put(bars, at, issued, STAGES, ring, kTileBytes, body + f * 16,
                                  (uint32_t)min((int64_t)kScanTileVecs, g.v1 - f) * 16u, policy);
                if (!ok) ring_drain(bars, issued, STAGES);
            }
            if (!__shfl_sync(kFull, ok, 0)) break;
        }
        return;
    }

    RingAt at;
    int64_t y = p.tokens.n == 1 && blockIdx.x < items ? p.tokens.at(row_of(blockIdx.x), 0) : 0;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t r = row_of(item), next = item + gridDim.x;
        bool skip = p.tokens.n == 1 && y == p.tokens.ignore_idx;
        if (p.tokens.n == 1 && next < items) y = p.tokens.at(row_of(next), 0);
        if (p.tokens.n > 1) skip = row_skipped(p.tokens, r);
        if (skip) {
            if (!p.part) write_skipped(p, r);
            continue;
        }
        const Segment g = segment<ES>(p, r, (int)(item - r * p.segs));
        // the elements before the body go with the first segment, those after it with the last
        const bool head = g.first && tid < g.sp.h1;
        const bool tail = g.last && g.sp.t0 + tid < p.V;
        const float xh = head ? VT::load1(g.x + tid * ES) : -INFINITY;
        const float xt = tail ? VT::load1(g.x + (g.sp.t0 + tid) * ES) : -INFINITY;
        Stat st = stat_identity();
        TopState ts = {};
        typename VT::Max gm[kScanVecs];
        int has = 0;
        if constexpr (TOP) {
            ts = top_start(top, p.top_k);
#pragma unroll
            for (int i = 0; i < kScanVecs; ++i) gm[i] = VT::max_init();
            if (head) has = 1;
        }
        const int ntiles = (int)((g.v1 - g.v0 + kScanTileVecs - 1) / kScanTileVecs);
        for (int t = 0; t < ntiles || t == 0; ++t) {
            const int64_t f = g.v0 + (int64_t)t * kScanTileVecs;
            const int n = (int)min((int64_t)kScanTileVecs, g.v1 - f);
            const T* tile = reinterpret_cast<const T*>(ring + (size_t)at.s * kTileBytes);
            uint4 raw[kScanVecs];
            bool have[kScanVecs];
            if (ntiles > 0) ring_wait(bars, at);
#pragma unroll
            for (int i = 0; i < kScanVecs; ++i) {
                have[i] = tid + i * kScanThreads < n;
                if (have[i]) raw[i] = reinterpret_cast<const uint4*>(tile)[tid + i * kScanThreads];
            }
            float mx = stat_tile<T, kScanVecs, ENT, TOP>(st, raw, have, p.L, gm);
            if constexpr (TOP) {
                const bool edge = t == 0 && head;
                bool raised = false;
                if (edge) mx = fmaxf(mx, xh);
                if (t == 0) {
#pragma unroll
                    for (int i = 0; i < kScanVecs; ++i) has |= have[i] ? 1 << i : 0;
                }
                if ((t & (t + 1)) == 0) raised = top_raise<T, kScanVecs>(top, ts, gm, has, edge ? xh : -INFINITY);
                top_tile<T>(top, ts, have[0] || edge, mx, tile, n, (uint32_t)(g.sp.h1 + f * VEC), edge, xh, tid);
                if (t == 0) ts.recount(top);
                else if (raised) ts.strict = true;
            }
            if (ntiles > 0) ring_release(bars, at, STAGES);
        }
        if (head) stat_add(st, xh, p.L);
        if (tail) stat_add(st, xt, p.L);
        int c = 0;
        if constexpr (TOP) {
            const bool more = tail && ts.takes(xt);
            if (scan_count(more) > 0) {
                if (ts.bound + VEC > kTopCap) ts.compact(top);
                if (more && ts.takes(xt)) top_push_one(top, xt, (uint32_t)(g.sp.t0 + tid));
            }
            ts.recount(top);
            if (ts.bound > 2 * p.top_k + 32) {
                top_raise<T, kScanVecs>(top, ts, gm, has, -INFINITY);
                top_prune(top, ts);
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
    if (tid == 0 && bars.gone) atomicOr(p.err, CE_DEVERR_TIMEOUT);
}

// A row's segments put together.
template <typename T>
__global__ void __launch_bounds__(kScanThreads) ce_join_kernel(const __grid_constant__ ScanArgs p) {
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float4 red[kScanThreads / 32];
    TopSmem& top = *reinterpret_cast<TopSmem*>(sm);
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    if (row_skipped(p.tokens, r)) {
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
    constexpr size_t smem = scan_smem(TOP);
    auto* k = ce_scan_kernel<T, TOP, ENT>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    int64_t grid = a.N * a.segs;
    if (grid > kScanSlots) grid = kScanSlots;
    k<<<(unsigned)grid, kScanThreads + 32, smem, s>>>(a);
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

cudaError_t launch_scan(const ScanArgs& a, int dtype, bool entropy, cudaStream_t s) {
    if (dtype == CE_F32) return launch_scan_type<float>(a, entropy, s);
    if (dtype == CE_BF16) return launch_scan_type<__nv_bfloat16>(a, entropy, s);
    return launch_scan_type<__half>(a, entropy, s);
}

size_t part_bytes(int64_t N, int segs) { return align_up((size_t)N * segs * sizeof(float4), 256); }

}  // namespace

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
