// ce_logprobs.cu -- log-probabilities of given tokens, the entropy and the largest
// logits of each row, and their C entry points.
//
//   lp_j = x_j - logsumexp(x),   H = -sum_j exp(lp_j) lp_j,
//   top: the K largest x in falling order (ties: the lower column first), with lp
//
// Bound by HBM: every logit is read once (with top_k a few hundred vectors of a row
// again, from L2); rows are claimed from a counter, since the CTAs are not equally fast (equal
// shares of 16384 x 32000 with the entropy and one alternative: 173 to 265 us).  ce_scan_kernel streams rows, or
// segments of few rows (ce_rowscan.cuh); a row in one piece is finished by its side warps, a row
// in segments by ce_join_kernel from their partial results.
// Measured on bf16 rows of 128000 columns, 4096 of them: the given token alone 154 us (6.8
// TB/s, the copy rate), with the entropy 155, with 20 likeliest 161, with 64 175 (5.9 TB/s),
// with 256 what the side warps' selection takes; 4096 x 50257 70, 74 and (20) 90 us;
// 256 x 128000 with the entropy and 20 likeliest, a row to a CTA, 31 us; 4 x 32000 with 5 likeliest, in
// segments, 12 us, two kernels' latency.  float32, 20 and 64 likeliest: 4096 x 128000, every row in two
// segments for its maxima's room, 330 and 361 us (5.8 TB/s), 4096 x 50257, in one piece, 143 and 170.
// Given tokens from the 33rd on are loaded 32 at a time, each load waited for: 32 of 4096 x 128000 bf16
// 164 us, 64 170, 256 201, 1024 378; 1024 of 4 x 32000 64 us.
#include <math.h>

#include "ce_rowscan.h"

namespace gbce {
namespace {

// A row's outputs by the lanes of one warp.
__device__ __forceinline__ void write_skipped(const ScanArgs& p, int64_t r) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        if (p.entropy) p.entropy[r] = 0.f;
        if (p.stats) p.stats[r] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int k = lane; k < p.tokens.n; k += 32) p.logprobs[r * p.tokens.n + k] = 0.f;
#pragma unroll 1
    for (int k = lane; k < p.top_k; k += 32) {
        p.top_tokens[r * p.top_k + k] = p.tokens.ignore_idx;
        p.top_logprobs[r * p.top_k + k] = 0.f;
    }
}

// A lane's given token of a row and its logit (the first 32 of them).
template <typename T>
struct Given {
    int64_t y = 0;
    float x = 0.f;
    __device__ __forceinline__ void load(const ScanArgs& p, int64_t r, const char* row, int k) {
        if (k >= p.tokens.n) return;
        y = p.tokens.at(r, k);
        if (y >= 0 && y < p.V) x = Vec<T>::load1(row + y * sizeof(T));
    }
};

// What is subtracted of a logit to give its log-probability; log d is +inf where nothing is
// allowed: every log-probability is -inf then.
struct RowNorm {
    float m, logd;
};

// A row's outputs from its statistics, but for its likeliest tokens.
template <typename T>
__device__ __forceinline__ RowNorm finish_row(const ScanArgs& p, int64_t r, const char* x, const Stat& t,
                                              Given<T> given) {
    const int lane = threadIdx.x & 31;
    const bool none = stat_none(t.m, t.d);
    const float logd = none ? 0.f : stat_logd(t, p.L);
    if (lane == 0) {
        const float h = none ? 0.f : stat_entropy(t);
        if (p.entropy) p.entropy[r] = h;
        if (p.stats) p.stats[r] = make_float4(t.m, logd, h, 0.f);
    }
#pragma unroll 1
    for (int k = lane; k < p.tokens.n; k += 32) {
        if (k >= 32) given.load(p, r, x, k);
        float lp = 0.f;
        if (given.y != p.tokens.ignore_idx) {
            if (given.y < 0 || given.y >= p.V) {
                lp = NAN;
                atomicOr(p.err, CE_DEVERR_TARGET_RANGE);
            } else {
                lp = none ? -INFINITY : (given.x - t.m) - logd;
            }
        }
        p.logprobs[r * p.tokens.n + k] = lp;
    }
    return none ? RowNorm{0.f, INFINITY} : RowNorm{t.m, logd};
}

// The likeliest tokens from the candidates in falling order (c of them).
__device__ __forceinline__ void finish_top(const ScanArgs& p, int64_t r, RowNorm n, const uint64_t* top, int c) {
#pragma unroll 1
    for (int k = threadIdx.x & 31; k < p.top_k; k += 32) {
        int64_t token = -1;  // NaN is no alternative: a row of fewer than K others ends so
        float lp = NAN;
        if (k < c) {
            token = key_column(top[k]);
            lp = (key_value(top[k]) - n.m) - n.logd;
        }
        p.top_tokens[r * p.top_k + k] = token;
        p.top_logprobs[r * p.top_k + k] = lp;
    }
}

// Shared memory: the ring, and with top_k each side warp's candidates and the groups'
// maxima of each place of the queue.
constexpr int kTileBytes = kTileVecs * 16;
constexpr int scan_stages(bool top) { return top ? 2 : 3; }
constexpr size_t scan_smem(bool top) {
    return (size_t)scan_stages(top) * kTileBytes + (top ? kSideWarps * sizeof(TopSmem) + kHeadsRoom * 2 : 0);
}

template <typename T, bool TOP, bool ENT>
__global__ void __launch_bounds__(kRowThreads, 2) ce_scan_kernel(const __grid_constant__ ScanArgs p) {
    using VT = Vec<T>;
    constexpr int ES = sizeof(T), STAGES = scan_stages(TOP);
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ RowBars bars;
    unsigned char* ring = sm;
    uint16_t* heads = reinterpret_cast<uint16_t*>(sm + (size_t)STAGES * kTileBytes);  // [p.places][p.heads]
    TopSmem* tops = reinterpret_cast<TopSmem*>(heads + kHeadsRoom);  // [kSideWarps]
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        row_bars_init(bars);
        if (p.part && blockIdx.x == 0) *p.err = 0u;
    }
    __syncthreads();
    griddep_launch_dependents();  // the kernel that puts segments together waits for this one's end itself

    if (threadIdx.x < kMainThreads) {
        Turn at, q;
        for (;; q.next(p.places)) {
            if (!warp_wait(bars, &bars.ready[q.s], q.ph)) return;
            const int64_t row = bars.item[q.s].row, nv = bars.item[q.s].nv;
            const int skip = bars.item[q.s].skip;
            if (row < 0) return;
            if (skip)
                warp_arrive(&bars.done[q.s]);
            else if (!main_stats<T, 8, ENT, TOP>(bars, at, STAGES, ring, q.s, nv, p.L, heads + q.s * p.heads))
                return;
            warp_arrive(&bars.free_[q.s]);
        }
    }

    if (threadIdx.x < kMainThreads + 32) {  // the copying warp
        const uint64_t policy = l2_evict_first_policy();
        Turn at, q;
        uint32_t issued = 0;
        bool ok = true;
        const int64_t items = p.N * p.segs;
        auto row_of = [&](int64_t item) { return p.segs == 1 ? item : item / p.segs; };
        const bool one = p.tokens.n == 1;
        auto token = [&](int64_t item) -> int64_t {
            return one && item < items ? p.tokens.at(row_of(item), 0) : 0;
        };
        const bool late = p.V * ES > STAGES * kTileBytes;
        int64_t item = blockIdx.x, next = item + gridDim.x;
        int64_t y = token(item), y1 = token(next);  // loaded an item ahead
        int ends = kSideWarps;  // an end mark for each side warp
        for (; ok && ends > 0; q.next(p.places)) {
            const bool more = item < items;
            if (!more) --ends;
            const int64_t r = more ? row_of(item) : -1;
            int64_t after = next + gridDim.x;
            const bool claims = p.claim && next < items && lane == 0;
            if (claims && !late) after = 2 * (int64_t)gridDim.x + atomicAdd(p.claim, 1u);
            bool skip = one && y == p.tokens.ignore_idx;
            if (more && p.tokens.n > 1) {  // left out when all are ignored
                bool keep = false;
#pragma unroll 1
                for (int k = lane; k < p.tokens.n; k += 32) keep |= p.tokens.at(r, k) != p.tokens.ignore_idx;
                skip = !__any_sync(kFull, keep);
            }
            if (lane == 0) {
                ok = row_wait(bars, &bars.free_[q.s], q.ph ^ 1u);
                if (ok) {
                    RowItem& it = bars.item[q.s];
                    it.row = r;
                    int64_t v0 = 0, v1 = 0;
                    const char* body = nullptr;
                    if (more) {
                        const int seg = (int)(item - r * p.segs);
                        const char* x = p.x + p.row.at(r) * ES;
                        const Span16 sp = span16<ES>(x, 0, p.V);
                        const bool last = seg == p.segs - 1;
                        v0 = min(sp.nv, seg * p.per);
                        v1 = last ? sp.nv : min(sp.nv, v0 + p.per);
                        body = x + sp.h1 * ES;
                        it.x = x;
                        it.item = item;
                        it.v0 = v0;
                        it.nv = v1 - v0;
                        // the elements before the body go with the first segment, those after it with the last
                        it.head = seg == 0 ? (int)sp.h1 : 0;
                        it.h1 = (int)sp.h1;
                        it.tail = (int)sp.t0;
                        it.tails = last ? (int)(p.V - sp.t0) : 0;
                        it.skip = skip;
                    }
                    mbar_arrive(&bars.ready[q.s]);
                    if (!skip)
                        for (int64_t v = v0; ok && v < v1; v += kTileVecs)
                            ok = ring_put(bars, at, issued, STAGES, ring, kTileBytes, body + v * 16,
                                          (uint32_t)min((int64_t)kTileVecs, v1 - v) * 16u, policy);
                }
                if (!ok) ring_drain(bars, issued, STAGES);
            }
            ok = __shfl_sync(kFull, (int)ok, 0);
            if (claims && late) after = 2 * (int64_t)gridDim.x + atomicAdd(p.claim, 1u);
            after = __shfl_sync(kFull, after, 0);
            item = next;
            next = after;
            y = y1;
            y1 = token(next);
        }
        return;
    }

    // a side warp takes every kSideWarps-th item
    const int side = (threadIdx.x - kMainThreads - 32) >> 5;
    TopSmem& top = tops[side];
    Turn q;
    for (int k = 0; k < side; ++k) q.next(p.places);
    for (;;) {
        if (!warp_wait(bars, &bars.ready[q.s], q.ph)) break;
        const RowItem& it = bars.item[q.s];
        const int64_t r = it.row;
        if (r < 0) break;
        if (it.skip) {
            if (!p.part) write_skipped(p, r);
        } else {
            Given<T> given;
            if (!p.part) given.load(p, r, it.x, lane);
            const int64_t ce = edge_column(it);
            const float xe = ce >= 0 ? VT::load1(it.x + ce * ES) : -INFINITY;
            if (!warp_wait(bars, &bars.done[q.s], q.ph)) break;
            const Stat st = row_stats<ENT>(bars.part[q.s], ce >= 0, xe, p.L);
            RowNorm norm = {};
            if (!p.part)
                norm = finish_row<T>(p, r, it.x, st, given);
            else if (lane == 0)
                p.part[it.item] = make_float4(st.m, st.d, st.s, 0.f);
            if constexpr (TOP) {
                const int groups = (int)((it.nv + kTileVecs - 1) / kTileVecs) * kMainThreads;
                const int64_t col0 = it.h1 + it.v0 * VT::kElems;
                const int c = top_select<T>(top, heads + q.s * p.heads, groups,
                                  reinterpret_cast<const uint4*>(it.x + col0 * ES), it.nv, (uint32_t)col0, p.top_k,
                                  ce >= 0, xe, (uint32_t)ce);
                if (!p.part) {
                    finish_top(p, it.row, norm, top.buf, c);
                } else {
                    if (lane == 0) p.part[it.item].w = __int_as_float(c);
#pragma unroll 1
                    for (int k = lane; k < c; k += 32) p.cand[it.item * p.top_k + k] = top.buf[k];
                }
            }
        }
        warp_arrive(&bars.free_[q.s]);
        for (int k = 0; k < kSideWarps; ++k) q.next(p.places);
    }
    if (lane == 0 && bars.gone) atomicOr(p.err, CE_DEVERR_TIMEOUT);
}

// A row's segments put together by a warp.
constexpr int kJoinWarps = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) ce_join_kernel(const __grid_constant__ ScanArgs p) {
    extern __shared__ __align__(128) unsigned char sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    TopSmem& top = reinterpret_cast<TopSmem*>(sm)[warp];
    const int64_t r = (int64_t)blockIdx.x * kJoinWarps + warp;
    griddep_wait();
    if (r >= p.N) return;
    const char* x = p.x + p.row.at(r) * sizeof(T);
    Given<T> given;
    given.load(p, r, x, lane);
    bool keep = p.tokens.n == 0;
#pragma unroll 1
    for (int k = lane; k < p.tokens.n; k += 32)
        keep |= (k == lane ? given.y : p.tokens.at(r, k)) != p.tokens.ignore_idx;
    if (!__any_sync(kFull, keep)) {
        write_skipped(p, r);
        return;
    }
    Stat st = stat_identity();
    const float4* part = p.part + r * p.segs;
    const uint64_t* cand = p.cand + r * p.segs * p.top_k;
    TopGate g(p.top_k, -INFINITY);
    // Many: what reaches the least of the segments' j-th largest is enough, j of every segment
    // being K at least (a segment with fewer gives no bound).  1 x 128000, 256 likeliest: 254 us
    // without, 85 with; 64: 62 and 34; 8, 256 candidates: 12.4 and 13.8, so not for those.
    uint64_t bound = 0;
    if (p.segs * p.top_k > 256) {
        const int j = (p.top_k + p.segs - 1) / p.segs;
        bound = ~(uint64_t)0;
#pragma unroll 1
        for (int k0 = lane; k0 < p.segs; k0 += 32) {
            const uint64_t key = cand[(int64_t)k0 * p.top_k + j - 1];
            bound = min(bound, __float_as_int(part[k0].w) >= j ? key : (uint64_t)0);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(kFull, bound, o);
            bound = min(bound, other);
        }
    }
    for (int k0 = 0; k0 < p.segs; k0 += 32) {
        const float4 v = k0 + lane < p.segs ? part[k0 + lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        st = stat_combine(st, Stat{v.x, v.y, v.z}, p.L);
        // the candidates of 32 segments, top_k places each
        const int have = __float_as_int(v.w), most = min(32, p.segs - k0) * p.top_k;
#pragma unroll 4
        for (int u0 = 0; u0 < most; u0 += 32) {
            const int u = u0 + lane, seg = u / max(p.top_k, 1);
            const int here = __shfl_sync(kFull, have, seg & 31);
            const bool held = u < most && u - seg * p.top_k < here;
            const uint64_t key = held ? cand[(int64_t)k0 * p.top_k + u] : 0;
            const bool ok = held && key >= bound;
            top_room(top, g, 32);
            const unsigned m = __ballot_sync(kFull, ok);
            if (ok) top.buf[g.held + __popc(m & ((1u << lane) - 1u))] = key;
            g.held += __popc(m);
        }
    }
    st = stat_warp<true>(st, p.L);
    top_sort(top, g.held);
    if (g.held > p.top_k) g.held = p.top_k;
    const RowNorm norm = finish_row<T>(p, r, x, st, given);
    finish_top(p, r, norm, top.buf, g.held);
}

template <typename T, bool TOP, bool ENT>
cudaError_t launch_scan_t(const ScanArgs& a, cudaStream_t s) {
    constexpr size_t smem = scan_smem(TOP);
    auto* k = ce_scan_kernel<T, TOP, ENT>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    int64_t grid = a.N * a.segs;
    if (grid > kScanSlots) grid = kScanSlots;
    k<<<(unsigned)grid, kRowThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scan_type(const ScanArgs& a, bool entropy, cudaStream_t s) {
    if (a.top_k > 0) return entropy ? launch_scan_t<T, true, true>(a, s) : launch_scan_t<T, true, false>(a, s);
    return entropy ? launch_scan_t<T, false, true>(a, s) : launch_scan_t<T, false, false>(a, s);
}

template <typename T>
cudaError_t launch_join(const ScanArgs& a, cudaStream_t s) {
    const size_t smem = kJoinWarps * sizeof(TopSmem);
    auto* k = ce_join_kernel<T>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    set_pdl_attr(&attr[0]);
    cfg.gridDim = dim3((unsigned)((a.N + kJoinWarps - 1) / kJoinWarps));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
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
    const ScanPlan pl = plan_scan(N, V, elem_size(dtype), top_k);
    if (pl.segs <= 1) return pl.segs ? kWsHeaderBytes : 0;
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
    const ScanPlan pl = plan_scan(N, V, elem_size(dtype), top_k);
    if (pl.segs == 0) return CE_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    ScanArgs a = {};
    a.x = static_cast<const char*>(logits);
    a.row = row_addr(strides[0], strides[1], dim0, dim1);
    a.N = N;
    a.V = V;
    a.L = kLog2e;
    a.segs = pl.segs;
    a.per = pl.per;
    a.places = pl.places;
    a.heads = pl.heads;
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
    // rows in segments: the first kernel starts the error word, the second one adds to it
    a.claim = a.part ? nullptr : reinterpret_cast<uint32_t*>(ws + kWsRowClaimOffset);
    cudaError_t e = a.part ? cudaSuccess : cudaMemsetAsync(ws, 0, kWsHeaderBytes, s);
    if (e == cudaSuccess) e = launch_scan(a, dtype, entropy || stats, s);
    if (e == cudaSuccess && a.part) {
        if (dtype == CE_F32) e = launch_join<float>(a, s);
        else if (dtype == CE_BF16) e = launch_join<__nv_bfloat16>(a, s);
        else e = launch_join<__half>(a, s);
    }
    return e == cudaSuccess ? CE_OK : launch_failed();
}
