// ce_distill.cu -- the divergence of a row's softmax from a teacher that is known by
// its top logits, and its C entry points.
//
// With s = 1 / temperature, z_k the teacher's logit of its token t_k:
//   q_k = exp(s z_k) / sum exp(s z)   (normalize; else exp(s z_k), the rest left out)
//   p_j = exp(s x_j) / sum exp(s x)
//   loss = temperature^2 sum_k q_k (log q_k - log p_{t_k})
//   grad_j = dloss temperature (Q p_j - sum_k q_k [t_k = j]),   Q = sum_k q_k
//
// Bound by HBM: a logit read, a gradient written.  ce_distill_kernel is a persistent
// grid whose CTAs own whole rows.  A warp keeps a ring of tiles filled with bulk copies;
// eight warps take them out: the row's statistics (ce_rowscan.cuh) in a first pass, the
// gradient in a second, whose tiles come from L2, which the first was asked to keep
// them in.  The row's list is worked on before its tiles: the teacher's softmax, the
// student's logits of its tokens, and a hash table that finds tokens listed twice;
// their columns are written again after the second pass.
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
    float* loss;             // [N]
    float4* stats;           // [N] {m, log d, the teacher's maximum, log of its sum}, or NULL
    uint32_t* err;
    const int64_t* n_count;  // rows that count
    // the gradient, at the logits' offset from 16 bytes
    char* out;
    RowAddr orow;
    const float* dloss;
    const int64_t* n_dev;    // n_count for the mean's gradient, else NULL
    float* mean_out;         // or NULL
    uint32_t* ticket;        // CTAs done
    int stages, slots;
};

// The teacher's table: its tokens and probabilities, and the slots of a hash table.
inline int teacher_slots(int K) {
    int n = 64;
    while (n < 2 * K) n *= 2;
    return n;
}
struct TeacherSmem {
    float* q;       // [K]
    int* token;     // [K], -1: left out
    int* key;       // [slots] token or -1
    int* first;     // [slots] the lowest k of that token
    int slots;
};

template <typename T, int NV, bool GRAD, int KE>  // KE: listed tokens a thread takes
__global__ void __launch_bounds__(kScanThreads + 32, NV == 4 ? 2 : 1)
ce_distill_kernel(const __grid_constant__ DistillArgs p) {
    using VT = Vec<T>;
    constexpr int ES = sizeof(T), PP = VT::kElems / 2;
    constexpr int TILE = kScanThreads * NV;  // vectors
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ RingBars bars;
    __shared__ float4 red4[kScanThreads / 32];
    __shared__ float red[3][kScanThreads / 32];
    __shared__ int last;
    unsigned char* ring = sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.tokens.n;
    if (tid == 0) ring_init(bars, p.stages);
    __syncthreads();

    if (tid >= kScanThreads) {  // the copying warp
        if (lane == 0) {
            // the first pass asks L2 to keep the row for the second
            const uint64_t keep = GRAD ? l2_evict_last_policy() : l2_evict_first_policy();
            const uint64_t drop = l2_evict_first_policy();
            RingAt at;
            uint32_t issued = 0;
            bool ok = true;
            int64_t y = p.tokens.at(blockIdx.x, 0);
            for (int64_t r = blockIdx.x; ok && r < p.N; r += gridDim.x) {
                const bool skip = y == p.tokens.ignore_idx;
                if (r + gridDim.x < p.N) y = p.tokens.at(r + gridDim.x, 0);
                if (skip) continue;
                const char* x = p.x + p.row.at(r) * ES;
                const Span16 sp = span16<ES>(x, 0, p.V);
                for (int pass = 0; ok && pass < (GRAD ? 2 : 1); ++pass)
                    for (int64_t f = 0; ok && f < sp.nv; f += TILE)
                        ok = ring_put(bars, at, issued, p.stages, ring, TILE * 16, x + sp.h1 * ES + f * 16,
                                      (uint32_t)min((int64_t)TILE, sp.nv - f) * 16u, pass == 0 ? keep : drop);
            }
            if (!ok) ring_drain(bars, issued, p.stages);
        }
        return;
    }

    TeacherSmem ts;
    ts.slots = p.slots;
    ts.q = reinterpret_cast<float*>(sm + (size_t)p.stages * TILE * 16);
    ts.token = reinterpret_cast<int*>(ts.q + K);
    ts.key = ts.token + K;
    ts.first = ts.key + p.slots;
    RingAt at;
    // the row count and the error word come from the kernel before this one, which
    // may still run: they are waited for where the first row needs them
    bool counted = false;
    float g_mean = 1.f;
    auto need_count = [&]() {
        if (counted) return;
        griddep_wait();
        if (p.n_dev) g_mean = (p.dloss ? __ldg(p.dloss) : 1.f) / (float)(*p.n_dev);
        counted = true;
    };
    // a row's first token and list are loaded one row ahead
    int64_t y0 = p.tokens.at(blockIdx.x, 0), y[KE];
    float z[KE];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < KE; ++i) {
            const int k = tid + i * kScanThreads;
            y[i] = k < K ? p.tokens.at(r, k) : p.tokens.ignore_idx;
            z[i] = k < K ? teacher_at(p.teacher, p.teacher_dtype, p.trow.at(r) + k * p.tstep) : -INFINITY;
        }
    };
    fetch(blockIdx.x);
    for (int64_t r = blockIdx.x; r < p.N; r += gridDim.x) {
        const char* x = p.x + p.row.at(r) * ES;
        char* out = GRAD ? p.out + p.orow.at(r) * ES : nullptr;
        const Span16 sp = span16<ES>(x, 0, p.V);
        const int64_t edge = span16_edge(sp, 0, p.V, tid);
        const int64_t next = r + gridDim.x;
        const bool skip = y0 == p.tokens.ignore_idx;
        if (next < p.N) y0 = p.tokens.at(next, 0);
        if (skip) {
            if (GRAD) {
                uint4* to = reinterpret_cast<uint4*>(out + sp.h1 * ES);
                for (int64_t v = tid; v < sp.nv; v += kScanThreads) stg128_stream(to + v, make_uint4(0, 0, 0, 0));
                if (edge >= 0) VT::store1(out + edge * ES, 0.f);
            }
            if (tid == 0) {
                p.loss[r] = 0.f;
                if (p.stats) p.stats[r] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
            }
            if (next < p.N) fetch(next);
            continue;
        }
        // the list: the student's logits, the teacher's softmax
        float xv[KE], q[KE], lq[KE];
        int col[KE];
        bool bad = false;
        float zm = -INFINITY;
        const float xe = edge >= 0 ? VT::load1(x + edge * ES) : -INFINITY;
#pragma unroll
        for (int i = 0; i < KE; ++i) {
            const bool there = y[i] != p.tokens.ignore_idx;
            const bool in = there && y[i] >= 0 && y[i] < p.V;
            bad |= there && !in;
            col[i] = in ? (int)y[i] : -1;
            xv[i] = in ? VT::load1(x + y[i] * ES) : 0.f;
            lq[i] = in ? z[i] : -INFINITY;
            zm = fmaxf(zm, lq[i]);
        }
        if (next < p.N) fetch(next);
        zm = scan_max(zm, red[0]);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < KE; ++i)
            if (lq[i] != -INFINITY) sum += ex2_approx((lq[i] - zm) * p.L);
        sum = scan_sum(sum, red[1]);
        const bool nothing = zm == -INFINITY && sum == 0.f;  // no token has any probability
        const float logs = nothing ? 0.f : logf(sum);
        const float Q = nothing       ? 0.f
                        : sum != sum  ? sum
                        : p.normalize ? 1.f
                                      : ex2_approx((zm * p.scale + logs) * kLog2e);
#pragma unroll
        for (int i = 0; i < KE; ++i) {
            const int k = tid + i * kScanThreads;
            q[i] = 0.f;
            if (lq[i] != -INFINITY) {
                lq[i] = p.normalize ? (lq[i] - zm) * p.scale - logs : lq[i] * p.scale;
                q[i] = ex2_approx(lq[i] * kLog2e);
            }
            if (GRAD && k < K) {
                ts.q[k] = q[i];
                ts.token[k] = col[i];
            }
        }
        // tokens listed twice: the first entry of each speaks for all
        if (GRAD) {
            for (int k = tid; k < ts.slots; k += kScanThreads) {
                ts.key[k] = -1;
                ts.first[k] = 0x7fffffff;
            }
            scan_sync();
            int slot[KE];
#pragma unroll
            for (int i = 0; i < KE; ++i) {
                slot[i] = -1;
                if (col[i] < 0) continue;
                uint32_t h = ((uint32_t)col[i] * 2654435761u) >> 7;
                for (;; ++h) {
                    h &= (uint32_t)ts.slots - 1u;
                    const int was = atomicCAS(&ts.key[h], -1, col[i]);
                    if (was == -1 || was == col[i]) break;
                }
                slot[i] = (int)h;
                atomicMin(&ts.first[h], tid + i * kScanThreads);
            }
            scan_sync();
            bool again = false;
#pragma unroll
            for (int i = 0; i < KE; ++i)
                if (slot[i] >= 0 && ts.first[slot[i]] != tid + i * kScanThreads) {
                    again = true;
                    slot[i] = -1;
                    col[i] = -2 - col[i];  // counts for the loss alone
                }
            if (scan_count(again) > 0) {
#pragma unroll
                for (int i = 0; i < KE; ++i) {
                    if (slot[i] < 0) continue;
                    float c = 0.f;
                    for (int k = 0; k < K; ++k)
                        if (ts.token[k] == col[i]) c += ts.q[k];
                    ts.q[tid + i * kScanThreads] = c;  // read by no other: its token is this thread's
                }
            }
        }

        // first pass: the row's statistics
        Stat st = stat_identity();
        typename VT::Max gm[NV];
        for (int64_t f = 0; f < sp.nv; f += TILE) {
            const int n = (int)min((int64_t)TILE, sp.nv - f);
            const uint4* tile = reinterpret_cast<const uint4*>(ring + (size_t)at.s * TILE * 16);
            ring_wait(bars, at);
            uint4 raw[NV];
            bool have[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                have[i] = tid + i * kScanThreads < n;
                if (have[i]) raw[i] = tile[tid + i * kScanThreads];
            }
            stat_tile<T, NV, false, false>(st, raw, have, p.L, gm);
            ring_release(bars, at, p.stages);
        }
        if (edge >= 0) stat_add(st, xe, p.L);
        st = stat_block(st, p.L, red4);
        const bool none = stat_none(st.m, st.d);
        const float logd = none ? 0.f : logf(st.d);
        float loss = 0.f;
#pragma unroll
        for (int i = 0; i < KE; ++i) {
            const float lp = none ? -INFINITY : (xv[i] - st.m) * p.scale - logd;
            loss += q[i] == 0.f ? 0.f : q[i] * (lq[i] - lp);
        }
        loss = scan_sum(loss, red[2]);
        const bool wrong = scan_count(bad) > 0;
        need_count();
        if (tid == 0) {
            if (wrong) atomicOr(p.err, CE_DEVERR_TARGET_RANGE);
            p.loss[r] = wrong ? NAN : p.tau * p.tau * loss;
            if (p.stats) p.stats[r] = make_float4(st.m, logd, zm, logs);
        }
        if constexpr (GRAD) {
            // second pass: p_j dloss temperature Q, and at the listed columns that less q
            const float gt = (p.n_dev ? g_mean : (p.dloss ? __ldg(p.dloss + r) : 1.f)) * p.tau;
            const bool zero = wrong || none;
            const float a = gt * Q, shift = -logd * kLog2e, nm = -st.m;
            const float2 NM = make_float2(nm, nm), LL = make_float2(p.L, p.L), SH = make_float2(shift, shift);
            const float2 A = make_float2(a, a);
            for (int64_t f = 0; f < sp.nv; f += TILE) {
                const int n = (int)min((int64_t)TILE, sp.nv - f);
                const uint4* tile = reinterpret_cast<const uint4*>(ring + (size_t)at.s * TILE * 16);
                uint4* to = reinterpret_cast<uint4*>(out + sp.h1 * ES) + f;
                ring_wait(bars, at);
                uint4 raw[NV];
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * kScanThreads < n) raw[i] = tile[tid + i * kScanThreads];
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (tid + i * kScanThreads >= n) continue;
                    float2 v[PP];
                    VT::unpack2(raw[i], v);
#pragma unroll
                    for (int k = 0; k < PP; ++k) {
                        const float2 e = __ffma2_rn(__fadd2_rn(v[k], NM), LL, SH);
                        v[k] = __fmul2_rn(make_float2(ex2_approx(e.x), ex2_approx(e.y)), A);
                    }
                    stg128_stream(to + tid + i * kScanThreads, zero ? make_uint4(0, 0, 0, 0) : VT::pack2(v));
                }
                ring_release(bars, at, p.stages);
            }
            auto grad = [&](float v) { return ex2_approx(fmaf(v + nm, p.L, shift)) * a; };
            if (edge >= 0) VT::store1(out + edge * ES, zero ? 0.f : grad(xe));
            scan_sync();
            if (!zero) {
#pragma unroll
                for (int i = 0; i < KE; ++i)
                    if (col[i] >= 0)
                        VT::store1(out + (int64_t)col[i] * ES,
                                   fmaf(-gt, ts.q[tid + i * kScanThreads], grad(xv[i])));
            }
            scan_sync();
        }
    }
    need_count();
    if (tid == 0 && bars.gone) atomicOr(p.err, CE_DEVERR_TIMEOUT);
    // the mean: the last CTA to finish sums the rows' losses in a fixed order
    if (p.mean_out) {
        __threadfence();
        scan_sync();
        if (tid == 0) {
            __threadfence();
            last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        }
        scan_sync();
        if (!last) return;
        __threadfence();
        __shared__ double dred[kScanThreads / 32];
        double acc = strided_sum_fixed(p.loss, p.N, tid, kScanThreads);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(kFull, acc, off);
        if (lane == 0) dred[warp] = acc;
        scan_sync();
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < kScanThreads / 32; ++w) t += dred[w];
            p.mean_out[0] = (float)(t / (double)(*p.n_count));  // NaN when every row is ignored
        }
    }
}

// Workspace: the header, the rows' losses, their statistics (a gradient at another
// offset from 16 bytes than the logits is written by ce_softgrad_kernel from them).
struct Layout {
    size_t loss, stats, bytes;
};
Layout layout(int64_t N) {
    Layout l;
    l.loss = kWsHeaderBytes;
    l.stats = l.loss + align_up((size_t)N * 4, 256);
    l.bytes = l.stats + align_up((size_t)N * 16, 256);
    return l;
}

template <typename T, int NV, bool GRAD, int KE>
cudaError_t launch_distill_k(DistillArgs a, cudaStream_t s) {
    auto* k = ce_distill_kernel<T, NV, GRAD, KE>;
    a.slots = GRAD ? teacher_slots(a.tokens.n) : 0;
    const size_t list = GRAD ? (size_t)a.tokens.n * 8 + (size_t)a.slots * 8 : 0;
    // six tiles; five where a long list would cost an SM its second CTA
    a.stages = NV == 4 && list > 8 * 1024 ? 5 : 6;
    const size_t smem = (size_t)a.stages * kScanThreads * NV * 16 + list;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    int64_t grid = NV == 4 ? kScanSlots : kScanSlots / 2;
    if (grid > a.N) grid = a.N;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    set_pdl_attr(&attr[0]);
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kScanThreads + 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs& a, cudaStream_t s) {
    const bool brief = a.tokens.n <= kScanThreads;
    if (!a.out) return brief ? launch_distill_k<T, 4, false, 1>(a, s) : launch_distill_k<T, 4, false, 4>(a, s);
    // rows over 128 KB: one CTA per SM with tiles of 32 KB, so fewer rows wait in L2 for
    // their second pass
    if (a.V * (int64_t)sizeof(T) > 128 * 1024)
        return brief ? launch_distill_k<T, 8, true, 1>(a, s) : launch_distill_k<T, 8, true, 4>(a, s);
    return brief ? launch_distill_k<T, 4, true, 1>(a, s) : launch_distill_k<T, 4, true, 4>(a, s);
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
    const Layout l = layout(N);
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
    if (N == 0) return !reduce || launch_reduce_mean(pb, loss_out, s) == cudaSuccess ? CE_OK : launch_failed();
    DistillArgs d = {};
    d.x = static_cast<const char*>(logits);
    d.row = row_addr(strides[0], strides[1], dim0, dim1);
    d.N = N;
    d.V = V;
    d.scale = 1.f / t.tau;
    d.L = kLog2e / t.tau;
    d.tau = t.tau;
    d.tokens = row_tokens(t.tokens, t.token_strides, t.n, dim0, dim1, t.ignore_idx);
    d.teacher = t.logits;
    d.teacher_dtype = t.dtype;
    d.trow = row_addr(t.strides[0], t.strides[1], dim0, dim1);
    d.tstep = t.strides[2];
    d.normalize = t.normalize;
    d.loss = pb.loss_rows;
    d.stats = reinterpret_cast<float4*>(stats_out);
    d.err = pb.err;
    d.n_count = pb.n_dev;
    d.mean_out = reduce ? loss_out : nullptr;
    d.ticket = pb.ticket;
    bool after = false;  // the gradient from the statistics, in a launch of its own
    if (grad) {
        const int64_t es = elem_size(dtype);
        after = (reinterpret_cast<uintptr_t>(grad) - reinterpret_cast<uintptr_t>(logits)) % 16 ||
                (dim0 > 1 && (grad_strides[0] - strides[0]) * es % 16) ||
                (dim1 > 1 && (grad_strides[1] - strides[1]) * es % 16);
        if (after) {
            d.stats = reinterpret_cast<float4*>(ws + l.stats);
        } else {
            d.out = static_cast<char*>(grad);
            d.orow = row_addr(grad_strides[0], grad_strides[1], dim0, dim1);
            d.dloss = dloss;
            d.n_dev = reduce ? pb.n_dev : nullptr;
        }
    }
    if (dtype == CE_F32) e = launch_distill_t<float>(d, s);
    else if (dtype == CE_BF16) e = launch_distill_t<__nv_bfloat16>(d, s);
    else e = launch_distill_t<__half>(d, s);
    if (e == cudaSuccess && after)
        e = launch_softgrad(grad_args(logits, dim0, dim1, V, strides, t, d.stats, dloss, reduce ? pb.n_dev : nullptr,
                                      grad, grad_strides),
                            dtype, s);
    return e == cudaSuccess ? CE_OK : launch_failed();
}

}  // namespace
}  // namespace gbce

extern "C" size_t ce_distill_workspace_bytes(int64_t N, int64_t V, ce_dtype dtype) {
    using namespace gbce;
    if (dtype < CE_F32 || dtype > CE_F16 || N < 0 || N > 0x7fffffffLL || V < 1 || V > 0x7fffffffLL) return 0;
    return layout(N).bytes;
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
