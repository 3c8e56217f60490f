// ce_distill.cu -- the divergence of a row's softmax from a teacher that is known by
// its top logits, and its C entry points.
//
// With s = 1 / temperature, z_k the teacher's logit of its token t_k:
//   q_k = exp(s z_k) / sum exp(s z)   (normalize; else exp(s z_k), the rest left out)
//   p_j = exp(s x_j) / sum exp(s x)
//   loss = temperature^2 sum_k q_k (log q_k - log p_{t_k})
//   grad_j = dloss temperature (Q p_j - sum_k q_k [t_k = j]),   Q = sum_k q_k
//
// Bound by HBM: a logit read, a gradient written.  ce_distill_kernel streams whole rows
// (ce_rowscan.cuh): the statistics in a first pass, the gradient in a second, whose tiles
// come from L2, which the first was asked to keep them in, as far as the rows that are begun
// fit: a row per SM (1 GB of logits in all: rows of 256 KB 1.02 times from HBM, of 512 KB 1.24,
// of 1 MB 1.84; 1024 x 256000 float32 447 us, 0.70 of the copy rate).  Each side warp takes every
// third row: its list while the rows before are streamed (the teacher's softmax, the
// student's logits of its tokens, a hash table that finds tokens listed twice), then
// its loss and, once its gradient is stored, its listed columns again.
// Measured, bf16: 4096 x 128000, 64 tokens, loss and gradient 311 us (6.4 TB/s), 0.96 of the
// copy rate; the loss alone of 2048 x 100277, 256 tokens, 77 us (5.4 TB/s).  Lists of 256
// tokens and more are bound by the side warps (4096 x 32000: 64 tokens 96 us, 256 169, 1024 343 of
// distinct tokens and 552 of tokens drawn with replacement, whose repeats are summed).
#include <math.h>

#include <type_traits>

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
    uint32_t* claim;         // rows handed out beyond each CTA's first three
    int stages, slots;
};

constexpr int kPlaces = 6;  // of the queue: a row in the stream, two ahead, three behind

// An entry of a row's list, in shared memory.
struct ListEntry {
    float q, lq;  // the teacher's probability and its log
    float x;      // the student's logit
    int col;      // -1: left out; below: token -2 - col, listed before (counts for the loss alone)
};
// What the main warps need of a row's list for its gradient.
struct ListRow {
    float Q;          // the summed probability
    float em, ed;     // statistics of the student's logits around the body
    int bad;          // a token out of range
};
inline int list_slots(int K) {
    int n = 64;
    while (n < 2 * K) n *= 2;
    return n;
}
inline size_t list_bytes(int K, bool grad) {  // of the three side warps
    return kSideWarps * ((size_t)K * sizeof(ListEntry) + (grad ? (size_t)list_slots(K) * 2 : 0));
}

template <typename T, int NV, bool GRAD>
__global__ void __launch_bounds__(kRowThreads, GRAD && NV == 8 ? 1 : 2) ce_distill_kernel(const __grid_constant__ DistillArgs p) {
    using VT = Vec<T>;
    constexpr int ES = sizeof(T), PP = VT::kElems / 2;
    constexpr int TILE = kMainThreads * NV;  // vectors
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ RowBars bars;
    __shared__ ListRow lists[kPlaces];
    __shared__ double dred[kSideWarps];
    __shared__ int last;
    unsigned char* ring = sm;
    const int lane = threadIdx.x & 31, K = p.tokens.n;
    if (threadIdx.x == 0) row_bars_init(bars);
    __syncthreads();

    // The row count and the error word come from the kernel before this one, which may
    // still run: a thread waits for it where it first needs them.
    bool counted = false;
    float g_mean = 1.f;
    auto need_count = [&]() {
        if (counted) return;
        griddep_wait();
        if (p.n_dev) g_mean = (p.dloss ? __ldg(p.dloss) : 1.f) / (float)(*p.n_dev);
        counted = true;
    };
    auto row_scale = [&](int64_t r) {
        need_count();
        return (p.n_dev ? g_mean : (p.dloss ? __ldg(p.dloss + r) : 1.f)) * p.tau;
    };

    if (threadIdx.x < kMainThreads) {
        const int tid = threadIdx.x;
        Turn at, q;
        for (;; q.next(kPlaces)) {
            if (!warp_wait(bars, &bars.ready[q.s], q.ph)) return;
            const RowItem& it = bars.item[q.s];
            const int64_t r = it.row, nv = it.nv;
            if (r < 0) return;
            uint4* to = GRAD ? reinterpret_cast<uint4*>(it.out + it.h1 * ES) + tid : nullptr;
            if (it.skip) {
                warp_arrive(&bars.done[q.s]);
                if (GRAD) {
                    for (int64_t v = tid; v < nv; v += kMainThreads, to += kMainThreads)
                        stg128_stream(to, make_uint4(0, 0, 0, 0));
                    warp_arrive(&bars.stored[q.s]);
                }
                warp_arrive(&bars.free_[q.s]);
                continue;
            }
            if (!main_stats<T, NV, false, false>(bars, at, p.stages, ring, q.s, nv, p.L, nullptr)) return;
            if constexpr (GRAD) {
                if (!warp_wait(bars, &bars.done[q.s], q.ph) || !warp_wait(bars, &bars.prep[q.s], q.ph)) return;
                const ListRow& l = lists[q.s];
                Stat st = stat_identity();
                if (lane < kMainThreads / 32) st = Stat{bars.part[q.s][lane].x, bars.part[q.s][lane].y, 0.f};
                else if (lane == kMainThreads / 32) st = Stat{l.em, l.ed, 0.f};
                st = stat_warp<false>(st, p.L);
                const bool zero = l.bad || stat_none(st.m, st.d);
                const float a = row_scale(r) * l.Q;
                // p = 2^(x L + R) in one fused step for outputs in 16 bits (rounding R costs 2^-24 of it in the
                // exponent, 3e-6 of p at most); else from the difference
                const float logd2 = stat_logd(st, p.L) * kLog2e, M = stat_ref(st.m, p.L);
                const bool fused = ES == 2 && fabsf(M) < 64.f;
                const float R = fused ? -(M + logd2) : 0.f;
                const float2 NM = make_float2(-st.m, -st.m), LL = make_float2(p.L, p.L);
                const float2 SH = fused ? make_float2(R, R) : make_float2(-logd2, -logd2), A = make_float2(a, a);
                auto vector = [&](uint4 raw, auto one) {
                    float2 v[PP];
                    VT::unpack2(raw, v);
#pragma unroll
                    for (int k = 0; k < PP; ++k) {
                        const float2 e = __ffma2_rn(decltype(one)::value ? v[k] : __fadd2_rn(v[k], NM), LL, SH);
                        v[k] = __fmul2_rn(make_float2(ex2_approx(e.x), ex2_approx(e.y)), A);
                    }
                    return VT::pack2(v);
                };
                for (int64_t f = 0; f < nv; f += TILE, to += TILE) {
                    const uint4* tile = reinterpret_cast<const uint4*>(ring + (size_t)at.s * TILE * 16) + tid;
                    if (!warp_wait(bars, &bars.full[at.s], at.ph)) return;
                    const int64_t n = nv - f - tid;  // vectors from this thread's first on
                    if (fused && !zero && nv - f >= TILE) {
                        uint4 raw[NV];
#pragma unroll
                        for (int i = 0; i < NV; ++i) raw[i] = tile[i * kMainThreads];
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            stg128_stream(to + i * kMainThreads, vector(raw[i], std::true_type()));
                    } else {
#pragma unroll
                        for (int i = 0; i < NV; ++i) {
                            if (i * kMainThreads >= n) break;
                            const uint4 raw = tile[i * kMainThreads];
                            uint4 o = fused ? vector(raw, std::true_type()) : vector(raw, std::false_type());
                            if (zero) o = make_uint4(0, 0, 0, 0);
                            stg128_stream(to + i * kMainThreads, o);
                        }
                    }
                    warp_arrive(&bars.empty[at.s]);
                    at.next(p.stages);
                }
                warp_arrive(&bars.stored[q.s]);
            }
            warp_arrive(&bars.free_[q.s]);
        }
    }

    if (threadIdx.x < kMainThreads + 32) {  // the copying warp
        if (lane == 0) {
            // the first pass asks L2 to keep the row for the second
            const uint64_t keep = GRAD ? l2_evict_last_policy() : l2_evict_first_policy();
            const uint64_t drop = l2_evict_first_policy();
            Turn at, q;
            uint32_t issued = 0;
            bool ok = true, started = false;
            // rows: the CTA's first three, then the next that no CTA has claimed; each is in the queue two
            // ahead of its copies, so the side warps work on its list meanwhile
            auto token = [&](int64_t r) { return r < p.N ? p.tokens.at(r, 0) : 0; };
            auto publish = [&](int64_t r, int64_t y) {
                ok = ok && row_wait(bars, &bars.free_[q.s], q.ph ^ 1u);
                if (!ok) return;
                RowItem& it = bars.item[q.s];
                it.row = r < p.N ? r : -1;
                if (r < p.N) {
                    const char* x = p.x + p.row.at(r) * ES;
                    const Span16 sp = span16<ES>(x, 0, p.V);
                    it.x = x;
                    it.out = GRAD ? p.out + p.orow.at(r) * ES : nullptr;
                    it.v0 = 0;
                    it.nv = sp.nv;
                    it.h1 = it.head = (int)sp.h1;
                    it.tail = (int)sp.t0;
                    it.tails = (int)(p.V - sp.t0);
                    it.skip = y == p.tokens.ignore_idx;
                }
                mbar_arrive(&bars.ready[q.s]);
                q.next(kPlaces);
            };
            int64_t r = blockIdx.x, r1 = r + gridDim.x, r2 = r1 + gridDim.x, r3 = 0;
            int64_t y = token(r), y1 = token(r1), y2 = token(r2), y3 = 0;
            auto claim = [&]() {
                r3 = p.N;
                if (r2 >= p.N) return;
                if (!started) griddep_wait();  // the kernel before zeroes the counter
                started = true;
                r3 = 3 * (int64_t)gridDim.x + atomicAdd(p.claim, 1u);
                y3 = token(r3);
            };
            publish(r, y);
            publish(r1, y1);
            while (ok && r < p.N) {
                publish(r2, y2);
                const bool skip = y == p.tokens.ignore_idx;
                const char* x = p.x + p.row.at(r) * ES;
                const Span16 sp = span16<ES>(x, 0, p.V);
                const char* body = x + sp.h1 * ES;
                auto pass = [&](uint64_t policy) {
                    for (int64_t f = 0; ok && f < sp.nv; f += TILE)
                        ok = ring_put(bars, at, issued, p.stages, ring, TILE * 16, body + f * 16,
                                      (uint32_t)min((int64_t)TILE, sp.nv - f) * 16u, policy);
                };
                const bool early = started;
                if (early) claim();
                if (!skip) pass(keep);
                if (!early) claim();
                if (!skip && GRAD) pass(drop);
                r = r1;
                y = y1;
                r1 = r2;
                y1 = y2;
                r2 = r3;
                y2 = y3;
            }
            publish(p.N, 0);  // an end mark for each side warp
            if (!ok) ring_drain(bars, issued, p.stages);
        }
        return;
    }

    // a side warp takes every kSideWarps-th row
    const int tid = threadIdx.x - kMainThreads - 32, side = tid >> 5;
    ListEntry* e = reinterpret_cast<ListEntry*>(sm + (size_t)p.stages * TILE * 16) + side * K;
    uint16_t* slots = reinterpret_cast<uint16_t*>(sm + (size_t)p.stages * TILE * 16 +
                                                  (size_t)kSideWarps * K * sizeof(ListEntry)) + side * p.slots;
    for (uint32_t turn = side;; turn += kSideWarps) {
        const int q = (int)(turn % kPlaces);
        const uint32_t ph = (turn / kPlaces) & 1u;
        if (!warp_wait(bars, &bars.ready[q], ph)) break;
        const RowItem& it = bars.item[q];
        const int64_t r = it.row;
        if (r < 0) break;
        const int64_t ce = edge_column(it);
        if (it.skip) {
            if (lane == 0) {
                p.loss[r] = 0.f;
                if (p.stats) p.stats[r] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
            }
            if (GRAD && ce >= 0) VT::store1(it.out + ce * ES, 0.f);
            warp_arrive(&bars.prep[q]);
            warp_arrive(&bars.free_[q]);
            continue;
        }
        const float xe = ce >= 0 ? VT::load1(it.x + ce * ES) : -INFINITY;
        bool bad = false;
        float zm = -INFINITY;
#pragma unroll 4
        for (int k = lane; k < K; k += 32) {
            const int64_t y = p.tokens.at(r, k);
            const float z = teacher_at(p.teacher, p.teacher_dtype, p.trow.at(r) + k * p.tstep);
            const bool there = y != p.tokens.ignore_idx, in = there && y >= 0 && y < p.V;
            bad |= there && !in;
            // without a gradient the row's logits are not replaced: they are fetched once it lies in L2
            e[k] = ListEntry{0.f, in ? z : -INFINITY, GRAD && in ? VT::load1(it.x + y * ES) : 0.f, in ? (int)y : -1};
            zm = fmaxf(zm, in ? z : -INFINITY);
        }
        bad = __any_sync(kFull, bad);
        zm = warp_max_redux(zm);
        float sum = 0.f;
#pragma unroll 1
        for (int k = lane; k < K; k += 32)
            if (e[k].lq != -INFINITY) sum += ex2_approx((e[k].lq - zm) * p.L);
        sum = warp_allsum(sum);
        const bool nothing = zm == -INFINITY && sum == 0.f;  // no token has any probability
        const float logs = nothing ? 0.f : logf(sum);
        const float Q = nothing       ? 0.f
                        : sum != sum  ? sum
                        : p.normalize ? 1.f
                                      : ex2_approx((zm * p.scale + logs) * kLog2e);
#pragma unroll 1
        for (int k = lane; k < K; k += 32) {
            if (e[k].lq == -INFINITY) continue;
            const float lq = p.normalize ? (e[k].lq - zm) * p.scale - logs : e[k].lq * p.scale;
            e[k].lq = lq;
            e[k].q = ex2_approx(lq * kLog2e);
        }
        bool again = false;
        if constexpr (GRAD) {
            // of a token's entries one, the first to find a slot, writes for all
#pragma unroll 1
            for (int k = lane; k < p.slots; k += 32) slots[k] = kSlotFree;
            __syncwarp();
#pragma unroll 1
            for (int k = lane; k < K; k += 32) {
                const int col = e[k].col;
                if (col < 0) continue;
                if (list_enter(slots, (uint32_t)p.slots, k, col, [&](int j) { return e[j].col; }, slot_cas)) {
                    again = true;
                    e[k].col = -2 - col;
                }
            }
            again = __any_sync(kFull, again);
            Stat es = stat_identity();
            if (ce >= 0) stat_add(es, xe, p.L);
            es = stat_warp<false>(es, p.L);
            if (lane == 0) lists[q] = ListRow{Q, es.m, es.d, bad};
        }
        warp_arrive(&bars.prep[q]);

        if (!warp_wait(bars, &bars.done[q], ph)) break;
        const Stat st = row_stats<false>(bars.part[q], ce >= 0, xe, p.L);
        const bool none = stat_none(st.m, st.d);
        const float logd = none ? 0.f : stat_logd(st, p.L);
        float loss = 0.f;
#pragma unroll 8
        for (int k = lane; k < K; k += 32) {
            if (e[k].q == 0.f) continue;
            const float x = GRAD ? e[k].x : VT::load1(it.x + (int64_t)e[k].col * ES);
            const float lp = none ? -INFINITY : (x - st.m) * p.scale - logd;
            loss += e[k].q * (e[k].lq - lp);
        }
        loss = warp_allsum(loss);
        need_count();
        if (lane == 0) {
            if (bad) atomicOr(p.err, CE_DEVERR_TARGET_RANGE);
            p.loss[r] = bad ? NAN : p.tau * p.tau * loss;
            if (p.stats) p.stats[r] = make_float4(st.m, logd, zm, logs);
        }
        if constexpr (GRAD) {
            const float gt = row_scale(r), a = gt * Q, shift = -logd * kLog2e, nm = -st.m;
            const bool zero = bad || none;
            auto grad = [&](float v) { return ex2_approx(fmaf(v + nm, p.L, shift)) * a; };
            if (ce >= 0) VT::store1(it.out + ce * ES, zero ? 0.f : grad(xe));
            if (again && !zero) {
                // the sum of a token's entries, in an order of their own, at the one that writes
#pragma unroll 1
                for (int h = lane; h < p.slots; h += 32) {
                    const unsigned mine = slots[h];
#pragma unroll 1
                    for (unsigned m = __ballot_sync(kFull, slot_twice(mine)); m; m &= m - 1u) {
                        const int k = slot_entry(__shfl_sync(kFull, mine, __ffs(m) - 1)), col = e[k].col;
                        float c = 0.f;
#pragma unroll 1
                        for (int j = lane; j < K; j += 32)
                            if (e[j].col == col || e[j].col == -2 - col) c += e[j].q;
                        c = warp_allsum(c);
                        __syncwarp();
                        if (lane == 0) e[k].q = c;
                        __syncwarp();
                    }
                }
            }
            if (!warp_wait(bars, &bars.stored[q], ph)) break;
            __syncwarp();  // a listed column may be one of the elements around the body, that another lane has stored
#pragma unroll 1
            for (int k = lane; k < K && !zero; k += 32) {
                const int col = e[k].col;
                if (col < 0) continue;
                VT::store1(it.out + (int64_t)col * ES, fmaf(-gt, e[k].q, grad(e[k].x)));
            }
        }
        warp_arrive(&bars.free_[q]);
    }
    need_count();
    if (lane == 0 && bars.gone) atomicOr(p.err, CE_DEVERR_TIMEOUT);
    // the mean: the last CTA to finish sums the rows' losses in a fixed order
    if (p.mean_out) {
        __threadfence();
        side_sync();
        if (tid == 0) {
            __threadfence();
            last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        }
        side_sync();
        if (!last) return;
        __threadfence();
        double acc = strided_sum_fixed(p.loss, p.N, tid, kSideThreads);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(kFull, acc, off);
        if (lane == 0) dred[tid >> 5] = acc;
        side_sync();
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < kSideWarps; ++w) t += dred[w];
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

// The header of the workspace, and (count) how many rows count: those whose first token is not
// ignore_idx.  One CTA; the kernel after it starts meanwhile.  (With the loss's count kernel,
// a cluster that sums class weights as well, a loss of 16 rows of 32000 takes 18.6 us
// in place of 16.)
constexpr int kCountThreads = 1024;
__global__ void __launch_bounds__(kCountThreads)
ce_distill_count_kernel(const int64_t* t, RowAddr row, int64_t N, int64_t ignore_idx, bool count, uint32_t* err,
                        uint32_t* ticket, uint32_t* claim, int64_t* n_ws, int64_t* n_out) {
    griddep_launch_dependents();
    __shared__ int total;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    int own = 0;
    if (count) {
        constexpr int B = 8;  // loads on their way
        for (int64_t r0 = threadIdx.x; r0 < N; r0 += kCountThreads * B) {
            int64_t y[B];
#pragma unroll
            for (int u = 0; u < B; ++u) {
                const int64_t r = r0 + u * kCountThreads;
                y[u] = r < N ? __ldg(t + row.at(r)) : ignore_idx;
            }
#pragma unroll
            for (int u = 0; u < B; ++u) own += y[u] != ignore_idx;
        }
    }
    own = (int)__reduce_add_sync(kFull, (unsigned)own);
    if ((threadIdx.x & 31) == 0 && own) atomicAdd(&total, own);
    __syncthreads();
    if (threadIdx.x == 0) {
        *err = 0u;
        *ticket = 0u;
        *claim = 0u;
        *n_ws = total;
        if (n_out) *n_out = total;
    }
}

template <typename T, int NV, bool GRAD>
cudaError_t launch_distill_k(DistillArgs a, cudaStream_t s) {
    auto* k = ce_distill_kernel<T, NV, GRAD>;
    a.slots = GRAD ? list_slots(a.tokens.n) : 0;
    const size_t list = list_bytes(a.tokens.n, GRAD);
    constexpr bool one = GRAD && NV == 8;  // CTA per SM
    constexpr size_t tile = kMainThreads * NV * 16, room = (one ? 222 : 111) * 1024;
    // (Without a gradient the lists leave three slots up to 320 tokens, two up to 1002 and then one; they bound
    // the kernel by then: 2048 x 100277 bf16 with 320 tokens 97 us, 1002 177, 1003 170, 1024 157.)
    a.stages = (int)((room - list) / tile);
    if (a.stages > kRingMost) a.stages = kRingMost;
    const size_t smem = a.stages * tile + list;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    int64_t grid = one ? kSMs : kScanSlots;
    if (grid > a.N) grid = a.N;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    set_pdl_attr(&attr[0]);
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs& a, cudaStream_t s) {
    if (!a.out) return launch_distill_k<T, 8, false>(a, s);
    // rows over 128 KB: one CTA per SM with tiles of 32 KB, so fewer rows wait in L2 for
    // their second pass (4096 rows of 128000 bf16 columns 326 us, with two CTAs per SM 378; of
    // 70000 193 and 197, of 60000 169 both ways; 8192 of 32000 262 and 175)
    return a.V * (int64_t)sizeof(T) > 128 * 1024 ? launch_distill_k<T, 8, true>(a, s) : launch_distill_k<T, 4, true>(a, s);
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
    Problem pb = {};
    pb.N = N;
    pb.err = reinterpret_cast<uint32_t*>(ws + kWsErrOffset);
    pb.n_dev = reinterpret_cast<int64_t*>(ws + kWsCountOffset);
    pb.ticket = reinterpret_cast<uint32_t*>(ws + kWsTicketOffset);
    pb.row_claim = reinterpret_cast<uint32_t*>(ws + kWsRowClaimOffset);
    pb.loss_rows = reduce ? reinterpret_cast<float*>(ws + l.loss) : loss_out;
    const RowTokens tokens = row_tokens(t.tokens, t.token_strides, t.n, dim0, dim1, t.ignore_idx);
    const bool count = reduce || n_out;
    ce_distill_count_kernel<<<1, count ? kCountThreads : 32, 0, s>>>(tokens.t, tokens.row, N, t.ignore_idx, count, pb.err,
                                                                    pb.ticket, pb.row_claim, pb.n_dev, n_out);
    cudaError_t e = cudaGetLastError();
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
    d.tokens = tokens;
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
    d.claim = pb.row_claim;
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
