// ce_api.cu -- the C ABI of libgbce: argument checks, the path planner and
// the launch sequence.  Every entry point is declared and documented in
// include/ce.h.
//
// One pass enqueues, on the caller's stream:
//   1. ce_count_kernel    -- n_non_ignore and the target range check (needed
//                            before any gradient: a kept row is scaled by
//                            dloss/n under reduce_loss);
//   2. the main kernel(s) -- the stream kernel (wide rows), the warp-per-row
//                            kernel (rows of one tile), the plain-load
//                            kernel (rows off the 16-byte grid), the
//                            row/cluster kernel, or the two stage kernels of
//                            the split path;
//   3. ce_mean_kernel     -- reduce_loss only, on the paths that do not take
//                            the mean in their last CTA: the fixed-order mean.
// Nothing is allocated and nothing waits for the device.
#include <math.h>
#include <string.h>

#include "ce_internal.h"

namespace gbce {

int elem_size(int dtype) { return dtype == CE_F32 ? 4 : 2; }

cudaError_t allow_smem(const void* kernel, size_t bytes) {
    if (bytes <= 16 * 1024) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess || bytes <= 40 * 1024) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

namespace {

constexpr int kMaxCluster = 16;
constexpr size_t kSmemLimit = 227 * 1024;

struct Plan {
    int path;  // CE_PATH_ROW / CLUSTER / TWO_STAGE / STREAM / WARP / VECROW, or < 0 on error
    FusedPlan fused;
    SplitPlan split;
    StreamPlan stream;
    RowsPlan rows;
    VecRowPlan vecrow;
};

// Warp-per-row kernel: the row must fit one tile of 16 or 32 KB; each of its
// 6 consumer warps owns stages/6 tiles, so stages is a multiple of 6.
bool plan_rows(int64_t row_bytes, int64_t N, const ce_options* o, RowsPlan* rp) {
    rp->tile_kb = (o && o->tune_tile_kb) ? o->tune_tile_kb : (row_bytes <= 16 * 1024 ? 16 : 32);
    if (row_bytes > (int64_t)rp->tile_kb * 1024) return false;
    // 16 KB tiles with many rows: two per warp (192 KB, one CTA per SM), so a
    // warp's next row lands while it works on this one (1 GB of 8192-column
    // bf16 rows: 0.373 ms against 0.390 ms); with few rows, one per warp and
    // two CTAs per SM (more warps in flight: 1024 such rows 16.1 us against
    // 17.5 us).  32 KB tiles: one per warp (192 KB).
    const int def = (rp->tile_kb == 16 && N >= 8192) ? 12 : 6;
    rp->stages = (o && o->tune_stages) ? o->tune_stages : def;
    if (rp->stages % 6 != 0) return false;
    rp->ctas_per_sm_cap = o ? o->tune_ctas_per_sm : 0;
    return rp->stages * (size_t)rp->tile_kb * 1024 + 1024 <= kSmemLimit;
}

// Row-streaming kernel: tiles of 16 or 32 KB consumed by 256 or 512 threads,
// `stages` of them in flight.  Defaults from sweeps over V = 32000 .. 256000
// bf16 (32 KB tiles and 256 threads best at every width; the ring depth is
// chosen by the caller from the row width).
// def_tile_kb / def_stages: the shape when the options leave it open (0:
// 32 KB tiles 5 deep, 16 KB tiles 12 deep).
bool plan_stream(const ce_options* o, StreamPlan* sp, int def_tile_kb = 0, int def_stages = 0) {
    sp->threads = (o && o->tune_threads) ? o->tune_threads : 256;
    sp->tile_kb = (o && o->tune_tile_kb) ? o->tune_tile_kb : (def_tile_kb ? def_tile_kb : 32);
    sp->stages = (o && o->tune_stages) ? o->tune_stages
                                       : (def_stages ? def_stages : (sp->tile_kb == 32 ? 5 : 12));
    sp->ctas_per_sm_cap = o ? o->tune_ctas_per_sm : 0;
    sp->l2_keep = (o && o->tune_l2_keep == 2) ? 0 : 1;
    const size_t tile = (size_t)sp->tile_kb * 1024;
    if (sp->threads != 256 && sp->threads != 512) return false;
    return sp->stages * tile + 1024 <= kSmemLimit;
}

int round_up_int(int64_t x, int64_t m) { return (int)((x + m - 1) / m * m); }

bool opts_clean(const ce_options* o) {
    if (!o) return true;
    for (int i = 0; i < 2; ++i)
        if (o->reserved[i] != 0) return false;
    if (o->tune_tile_kb != 0 && o->tune_tile_kb != 16 && o->tune_tile_kb != 32) return false;
    if (o->force_path < 0 || o->force_path > CE_PATH_VECROW) return false;
    if (o->num_vocab_chunks < 0) return false;
    if (o->tune_threads != 0 && o->tune_threads != 256 && o->tune_threads != 512 &&
        o->tune_threads != 32 && o->tune_threads != 1024)
        return false;
    if (o->tune_stages < 0 || o->tune_stages > 12 || o->tune_stages == 1) return false;
    if (o->tune_ctas_per_sm < 0) return false;
    if (o->tune_l2_keep < 0 || o->tune_l2_keep > 2) return false;
    return true;
}

// Choose the fused-kernel shape; returns false when the fused kernel cannot
// take this problem (V too large for 16 CTAs, a forced K it cannot honour).
bool plan_fused(int dtype, int64_t V, const ce_options* o, bool want_cluster, FusedPlan* fp) {
    const int es = elem_size(dtype);
    const int vec = 16 / es;
    const int K = o ? o->num_vocab_chunks : 0;
    int C;
    if (K > 0) {
        C = K;
    } else {
        // prefer 256-thread CTAs (several resident per SM); 512-thread CTAs
        // only when 16 of the smaller ones cannot hold a row
        C = (int)((V + 8191) / 8192);
        if (C > kMaxCluster) C = (int)((V + 16383) / 16384);
        if (want_cluster && C < 2) C = 2;
    }
    if (C < 1 || C > kMaxCluster) return false;
    if (o && o->tune_threads && o->tune_threads != 256 && o->tune_threads != 512) return false;
    const int64_t chunk = round_up_int((V + C - 1) / C, vec);
    int threads = (o && o->tune_threads) ? o->tune_threads : (chunk <= 8192 ? 256 : 512);
    if (chunk > (int64_t)fused_capacity(dtype, threads)) {
        if (o && o->tune_threads) return false;
        threads = 512;
        if (chunk > (int64_t)fused_capacity(dtype, threads)) return false;
    }
    const size_t stage_bytes = align_up((size_t)chunk * es, 128);
    int stages = (o && o->tune_stages) ? o->tune_stages : (stage_bytes <= 40 * 1024 ? 3 : 2);
    if (stages > 4) return false;
    while (stages > 2 && stages * stage_bytes + 2048 > kSmemLimit) --stages;
    if (stages * stage_bytes + 2048 > kSmemLimit) return false;
    fp->threads = threads;
    fp->cluster = C;
    fp->chunk = (int)chunk;
    fp->stages = stages;
    fp->ctas_per_sm_cap = o ? o->tune_ctas_per_sm : 0;
    return true;
}

int split_chunks(int64_t V, const ce_options* o) {
    const int K = o ? o->num_vocab_chunks : 0;
    if (K > 0) return (int)(K < V ? K : V);
    return split_auto_chunks(V);
}

Plan make_plan(const Problem& p, const ce_options* o) {
    Plan pl;
    memset(&pl, 0, sizeof pl);
    const int force = o ? o->force_path : CE_PATH_AUTO;
    const bool aligned = fused_aligned(p) && p.V <= 0x7fffffffLL;
    if (o && o->class_weights) {
        // the class-weighted pass: the stream kernel (256-thread shapes) when
        // the rows and the weight vector are 16-byte aligned and no split is
        // asked for, the two-stage kernels otherwise
        const bool cw_aligned = reinterpret_cast<uintptr_t>(o->class_weights) % 16 == 0;
        // each gradient tile brings its weights (4/s times its bytes) into
        // the next ring slots: 16 KB tiles 6 deep unless tuned (two CTAs per
        // SM), and room for two tiles with their weights
        const int group = 1 + 4 / (int)p.es;
        if ((force == CE_PATH_AUTO || force == CE_PATH_STREAM) && aligned && cw_aligned &&
            o->num_vocab_chunks == 0 && plan_stream(o, &pl.stream, 16, 6) &&
            pl.stream.threads == 256 && pl.stream.stages >= 2 * group) {
            pl.path = CE_PATH_STREAM;
            return pl;
        }
        if (force != CE_PATH_AUTO && force != CE_PATH_TWO_STAGE) {
            pl.path = -2;
            return pl;
        }
        pl.path = CE_PATH_TWO_STAGE;
        pl.split.chunks = split_chunks(p.V, o);
        pl.split.chunk = (p.V + pl.split.chunks - 1) / pl.split.chunks;
        return pl;
    }
    const int K = o ? o->num_vocab_chunks : 0;
    const int64_t row_bytes = p.V * p.es;
    const int def_tile = row_bytes <= 128 * 1024 ? 16 : 32;
    // A vocabulary split asked for on aligned rows: the stream kernel streams
    // each chunk of ceil(V/K) columns (rounded up to 16 bytes) as its own run
    // of tiles and combines the chunks' partials in chunk order (256
    // consuming threads).  16 KB tiles, two CTAs per SM, at any width: the
    // chunk-end sums and part-filled tiles want the extra warps.  Same-GPU
    // sweep, 2.1 GB of bf16 logits, ms per launch (stream / two-stage /
    // cluster): 128000 columns K = 8 0.677 (0.813 with 32 KB tiles) / 1.040;
    // K = 16 0.745 / 1.251 / 1.932; K = 32 1.222 / 1.961; 65536 columns K = 16
    // 1.201 / 1.911 / 3.315; 32000 columns K = 4 0.820 / 1.252 / 1.448.  More
    // chunks than 32 go to the two-stage kernels.
    if (K > 0 && aligned && (force == CE_PATH_AUTO || force == CE_PATH_STREAM)) {
        const int vec = 16 / p.es;
        const int64_t C = round_up_int((p.V + K - 1) / K, vec);
        const int64_t nch = (p.V + C - 1) / C;
        // (a chunk's byte count is kept in 32 bits)
        if (nch <= kMaxStreamChunks && C * p.es <= 0xffffffffLL && plan_stream(o, &pl.stream, 16, 6) &&
            pl.stream.threads == 256) {
            pl.stream.geo = kStreamChunks;
            pl.stream.chunk_elems = C;
            pl.stream.nchunks = (int)nch;
            pl.path = CE_PATH_STREAM;
            return pl;
        }
        if (force == CE_PATH_STREAM) {
            pl.path = -2;
            return pl;
        }
    }
    // Rows off the 16-byte grid wider than 32 KB (odd widths such as 50257 or
    // 100277 in 16-bit types, shifted views): the stream kernel copies each
    // row's aligned body with TMA and takes the at most 2 (16/s - 1) elements
    // around it one per thread.  Narrower ones, and shapes the stream kernel
    // does not have (tune_threads other than 256), take the plain-load kernel
    // below.
    const bool edges_auto = force == CE_PATH_AUTO && !aligned && K == 0 && row_bytes > 32 * 1024;
    const bool edges_forced = force == CE_PATH_STREAM && !aligned && K == 0;
    if ((edges_auto || edges_forced) && p.V <= 0x7fffffffLL) {
        if (plan_stream(o, &pl.stream, def_tile, 6) && pl.stream.threads == 256) {
            pl.stream.geo = kStreamEdges;
            pl.path = CE_PATH_STREAM;
            return pl;
        }
        if (edges_forced) {
            pl.path = -2;
            return pl;
        }
        memset(&pl.stream, 0, sizeof pl.stream);
    }
    // Short rows (one 32 KB tile or less): a warp per row; wider rows: the
    // stream kernel; a requested vocabulary split: the cluster kernel.
    const bool warp_auto = force == CE_PATH_AUTO && aligned && K == 0 && row_bytes <= 32 * 1024;
    if (force == CE_PATH_WARP || warp_auto) {
        if (!aligned || !plan_rows(row_bytes, p.N, o, &pl.rows)) {
            pl.path = -2;
            return pl;
        }
        pl.path = CE_PATH_WARP;
        return pl;
    }
    // Rows off the 16-byte grid up to 32 KB (or forced): plain 16-byte loads,
    // the second pass from L2.  A requested vocabulary split still goes to
    // the two-stage kernels.
    if (force == CE_PATH_VECROW || (force == CE_PATH_AUTO && !aligned && K == 0)) {
        // Shapes by row width (tune_threads overrides): up to 32 KB a warp per
        // row; up to 320 KB 512-thread CTAs, two per SM; wider rows
        // 1024-thread CTAs, one per SM, so half as many rows wait in L2
        // between their passes.  Same-GPU sweep, ~2.1 GB of bf16 logits, ms
        // per launch: 16383 columns warp 0.842 / CTA 1.049; 100277 512-thread
        // 0.798 / 1024-thread 0.949; 151937 0.855 / 0.878; 200019 0.935 /
        // 0.907; fp32 100003 0.946 / 0.892.
        pl.path = (K == 0 && p.V <= 0x7fffffffLL) ? CE_PATH_VECROW : -2;
        const int tt = o ? o->tune_threads : 0;
        pl.vecrow.warp_rows = tt == 32 || (tt == 0 && row_bytes <= 32 * 1024);
        pl.vecrow.threads = tt > 32 ? tt : (row_bytes <= 320 * 1024 ? 512 : 1024);
        pl.vecrow.ctas_per_sm_cap = o ? o->tune_ctas_per_sm : 0;
        return pl;
    }
    const bool stream_auto = force == CE_PATH_AUTO && aligned && K == 0;
    if (force == CE_PATH_STREAM || stream_auto) {
        // Rows up to 128 KB: 16 KB tiles 6 deep, two CTAs per SM (twice the
        // warps; two CTAs' rows between their passes still fit L2).  Wider
        // rows: 32 KB tiles 6 deep, one CTA per SM, so fewer rows wait in L2
        // for their second pass.  Same-GPU sweep, ~2.1 GB of bf16 logits per
        // width, ms per launch (16 KB x 6 / 32 KB x 6): 32 KB rows 0.795 /
        // 1.203, 62 KB 0.604 / 0.743, 98 KB 0.605 / 0.728, 128 KB 0.608 /
        // 0.617, 160 KB 0.618 / 0.598, 250 KB 0.679 / 0.601, 500 KB 0.836 /
        // 0.681.
        // The same shape with or without a gradient, so a forward-only pass
        // gives the fused pass's losses bit for bit (one CTA's partial sums
        // group the same way); two CTAs per SM would speed a forward-only pass
        // of wider rows too (split step at 128000 columns: 1.822 ms against
        // 1.846 ms), not worth losing that.
        if (!aligned || !plan_stream(o, &pl.stream, def_tile, 6)) {
            pl.path = -2;
            return pl;
        }
        pl.path = CE_PATH_STREAM;
        return pl;
    }
    if (force == CE_PATH_TWO_STAGE || (force == CE_PATH_AUTO && !aligned)) {
        pl.path = CE_PATH_TWO_STAGE;
    } else if (!aligned) {
        pl.path = -2;  // row / cluster forced on rows that are not 16-byte aligned
        return pl;
    } else if (plan_fused(p.dtype, p.V, o, force == CE_PATH_CLUSTER, &pl.fused)) {
        pl.path = pl.fused.cluster == 1 ? CE_PATH_ROW : CE_PATH_CLUSTER;
        if (force == CE_PATH_ROW && pl.path != CE_PATH_ROW) pl.path = -2;
        if (force == CE_PATH_CLUSTER && pl.path != CE_PATH_CLUSTER) pl.path = -2;
        return pl;
    } else if (force == CE_PATH_AUTO) {
        pl.path = CE_PATH_TWO_STAGE;
    } else {
        pl.path = -2;
        return pl;
    }
    pl.split.chunks = split_chunks(p.V, o);
    pl.split.chunk = (p.V + pl.split.chunks - 1) / pl.split.chunks;
    return pl;
}

size_t workspace_need(int64_t N, int64_t V, const ce_options* o) {
    const size_t rows = align_up((size_t)N * sizeof(float), 256);
    const size_t parts = align_up((size_t)N * (size_t)split_chunks(V, o) * sizeof(float4), 256);
    return kWsHeaderBytes + rows + parts;
}

ce_status check_common(const void* logits, int dtype, int layout, int64_t dim0, int64_t dim1,
                       int64_t V, const int64_t* strides, const int64_t* targets,
                       const int64_t* tstrides, float a, int reduce, float* loss_out, void* ws,
                       size_t ws_bytes, const ce_options* o) {
    if (dtype < CE_F32 || dtype > CE_F16) return CE_ERR_UNSUPPORTED_DTYPE;
    if (layout != CE_LAYOUT_BSV && layout != CE_LAYOUT_SBV) return CE_ERR_INVALID_ARG;
    if (!ws || !strides || !tstrides) return CE_ERR_INVALID_ARG;
    if (dim0 < 0 || dim1 < 0 || V < 1 || V > 0x7fffffffLL) return CE_ERR_INVALID_ARG;
    // with no rows the logits, targets and per-row losses may be empty (NULL);
    // a mean still needs its one output value
    const bool empty = dim0 * dim1 == 0;
    if (!empty && (!logits || !targets || !loss_out)) return CE_ERR_INVALID_ARG;
    if (empty && reduce && !loss_out) return CE_ERR_INVALID_ARG;
    if (!(a >= 0.f && a <= 1.f)) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % elem_size(dtype)) return CE_ERR_INVALID_ARG;
    if (!opts_clean(o)) return CE_ERR_INVALID_ARG;
    if (strides[2] != 1 || strides[0] < 0 || strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (tstrides[0] < 0 || tstrides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (reinterpret_cast<uintptr_t>(ws) % 16) return CE_ERR_INVALID_ARG;
    if (ws_bytes < workspace_need(dim0 * dim1, V, o)) return CE_ERR_WORKSPACE_TOO_SMALL;
    return CE_OK;
}

cudaError_t launch_planned(const Problem& pb, const Plan& pl, float4* parts, cudaStream_t s) {
    if (pl.path == CE_PATH_TWO_STAGE) return launch_split(pb, pl.split, parts, s);
    if (pl.path == CE_PATH_STREAM)
        return pl.stream.geo == kStreamAligned ? launch_stream(pb, pl.stream, s)
                                               : launch_stream_geo(pb, pl.stream, parts, s);
    if (pl.path == CE_PATH_WARP) return launch_rows(pb, pl.rows, s);
    if (pl.path == CE_PATH_VECROW) return launch_vecrow(pb, pl.vecrow, s);
    return launch_fused(pb, pl.fused, s);
}

ce_status run_pass(Problem& pb, const ce_options* o, float* loss_out, int64_t* n_out,
                   void* ws, cudaStream_t s) {
    Plan pl = make_plan(pb, o);
    if (pl.path < 0) return CE_ERR_UNSUPPORTED_PATH;
    char* w = static_cast<char*>(ws);
    pb.err = reinterpret_cast<uint32_t*>(w + kWsErrOffset);
    pb.n_dev = reinterpret_cast<int64_t*>(w + kWsCountOffset);
    pb.ticket = reinterpret_cast<uint32_t*>(w + kWsTicketOffset);
    pb.cw = o ? o->class_weights : nullptr;
    pb.wdenom = reinterpret_cast<double*>(w + kWsWeightDenomOffset);
    pb.wsum = reinterpret_cast<double*>(w + kWsWeightSumOffset);
    pb.row_claim = reinterpret_cast<uint32_t*>(w + kWsRowClaimOffset);
    pb.row_done = reinterpret_cast<uint32_t*>(w + kWsRowDoneOffset);
    // the stream and warp kernels compute the mean themselves (their last CTA)
    const bool mean_in_kernel =
        pb.reduce && (pl.path == CE_PATH_STREAM || pl.path == CE_PATH_WARP) && pb.N > 0;
    pb.mean_out = mean_in_kernel ? loss_out : nullptr;
    float* rows = reinterpret_cast<float*>(w + kWsHeaderBytes);
    float4* parts = reinterpret_cast<float4*>(
        w + kWsHeaderBytes + align_up((size_t)pb.N * sizeof(float), 256));
    pb.loss_rows = pb.reduce ? rows : loss_out;

    if (launch_count(pb, n_out, s) != cudaSuccess) return launch_failed();
    cudaEvent_t eb = o ? static_cast<cudaEvent_t>(o->event_begin) : nullptr;
    cudaEvent_t ee = o ? static_cast<cudaEvent_t>(o->event_end) : nullptr;
    if (eb && cudaEventRecord(eb, s) != cudaSuccess) return launch_failed();
    if (pb.N > 0 && launch_planned(pb, pl, parts, s) != cudaSuccess) return launch_failed();
    if (ee && cudaEventRecord(ee, s) != cudaSuccess) return launch_failed();
    if (pb.reduce && !mean_in_kernel && launch_reduce_mean(pb, loss_out, s) != cudaSuccess)
        return launch_failed();
    return CE_OK;
}

// True when distinct rows never share an element: with the two row strides
// sorted, the inner one spans at least a row of V and the outer one spans
// every inner step.  (Sufficient, not necessary; covers contiguous, padded and
// transposed layouts.)  Required of the in-place gradient pass.
bool rows_disjoint(int64_t dim0, int64_t dim1, int64_t V, int64_t s0, int64_t s1) {
    int64_t in_s = s1, in_n = dim1, out_s = s0, out_n = dim0;
    if (in_n <= 1 || (out_n > 1 && s0 < s1)) {
        in_s = s0; in_n = dim0; out_s = s1; out_n = dim1;
    }
    if (in_n > 1 && in_s < V) return false;
    if (out_n > 1 && out_s < (in_n > 1 ? in_s * in_n : V)) return false;
    return true;
}

void fill_problem(Problem& pb, const void* logits, int dtype, int64_t dim0, int64_t dim1,
                  int64_t V, const int64_t* strides, const int64_t* targets, const int64_t* tstrides,
                  float a, int64_t ignore_idx, int reduce) {
    memset(&pb, 0, sizeof pb);
    pb.logits = static_cast<char*>(const_cast<void*>(logits));
    pb.dtype = dtype;
    pb.es = elem_size(dtype);
    pb.dim0 = dim0;
    pb.dim1 = dim1;
    pb.N = dim0 * dim1;
    pb.V = V;
    pb.s0 = strides[0];
    pb.s1 = strides[1];
    pb.targets = targets;
    pb.ts0 = tstrides[0];
    pb.ts1 = tstrides[1];
    pb.a = a;
    pb.ignore_idx = ignore_idx;
    pb.reduce = reduce ? 1 : 0;
}

// The backward of ce_bwd and ce_vp_bwd: the gradient of V columns of the
// logits that start at vocabulary column vocab_offset of a V_total vocabulary.
ce_status bwd_common(const void* logits, int dtype, int64_t dim0, int64_t dim1, int64_t V,
                     int64_t vocab_offset, int64_t V_total, const int64_t* strides,
                     const int64_t* targets, const int64_t* target_strides, const float* lse,
                     float label_smoothing, int64_t ignore_idx, int reduce_loss, const float* dloss,
                     const int64_t* n_non_ignore, void* grad, const int64_t* grad_strides,
                     cudaStream_t stream) {
    if (dtype < CE_F32 || dtype > CE_F16) return CE_ERR_UNSUPPORTED_DTYPE;
    if (!strides || !target_strides || !grad_strides) return CE_ERR_INVALID_ARG;
    if (dim0 < 0 || dim1 < 0 || V < 1 || vocab_offset < 0 || V_total < vocab_offset + V ||
        V_total > 0x7fffffffLL)
        return CE_ERR_INVALID_ARG;
    if (!(label_smoothing >= 0.f && label_smoothing <= 1.f)) return CE_ERR_INVALID_ARG;
    const int64_t N = dim0 * dim1;
    if (N > 0 && (!logits || !targets || !lse || !grad)) return CE_ERR_INVALID_ARG;
    if (N > 0 && reduce_loss && !n_non_ignore) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % elem_size(dtype) ||
        reinterpret_cast<uintptr_t>(grad) % elem_size(dtype))
        return CE_ERR_INVALID_ARG;
    if (strides[2] != 1 || strides[0] < 0 || strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (grad_strides[2] != 1 || grad_strides[0] < 0 || grad_strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (target_strides[0] < 0 || target_strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (!rows_disjoint(dim0, dim1, V, grad_strides[0], grad_strides[1])) return CE_ERR_BAD_STRIDE;
    if (grad == logits && (grad_strides[0] != strides[0] || grad_strides[1] != strides[1]))
        return CE_ERR_BAD_STRIDE;
    if (N == 0) return CE_OK;
    BwdProblem bp;
    memset(&bp, 0, sizeof bp);
    const int es = elem_size(dtype);
    bp.logits = static_cast<const char*>(logits);
    bp.grad = static_cast<char*>(grad);
    bp.dtype = dtype;
    bp.dim1 = dim1;
    bp.N = N;
    bp.V = V;
    bp.s0 = strides[0];
    bp.s1 = strides[1];
    bp.gs0 = grad_strides[0];
    bp.gs1 = grad_strides[1];
    bp.targets = targets;
    bp.ts0 = target_strides[0];
    bp.ts1 = target_strides[1];
    bp.ignore_idx = ignore_idx;
    bp.lse = lse;
    bp.a = label_smoothing;
    bp.reduce = reduce_loss ? 1 : 0;
    bp.dloss = dloss;
    bp.n_dev = n_non_ignore;
    bp.vocab_offset = vocab_offset;
    bp.V_total = V_total;
    // 16-byte vectors when every gradient row sits at its logits row's offset
    // from a 16-byte boundary (always so in place)
    bp.vec_ok = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(grad)) % 16 == 0 &&
                ((strides[0] - grad_strides[0]) * es) % 16 == 0 &&
                ((strides[1] - grad_strides[1]) * es) % 16 == 0;
    if (launch_bwd(bp, stream) != cudaSuccess) return launch_failed();
    return CE_OK;
}

}  // namespace

// The main kernel(s) of one pass, planned as ce_fwd_bwd would, for a caller
// that has already run the count kernel (pb.n_dev, pb.err set) and wants the
// per-row losses in pb.loss_rows (no in-kernel mean).  `partials` holds the
// two-stage partials when that path is planned.
cudaError_t launch_main_pass(Problem& pb, const ce_options* o, float4* partials, size_t partial_bytes,
                             cudaStream_t s) {
    Plan pl = make_plan(pb, o);
    if (pl.path < 0) return cudaErrorInvalidValue;
    if (pl.path == CE_PATH_TWO_STAGE &&
        (size_t)pb.N * (size_t)pl.split.chunks * sizeof(float4) > partial_bytes)
        return cudaErrorInvalidValue;
    pb.mean_out = nullptr;
    if (pb.N == 0) return cudaSuccess;
    return launch_planned(pb, pl, partials, s);
}

size_t partial_bytes_for(int64_t N, int64_t V) {
    return align_up((size_t)N * (size_t)split_chunks(V, nullptr) * sizeof(float4), 256);
}

void problem_init(Problem& pb, const void* logits, int dtype, int64_t dim0, int64_t dim1, int64_t V,
                  const int64_t* strides, const int64_t* targets, const int64_t* tstrides, float a,
                  int64_t ignore_idx, int reduce) {
    fill_problem(pb, logits, dtype, dim0, dim1, V, strides, targets, tstrides, a, ignore_idx, reduce);
}

}  // namespace gbce

using namespace gbce;

extern "C" {

size_t ce_workspace_bytes(int64_t dim0, int64_t dim1, int64_t V, ce_dtype dtype,
                          const ce_options* opts) {
    if (dim0 < 0 || dim1 < 0 || V < 1 || (int)dtype < CE_F32 || (int)dtype > CE_F16) return 0;
    if (!opts_clean(opts)) return 0;
    return workspace_need(dim0 * dim1, V, opts);
}

ce_status ce_fwd_bwd(void* logits, ce_dtype dtype, ce_layout layout, int64_t dim0, int64_t dim1,
                     int64_t V, const int64_t strides[3], const int64_t* targets,
                     const int64_t target_strides[2], float label_smoothing, int64_t ignore_idx,
                     int reduce_loss, const float* dloss, float* loss_out, void* grad_inplace,
                     int64_t* n_non_ignore_out, void* workspace, size_t workspace_bytes,
                     const ce_options* opts, void* stream) {
    ce_status st = check_common(logits, dtype, layout, dim0, dim1, V, strides, targets,
                                target_strides, label_smoothing, reduce_loss, loss_out,
                                workspace, workspace_bytes, opts);
    if (st != CE_OK) return st;
    if (grad_inplace != logits) return CE_ERR_INVALID_ARG;
    if (!rows_disjoint(dim0, dim1, V, strides[0], strides[1])) return CE_ERR_BAD_STRIDE;
    Problem pb;
    fill_problem(pb, logits, dtype, dim0, dim1, V, strides, targets, target_strides,
                 label_smoothing, ignore_idx, reduce_loss);
    pb.dloss = dloss;
    pb.grad = true;
    return run_pass(pb, opts, loss_out, n_non_ignore_out, workspace,
                    static_cast<cudaStream_t>(stream));
}

ce_status ce_fwd_only(const void* logits, ce_dtype dtype, ce_layout layout, int64_t dim0,
                      int64_t dim1, int64_t V, const int64_t strides[3], const int64_t* targets,
                      const int64_t target_strides[2], float label_smoothing, int64_t ignore_idx,
                      int reduce_loss, float* loss_out, float* lse_out, int64_t* n_non_ignore_out,
                      void* workspace, size_t workspace_bytes, const ce_options* opts,
                      void* stream) {
    ce_status st = check_common(logits, dtype, layout, dim0, dim1, V, strides, targets,
                                target_strides, label_smoothing, reduce_loss, loss_out,
                                workspace, workspace_bytes, opts);
    if (st != CE_OK) return st;
    Problem pb;
    fill_problem(pb, logits, dtype, dim0, dim1, V, strides, targets, target_strides,
                 label_smoothing, ignore_idx, reduce_loss);
    pb.lse_out = lse_out;
    pb.grad = false;
    return run_pass(pb, opts, loss_out, n_non_ignore_out, workspace,
                    static_cast<cudaStream_t>(stream));
}

ce_status ce_bwd(const void* logits, ce_dtype dtype, ce_layout layout, int64_t dim0, int64_t dim1,
                 int64_t V, const int64_t strides[3], const int64_t* targets,
                 const int64_t target_strides[2], const float* lse, float label_smoothing,
                 int64_t ignore_idx, int reduce_loss, const float* dloss,
                 const int64_t* n_non_ignore, void* grad, const int64_t grad_strides[3],
                 void* stream) {
    if (layout != CE_LAYOUT_BSV && layout != CE_LAYOUT_SBV) return CE_ERR_INVALID_ARG;
    return bwd_common(logits, dtype, dim0, dim1, V, 0, V, strides, targets, target_strides, lse,
                      label_smoothing, ignore_idx, reduce_loss, dloss, n_non_ignore, grad,
                      grad_strides, static_cast<cudaStream_t>(stream));
}

ce_status ce_vp_partials(const void* shard_logits, ce_dtype dtype, int64_t dim0, int64_t dim1,
                         int64_t V_shard, const int64_t strides[3], const int64_t* targets,
                         const int64_t target_strides[2], int64_t vocab_offset, int64_t ignore_idx,
                         float* partials, void* stream) {
    if (dtype < CE_F32 || dtype > CE_F16) return CE_ERR_UNSUPPORTED_DTYPE;
    if (!strides || !target_strides) return CE_ERR_INVALID_ARG;
    if (dim0 < 0 || dim1 < 0 || V_shard < 1 || vocab_offset < 0) return CE_ERR_INVALID_ARG;
    const int64_t N = dim0 * dim1;
    if (N > 0 && (!shard_logits || !targets || !partials)) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(partials) % 16) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(shard_logits) % elem_size(dtype)) return CE_ERR_INVALID_ARG;
    if (strides[2] != 1 || strides[0] < 0 || strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (target_strides[0] < 0 || target_strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (N == 0) return CE_OK;
    VpPartProblem vp;
    vp.logits = static_cast<const char*>(shard_logits);
    vp.dtype = dtype;
    vp.s0 = strides[0];
    vp.s1 = strides[1];
    vp.dim1 = dim1;
    vp.N = N;
    vp.V = V_shard;
    vp.vocab_offset = vocab_offset;
    vp.targets = targets;
    vp.ts0 = target_strides[0];
    vp.ts1 = target_strides[1];
    vp.ignore_idx = ignore_idx;
    vp.part = reinterpret_cast<float4*>(partials);
    if (launch_vp_partials(vp, static_cast<cudaStream_t>(stream)) != cudaSuccess) return launch_failed();
    return CE_OK;
}

ce_status ce_vp_combine(const float* partials, int num_shards, const int64_t* shard_offsets,
                        int64_t dim0, int64_t dim1, const int64_t* targets,
                        const int64_t target_strides[2], float label_smoothing, int64_t ignore_idx,
                        int reduce_loss, float* loss_out, float* lse_out,
                        int64_t* n_non_ignore_out, void* workspace, size_t workspace_bytes,
                        void* stream) {
    if (num_shards < 1 || num_shards > kVpMaxShards || !shard_offsets || !target_strides)
        return CE_ERR_INVALID_ARG;
    if (shard_offsets[0] != 0) return CE_ERR_INVALID_ARG;
    for (int k = 0; k < num_shards; ++k)
        if (shard_offsets[k + 1] <= shard_offsets[k]) return CE_ERR_INVALID_ARG;
    const int64_t V = shard_offsets[num_shards];
    if (dim0 < 0 || dim1 < 0 || V > 0x7fffffffLL) return CE_ERR_INVALID_ARG;
    if (!(label_smoothing >= 0.f && label_smoothing <= 1.f)) return CE_ERR_INVALID_ARG;
    const int64_t N = dim0 * dim1;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return CE_ERR_INVALID_ARG;
    if (N > 0 && (!partials || !targets || !loss_out || !lse_out)) return CE_ERR_INVALID_ARG;
    if (N == 0 && reduce_loss && !loss_out) return CE_ERR_INVALID_ARG;
    if (target_strides[0] < 0 || target_strides[1] < 0) return CE_ERR_BAD_STRIDE;
    if (workspace_bytes < workspace_need(N, V, nullptr)) return CE_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    static const int64_t unit_strides[3] = {0, 0, 1};
    Problem pb;
    fill_problem(pb, nullptr, CE_F32, dim0, dim1, V, unit_strides, targets, target_strides,
                 label_smoothing, ignore_idx, reduce_loss);
    char* w = static_cast<char*>(workspace);
    pb.err = reinterpret_cast<uint32_t*>(w + kWsErrOffset);
    pb.n_dev = reinterpret_cast<int64_t*>(w + kWsCountOffset);
    pb.ticket = reinterpret_cast<uint32_t*>(w + kWsTicketOffset);
    pb.loss_rows = reduce_loss ? reinterpret_cast<float*>(w + kWsHeaderBytes) : loss_out;
    if (launch_count(pb, n_non_ignore_out, s) != cudaSuccess) return launch_failed();
    VpCombineProblem vc;
    vc.part = reinterpret_cast<const float4*>(partials);
    vc.R = num_shards;
    vc.off = shard_offsets;
    vc.dim1 = dim1;
    vc.N = N;
    vc.targets = targets;
    vc.ts0 = target_strides[0];
    vc.ts1 = target_strides[1];
    vc.ignore_idx = ignore_idx;
    vc.a = label_smoothing;
    vc.loss = pb.loss_rows;
    vc.lse = lse_out;
    if (launch_vp_combine(vc, s) != cudaSuccess) return launch_failed();
    if (reduce_loss && launch_reduce_mean(pb, loss_out, s) != cudaSuccess) return launch_failed();
    return CE_OK;
}

ce_status ce_vp_bwd(const void* shard_logits, ce_dtype dtype, int64_t dim0, int64_t dim1,
                    int64_t V_shard, const int64_t strides[3], const int64_t* targets,
                    const int64_t target_strides[2], int64_t vocab_offset, int64_t V_total,
                    const float* lse, float label_smoothing, int64_t ignore_idx, int reduce_loss,
                    const float* dloss, const int64_t* n_non_ignore, void* grad,
                    const int64_t grad_strides[3], void* stream) {
    return bwd_common(shard_logits, dtype, dim0, dim1, V_shard, vocab_offset, V_total, strides,
                      targets, target_strides, lse, label_smoothing, ignore_idx, reduce_loss, dloss,
                      n_non_ignore, grad, grad_strides, static_cast<cudaStream_t>(stream));
}

ce_status ce_get_error(const void* workspace, void* stream, uint32_t* host_err) {
    if (!workspace || !host_err) return CE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, static_cast<const char*>(workspace) + kWsErrOffset, sizeof v,
                        cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return launch_failed();
    if (cudaStreamSynchronize(s) != cudaSuccess) return launch_failed();
    *host_err = v;
    if (v & CE_DEVERR_TIMEOUT) return CE_ERR_DEVICE_TIMEOUT;
    if (v & CE_DEVERR_TARGET_RANGE) return CE_ERR_TARGET_RANGE;
    return CE_OK;
}

ce_status ce_wait_timeout_probe(void* workspace, size_t workspace_bytes, void* stream) {
    if (!workspace || workspace_bytes < kWsHeaderBytes) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return CE_ERR_INVALID_ARG;
    uint32_t* err = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + kWsErrOffset);
    if (launch_wait_probe(err, static_cast<cudaStream_t>(stream)) != cudaSuccess) return launch_failed();
    return CE_OK;
}

const char* ce_status_string(ce_status status) {
    switch (status) {
        case CE_OK: return "ok";
        case CE_ERR_INVALID_ARG: return "invalid argument";
        case CE_ERR_UNSUPPORTED_DTYPE: return "unsupported dtype";
        case CE_ERR_BAD_STRIDE:
            return "bad stride: the vocabulary stride must be 1, no stride negative, and (for the "
                   "in-place gradient) no two rows may share memory";
        case CE_ERR_WORKSPACE_TOO_SMALL: return "workspace smaller than ce_workspace_bytes()";
        case CE_ERR_LAUNCH: return "a CUDA launch or runtime call failed";
        case CE_ERR_TARGET_RANGE: return "a target outside [0, V) that is not ignore_idx";
        case CE_ERR_DEVICE_TIMEOUT: return "a bounded wait inside a kernel gave up";
        case CE_ERR_UNSUPPORTED_PATH: return "the forced path cannot run this shape";
    }
    return "unknown status";
}

int ce_plan_path(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                 const int64_t strides[3], const ce_options* opts, int* chunks_out) {
    if ((int)dtype < CE_F32 || (int)dtype > CE_F16 || !strides || V < 1 || dim0 < 0 || dim1 < 0)
        return -1;
    if (strides[2] != 1 || strides[0] < 0 || strides[1] < 0 || !opts_clean(opts)) return -1;
    static const int64_t zero_t[2] = {0, 0};
    Problem pb;
    fill_problem(pb, logits, dtype, dim0, dim1, V, strides, nullptr, zero_t, 0.f, -100, 0);
    Plan pl = make_plan(pb, opts);
    if (pl.path < 0) return pl.path;
    if (chunks_out)
        *chunks_out = pl.path == CE_PATH_TWO_STAGE ? pl.split.chunks
                      : pl.path == CE_PATH_STREAM  ? (pl.stream.geo == kStreamChunks ? pl.stream.nchunks : 1)
                      : (pl.path == CE_PATH_WARP || pl.path == CE_PATH_VECROW) ? 1
                                                                               : pl.fused.cluster;
    return pl.path;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// ce_fwd_bwd_noalloc: the pass with its scratch in a fixed device array.
//
// Scratch (error word, row count, per-row losses of the mean, two-stage
// partials) normally lives in the caller's workspace.  This entry point takes
// it from g_noalloc_scratch, a file-scope __device__ array that every GPU
// loading the library holds until the process exits.  In host code the name
// g_noalloc_scratch denotes a host-side shadow, not device memory, so it is
// never handed to a kernel: its device address is looked up once per device
// with cudaGetSymbolAddress (with that device current) and cached.
// ---------------------------------------------------------------------------
#include <mutex>

namespace gbce {
namespace {

constexpr size_t kNoAllocScratchBytes = (size_t)2 << 20;  // 2 MiB per GPU
constexpr int kNoAllocMaxDevices = 64;

static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

std::mutex g_noalloc_mutex;
void* g_noalloc_device_ptr[kNoAllocMaxDevices];  // device address per device, set once

// Device address of the scratch on the current device (set-up on first use).
ce_status noalloc_scratch(void** out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kNoAllocMaxDevices)
        return launch_failed();
    std::lock_guard<std::mutex> lock(g_noalloc_mutex);
    if (!g_noalloc_device_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return launch_failed();
        g_noalloc_device_ptr[dev] = p;
    }
    *out = g_noalloc_device_ptr[dev];
    return CE_OK;
}

// Scratch bytes the planned pass actually touches: the header, the per-row
// loss slots, and the two-stage partials when that path runs.
size_t noalloc_need(const Problem& pb, const Plan& pl) {
    size_t need = kWsHeaderBytes + align_up((size_t)pb.N * sizeof(float), 256);
    if (pl.path == CE_PATH_TWO_STAGE)
        need += align_up((size_t)pb.N * (size_t)pl.split.chunks * sizeof(float4), 256);
    if (pl.path == CE_PATH_STREAM && pl.stream.geo == kStreamChunks)
        need += align_up((size_t)pb.N * (size_t)pl.stream.nchunks * sizeof(float4), 256);
    return need;
}

}  // namespace
}  // namespace gbce

extern "C" ce_status ce_fwd_bwd_noalloc(void* logits, ce_dtype dtype, ce_layout layout,
                                        int64_t dim0, int64_t dim1, int64_t V,
                                        const int64_t strides[3], const int64_t* targets,
                                        const int64_t target_strides[2], float label_smoothing,
                                        int64_t ignore_idx, int reduce_loss, const float* dloss,
                                        float* loss_out, void* grad_inplace,
                                        int64_t* n_non_ignore_out, const ce_options* opts,
                                        void* stream) {
    if (dim0 < 0 || dim1 < 0 || V < 1 || V > 0x7fffffffLL || !strides) return CE_ERR_INVALID_ARG;
    // argument checks of ce_fwd_bwd; the workspace test is replaced by the
    // scratch-size test below, so a placeholder aligned pointer stands in here
    ce_status st = check_common(logits, dtype, layout, dim0, dim1, V, strides, targets,
                                target_strides, label_smoothing, reduce_loss, loss_out,
                                reinterpret_cast<void*>(256), workspace_need(dim0 * dim1, V, opts),
                                opts);
    if (st != CE_OK) return st;
    if (grad_inplace != logits) return CE_ERR_INVALID_ARG;
    if (!rows_disjoint(dim0, dim1, V, strides[0], strides[1])) return CE_ERR_BAD_STRIDE;
    Problem pb;
    fill_problem(pb, logits, dtype, dim0, dim1, V, strides, targets, target_strides,
                 label_smoothing, ignore_idx, reduce_loss);
    pb.dloss = dloss;
    pb.grad = true;
    Plan pl = make_plan(pb, opts);
    if (pl.path < 0) return CE_ERR_UNSUPPORTED_PATH;
    if (noalloc_need(pb, pl) > kNoAllocScratchBytes) return CE_ERR_WORKSPACE_TOO_SMALL;
    void* scratch = nullptr;
    st = noalloc_scratch(&scratch);
    if (st != CE_OK) return st;
    return run_pass(pb, opts, loss_out, n_non_ignore_out, scratch,
                    static_cast<cudaStream_t>(stream));
}

extern "C" ce_status ce_noalloc_get_error(void* stream, uint32_t* host_err) {
    if (!host_err) return CE_ERR_INVALID_ARG;
    void* scratch = nullptr;
    const ce_status st = gbce::noalloc_scratch(&scratch);
    if (st != CE_OK) return st;
    return ce_get_error(scratch, stream, host_err);
}
