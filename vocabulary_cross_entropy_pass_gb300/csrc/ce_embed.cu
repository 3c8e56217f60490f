// ce_embed.cu -- rows of the (V, H) vocabulary matrix by token, and their
// gradient.
//
//   out_i = scale * W[t_i]           (t_i == ignore_idx: zeros; outside [0, V): NaN)
//   dW_v (+)= scale * sum over i with t_i = v of g_i
//
// Forward: one gathered read and one write per element, bound by HBM (32768 tokens
// of 4096 bf16, 128000 rows: 60 us, 0.91 of the copy rate for distinct rows read
// once; off the 16-byte grid 0.5 to 0.7).
//
// Gradient: equal tokens meet, so the sum is taken over the tokens in sorted
// order, which makes it the same on every run.
//   1. ce_embed_sort_kernel: a stable radix sort of (token, position) by one
//      cluster of up to eight CTAs: each warp counts the digits of its own run of
//      tokens in shared memory, the CTAs exchange their counts over distributed
//      shared memory, each warp then sends its run in order to the CTAs that hold
//      the places (up to 65536 tokens stay on chip between the digits).
//      Ignored and out-of-range tokens become key V and sort to the end.  The
//      sort is a chain of latencies on eight SMs: the launch's other CTAs zero
//      the gradient meanwhile, where it is to be written whole.
//   2. ce_embed_grad_kernel: a CTA sums a fixed number of sorted entries over
//      a slab of columns, in registers, a gradient row at a time; a token
//      whose entries all lie in the chunk is written at once, one that crosses
//      a chunk border leaves its float32 part in the workspace.
//   3. ce_embed_join_kernel: the parts of tokens that cross chunk borders,
//      added in chunk order.
// Few tokens (those launches' latencies would be most of the time): one kernel in
// which each token's CTA looks through all tokens, the first of each value sums
// its rows in order, and further CTAs zero the rows of tokens that do not occur.
// 16384 tokens of 4096 bf16 added to a 128000-row float32 gradient: 12.5 us of
// sorting, 61 us of sums (360 MB, 0.88 of the copy rate), 10 us of joining (the most
// frequent token's 29 parts), 88 us together; 65536 tokens 253 us, 131072 (sorted
// through global memory) 464, 0.69 of the copy rate.
#include "ce_device.cuh"
#include "ce_internal.h"
#include "ce_pack.cuh"
#include "ce_span.cuh"

namespace gbce {
namespace {

struct EmbedFwdArgs {
    const int64_t* tok;
    int64_t dim1, ts0, ts1, N;
    int flat;
    const char* w;
    char* out;
    int64_t ws, os;        // row strides in bytes
    int64_t V, H, ignore;
    float scale;
    uint32_t* err;         // or NULL
};

__device__ __forceinline__ int64_t token_at(const int64_t* tok, int64_t dim1, int64_t ts0, int64_t ts1, int flat,
                                            int64_t i) {
    if (flat) return __ldg(tok + i * ts1);
    const int64_t a = i / dim1;
    return __ldg(tok + a * ts0 + (i - a * dim1) * ts1);
}

// One CTA (128 threads) or, for rows of at most 128 vectors, one warp per token
// and slab of U vectors of 16 bytes a thread.  SHIFT: rows off
// the 16-byte grid (odd widths, views): the output's vectors, each cut out of
// the two vectors of the matrix's row that hold it, the elements around them one
// per thread.
template <typename T, int U, bool SHIFT>
__global__ void __launch_bounds__(128) ce_embed_fwd_kernel(const __grid_constant__ EmbedFwdArgs p) {
    constexpr int ES = sizeof(T);
    constexpr int VEC = 16 / ES;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.N) return;
    const int TX = blockDim.x;
    const int v0 = blockIdx.y * (TX * U) + threadIdx.x;
    const int64_t t = token_at(p.tok, p.dim1, p.ts0, p.ts1, p.flat, row);
    char* out = p.out + row * p.os;
    const bool in = t >= 0 && t < p.V && t != p.ignore;
    const float fill = t == p.ignore ? 0.f : __int_as_float(0x7fc00000);
    if (!in && t != p.ignore && p.err && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.err, CE_DEVERR_TARGET_RANGE);
    const char* src = p.w + (in ? t : 0) * p.ws;
    int nv = (int)(p.H / VEC);
    int safe0 = 0, safe1 = nv;
    uint32_t ph = 0;
    if (SHIFT) {
        const Span16 sp = span16<ES>(out, 0, p.H);
        nv = (int)sp.nv;
        const int64_t e = span16_edge(sp, 0, p.H, threadIdx.x);
        if (e >= 0 && blockIdx.y == 0) {
            T o;
            from_f32(o, in ? to_f32(reinterpret_cast<const T*>(src)[e]) * p.scale : fill);
            reinterpret_cast<T*>(out)[e] = o;
        }
        const int64_t at = sp.h1 * ES;
        out += at;
        ph = (uint32_t)(reinterpret_cast<uintptr_t>(src + at) & 15u);
        src += at - ph;
        // a shifted vector's two lie inside the row: not before its first element,
        // not past its last
        safe0 = at < (int64_t)ph ? 1 : 0;
        const int64_t room = (p.H * ES - at + ph) / 16 - (ph ? 1 : 0);
        safe1 = (int)(room < nv ? room : nv);
    }
    Pack<T, VEC> a[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = v0 + u * TX;
        if (!in || v >= nv) continue;
        const uint4* q = reinterpret_cast<const uint4*>(src) + v;
        if (!SHIFT || (ph == 0u && v < safe1)) {
            a[u].raw = __ldg(q);
        } else if (v >= safe0 && v < safe1) {
            a[u].raw = shift_bytes(__ldg(q), __ldg(q + 1), ph);
        } else {
            const T* x = reinterpret_cast<const T*>(src + ph) + (int64_t)v * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) a[u].v[i] = x[i];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = v0 + u * TX;
        if (v >= nv) continue;
        Pack<T, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.set(i, in ? a[u].f(i) * p.scale : fill);
        o.store(out + (int64_t)v * 16);
    }
}

// ----------------------------------------------------------------- sorted tokens
constexpr int kSortThreads = 512;
constexpr int kSortWarps = 16;
constexpr int kMaxDigitBits = 9;         // one bin per thread
constexpr int kSortCluster = 8;
constexpr int kOnChip = 8192;            // entries a CTA holds in shared memory, at most

struct SortArgs {
    const int64_t* tok;
    int64_t dim1, ts0, ts1;
    int flat;
    uint32_t N, V;
    int64_t ignore;
    int passes, bits;      // digits of `bits` bits, least first
    int on_chip;           // entries per CTA kept in shared memory between the digits, or 0: in a and b
    uint32_t* err;
    uint2* a;              // (key, position): the sorted ones end here
    uint2* b;
    char* zero;            // the gradient to be zeroed, or NULL
    int64_t zrows, zstride, zbytes;  // its rows, their stride and bytes
};

__device__ __forceinline__ uint32_t ld_dsmem_u32(const uint32_t* local, uint32_t rank) {
    uint32_t remote, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
    return v;
}
__device__ __forceinline__ void st_dsmem_u2(uint2* local, uint32_t rank, uint2 v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(remote), "r"(v.x), "r"(v.y) : "memory");
}

// Zero one row (a warp): 16-byte vectors between a head and a tail of two-byte
// pieces.
__device__ __forceinline__ void zero_row(char* row, int64_t bytes) {
    const int lane = threadIdx.x & 31;
    int64_t head = (int64_t)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u);
    if (head > bytes) head = bytes;
    const int64_t nv = (bytes - head) / 16;
    uint4* body = reinterpret_cast<uint4*>(row + head);
#pragma unroll 4
    for (int64_t v = lane; v < nv; v += 32) __stcs(body + v, make_uint4(0, 0, 0, 0));
    const int64_t t0 = head + nv * 16;  // lanes 0..7 the head, 8..15 the tail
    const int64_t at = lane < 8 ? lane * 2 : t0 + (lane - 8) * 2;
    if (lane < 8 ? at < head : (lane < 16 && at < bytes)) *reinterpret_cast<uint16_t*>(row + at) = 0;
}

__global__ void __launch_bounds__(kSortThreads) ce_embed_sort_kernel(const __grid_constant__ SortArgs p) {
    extern __shared__ __align__(16) uint32_t sm[];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank(), nc = cluster_nctarank();
    if (cluster_id_x() > 0) {
        const int64_t step = ((int64_t)gridDim.x - nc) * kSortWarps;
        for (int64_t r = ((int64_t)blockIdx.x - nc) * kSortWarps + warp; r < p.zrows; r += step)
            zero_row(p.zero + r * p.zstride, p.zbytes);
        return;
    }
    const int bins = 1 << p.bits;
    uint32_t* hist = sm;                          // [16][bins]: a warp's digit counts, then its next places
    uint32_t* total = sm + kSortWarps * bins;     // [bins + 1]: this CTA's counts, and whether a token is out of range
    uint32_t* start = total + bins + 4;           // [bins]: where this CTA's entries of the digit go
    uint32_t* wsum = start + bins;                // [16]
    uint2* here = reinterpret_cast<uint2*>(wsum + 16);  // [2][on_chip]
    const uint32_t mask = (uint32_t)bins - 1;

    // each warp owns a run of tokens, in order over warps and CTAs
    const uint32_t per = (p.N + nc * kSortThreads - 1) / (nc * kSortThreads) * 32;
    const uint64_t from = (uint64_t)(rank * kSortWarps + warp) * per;
    const uint32_t i0 = (uint32_t)(from < p.N ? from : p.N);
    const uint32_t i1 = (uint32_t)(from + per < p.N ? from + per : p.N);
    const uint32_t per_cta = kSortWarps * per, mine0 = rank * per_cta;  // its entries, the first one
    // at / per_cta is the upper half of at times this: exact while at times the
    // rounding (below per_cta) is below 2^32, and on chip both are at most 2^16
    const uint32_t per_cta_inv = per_cta ? 0xffffffffu / per_cta + 1u : 0u;
    if (tid == 0) total[bins] = 0u;

    for (int pass = 0; pass < p.passes; ++pass) {
        const bool last = pass + 1 == p.passes;
        const int shift = pass * p.bits;
        // read from `src` at i: this CTA's shared memory, or b and a in turn (the
        // last digit is written to a)
        uint2* chip = here + (pass & 1 ? p.on_chip : 0);
        uint2* next = here + (pass & 1 ? 0 : p.on_chip);
        uint2* src = ((p.passes - pass) & 1) ? p.b : p.a;
        uint2* dst = ((p.passes - pass) & 1) ? p.a : p.b;
        auto entry = [&](uint32_t i) -> uint2 { return p.on_chip ? chip[i - mine0] : __ldcg(src + i); };
        for (int i = tid; i < kSortWarps * bins / 4; i += kSortThreads)
            reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint32_t* mine = hist + warp * bins;
        if (pass == 0) {
            bool out = false;
            for (uint32_t base = i0; base < i1; base += 128) {
                int64_t t[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t i = base + u * 32 + lane;
                    if (i < i1) t[u] = token_at(p.tok, p.dim1, p.ts0, p.ts1, p.flat, i);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t i = base + u * 32 + lane;
                    if (i < i1) {
                        const bool ok = t[u] >= 0 && t[u] < (int64_t)p.V && t[u] != p.ignore;
                        const uint32_t key = ok ? (uint32_t)t[u] : p.V;
                        out |= !ok && t[u] != p.ignore;
                        // what this thread sends on below
                        if (p.on_chip) chip[i - mine0] = make_uint2(key, i);
                        else src[i] = make_uint2(key, i);
                        atomicAdd(&mine[key & mask], 1u);
                    }
                }
            }
            if (out) total[bins] = 1u;
        } else {
            for (uint32_t i = i0 + lane; i < i1; i += 32) atomicAdd(&mine[(entry(i).x >> shift) & mask], 1u);
        }
        __syncthreads();
        // each bin (one per thread): exclusive prefix over the warps, the CTA's total
        if (tid < bins) {
            uint32_t c[kSortWarps], run = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * bins + tid];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                hist[w * bins + tid] = run;
                run += c[w];
            }
            total[tid] = run;
        }
        if (nc > 1) cluster_sync(); else __syncthreads();
        uint32_t before = 0, all = 0;
        if (tid < bins) {
            uint32_t c[kSortCluster];
#pragma unroll
            for (uint32_t r = 0; r < kSortCluster; ++r) c[r] = r < nc ? ld_dsmem_u32(total + tid, r) : 0u;
#pragma unroll
            for (uint32_t r = 0; r < kSortCluster; ++r) {
                if (r < rank) before += c[r];
                all += c[r];
            }
        }
        if (pass == 0 && rank == 0 && tid < 32) {
            const bool out = lane < (int)nc && ld_dsmem_u32(total + bins, lane) != 0u;
            const bool any = __any_sync(kFull, out);
            if (lane == 0) *p.err = any ? CE_DEVERR_TARGET_RANGE : 0u;
        }
        // exclusive scan of `all` over the bins
        uint32_t inc = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        uint32_t ws = lane < kSortWarps ? wsum[lane] : 0u;
#pragma unroll
        for (int o = 1; o < kSortWarps; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, ws, o);
            if (lane >= o) ws += u;
        }
        const uint32_t upto = __shfl_sync(kFull, ws, warp == 0 ? 0 : warp - 1);
        if (tid < bins) start[tid] = (warp == 0 ? 0u : upto) + inc - all + before;
        // this CTA has read the others' counts: with the last digit it only
        // has to stay until they have read its own
        if (last && nc > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        __syncthreads();
        for (uint32_t base = i0; base < i1; base += 32) {
            const uint32_t i = base + lane;
            const bool on = i < i1;
            const uint2 e = on ? entry(i) : make_uint2(0u, 0u);
            const uint32_t d = (e.x >> shift) & mask;
            // the lanes with the same digit, a bit of it at a time (bits past the
            // digit's are zero everywhere)
            unsigned peers = __ballot_sync(kFull, on);
#pragma unroll
            for (int k = 0; k < kMaxDigitBits; ++k) {
                const unsigned one = __ballot_sync(kFull, (d >> k) & 1u);
                peers &= (d >> k) & 1u ? one : ~one;
            }
            uint32_t at = 0;
            if (on) at = start[d] + mine[d] + __popc(peers & ((1u << lane) - 1u));
            __syncwarp();
            if (on && lane == __ffs(peers) - 1) mine[d] += __popc(peers);
            __syncwarp();
            if (on) {
                if (last || !p.on_chip) {
                    dst[at] = e;
                } else {
                    const uint32_t to = __umulhi(at, per_cta_inv);
                    st_dsmem_u2(next + (at - to * per_cta), to, e);
                }
            }
        }
        if (last) break;
        if (!p.on_chip) __threadfence();
        if (nc > 1) cluster_sync(); else __syncthreads();  // the next pass reads what all CTAs wrote
    }
    if (nc > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ----------------------------------------------------------------- sums of runs
struct GradArgs {
    const uint2* ent;      // sorted (token, position)
    uint32_t N, V;
    int64_t H;
    const char* g;
    int64_t gs;            // gradient row stride in bytes
    char* dw;
    int64_t dws;           // in bytes
    float* part;           // [chunks][2][H]
    int nv;                // vectors per row
    int R;                 // entries per chunk
    int chunks;
    int accumulate;
    float scale;
};

constexpr int kGradThreads = 128;
constexpr int kMaxR = 64;

// One run's sum.  Adding goes through L2's reductions: a row has one writer, so
// the result does not depend on any order, and the thread does not wait for what
// is there (a load in its place held every run's end up for an HBM latency).
// L2 takes values below 2^-126 as zeros.
template <typename TW, int VEC>
__device__ __forceinline__ void write_row(char* row, int64_t col, const float* acc, float scale, int accumulate) {
    if constexpr (sizeof(TW) == 4) {
        float* q = reinterpret_cast<float*>(row) + col;
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = acc[i] * scale;
        if (!accumulate) {
            store_f32<VEC>(q, o);
        } else if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4)
                asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(q + i), "f"(o[i]), "f"(o[i + 1]),
                             "f"(o[i + 2]), "f"(o[i + 3])
                             : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) asm volatile("red.global.add.f32 [%0], %1;" ::"l"(q + i), "f"(o[i]) : "memory");
        }
    } else {
        Pack<TW, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.set(i, acc[i] * scale);
        o.store(row + col * (int64_t)sizeof(TW));
    }
}

template <typename T, typename TW, int VEC>
__global__ void __launch_bounds__(kGradThreads) ce_embed_grad_kernel(const __grid_constant__ GradArgs p) {
    constexpr int ES = sizeof(T);
    constexpr int U = 8;
    const int v = blockIdx.y * kGradThreads + threadIdx.x;
    const bool on = v < p.nv;
    const int64_t col = (int64_t)v * VEC;
    __shared__ uint2 ent[kMaxR + 2];  // the chunk's entries between its neighbours
    griddep_wait();
    griddep_launch_dependents();
    // tokens without a gradient have key V and lie at the end: no chunk's run
    // reaches into them
    const uint32_t c0 = blockIdx.x * (uint32_t)p.R;
    int mine = 0;
    if ((int)threadIdx.x < p.R + 2) {
        const int64_t at = (int64_t)c0 + threadIdx.x - 1;
        uint2 e = make_uint2(0xffffffffu, 0u);
        if (at >= 0 && at < (int64_t)p.N) e = p.ent[at];
        if (e.x >= p.V) e.x = 0xffffffffu;
        ent[threadIdx.x] = e;
        mine = threadIdx.x >= 1 && (int)threadIdx.x <= p.R && e.x != 0xffffffffu;
    }
    const int len = __syncthreads_count(mine);
    if (!on) return;
    const char* g = p.g + col * ES;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    int begin = 1;  // first entry of the current run
    for (int b = 1; b <= len; b += U) {
        Pack<T, VEC> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b + u <= len) x[u].load_cs(g + (int64_t)ent[b + u].y * p.gs);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = b + u;
            if (k > len) break;
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += x[u].f(i);
            const uint32_t key = ent[k].x;
            const bool last = ent[k + 1].x != key;
            if (last || k == len) {
                const bool from_here = begin > 1 || ent[0].x != key;
                if (from_here && last) {
                    write_row<TW, VEC>(p.dw + (int64_t)key * p.dws, col, acc, p.scale, p.accumulate);
                } else {
                    float* q = p.part + ((int64_t)blockIdx.x * 2 + (from_here ? 1 : 0)) * p.H + col;
                    store_f32<VEC>(q, acc);
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
                begin = k + 1;
            }
        }
    }
}

// A run that crosses chunk borders begins in one chunk (its part is that chunk's
// second) and fills whole chunks (their first parts) up to its last.
template <typename TW, int VEC>
__global__ void __launch_bounds__(kGradThreads) ce_embed_join_kernel(const __grid_constant__ GradArgs p) {
    griddep_wait();
    const uint32_t n = p.N;
    const uint64_t c0 = (uint64_t)blockIdx.x * p.R, c1 = c0 + p.R;
    if (c1 >= n) return;                        // the last chunk's last run ends there
    const uint32_t key = p.ent[c1 - 1].x, over = p.ent[c1].x;
    const uint32_t at0 = p.ent[c0].x, prev = c0 > 0 ? p.ent[c0 - 1].x : 0xffffffffu;
    if (over != key || key >= p.V) return;      // no run crosses this border
    if (at0 == key && prev == key) return;      // it began in an earlier chunk
    // the last chunk that begins with the token, 32 chunks at a look
    const int lane = threadIdx.x & 31;
    int64_t last = blockIdx.x + 1;
    for (;;) {
        const int64_t c = last + 1 + lane;
        const uint64_t i = (uint64_t)c * p.R;
        const unsigned same = __ballot_sync(kFull, i < n && p.ent[i < n ? i : 0].x == key);
        const int k = same == kFull ? 32 : __ffs(~same) - 1;
        last += k;
        if (k < 32) break;
    }
    const int64_t col = ((int64_t)blockIdx.y * kGradThreads + threadIdx.x) * VEC;
    if (col >= p.H) return;
    constexpr int B = 8;
    float acc[VEC];
    load_f32<VEC>(p.part + ((int64_t)blockIdx.x * 2 + 1) * p.H + col, acc);
    for (int64_t c = blockIdx.x + 1; c <= last; c += B) {
        float v[B][VEC];
#pragma unroll
        for (int u = 0; u < B; ++u)
            if (c + u <= last) load_f32<VEC>(p.part + (c + u) * 2 * p.H + col, v[u]);
#pragma unroll
        for (int u = 0; u < B; ++u)
            if (c + u <= last)
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] += v[u][i];
    }
    write_row<TW, VEC>(p.dw + (int64_t)key * p.dws, col, acc, p.scale, p.accumulate);
}

// ----------------------------------------------------------------- few tokens
constexpr int kFewThreads = 256;
constexpr int kFewTokens = 1024;         // at most
constexpr int kFewCols = 256;            // columns of a CTA
constexpr int kZeroRows = 4096;          // rows of a CTA that zeroes, at most

struct FewArgs {
    const int64_t* tok;
    int64_t dim1, ts0, ts1;
    int flat;
    int N;
    int64_t V, H, ignore;
    const char* g;
    int64_t gs;            // in bytes
    char* dw;
    int64_t dws, row_bytes;
    uint32_t* err;
    int zero_rows;         // rows of each zeroing CTA (blockIdx.x >= N)
    int accumulate;
    float scale;
};

// A CTA per token and 256 columns.  All but the first CTA of a value leave; it
// lists the value's places in order, its eight warps take every eighth of
// those rows, and the warps' sums are added in order.
template <typename T, typename TW, int VEC>
__global__ void __launch_bounds__(kFewThreads) ce_embed_few_kernel(const __grid_constant__ FewArgs p) {
    constexpr int ES = sizeof(T);
    constexpr int NW = kFewThreads / 32;
    constexpr int NV = 8 / VEC;            // vectors of a lane: eight columns
    constexpr int U = 4;
    constexpr int IT = kFewTokens / kFewThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto token = [&](int k) { return token_at(p.tok, p.dim1, p.ts0, p.ts1, p.flat, k); };
    if ((int)blockIdx.x >= p.N) {
        if (blockIdx.y > 0) return;
        __shared__ uint32_t used[kZeroRows / 32];
        const int64_t r0 = (int64_t)(blockIdx.x - p.N) * p.zero_rows, r1 = min(p.V, r0 + p.zero_rows);
        for (int k = tid; k < kZeroRows / 32; k += kFewThreads) used[k] = 0u;
        __syncthreads();
        for (int k = tid; k < p.N; k += kFewThreads) {
            const int64_t t = token(k);
            if (t >= r0 && t < r1 && t != p.ignore) atomicOr(&used[(t - r0) >> 5], 1u << ((t - r0) & 31));
        }
        __syncthreads();
        for (int64_t r = r0 + warp; r < r1; r += NW)
            if (!((used[(r - r0) >> 5] >> ((r - r0) & 31)) & 1u)) zero_row(p.dw + r * p.dws, p.row_bytes);
        return;
    }
    __shared__ uint16_t place[kFewTokens];
    __shared__ int count[IT * NW];
    __shared__ __align__(16) float sums[NW][kFewCols];  // written as float4
    const int i = blockIdx.x;
    const int64_t mine = token(i);
    int64_t t[IT];
#pragma unroll
    for (int q = 0; q < IT; ++q) {
        const int k = q * kFewThreads + tid;
        t[q] = k < p.N ? token(k) : p.ignore;
    }
    if (i == 0 && blockIdx.y == 0) {
        bool out = false;
#pragma unroll
        for (int q = 0; q < IT; ++q) out |= t[q] != p.ignore && (t[q] < 0 || t[q] >= p.V);
        const int any = __syncthreads_or(out);
        if (tid == 0) *p.err = any ? CE_DEVERR_TARGET_RANGE : 0u;
    }
    if (mine == p.ignore || mine < 0 || mine >= p.V) return;
    bool earlier = false;
    unsigned same[IT];
#pragma unroll
    for (int q = 0; q < IT; ++q) {
        const bool s = q * kFewThreads + tid < p.N && t[q] == mine;
        earlier |= s && q * kFewThreads + tid < i;
        same[q] = __ballot_sync(kFull, s);
        if (lane == 0) count[q * NW + warp] = __popc(same[q]);
    }
    if (__syncthreads_or(earlier)) return;
    // the value's places in order: token k is in row k / 256 of the loop, then by warp
    int before = 0, m = 0;
#pragma unroll
    for (int q = 0; q < IT; ++q) {
        for (int w = 0; w < NW; ++w) {
            if (w == warp) before = m;
            m += count[q * NW + w];
        }
        if ((same[q] >> lane) & 1u)
            place[before + __popc(same[q] & ((1u << lane) - 1u))] = (uint16_t)(q * kFewThreads + tid);
    }
    __syncthreads();
    float acc[NV][VEC];
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[e][k] = 0.f;
    const int64_t c0 = (int64_t)blockIdx.y * kFewCols;
    for (int j = warp; j < m; j += NW * U) {
        Pack<T, VEC> x[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * NW < m) {
                const char* row = p.g + (int64_t)place[j + u * NW] * p.gs;
#pragma unroll
                for (int e = 0; e < NV; ++e) {
                    const int64_t c = c0 + (e * 32 + lane) * VEC;
                    x[u][e].zero();
                    if (c < p.H) x[u][e].load_cs(row + c * ES);
                }
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * NW < m)
#pragma unroll
                for (int e = 0; e < NV; ++e)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) acc[e][k] += x[u][e].f(k);
    }
    const int warps = m < NW ? m : NW;     // warps that have a sum
    if (warp < warps) {
#pragma unroll
        for (int e = 0; e < NV; ++e) store_f32<VEC>(&sums[warp][(e * 32 + lane) * VEC], acc[e]);
    }
    __syncthreads();
    if (c0 + tid < p.H) {
        float f = sums[0][tid];
        for (int w = 1; w < warps; ++w) f += sums[w][tid];
        write_row<TW, 1>(p.dw + mine * p.dws, c0 + tid, &f, p.scale, p.accumulate);
    }
}

// entries per chunk, from the sizes alone (the workspace holds two float32
// rows for each chunk)
int chunk_entries(int64_t N) { return N >= 8192 ? 32 : (N >= 1024 ? 16 : 8); }

// Whether one kernel takes all (every CTA looks through all tokens).  Added to a tied
// gradient, few / sorted: 16 tokens of 4096 2.7 / 8.3 us, 100 of 4096 (1600 CTAs)
// 5.9 / 9.3, 256 of 4096 (4096 CTAs) 11.2 / 9.9.
bool few_tokens(int64_t N, int64_t H) {
    return N > 0 && N <= kFewTokens && N * ((H + kFewCols - 1) / kFewCols) <= 2048;
}

struct EmbedWs {
    size_t a, b, part, bytes;
    int R, chunks;
};
EmbedWs embed_ws(int64_t N, int64_t H) {
    EmbedWs w;
    w.R = chunk_entries(N);
    w.chunks = (int)((N + w.R - 1) / w.R);
    w.a = kWsHeaderBytes;
    w.b = w.a + align_up((size_t)N * 8, 256);
    w.part = w.b + align_up((size_t)N * 8, 256);
    w.bytes = w.part + (size_t)w.chunks * 2 * (size_t)H * 4;
    return w;
}

bool bad_dtype(int d) { return d < CE_F32 || d > CE_F16; }
bool off_grid(const void* p, int es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }
bool bad_sizes(int64_t N, int64_t H, int64_t V) {
    return N < 0 || N > 0x7ffffff0LL || H < 1 || H > (1 << 20) || V < 1 || V > 0x7fffffffLL;
}
// N of (dim0, dim1), or -1
int64_t count_of(int64_t d0, int64_t d1) {
    if (d0 < 0 || d1 < 0 || d0 > 0x7fffffffLL || d1 > 0x7fffffffLL) return -1;
    return d0 * d1;
}
bool tokens_flat(int64_t d0, int64_t d1, const int64_t* ts) { return d0 == 1 || ts[0] == d1 * ts[1]; }

template <typename T, bool SHIFT>
cudaError_t launch_fwd(const EmbedFwdArgs& a, cudaStream_t s) {
    const int64_t nv = (a.H * (int64_t)sizeof(T) + 15) / 16;
    // few tokens: a vector a thread over more CTAs
    if (a.N * ((nv + 511) / 512) < 1024)
        ce_embed_fwd_kernel<T, 1, SHIFT><<<dim3((unsigned)a.N, (unsigned)((nv + 127) / 128)), 128, 0, s>>>(a);
    else if (nv <= 128)
        ce_embed_fwd_kernel<T, 4, SHIFT><<<(unsigned)((a.N + 3) / 4), dim3(32, 4), 0, s>>>(a);
    else
        ce_embed_fwd_kernel<T, 4, SHIFT><<<dim3((unsigned)a.N, (unsigned)((nv + 511) / 512)), 128, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_fwd_t(const EmbedFwdArgs& a, int vb, cudaStream_t s) {
    return vb == 16 ? launch_fwd<T, false>(a, s) : launch_fwd<T, true>(a, s);
}

// A kernel that may start while the one before it ends.
template <typename K, typename A>
cudaError_t launch_behind(K* k, dim3 grid, int threads, const A& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    set_pdl_attr(at);
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename T, typename TW, int VEC>
cudaError_t launch_grad(GradArgs& a, cudaStream_t s) {
    if (a.chunks == 0) return cudaSuccess;
    a.nv = (int)(a.H / VEC);
    const dim3 grid((unsigned)a.chunks, (unsigned)((a.nv + kGradThreads - 1) / kGradThreads));
    cudaError_t e = launch_behind(ce_embed_grad_kernel<T, TW, VEC>, grid, kGradThreads, a, s);
    if (e != cudaSuccess || a.chunks == 1) return e;
    constexpr int JV = VEC >= 4 ? 4 : 1;  // floats of the parts per thread
    const dim3 join((unsigned)(a.chunks - 1), (unsigned)((a.H / JV + kGradThreads - 1) / kGradThreads));
    return launch_behind(ce_embed_join_kernel<TW, JV>, join, kGradThreads, a, s);
}
template <typename T>
cudaError_t launch_grad_t(GradArgs& a, bool w32, int vb, cudaStream_t s) {
    constexpr int ES = sizeof(T);
    if (w32) {
        if (vb == 16) return launch_grad<T, float, 16 / ES>(a, s);
        if constexpr (ES == 2)
            if (vb == 4) return launch_grad<T, float, 2>(a, s);
        return launch_grad<T, float, 1>(a, s);
    }
    if constexpr (ES == 2) {
        if (vb == 16) return launch_grad<T, T, 8>(a, s);
        if (vb == 4) return launch_grad<T, T, 2>(a, s);
        return launch_grad<T, T, 1>(a, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T, typename TW, int VEC>
cudaError_t launch_few_v(const FewArgs& a, cudaStream_t s) {
    const int64_t zero = a.zero_rows ? (a.V + a.zero_rows - 1) / a.zero_rows : 0;
    // the zeroing CTAs go by the first slab alone
    const unsigned slabs = (unsigned)((a.H + kFewCols - 1) / kFewCols);
    ce_embed_few_kernel<T, TW, VEC><<<dim3((unsigned)(a.N + zero), slabs), kFewThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_few(const FewArgs& a, bool w32, int vb, cudaStream_t s) {
    constexpr int ES = sizeof(T);
    if constexpr (ES == 4) {
        return vb == 16 ? launch_few_v<T, float, 4>(a, s) : launch_few_v<T, float, 1>(a, s);
    } else {
        if (w32) return vb == 16 ? launch_few_v<T, float, 8>(a, s) : launch_few_v<T, float, 1>(a, s);
        return vb == 16 ? launch_few_v<T, T, 8>(a, s) : launch_few_v<T, T, 1>(a, s);
    }
}

cudaError_t launch_sort(SortArgs& a, cudaStream_t s) {
    const int bins = 1 << a.bits;
    int nc = 1;
    while (nc < kSortCluster && (int64_t)nc * 1024 < a.N) nc *= 2;
    const int64_t each = ((int64_t)a.N + nc * kSortThreads - 1) / (nc * kSortThreads) * kSortThreads;
    const size_t counts = (size_t)(kSortWarps * bins + 2 * bins + 20) * 4;
    a.on_chip = each <= kOnChip && counts + (size_t)each * 16 <= 220 * 1024 ? (int)each : 0;
    const size_t smem = counts + (size_t)a.on_chip * 16;
    cudaError_t e;
    if (smem > 40 * 1024 &&
        (e = cudaFuncSetAttribute(ce_embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
            cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    // a warp for every row to zero, up to two CTAs on each of the other SMs
    int extra = 0;
    if (a.zero) {
        const int64_t want = (a.zrows + kSortWarps - 1) / kSortWarps;
        extra = (int)(want < 288 ? want : 288);
        extra = (extra + nc - 1) / nc * nc;
    }
    cfg.gridDim = dim3(nc + extra);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = nc;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ce_embed_sort_kernel, a);
}

}  // namespace
}  // namespace gbce

using namespace gbce;

extern "C" ce_status ce_embed_fwd(const int64_t* tokens, int64_t dim0, int64_t dim1, const int64_t token_strides[2],
                                  const void* weight, ce_dtype dtype, int64_t V, int64_t H, int64_t weight_stride,
                                  float scale, int64_t ignore_idx, void* out, int64_t out_stride, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype)) return CE_ERR_UNSUPPORTED_DTYPE;
    const int64_t N = count_of(dim0, dim1);
    if (bad_sizes(N, H, V) || !token_strides) return CE_ERR_INVALID_ARG;
    if (workspace && (reinterpret_cast<uintptr_t>(workspace) % 16)) return CE_ERR_INVALID_ARG;
    if (workspace && workspace_bytes < kWsHeaderBytes) return CE_ERR_WORKSPACE_TOO_SMALL;
    if (N > 0) {
        if (!tokens || !weight || !out) return CE_ERR_INVALID_ARG;
        const int es = elem_size(dtype);
        if (off_grid(weight, es) || off_grid(out, es) || off_grid(tokens, 8)) return CE_ERR_INVALID_ARG;
        if (token_strides[0] < 0 || token_strides[1] < 0) return CE_ERR_BAD_STRIDE;
        if ((V > 1 && weight_stride < H) || (N > 1 && out_stride < H)) return CE_ERR_BAD_STRIDE;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    EmbedFwdArgs a;
    a.err = workspace ? reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + kWsErrOffset) : nullptr;
    if (a.err && cudaMemsetAsync(a.err, 0, 4, s) != cudaSuccess) return launch_failed();
    if (N == 0) return CE_OK;
    const int es = elem_size(dtype);
    a.tok = tokens;
    a.dim1 = dim1;
    a.ts0 = token_strides[0];
    a.ts1 = token_strides[1];
    a.N = N;
    a.flat = tokens_flat(dim0, dim1, token_strides);
    a.w = static_cast<const char*>(weight);
    a.out = static_cast<char*>(out);
    a.ws = weight_stride * es;
    a.os = out_stride * es;
    a.V = V;
    a.H = H;
    a.ignore = ignore_idx;
    a.scale = scale;
    const uint64_t vals[] = {(uint64_t)(uintptr_t)weight, (uint64_t)(uintptr_t)out, (uint64_t)(V > 1 ? a.ws : 0),
                             (uint64_t)(N > 1 ? a.os : 0), (uint64_t)H * es};
    const int vb = common_vector_bytes(vals, 5, es);
    cudaError_t e = dtype == CE_F32    ? launch_fwd_t<float>(a, vb, s)
                    : dtype == CE_BF16 ? launch_fwd_t<__nv_bfloat16>(a, vb, s)
                                       : launch_fwd_t<__half>(a, vb, s);
    return e == cudaSuccess ? CE_OK : launch_failed();
}

extern "C" size_t ce_embed_bwd_workspace_bytes(int64_t N, int64_t H, int64_t V) {
    if (bad_sizes(N, H, V)) return 0;
    return embed_ws(N, H).bytes;
}

extern "C" ce_status ce_embed_bwd(const void* grad_out, ce_dtype dtype, int64_t grad_out_stride,
                                  const int64_t* tokens, int64_t dim0, int64_t dim1,
                                  const int64_t token_strides[2], int64_t V, int64_t H, float scale,
                                  int64_t ignore_idx, void* grad_weight, ce_dtype grad_dtype,
                                  int64_t grad_weight_stride, int accumulate, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype) || (grad_dtype != CE_F32 && grad_dtype != dtype)) return CE_ERR_UNSUPPORTED_DTYPE;
    if (accumulate && grad_dtype != CE_F32) return CE_ERR_UNSUPPORTED_DTYPE;
    const int64_t N = count_of(dim0, dim1);
    if (bad_sizes(N, H, V) || !token_strides || !grad_weight || !workspace) return CE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return CE_ERR_INVALID_ARG;
    const int es = elem_size(dtype), wes = elem_size(grad_dtype);
    if (off_grid(grad_weight, wes)) return CE_ERR_INVALID_ARG;
    if (V > 1 && grad_weight_stride < H) return CE_ERR_BAD_STRIDE;
    if (N > 0) {
        if (!grad_out || !tokens || off_grid(grad_out, es) || off_grid(tokens, 8)) return CE_ERR_INVALID_ARG;
        if (token_strides[0] < 0 || token_strides[1] < 0 || grad_out_stride < 0) return CE_ERR_BAD_STRIDE;
    }
    const EmbedWs w = embed_ws(N, H);
    if (workspace_bytes < w.bytes) return CE_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* base = static_cast<char*>(workspace);
    const uint64_t vals[] = {(uint64_t)(uintptr_t)grad_out, (uint64_t)(N > 1 ? grad_out_stride * es : 0),
                             (uint64_t)H * es, (uint64_t)(uintptr_t)grad_weight,
                             (uint64_t)(V > 1 ? grad_weight_stride * wes : 0)};
    const int vb = common_vector_bytes(vals, 5, es);
    const bool w32 = grad_dtype == CE_F32;

    if (few_tokens(N, H)) {
        FewArgs fa;
        fa.tok = tokens;
        fa.dim1 = dim1 > 0 ? dim1 : 1;
        fa.ts0 = token_strides[0];
        fa.ts1 = token_strides[1];
        fa.flat = tokens_flat(dim0, dim1, token_strides);
        fa.N = (int)N;
        fa.V = V;
        fa.H = H;
        fa.ignore = ignore_idx;
        fa.g = static_cast<const char*>(grad_out);
        fa.gs = grad_out_stride * es;
        fa.dw = static_cast<char*>(grad_weight);
        fa.dws = grad_weight_stride * wes;
        fa.row_bytes = H * wes;
        fa.err = reinterpret_cast<uint32_t*>(base + kWsErrOffset);
        // zeroing: about two CTAs on each SM, more for more rows than they take
        const int64_t per = (V + 303) / 304;
        fa.zero_rows = accumulate ? 0 : (int)(per < 8 ? 8 : (per > kZeroRows ? kZeroRows : per));
        fa.accumulate = accumulate ? 1 : 0;
        fa.scale = scale;
        cudaError_t e = dtype == CE_F32    ? launch_few<float>(fa, true, vb, s)
                        : dtype == CE_BF16 ? launch_few<__nv_bfloat16>(fa, w32, vb, s)
                                           : launch_few<__half>(fa, w32, vb, s);
        return e == cudaSuccess ? CE_OK : launch_failed();
    }

    SortArgs sa;
    sa.tok = tokens;
    sa.dim1 = dim1 > 0 ? dim1 : 1;
    sa.ts0 = token_strides[0];
    sa.ts1 = token_strides[1];
    sa.flat = tokens_flat(dim0, dim1, token_strides);
    sa.N = (uint32_t)N;
    sa.V = (uint32_t)V;
    sa.ignore = ignore_idx;
    int bits = 1;
    while (((uint64_t)V >> bits) != 0) ++bits;  // keys 0 .. V
    sa.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    sa.bits = (bits + sa.passes - 1) / sa.passes;
    if (sa.bits < 2) sa.bits = 2;
    sa.err = reinterpret_cast<uint32_t*>(base + kWsErrOffset);
    uint2* a = reinterpret_cast<uint2*>(base + w.a);
    sa.a = a;
    sa.b = reinterpret_cast<uint2*>(base + w.b);
    sa.zero = accumulate ? nullptr : static_cast<char*>(grad_weight);
    sa.zrows = V;
    sa.zstride = grad_weight_stride * wes;
    sa.zbytes = H * wes;
    if (sa.zero && (V == 1 || sa.zstride == sa.zbytes)) {
        // one run of memory: rows of 16 KB
        const int64_t all = V * sa.zbytes, row = 16384;
        if (all % row == 0 || all < row) {
            sa.zrows = all < row ? 1 : all / row;
            sa.zstride = sa.zbytes = all < row ? all : row;
        }
    }
    if (launch_sort(sa, s) != cudaSuccess) return launch_failed();
    if (N == 0) return CE_OK;

    GradArgs ga;
    ga.ent = a;
    ga.N = sa.N;
    ga.V = sa.V;
    ga.H = H;
    ga.g = static_cast<const char*>(grad_out);
    ga.gs = grad_out_stride * es;
    ga.dw = static_cast<char*>(grad_weight);
    ga.dws = grad_weight_stride * wes;
    ga.part = reinterpret_cast<float*>(base + w.part);
    ga.R = w.R;
    ga.chunks = w.chunks;
    ga.accumulate = accumulate ? 1 : 0;
    ga.scale = scale;
    cudaError_t e = dtype == CE_F32    ? launch_grad_t<float>(ga, true, vb, s)
                    : dtype == CE_BF16 ? launch_grad_t<__nv_bfloat16>(ga, w32, vb, s)
                                       : launch_grad_t<__half>(ga, w32, vb, s);
    return e == cudaSuccess ? CE_OK : launch_failed();
}
