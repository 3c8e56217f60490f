// ce_rowscan.cuh -- what the passes over rows of logits share: a row's softmax
// statistics, and the exact selection of its largest logits on the way.
//
// Statistics of a set of logits x at the scale L = log2(e) / temperature: the maximum m,
// d = sum 2^y and s = sum y 2^y with y = x L - M, M = m L rounded (one fused step from x, and
// M is a reference like any other: what its rounding shifts is given back in log d), so
//   log d = ln 2 (log2 d - (m L - M)),  log-probability = (x - m) / temperature - log d,
//   entropy = ln 2 (log2 d - s / d).
// Where M leaves float32 (a row at the type's lowest value) y = (x - m) L.  A logit of
// -inf counts for nothing in d and s; a NaN makes both NaN.
//
// The streaming kernels built on this (ce_logprobs.cu, ce_distill.cu) are persistent;
// the warps of a CTA have three parts and meet at mbarriers alone:
//   the copying warp  takes rows (or segments of rows), describes each in a slot of a short
//                     queue and copies its 16-byte aligned body tile by tile into a ring
//                     (1-D bulk copies);
//   eight main warps  take the tiles out, sum the statistics and, where a gradient
//                     is written, take the row's tiles a second time; a row costs
//                     them a warp reduction and no barrier of their own;
//   four side warps   do what a row has beside its stream, while the main warps are
//                     on the next: the elements around the body, the given or listed
//                     tokens, the largest logits, the outputs.
// (With the eight warps doing all of it between barriers, a row of 32000 columns cost
// them as much again as its tiles did: 16384 rows 210 us.)
//
// Selection of the K largest, ties to the lowest column: a candidate is the key
// (value, ~column), so keys differ and their order is the answer's.  The main warps
// leave the maximum of each group of 32 vectors (K over 64: of 8) of the row; T, the
// K-th largest of them, is a value that K logits at least are not below, so only the
// groups that reach it are read again, from L2, and of random logits 1.1 K to 1.4 K are
// candidates.  Short rows have too few groups: their vectors' maxima are taken first.
// Groups are read in the order of their columns, in batches that the buffer has room
// for after it was sorted and cut to K, and once K candidates are held only what is
// above T counts: equal or ordered logits cost time, not exactness.
#pragma once

#include "ce_device.cuh"
#include "ce_internal.h"
#include "ce_pack.cuh"
#include "ce_rowscan_plan.h"
#include "ce_span.cuh"

namespace gbce {

// ----------------------------------------------------------------- statistics
struct Stat {
    float m, d, s;
};
__device__ __forceinline__ Stat stat_identity() { return Stat{-INFINITY, 0.f, 0.f}; }

constexpr float kFarBelow = -1e4f;  // 2^kFarBelow is 0, and so is its product with it
constexpr float kRefMost = 1e38f;   // a reference this far out is not used
constexpr float kLn2f = 0.6931471805599453f;

__device__ __forceinline__ float stat_ref(float m, float L) { return __fmul_rn(m, L); }
// The exponent by which what is relative to m counts relative to the larger top.
__device__ __forceinline__ float stat_shift(float m, float top, float L) {
    return m == top ? 0.f : fmaxf(stat_ref(m, L) - stat_ref(top, L), kFarBelow);
}

__device__ __forceinline__ Stat stat_combine(const Stat& a, const Stat& b, float L) {
    const float m = fmaxf(a.m, b.m);
    const float ya = stat_shift(a.m, m, L), yb = stat_shift(b.m, m, L);
    const float fa = ex2_approx(ya), fb = ex2_approx(yb);
    return Stat{m, fa * a.d + fb * b.d, fa * fmaf(a.d, ya, a.s) + fb * fmaf(b.d, yb, b.s)};
}

// The warp's statistics, in every lane: one maximum, one factor a lane, plain sums.
template <bool ENT>
__device__ __forceinline__ Stat stat_warp(Stat a, float L) {
    const float m = warp_max_redux(a.m);
    const float y = stat_shift(a.m, m, L), f = ex2_approx(y);
    Stat r{m, f * a.d, ENT ? f * fmaf(a.d, y, a.s) : 0.f};
    r.d = warp_allsum(r.d);
    if (ENT) r.s = warp_allsum(r.s);
    return r;
}

// log sum exp((x - m) / temperature), 0 where nothing is allowed.
__device__ __forceinline__ float stat_logd(const Stat& t, float L) {
    const float M = stat_ref(t.m, L);
    return kLn2f * (log2f(t.d) - (fabsf(M) < kRefMost ? fmaf(t.m, L, -M) : 0.f));
}
__device__ __forceinline__ float stat_entropy(const Stat& t) { return kLn2f * (log2f(t.d) - t.s / t.d); }

// Nothing is allowed in the row (every logit -inf).
__device__ __forceinline__ bool stat_none(float m, float d) { return m == -INFINITY && d == d; }

// One logit more.
__device__ __forceinline__ void stat_add(Stat& a, float x, float L) {
    const float M = stat_ref(x, L), y = fabsf(M) < kRefMost ? fmaf(x, L, -M) : 0.f;
    Stat b{x, ex2_approx(y), 0.f};
    b.s = b.d * y;
    if (x == -INFINITY) b.d = 0.f;
    if (x == INFINITY || x != x) b = Stat{x == x ? x : -INFINITY, NAN, NAN};
    a = stat_combine(a, b, L);
}

// e = 2^y of one vector's logits relative to m, added to d2 and (ENT) with y to s2.  FAR: y
// = (x - m) L, ref = -m (else ref = -M); LOW: some logit may be -inf.
template <typename T, bool ENT, bool FAR, bool LOW>
__device__ __forceinline__ void stat_vector(const uint4& raw, float ref, float L, float2& d2, float2& s2) {
    using VT = Vec<T>;
    constexpr int PP = VT::kElems / 2;
    const float2 R = make_float2(ref, ref), LL = make_float2(L, L);
    float2 x[PP];
    VT::unpack2(raw, x);
#pragma unroll
    for (int k = 0; k < PP; ++k) {
        float2 y = FAR ? __fmul2_rn(__fadd2_rn(x[k], R), LL) : __ffma2_rn(x[k], LL, R);
        const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        d2 = __fadd2_rn(d2, e);
        if (ENT) {
            if (LOW) y = make_float2(fmaxf(y.x, kFarBelow), fmaxf(y.y, kFarBelow));
            s2 = __ffma2_rn(e, y, s2);
        }
    }
}
// What is rarely met, out of the way: a row at the type's lowest value, logits of -inf
// under an entropy.
template <typename T, bool ENT>
__device__ __forceinline__ float4 stat_far(const uint4* src, int n, float m, float L) {
    float2 d2 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
    const bool near = fabsf(stat_ref(m, L)) < kRefMost || m == -INFINITY;
    const float ref = m == -INFINITY ? 0.f : (near ? -stat_ref(m, L) : -m);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        if (near) stat_vector<T, ENT, false, true>(src[i * kMainThreads], ref, L, d2, s2);
        else stat_vector<T, ENT, true, true>(src[i * kMainThreads], ref, L, d2, s2);
    }
    return make_float4(d2.x, d2.y, s2.x, s2.y);
}

// A thread's vectors of a tile: src[0], src[kMainThreads], ..., n of them (FULL: NV).
// ENT: s as well.  GM: each vector's maximum into gm (-inf where there is none).
template <typename T, int NV, bool FULL, bool ENT, bool GM>
__device__ __forceinline__ void stat_tile(Stat& a, const uint4* src, int n, float L, float (&gm)[NV]) {
    using VT = Vec<T>;
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (FULL || i < n) raw[i] = src[i * kMainThreads];
    float top;
    if (GM) {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            gm[i] = FULL || i < n ? VT::vmax(raw[i]) : -INFINITY;
            top = fmaxf(top, gm[i]);
        }
    } else {
        typename VT::Max tm = VT::max_init();
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (FULL || i < n) tm = VT::max_acc(tm, raw[i]);
        top = VT::max_done(tm);
    }
    if (top > a.m) {
        const float y = stat_shift(a.m, top, L), f = ex2_approx(y);
        if (ENT) a.s = f * fmaf(a.d, y, a.s);
        a.d *= f;
        a.m = top;
    }
    float2 d2 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
    const float ref = a.m == -INFINITY ? 0.f : -stat_ref(a.m, L);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (FULL || i < n) stat_vector<T, ENT, false, false>(raw[i], ref, L, d2, s2);
    // (0 times -inf, or a NaN, which d shows too)
    if (!(fabsf(ref) < kRefMost) || (ENT && s2.x + s2.y != s2.x + s2.y)) {
        const float4 v = stat_far<T, ENT>(src, FULL ? NV : n, a.m, L);
        d2 = make_float2(v.x, v.y);
        s2 = make_float2(v.z, v.w);
    }
    a.d += d2.x + d2.y;
    if (ENT) a.s += s2.x + s2.y;
}

// ----------------------------------------------------------------- side warps
// The kSideThreads threads of the side warps (and of the kernels that are all of
// them), numbered from 0.  Not the aligned form (bar.sync): a warp's lanes may come one
// by one, after a lane's own work or a wait.
__device__ __forceinline__ void side_sync() {
    __syncwarp();
    asm volatile("barrier.sync 1, %0;" ::"n"(kSideThreads) : "memory");
}
__device__ __forceinline__ bool side_any(bool v) {
    uint32_t n;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(n)
        : "r"((uint32_t)v), "n"(kSideThreads)
        : "memory");
    return n != 0;
}
// Over the side warps, in a fixed order; `red` is not used by others until the next barrier.
__device__ __forceinline__ float side_sum(float v, float* red, int tid) {
    v = warp_allsum(v);
    if ((tid & 31) == 0) red[tid >> 5] = v;
    side_sync();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSideThreads / 32; ++w) t += red[w];
    return t;
}
__device__ __forceinline__ float side_max(float v, float* red, int tid) {
    v = warp_allmax(v);
    if ((tid & 31) == 0) red[tid >> 5] = v;
    side_sync();
    float t = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSideThreads / 32; ++w) t = fmaxf(t, red[w]);
    return t;
}

// ----------------------------------------------------------------- the largest
// Keys grow with the value (-0 as 0) and fall with the column; 0 is below all.
__device__ __forceinline__ uint64_t top_key(float x, uint32_t column) {
    const uint32_t b = __float_as_uint(x + 0.f);
    const uint32_t o = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
    return ((uint64_t)o << 32) | (0xffffffffu - column);
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t key_column(uint64_t k) { return 0xffffffffu - (uint32_t)k; }
// The first 16 bits of a value's key: they order values rounded down to them (a NaN, the
// maximum of nothing else, as -inf).
constexpr uint32_t kLowestHead = 0x007fu;
__device__ __forceinline__ uint32_t value_head(float x) {
    return x == x ? (uint32_t)(top_key(x, 0) >> 48) : kLowestHead;
}

struct TopSmem {
    uint64_t buf[kTopCap];
    uint16_t vheads[kTopHeads];  // of a short row's vectors
    uint16_t list[kTopHeads];    // groups to be read again
    int count, listed;
    uint32_t kth;
};

// The largest head that at least K of the n heads reach; 0: fewer than K are not 0.  One warp.
__device__ __forceinline__ uint32_t kth_head(const uint16_t* heads, int n, int K) {
    const int lane = threadIdx.x & 31;
    uint32_t kth = 0;
    for (int b = 15; b >= 0; --b) {
        const uint32_t cand = kth | (1u << b);
        int own = 0;
        for (int k = lane * 8; k < n; k += 256) {
            const uint4 u = *reinterpret_cast<const uint4*>(heads + k);  // past n: zeros
            own += ((u.x & 0xffffu) >= cand) + ((u.x >> 16) >= cand) + ((u.y & 0xffffu) >= cand) +
                   ((u.y >> 16) >= cand) + ((u.z & 0xffffu) >= cand) + ((u.z >> 16) >= cand) +
                   ((u.w & 0xffffu) >= cand) + ((u.w >> 16) >= cand);
        }
        const int c = (int)__reduce_add_sync(kFull, (unsigned)own);
        if (c >= K) kth = cand;
        if (c == K) break;
    }
    return kth;
}

// The first c keys of buf in falling order.  All side threads, between barriers.
__device__ __forceinline__ void top_sort(TopSmem& s, int c, int tid) {
    if (c <= 2 * kSideThreads) {
        // few: a key's rank is the number of larger ones
        const uint64_t k0 = tid < c ? s.buf[tid] : 0, k1 = tid + kSideThreads < c ? s.buf[tid + kSideThreads] : 0;
        int r0 = 0, r1 = 0;
        if ((tid & ~31) < c) {
#pragma unroll 4
            for (int k = 0; k < c; ++k) {
                const uint64_t o = s.buf[k];
                r0 += o > k0;
                r1 += o > k1;
            }
        }
        side_sync();
        if (tid < c) s.buf[r0] = k0;
        if (tid + kSideThreads < c) s.buf[r1] = k1;
        side_sync();
        return;
    }
    int n = 4 * kSideThreads;
    while (n < c) n *= 2;
    for (int k = c + tid; k < n; k += kSideThreads) s.buf[k] = 0;
    side_sync();
    for (int size = 2; size <= n; size *= 2) {
        for (int step = size / 2; step > 0; step /= 2) {
            for (int p = tid; p < n / 2; p += kSideThreads) {
                const int lo = p & (step - 1), i = 2 * (p - lo) + lo, j = i + step;
                const uint64_t a = s.buf[i], b = s.buf[j];
                if ((a < b) == ((i & size) == 0)) {
                    s.buf[i] = b;
                    s.buf[j] = a;
                }
            }
            side_sync();
        }
    }
}

// What a selection lets in, the same in every side thread.
struct TopGate {
    int K;
    float T;
    bool all;      // no threshold: every number counts
    bool strict;   // K candidates not below T are held, of columns before: only what is above T counts
    __device__ __forceinline__ bool takes(float x) const { return all ? x == x : (strict ? x > T : x >= T); }
};

// How many candidates are held; sorted and cut to K where there is no room for `more`.
__device__ __forceinline__ int top_room(TopSmem& s, TopGate& g, int more, int tid) {
    side_sync();
    int c = s.count;
    if (c + more > kTopCap) {
        top_sort(s, c, tid);
        if (c >= g.K) {
            c = g.K;
            g.T = key_value(s.buf[c - 1]);
            g.all = false;
        }
        side_sync();
        if (tid == 0) s.count = c;
    }
    g.strict = !g.all && c >= g.K;
    side_sync();
    return c;
}
__device__ __forceinline__ void top_push(TopSmem& s, bool ok, float x, uint32_t column) {
    const unsigned m = __ballot_sync(kFull, ok);
    if (m == 0u) return;
    const int lane = threadIdx.x & 31;
    int base = 0;
    if (lane == 0) base = atomicAdd(&s.count, __popc(m));
    base = __shfl_sync(kFull, base, 0);
    if (ok) s.buf[base + __popc(m & ((1u << lane) - 1u))] = top_key(x, column);
}

// The candidates' buffer sorted and cut to K; how many there are.
__device__ __forceinline__ int top_finish(TopSmem& s, int K, int tid) {
    side_sync();
    const int c = s.count;
    top_sort(s, c, tid);
    return c < K ? c : K;
}

// The K largest of a row's (segment's) logits into the front of s.buf, in falling order;
// returns how many there are.  body: its nv vectors in global memory, their first logit of
// column col0; heads: the groups' maxima, G of them (zeros up to a multiple of 256), `unit`
// vectors each.  xe, ce: the thread's element around the body (before: it lies before the
// body), where has_edge.  All side threads.
template <typename T>
__device__ __forceinline__ int top_select(TopSmem& s, const uint16_t* heads, int G, int unit, const uint4* body,
                                          int64_t nv, uint32_t col0, int K, bool has_edge, bool before, float xe,
                                          uint32_t ce, int tid) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems;
    const int lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s.count = 0;
    if (G < 2 * K && nv <= kTopHeads) {
        for (int v = tid; v < kTopHeads; v += kSideThreads) {
            uint32_t h = 0;
            if (v < nv) h = value_head(VT::vmax(__ldg(body + v)));
            s.vheads[v] = (uint16_t)h;
            if (v >= ((nv + 255) & ~255)) break;
        }
        heads = s.vheads;
        G = (int)nv;
        unit = 1;
    }
    side_sync();
    if (warp == 0) {
        const uint32_t kth = kth_head(heads, G, K);
        int n = 0;
        for (int k0 = 0; k0 < G; k0 += 32) {
            const bool in = k0 + lane < G && heads[k0 + lane] >= (kth ? kth : 1u);
            const unsigned m = __ballot_sync(kFull, in);
            if (in) s.list[n + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(k0 + lane);
            n += __popc(m);
        }
        if (lane == 0) {
            s.kth = kth;
            s.listed = n;
        }
    }
    side_sync();
    const uint32_t kth = s.kth;
    TopGate g;
    g.K = K;
    g.all = kth == 0;
    g.strict = false;
    g.T = kth <= kLowestHead ? -INFINITY : key_value((uint64_t)kth << 48);
    top_push(s, has_edge && before && g.takes(xe), xe, ce);
    // a warp takes 32 vectors at a time, twice in a batch; the next batch's are on their way
    constexpr int STEPS = 2, WARPS = kSideThreads / 32;
    const int per = 32 / unit, batch = STEPS * WARPS * per, listed = s.listed;
    uint4 next[STEPS];
    int64_t vn[STEPS];
    auto fetch = [&](int b) {
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            const int e = b + (u * WARPS + warp) * per + lane / unit;
            vn[u] = e < listed ? (int64_t)s.list[e] * unit + lane % unit : nv;
            if (vn[u] < nv) next[u] = __ldg(body + vn[u]);
        }
    };
    fetch(0);
    for (int b = 0; b < listed; b += batch) {
        uint4 raw[STEPS];
        int64_t v[STEPS];
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            raw[u] = next[u];
            v[u] = vn[u];
        }
        fetch(b + batch);
        top_room(s, g, STEPS * kSideThreads * VEC, tid);
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            const bool hit = v[u] < nv && (g.all || g.takes(VT::vmax(raw[u])));
            if (!__any_sync(kFull, hit)) continue;
            float x[VEC];
            VT::unpack(raw[u], x);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                top_push(s, hit && g.takes(x[k]), x[k], col0 + (uint32_t)(v[u] * VEC + k));
        }
    }
    top_room(s, g, kSideThreads, tid);
    top_push(s, has_edge && !before && g.takes(xe), xe, ce);
    return top_finish(s, K, tid);
}

// ----------------------------------------------------------------- the ring and the queue
// full[s] completes when the tile in slot s has landed, empty[s] when every main warp
// is done with it.  A row's slot in the queue: ready when the copying warp has described
// it, done when every main warp has left its statistics, stored when every main warp has
// stored its gradient, prep when the side warps have worked on its list, and free when
// the main warps and the side warps need it no more.  Every wait is bounded: one that
// gives up raises `gone`, which ends all others; the copying warp then issues no more and
// leaves when what it has issued has landed (bounded too).
constexpr int kRingMost = 6;
constexpr int kQueue = 3;  // places at most
struct RowItem {
    const char* x;      // the row
    char* out;          // its gradient, or NULL
    int64_t row;        // -1: no more
    int64_t v0, nv;     // its first vector of the body and how many
    int64_t item;       // number of the row or segment
    int h1;             // where the body starts
    int head, tail;     // elements before it that go with the item, where those after it start
    int tails;          // how many
    int skip;           // not read
};
struct RowBars {
    uint64_t full[kRingMost], empty[kRingMost];
    uint64_t ready[kQueue], done[kQueue], stored[kQueue], prep[kQueue], free_[kQueue];
    RowItem item[kQueue];
    float4 part[kQueue][kMainThreads / 32];
    volatile int gone;
};
__device__ __forceinline__ void row_bars_init(RowBars& b) {
    constexpr int W = kMainThreads / 32;
    for (int s = 0; s < kRingMost; ++s) {
        mbar_init(&b.full[s], 1);
        mbar_init(&b.empty[s], W);
    }
    for (int s = 0; s < kQueue; ++s) {
        mbar_init(&b.ready[s], 1);
        mbar_init(&b.done[s], W);
        mbar_init(&b.stored[s], W);
        mbar_init(&b.prep[s], 1);
        mbar_init(&b.free_[s], W + 1);
    }
    b.gone = 0;
    fence_barrier_init();
}
// False: gave up, or another wait has.
__device__ __forceinline__ bool row_wait(RowBars& b, uint64_t* bar, uint32_t ph) {
    if (mbar_try_wait(bar, ph)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1; !b.gone; ++it) {
        if (mbar_try_wait(bar, ph)) return true;
        if ((it & 255u) == 0u && global_timer_ns() - t0 > kWaitLimitNs) b.gone = 1;
    }
    return false;
}
// A place in the ring or the queue: slot and phase.
struct Turn {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            ph ^= 1u;
        }
    }
};
// The copying thread: a tile of `bytes` (a multiple of 16, not 0) into the next slot.
__device__ __forceinline__ bool ring_put(RowBars& b, Turn& at, uint32_t& issued, int stages, unsigned char* ring,
                                         int slot_bytes, const void* src, uint32_t bytes, uint64_t policy) {
    if (!row_wait(b, &b.empty[at.s], at.ph ^ 1u)) return false;
    mbar_arrive_expect_tx(&b.full[at.s], bytes);
    tma_load_1d(ring + (size_t)at.s * slot_bytes, src, bytes, &b.full[at.s], policy);
    at.next(stages);
    ++issued;
    return true;
}
// Before the copying thread leaves early: every copy issued lands.
__device__ __forceinline__ void ring_drain(RowBars& b, uint32_t issued, int stages) {
    for (int s = 0; s < stages; ++s)
        if (issued > (uint32_t)s)
            (void)mbar_wait_bounded(&b.full[s], ((issued - 1u - (uint32_t)s) / (uint32_t)stages) & 1u);
}
// A warp is done with something: lane 0 arrives for all.  A ring's slot is handed back
// once its values have been used, not behind the loads: where the warp's global stores
// were backed up, the loads waited behind them and the arrival did not, and the next tile
// landed first (in one of 100 launches of 1219 rows of 20011 float32 columns).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// First pass over a row's tiles by the main warps: the warp's statistics go to part, and
// (GM: 1 a group of 32 vectors, 2 of 8) the groups' maxima to heads.
template <typename T, int NV, bool ENT, int GM>
__device__ __forceinline__ bool main_stats(RowBars& b, Turn& at, int stages, const unsigned char* ring, int q,
                                           int64_t nv, float L, uint16_t* heads) {
    constexpr int TILE = kMainThreads * NV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Stat st = stat_identity();
    for (; nv > 0; nv -= TILE) {
        const uint4* src = reinterpret_cast<const uint4*>(ring + (size_t)at.s * TILE * 16) + tid;
        float gm[NV];
        if (!row_wait(b, &b.full[at.s], at.ph)) return false;
        int mine = NV;
        if (nv >= TILE) {
            stat_tile<T, NV, true, ENT, GM != 0>(st, src, NV, L, gm);
        } else {
            mine = max(0, min(NV, ((int)nv - tid + kMainThreads - 1) / kMainThreads));
            stat_tile<T, NV, false, ENT, GM != 0>(st, src, mine, L, gm);
        }
        warp_arrive(&b.empty[at.s]);
        at.next(stages);
        if (GM == 1) {
            // lane i keeps group i's; 0 where the group has no vector
            float own = -INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float m = warp_max_redux(gm[i]);
                if (lane == i) own = m;
            }
            if (lane < NV)
                heads[lane * (kMainThreads / 32) + warp] =
                    (uint16_t)(lane * kMainThreads + warp * 32 < nv ? value_head(own) : 0u);
            heads += TILE / 32;
        } else if (GM == 2) {
            float own = -INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float m = gm[i];
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
                if ((lane & 7) == i) own = m;
            }
            const int i = lane & 7, first = i * kMainThreads + (tid & ~7);
            if (i < NV) heads[first / 8] = (uint16_t)(first < nv ? value_head(own) : 0u);
            heads += TILE / 8;
        }
    }
    st = stat_warp<ENT>(st, L);
    if (lane == 0) b.part[q][warp] = make_float4(st.m, st.d, st.s, 0.f);
    warp_arrive(&b.done[q]);
    return true;
}

// A row's statistics from the main warps' and the elements around its body (lanes 8 and
// on hold one each); the same in every lane.
template <bool ENT>
__device__ __forceinline__ Stat row_stats(const float4* part, bool has_edge, float xe, float L) {
    constexpr int W = kMainThreads / 32;
    const int lane = threadIdx.x & 31;
    Stat st = stat_identity();
    if (lane < W) {
        const float4 v = part[lane];
        st = Stat{v.x, v.y, v.z};
    } else if (has_edge) {
        stat_add(st, xe, L);
    }
    return stat_warp<ENT>(st, L);
}
// The element around the body that lane 8 + k takes, k counting those before it first: its
// column, or -1.
__device__ __forceinline__ int64_t edge_column(const RowItem& it) {
    const int k = (int)(threadIdx.x & 31) - kMainThreads / 32;
    if (k < 0) return -1;
    if (k < it.head) return k;
    return k - it.head < it.tails ? it.tail + (k - it.head) : -1;
}

// ----------------------------------------------------------------- rows
struct RowAddr {
    int64_t s0, s1, dim1;
    int flat;  // row r at r * s1
    __device__ __forceinline__ int64_t at(int64_t r) const {
        if (flat) return r * s1;
        const int64_t i = r / dim1;
        return i * s0 + (r - i * dim1) * s1;
    }
};
inline RowAddr row_addr(int64_t s0, int64_t s1, int64_t dim0, int64_t dim1) {
    RowAddr a{s0, s1, dim1, 0};
    a.flat = dim0 == 1 || dim1 == 1 || s0 == dim1 * s1 ? 1 : 0;
    if (dim1 == 1 && dim0 != 1) a.s1 = s0;  // row r is (r, 0)
    return a;
}

// A list of tokens for each row (given ones, or a teacher's).
struct RowTokens {
    const int64_t* t;   // NULL: none
    RowAddr row;
    int64_t step;       // between a row's tokens
    int n;
    int64_t ignore_idx;
    __device__ __forceinline__ int64_t at(int64_t r, int k) const { return __ldg(t + row.at(r) + k * step); }
};

}  // namespace gbce
