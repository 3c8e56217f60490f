// ce_rowscan.cuh -- what the passes over rows of logits share: a row's softmax
// statistics, and the exact selection of its largest logits on the way.
//
// Statistics of a set of logits x at the scale L = log2(e) / temperature, with
// y = (x - m) L: the maximum m, d = sum 2^y and s = sum y 2^y, so that
//   log-probability = (x - m) / temperature - log d,   entropy = log d - ln 2 * s / d
// (the differences x - m are taken first: a row that lies at -3e4, or at the type's
// lowest value, keeps its digits).  An infinite or missing logit counts for
// nothing in d and s; a NaN makes both NaN.
//
// Selection of the K largest, ties to the lowest column: a candidate is the key
// (value, ~column), so keys differ and their order is the answer's.  A threshold T
// under which no logit can be among the K largest keeps nearly all logits out: the
// K-th largest of the maxima of 256 (K over 64: 1024) groups of the logits read so
// far, which K logits at least are not below.  It is taken in the first tile and
// again in tiles 1, 3, 7, ..., so of random logits about K (1 + ln 2) come in at
// each and 1.2 K to 1.4 K are left at the end; in between only what is above T
// counts, since K logits not below it lie in columns before.
// A tile that could overfill the buffer (equal or rising logits) is taken vector by
// vector with the buffer sorted in between, so any row is exact in bounded time.
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

__device__ __forceinline__ Stat stat_combine(const Stat& a, const Stat& b, float L) {
    const float m = fmaxf(a.m, b.m);
    const float ya = a.m == m ? 0.f : fmaxf((a.m - m) * L, kFarBelow);
    const float yb = b.m == m ? 0.f : fmaxf((b.m - m) * L, kFarBelow);
    const float fa = ex2_approx(ya), fb = ex2_approx(yb);
    return Stat{m, fa * a.d + fb * b.d, fa * fmaf(a.d, ya, a.s) + fb * fmaf(b.d, yb, b.s)};
}

__device__ __forceinline__ Stat stat_warp(Stat a, float L) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(kFull, a.m, off);
        b.d = __shfl_xor_sync(kFull, a.d, off);
        b.s = __shfl_xor_sync(kFull, a.s, off);
        a = stat_combine(a, b, L);
    }
    return a;
}

// Nothing is allowed in the row (every logit -inf).
__device__ __forceinline__ bool stat_none(float m, float d) { return m == -INFINITY && d == d; }

// One logit more.
__device__ __forceinline__ void stat_add(Stat& a, float x, float L) {
    Stat b{x == x ? x : -INFINITY, x == -INFINITY ? 0.f : (x == x && x != INFINITY ? 1.f : NAN), 0.f};
    a = stat_combine(a, b, L);
}

// The vectors of one tile that a thread holds (have: those that are there).  ENT: s as
// well.  GM: the running maxima of the thread's vector places, kept packed.
template <typename T, int NV, bool ENT, bool GM>
__device__ __forceinline__ float stat_tile(Stat& a, const uint4 (&raw)[NV], const bool (&have)[NV], float L,
                                           typename Vec<T>::Max (&gm)[NV]) {
    using VT = Vec<T>;
    constexpr int PP = VT::kElems / 2;
    typename VT::Max tm = VT::max_init();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!have[i]) continue;
        tm = VT::max_acc(tm, raw[i]);
        if (GM) gm[i] = VT::max_acc(gm[i], raw[i]);
    }
    const float top = VT::max_done(tm);
    if (top > a.m) {
        const float y = fmaxf((a.m - top) * L, kFarBelow), f = ex2_approx(y);
        if (ENT) a.s = f * fmaf(a.d, y, a.s);
        a.d *= f;
        a.m = top;
    }
    const float nm = a.m == -INFINITY ? 0.f : -a.m;
    const float2 NM = make_float2(nm, nm), LL = make_float2(L, L);
    float2 d2 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (have[i]) {
            float2 x[PP];
            VT::unpack2(raw[i], x);
#pragma unroll
            for (int k = 0; k < PP; ++k) {
                float2 y = __fmul2_rn(__fadd2_rn(x[k], NM), LL);
                const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                d2 = __fadd2_rn(d2, e);
                if (ENT) {
                    y.x = fmaxf(y.x, kFarBelow);
                    y.y = fmaxf(y.y, kFarBelow);
                    s2 = __ffma2_rn(e, y, s2);
                }
            }
        }
    }
    a.d += d2.x + d2.y;
    if (ENT) a.s += s2.x + s2.y;
    return top;
}

// ----------------------------------------------------------------- barriers
// Over the kScanThreads threads that read tiles (others may belong to the CTA).  Not the
// aligned form (bar.sync): that one says that the warp's lanes arrive together, and
// where they do not (after a lane's own work or a wait that lanes leave one by one)
// a later __syncwarp is taken for done and lane 0 hands a slot back before the others
// have read it.
__device__ __forceinline__ void scan_sync() {
    __syncwarp();
    asm volatile("barrier.sync 1, %0;" ::"n"(kScanThreads) : "memory");
}
__device__ __forceinline__ int scan_count(bool v) {  // how many threads passed true
    uint32_t n;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.popc.u32 %0, 1, %2, p;\n\t}"
        : "=r"(n)
        : "r"((uint32_t)v), "n"(kScanThreads)
        : "memory");
    return (int)n;
}

// Every thread's statistics combined in a fixed order; all threads get them.
// `red`: a slot for each warp, not used by others until the next barrier.
__device__ __forceinline__ Stat stat_block(Stat a, float L, float4* red) {
    a = stat_warp(a, L);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float4(a.m, a.d, a.s, 0.f);
    scan_sync();
    Stat t = stat_identity();
#pragma unroll
    for (int w = 0; w < kScanThreads / 32; ++w) {
        const float4 v = red[w];
        t = stat_combine(t, Stat{v.x, v.y, v.z}, L);
    }
    return t;
}
__device__ __forceinline__ float scan_sum(float v, float* red) {
    v = warp_allsum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    scan_sync();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kScanThreads / 32; ++w) t += red[w];
    return t;
}
__device__ __forceinline__ float scan_max(float v, float* red) {
    v = warp_allmax(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    scan_sync();
    float t = -INFINITY;
#pragma unroll
    for (int w = 0; w < kScanThreads / 32; ++w) t = fmaxf(t, red[w]);
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

struct TopSmem {
    uint64_t buf[kTopCap];
    int cnt[16];
    int count;
};

// The largest 16-bit head of an ordered value that at least K of the groups' maxima
// reach, where each thread brings n of them (v); as the value it stands for, rounded
// down.  False: there are fewer than K groups (a group without logits is no group).
template <int NG>
__device__ __forceinline__ bool kth_group(TopSmem& s, const uint32_t (&v)[NG], int K, float& T) {
    uint32_t head = 0;
    if (NG > 1) {
        if (threadIdx.x < 16) s.cnt[threadIdx.x] = 0;
        scan_sync();
    }
    for (int b = 15; b >= 0; --b) {
        const uint32_t cand = head | (1u << b);
        int n;
        if (NG == 1) {
            n = scan_count(v[0] >= cand);
        } else {
            int own = 0;
#pragma unroll
            for (int i = 0; i < NG; ++i) own += v[i] >= cand;
            own = (int)__reduce_add_sync(kFull, (unsigned)own);
            if ((threadIdx.x & 31) == 0) atomicAdd(&s.cnt[b], own);
            scan_sync();
            n = s.cnt[b];
        }
        if (n >= K) head = cand;
        if (n == K) break;
    }
    T = head <= 0x007fu ? -INFINITY : key_value((uint64_t)head << 48);
    return head != 0;
}
__device__ __forceinline__ uint32_t value_head(float x) { return (uint32_t)(top_key(x, 0) >> 48); }

// The first c keys of buf in falling order.  All threads, between barriers.
__device__ __forceinline__ void top_sort(TopSmem& s, int c) {
    const int tid = threadIdx.x;
    if (c <= kScanThreads) {
        // few: each key's rank is the number of larger ones
        const uint64_t own = tid < c ? s.buf[tid] : 0;
        int r = 0;
        if ((tid & ~31) < c)
            for (int k = 0; k < c; ++k) r += s.buf[k] > own;
        scan_sync();
        if (tid < c) s.buf[r] = own;
        scan_sync();
        return;
    }
    int n = 2 * kScanThreads;
    while (n < c) n *= 2;
    for (int k = c + tid; k < n; k += kScanThreads) s.buf[k] = 0;
    scan_sync();
    for (int size = 2; size <= n; size *= 2) {
        for (int step = size / 2; step > 0; step /= 2) {
            for (int p = tid; p < n / 2; p += kScanThreads) {
                const int lo = p & (step - 1), i = 2 * (p - lo) + lo, j = i + step;
                const uint64_t a = s.buf[i], b = s.buf[j];
                if ((a < b) == ((i & size) == 0)) {
                    s.buf[i] = b;
                    s.buf[j] = a;
                }
            }
            scan_sync();
        }
    }
}

// The state of a selection, the same in every thread of the CTA.
struct TopState {
    int K;
    int bound;     // candidates held, at most
    float T;
    bool all;      // no threshold yet: every logit counts
    bool strict;   // K logits not below T are held: only what is above it counts

    __device__ __forceinline__ bool takes(float x) const { return all ? x == x : (strict ? x > T : x >= T); }

    // Sorts what is held and keeps the K largest.
    __device__ __forceinline__ void compact(TopSmem& s) {
        scan_sync();
        const int c = s.count;
        top_sort(s, c);
        bound = c < K ? c : K;
        if (c >= K) {
            T = key_value(s.buf[K - 1]);
            all = false;
            strict = true;
        }
        scan_sync();
        if (threadIdx.x == 0) s.count = bound;
        scan_sync();
    }

    // What the buffer holds now.
    __device__ __forceinline__ void recount(TopSmem& s) {
        scan_sync();
        bound = s.count;
        if (!all && bound >= K) strict = true;
        scan_sync();
    }
};

// Vectors [i0, i1) of each lane that `hit`: a warp takes a lane's logits together.
// tile: its vectors, nvec of them; col0: the column of its first logit.
template <typename T>
__device__ __forceinline__ void top_push(TopSmem& s, const TopState& st, bool hit, const T* tile, int nvec,
                                         uint32_t col0, int i0, int i1) {
    constexpr int VEC = Vec<T>::kElems;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned todo = __ballot_sync(kFull, hit);
    const int i = i0 + lane / VEC, e = lane % VEC;  // VEC * kScanVecs <= 32
    while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int v = warp * 32 + src + i * kScanThreads;
        float x = NAN;
        if (i < i1 && v < nvec) x = to_f32(tile[v * VEC + e]);
        const bool ok = st.takes(x);
        const unsigned m = __ballot_sync(kFull, ok);
        if (m == 0u) continue;
        int base = 0;
        if (lane == 0) base = atomicAdd(&s.count, __popc(m));
        base = __shfl_sync(kFull, base, 0);
        if (ok) s.buf[base + __popc(m & ((1u << lane) - 1u))] = top_key(x, col0 + (uint32_t)(v * VEC + e));
    }
}
__device__ __forceinline__ void top_push_one(TopSmem& s, float x, uint32_t column) {
    s.buf[atomicAdd(&s.count, 1)] = top_key(x, column);
}

__device__ __forceinline__ TopState top_start(TopSmem& s, int K) {
    TopState st;
    st.K = K;
    st.bound = 0;
    st.T = -INFINITY;
    st.all = true;
    st.strict = false;
    if (threadIdx.x == 0) s.count = 0;
    return st;
}

// Raises the threshold from the groups' running maxima (has: the thread's group i has a
// logit).  What is held and not below the new threshold was let in by the old one; the
// present tile is to be taken with `takes` as it is then.
template <typename T, int NV>
__device__ __forceinline__ bool top_raise(TopSmem& s, TopState& st, const typename Vec<T>::Max (&gm)[NV], int has,
                                          float edge) {
    using VT = Vec<T>;
    float t;
    bool ok;
    if (st.K <= 64) {
        float f = edge;
#pragma unroll
        for (int i = 0; i < NV; ++i) f = fmaxf(f, VT::max_done(gm[i]));
        const uint32_t v[1] = {has ? value_head(f) : 0u};
        ok = kth_group<1>(s, v, st.K, t);
    } else {
        uint32_t v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float f = VT::max_done(gm[i]);
            v[i] = (has >> i) & 1 ? value_head(i == 0 ? fmaxf(f, edge) : f) : 0u;
        }
        ok = kth_group<NV>(s, v, st.K, t);
    }
    const bool up = ok && (st.all || t > st.T);
    if (up) {
        st.T = t;
        st.all = false;
        st.strict = false;
    }
    return up;
}

// Drops what is held below the threshold.
__device__ __forceinline__ void top_prune(TopSmem& s, TopState& st) {
    constexpr int EACH = kTopCap / kScanThreads;
    const int lane = threadIdx.x & 31;
    scan_sync();
    const int c = s.count;
    uint64_t k[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int at = i * kScanThreads + threadIdx.x;
        k[i] = at < c ? s.buf[at] : 0;
    }
    scan_sync();
    if (threadIdx.x == 0) s.count = 0;
    scan_sync();
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (i * kScanThreads >= c) break;
        const bool ok = k[i] != 0 && (st.all || key_value(k[i]) >= st.T);
        const unsigned m = __ballot_sync(kFull, ok);
        int base = 0;
        if (lane == 0 && m) base = atomicAdd(&s.count, __popc(m));
        base = __shfl_sync(kFull, base, 0);
        if (ok) s.buf[base + __popc(m & ((1u << lane) - 1u))] = k[i];
    }
}

// A tile's candidates.  top: the maximum of the thread's logits in it (and of
// `edge`, an element before the tile's vectors, where has_edge).
template <typename T>
__device__ __forceinline__ void top_tile(TopSmem& s, TopState& st, bool has, float top, const T* tile, int nvec,
                                         uint32_t col0, bool has_edge, float edge, uint32_t edge_col) {
    constexpr int VEC = Vec<T>::kElems;
    constexpr int EACH = VEC * kScanVecs + 1;
    bool hit = has && st.takes(top);
    int nh = scan_count(hit);
    if (nh == 0) return;
    if (st.bound + nh * EACH > kTopCap) {
        st.recount(s);
        if (st.bound >= 2 * st.K && st.bound >= 64) {
            st.compact(s);
            hit = has && st.takes(top);
            nh = scan_count(hit);
            if (nh == 0) return;
        }
    }
    if (st.bound + nh * EACH <= kTopCap) {
        if (hit && has_edge && st.takes(edge)) top_push_one(s, edge, edge_col);
        top_push<T>(s, st, hit, tile, nvec, col0, 0, kScanVecs);
        st.bound += nh * EACH;
        return;
    }
    if (hit && has_edge && st.takes(edge)) top_push_one(s, edge, edge_col);  // fewer than VEC in all
    for (int i = 0; i < kScanVecs; ++i) {
        st.recount(s);
        if (st.bound + kScanThreads * VEC > kTopCap) st.compact(s);
        top_push<T>(s, st, hit, tile, nvec, col0, i, i + 1);
    }
    st.recount(s);
}

// ----------------------------------------------------------------- the ring
// Tiles of a row's 16-byte aligned body, copied into a ring of shared memory by one
// thread of a warp of its own (1-D bulk copies).  full[s] completes when the tile in slot
// s has landed, empty[s] when every reading warp is done with it.  Every wait is
// bounded: one that gives up raises `gone` and the error word; the copying thread then
// issues no more, waits (bounded) for what it has issued and leaves, and the readers
// run through their rows without waiting.
constexpr int kRingMost = 12;
struct RingBars {
    uint64_t full[kRingMost], empty[kRingMost];
    volatile int gone;
};
struct RingAt {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) {
            s = 0;
            ph ^= 1u;
        }
    }
};
__device__ __forceinline__ void ring_init(RingBars& b, int stages) {
    for (int s = 0; s < stages; ++s) {
        mbar_init(&b.full[s], 1);
        mbar_init(&b.empty[s], kScanThreads / 32);
    }
    b.gone = 0;
    fence_barrier_init();
}
// The copying thread: `bytes` (a multiple of 16, not 0) of src into the next slot.
__device__ __forceinline__ bool ring_put(RingBars& b, RingAt& at, uint32_t& issued, int stages, unsigned char* ring,
                                         int slot_bytes, const void* src, uint32_t bytes, uint64_t policy) {
    if (!mbar_wait_bounded(&b.empty[at.s], at.ph ^ 1u)) {
        b.gone = 1;
        return false;
    }
    mbar_arrive_expect_tx(&b.full[at.s], bytes);
    tma_load_1d(ring + (size_t)at.s * slot_bytes, src, bytes, &b.full[at.s], policy);
    at.next(stages);
    ++issued;
    return true;
}
// Before the copying thread leaves early: every copy issued lands.
__device__ __forceinline__ void ring_drain(RingBars& b, uint32_t issued, int stages) {
    for (int s = 0; s < stages; ++s)
        if (issued > (uint32_t)s)
            (void)mbar_wait_bounded(&b.full[s], ((issued - 1u - (uint32_t)s) / (uint32_t)stages) & 1u);
}
// A reading thread: the slot `at` has landed (or the ring is gone).
__device__ __forceinline__ void ring_wait(RingBars& b, const RingAt& at) {
    if (!b.gone && !mbar_wait_bounded(&b.full[at.s], at.ph)) b.gone = 1;
}
__device__ __forceinline__ void ring_release(RingBars& b, RingAt& at, int stages) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&b.empty[at.s]);
    at.next(stages);
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
