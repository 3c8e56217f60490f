// ce_rowscan.cuh -- what the passes over rows of logits share: a row's softmax
// statistics, and the exact selection of its largest logits on the way.
//
// Statistics of a set of logits x at the scale L = log2(e) / temperature: the maximum m,
// d = sum 2^y and s = sum y 2^y with y = x L - M, M = m L rounded (one fused step from x, and
// M is a reference like any other: what its rounding shifts is given back in log d), so
//   log d = ln 2 (log2 d - (m L - M)),  log-probability = (x - m) / temperature - log d,
//   entropy = ln 2 (log2 d - s / d).
// Where M is so large that its rounding would carry 2^y out of float32 (a row, or what a thread
// has seen of it, at a mask's -1e30: y is off by 2^76 there) y = (x - m) L.  A logit of -inf
// counts for nothing in d and s; a NaN makes both NaN.
//
// The streaming kernels built on this (ce_logprobs.cu, ce_distill.cu) are persistent;
// the warps of a CTA have three parts and meet at mbarriers alone:
//   the copying warp  takes rows (or segments of rows), describes each in a slot of a short
//                     queue and copies its 16-byte aligned body tile by tile into a ring
//                     (1-D bulk copies);
//   eight main warps  take the tiles out, sum the statistics and, where a gradient
//                     is written, take the row's tiles a second time; a row costs
//                     them a warp reduction and no barrier of their own;
//   the side warps    do what a row has beside its stream, while the main warps are
//                     on the next ones: the elements around the body, the given or
//                     listed tokens, the largest logits, the outputs.
// (With the eight warps doing all of it between barriers, a row of 32000 columns cost
// them as much again as its tiles did: 16384 rows 210 us.)
//
// Selection of the K largest, ties to the lowest column: a candidate is the key
// (value, ~column), so keys differ and their order is the answer's.  Each main thread
// leaves the maximum of its vectors of a tile, eight neighbours (a line of 128 bytes), which
// the statistics want anyway (over eight threads' vectors, by shuffles, it cost half as
// much again as the statistics).
// T, the K-th largest of these, is a value that K logits at least are not below, so only
// the groups that reach it are read again, from L2, and of random logits 1.1 K to 1.4 K
// are candidates.  Short rows have too few groups: their vectors' maxima are taken first.
// Where the buffer of candidates has no room it is sorted and cut to K, and what comes
// later has to be above the K-th key; where equal logits abound (a mask) only groups
// above T are read, and the equals in order from the row's start.  So any row is exact.
// A row's selection is one warp's work, without barriers, and three rows' go on at a time
// (four warps at one row's, with a barrier for each step: 17 us a row of 128000 columns,
// K = 64, beside the stream).  Its code and the main loop share the instruction cache, and
// outgrew it once: loops are not unrolled here (8 of 16384 x 32000 with entropy: 259 us
// unrolled, 219 not).
#pragma once

#include "ce_device.cuh"
#include "ce_internal.h"
#include "ce_pack.cuh"
#include "ce_rowscan_plan.h"
#include "ce_span.cuh"

#include <type_traits>

namespace gbce {

// ----------------------------------------------------------------- statistics
struct Stat {
    float m, d, s;
};
__device__ __forceinline__ Stat stat_identity() { return Stat{-INFINITY, 0.f, 0.f}; }

constexpr float kFarBelow = -1e4f;  // 2^kFarBelow is 0, and so is its product with it
// 2^31: a product below is off by 64 at most, so no 2^y leaves float32 for it.  A larger one is no reference.
constexpr float kRefMost = 2147483648.f;
constexpr float kLn2f = 0.6931471805599453f;

__device__ __forceinline__ float stat_ref(float m, float L) { return __fmul_rn(m, L); }
// By how much the reference M falls short of m L; 0 where m itself is the reference.
__device__ __forceinline__ float stat_short(float m, float M, float L) {
    return fabsf(M) < kRefMost ? fmaf(m, L, -M) : 0.f;
}
// The exponent by which what is relative to m's reference counts relative to the larger top's.  Next to a
// reference that is no product the smaller counts for nothing: two logits there lie 2^7 apart in the
// exponent.  (Where m alone is so far, below, M - T is -128 at most, its sum 2^31 at most and top's 2^-64 at
// least: less than a rounding.)
__device__ __forceinline__ float stat_shift(float m, float top, float L) {
    const float T = stat_ref(top, L);
    const float y = fabsf(T) < kRefMost ? fmaxf(stat_ref(m, L) - T, kFarBelow) : kFarBelow;
    return m == top ? 0.f : y;
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
    return kLn2f * (log2f(t.d) - stat_short(t.m, M, L));
}
__device__ __forceinline__ float stat_entropy(const Stat& t) { return kLn2f * (log2f(t.d) - t.s / t.d); }

// Nothing is allowed in the row (every logit -inf).
__device__ __forceinline__ bool stat_none(float m, float d) { return m == -INFINITY && d == d; }

// One logit more.
__device__ __forceinline__ void stat_add(Stat& a, float x, float L) {
    const float y = stat_short(x, stat_ref(x, L), L);
    Stat b{x, ex2_approx(y), 0.f};
    b.s = b.d * y;
    if (x == -INFINITY) b.d = 0.f;
    if (x == INFINITY || x != x) b = Stat{x == x ? x : -INFINITY, NAN, NAN};
    a = stat_combine(a, b, L);
}

// The larger of two, a NaN where either is one.
__device__ __forceinline__ uint32_t max_nan(uint32_t a, float b, float) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(b));
    return __float_as_uint(r);
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, float b, __nv_bfloat16) {
    return bf162_bits(__hmax2_nan(as_bf162(a), __float2bfloat162_rn(b)));
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, float b, __half) {
    return h2_bits(__hmax2_nan(as_h2(a), __float2half2_rn(b)));
}

// e = 2^y of one vector's logits, added to d2 and (ENT) with y to s2: y = (x + add) L +
// ref, add 0 but where SLOW.  least (ENT): where 2^y is 0, a logit counts as this one, so no
// 0 is multiplied with -inf; taken on packed pairs in 16 bits (SLOW: on y).
template <typename T, bool ENT, bool SLOW>
__device__ __forceinline__ void stat_vector(uint4 raw, float ref, float add, float least, float L, float2& d2,
                                            float2& s2) {
    using VT = Vec<T>;
    constexpr int PP = VT::kElems / 2;
    const float2 R = make_float2(ref, ref), AD = make_float2(add, add), LL = make_float2(L, L);
    if (ENT && !SLOW) {
        raw.x = max_nan(raw.x, least, T());
        raw.y = max_nan(raw.y, least, T());
        raw.z = max_nan(raw.z, least, T());
        raw.w = max_nan(raw.w, least, T());
    }
    float2 x[PP];
    VT::unpack2(raw, x);
#pragma unroll
    for (int k = 0; k < PP; ++k) {
        float2 y = __ffma2_rn(SLOW ? __fadd2_rn(x[k], AD) : x[k], LL, R);
        const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        d2 = __fadd2_rn(d2, e);
        if (ENT) {
            if (SLOW) y = make_float2(fmaxf(y.x, kFarBelow), fmaxf(y.y, kFarBelow));
            s2 = __ffma2_rn(e, y, s2);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 all_low() {  // a vector of -inf, which counts for nothing
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
}
// A warp is done with something: lane 0 arrives for all.  A ring's slot is handed back
// once its values have been used, not behind the loads: where the warp's global stores
// were backed up, the loads waited behind them and the arrival did not, and the next tile
// landed first (in one of 100 launches of 1219 rows of 20011 float32 columns).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint4 ld_smem(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// A thread's vectors of a tile: NV neighbours, n of them there.  It takes them in an order of
// its own (`turn`), so eight threads next to each other meet in no bank of shared memory.
template <int NV>
__device__ __forceinline__ int tile_turn() {
    return NV == 8 ? threadIdx.x & 7 : (threadIdx.x >> 1) & 3;
}
// ENT: s as well.  Returns their maximum.  The tile is handed back (empty) when every
// lane's maximum is known, so all have their values, and the sums go on in registers: with two
// slots both are in flight most of the time.
template <typename T, int NV, bool ENT>
__device__ __forceinline__ float stat_tile(Stat& a, const uint4* tile, int nv, float L, uint64_t* empty) {
    using VT = Vec<T>;
    static_assert(NV == 8 || NV == 4, "the orders");
    const uint4* src = tile + threadIdx.x * NV;
    const int turn = tile_turn<NV>(), n = min(NV, nv - (int)threadIdx.x * NV);
    const uint32_t at = smem_u32(src) + turn * 16u;  // of 16 bytes times NV: the i-th one's is at ^ 16 i
    uint4 raw[NV];
    if (n == NV) {
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[i] = ld_smem(at ^ (16u * i));
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw[i] = all_low<T>();
            if ((i ^ turn) < n) raw[i] = ld_smem(at ^ (16u * i));
        }
    }
    typename VT::Max tm = VT::max_init();
#pragma unroll
    for (int i = 0; i < NV; ++i) tm = VT::max_acc(tm, raw[i]);
    const float top = VT::max_done(tm);
    if (top > a.m) {
        const float y = stat_shift(a.m, top, L), f = ex2_approx(y);
        if (ENT) a.s = f * fmaf(a.d, y, a.s);
        a.d *= f;
        a.m = top;
    }
    const float ref = a.m == -INFINITY ? 0.f : -stat_ref(a.m, L);
    // 2^y is 0 from 150 down; the distance leaves room for the rounding to 16 bits (2^-9 of
    // the maximum).  Without a maximum 2^y is 0 for any logit there is.
    const float top_or_low = a.m == -INFINITY ? kFarBelow : a.m;
    const float least = ENT ? top_or_low - fmaxf(200.f / L, fabsf(top_or_low) * 0.015625f) : 0.f;
    // rarely met: a thread that has seen only a mask's large values (in float16, where `least` is none of its).
    // 4096 x 128000 bf16 with entropy, one token of 64 allowed, the rest -1e30: 193 us, -1e9 or -inf: 164
    const bool far = !(fabsf(ref) < kRefMost);
    const bool slow = far || (ENT && std::is_same<T, __half>::value && least < -65504.f);
    const bool again = __any_sync(kFull, slow);
    if (!again) warp_arrive(empty);
    float2 d2 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) stat_vector<T, ENT, false>(raw[i], ref, 0.f, least, L, d2, s2);
    if (slow) {
        d2 = s2 = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int i = 0; i < n; ++i)
            stat_vector<T, ENT, true>(src[i], far ? 0.f : ref, far ? -a.m : 0.f, 0.f, L, d2, s2);
    }
    if (again) warp_arrive(empty);
    a.d += d2.x + d2.y;
    if (ENT) a.s += s2.x + s2.y;
    return top;
}

// ----------------------------------------------------------------- side warps
// The kSideThreads threads of the side warps (and of the kernels that are all of
// them), numbered from 0.  Not the aligned form (bar.sync): a warp's lanes may come one
// by one, after a lane's own work or a wait.
__device__ __forceinline__ void side_sync() {
    __syncwarp();
    asm volatile("barrier.sync 1, %0;" ::"n"(kSideThreads) : "memory");
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
// A value's place among the values of T in 16 bits: exact in the 16-bit types, of float32
// the first 16 bits of its key, which order values rounded down to them.  A NaN (the
// maximum of nothing else) counts as -inf, the lowest.
template <typename T>
struct Head;
template <>
struct Head<float> {
    static constexpr uint32_t lowest = 0x007fu;
    static constexpr bool exact = false;
    __device__ __forceinline__ static uint32_t of(float x) { return x == x ? (uint32_t)(top_key(x, 0) >> 48) : lowest; }
    __device__ __forceinline__ static float value(uint32_t h) { return key_value((uint64_t)h << 48); }
};
template <>
struct Head<__nv_bfloat16> {
    static constexpr uint32_t lowest = 0x007fu;
    static constexpr bool exact = true;
    __device__ __forceinline__ static uint32_t of(float x) { return Head<float>::of(x); }
    __device__ __forceinline__ static float value(uint32_t h) { return __uint_as_float((h & 0x8000u ? h & 0x7fffu : ~h & 0xffffu) << 16); }
};
template <>
struct Head<__half> {
    static constexpr uint32_t lowest = 0x03ffu;
    static constexpr bool exact = true;
    __device__ __forceinline__ static uint32_t of(float x) {
        const uint32_t b = __half_as_ushort(__float2half_rn(x + 0.f));
        return x == x ? (b & 0x8000u ? ~b & 0xffffu : b | 0x8000u) : lowest;
    }
    __device__ __forceinline__ static float value(uint32_t h) {
        return __half2float(__ushort_as_half((unsigned short)(h & 0x8000u ? h & 0x7fffu : ~h)));
    }
};

// The candidates of one warp's selection.
struct alignas(16) TopSmem {
    uint64_t buf[kTopCap];
    int bins[160];  // of heads; then vectors to be looked at: 31 left over and 128 more
};

// Few keys: a key's rank is the number of larger ones (75 keys: half the instructions of
// a sorting network).
template <int NK>
__device__ __forceinline__ void sort_by_rank(TopSmem& s, int c) {
    const int lane = threadIdx.x & 31;
    uint64_t k[NK];
    int r[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        k[i] = 32 * i + lane < c ? s.buf[32 * i + lane] : 0;
        r[i] = 0;
    }
#pragma unroll 4
    for (int j = 0; j < c; ++j) {
        const uint64_t o = s.buf[j];
#pragma unroll
        for (int i = 0; i < NK; ++i) r[i] += o > k[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NK; ++i)
        if (32 * i + lane < c) s.buf[r[i]] = k[i];
    __syncwarp();
}

// The first c keys of buf in falling order.  One warp.  Neither unrolled nor inlined, like the
// searches below: the side warps' code shares the instruction cache with the main loop.
static __device__ __noinline__ void top_sort(TopSmem& s, int c) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if (c <= 1) return;
    if (c <= 32) return sort_by_rank<1>(s, c);
    if (c <= 64) return sort_by_rank<2>(s, c);
    if (c <= 128) return sort_by_rank<4>(s, c);
    int n = 256;
    while (n < c) n *= 2;
#pragma unroll 1
    for (int k = c + lane; k < n; k += 32) s.buf[k] = 0;
    __syncwarp();
#pragma unroll 1
    for (int size = 2; size <= n; size *= 2) {
#pragma unroll 1
        for (int step = size / 2; step > 0; step /= 2) {
#pragma unroll 2
            for (int p = lane; p < n / 2; p += 32) {
                const int lo = p & (step - 1), i = 2 * (p - lo) + lo, j = i + step;
                const uint64_t a = s.buf[i], b = s.buf[j];
                if ((a < b) == ((i & size) == 0)) {
                    s.buf[i] = b;
                    s.buf[j] = a;
                }
            }
            __syncwarp();
        }
    }
}

// What a selection lets in, the same in every lane: logits above T, and those equal to it of
// columns below C.
struct TopGate {
    int K;
    int held;      // candidates
    float T;
    uint32_t C;

    __device__ __forceinline__ TopGate(int K, float T) : K(K), held(0), T(T), C(0xffffffffu) {}
    __device__ __forceinline__ bool takes(float x, uint32_t col) const { return x > T || (x == T && col < C); }
};

// Room for `more` candidates: where there is none, what is held is sorted and cut to K.
__device__ __forceinline__ void top_room(TopSmem& s, TopGate& g, int more) {
    if (g.held + more <= kTopCap) return;
    top_sort(s, g.held);
    if (g.held >= g.K) {
        g.held = g.K;
        g.T = key_value(s.buf[g.K - 1]);
        g.C = key_column(s.buf[g.K - 1]);
    }
    __syncwarp();
}

// The k-th logit of a vector.
__device__ __forceinline__ uint32_t pick_word(const uint4& r, int k) {
    return k & 2 ? (k & 1 ? r.w : r.z) : (k & 1 ? r.y : r.x);
}
template <typename T>
__device__ __forceinline__ float pick(const uint4& r, int k) {
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(pick_word(r, k));
    } else {
        const float2 v = Vec<T>::unpack_pair(pick_word(r, k >> 1));
        return k & 1 ? v.y : v.x;
    }
}
// The logits of each lane's vector (have: it has one) that the gate lets in; col: the
// column of its first.  equal: those equal to T alone.
template <typename T>
__device__ __forceinline__ void top_push(TopSmem& s, TopGate& g, bool have, const uint4& raw, uint32_t col,
                                         bool equal = false) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems;
    const int lane = threadIdx.x & 31;
    unsigned ok = 0;
    if (__any_sync(kFull, have && VT::vmax(raw) >= g.T)) {
        float x[VEC];
        VT::unpack(raw, x);
#pragma unroll
        for (int k = 0; k < VEC; ++k) ok |= x[k] >= g.T && !(equal && x[k] > g.T) ? 1u << k : 0u;
        if (!have) ok = 0;
    }
    while (__any_sync(kFull, ok != 0u)) {
        bool in = false;
        uint64_t key = 0;
        if (ok) {
            const int k = __ffs(ok) - 1;
            const float x = pick<T>(raw, k);
            key = top_key(x, col + (uint32_t)k);
            in = g.takes(x, col + (uint32_t)k);
            ok &= ok - 1u;
        }
        const unsigned m = __ballot_sync(kFull, in);
        if (in) s.buf[g.held + __popc(m & ((1u << lane) - 1u))] = key;
        g.held += __popc(m);
    }
}
__device__ __forceinline__ void top_push_one(TopSmem& s, TopGate& g, bool ok, float x, uint32_t col) {
    const unsigned m = __ballot_sync(kFull, ok && g.takes(x, col));
    const int lane = threadIdx.x & 31;
    if ((m >> lane) & 1u) s.buf[g.held + __popc(m & ((1u << lane) - 1u))] = top_key(x, col);
    g.held += __popc(m);
}

__device__ __forceinline__ uint32_t head_of_eight(const uint16_t* heads, int k) {  // maxima in both halves
    const uint4 u = *reinterpret_cast<const uint4*>(heads + k);
    return __vmaxu2(__vmaxu2(u.x, u.y), __vmaxu2(u.z, u.w));
}
// Heads (of eight, or two, the maximum: fold) counted by their distance below `top` (those
// above it as none) in 128 bins of 2^shift: the bin in which the K-th lies, and in the
// upper half how many lie in it and above it.  128: in none.
static __device__ __noinline__ uint32_t head_bin(TopSmem& s, const uint16_t* heads, int n, int K, uint32_t top,
                                                 int shift, int fold) {
    const int lane = threadIdx.x & 31;
    const uint32_t span = 128u << shift;
    *reinterpret_cast<int4*>(s.bins + 4 * lane) = make_int4(0, 0, 0, 0);
    __syncwarp();
    auto bin = [&](uint32_t h) {
        const uint32_t d = h < top ? top - h : 0u;
        if (d < span && h) atomicAdd(&s.bins[d >> shift], 1);
    };
    if (fold == 8) {
#pragma unroll 1
        for (int k = lane * 8; k < n; k += 256) {
            const uint32_t v = head_of_eight(heads, k);
            bin(max(v & 0xffffu, v >> 16));
        }
    } else {
#pragma unroll 1
        for (int k = lane * 2; k < n; k += 64) {
            const uint32_t u = *reinterpret_cast<const uint32_t*>(heads + k);
            const uint32_t a = u & 0xffffu, c = u >> 16;
            bin(max(a, c));
            if (fold == 1) bin(min(a, c));
        }
    }
    __syncwarp();
    const int4 c = *reinterpret_cast<const int4*>(s.bins + 4 * lane);
    const int own = c.x + c.y + c.z + c.w;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += u;
    }
    __syncwarp();
    const unsigned there = __ballot_sync(kFull, sum >= K);
    if (there == 0u) return 128u;
    const int l = __ffs(there) - 1, before = sum - own;
    const int e0 = before + c.x, e1 = e0 + c.y, e2 = e1 + c.z;
    const int b = e0 >= K ? 0 : e1 >= K ? 1 : e2 >= K ? 2 : 3;
    const uint32_t said = (uint32_t)(4 * lane + b) | (uint32_t)(b == 0 ? e0 : b == 1 ? e1 : b == 2 ? e2 : sum) << 16;
    return __shfl_sync(kFull, said, l);
}

// The least head that is read again: at least K of the n heads reach it (0: fewer than K are
// not 0).  It is sought below the largest head, in wider bins where K lie further down.
// Of many heads for each of the K only the maximum of eight, or two, counts: few more than
// K reach that too.  Where many more than K do (equal heads: a mask, a constant row), the
// K-th itself is sought (many).
__device__ __forceinline__ uint32_t kth_head(TopSmem& s, const uint16_t* heads, int n, int K, bool& many) {
    const int lane = threadIdx.x & 31;
    many = false;
    uint32_t top = 0;
#pragma unroll 1
    for (int k = lane * 8; k < n; k += 256) top = __vmaxu2(top, head_of_eight(heads, k));
    top = __reduce_max_sync(kFull, max(top & 0xffffu, top >> 16));
    if (top == 0) return 0;
    if (K == 1) {
        many = true;  // the K-th itself
        return top;
    }
    if (n <= 32) {
        // a head a lane: its bits from the first
        const uint32_t h = lane < n ? heads[lane] : 0u;
        uint32_t kth = 0;
#pragma unroll 1
        for (uint32_t bit = 0x8000u; bit; bit >>= 1)
            if (__popc(__ballot_sync(kFull, h >= (kth | bit))) >= K) kth |= bit;
        many = true;
        return kth;
    }
    int fold = n >= 24 * K ? 8 : (n >= 6 * K ? 2 : 1);
    int shift = 1;
#pragma unroll 1
    for (;;) {
        const uint32_t said = head_bin(s, heads, n, K, top, shift, fold), b = said & 0xffffu;
        const int upto = (int)(said >> 16);
        if (b == 128u) {  // further down, or (a second time, without folding) nowhere
            if (shift == 9 && fold == 1) return 0;
            if (shift == 9) fold = 1;
            else shift += 4;
            continue;
        }
        if (!many && upto <= 2 * K + 16) {
            const uint32_t far = ((b + 1u) << shift) - 1u;  // the bin's far end
            return top > far ? top - far : 1u;
        }
        // what lies above the bin counts in the next, finer one's first bin
        const uint32_t near = b << shift;
        top = top > near ? top - near : 1u;
        if (many && shift == 0) return top;
        shift = !many ? shift : shift > 5 ? 5 : shift > 1 ? 1 : 0;
        if (!many && shift == 1) shift = 0;
        many = true;
        fold = 1;
    }
}

// How many heads reach `least`, 1 at least.
__device__ __forceinline__ int count_heads(const uint16_t* heads, int n, uint32_t least) {
    const uint32_t two = least | (least << 16);
    uint32_t sum = 0;
#pragma unroll 1
    for (int k = (threadIdx.x & 31) * 8; k < n; k += 256) {
        const uint4 u = *reinterpret_cast<const uint4*>(heads + k);
        sum += __vsetgeu2(u.x, two) + __vsetgeu2(u.y, two) + __vsetgeu2(u.z, two) + __vsetgeu2(u.w, two);
    }
    return __reduce_add_sync(kFull, (sum & 0xffffu) + (sum >> 16));
}

// The heads that reach `least` (1 at least), listed in place by their numbers: the list never
// reaches a head that has not been looked at.  How many there are.
__device__ __forceinline__ int list_heads(uint16_t* heads, int n, uint32_t least) {
    const int lane = threadIdx.x & 31;
    if (least == 0) least = 1;
    int listed = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += 256) {
        const int k = k0 + lane * 8;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (k < n) u = *reinterpret_cast<const uint4*>(heads + k);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        unsigned ok = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ok |= (w[i] & 0xffffu) >= least ? 1u << (2 * i) : 0u;
            ok |= (w[i] >> 16) >= least ? 2u << (2 * i) : 0u;
        }
#pragma unroll 1
        for (unsigned m; (m = __ballot_sync(kFull, ok != 0u)) != 0u; ok &= ok - 1u) {  // few: one of a lane's at a time
            if (ok) heads[listed + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(k + __ffs(ok) - 1);
            listed += __popc(m);
        }
        __syncwarp();
    }
    __syncwarp();
    return listed;
}

// The listed groups' vectors, 32 at a time and the next ones on their way.  wide: a group is
// eight vectors, else one.  equal: every vector from the
// first on, for logits equal to T alone, until `equal` of them are held (or K and all after
// them come behind those).  Most vectors of a listed group have no candidate: those that
// reach T are queued first and looked at when each lane has one (read twice, but a third
// of the instructions).
template <typename T>
__device__ __forceinline__ void top_take(TopSmem& s, TopGate& g, const uint16_t* list, int listed, bool wide,
                                         const uint4* body, int64_t nv, uint32_t col0, int equal) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems, AHEAD = 2;
    static_assert(kTileVecs == 8 * kMainThreads, "eight vectors of a tile a thread");
    const int lane = threadIdx.x & 31, per = wide ? 4 : 32, had = g.held;
    const int last = nv < 0x7fffffff ? (int)nv : 0x7fffffff;
    if (equal) listed = last;
    int* queue = s.bins;  // vectors
    int queued = 0;
    uint4 raw[AHEAD];
    int v[AHEAD];  // the vector, or -1
    auto fetch = [&](int b, uint4& to, int& vec) {
        const int e = b + (wide ? lane >> 3 : lane);
        vec = -1;
        if (e < listed) {
            int at = equal ? e : (int)list[e];
            if (wide) at = at * 8 + (lane & 7);
            if (at < last) {
                vec = at;
                to = __ldg(body + at);
            }
        }
    };
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) fetch(a * per, raw[a], v[a]);
    bool more = listed > 0;
#pragma unroll 1
    for (int b = 0; more || queued > 0; b += AHEAD * per) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const float most = VT::vmax(raw[a]);
            bool hit = v[a] >= 0 && most >= g.T;
            if (g.C != 0xffffffffu) hit = hit && g.takes(most, col0 + (uint32_t)(v[a] * VEC));  // many equals
            const unsigned m = __ballot_sync(kFull, hit);
            if (hit) queue[queued + __popc(m & ((1u << lane) - 1u))] = v[a];
            queued += __popc(m);
            fetch(b + (AHEAD + a) * per, raw[a], v[a]);
        }
        more = b + AHEAD * per < listed;
        __syncwarp();
        int at = 0;
#pragma unroll 1
        for (; queued - at >= 32 || (!more && queued > at); at += 32) {
            const int vec = at + lane < queued ? queue[at + lane] : -1;
            uint4 now = make_uint4(0, 0, 0, 0);
            if (vec >= 0) now = __ldg(body + vec);
            top_room(s, g, 32 * VEC);
            if (equal && (g.held >= had + equal || g.C != 0xffffffffu)) return;
            top_push<T>(s, g, vec >= 0, now, col0 + (uint32_t)(vec * VEC), equal != 0);
        }
        const int left = max(0, queued - at);  // fewer than 32
        const int keep = lane < left ? queue[at + lane] : 0;
        __syncwarp();
        if (lane < left) queue[lane] = keep;
        __syncwarp();
        queued = left;
    }
}

// The K largest of a row's (segment's) logits into the front of s.buf, in falling order;
// returns how many there are.  One warp.  body: its nv vectors in global memory, their
// first logit of column col0; heads: the groups' maxima, G of them (zeros up to a multiple
// of eight), overwritten.  xe, ce: the lane's element around the body, where has_edge.
template <typename T>
__device__ __forceinline__ int top_select(TopSmem& s, uint16_t* heads, int G, const uint4* body, int64_t nv,
                                          uint32_t col0, int K, bool has_edge, float xe, uint32_t ce) {
    using VT = Vec<T>;
    const int lane = threadIdx.x & 31;
    const bool brief = G < 2 * K && nv <= kTopHeads;  // too few groups: each vector is one
    if (brief) {
#pragma unroll 1
        for (int v = lane; v < (((int)nv + 255) & ~255); v += 32)
            heads[v] = (uint16_t)(v < nv ? Head<T>::of(VT::vmax(__ldg(body + v))) : 0u);
        G = (int)nv;
        __syncwarp();
    }
    bool many;
    const uint32_t kth = kth_head(s, heads, G, K, many);
    // Where the head says the value and many groups reach it, its equals are not all read.
    const bool exact = many && (Head<T>::exact || kth <= Head<T>::lowest) && count_heads(heads, G, kth) > 2 * K + 32;
    const int listed = list_heads(heads, G, exact ? kth + 1 : kth);
    const float T0 = kth <= Head<T>::lowest ? -INFINITY : Head<T>::value(kth);
    TopGate g(K, T0);
    top_push_one(s, g, has_edge, xe, ce);
    if (exact) g.C = 0;  // first what is above T
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        top_take<T>(s, g, heads, listed, !brief && pass == 0, body, nv, col0, pass ? K : 0);
        if (pass || !exact || g.T != T0) break;  // (T has risen where K are above T0)
        g.C = 0xffffffffu;
    }
    top_sort(s, g.held);
    return g.held < K ? g.held : K;
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
// The same answer in every lane.
__device__ __forceinline__ bool warp_wait(RowBars& b, uint64_t* bar, uint32_t ph) {
    return __all_sync(kFull, row_wait(b, bar, ph));
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
// First pass over a row's tiles by the main warps: the warp's statistics go to part, and
// with GM the maximum of each thread's vectors of a tile to heads.  A warp without a vector
// of a last tile passes it by; there is one body for every tile (a second one for half a tile cost
// more, beside the side warps' code in the instruction cache, than it saved).
template <typename T, int NV, bool ENT, bool GM>
__device__ __forceinline__ bool main_stats(RowBars& b, Turn& at, int stages, const unsigned char* ring, int q,
                                           int64_t nv, float L, uint16_t* heads) {
    constexpr int TILE = kMainThreads * NV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Stat st = stat_identity();
    for (; nv > 0; nv -= TILE) {
        const uint4* tile = reinterpret_cast<const uint4*>(ring + (size_t)at.s * TILE * 16);
        if (!warp_wait(b, &b.full[at.s], at.ph)) return false;
        const int left = nv < TILE ? (int)nv : TILE;
        float top = -INFINITY;
        if (left > warp * 32 * NV)
            top = stat_tile<T, NV, ENT>(st, tile, left, L, &b.empty[at.s]);
        else
            warp_arrive(&b.empty[at.s]);
        if constexpr (GM) {
            heads[tid] = (uint16_t)(tid * NV < left ? Head<T>::of(top) : 0u);  // 0: no vector
            heads += kMainThreads;
        }
        at.next(stages);
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
