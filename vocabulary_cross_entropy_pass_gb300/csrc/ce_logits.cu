// ce_logits.cu -- penalties, biases, a grammar's bit mask and the temperature
// on the logits, and the gradient through them.
//
// Per row, with c_j the number of times token j occurs in the answer so far
// (the history past its first prompt_length tokens), s_j whether it occurs in
// the history at all, b_j the summed biases given for it:
//   z_j = s_j ? (x_j > 0 ? x_j / rep : x_j rep) : x_j
//   y_j = (z_j - freq c_j - pres [c_j > 0] + b_j) / temp
//   out_j = allowed_j ? y_j : mask_value
// Backward: dx_j = allowed_j ? dy_j / temp * (s_j ? (x_j > 0 ? 1/rep : rep) : 1) : 0.
//
// Bound by HBM: each allowed logit is read once and each output written once.
// A CTA streams a run of one row's columns with nothing but the mask and the
// temperature applied; a 16-byte vector whose mask bits are all clear is
// written without being read.  (HBM is read in 128-byte lines: with one token of
// 64 allowed at random, two lines of three.)  The few columns that the history
// or the biases touch are written again after the stream has passed over them.
// Where they and their outputs come from:
//   few columns in all (a decoding step of a few rows, where latency counts): the
//           CTA itself reads the row's lists, with a count per column in shared
//           memory (integer atomics: any order gives the same counts; who
//           raises a column from zero lists it).
//   many    a kernel before it, a CTA per row: a bit per column, a scan of the
//           bits that gives each touched column its place in the row's table in
//           the workspace, then counts on the table's entries.  The stream's CTAs
//           find their part of the table ready, so the lists' chain of
//           dependent steps is not paid for in each of them, and read the
//           logits of its columns again while L2 still holds them (read by the
//           first kernel they came from HBM a second time, 64 bytes for each).
// Biases of one column are added in list order by one warp.
// bf16, 512 rows of 128000 columns: 40.6 us without lists and mask (6.5 TB/s, 0.97
// of the copy rate), 41.5 us under masks of which one row of four is free (235 MB in
// 128-byte lines: 35 us), 77 us with histories of 4096 and 64 biases as well (17.1 us
// of it the list kernel, which its shared-memory atomics and scans keep busy).
#include "ce_device.cuh"
#include "ce_internal.h"
#include "ce_logits_plan.h"
#include "ce_pack.cuh"
#include "ce_span.cuh"

namespace gbce {
namespace {

constexpr int kThreads = kLogitThreads;
constexpr uint32_t kBiased = 0x40000000u;  // a bias is given for the column
constexpr uint32_t kSeen = 0x80000000u;    // the token occurs; the low 30 bits count it in the answer

struct LogitArgs : LogitSizes {
    const char* x;         // logits (backward: read where the history touches them)
    const char* g;         // backward: the gradient of the outputs, else NULL
    char* out;
    int64_t xs0, xs1, gs0, gs1, os0, os1;  // in elements
    int64_t dim1;
    int listed;            // the history or the biases touch columns
    int in_place;
    uint2* table;          // [N][parts][entries] touched (column in its run, count and flags), by column; or NULL
    float* tbias;          // [N][parts][entries] their summed biases
    uint32_t* start;       // [N][runs][2] a run's first and last + 1 entry of its part's table
    const int64_t* hist;
    int64_t hist_stride;
    const int64_t* hist_len;
    const int64_t* prompt_len;
    const float* rep;
    const float* freq;
    const float* pres;
    const int64_t* btok;
    const float* bval;
    int64_t btok_stride, bval_stride;
    const uint32_t* mask;
    int64_t mask_stride;
    const float* temp;
    float mask_value;
};

// v / d, inv being 1 / d rounded.  In 16 bits a product with it: at most 2^-23 more
// before a rounding of 2^-9 or 2^-12.  Outputs in float32 get the quotient rounded
// once: v - q d is exact in one fused step, and q plus inv times that, taken twice,
// is the rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990).  A zero keeps
// its sign, an infinity its product.  (The divide operator in its place: 512 rows of
// 128000 under masks 82 -> 91 us, by the registers its rare branch takes.)
template <typename T>
__device__ __forceinline__ float quotient(float v, float d, float inv) {
    const float p = v * inv;
    if (sizeof(T) != 4) return p;
    float q = fmaf(fmaf(-p, d, v), inv, p);
    const float r = fmaf(-q, d, v);
    q = fmaf(r, inv, q);
    return p != 0.f && fabsf(r) <= 3.4e38f ? q : p;
}

// One column's value (or gradient).
struct RowScalars {
    float rep, inv_rep, freq, pres;
};

template <typename T, bool BWD>
__device__ __forceinline__ float special(float v, float x, uint32_t word, float bias, const RowScalars& r) {
    const bool seen = (word & ~kBiased) != 0u;
    if (BWD) return seen ? (x > 0.f ? quotient<T>(v, r.rep, r.inv_rep) : v * r.rep) : v;
    float z = seen ? (x > 0.f ? quotient<T>(x, r.rep, r.inv_rep) : x * r.rep) : x;
    const uint32_t c = word & ~(kSeen | kBiased);
    if (c) z = fmaf(-r.freq, (float)c, z) - r.pres;
    return z + bias;
}

// One row's pointers at column c0.
struct RowPtrs {
    const char* x;
    const char* src;       // what is streamed: the logits, or the outputs' gradient
    char* out;
    const uint32_t* mask;
    float temp, inv_temp;
};
template <int ES, bool BWD>
__device__ __forceinline__ RowPtrs row_ptrs(const LogitArgs& p, int64_t row, int64_t c0) {
    int64_t i = 0, j = row;
    if (p.dim1 < p.N) {
        i = row / p.dim1;
        j = row - i * p.dim1;
    }
    RowPtrs r;
    r.x = p.x + (i * p.xs0 + j * p.xs1 + c0) * ES;
    r.src = BWD ? p.g + (i * p.gs0 + j * p.gs1 + c0) * ES : r.x;
    r.out = p.out + (i * p.os0 + j * p.os1 + c0) * ES;
    r.mask = p.mask ? p.mask + row * p.mask_stride + c0 / 32 : nullptr;
    r.temp = p.temp ? __ldg(p.temp + row) : 1.f;
    r.inv_temp = 1.f / r.temp;
    return r;
}
__device__ __forceinline__ bool allowed(const uint32_t* mask, int c) {
    return !mask || ((__ldg(mask + (c >> 5)) >> (c & 31)) & 1u);
}

__device__ __forceinline__ RowScalars row_scalars(const LogitArgs& p, int64_t row) {
    RowScalars rs;
    rs.rep = p.rep ? __ldg(p.rep + row) : 1.f;
    rs.inv_rep = 1.f / rs.rep;
    rs.freq = p.freq ? __ldg(p.freq + row) : 0.f;
    rs.pres = p.pres ? __ldg(p.pres + row) : 0.f;
    return rs;
}

// A token's column in the run that starts at c0, or at least 2^31.
// (c0 < 2^31: a token's upper half is zero or the token lies nowhere.)
__device__ __forceinline__ uint32_t column_of(int64_t t, int64_t c0) {
    const uint32_t lo = (uint32_t)t, hi = (uint32_t)((uint64_t)t >> 32);
    return hi == 0u && lo >= (uint32_t)c0 ? lo - (uint32_t)c0 : 0xffffffffu;
}

// The listed columns of this run: col[0 .. returned count), each one's output in
// cnt[column].  Shared memory: cnt[cols], bias[cols] (with biases), col[cols].
struct Listed {
    uint32_t* cnt;
    uint16_t* col;
    int n;
};
template <typename T, bool BWD>
__device__ __forceinline__ Listed find_listed(const LogitArgs& p, const RowPtrs& rp, int64_t row, int64_t c0, int n,
                                              uint32_t* sm) {
    using VT = Vec<T>;
    constexpr int ES = sizeof(T);
    __shared__ int nl;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t* cnt = sm;
    float* bias = reinterpret_cast<float*>(cnt + p.cols);
    uint16_t* col = reinterpret_cast<uint16_t*>(bias + (!BWD && p.bias_max > 0 ? p.cols : 0));

    int64_t len = 0, prompt = 0;
    const int64_t* h = p.hist + row * p.hist_stride;
    if (p.hist_max > 0) {
        len = p.hist_len ? __ldg(p.hist_len + row) : p.hist_max;
        len = len < 0 ? 0 : (len > p.hist_max ? p.hist_max : len);
        prompt = p.prompt_len ? __ldg(p.prompt_len + row) : 0;
    }
    for (int k = tid; k < p.cols / 4; k += kThreads) reinterpret_cast<uint4*>(cnt)[k] = make_uint4(0, 0, 0, 0);
    if (!BWD && p.bias_max > 0)
        for (int k = tid; k < p.cols / 4; k += kThreads)
            reinterpret_cast<float4*>(bias)[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tid == 0) nl = 0;
    __syncthreads();
    // the one that finds a column untouched lists it
    auto hit = [&](uint32_t c, uint32_t bit) {
        const uint32_t old = bit ? atomicOr(&cnt[c], bit) : atomicAdd(&cnt[c], 1u);
        if (old == 0u) col[atomicAdd(&nl, 1)] = (uint16_t)c;
    };
    for (int64_t k0 = 0; k0 < len; k0 += kThreads * 4) {
        int64_t t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t k = k0 + u * kThreads + tid;
            t[u] = k < len ? __ldg(h + k) : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t c = column_of(t[u], c0);
            if (c < (uint32_t)n) hit(c, k0 + u * kThreads + tid < prompt ? kSeen : 0u);
        }
    }
    if (!BWD && p.bias_max > 0 && warp == kThreads / 32 - 1) {
        const int64_t* bt = p.btok + row * p.btok_stride;
        const float* bv = p.bval + row * p.bval_stride;
        for (int64_t k0 = 0; k0 < p.bias_max; k0 += 32) {
            const int64_t k = k0 + lane;
            const uint32_t c = k < p.bias_max ? column_of(__ldg(bt + k), c0) : 0xffffffffu;
            const bool in = c < (uint32_t)n;
            if (!__any_sync(kFull, in)) continue;
            const float b = in ? __ldg(bv + k) : 0.f;
            const unsigned peers = __match_any_sync(kFull, in ? c : 0xffffffffu);
            const bool lead = in && lane == __ffs(peers) - 1;
            // the leader adds its column's biases in list order
            unsigned todo = lead ? peers : 0u;
            float sum = lead ? bias[c] : 0.f;
            while (__any_sync(kFull, todo != 0u)) {
                const float v = __shfl_sync(kFull, b, todo ? __ffs(todo) - 1 : 0);
                if (todo) {
                    sum += v;
                    todo &= todo - 1;
                }
            }
            if (lead) {
                bias[c] = sum;
                hit(c, kBiased);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    const RowScalars rs = row_scalars(p, row);
    const int m = nl;
    for (int e = tid; e < m; e += kThreads) {
        const int c = col[e];
        const float xv = VT::load1(rp.x + c * ES);
        const float v = BWD ? VT::load1(rp.src + c * ES) : xv;
        float o = BWD ? 0.f : p.mask_value;
        if (allowed(rp.mask, c))
            o = quotient<T>(special<T, BWD>(v, xv, cnt[c], (!BWD && p.bias_max > 0) ? bias[c] : 0.f, rs), rp.temp,
                            rp.inv_temp);
        cnt[c] = __float_as_uint(o);
    }
    return Listed{cnt, col, m};
}

// The stream over n columns, by the output's 16-byte vectors, with the elements
// around them one per thread.  SHIFT: the inputs lie at another offset from 16
// bytes than the outputs.  behind(0) and behind(1) are called once each, after
// the first and the second batch of loads are on their way.
template <typename T, bool BWD, bool SHIFT, bool MASK, typename F>
__device__ __forceinline__ void stream_run(const LogitArgs& p, const RowPtrs& rp, int64_t c0, int n, const Span16& sp,
                                           F behind) {
    using VT = Vec<T>;
    constexpr int VEC = VT::kElems;
    constexpr int ES = sizeof(T);
    constexpr int TH = kThreads;
    // vectors per thread and batch: with a mask, two dependent loads each and few
    // bytes, more CTAs count for more (512 x 128000 with lists 83 -> 77 us, 4096
    // x 50257 205 -> 179 us; without a mask 66 -> 72 us)
    constexpr int U = MASK ? 2 : 4;
    constexpr uint32_t ALL = (1u << VEC) - 1u;
    const int tid = threadIdx.x;
    const float blocked = BWD ? 0.f : p.mask_value;
    const int nv = (int)sp.nv, off = (int)sp.h1;
    {
        const int e = (int)span16_edge(sp, 0, n, TH - 1 - tid);
        if (e >= 0)
            VT::store1(rp.out + e * ES,
                       allowed(rp.mask, e) ? quotient<T>(VT::load1(rp.src + e * ES), rp.temp, rp.inv_temp) : blocked);
    }
    const uint32_t ph = (uint32_t)(reinterpret_cast<uintptr_t>(rp.src + off * ES) & 15u);
    const uint4* in = reinterpret_cast<const uint4*>(rp.src + off * ES - ph);  // on the 16-byte grid
    uint4* to = reinterpret_cast<uint4*>(rp.out + off * ES);
    // a shifted vector reads two that must lie inside the row: not before its
    // first element, not past its last
    const int safe0 = SHIFT && c0 + off < (int64_t)(ph / ES) ? 1 : 0;
    const int64_t room = ((p.V - c0 - off) * ES + ph) / 16 - 1;
    const int safe1 = (int)(room < nv ? room : nv);
    auto load = [&](int v) -> uint4 {
        if constexpr (!SHIFT) {
            return __ldcs(in + v);
        } else {
            if (v >= safe0 && v < safe1) return shift_bytes(__ldg(in + v), __ldg(in + v + 1), ph);
            float f[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] = VT::load1(rp.src + (off + v * VEC + k) * ES);
            return VT::pack(f);
        }
    };
    const uint8_t* mb = reinterpret_cast<const uint8_t*>(rp.mask);  // bit c % 8 of byte c / 8
    auto bits_of = [&](int v) -> uint32_t {
        const int c = off + v * VEC, s = c & 7;
        uint32_t m = __ldg(mb + (c >> 3));
        if (s + VEC > 8) m |= (uint32_t)__ldg(mb + (c >> 3) + 1) << 8;
        return (m >> s) & ALL;
    };
    const float2 T2 = make_float2(rp.inv_temp, rp.inv_temp);
    int step = 0;
    for (int v0 = tid; v0 < nv; v0 += TH * U) {
        uint4 raw[U];
        uint32_t on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u * TH;
            on[u] = v >= nv ? 0u : (MASK ? bits_of(v) : ALL);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (on[u]) raw[u] = load(v0 + u * TH);
        if (step < 2) behind(step++);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v0 + u * TH >= nv) continue;
            float2 f[VEC / 2];
            VT::unpack2(raw[u], f);
#pragma unroll
            for (int k = 0; k < VEC / 2; ++k) {
                if (ES == 4) f[k] = make_float2(quotient<T>(f[k].x, rp.temp, rp.inv_temp), quotient<T>(f[k].y, rp.temp, rp.inv_temp));
                else f[k] = __fmul2_rn(f[k], T2);
                if (MASK) {
                    f[k].x = (on[u] >> (2 * k)) & 1u ? f[k].x : blocked;
                    f[k].y = (on[u] >> (2 * k + 1)) & 1u ? f[k].y : blocked;
                }
            }
            stg128_stream(to + v0 + u * TH, VT::pack2(f));
        }
    }
    while (step < 2) behind(step++);
}

template <typename T, bool BWD, bool MASK>
__global__ void __launch_bounds__(kThreads, MASK ? 8 : 6) ce_logits_kernel(const __grid_constant__ LogitArgs p) {
    using VT = Vec<T>;
    constexpr int ES = sizeof(T);
    extern __shared__ __align__(16) uint32_t sm[];
    const int run = blockIdx.x, tid = threadIdx.x;
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (row >= p.N) return;
    const int64_t c0 = (int64_t)run * p.cols;
    const int n = (int)min((int64_t)p.cols, p.V - c0);
    const RowPtrs rp = row_ptrs<ES, BWD>(p, row, c0);
    Listed l = {};
    uint2 range = make_uint2(0u, 0u);  // this run's entries of the table
    RowScalars rs = {};
    if (p.table) {
        griddep_wait();
        range = __ldcg(reinterpret_cast<const uint2*>(p.start) + row * p.runs + run);
        rs = row_scalars(p, row);
    } else if (p.listed) {
        l = find_listed<T, BWD>(p, rp, row, c0, n, sm);
        if (p.in_place) __syncthreads();
    }
    const int64_t t0 = (row * p.parts + run / p.part_runs) * p.entries;
    auto bias_of = [&](uint32_t e, uint32_t word) {
        return !BWD && (word & kBiased) ? __ldcg(p.tbias + t0 + e) : 0.f;
    };
    auto output = [&](uint32_t e, int c, uint32_t word) {
        if (!allowed(rp.mask, c)) return BWD ? 0.f : p.mask_value;
        const float xv = VT::load1(rp.x + c * ES);
        const float v = BWD ? VT::load1(rp.src + c * ES) : xv;
        return quotient<T>(special<T, BWD>(v, xv, word, bias_of(e, word), rs), rp.temp, rp.inv_temp);
    };
    if (p.in_place && range.x < range.y) {
        // what the logits give is taken before the stream replaces them
        for (uint32_t e = range.x + tid; e < range.y; e += kThreads) {
            const uint2 t = __ldcg(p.table + t0 + e);
            p.table[t0 + e].y = __float_as_uint(output(e, (int)t.x, t.y));
        }
        __syncthreads();
    }
    // a thread's first entry, then what its output needs, fetched behind the
    // stream's loads
    uint2 mine = make_uint2(0u, 0u);
    float xv = 0.f, v = 0.f, bv = 0.f;
    bool ok = false;
    const bool have = range.x + tid < range.y;
    auto gather = [&](int c) {
        xv = VT::load1(rp.x + c * ES);
        v = BWD ? VT::load1(rp.src + c * ES) : xv;
    };
    auto fetch = [&](int step) {
        if (!have) return;
        if (step == 0) {
            mine = __ldcg(p.table + t0 + range.x + tid);
        } else if (!p.in_place) {
            const int c = (int)mine.x;
            ok = allowed(rp.mask, c);
            bv = bias_of(range.x + tid, mine.y);
            if (!MASK) gather(c);
        }
    };
    const Span16 sp = span16<ES>(rp.out, 0, n);
    if (((reinterpret_cast<uintptr_t>(rp.src) ^ reinterpret_cast<uintptr_t>(rp.out)) & 15u) == 0)
        stream_run<T, BWD, false, MASK>(p, rp, c0, n, sp, fetch);
    else
        stream_run<T, BWD, true, MASK>(p, rp, c0, n, sp, fetch);
    if (range.x < range.y) {
        if (MASK && have && ok && !p.in_place) gather((int)mine.x);  // a forbidden logit's line may never have been read
        __syncthreads();
        if (have) {
            const float o = p.in_place ? __uint_as_float(mine.y)
                            : ok       ? quotient<T>(special<T, BWD>(v, xv, mine.y, bv, rs), rp.temp, rp.inv_temp)
                                       : (BWD ? 0.f : p.mask_value);
            VT::store1(rp.out + (int)mine.x * ES, o);
        }
        for (uint32_t e = range.x + tid + kThreads; e < range.y; e += kThreads) {
            const uint2 t = __ldcg(p.table + t0 + e);
            const int c = (int)t.x;
            VT::store1(rp.out + c * ES, p.in_place ? __uint_as_float(t.y) : output(e, c, t.y));
        }
    } else if (l.n > 0) {
        __syncthreads();
        for (int e = tid; e < l.n; e += kThreads)
            VT::store1(rp.out + l.col[e] * ES, __uint_as_float(l.cnt[l.col[e]]));
    }
}

// The table of one part of a row.  Shared memory: bits[words] (a whole number of
// 16-byte vectors), cnt[entries], keys[slots] and sums[sums] of the biased entries
// (without slots a sum for each entry), first[words] (entries before each word:
// 16 bits, a part has at most 65535), col[entries] (columns in their runs: 16 bits,
// a run is a power of two of at most 65536).
template <int TH, int U>
__global__ void __launch_bounds__(TH, 2048 / TH) ce_logits_lists_kernel(const __grid_constant__ LogitArgs p) {
    extern __shared__ __align__(16) uint32_t sm[];
    __shared__ uint32_t wsum[TH / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (row >= p.N) return;
    const int64_t cols = (int64_t)p.part_runs * p.cols, c0 = blockIdx.x * cols;
    const int n = (int)min(cols, p.V - c0);
    const int words = (int)(cols / 32);
    uint32_t* bits = sm;
    uint32_t* cnt = bits + words;
    uint32_t* keys = cnt + p.entries;
    float* sums = reinterpret_cast<float*>(keys + p.slots);
    uint16_t* first = reinterpret_cast<uint16_t*>(sums + p.sums);
    uint16_t* col = first + words;
    const uint32_t in_run = (uint32_t)p.cols - 1;
    const int64_t t0 = (row * p.parts + blockIdx.x) * p.entries;
    uint2* table = p.table + t0;
    const int64_t* h = p.hist + row * p.hist_stride;
    const int64_t* bt = p.btok + row * p.btok_stride;
    const float* bv = p.bval + row * p.bval_stride;

    const int hist_max = (int)p.hist_max;
    uint32_t tc[U];  // this thread's first tokens, as columns of the part
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k = u * TH + tid;
        tc[u] = k < hist_max ? column_of(__ldg(h + k), c0) : 0xffffffffu;
    }
    int len = 0, prompt = 0;
    if (hist_max > 0) {
        const int64_t l = p.hist_len ? __ldg(p.hist_len + row) : hist_max;
        const int64_t q = p.prompt_len ? __ldg(p.prompt_len + row) : 0;
        len = l < 0 ? 0 : (l > hist_max ? hist_max : (int)l);
        prompt = q < 0 ? 0 : (q > hist_max ? hist_max : (int)q);
    }
    for (int k = tid; k < words / 4; k += TH) reinterpret_cast<uint4*>(bits)[k] = make_uint4(0, 0, 0, 0);
    if (p.bias_max > 0)
        for (int k = tid; k < p.slots; k += TH) {
            keys[k] = 0xffffffffu;
            sums[k] = 0.f;
        }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u * TH + tid >= len) tc[u] = 0xffffffffu;
    __syncthreads();
    auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (tc[u] < (uint32_t)n) f(tc[u], u * TH + tid < prompt);
        for (int k0 = U * TH; k0 < len; k0 += TH * 4) {
            uint32_t c[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u * TH + tid;
                c[u] = k < len ? column_of(__ldg(h + k), c0) : 0xffffffffu;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c[u] < (uint32_t)n) f(c[u], k0 + u * TH + tid < prompt);
        }
    };
    each([&](uint32_t c, bool) { atomicOr(&bits[c >> 5], 1u << (c & 31)); });
    for (int64_t k = tid; k < p.bias_max; k += TH) {
        const uint32_t c = column_of(__ldg(bt + k), c0);
        if (c < (uint32_t)n) atomicOr(&bits[c >> 5], 1u << (c & 31));
    }
    __syncthreads();
    // entries before each word: a thread's run of words, then over the threads
    const int per = (words / 4 + TH - 1) / TH * 4;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    uint32_t own = 0;
    for (int k = w0; k < w1; k += 4) {
        const uint4 b = *reinterpret_cast<const uint4*>(bits + k);
        own += __popc(b.x) + __popc(b.y) + __popc(b.z) + __popc(b.w);
    }
    uint32_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    uint32_t ws = lane < TH / 32 ? wsum[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, ws, o);
        if (lane >= o) ws += u;
    }
    const int ne = (int)__shfl_sync(kFull, ws, TH / 32 - 1);
    uint32_t before = __shfl_sync(kFull, ws, warp == 0 ? 0 : warp - 1);
    before = (warp == 0 ? 0u : before) + inc - own;
    for (int k = w0; k < w1; k += 4) {
        const uint4 b = *reinterpret_cast<const uint4*>(bits + k);
        ushort4 f;
        f.x = (unsigned short)before;
        f.y = (unsigned short)(before += __popc(b.x));
        f.z = (unsigned short)(before += __popc(b.y));
        f.w = (unsigned short)(before += __popc(b.z));
        before += __popc(b.w);
        *reinterpret_cast<ushort4*>(first + k) = f;
    }
    for (int k = tid; k < ne; k += TH) {
        cnt[k] = 0u;
        if (p.bias_max > 0 && p.slots == 0) sums[k] = 0.f;
    }
    __syncthreads();
    // where each run's entries are
    const int r0 = blockIdx.x * p.part_runs;
    for (int k = tid; k < p.part_runs && r0 + k < p.runs; k += TH) {
        const uint32_t a = first[k * (p.cols / 32)];
        const uint32_t b = r0 + k + 1 < p.runs && k + 1 < p.part_runs ? first[(k + 1) * (p.cols / 32)] : (uint32_t)ne;
        reinterpret_cast<uint2*>(p.start)[row * p.runs + r0 + k] = make_uint2(a, b);
    }
    // counts; whoever raises an entry from zero names its column
    auto place = [&](uint32_t c) { return first[c >> 5] + __popc(bits[c >> 5] & ((1u << (c & 31)) - 1u)); };
    each([&](uint32_t c, bool in_prompt) {
        const uint32_t e = place(c);
        const uint32_t old = in_prompt ? atomicOr(&cnt[e], kSeen) : atomicAdd(&cnt[e], 1u);
        if (old == 0u) col[e] = (uint16_t)(c & in_run);
    });
    if (p.bias_max > 0 && warp == TH / 32 - 1) {
        for (int64_t k0 = 0; k0 < p.bias_max; k0 += 32) {
            const int64_t k = k0 + lane;
            const uint32_t c = k < p.bias_max ? column_of(__ldg(bt + k), c0) : 0xffffffffu;
            const float b = k < p.bias_max ? __ldg(bv + k) : 0.f;
            const bool in = c < (uint32_t)n;
            if (!__any_sync(kFull, in)) continue;
            const uint32_t e = in ? place(c) : 0xffffffffu;
            const unsigned peers = __match_any_sync(kFull, e);
            const bool lead = in && lane == __ffs(peers) - 1;
            uint32_t slot = 0;
            if (lead && p.slots == 0) {
                slot = e;
            } else if (lead) {  // the entry's slot, a new one for its first bias
                slot = (e * 2654435761u) & (p.slots - 1);
                for (;;) {
                    const uint32_t was = atomicCAS(&keys[slot], 0xffffffffu, e);
                    if (was == 0xffffffffu || was == e) break;
                    slot = (slot + 1) & (p.slots - 1);
                }
            }
            // the leader adds its column's biases in list order
            unsigned todo = lead ? peers : 0u;
            float sum = lead ? sums[slot] : 0.f;
            while (__any_sync(kFull, todo != 0u)) {
                const float v = __shfl_sync(kFull, b, todo ? __ffs(todo) - 1 : 0);
                if (todo) {
                    sum += v;
                    todo &= todo - 1;
                }
            }
            if (lead) {
                sums[slot] = sum;
                if (atomicOr(&cnt[e], kBiased) == 0u) col[e] = (uint16_t)(c & in_run);
            }
            __syncwarp();
        }
    }
    griddep_launch_dependents();  // earlier the waiting stream takes the place of lists not yet begun
    __syncthreads();
    for (int e = tid; e < ne; e += TH) {
        table[e] = make_uint2(col[e], cnt[e]);
        if (p.bias_max > 0 && p.slots == 0 && (cnt[e] & kBiased)) p.tbias[t0 + e] = sums[e];
    }
    if (p.bias_max > 0)
        for (int k = tid; k < p.slots; k += TH)
            if (keys[k] != 0xffffffffu) p.tbias[t0 + keys[k]] = sums[k];
}

template <typename T, bool BWD>
cudaError_t launch_logits_t(const LogitArgs& a, cudaStream_t s) {
    cudaError_t e;
    auto allow = [](auto* k, size_t smem) { return allow_smem(reinterpret_cast<const void*>(k), smem); };
    const int64_t rows = a.N < 65535 ? a.N : 65535;
    const unsigned deep = (unsigned)((a.N + rows - 1) / rows);
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    if (a.table) {
        const size_t smem = list_bytes(a);
        // short lists: small CTAs, more rows at a time
        const bool brief = a.hist_max + a.bias_max <= 512;
        auto* k = brief ? ce_logits_lists_kernel<128, 4> : ce_logits_lists_kernel<512, 8>;
        if ((e = allow(k, smem)) != cudaSuccess) return e;
        k<<<dim3((unsigned)a.parts, (unsigned)rows, deep), brief ? 128 : 512, smem, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        set_pdl_attr(at);
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    cfg.gridDim = dim3((unsigned)a.runs, (unsigned)rows, deep);
    cfg.blockDim = dim3(kThreads);
    // the CTA's own counts, biases and list
    if (a.listed && !a.table) cfg.dynamicSmemBytes = (size_t)a.cols * (a.bias_max > 0 ? 10 : 6);
    auto* k = a.mask ? ce_logits_kernel<T, BWD, true> : ce_logits_kernel<T, BWD, false>;
    if ((e = allow(k, cfg.dynamicSmemBytes)) != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <bool BWD>
cudaError_t launch_logits(const LogitArgs& a, int dtype, cudaStream_t s) {
    if (dtype == CE_F32) return launch_logits_t<float, BWD>(a, s);
    if (dtype == CE_BF16) return launch_logits_t<__nv_bfloat16, BWD>(a, s);
    return launch_logits_t<__half, BWD>(a, s);
}

// The runs' entries, the tables, the biases.
size_t start_bytes(const LogitArgs& a) { return align_up((size_t)a.N * a.runs * 8, 256); }
size_t table_bytes(const LogitArgs& a) { return align_up((size_t)a.N * a.parts * a.entries * 8, 256); }
size_t logits_workspace(const LogitArgs& a) {
    return start_bytes(a) + table_bytes(a) + (a.bias_max > 0 ? table_bytes(a) / 2 : 0);
}

}  // namespace

bool rows_apart(int64_t d0, int64_t d1, int64_t V, const int64_t* s) {
    int64_t in_s = s[1], in_n = d1, out_s = s[0], out_n = d0;
    if (in_n <= 1 || (out_n > 1 && s[0] < s[1])) {
        in_s = s[0]; in_n = d0; out_s = s[1]; out_n = d1;
    }
    if (in_n > 1 && in_s < V) return false;
    if (out_n > 1 && out_s < (in_n > 1 ? in_s * in_n : V)) return false;
    return true;
}

namespace {

ce_status logits_common(const void* grad, const int64_t* grad_strides, const void* logits, ce_dtype dtype,
                        int64_t dim0, int64_t dim1, int64_t V, const int64_t* strides,
                        const ce_logits_params* q, void* out, const int64_t* out_strides, bool bwd, void* workspace,
                        size_t workspace_bytes, cudaStream_t s) {
    if (dtype < CE_F32 || dtype > CE_F16) return CE_ERR_UNSUPPORTED_DTYPE;
    if (!strides || !out_strides || !q || (bwd && !grad_strides)) return CE_ERR_INVALID_ARG;
    if (dim0 < 0 || dim1 < 0 || dim0 > 0x7fffffffLL || dim1 > 0x7fffffffLL || V < 1 || V > 0x7fffffffLL)
        return CE_ERR_INVALID_ARG;
    const int64_t N = dim0 * dim1;
    for (int k = 0; k < 2; ++k)
        if (q->reserved[k] != 0) return CE_ERR_INVALID_ARG;
    if (q->history_max < 0 || q->bias_max < 0 || q->history_max >= 0x40000000LL || q->bias_max > 0x40000000LL)
        return CE_ERR_INVALID_ARG;
    if (N > 0) {
        if (!logits || !out || (bwd && !grad)) return CE_ERR_INVALID_ARG;
        const uintptr_t all = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out) |
                              reinterpret_cast<uintptr_t>(bwd ? grad : out);
        if (all % elem_size(dtype)) return CE_ERR_INVALID_ARG;
        if (q->history_max > 0 && !q->history) return CE_ERR_INVALID_ARG;
        if (q->bias_max > 0 && (!q->bias_tokens || !q->bias_values)) return CE_ERR_INVALID_ARG;
        if (strides[2] != 1 || strides[0] < 0 || strides[1] < 0) return CE_ERR_BAD_STRIDE;
        if (bwd && (grad_strides[2] != 1 || grad_strides[0] < 0 || grad_strides[1] < 0)) return CE_ERR_BAD_STRIDE;
        if (out_strides[2] != 1 || out_strides[0] < 0 || out_strides[1] < 0) return CE_ERR_BAD_STRIDE;
        if (!rows_apart(dim0, dim1, V, out_strides)) return CE_ERR_BAD_STRIDE;
        if (q->history_stride < 0 || q->bias_tokens_stride < 0 || q->bias_values_stride < 0 || q->mask_stride < 0)
            return CE_ERR_BAD_STRIDE;
        if (q->mask && q->mask_stride != 0 && q->mask_stride < (V + 31) / 32) return CE_ERR_BAD_STRIDE;
        const int64_t* in_s = bwd ? grad_strides : strides;
        if (out == (bwd ? grad : logits) && (out_strides[0] != in_s[0] || out_strides[1] != in_s[1]))
            return CE_ERR_BAD_STRIDE;  // in place means the same strides
        if (bwd && out == logits) return CE_ERR_INVALID_ARG;
    }
    if (N == 0) return CE_OK;
    LogitArgs a = {};
    a.x = static_cast<const char*>(logits);
    a.g = static_cast<const char*>(grad);
    a.out = static_cast<char*>(out);
    a.xs0 = strides[0];
    a.xs1 = strides[1];
    a.gs0 = bwd ? grad_strides[0] : 0;
    a.gs1 = bwd ? grad_strides[1] : 0;
    a.os0 = out_strides[0];
    a.os1 = out_strides[1];
    a.dim1 = dim1;
    a.N = N;
    a.V = V;
    a.hist = q->history;
    a.hist_stride = q->history_stride;
    a.hist_max = q->history_max;
    a.hist_len = q->history_lengths;
    a.prompt_len = q->prompt_lengths;
    a.rep = q->repetition_penalty;
    a.freq = q->frequency_penalty;
    a.pres = q->presence_penalty;
    a.btok = q->bias_tokens;
    a.bval = q->bias_values;
    a.btok_stride = q->bias_tokens_stride;
    a.bval_stride = q->bias_values_stride;
    a.bias_max = q->bias_max;
    a.mask = reinterpret_cast<const uint32_t*>(q->mask);
    a.mask_stride = q->mask_stride;
    a.temp = q->temperature;
    a.mask_value = q->mask_value;
    a.in_place = out == (bwd ? grad : logits);
    // the plan (and so the workspace) goes by the lists' sizes alone; then what
    // nothing looks at is left out: a history without a penalty, and for the
    // gradient all but the repetition penalty
    if (N > 65535LL * 65535) return CE_ERR_INVALID_ARG;
    const bool tables = plan_logits(a, elem_size(dtype));
    a.table = nullptr;
    a.start = nullptr;
    a.tbias = nullptr;
    if (tables) {
        if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return CE_ERR_INVALID_ARG;
        if (workspace_bytes < logits_workspace(a)) return CE_ERR_WORKSPACE_TOO_SMALL;
        char* w = static_cast<char*>(workspace);
        a.start = reinterpret_cast<uint32_t*>(w);
        a.table = reinterpret_cast<uint2*>(w + start_bytes(a));
        a.tbias = reinterpret_cast<float*>(w + start_bytes(a) + table_bytes(a));
    }
    if (bwd) a.bias_max = 0;
    if (bwd ? !a.rep : !(a.rep || a.freq || a.pres)) a.hist_max = 0;
    a.listed = a.hist_max + a.bias_max > 0;
    if (!a.listed) a.table = nullptr;
    cudaError_t e = bwd ? launch_logits<true>(a, dtype, s) : launch_logits<false>(a, dtype, s);
    return e == cudaSuccess ? CE_OK : launch_failed();
}

}  // namespace
}  // namespace gbce

extern "C" size_t ce_logits_workspace_bytes(int64_t N, int64_t V, ce_dtype dtype, int64_t history_max,
                                            int64_t bias_max) {
    using namespace gbce;
    if (dtype < CE_F32 || dtype > CE_F16 || N < 0 || N > 65535LL * 65535 || V < 1 || V > 0x7fffffffLL ||
        history_max < 0 || bias_max < 0 || history_max > 0x40000000LL || bias_max > 0x40000000LL)
        return 0;
    LogitArgs a = {};
    a.N = N;
    a.V = V;
    a.hist_max = history_max;
    a.bias_max = bias_max;
    return N > 0 && plan_logits(a, elem_size(dtype)) ? logits_workspace(a) : 0;
}

extern "C" ce_status ce_logits_process(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                       const int64_t strides[3], const ce_logits_params* params, void* out,
                                       const int64_t out_strides[3], void* workspace, size_t workspace_bytes,
                                       void* stream) {
    return gbce::logits_common(nullptr, nullptr, logits, dtype, dim0, dim1, V, strides, params, out, out_strides,
                               false, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" ce_status ce_logits_process_bwd(const void* grad_out, const int64_t grad_out_strides[3],
                                           const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                                           const int64_t strides[3], const ce_logits_params* params, void* grad,
                                           const int64_t grad_strides[3], void* workspace, size_t workspace_bytes,
                                           void* stream) {
    return gbce::logits_common(grad_out, grad_out_strides, logits, dtype, dim0, dim1, V, strides, params, grad,
                               grad_strides, true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
