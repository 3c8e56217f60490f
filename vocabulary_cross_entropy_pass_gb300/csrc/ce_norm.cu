// ce_norm.cu -- the residual's addition and the root-mean-square norm, and
// their gradients.
//
//   h = x + r                      (r optional; stored rounded to the input type)
//   y_j = h_j rstd w_j,            rstd = 1 / sqrt(mean_j h_j^2 + eps)
//   8 bits: for each group of columns  s = max(max|y_j| / top, 2^-126),
//           q_j = round(y_j / s) saturated at +-top (448 for e4m3, 57344 for e5m2)
//
// y comes from the unrounded float32 h, so the stored h and y each carry one
// rounding.  Backward, from the stored h with n_j = h_j rstd, c = mean_j(g_j w_j n_j):
//   dx_j = rstd (g_j w_j - n_j c) + dh_j,     dw_j = sum over rows of g_j n_j
// where dh is the gradient that reaches h from the residual stream; x and r
// share dx.  rstd is computed again from h (the row is in registers anyway),
// so the forward saves nothing but h.
//
// Bound by HBM: forward reads x, r and writes h, y; backward reads h, g, dh and
// writes dx.  A row's elements stay in registers between the statistics and
// the output.  Measured, of the GPU's 6.70 TB/s copy rate (bf16, GPU time of a call in
// a graph): forward of 16384 x 4096 with a residual 80.4 us, 6.68 TB/s; to e4m3 with a
// scale for 128 columns, 8192 x 8192, 83.2 us, 5.7 TB/s (its conversions keep the
// schedulers at 75 %); gradients of 16384 x 4096 88.1 us, 6.1 TB/s.  Rows off the
// 16-byte grid, 16384 x 4097: forward 154 us (0.52 of the copy rate), gradients 133
// (0.60), e4m3 230 (0.30); short ones, 32768 x 511 and 777, 0.3 to 0.5.  A float32
// weight under 16-bit rows, which is loaded an element at a time: forward of 16384 x
// 4096 92 us, gradients 89.7.
#include <cuda_fp8.h>

#include "ce_device.cuh"
#include "ce_internal.h"
#include "ce_pack.cuh"

namespace gbce {
namespace {

constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126: 1 / scale stays finite

struct NormFwdArgs {
    const char* x;
    const char* r;         // or NULL
    const char* w;
    char* y;
    char* h;               // or NULL
    float* scales;         // [N][groups]
    int64_t N, H;
    int64_t xs, rs, ys, hs;  // row strides in bytes
    float eps, inv_h, top;
    int w32;               // the weight is float32
    int group, groups;     // columns per scale and scales per row (8 bits)
    int kind;              // 1 e4m3, 2 e5m2
};

// Sum over the CTA; every thread gets it.  `red` holds a float per warp, twice
// (two calls in a row use alternate halves, so one barrier each is enough).
__device__ __forceinline__ float cta_sum(float v, float* red) {
    v = warp_allsum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const float t = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f;
    return warp_allsum(t);
}
__device__ __forceinline__ float cta_max(float v, float* red) {
    v = warp_allmax(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const float t = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f;
    return warp_allmax(t);
}

// 8-bit values of a group, from t_j = h_j w_j (y_j = t_j rstd): with m = max|t| the
// scale is m / top rstd and q_j = t_j top / m.  The factor top / m is kept as a
// float and what that leaves (hi + lo), so q_j takes one rounding before that to 8
// bits and a value on a rounding border goes to the definition's side (34 million
// values of bf16 rows in groups of 128: none off the rounded definition; with a
// factor of one float 11 of a million, and 80.1 us for 8192 x 8192, its outputs given,
// against 81.9).
// A scale at its least value, or an m whose reciprocal may not be finite: y_j times
// 1 / scale.
struct Group {
    float hi, lo, scale;
    bool direct;           // t_j is taken, not y_j
};
__device__ __forceinline__ Group group_of(float m, float to_scale, float top) {
    Group g;
    g.scale = fmaxf(m * to_scale, kTinyScale);
    g.direct = g.scale > kTinyScale && m > 0x1p-100f && m < 0x1p100f;
    const float d = g.direct ? m : g.scale, n = g.direct ? top : 1.f;
    const float inv = __fdividef(1.f, d);
    g.hi = n * inv;
    g.lo = fmaf(-g.hi, d, n) * inv;
    return g;
}
// PAIRS: two values to an instruction (in the wide kernel they took more than they
// gave: 2048 x 20480 in float32 150 -> 162 us).
template <int VEC, bool PAIRS = true>
__device__ __forceinline__ void store_q8(char* p, float* t, const Group& g, float rstd, int kind) {
    Pack<uint8_t, VEC> o;
    if (!g.direct) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) t[i] *= rstd;
    }
    const __nv_fp8_interpretation_t k = kind == 1 ? __NV_E4M3 : __NV_E5M2;
    if constexpr (VEC >= 2) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const float2 f = make_float2(t[i], t[i + 1]);
            const float2 q = PAIRS ? __ffma2_rn(f, make_float2(g.hi, g.hi), __fmul2_rn(f, make_float2(g.lo, g.lo)))
                                   : make_float2(fmaf(f.x, g.hi, f.x * g.lo), fmaf(f.y, g.hi, f.y * g.lo));
            const uint16_t two = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, k);
            o.v[i] = (uint8_t)two;
            o.v[i + 1] = (uint8_t)(two >> 8);
        }
    } else {
        o.v[0] = __nv_cvt_float_to_fp8(fmaf(t[0], g.hi, t[0] * g.lo), __NV_SATFINITE, k);
    }
    o.store(p);
}

template <typename T, int VEC>
__device__ __forceinline__ void load_w(const NormFwdArgs& p, int64_t col, float* w) {
    if (p.w32) {
        const float* q = reinterpret_cast<const float*>(p.w) + col;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = __ldg(q + i);
    } else {
        Pack<T, VEC> t;
        t.load_nc(p.w + col * (int64_t)sizeof(T));
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = t.f(i);
    }
}

// One CTA (or warp) per row, VPT vectors of VEC elements per thread in registers.
// PHASED: the rows of x, r, y and h lie off the 16-byte grid, all at the same
// offset: a thread's vectors are those of the grid, the row's first and last only
// in part (element i of vector v is column v * VEC + i - sh).
template <typename T, int VEC, int VPT, bool Q8, bool PHASED>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) ce_rmsnorm_fwd_kernel(const __grid_constant__ NormFwdArgs p) {
    constexpr int ES = sizeof(T);
    __shared__ float red[64];
    extern __shared__ float stage[];  // STAGED: the row's y
    // 8-bit groups go by columns: lanes of vectors hold them whole on the grid only
    constexpr bool STAGED = Q8 && (PHASED || VEC == 1);
    // rows of at most 128 vectors: a warp to each, eight in a CTA (blockDim.y)
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.N) return;
    const int tid = threadIdx.x, TH = blockDim.x;
    const char* x = p.x + row * p.xs;
    const char* r = p.r ? p.r + row * p.rs : nullptr;
    const int sh = PHASED ? (int)(reinterpret_cast<uintptr_t>(x) & 15u) / ES : 0;
    const int nv = PHASED ? (int)((p.H + sh + VEC - 1) / VEC) : (int)(p.H / VEC);
    auto edge = [&](int v) { return PHASED && (v == 0 || v == nv - 1); };
    auto inside = [&](int v, int i) {
        const int64_t c = (int64_t)v * VEC + i - sh;
        return c >= 0 && c < p.H;
    };
    auto take = [&](const char* row_at, int v) {
        Pack<T, VEC> a;
        if (edge(v) || v >= nv) a.zero();
        if (edge(v)) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (inside(v, i)) a.v[i] = reinterpret_cast<const T*>(row_at)[(int64_t)v * VEC + i - sh];
        } else if (v < nv) {
            a.load_cs(row_at + ((int64_t)v * VEC - sh) * ES);
        }
        return a;
    };
    auto give = [&](char* row_at, int v, const float* f) {
        Pack<T, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.set(i, f[i]);
        if (edge(v)) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (inside(v, i)) reinterpret_cast<T*>(row_at)[(int64_t)v * VEC + i - sh] = o.v[i];
        } else if (v < nv) {
            o.store(row_at + ((int64_t)v * VEC - sh) * ES);
        }
    };

    float h[VPT][VEC];
    {
        Pack<T, VEC> a[VPT], b[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) a[k] = take(x, tid + k * TH);
        if (r) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) b[k] = take(r, tid + k * TH);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[k][i] = a[k].f(i) + b[k].f(i);
        } else {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[k][i] = a[k].f(i);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss = fmaf(h[k][i], h[k][i], ss);
    if (p.h) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) give(p.h + row * p.hs, tid + k * TH, h[k]);
    }
    ss = cta_sum(ss, red);
    const float rstd = rsqrtf(fmaf(ss, p.inv_h, p.eps));
    const bool w_grid = PHASED && !p.w32 && (reinterpret_cast<uintptr_t>(p.w) & 15u) == 0;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = tid + k * TH;
        float w[VEC];
        if (v < nv) {
            if constexpr (PHASED) {
                if (w_grid && v > 0 && (int64_t)(v + 1) * VEC <= p.H) {
                    // the weight's own vectors v - 1 and v hold these columns
                    const uint4* q = reinterpret_cast<const uint4*>(p.w) + v;
                    Pack<T, VEC> t;
                    t.raw = sh ? shift_bytes(__ldg(q - 1), __ldg(q), 16u - (uint32_t)sh * ES) : __ldg(q);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) w[i] = t.f(i);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        w[i] = 0.f;
                        if (!edge(v) || inside(v, i)) load_w<T, 1>(p, (int64_t)v * VEC + i - sh, w + i);
                    }
                }
            } else {
                load_w<T, VEC>(p, (int64_t)v * VEC, w);
            }
            // 8 bits: t, and rstd goes into the scales
            if constexpr (Q8 && VEC % 2 == 0) {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const float2 t = __fmul2_rn(make_float2(h[k][i], h[k][i + 1]), make_float2(w[i], w[i + 1]));
                    h[k][i] = t.x;
                    h[k][i + 1] = t.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[k][i] *= Q8 ? w[i] : rstd * w[i];
            }
        }
    }
    char* y = p.y + row * p.ys;
    if constexpr (!Q8) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) give(y, tid + k * TH, h[k]);
    } else {
        float am[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            am[k] = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) am[k] = fmaxf(am[k], fabsf(h[k][i]));
            if (tid + k * TH >= nv) am[k] = 0.f;
        }
        float* sc = p.scales + row * (int64_t)p.groups;
        const float to_scale = rstd / p.top;
        Group whole = {};  // of all columns, where there is one group
        if (p.groups == 1) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k) m = fmaxf(m, am[k]);
            whole = group_of(cta_max(m, red + 32), to_scale, p.top);
            if (tid == 0) sc[0] = whole.scale;
        }
        if constexpr (STAGED) {
            // the row's float32 t in shared memory; then a warp to each group of
            // columns, lanes side by side
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * TH;
                if (v < nv)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (!edge(v) || inside(v, i)) stage[(int64_t)v * VEC + i - sh] = h[k][i];
            }
            __syncthreads();
            const int lane = tid & 31, nw = TH >> 5;
            const int per = p.groups == 1 ? 4 : p.group / 32, run = per * 32;
            const bool four = per == 4 && (reinterpret_cast<uintptr_t>(y) & 3u) == 0;
            for (int g = tid >> 5; (int64_t)g * run < p.H; g += nw) {
                const int64_t c0 = (int64_t)g * run + lane * per;
                float f[4];
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = i < per && c0 + i < p.H ? stage[c0 + i] : 0.f;
                    m = fmaxf(m, fabsf(f[i]));
                }
                Group s = whole;
                if (p.groups > 1) {
                    s = group_of(warp_allmax(m), to_scale, p.top);
                    if (lane == 0) sc[g] = s.scale;
                }
                if (four && c0 + 4 <= p.H) {
                    store_q8<4>(y + c0, f, s, rstd, p.kind);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < per && c0 + i < p.H) store_q8<1>(y + c0 + i, f + i, s, rstd, p.kind);
                }
            }
        } else {
            const int gl = p.group / VEC;  // vectors (lanes) per group: at most 32
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * TH;
                Group s = whole;
                if (p.groups > 1) {
                    for (int o = gl >> 1; o > 0; o >>= 1) am[k] = fmaxf(am[k], __shfl_xor_sync(kFull, am[k], o));
                    s = group_of(am[k], to_scale, p.top);
                    if (v < nv && (v & (gl - 1)) == 0) sc[v / gl] = s.scale;
                }
                if (v < nv) store_q8<VEC>(y + (int64_t)v * VEC, h[k], s, rstd, p.kind);
            }
        }
    }
}

// Rows too wide for registers: two passes (three with 8 bits) over the row,
// the later ones from L2.  h and y are written in the last pass only, each
// element by the thread that has just read it, so they may replace x or r.
template <typename T, int VEC, bool Q8>
__global__ void __launch_bounds__(512) ce_rmsnorm_fwd_wide_kernel(const __grid_constant__ NormFwdArgs p) {
    constexpr int ES = sizeof(T);
    __shared__ float red[64];
    extern __shared__ uint32_t gmax[];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, TH = blockDim.x;
    const int64_t nv = p.H / VEC;
    const char* x = p.x + row * p.xs;
    const char* r = p.r ? p.r + row * p.rs : nullptr;
    auto get = [&](int64_t v, float* h) {
        Pack<T, VEC> a, b;
        a.load(x + v * VEC * ES);
        if (r) b.load(r + v * VEC * ES);
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] = r ? a.f(i) + b.f(i) : a.f(i);
    };
    float ss = 0.f;
#pragma unroll 4
    for (int64_t v = tid; v < nv; v += TH) {
        float h[VEC];
        get(v, h);
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss = fmaf(h[i], h[i], ss);
    }
    ss = cta_sum(ss, red);
    const float rstd = rsqrtf(fmaf(ss, p.inv_h, p.eps));
    float* sc = p.scales + row * (int64_t)p.groups;
    const float to_scale = rstd / p.top;
    if constexpr (Q8) {
        for (int g = tid; g < p.groups; g += TH) gmax[g] = 0u;
        __syncthreads();
        for (int64_t v0 = 0; v0 < nv; v0 += TH) {
            const int64_t v = v0 + tid;
            float m = 0.f;
            if (v < nv) {
                float h[VEC], w[VEC];
                get(v, h);
                load_w<T, VEC>(p, v * VEC, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(h[i] * w[i]));
                atomicMax(&gmax[v * VEC / p.group], __float_as_uint(m));
            }
        }
        __syncthreads();
        for (int g = tid; g < p.groups; g += TH) sc[g] = group_of(__uint_as_float(gmax[g]), to_scale, p.top).scale;
    }
    char* y = p.y + row * p.ys;
    char* ho = p.h ? p.h + row * p.hs : nullptr;
#pragma unroll 2
    for (int64_t v = tid; v < nv; v += TH) {
        float h[VEC], w[VEC];
        get(v, h);
        load_w<T, VEC>(p, v * VEC, w);
        Pack<T, VEC> o;
        if (ho) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o.set(i, h[i]);
            o.store(ho + v * VEC * ES);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] *= Q8 ? w[i] : rstd * w[i];
        if constexpr (Q8) {
            store_q8<VEC, false>(y + v * VEC, h, group_of(__uint_as_float(gmax[v * VEC / p.group]), to_scale, p.top),
                                 rstd, p.kind);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o.set(i, h[i]);
            o.store(y + v * VEC * ES);
        }
    }
}

template <typename T, int VEC, bool Q8, bool PHASED = false>
cudaError_t launch_fwd(const NormFwdArgs& a, cudaStream_t s) {
    const int64_t nv = PHASED ? (a.H + VEC - 1 + VEC - 1) / VEC : a.H / VEC;
    size_t smem = Q8 ? (size_t)a.groups * 4 : 0;  // the wide kernel's maxima
    constexpr int MAXV = VEC >= 8 ? 4 : (VEC == 4 ? 8 : 16);  // 512 threads hold 512 * MAXV vectors
    if (nv > 512 * MAXV) {
        auto* k = ce_rmsnorm_fwd_wide_kernel<T, PHASED ? 1 : VEC, Q8>;
        if (smem > 40 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        k<<<(unsigned)a.N, 512, smem, s>>>(a);
        return cudaGetLastError();
    }
    smem = Q8 && (PHASED || VEC == 1) ? (size_t)a.H * 4 : 0;
    auto go = [&](auto* k, int th) {
        if (smem > 40 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        k<<<(unsigned)a.N, th, smem, s>>>(a);
        return cudaGetLastError();
    };
    const auto th = [&](int v) { return (int)((nv + 32 * v - 1) / (32 * v) * 32); };
    if (nv <= (PHASED ? 32 : 128) && a.N > 304 && smem == 0) {
        // many short rows (32768 of 128 elements 18.3 -> 8.2 us; of 777, off the
        // grid, 60 -> 75 us, so those keep a CTA)
        const dim3 block(32, 8);
        const unsigned grid = (unsigned)((a.N + 7) / 8);
        if (nv <= 32) ce_rmsnorm_fwd_kernel<T, VEC, 1, Q8, PHASED><<<grid, block, 0, s>>>(a);
        else ce_rmsnorm_fwd_kernel<T, VEC, 4, Q8, PHASED><<<grid, block, 0, s>>>(a);
        return cudaGetLastError();
    }
    if (nv <= 256 || (a.N <= 304 && nv <= 1024)) return go(ce_rmsnorm_fwd_kernel<T, VEC, 1, Q8, PHASED>, th(1));
    if (nv <= 2048) return go(ce_rmsnorm_fwd_kernel<T, VEC, 4, Q8, PHASED>, th(4));
    return go(ce_rmsnorm_fwd_kernel<T, VEC, MAXV, Q8, PHASED>, th(MAXV));
}

template <typename T>
cudaError_t launch_fwd_t(const NormFwdArgs& a, int vb, cudaStream_t s) {
    constexpr int ES = sizeof(T);
    const bool q = a.kind != 0;
    if (vb == 16) return q ? launch_fwd<T, 16 / ES, true>(a, s) : launch_fwd<T, 16 / ES, false>(a, s);
    auto at = [](const void* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u); };
    bool phased = (q || at(a.y) == at(a.x)) && (!a.r || at(a.r) == at(a.x)) && (!a.h || at(a.h) == at(a.x));
    if (a.N > 1)
        phased = phased && (q || (a.ys - a.xs) % 16 == 0) && (!a.r || (a.rs - a.xs) % 16 == 0) &&
                 (!a.h || (a.hs - a.xs) % 16 == 0);
    if (phased) return q ? launch_fwd<T, 16 / ES, true, true>(a, s) : launch_fwd<T, 16 / ES, false, true>(a, s);
    if constexpr (ES == 2)
        if (vb == 4 && !q) return launch_fwd<T, 2, false>(a, s);
    return q ? launch_fwd<T, 1, true>(a, s) : launch_fwd<T, 1, false>(a, s);
}

// ----------------------------------------------------------------- backward
struct NormBwdArgs {
    const char* g;
    const char* h;
    const char* w;
    const char* dh;        // or NULL
    char* dx;
    float* part;           // [gridDim.x][part_pitch] partial sums of dw, or NULL
    int64_t N, H;
    int64_t gs, hs, dhs, dxs;  // row strides in bytes
    float eps, inv_h;
    int w32;
    uint32_t* err;         // the workspace's error word, or NULL
};

// Floats between the partial rows of dw.
__host__ __device__ __forceinline__ int64_t part_pitch(int64_t H) { return (H + 15) / 4 * 4 + 4; }

// A persistent grid over the rows; a thread keeps its columns' dw sums in
// registers over all rows of its CTA and writes them once.  The rows come in by
// bulk copies (TMA) into a ring of `stages` row sets (g, h and dh): the next ones
// are on their way while one is worked on, and both passes over a row read
// shared memory.  A row off the 16-byte grid is copied from the boundary before
// it to the boundary after it, as far as that stays between the tensor's first
// and last element, the rest element by element.
// MODE, by how the rows of g, h, dh and dx lie:
//   kOnGrid  all on the 16-byte grid, a whole number of vectors each;
//   kPhased  off it, but all at the same offset, row for row: a thread's
//            vectors are those of the 16-byte grid, the row's first and last only
//            in part.  Every row of a CTA has the same offset (the grid is a
//            multiple of 8 CTAs), so a thread's columns stay its own;
//   kLoose   anything else: single elements, TH apart.
// One barrier per row: it hands the sums over, and past it the row before
// has been read by all, so its place is filled again.  A copy that does not
// arrive sets the workspace's error word, and every thread leaves at the row's barrier.
constexpr int kOnGrid = 0, kPhased = 1, kLoose = 2;
struct RingArgs {
    NormBwdArgs n;
    int stages, slot;      // bytes of one tensor's row in the ring (a multiple of 16)
};

template <int ES>
struct RowSpan {           // what of a row the bulk copy takes
    const char* from;
    uint32_t bytes;        // 0: nothing
    int at;                // byte of the slot where `from` lands; the row begins at byte `phase`
    int phase;
};
template <int ES>
__device__ __forceinline__ RowSpan<ES> row_span(const char* base, int64_t stride, int64_t row, int64_t rows, int64_t len) {
    const char* a = base + row * stride;
    const uintptr_t u = reinterpret_cast<uintptr_t>(a), e = u + (uintptr_t)len;
    const uintptr_t first = reinterpret_cast<uintptr_t>(base);
    const uintptr_t last = first + (uintptr_t)((rows - 1) * stride + len);  // past the last element
    uintptr_t lo = u & ~(uintptr_t)15, hi = (e + 15) & ~(uintptr_t)15;
    const int phase = (int)(u - lo);
    if (lo < first) lo = (u + 15) & ~(uintptr_t)15;
    if (hi > last) hi = e & ~(uintptr_t)15;
    RowSpan<ES> s;
    s.phase = phase;
    s.from = reinterpret_cast<const char*>(lo);
    s.bytes = hi > lo ? (uint32_t)(hi - lo) : 0u;
    s.at = (int)(lo - (u - phase));
    return s;
}

template <typename T, int VPT, int MODE, bool RES>
__global__ void __launch_bounds__(512) ce_rmsnorm_bwd_kernel(const __grid_constant__ RingArgs q) {
    constexpr int ES = sizeof(T);
    constexpr bool GRID = MODE == kOnGrid;
    constexpr int VEC = MODE == kLoose ? 1 : 16 / ES;
    constexpr int NT = RES ? 3 : 2;            // tensors per row set
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[16];
    __shared__ float2 red[2][16];
    __shared__ int gave_up;
    const NormBwdArgs& p = q.n;
    const int tid = threadIdx.x, TH = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = TH >> 5;
    const int64_t len = p.H * ES;
    // kPhased: the elements by which the CTA's rows lie past the grid; element i of
    // vector v is column v * VEC + i - sh
    const int sh = MODE == kPhased ? (int)((reinterpret_cast<uintptr_t>(p.h) + blockIdx.x * (uint64_t)p.hs) & 15u) / ES : 0;
    const int nv = MODE == kPhased ? (int)((p.H + sh + VEC - 1) / VEC) : (int)(p.H / VEC);
    auto edge = [&](int v) { return MODE == kPhased && (v == 0 || v == nv - 1); };
    auto inside = [&](int v, int i) {
        const int64_t c = (int64_t)v * VEC + i - sh;
        return c >= 0 && c < p.H;
    };
    const uint64_t policy = l2_evict_first_policy();
    if (tid == 0) {
        for (int k = 0; k < q.stages; ++k) mbar_init(&full[k], 1);
        gave_up = 0;
        if (blockIdx.x == 0 && p.err) *p.err = 0u;
        fence_barrier_init();
    }
    __syncthreads();

    auto base_of = [&](int t) { return t == 0 ? p.g : (t == 1 ? p.h : p.dh); };
    auto stride_of = [&](int t) { return t == 0 ? p.gs : (t == 1 ? p.hs : p.dhs); };
    auto span_of = [&](int t, int64_t row) { return row_span<ES>(base_of(t), stride_of(t), row, p.N, len); };
    auto issue = [&](int64_t row, int stage) {  // one thread
        unsigned char* at = ring + (size_t)stage * NT * q.slot;
        if (GRID) {
            mbar_arrive_expect_tx(&full[stage], (uint32_t)(NT * len));
#pragma unroll
            for (int t = 0; t < NT; ++t)
                tma_load_1d(at + t * q.slot, base_of(t) + row * stride_of(t), (uint32_t)len, &full[stage], policy);
        } else {
            uint32_t bytes = 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) bytes += span_of(t, row).bytes;
            mbar_arrive_expect_tx(&full[stage], bytes);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const RowSpan<ES> s = span_of(t, row);
                if (s.bytes) tma_load_1d(at + t * q.slot + s.at, s.from, s.bytes, &full[stage], policy);
            }
        }
    };
    if (tid == 0)
        for (int k = 0; k < q.stages; ++k) {
            const int64_t row = blockIdx.x + (int64_t)k * gridDim.x;
            if (row < p.N) issue(row, k);
        }

    float w32[VPT][VEC], dw[VPT][VEC];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = tid + k * TH;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            dw[k][i] = 0.f;
            w32[k][i] = 0.f;
            if (v < nv && (!edge(v) || inside(v, i)))
                w32[k][i] = p.w32 ? __ldg(reinterpret_cast<const float*>(p.w) + (int64_t)v * VEC + i - sh)
                                  : to_f32(reinterpret_cast<const T*>(p.w)[(int64_t)v * VEC + i - sh]);
        }
    }

    int stage = 0, flip = 0;
    uint32_t parity = 0;
    int64_t done = -1;     // stage whose row all threads have read once they pass the next barrier
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x, flip ^= 1) {
        const unsigned char* at = ring + (size_t)stage * NT * q.slot;
        if (!mbar_wait_bounded(&full[stage], parity)) {
            if (p.err) atomicOr(p.err, CE_DEVERR_TIMEOUT);
            gave_up = 1;
        }
        int ph[3] = {0, 0, 0};
        if (!GRID) {
            // rows within 16 bytes of a tensor's ends may have elements that no copy
            // could take
            bool ends = false;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int64_t off = row * stride_of(t);
                ends |= off < 16 || (p.N - 1 - row) * stride_of(t) < 16;
                ph[t] = (int)((reinterpret_cast<uintptr_t>(base_of(t)) + (uintptr_t)off) & 15u);
            }
            if (ends) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const RowSpan<ES> s = span_of(t, row);
                    // elements before the copy, and the first one after it
                    const int64_t head = min(p.H, s.at > s.phase ? (int64_t)((s.at - s.phase) / ES) : (int64_t)0);
                    const int64_t tail0 = s.bytes ? ((int64_t)s.at + s.bytes - s.phase) / ES : head;
                    const T* a = reinterpret_cast<const T*>(base_of(t) + row * stride_of(t));
                    T* to = reinterpret_cast<T*>(ring + (size_t)stage * NT * q.slot + t * q.slot + s.phase);
                    for (int64_t c = tid; c < head; c += TH) to[c] = a[c];
                    for (int64_t c = tail0 + tid; c < p.H; c += TH) to[c] = a[c];
                }
                fence_proxy_async_smem();  // a later copy may land on these bytes
                __syncthreads();
            }
        }
        auto get = [&](int t, int v) {
            Pack<T, VEC> x;
            x.load(at + t * q.slot + (MODE == kLoose ? ph[t] : 0) + (size_t)v * VEC * ES);
            if (edge(v)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (!inside(v, i)) x.set(i, 0.f);
            }
            return x;
        };
        float ss = 0.f, c = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * TH;
            if (v < nv) {
                const Pack<T, VEC> g = get(0, v), h = get(1, v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float hv = h.f(i);
                    ss = fmaf(hv, hv, ss);
                    c = fmaf(g.f(i) * w32[k][i], hv, c);
                }
            }
        }
        ss = warp_allsum(ss);
        c = warp_allsum(c);
        if (lane == 0) red[flip][warp] = make_float2(ss, c);
        __syncthreads();
        if (gave_up) break;
        if (tid == 0 && done >= 0) {
            // the row before this one has been read by all
            const int64_t next = row + (int64_t)(q.stages - 1) * gridDim.x;
            if (next < p.N) issue(next, (int)done);
        }
        {
            const float2 t = lane < nw ? red[flip][lane] : make_float2(0.f, 0.f);
            ss = warp_allsum(t.x);
            c = warp_allsum(t.y);
        }
        const float rstd = rsqrtf(fmaf(ss, p.inv_h, p.eps));
        const float cc = c * rstd * p.inv_h;  // mean of g w n
        char* xp = p.dx + row * p.dxs;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * TH;
            if (v < nv) {
                const Pack<T, VEC> g = get(0, v), h = get(1, v);
                Pack<T, VEC> d, o;
                if (RES) d = get(2, v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float n = h.f(i) * rstd, gv = g.f(i);
                    dw[k][i] = fmaf(gv, n, dw[k][i]);
                    float t = rstd * fmaf(-n, cc, gv * w32[k][i]);
                    if (RES) t += d.f(i);
                    o.set(i, t);
                }
                if (edge(v)) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (inside(v, i)) reinterpret_cast<T*>(xp)[(int64_t)v * VEC + i - sh] = o.v[i];
                } else {
                    o.store_cs(xp + ((int64_t)v * VEC - sh) * ES);
                }
            }
        }
        done = stage;
        if (++stage == q.stages) {
            stage = 0;
            parity ^= 1u;
        }
    }
    if (gave_up) {
        // no copy may land after this CTA has left
        if (tid == 0)
            for (int k = 0; k < q.stages; ++k) mbar_wait_bounded(&full[k], k >= stage ? parity : parity ^ 1u);
        __syncthreads();
        return;
    }
    if (p.part) {
        // kPhased: shifted like the rows
        float* out = p.part + (int64_t)blockIdx.x * part_pitch(p.H);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * TH;
            if (v < nv) store_f32<VEC>(out + (int64_t)v * VEC, dw[k]);
        }
    }
}

// Rows too wide for registers: two passes over each row, dw summed in this
// CTA's own partial row.
template <typename T, int VEC>
__global__ void __launch_bounds__(512) ce_rmsnorm_bwd_wide_kernel(const __grid_constant__ NormBwdArgs p) {
    constexpr int ES = sizeof(T);
    __shared__ float2 red[2][32];
    const int tid = threadIdx.x, TH = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = TH >> 5;
    const int64_t nv = p.H / VEC;
    float* out = p.part ? p.part + (int64_t)blockIdx.x * part_pitch(p.H) : nullptr;
    if (blockIdx.x == 0 && tid == 0 && p.err) *p.err = 0u;
    auto wat = [&](int64_t c) {
        return p.w32 ? __ldg(reinterpret_cast<const float*>(p.w) + c) : to_f32(reinterpret_cast<const T*>(p.w)[c]);
    };
    int flip = 0;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x, flip ^= 1, first = false) {
        const char* gp = p.g + row * p.gs;
        const char* hp = p.h + row * p.hs;
        float ss = 0.f, c = 0.f;
#pragma unroll 2
        for (int64_t v = tid; v < nv; v += TH) {
            Pack<T, VEC> g, h;
            g.load(gp + v * VEC * ES);
            h.load(hp + v * VEC * ES);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float hv = h.f(i);
                ss = fmaf(hv, hv, ss);
                c = fmaf(g.f(i) * wat(v * VEC + i), hv, c);
            }
        }
        ss = warp_allsum(ss);
        c = warp_allsum(c);
        if (lane == 0) red[flip][warp] = make_float2(ss, c);
        __syncthreads();
        const float2 t = lane < nw ? red[flip][lane] : make_float2(0.f, 0.f);
        ss = warp_allsum(t.x);
        c = warp_allsum(t.y);
        const float rstd = rsqrtf(fmaf(ss, p.inv_h, p.eps));
        const float cc = c * rstd * p.inv_h;
        char* xp = p.dx + row * p.dxs;
        for (int64_t v = tid; v < nv; v += TH) {
            Pack<T, VEC> g, h, d, o;
            g.load(gp + v * VEC * ES);
            h.load(hp + v * VEC * ES);
            if (p.dh) d.load(p.dh + row * p.dhs + v * VEC * ES);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float n = h.f(i) * rstd, gv = g.f(i);
                if (out) {
                    float* q = out + v * VEC + i;
                    *q = first ? gv * n : fmaf(gv, n, *q);
                }
                float t2 = rstd * fmaf(-n, cc, gv * wat(v * VEC + i));
                if (p.dh) t2 += d.f(i);
                o.set(i, t2);
            }
            o.store(xp + v * VEC * ES);
        }
    }
}

// Rows of at most kShortWidth elements: a warp to each, straight into registers,
// U rows at once, without barriers; a lane's columns' dw stay in its registers over
// all of its warp's rows, and the CTA's eight warps are added in order at the end.
// EPL: elements of a lane (32 * EPL is at least the width).
// Against the ring above with a CTA to a row (bf16 with a residual, GPU us of a call,
// here / ring): 262144 x 128 51 / 109, 32768 x 256 17 / 24, 131072 x 512 92 / 99; off
// the grid 32768 x 511 47 / 66, 4708 x 396 8.6 / 17.4; 64 x 128 4.2 / 5.5.
constexpr int64_t kShortWidth = 512;
constexpr int kShortWarps = 8;
// CTAs per SM, two / four: 262144 x 128 72 / 51 us, 262144 x 64 66 / 46; 32768 x 256
// 16.8 / 19.6, 32768 x 512 25.7 / 28.6 (fewer partial rows of dw to write and add).
// Three, six and eight were behind the better of these at nearly all sizes.
constexpr int short_per_sm(int64_t H) { return H <= 128 ? 4 : 2; }
template <typename T, int EPL, int VEC>
__global__ void __launch_bounds__(kShortWarps * 32) ce_rmsnorm_bwd_short_kernel(const __grid_constant__ NormBwdArgs p) {
    constexpr int ES = sizeof(T);
    constexpr int VPT = EPL / VEC;
    constexpr int U = EPL <= 8 ? 2 : 1;
    __shared__ __align__(16) float sum[kShortWarps][EPL * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int H = (int)p.H, nv = H / VEC;
    if (blockIdx.x == 0 && tid == 0 && p.err) *p.err = 0u;
    float w32[VPT][VEC], dw[VPT][VEC];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = lane + k * 32;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            dw[k][i] = 0.f;
            w32[k][i] = 0.f;
            if (v < nv)
                w32[k][i] = p.w32 ? __ldg(reinterpret_cast<const float*>(p.w) + v * VEC + i)
                                  : to_f32(reinterpret_cast<const T*>(p.w)[v * VEC + i]);
        }
    }
    const int64_t step = (int64_t)gridDim.x * kShortWarps;
    for (int64_t row = (int64_t)blockIdx.x * kShortWarps + warp; row < p.N; row += U * step) {
        Pack<T, VEC> g[U][VPT], h[U][VPT], d[U][VPT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = row + u * step;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = lane + k * 32;
                g[u][k].zero();
                h[u][k].zero();
                d[u][k].zero();
                if (r < p.N && v < nv) {
                    g[u][k].load_cs(p.g + r * p.gs + v * (VEC * ES));
                    h[u][k].load_cs(p.h + r * p.hs + v * (VEC * ES));
                    if (p.dh) d[u][k].load_cs(p.dh + r * p.dhs + v * (VEC * ES));
                }
            }
        }
        float ss[U], c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ss[u] = c[u] = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float hv = h[u][k].f(i);
                    ss[u] = fmaf(hv, hv, ss[u]);
                    c[u] = fmaf(g[u][k].f(i) * w32[k][i], hv, c[u]);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ss[u] = warp_allsum(ss[u]);
            c[u] = warp_allsum(c[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = row + u * step;
            if (r >= p.N) break;
            const float rstd = rsqrtf(fmaf(ss[u], p.inv_h, p.eps));
            const float cc = c[u] * rstd * p.inv_h;  // mean of g w n
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = lane + k * 32;
                Pack<T, VEC> o;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float n = h[u][k].f(i) * rstd, gv = g[u][k].f(i);
                    dw[k][i] = fmaf(gv, n, dw[k][i]);
                    float t = rstd * fmaf(-n, cc, gv * w32[k][i]);
                    if (p.dh) t += d[u][k].f(i);
                    o.set(i, t);
                }
                if (v < nv) o.store_cs(p.dx + r * p.dxs + v * (VEC * ES));
            }
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int k = 0; k < VPT; ++k) store_f32<VEC>(&sum[warp][(lane + k * 32) * VEC], dw[k]);
    __syncthreads();
    for (int c = tid; c < H; c += kShortWarps * 32) {
        float t = sum[0][c];
#pragma unroll
        for (int w = 1; w < kShortWarps; ++w) t += sum[w][c];
        p.part[(int64_t)blockIdx.x * part_pitch(p.H) + c] = t;
    }
}

// dw_j = the partial rows' column sums, in a fixed order: 32 columns per CTA, a
// warp to every 32nd partial row, then the warps' sums in order.
// Partial row r lies (low + r * step) mod 16 bytes / es past its start.
__global__ void __launch_bounds__(1024) ce_rmsnorm_dw_kernel(const float* part, int rows, int64_t H, float* dw,
                                                             uint32_t low, uint32_t step, int es) {
    __shared__ float sh[32][33];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float acc = 0.f;
    if (c < H) {
#pragma unroll 8
        for (int r = warp; r < rows; r += 32) acc += __ldcg(part + r * part_pitch(H) + c + ((low + r * step) & 15u) / es);
    }
    sh[warp][lane] = acc;
    __syncthreads();
    // warp w adds column w's 32 sums pairwise, the same pairs on every run
    const float t = warp_allsum(sh[lane][warp]);
    const int64_t col = (int64_t)blockIdx.x * 32 + warp;
    if (lane == 0 && col < H) dw[col] = t;
}

// CTAs of the backward grid, from the sizes alone (the workspace holds a
// partial row for each): two per SM, more for short rows, whose barrier each is
// paid over fewer bytes (bf16, 32768 rows, GB/s of algorithmic bytes with two /
// four / eight per SM: 2048 wide 5290 / 5840, 1024 wide with four / eight 4820 /
// 5330; 4096 wide with two / three 6000 / 5840).  A ring has up to eight row
// sets in such a share of the SM's shared memory.  Where fewer than three fit (bf16
// with a residual: 776 to 1023, 1544 to 2047, 3080 to 4095 and more than 6144
// columns), it takes up to eight from all of it; fewer CTAs than these are then
// resident, and the grid runs in waves.
int bwd_per_sm(int64_t H) { return H >= 4096 ? 2 : (H >= 2048 ? 4 : (H >= 1024 ? 8 : 16)); }
int bwd_grid(int64_t N, int64_t H) {
    if (H <= kShortWidth) {
        const int64_t ctas = (N + kShortWarps - 1) / kShortWarps;
        const int64_t full = 152 * short_per_sm(H);
        return (int)(ctas < full ? ctas : full);
    }
    const int64_t most = 152 * bwd_per_sm(H);
    return (int)(N < most ? N : most);
}

template <typename T, int MODE, int VPT>
cudaError_t launch_ring(RingArgs& q, int threads, size_t smem, cudaStream_t s) {
    auto* k = q.n.dh ? ce_rmsnorm_bwd_kernel<T, VPT, MODE, true> : ce_rmsnorm_bwd_kernel<T, VPT, MODE, false>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem); e != cudaSuccess) return e;
    k<<<bwd_grid(q.n.N, q.n.H), threads, smem, s>>>(q);
    return cudaGetLastError();
}

// The widest row that the ring kernel takes: 512 threads' registers, and two row
// sets in shared memory.
template <typename T, int MODE>
cudaError_t launch_bwd_m(const NormBwdArgs& a, bool* shifted, cudaStream_t s) {
    constexpr int ES = sizeof(T);
    constexpr int VEC = MODE == kLoose ? 1 : 16 / ES;
    constexpr int M = MODE == kLoose ? 4 : (VEC == 8 ? 1 : 2);  // a step of vectors per thread: 8 elements, 4 if loose
    const int64_t nv = MODE == kPhased ? (a.H + VEC - 1 + VEC - 1) / VEC : a.H / VEC;
    RingArgs q;
    q.n = a;
    q.slot = (int)((a.H * ES + 15) / 16 * 16 + (MODE == kOnGrid ? 0 : 16));
    const int64_t set = (int64_t)q.slot * (a.dh ? 3 : 2);
    int64_t room = 216 * 1024 / bwd_per_sm(a.H);
    if (room < 3 * set) room = 216 * 1024;
    q.stages = (int)(room / set < 8 ? room / set : 8);
    if (q.stages >= 2 && nv <= 512 * 4 * M) {
        *shifted = MODE == kPhased;
        const size_t smem = (size_t)q.stages * set;
        const auto th = [&](int v) { return (int)((nv + 32 * v - 1) / (32 * v) * 32); };
        if (nv <= 256 * M) return launch_ring<T, MODE, M>(q, th(M), smem, s);
        if (nv <= 1024 * M) return launch_ring<T, MODE, 2 * M>(q, th(2 * M), smem, s);
        return launch_ring<T, MODE, 4 * M>(q, th(4 * M), smem, s);
    }
    constexpr int WV = MODE == kOnGrid ? VEC : 1;
    ce_rmsnorm_bwd_wide_kernel<T, WV><<<bwd_grid(a.N, a.H), 512, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int EPL>
cudaError_t launch_short(const NormBwdArgs& a, int vb, cudaStream_t s) {
    constexpr int FULL = 16 / (int)sizeof(T) < EPL ? 16 / (int)sizeof(T) : EPL;
    auto* k = vb == 16                  ? ce_rmsnorm_bwd_short_kernel<T, EPL, FULL>
              : vb == 4 && sizeof(T) == 2 ? ce_rmsnorm_bwd_short_kernel<T, EPL, sizeof(T) == 2 ? 2 : 1>
                                          : ce_rmsnorm_bwd_short_kernel<T, EPL, 1>;
    k<<<bwd_grid(a.N, a.H), kShortWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd_t(const NormBwdArgs& a, int vb, bool* shifted, cudaStream_t s) {
    if (a.H <= 128) return launch_short<T, 4>(a, vb, s);
    if (a.H <= 256) return launch_short<T, 8>(a, vb, s);
    if (a.H <= kShortWidth) return launch_short<T, 16>(a, vb, s);
    if (vb == 16) return launch_bwd_m<T, kOnGrid>(a, shifted, s);
    auto at = [](const void* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u); };
    const bool many = a.N > 1;
    bool phased = at(a.g) == at(a.h) && at(a.dx) == at(a.h) && (!a.dh || at(a.dh) == at(a.h));
    if (many)
        phased = phased && (a.gs - a.hs) % 16 == 0 && (a.dxs - a.hs) % 16 == 0 && (!a.dh || (a.dhs - a.hs) % 16 == 0);
    if (phased) return launch_bwd_m<T, kPhased>(a, shifted, s);
    return launch_bwd_m<T, kLoose>(a, shifted, s);
}

constexpr int64_t kMaxWidth = 1 << 20;

bool bad_dtype(int d) { return d < CE_F32 || d > CE_F16; }
bool off_grid(const void* p, int es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

}  // namespace
}  // namespace gbce

using namespace gbce;

extern "C" ce_status ce_rmsnorm_fwd(const void* x, const void* residual, const void* weight, ce_dtype dtype,
                                    ce_dtype weight_dtype, int64_t N, int64_t H, int64_t x_stride,
                                    int64_t residual_stride, float eps, void* out, int64_t out_stride,
                                    ce_quant quant, int group_size, float* scales, void* residual_out,
                                    int64_t residual_out_stride, void* stream) {
    if (bad_dtype(dtype) || (weight_dtype != dtype && weight_dtype != CE_F32)) return CE_ERR_UNSUPPORTED_DTYPE;
    if (quant < CE_QUANT_NONE || quant > CE_QUANT_E5M2) return CE_ERR_UNSUPPORTED_DTYPE;
    if (N < 0 || N > 0x7fffffffLL || H < 1 || H > kMaxWidth) return CE_ERR_INVALID_ARG;
    if (!(eps >= 0.f && eps <= 3.4e38f)) return CE_ERR_INVALID_ARG;
    if (quant && group_size != 0 && group_size != 32 && group_size != 64 && group_size != 128)
        return CE_ERR_INVALID_ARG;
    if (!quant && (group_size != 0 || scales)) return CE_ERR_INVALID_ARG;
    if (N == 0) return CE_OK;
    if (!x || !weight || !out || (quant && !scales)) return CE_ERR_INVALID_ARG;
    if (residual && !residual_out) return CE_ERR_INVALID_ARG;
    if (out == residual_out) return CE_ERR_INVALID_ARG;
    const int es = elem_size(dtype);
    if (off_grid(x, es) || off_grid(residual, es) || off_grid(weight, elem_size(weight_dtype)) ||
        off_grid(residual_out, es) || (!quant && off_grid(out, es)) || off_grid(scales, 4))
        return CE_ERR_INVALID_ARG;
    // input rows may repeat (stride 0); output rows may not share memory
    if (x_stride < 0 || residual_stride < 0) return CE_ERR_BAD_STRIDE;
    if (N > 1 && (out_stride < H || (residual_out && residual_out_stride < H))) return CE_ERR_BAD_STRIDE;
    if (quant && (out == x || out == residual)) return CE_ERR_INVALID_ARG;
    // an output that replaces an input takes its strides
    if (N > 1 && ((out == x && out_stride != x_stride) || (out == residual && out_stride != residual_stride) ||
                  (residual_out && residual_out == x && residual_out_stride != x_stride) ||
                  (residual_out && residual_out == residual && residual_out_stride != residual_stride)))
        return CE_ERR_BAD_STRIDE;

    NormFwdArgs a;
    a.x = static_cast<const char*>(x);
    a.r = static_cast<const char*>(residual);
    a.w = static_cast<const char*>(weight);
    a.y = static_cast<char*>(out);
    a.h = static_cast<char*>(residual_out);
    a.scales = scales;
    a.N = N;
    a.H = H;
    const int ys = quant ? 1 : es;
    a.xs = x_stride * es;
    a.rs = residual_stride * es;
    a.ys = out_stride * ys;
    a.hs = residual_out_stride * es;
    a.eps = eps;
    a.inv_h = 1.f / (float)H;
    a.w32 = weight_dtype == CE_F32 && dtype != CE_F32;
    a.kind = quant;
    a.top = quant == CE_QUANT_E5M2 ? 57344.f : 448.f;
    a.group = quant ? (group_size ? group_size : (int)H) : (int)H;
    a.groups = (int)((H + a.group - 1) / a.group);
    const int q = es / ys;  // the output's bytes scaled to the input's vectors
    const uint64_t vals[] = {(uint64_t)(uintptr_t)x, (uint64_t)(uintptr_t)residual,
                             (uint64_t)(a.w32 ? 0 : (uintptr_t)weight),
                             (uint64_t)(uintptr_t)out * (uint64_t)q, (uint64_t)(uintptr_t)residual_out,
                             (uint64_t)(N > 1 ? a.xs : 0), (uint64_t)(N > 1 && residual ? a.rs : 0),
                             (uint64_t)(N > 1 ? a.ys * q : 0), (uint64_t)(N > 1 && residual_out ? a.hs : 0),
                             (uint64_t)H * es};
    const int vb = common_vector_bytes(vals, 10, es);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == CE_F32    ? launch_fwd_t<float>(a, vb, s)
                    : dtype == CE_BF16 ? launch_fwd_t<__nv_bfloat16>(a, vb, s)
                                       : launch_fwd_t<__half>(a, vb, s);
    return e == cudaSuccess ? CE_OK : launch_failed();
}

extern "C" size_t ce_rmsnorm_bwd_workspace_bytes(int64_t N, int64_t H) {
    if (N < 0 || N > 0x7fffffffLL || H < 1 || H > kMaxWidth) return 0;
    return kWsHeaderBytes + (size_t)bwd_grid(N, H) * (size_t)part_pitch(H) * sizeof(float);
}

extern "C" ce_status ce_rmsnorm_bwd(const void* grad_out, const void* h, const void* weight, const void* grad_h,
                                    ce_dtype dtype, ce_dtype weight_dtype, int64_t N, int64_t H,
                                    int64_t grad_out_stride, int64_t h_stride, int64_t grad_h_stride, float eps,
                                    void* grad_x, int64_t grad_x_stride, float* grad_weight, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype) || (weight_dtype != dtype && weight_dtype != CE_F32)) return CE_ERR_UNSUPPORTED_DTYPE;
    if (N < 0 || N > 0x7fffffffLL || H < 1 || H > kMaxWidth) return CE_ERR_INVALID_ARG;
    if (!(eps >= 0.f && eps <= 3.4e38f)) return CE_ERR_INVALID_ARG;
    const int es = elem_size(dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (off_grid(grad_weight, 4)) return CE_ERR_INVALID_ARG;
    if (N > 0) {
        if (!grad_out || !h || !weight || !grad_x) return CE_ERR_INVALID_ARG;
        if (off_grid(grad_out, es) || off_grid(h, es) || off_grid(grad_h, es) || off_grid(grad_x, es) ||
            off_grid(weight, elem_size(weight_dtype)))
            return CE_ERR_INVALID_ARG;
        if (grad_out_stride < 0 || h_stride < 0 || grad_h_stride < 0) return CE_ERR_BAD_STRIDE;
        if (N > 1 && grad_x_stride < H) return CE_ERR_BAD_STRIDE;
        if (N > 1 && ((grad_x == grad_out && grad_x_stride != grad_out_stride) ||
                      (grad_x == h && grad_x_stride != h_stride) ||
                      (grad_x == grad_h && grad_x_stride != grad_h_stride)))
            return CE_ERR_BAD_STRIDE;
        if (grad_weight) {
            if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return CE_ERR_INVALID_ARG;
            if (workspace_bytes < ce_rmsnorm_bwd_workspace_bytes(N, H)) return CE_ERR_WORKSPACE_TOO_SMALL;
        }
    } else {
        // no rows: the weight's gradient is an empty sum
        if (grad_weight && cudaMemsetAsync(grad_weight, 0, (size_t)H * 4, s) != cudaSuccess) return launch_failed();
        return CE_OK;
    }
    NormBwdArgs a;
    a.g = static_cast<const char*>(grad_out);
    a.h = static_cast<const char*>(h);
    a.w = static_cast<const char*>(weight);
    a.dh = static_cast<const char*>(grad_h);
    a.dx = static_cast<char*>(grad_x);
    a.part = grad_weight ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeaderBytes) : nullptr;
    a.N = N;
    a.H = H;
    a.gs = grad_out_stride * es;
    a.hs = h_stride * es;
    a.dhs = grad_h_stride * es;
    a.dxs = grad_x_stride * es;
    a.eps = eps;
    a.inv_h = 1.f / (float)H;
    a.w32 = weight_dtype == CE_F32 && dtype != CE_F32;
    const uint64_t vals[] = {(uint64_t)(uintptr_t)grad_out, (uint64_t)(uintptr_t)h, (uint64_t)(uintptr_t)grad_h,
                             (uint64_t)(uintptr_t)grad_x, (uint64_t)(N > 1 ? a.gs : 0),
                             (uint64_t)(N > 1 ? a.hs : 0), (uint64_t)(N > 1 && grad_h ? a.dhs : 0),
                             (uint64_t)(N > 1 ? a.dxs : 0), (uint64_t)H * es};
    const int vb = common_vector_bytes(vals, 9, es);
    a.err = grad_weight ? reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + kWsErrOffset) : nullptr;
    bool shifted = false;
    cudaError_t e = dtype == CE_F32    ? launch_bwd_t<float>(a, vb, &shifted, s)
                    : dtype == CE_BF16 ? launch_bwd_t<__nv_bfloat16>(a, vb, &shifted, s)
                                       : launch_bwd_t<__half>(a, vb, &shifted, s);
    if (e != cudaSuccess) return launch_failed();
    if (grad_weight) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((H + 31) / 32));
        cfg.blockDim = dim3(1024);
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        set_pdl_attr(at);
        cfg.attrs = at;
        cfg.numAttrs = 1;
        const uint32_t low = shifted ? (uint32_t)(reinterpret_cast<uintptr_t>(h) & 15u) : 0u;
        const uint32_t step = shifted && N > 1 ? (uint32_t)(a.hs & 15) : 0u;
        if (cudaLaunchKernelEx(&cfg, ce_rmsnorm_dw_kernel, (const float*)a.part, bwd_grid(N, H), H, grad_weight, low,
                               step, es) != cudaSuccess)
            return launch_failed();
    }
    return CE_OK;
}
