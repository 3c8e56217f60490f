// ce_pack.cuh -- runs of VEC elements moved in one load or store, for the
// operators whose rows may sit on any multiple of the element size (the norm,
// the embedding rows): VEC * sizeof(T) is 16 bytes when base, stride and width
// allow it, else 4 bytes or one element.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gbce {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(__half& d, float x) { d = __float2half_rn(x); }

template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<1> { using type = uint8_t; };

template <typename T, int VEC>
union Pack {
    using Raw = typename RawOf<sizeof(T) * VEC>::type;
    Raw raw;
    T v[VEC];
    __device__ __forceinline__ Pack() {}
    __device__ __forceinline__ void zero() {
        Raw z = {};
        raw = z;
    }
    // data read once: streamed past L1
    __device__ __forceinline__ void load_cs(const void* p) { raw = __ldcs(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void load(const void* p) { raw = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ void load_nc(const void* p) { raw = __ldg(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<Raw*>(p) = raw; }
    __device__ __forceinline__ void store_cs(void* p) const { __stcs(reinterpret_cast<Raw*>(p), raw); }
    __device__ __forceinline__ float f(int i) const { return to_f32(v[i]); }
    __device__ __forceinline__ void set(int i, float x) { from_f32(v[i], x); }
};

// VEC floats at p: p is a multiple of 16 bytes when VEC is a multiple of 4
template <int VEC>
__device__ __forceinline__ void store_f32(float* p, const float* x) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = x[i];
    }
}
template <int VEC>
__device__ __forceinline__ void load_f32(const float* p, float* x) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = p[i];
    }
}

// The 16 bytes that start `ph` bytes into the two 16-byte vectors a, b (rows that
// lie at different offsets from 16 bytes).
__device__ __forceinline__ uint4 shift_bytes(uint4 a, uint4 b, uint32_t ph) {
    uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (ph & 8u) {
#pragma unroll
        for (int k = 0; k < 6; ++k) r[k] = r[k + 2];
    }
    if (ph & 4u) {
#pragma unroll
        for (int k = 0; k < 5; ++k) r[k] = r[k + 1];
    }
    const uint32_t s = (ph & 3u) * 8u;
    return make_uint4(__funnelshift_r(r[0], r[1], s), __funnelshift_r(r[1], r[2], s),
                      __funnelshift_r(r[2], r[3], s), __funnelshift_r(r[3], r[4], s));
}

// Widest run of elements (in bytes) that divides every given address or byte stride.
inline int common_vector_bytes(const uint64_t* vals, int n, int es) {
    uint64_t all = 0;
    for (int i = 0; i < n; ++i) all |= vals[i];
    if (all % 16 == 0) return 16;
    if (es == 2 && all % 4 == 0) return 4;
    return es;
}

}  // namespace gbce
