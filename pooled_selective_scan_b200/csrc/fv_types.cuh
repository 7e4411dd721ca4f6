// fv_types.cuh -- element types of the operators that take more than fp32, and their vector accesses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fv {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

// Two values packed into 32 bits, rounded to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// V consecutive values as fp32; p aligned to their size, up to 16 bytes.  STREAM: read once, evict first.
template <typename T, int V, bool STREAM>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4* q = reinterpret_cast<const float4*>(p + i);
            const float4 v = STREAM ? __ldcs(q) : __ldg(q);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else if constexpr (V == 8) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        const uint4 v = STREAM ? __ldcs(q) : __ldg(q);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(w[i]);
            x[2 * i] = f.x; x[2 * i + 1] = f.y;
        }
    } else {
        static_assert(V == 4, "vectors of 4 or 8 values");
        const uint2* q = reinterpret_cast<const uint2*>(p);
        const uint2 v = STREAM ? __ldcs(q) : __ldg(q);
        const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y);
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            __stcs(reinterpret_cast<float4*>(p + i), make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
    } else if constexpr (V == 8) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]),
                                                       pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7])));
    } else {
        static_assert(V == 4, "vectors of 4 or 8 values");
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3])));
    }
}

// V consecutive values as they lie in memory (streamed), zeros where they are not loaded.
template <typename T, int V>
struct Raw {
    static constexpr int kWords = V * (int)sizeof(T) / 4, kVec = kWords < 4 ? kWords : 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p, bool in) {
#pragma unroll
        for (int i = 0; i < kWords; i += kVec) {
            if constexpr (kVec == 4) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (in) v = __ldcs(reinterpret_cast<const uint4*>(p) + i / 4);
                w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
            } else {
                uint2 v = make_uint2(0u, 0u);
                if (in) v = __ldcs(reinterpret_cast<const uint2*>(p));
                w[0] = v.x; w[1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void unpack(float (&x)[V]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const float2 f = unpack2<T>(w[i]);
                x[2 * i] = f.x; x[2 * i + 1] = f.y;
            }
        }
    }
};

}  // namespace fv
