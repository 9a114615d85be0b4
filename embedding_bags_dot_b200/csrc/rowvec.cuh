// Runs of VEC consecutive row elements of type T, widened to fp32 on load and
// rounded once (to nearest) on store. A run is one access of VEC * sizeof(T)
// bytes, or several of 16; its address is a multiple of min(16, VEC * sizeof(T)).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dlrm {

template <int BYTES> struct RawBytes;
template <> struct RawBytes<1> { using t = uint8_t; };
template <> struct RawBytes<2> { using t = uint16_t; };
template <> struct RawBytes<4> { using t = uint32_t; };
template <> struct RawBytes<8> { using t = uint2; };
template <> struct RawBytes<16> { using t = uint4; };

// Two neighbouring elements at a time: one instruction widens or rounds both.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 to_f(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t from_f(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <> struct Pair<__half> {
    static __device__ __forceinline__ float2 to_f(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
    static __device__ __forceinline__ uint32_t from_f(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// The stored form of a run: kept in this form while a load is in flight (half the registers of fp32).
template <typename T, int VEC>
struct RowRaw {
    static constexpr int BYTES = VEC * (int)sizeof(T);
    static constexpr int ACC = BYTES < 16 ? BYTES : 16;   // bytes per access
    static constexpr int NA = BYTES / ACC;
    union {
        typename RawBytes<ACC>::t a[NA];
        T e[VEC];
        uint32_t w[BYTES < 4 ? 1 : BYTES / 4];
    };
    static constexpr bool PAIRS = sizeof(T) == 2 && VEC >= 2;
    __device__ __forceinline__ RowRaw() {}
    __device__ __forceinline__ void load(const T* p) {
        const typename RawBytes<ACC>::t* q = reinterpret_cast<const typename RawBytes<ACC>::t*>(p);
#pragma unroll
        for (int i = 0; i < NA; ++i) a[i] = q[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = Cvt<T>::from_f(0.f);
    }
    __device__ __forceinline__ void get(float (&v)[VEC]) const {
        if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const float2 f = Pair<T>::to_f(w[i / 2]);
                v[i] = f.x;
                v[i + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = Cvt<T>::to_f(e[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[VEC]) {
        if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) w[i / 2] = Pair<T>::from_f(v[i], v[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) e[i] = Cvt<T>::from_f(v[i]);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        typename RawBytes<ACC>::t* q = reinterpret_cast<typename RawBytes<ACC>::t*>(p);
#pragma unroll
        for (int i = 0; i < NA; ++i) q[i] = a[i];
    }
};

// VEC fp32 values as e4m3 codes (round to nearest even; magnitudes beyond 448 become 448, NaN stays NaN).
template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = (uint8_t)__nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        union {
            __nv_fp8x2_storage_t h[VEC / 2];
            typename RawBytes<VEC>::t w;
        } u;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            u.h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<typename RawBytes<VEC>::t*>(p) = u.w;
    }
}

// Whether p and a row pitch (bytes) keep every row on a multiple of `bytes` (a power of two).
inline bool rows_on(const void* p, long long pitch, int bytes) {
    return ((((uintptr_t)p) | (uintptr_t)pitch) & (uintptr_t)(bytes - 1)) == 0;
}

// Streaming multiprocessors of the current device (asked once per device).
inline int device_sms() {
    static int n[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return 148;
    if (!n[dev]) {
        int v = 0;
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        n[dev] = v > 0 ? v : 148;
    }
    return n[dev];
}

}  // namespace dlrm
