// Device-side pieces of the dense operators (products, activations, their
// gradients): element conversion, activations.
#pragma once

#include "common.hpp"

namespace moe {

// An offset past the end of any buffer resource: a load there returns zeros and
// touches no memory.
constexpr uint32_t kOutside = 0x80000000u;

// ---- element types ---------------------------------------------------------

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(__bf16 v) { return (float)v; }

// one rounding to nearest even (none for float)
template <typename T> __device__ __forceinline__ T from_f32(float v) { return (T)v; }

// N consecutive elements as floats. The address is a multiple of the vector's size.
template <typename T, int N> struct Vec {
    typedef T type __attribute__((ext_vector_type(N)));
    static __device__ __forceinline__ void load(const T *p, float (&v)[N])
    {
        const type x = *reinterpret_cast<const type *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = to_f32(x[i]);
    }
    template <bool NT = false>  // NT: non-temporal
    static __device__ __forceinline__ void store(T *p, const float (&v)[N])
    {
        type x;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = from_f32<T>(v[i]);
        if constexpr (NT)
            __builtin_nontemporal_store(x, reinterpret_cast<type *>(p));
        else
            *reinterpret_cast<type *>(p) = x;
    }
};

// 8 elements at a 16-byte aligned address. NT: stored non-temporally
template <typename T> __device__ __forceinline__ void load8(const T *p, float (&v)[8])
{
    if constexpr (sizeof(T) == 2) {
        Vec<T, 8>::load(p, v);
    } else {
        float a[4], b[4];
        Vec<T, 4>::load(p, a);
        Vec<T, 4>::load(p + 4, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}
template <typename T, bool NT = false>
__device__ __forceinline__ void store8(T *p, const float (&v)[8])
{
    if constexpr (sizeof(T) == 2) {
        Vec<T, 8>::template store<NT>(p, v);
    } else {
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        Vec<T, 4>::template store<NT>(p, a);
        Vec<T, 4>::template store<NT>(p + 4, b);
    }
}

// ---- activations (in 32 bits) ----------------------------------------------
// silu(z) = z s, s = 1 / (1 + e^-z); gelu(z) = z Phi(z), Phi(z) = erfc(-z / sqrt 2) / 2
// (erfc, not 1 + erf: for negative z the sum would cancel). NaN stays NaN.

enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

__device__ __forceinline__ float act_apply(float z, int act)
{
    switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;
    case kActSilu: return z / (1.f + expf(-z));
    case kActGelu: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    default: return z;
    }
}

// a = act(z), the return value act'(z):
//   relu' = [z > 0]; silu' = s (1 + z (1 - s)); gelu' = Phi(z) + z phi(z)
__device__ __forceinline__ float act_slope(float z, int act, float &a)
{
    switch (act) {
    case kActRelu: a = z < 0.f ? 0.f : z; return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    case kActSilu: {
        const float s = 1.f / (1.f + expf(-z));
        a = z * s;
        return s * (1.f + z * (1.f - s));
    }
    case kActGelu: {
        const float c = 0.5f * erfcf(-0.70710678118654752f * z);
        a = z * c;
        return c + z * (0.39894228040143268f * expf(-0.5f * z * z));
    }
    default: a = z; return 1.f;
    }
}

}  // namespace moe
