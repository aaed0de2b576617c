// What the norms share: vectors of a row, at any element address.
#pragma once

#include "common.h"

namespace sdm {

template <typename T> struct NormVec;
template <> struct NormVec<float> {
    static constexpr int V = 4;
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    static __device__ __forceinline__ void unpack(const raw &x, float (&o)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = x[j];
    }
    static __device__ __forceinline__ raw part(const float *p, int n) {   // the first n elements, zeros after them
        raw x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = j < n ? p[j] : 0.0f;
        return x;
    }
    static __device__ __forceinline__ void load(const float *p, float (&o)[4]) { unpack(*reinterpret_cast<const raw *>(p), o); }
    static __device__ __forceinline__ void store(float *p, const float (&o)[4]) {
        *reinterpret_cast<raw *>(p) = raw{o[0], o[1], o[2], o[3]};
    }
};
template <> struct NormVec<bf16> {
    static constexpr int V = 8;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    static __device__ __forceinline__ void unpack(const raw &x, float (&o)[8]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[2 * j] = __uint_as_float(x[j] << 16);
            o[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ raw part(const bf16 *p, int n) {   // the first n elements, zeros after them
        raw x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = (2 * j < n ? uint32_t(p[2 * j].bits) : 0u) | (2 * j + 1 < n ? uint32_t(p[2 * j + 1].bits) << 16 : 0u);
        return x;
    }
    static __device__ __forceinline__ void load(const bf16 *p, float (&o)[8]) { unpack(*reinterpret_cast<const raw *>(p), o); }
    static __device__ __forceinline__ void store(bf16 *p, const float (&o)[8]) {
        raw x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = f32x2_to_bf16x2(o[2 * j], o[2 * j + 1]);
        *reinterpret_cast<raw *>(p) = x;
    }
};

// V elements of type T at any element address.
template <typename T, int V> __device__ __forceinline__ void norm_load(const T *p, float (&o)[V]) {
    if constexpr (V == NormVec<T>::V) NormVec<T>::load(p, o);
    else {   // float32 parameters beside bfloat16 rows
        float a[4], b[4];
        NormVec<T>::load(p, a);
        NormVec<T>::load(p + 4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[j] = a[j];
            o[4 + j] = b[j];
        }
    }
}

// Vector i of a row of n columns at p: `fill` past its end.
template <typename T, int V>
__device__ __forceinline__ void norm_get(const T *p, int i, int n, float fill, float (&o)[V]) {
    const int c = i * V;
    if (c + V <= n) norm_load<T, V>(p + c, o);
    else {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = c + j < n ? to_f32(p[c + j]) : fill;
    }
}
template <typename T, int V> __device__ __forceinline__ void norm_put(T *p, int i, int n, const float (&o)[V]) {
    const int c = i * V;
    if (c + V <= n) NormVec<T>::store(p + c, o);
    else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < n) p[c + j] = from_f32<T>(o[j]);
    }
}

}  // namespace sdm
