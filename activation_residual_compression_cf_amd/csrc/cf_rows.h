// Device helpers of the operators on rows of heads: row addresses by token and head, and
// eight channels of a row as bf16 or fp32.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf_internal.h"
#include "cf_vec.h"

namespace cf {

typedef __bf16 vb2 __attribute__((ext_vector_type(2)));
typedef __bf16 vb8 __attribute__((ext_vector_type(8)));

template <typename T>
__device__ __forceinline__ T* row_ptr(const RowSet& r, int64_t token, int head) {
    return static_cast<T*>(r.data) + token * r.token_stride + head * r.head_stride;
}

// Eight consecutive channels; loads and stores are 16 bytes wide.
template <typename T>
struct Row8;

template <>
struct Row8<__bf16> {
    vb8 v;
    __device__ __forceinline__ void load(const __bf16* p) { v = *reinterpret_cast<const vb8*>(p); }
    __device__ __forceinline__ void store(__bf16* p) const { *reinterpret_cast<vb8*>(p) = v; }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(v[i]);
    }
    // rounds to nearest, ties to even; NaN stays NaN
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = static_cast<__bf16>(x[i]);
    }
};

template <>
struct Row8<float> {
    vf4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const vf4*>(p);
        b = *reinterpret_cast<const vf4*>(p + 4);
    }
    __device__ __forceinline__ void store(float* p) const {
        *reinterpret_cast<vf4*>(p) = a;
        *reinterpret_cast<vf4*>(p + 4) = b;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = a[i], x[i + 4] = b[i];
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = x[i], b[i] = x[i + 4];
    }
};

}  // namespace cf
