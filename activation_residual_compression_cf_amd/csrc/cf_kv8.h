// The 8-bit K/V cache's block layout (the format is described at cf_kv8_append in cf.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace cf {

constexpr int kKv8Block = 16;  // tokens that share a scale
// Exponents of the scales.  Every value the cache can hold, +-448 * 2^7 down to 2^-24, is then a
// half-precision number, which is what the attention multiplies V in for bf16 queries.
constexpr int kKv8ExpMin = -15, kKv8ExpMax = 7;

// Byte offsets inside the block of one page and head: P tokens of D channels.
struct Kv8Block {
    int page, dim;
    __host__ __device__ constexpr int64_t bytes() const { return 2 * int64_t(page) * dim + (page > 128 ? page / 8 : 16); }
    __host__ __device__ constexpr int k_code(int t) const { return t * dim; }
    __host__ __device__ constexpr int v_code(int t, int c) const { return page * dim + ((t >> 3) * dim + c) * 8 + (t & 7); }
    __host__ __device__ constexpr int k_scale(int t) const { return 2 * page * dim + (t >> 4); }
    __host__ __device__ constexpr int v_scale(int t) const { return 2 * page * dim + (page >> 4) + (t >> 4); }
};

// The cache as the kernels see it.
struct Kv8Cache {
    uint8_t* data;
    int64_t pages;
    int heads;
    Kv8Block block;
    int shift;  // log2 of the page's tokens
    __device__ __forceinline__ uint8_t* at(int64_t page, int head) const {
        return data + (page * heads + head) * block.bytes();
    }
};

}  // namespace cf
