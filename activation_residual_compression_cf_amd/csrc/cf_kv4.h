// The 4-bit K/V cache's block layout (the format is described at cf_kv4_append in cf.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace cf {

constexpr int kKvGroup = 32;  // channels that share a scale
// Exponents of the scales.  Every value the cache can hold, +-6 * 2^13 down to 2^-23, is then
// a half-precision number, which is what the attention multiplies V in for bf16 queries.
constexpr int kKvExpMin = -22, kKvExpMax = 13;
constexpr uint32_t kKvNan = 255;     // scale byte of a group that holds a NaN or an infinity
constexpr uint32_t kKvNanFrom = 192; // bytes from here on read as NaN

// Byte offsets inside the block of one page and head: P tokens of D channels.
struct KvBlock {
    int page, dim;
    __host__ __device__ constexpr int64_t bytes() const { return int64_t(page) * dim * 17 / 16; }
    __host__ __device__ constexpr int k_code(int t) const { return t * (dim / 2); }
    // piece n of 16: channels n * dim/16 ..
    __host__ __device__ constexpr int v_code(int t, int n) const {
        return page * (dim / 2) + (((t >> 3) * 16 + n) * 8 + (t & 7)) * (dim / 32);
    }
    __host__ __device__ constexpr int k_scale(int t, int g) const { return page * dim + t * (dim / 32) + g; }
    __host__ __device__ constexpr int v_scale(int t, int g) const {
        return page * dim + page * (dim / 32) + ((t >> 3) * (dim / 32) + g) * 8 + (t & 7);
    }
};

// The cache as the kernels see it.
struct KvCache {
    uint8_t* data;
    int64_t pages;
    int heads;
    KvBlock block;
    int shift;  // log2 of the page's tokens
    __device__ __forceinline__ uint8_t* at(int64_t page, int head) const {
        return data + (page * heads + head) * block.bytes();
    }
};

}  // namespace cf
