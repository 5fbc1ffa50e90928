// What the attention kernels over the 8-bit cache share beside the plan: the cache's codes.
#pragma once

#include "cf_attn_plan.h"
#include "cf_kv8.h"

namespace cf {
namespace {

using Attn8Args = PagedArgs<Kv8Cache>;

// Bit 7 of each of four codes that reads NaN (magnitude bits all set).
__device__ __forceinline__ uint32_t nan_codes(uint32_t c) { return ((c & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// From bits 7 of bytes: the bytes in full, and four bits.
__device__ __forceinline__ uint32_t full_bytes(uint32_t b) { return (b >> 7) * 0xffu; }
__device__ __forceinline__ uint32_t four_bits(uint32_t b) { return (b >> 7 & 1u) | (b >> 14 & 2u) | (b >> 21 & 4u) | (b >> 28 & 8u); }

// Eight codes as eight values.
__device__ __forceinline__ vb8 bf16_codes(uint32_t lo, uint32_t hi, float s) {
    const vu4 w{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true))};
    return __builtin_bit_cast(vb8, w);
}
__device__ __forceinline__ vh8 f16_codes(uint32_t lo, uint32_t hi, float s) {
    const vu4 w{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, true))};
    return __builtin_bit_cast(vh8, w);
}

// V's codes as what they are multiplied in (Prob has the reasons).
template <typename T>
struct Codes8 {
    static __device__ __forceinline__ vh8 frag(uint32_t lo, uint32_t hi, float s) { return f16_codes(lo, hi, s); }
};
template <>
struct Codes8<float> {
    static __device__ __forceinline__ vb8 frag(uint32_t lo, uint32_t hi, float s) { return bf16_codes(lo, hi, s); }
};

}  // namespace
}  // namespace cf
