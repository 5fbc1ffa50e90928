// What the kernels of the attention over the 4-bit cache share beside the plan: the cache and its codes.
#pragma once

#include "cf_attn_plan.h"
#include "cf_kv4.h"

namespace cf {
namespace {

using AttnArgs = PagedArgs<KvCache>;

// A workgroup takes at least so many units of 32 keys, or joining would cost more than it saves.
constexpr int kMinUnits = 8;

// bf16 pair of byte B of codes c.
template <int B>
__device__ __forceinline__ uint32_t to_bf16(uint32_t c, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, B));
}
template <int B>
__device__ __forceinline__ uint32_t to_f16(uint32_t c, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, B));
}

// What V's codes are multiplied as: fp16 beside the fp16 probabilities of bf16 queries, bf16 beside three parts.
template <typename T, int B>
__device__ __forceinline__ uint32_t decode4(uint32_t c, float s) {
    if constexpr (sizeof(T) == 4)
        return to_bf16<B>(c, s);
    else
        return to_f16<B>(c, s);
}

}  // namespace
}  // namespace cf
