// cf_kv4.hip - writer and reader of the 4-bit K/V cache.
//
// A group of 32 channels is held as 32 E2M1 codes and the exponent e of one scale:
//   e = the least integer with max|x| <= 6 * 2^e, within [-22, 13]
//   code = the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6} to x * 2^-e, ties to the even code;
//          above 6 (only where e is at its upper end) 6
// x * 2^-e is exact, so the codes are too: the same for fp32 and bf16 rows of equal values.
//
// Bound by memory: 2 * D * (2 or 4) bytes of rows in, 2 * D * 17/32 bytes out, per token and
// head, and the reverse for the reader.  17550 tokens of 30 heads of 64 in bf16: 47 us in (171 MB,
// 3.6 TB/s where the best copy reaches 6.2: at 64 channels V's codes leave two bytes at a time)
// and 29 us back, from the last-level cache; 1024 tokens of 24 heads of 128 in fp32 7 and 9 us.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf.h"
#include "cf_internal.h"
#include "cf_kv4.h"
#include "cf_rows.h"

namespace cf {
namespace {

constexpr int kThreads = 256;

struct StoreArgs {
    RowSet k, v;
    const int64_t* slots;
    int64_t tokens;
    KvCache cache;
};

// Eight channels a lane, four lanes a group: the group's scale byte, and the lane's codes.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], uint32_t* byte) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1, 64)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2, 64)));
    // bit patterns of magnitudes order as the magnitudes do, and NaN above infinity
    if (top >= 0x7f800000u) {
        *byte = kKvNan;
        return 0;
    }
    // top = 1.m * 2^(E - 127); 6 = 1.5 * 2^2
    int e = static_cast<int>(top >> 23) - 127 - 2 + ((top & 0x7fffffu) > 0x400000u);
    e = min(max(e, kKvExpMin), kKvExpMax);
    *byte = static_cast<uint32_t>(e + 127);
    // the conversion divides by the scale, rounds to nearest even and saturates
    const float s = __uint_as_float(*byte << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
    return c;
}

// D/8 lanes a row; the rows of a block are consecutive tokens of one head, so that the codes
// of V, which lie eight tokens together, leave a wave in runs.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void append_kernel(const StoreArgs p) {
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int head = blockIdx.y;
    const int64_t t = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes;
    if (t >= p.tokens) return;
    const int64_t slot = p.slots[t];
    const int64_t page = slot >> p.cache.shift;
    if (slot < 0 || page >= p.cache.pages) return;
    const int in = static_cast<int>(slot - page * p.cache.block.page);
    const KvBlock blk{p.cache.block.page, D};
    uint8_t* const base = p.cache.data + (page * p.cache.heads + head) * blk.bytes();

    Row8<T> kr, vr;
    kr.load(row_ptr<T>(p.k, t, head) + lane * 8);
    vr.load(row_ptr<T>(p.v, t, head) + lane * 8);
    float x[8];
    uint32_t byte;
    kr.get(x);
    const uint32_t kc = quantize8(x, &byte);
    *reinterpret_cast<uint32_t*>(base + blk.k_code(in) + lane * 4) = kc;
    if ((lane & 3) == 0) base[blk.k_scale(in, lane / 4)] = static_cast<uint8_t>(byte);
    vr.get(x);
    const uint32_t vc = quantize8(x, &byte);
    if constexpr (D == 128) {
        *reinterpret_cast<uint32_t*>(base + blk.v_code(in, lane)) = vc;
    } else {
        static_assert(D == 64);
        *reinterpret_cast<uint16_t*>(base + blk.v_code(in, 2 * lane)) = static_cast<uint16_t>(vc);
        *reinterpret_cast<uint16_t*>(base + blk.v_code(in, 2 * lane + 1)) = static_cast<uint16_t>(vc >> 16);
    }
    if ((lane & 3) == 0) base[blk.v_scale(in, lane / 4)] = static_cast<uint8_t>(byte);
}

// The eight values of a lane's codes.
__device__ __forceinline__ void values8(uint32_t c, uint32_t byte, float (&x)[8]) {
    typedef float vf2 __attribute__((ext_vector_type(2)));
    const bool nan = byte >= kKvNanFrom;
    const float s = __uint_as_float(byte << 23);
    const vf2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    const vf2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    const vf2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
    const vf2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    const float y[8] = {a.x, a.y, b.x, b.y, d.x, d.y, e.x, e.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = nan ? __builtin_nanf("") : y[i];
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(const StoreArgs p) {
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int head = blockIdx.y;
    const int64_t t = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes;
    if (t >= p.tokens) return;
    const int64_t slot = p.slots[t];
    const int64_t page = slot >> p.cache.shift;
    float k[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.f;
    if (slot >= 0 && page < p.cache.pages) {
        const int in = static_cast<int>(slot - page * p.cache.block.page);
        const KvBlock blk{p.cache.block.page, D};
        const uint8_t* const base = p.cache.data + (page * p.cache.heads + head) * blk.bytes();
        const uint32_t kc = *reinterpret_cast<const uint32_t*>(base + blk.k_code(in) + lane * 4);
        uint32_t vc;
        if constexpr (D == 128) {
            vc = *reinterpret_cast<const uint32_t*>(base + blk.v_code(in, lane));
        } else {
            vc = *reinterpret_cast<const uint16_t*>(base + blk.v_code(in, 2 * lane)) |
                 uint32_t(*reinterpret_cast<const uint16_t*>(base + blk.v_code(in, 2 * lane + 1))) << 16;
        }
        values8(kc, base[blk.k_scale(in, lane / 4)], k);
        values8(vc, base[blk.v_scale(in, lane / 4)], v);
    }
    Row8<T> r;
    r.set(k);
    r.store(row_ptr<T>(p.k, t, head) + lane * 8);
    r.set(v);
    r.store(row_ptr<T>(p.v, t, head) + lane * 8);
}

template <typename T, int D>
void launch_rows(bool read, const StoreArgs& p, hipStream_t stream) {
    constexpr int kRows = kThreads / (D / 8);
    const dim3 grid(static_cast<uint32_t>((p.tokens + kRows - 1) / kRows), p.cache.heads);
    if (read)
        read_kernel<T, D><<<grid, kThreads, 0, stream>>>(p);
    else
        append_kernel<T, D><<<grid, kThreads, 0, stream>>>(p);
}

hipError_t launch(bool read, int a_dtype, const StoreArgs& p, hipStream_t stream) {
    if (a_dtype == CF_BF16)
        p.cache.block.dim == 64 ? launch_rows<__bf16, 64>(read, p, stream) : launch_rows<__bf16, 128>(read, p, stream);
    else
        p.cache.block.dim == 64 ? launch_rows<float, 64>(read, p, stream) : launch_rows<float, 128>(read, p, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(int a_dtype, const RowSet& k, const RowSet& v, const int64_t* slots, int64_t tokens,
                             const KvCache& cache, hipStream_t stream) {
    return launch(false, a_dtype, StoreArgs{k, v, slots, tokens, cache}, stream);
}

hipError_t launch_kv4_read(int a_dtype, const RowSet& k, const RowSet& v, const int64_t* slots, int64_t tokens,
                           const KvCache& cache, hipStream_t stream) {
    return launch(true, a_dtype, StoreArgs{k, v, slots, tokens, cache}, stream);
}

}  // namespace cf
