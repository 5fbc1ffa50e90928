// What the kernels of the attention over the 4-bit cache share: a call's arguments, which keys a row
// sees, and how the work is cut.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf.h"
#include "cf_internal.h"
#include "cf_kv4.h"
#include "cf_rows.h"

namespace cf {
namespace {

typedef _Float16 vh8 __attribute__((ext_vector_type(8)));
typedef float vf16 __attribute__((ext_vector_type(16)));
typedef uint32_t vu4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnit = 32;  // keys
constexpr int kUnitsOfGpu = 256;  // compute units
// A workgroup takes at least so many units, or joining would cost more than it saves.
constexpr int kMinUnits = 8;
// p = 2^(x - m + kLift) where m is at most kSlack below the row's largest score so far: the
// reference moves, and O is rescaled, only when a score exceeds it by more.  p stays below
// 2^(kLift + kSlack) < 65504, and the lift keeps the fp16 of small p off the subnormals.
constexpr float kLift = 7.f, kSlack = 8.f;
// With P in fp16 the reference falls too, where a whole tile's largest p is below 2^-kDrop, fp16's smallest
// normal number: behind a key that outweighs the rest, their p would be subnormals or zero (a tail e^-22 below
// lost 13% in 16385 keys, one e^-26 below half or more).  So a p is off by at most 2^-11 of itself or of its
// tile's largest.  Queries and keys with channels 20 times the others' meet falls in many tiles: 4096 over 16384
// keys take 4% more with them, 2925 over 17550 2.7% (kDrop 10: 1% more again), few rows up to 3%.  It falls at most
// kDeep below its highest: O, 2^(kLift + kSlack + kDeep) times 2^31 keys times 2^16, fits fp32.
constexpr float kDrop = 14.f, kDeep = 60.f;
constexpr float kNone = -__builtin_inff();

struct AttnArgs {
    RowSet q, out;
    KvCache cache;
    const int32_t* table;
    int width;  // pages of a table row
    const int32_t* kv_lens;
    const int32_t* q_starts;  // or null: q_each queries for each sequence
    int total_q, q_each;
    int batch, q_heads, share;  // share: query heads of a K/V head
    int causal, window;
    float scale_log2;
    float* lse;
    float* part;    // partial O, m and sum
    int32_t* joins; // what each workgroup leaves to be joined, kJoin numbers each
    int groups;
};

// What a workgroup with an item's last units, but not its first, leaves for the second kernel: the workgroup
// with its first (-1 where there is nothing to join), the K/V head, the sequence's first query
// token, the item's first row and its rows.
constexpr int kJoin = 8;

// One sequence's rows and keys.
struct Seq {
    int q0, nq;  // query tokens
    int len;     // keys
};

// Loads through the scalar cache: the address is the same in every lane, and nothing writes there
// while the kernel runs.
__device__ __forceinline__ int32_t scalar_load(const int32_t* p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(reinterpret_cast<uintptr_t>(p));
}

__device__ __forceinline__ Seq cut_seq(const AttnArgs& p, int len, int lo, int hi) {
    Seq s;
    s.len = min(max(len, 0), p.width << p.cache.shift);
    s.q0 = min(max(lo, 0), p.total_q);
    s.nq = min(max(hi, s.q0), p.total_q) - s.q0;
    return s;
}

// b differs from lane to lane.
__device__ __forceinline__ Seq seq_of(const AttnArgs& p, int b) {
    const int len = p.kv_lens[b];
    if (p.q_starts) return cut_seq(p, len, p.q_starts[b], p.q_starts[b + 1]);
    return cut_seq(p, len, b * p.q_each, (b + 1) * p.q_each);
}

// b is the same in every lane.
__device__ __forceinline__ Seq seq_at(const AttnArgs& p, int b) {
    const int len = scalar_load(p.kv_lens + b);
    if (p.q_starts) return cut_seq(p, len, scalar_load(p.q_starts + b), scalar_load(p.q_starts + b + 1));
    return cut_seq(p, len, b * p.q_each, (b + 1) * p.q_each);
}

// Keys [lo, hi) that a query token sees; hi may be below lo.
__device__ __forceinline__ int seen_lo(const AttnArgs& p, const Seq& s, int token) {
    return p.window ? static_cast<int>(max(int64_t(s.len) - s.nq + token - p.window + 1, int64_t(0))) : 0;
}
__device__ __forceinline__ int seen_hi(const AttnArgs& p, const Seq& s, int token) {
    return p.causal ? min(s.len - s.nq + token + 1, s.len) : s.len;
}

// Row r of a sequence's rows for one K/V head: query token and query head.
__device__ __forceinline__ int token_of(const AttnArgs& p, int row) {
    return p.share == 1 ? row : static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(p.share));
}

// Units [u0, u0 + n) of an item; at least one, so that rows that see nothing are written too.
template <int ROWS, int UNIT>
__device__ __forceinline__ int units_of(const AttnArgs& p, const Seq& s, int tile, int* u0) {
    const int rows = s.nq * p.share;
    const int lo = seen_lo(p, s, token_of(p, tile * ROWS));
    const int hi = seen_hi(p, s, token_of(p, min(tile * ROWS + ROWS, rows) - 1));
    *u0 = lo / UNIT;
    return max((hi + UNIT - 1) / UNIT - *u0, 1);
}

template <int ROWS>
__device__ __forceinline__ int tiles_of(const AttnArgs& p, const Seq& s) {
    return (s.nq * p.share + ROWS - 1) / ROWS;
}

__device__ __forceinline__ int64_t uniform(int64_t v) { return wave_uniform(v); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
    const int lo = __shfl(static_cast<int>(v), lane, 64), hi = __shfl(static_cast<int>(v >> 32), lane, 64);
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo));
}

// Sum of v over the lanes up to this one, in 32 bits: within rows of 16 lanes, and then from row to row.
__device__ __forceinline__ uint32_t wave_scan32(uint32_t v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // one lane up
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row 0's last to row 1, 2's to 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row 1's last to rows 2 and 3
    return v;
}

// Inclusive sums over the wave's lanes, of values that are not negative.
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
    if (__all(v < int64_t(1) << 25)) return wave_scan32(static_cast<uint32_t>(v));
    const int lane = threadIdx.x & 63;
#pragma unroll 1
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t x = shfl64(v, lane - d);
        if (lane >= d) v += x;
    }
    return v;
}

// Where a workgroup's run of the work begins, and its length.  An item costs its units and PAD
// more: what starting and finishing one takes, in units.
struct Place {
    int me;  // which run
    int64_t at, end, chunk;
    int b, head, tile;
    int64_t rest;  // of at, from the item's start
};

// Every wave works it out by itself: a group of lanes takes a sequence and shares its tiles.
template <int ROWS, int UNIT, int PAD>
__device__ __forceinline__ bool place_of(const AttnArgs& p, Place* x) {
    const int lane = threadIdx.x & 63;
    int sub = 64;  // lanes of a sequence
    while (sub > 1 && 64 / sub < p.batch) sub >>= 1;
    const int each = 64 / sub;
    const auto head_cost = [&](int b) -> int64_t {
        int64_t n = 0;
        int tiles = 0;
        if (b < p.batch) {
            const Seq s = seq_of(p, b);
            tiles = tiles_of<ROWS>(p, s);
            int u0;
            for (int i = lane & (sub - 1); i < tiles; i += sub) n += units_of<ROWS, UNIT>(p, s, i, &u0) + PAD;
        }
        if (__all(tiles <= 1)) return shfl64(n, lane & ~(sub - 1));
        for (int d = 1; d < sub; d <<= 1) n += shfl64(n, lane ^ d);
        return n;
    };
    // with up to 64 sequences one round does it, and its sums are kept
    int64_t total = 0, own = 0, sum = 0;
    for (int b0 = 0; b0 < p.batch; b0 += each) {
        own = head_cost(b0 + lane / sub);
        sum = wave_scan((lane & (sub - 1)) == 0 ? own * p.cache.heads : 0);
        total += uniform(shfl64(sum, 63));
    }
    int64_t chunk = (total + p.groups - 1) / p.groups;
    chunk = max(chunk, int64_t(kMinUnits * kUnit / UNIT + PAD));
    x->chunk = chunk;
    // Workgroups are dealt to the eight XCDs in turn.  Neighbours in the order of the work share keys:
    // each XCD takes an eighth of the runs there are, side by side, and so one part of L2's keys.
    const int each_xcd = static_cast<int>((total + chunk - 1) / chunk + 7) / 8;
    const int bid = blockIdx.x;
    x->me = bid < 8 * each_xcd ? (bid & 7) * each_xcd + (bid >> 3) : bid;
    x->at = x->me * chunk;
    x->end = min(x->at + chunk, total);
    if (x->at >= x->end) return false;
    int64_t before = 0;
    int b0 = 0;
    if (p.batch > each) {
        for (;; b0 += each) {
            own = head_cost(b0 + lane / sub);
            sum = wave_scan((lane & (sub - 1)) == 0 ? own * p.cache.heads : 0);
            const int64_t all = before + uniform(shfl64(sum, 63));
            if (x->at < all) break;  // at < total, so some round gets here
            before = all;
        }
    }
    const int at_lane = __builtin_ctzll(__ballot(x->at < before + sum));  // a sequence's first lane
    x->b = uniform(b0 + at_lane / sub);
    const int64_t per_head = uniform(shfl64(own, at_lane));
    int64_t rest = x->at - before - uniform(shfl64(sum, at_lane)) + per_head * p.cache.heads;
    if ((rest | per_head) >> 31 == 0)
        x->head = uniform(static_cast<int>(static_cast<uint32_t>(rest) / static_cast<uint32_t>(per_head)));
    else
        x->head = uniform(static_cast<int>(rest / per_head));
    rest -= x->head * per_head;
    const Seq s = seq_at(p, x->b);
    const int tiles = tiles_of<ROWS>(p, s);
    if (tiles == 1) {
        x->tile = 0;
        x->rest = rest;
        return true;
    }
    for (int t0 = 0;; t0 += 64) {
        int u0;
        const int cost = t0 + lane < tiles ? units_of<ROWS, UNIT>(p, s, t0 + lane, &u0) + PAD : 0;
        const int64_t upto = wave_scan(cost);
        const int64_t all = uniform(shfl64(upto, 63));
        if (rest < all) {
            const int i = __builtin_ctzll(__ballot(rest < upto));
            x->tile = uniform(t0 + i);
            x->rest = rest - uniform(shfl64(upto - cost, i));
            return true;
        }
        rest -= all;
    }
}

// v over the lanes n, n + 16, n + 32, n + 48 that hold a row.
__device__ __forceinline__ float across_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float across_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// The leading eight bits of an fp32 number, which it loses: three in turn are all of it.  Cut off, not
// rounded: rounded, numbers from 3.396e38 on would become infinite.
__device__ __forceinline__ __bf16 take_bf16(float* rest) {
    const uint32_t top = __float_as_uint(*rest) & 0xffff0000u;
    *rest -= __uint_as_float(top);
    return __builtin_bit_cast(__bf16, static_cast<uint16_t>(top >> 16));
}

// bf16 pair of byte B of codes c.
template <int B>
__device__ __forceinline__ uint32_t to_bf16(uint32_t c, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, B));
}
template <int B>
__device__ __forceinline__ uint32_t to_f16(uint32_t c, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, B));
}

// What probabilities and V are multiplied in.  bf16 queries: P rounded to fp16 (half a step is 2^-11 of it).
// fp32 queries: three bf16 parts that add up to P, whatever its size (two fp16 parts run out of exponents: a
// tail e^-22 below one key was 10% off, and one e^-26 below was lost).
template <typename T>
struct Prob;

template <>
struct Prob<__bf16> {
    static constexpr int kParts = 1;
    static constexpr bool kFalls = true;  // the reference
    using Frag = vh8;
    template <int K>
    static __device__ __forceinline__ void set(Frag (&f)[K], int i, float e) {
        f[0][i] = static_cast<_Float16>(e);
    }
    template <int B>
    static __device__ __forceinline__ uint32_t decode(uint32_t c, float s) {
        return to_f16<B>(c, s);
    }
    static __device__ __forceinline__ vf4 mul16(Frag a, Frag b, vf4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ vf16 mul32(Frag a, Frag b, vf16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Prob<float> {
    static constexpr int kParts = 3;
    static constexpr bool kFalls = false;
    using Frag = vb8;
    template <int K>
    static __device__ __forceinline__ void set(Frag (&f)[K], int i, float e) {
#pragma unroll
        for (int k = 0; k < K; ++k) f[k][i] = take_bf16(&e);
    }
    template <int B>
    static __device__ __forceinline__ uint32_t decode(uint32_t c, float s) {
        return to_bf16<B>(c, s);
    }
    static __device__ __forceinline__ vf4 mul16(Frag a, Frag b, vf4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ vf16 mul32(Frag a, Frag b, vf16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

// Where a row's reference goes: up to its tile's largest score, in units of log2, where that is above it (lowered
// by kLift); down to it, with P in fp16, from far above; high is the highest it has been.
template <typename T>
__device__ __forceinline__ float next_ref(float top, float m, float* high) {
    float r = fmaxf(top - kLift, m);
    if constexpr (Prob<T>::kFalls) {
        // a tile that the row sees nothing of moves nothing
        if (top < m - kDrop && top > kNone) r = fmaxf(top - kLift, *high - kDeep);
        *high = fmaxf(*high, r);
    }
    return r;
}

// log sum exp of a row from its reference, in units of log2, and its sum.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? kNone : (m + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Whether a page number names a page of the cache (a sequence without keys has none).
__device__ __forceinline__ bool page_on(const AttnArgs& p, const Seq& s, int page) {
    return s.len > 0 && static_cast<uint32_t>(page) < static_cast<uint32_t>(p.cache.pages);
}

}  // namespace
}  // namespace cf
