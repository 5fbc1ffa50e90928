// cf_kv4_attn.hip - attention over the 4-bit K/V cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i k_j - m_i),  lse_i = m_i + log sum_j p_ij
// over the keys j that row i may see, in one pass over the keys with a running reference m
// and sum.  A row of the product is one (query token, query head); the rows of the query
// heads that share a K/V head are worked on together.
//
// What one wave does with 32 keys and 16 rows (matrix products of 16 x 16 with 32 terms;
// lane = 16 g + n):
//   S^T = K Q^T   K rows are keys; lane (g, n) holds a quarter of key row n's channels, which
//                 is one load of codes, and the codes become bf16 by the hardware's
//                 conversion with the group's scale.  Rows are keys in such an order that
//                 lane (g, n) ends up with the scores of keys 8g .. 8g+7 for row n.
//   O^T = V^T P^T the terms are keys: lane (g, n) needs keys 8g .. 8g+7 of its rows, which it
//                 has, and of channel piece n, which is how the cache lays V out: one load.
//                 Conversions give pairs of channels of one key; a byte permutation makes
//                 pairs of keys of them.
// So nothing passes through shared memory, and m, the sum and the rescaling of O are a
// lane's own.  K is exact in bf16 and V in fp16 (the cache's exponents see to that), and so are
// bf16 queries; fp32 queries are split into three bf16 parts that add up to them.  P is
// rounded to fp16 (11 bits: half a step is 2^-12), from fp32 queries to a sum of two fp16.
// All sums are fp32.
//
// The work is cut into units of 32 keys of one item, an item being up to kRows rows of one
// sequence and K/V head.  Every workgroup takes an equal run of units, whatever items they
// are of: a batch of unequal lengths, and causal rows, leave no workgroup behind.  Items that
// end up in several workgroups leave partial results in the workspace, which a second kernel
// joins in the order of the keys.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf.h"
#include "cf_internal.h"
#include "cf_kv4.h"
#include "cf_rows.h"

namespace cf {
namespace {

typedef _Float16 vh2 __attribute__((ext_vector_type(2)));
typedef _Float16 vh8 __attribute__((ext_vector_type(8)));
typedef uint32_t vu4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnit = 32;  // keys
// Workgroups of a call: what is resident on 256 compute units, more where a workgroup's
// registers allow it.
constexpr int kGroupsSmall = 1024, kGroupsLarge = 256;
#ifndef KWB
#define KWB 1
#endif
constexpr int kWideBlocks = KWB;
// A workgroup takes at least so many units, or joining would cost more than it saves.
constexpr int kMinUnits = 8;
// p = 2^(x - m + kLift) where m is at most kSlack below the row's largest score so far: the
// reference moves, and O is rescaled, only when a score exceeds it by more.  p stays below
// 2^(kLift + kSlack) < 65504, and the lift keeps the fp16 of small p off the subnormals.
constexpr float kLift = 7.f, kSlack = 8.f;
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
    int32_t* joins; // what each workgroup leaves to be joined
    int groups;
};

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
    return p.window ? max(s.len - s.nq + token - p.window + 1, 0) : 0;
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

// Inclusive sums over the wave's lanes.
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
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
        if (b < p.batch) {
            const Seq s = seq_of(p, b);
            const int tiles = tiles_of<ROWS>(p, s);
            int u0;
            for (int i = lane & (sub - 1); i < tiles; i += sub) n += units_of<ROWS, UNIT>(p, s, i, &u0) + PAD;
        }
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

// bf16 pair of byte B of codes c.
template <int B>
__device__ __forceinline__ uint32_t to_bf16(uint32_t c, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, B));
}
template <int B>
__device__ __forceinline__ uint32_t to_f16(uint32_t c, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, B));
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ bool page_on(const AttnArgs& p, const Seq& s, int page) {
    return s.len > 0 && static_cast<uint32_t>(page) < static_cast<uint32_t>(p.cache.pages);
}

// One wave's share of 32 keys, as loaded.
template <int D>
struct Keys {
    uint32_t k[2][D / 32];  // two rows of keys, a quarter of the channels each
    uint32_t ks[2];         // their scale bytes
    uint32_t v[D / 16];     // eight keys of a channel piece
    uint32_t vs[2];         // their scale bytes
    bool ok[2];             // the first and the last 16 keys have a page
};

// The two pages of a unit's first and last 16 keys (one page, where it has 32 tokens or more).
struct Pages {
    int at[2];
};

__device__ __forceinline__ Pages pages_of(const AttnArgs& p, const Seq& s, int b, int unit) {
    Pages x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // keys behind the last are read from its page (and masked later): always inside the cache
        const int i = min(unit * kUnit + 16 * h, max(s.len - 1, 0)) >> p.cache.shift;
        const int64_t at = int64_t(b) * p.width + i;
        x.at[h] = p.table ? scalar_load(p.table + at) : static_cast<int>(at);
    }
    return x;
}

// Where a lane's loads lie in a page's block, from the unit's first key on.
struct Offsets {
    uint32_t k, ks, v, vs;
};

template <int D>
__device__ __forceinline__ Offsets offsets_of(const AttnArgs& p) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const KvBlock blk{p.cache.block.page, D};
    const int mask = min(blk.page, kUnit) - 1;
    const int row = 8 * (n >> 2) + (n & 3);
    Offsets o;
    o.k = blk.k_code(row & mask) + g * (D / 8);
    o.ks = blk.k_scale(row & mask, g * (D / 4) / kKvGroup);
    o.v = blk.v_code(8 * g & mask, n);
    o.vs = blk.v_scale(8 * g & mask, n * (D / 16) / kKvGroup);
    return o;
}

template <int D>
__device__ __forceinline__ void load_keys(Keys<D>& x, const AttnArgs& p, const Seq& s, const Pages& pages,
                                          const Offsets& o, int head, int unit) {
    const int lane = threadIdx.x & 63;
    const KvBlock blk{p.cache.block.page, D};
    const int in = unit * kUnit & (blk.page - 1);
    const uint8_t* base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        x.ok[h] = page_on(p, s, pages.at[h]);
        base[h] = p.cache.at(x.ok[h] ? pages.at[h] : 0, head);
    }
    const uint8_t* const kb = lane & 8 ? base[1] : base[0];
    const uint8_t* const vb = lane & 32 ? base[1] : base[0];
    const uint8_t* const kc = kb + (o.k + in * (D / 2));
    const uint8_t* const vc = vb + (o.v + in * (D / 2));
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // four tokens further
        if constexpr (D == 128) {
            const vu4 w = *reinterpret_cast<const vu4*>(kc + 4 * h * (D / 2));
            x.k[h][0] = w.x, x.k[h][1] = w.y, x.k[h][2] = w.z, x.k[h][3] = w.w;
        } else {
            const vu2 w = *reinterpret_cast<const vu2*>(kc + 4 * h * (D / 2));
            x.k[h][0] = w.x, x.k[h][1] = w.y;
        }
        x.ks[h] = kb[o.ks + in * (D / 32) + 4 * h * (D / 32)];
    }
#pragma unroll
    for (int i = 0; i < D / 16; i += 4) {
        const vu4 w = *reinterpret_cast<const vu4*>(vc + 4 * i);
        x.v[i] = w.x, x.v[i + 1] = w.y, x.v[i + 2] = w.z, x.v[i + 3] = w.w;
    }
    const vu2 w = *reinterpret_cast<const vu2*>(vb + (o.vs + in * (D / 32)));
    x.vs[0] = w.x, x.vs[1] = w.y;
}

// Queries of 16 rows: bf16 parts that add up to them, channel order as in K's codes.
template <int D, int PARTS>
struct Rows {
    vb8 q[PARTS][D / 32];
};

template <typename T, int D, int PARTS>
__device__ __forceinline__ void load_rows(Rows<D, PARTS>& x, const AttnArgs& p, const Seq& s, int head, int row,
                                          int token, bool on) {
    const int g = (threadIdx.x & 63) >> 4;
    const T* const q = row_ptr<T>(p.q, s.q0 + token, head * p.share + row - token * p.share);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        float f[8];
        Row8<T> r;
        if (on) {
            r.load(q + g * (D / 4) + 8 * i);
            r.get(f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float rest = on ? f[j] : 0.f;
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const __bf16 h = static_cast<__bf16>(rest);
                x.q[k][i][j] = h;
                rest -= static_cast<float>(h);
            }
        }
    }
}

// PARTS: bf16 parts of a query (1 or 3); PP: fp16 parts of a probability.  NQ: sixteens of
// rows a wave holds.  SPLIT: the four waves share the item's rows and split its units;
// otherwise each has rows of its own.
template <typename T, int D, int NQ, bool SPLIT>
struct Shape {
    static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
    static constexpr int kP = sizeof(T) == 4 ? 2 : 1;
    static constexpr int kRows = 16 * NQ * (SPLIT ? 1 : kWaves);
    static constexpr int kPad = SPLIT ? 8 : 2;
};

// Floats of one partial result: rows x (D values, the reference, the sum).
template <int D>
__host__ __device__ constexpr int64_t part_floats(int rows) {
    return int64_t(rows) * (D + 2);
}

template <typename T>
__device__ __forceinline__ void store_out(T* o, const float (&x)[8]) {
    Row8<T> r;
    r.set(x);
    r.store(o);
}

template <typename T, int D, int NQ, bool SPLIT>
__global__ __launch_bounds__(kThreads, NQ == 1 ? 2 : 1) void attn_kernel(const AttnArgs p) {
    using S = Shape<T, D, NQ, SPLIT>;
    constexpr int kRows = S::kRows, kPad = S::kPad, kParts = S::kParts, kP = S::kP;
    constexpr int kJ = D / 16;  // O^T tiles of 16 channel pieces
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 15, g = lane >> 4;

    __shared__ float stage[SPLIT ? kWaves * 16 * (D + 4) : 1];
    __shared__ float stage_m[SPLIT ? kWaves * 16 : 1], stage_l[SPLIT ? kWaves * 16 : 1];

    Place w;
    const bool work = place_of<kRows, kUnit, kPad>(p, &w);
    const int me = w.me;
    if (threadIdx.x == 0) p.joins[me * 4] = -1;
    if (!work) return;
    const Offsets offs = offsets_of<D>(p);
    Seq s = seq_at(p, w.b);

    while (w.at < w.end) {
        // units [a, z) of this item
        int u0;
        const int count = units_of<kRows, kUnit>(p, s, w.tile, &u0);
        const int64_t take = min(w.end - w.at, count + kPad - w.rest);
        const int a = max(static_cast<int>(w.rest) - kPad, 0), z = static_cast<int>(w.rest + take) - kPad;
        w.at += take;
        if (z <= 0) break;  // the next workgroup begins this item
        const int rows = s.nq * p.share;
        const int row0 = w.tile * kRows + (SPLIT ? 0 : wave * 16 * NQ);
        const int head = w.head;

        constexpr int kStep = SPLIT ? kWaves : 1;
        const int first = a + (SPLIT ? wave : 0);
        Pages pages = pages_of(p, s, w.b, u0 + first);
        Keys<D> next;
        if (first < z) load_keys<D>(next, p, s, pages, offs, head, u0 + first);
        if (first + kStep < z) pages = pages_of(p, s, w.b, u0 + first + kStep);

        Rows<D, kParts> q[NQ];
        int lo[NQ], hi[NQ];                   // keys that row n of each sixteen sees
        int full_lo = 0, full_hi = INT32_MAX; // keys that all of the wave's rows see
        {
            const int last = min(row0 + 16 * NQ, rows) - 1;
            if (last >= row0) {
                full_lo = seen_lo(p, s, token_of(p, last));
                full_hi = seen_hi(p, s, token_of(p, row0));
            }
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int row = row0 + i * 16 + n;
            const bool on = row < rows;
            const int token = token_of(p, on ? row : row0 < rows ? row0 : 0);
            load_rows<T, D, kParts>(q[i], p, s, head, on ? row : 0, on ? token : 0, on);
            lo[i] = on ? seen_lo(p, s, token) : 0;
            hi[i] = on ? seen_hi(p, s, token) : 0;
        }

        vf4 o[NQ][kJ];
        float m[NQ], sum[NQ];  // m: reference in units of log2, raised by kLift
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            m[i] = kNone, sum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < kJ; ++j) o[i][j] = vf4{0.f, 0.f, 0.f, 0.f};
        }

        for (int u = first; u < z; u += kStep) {
            Keys<D> x = next;
            if (u + kStep < z) load_keys<D>(next, p, s, pages, offs, head, u0 + u + kStep);
            if (u + 2 * kStep < z) pages = pages_of(p, s, w.b, u0 + u + 2 * kStep);
            const int key0 = (u0 + u) * kUnit;
            // the lane's own eight keys
            const int mine0 = key0 + 8 * g;
            const bool ok = lane & 32 ? x.ok[1] : x.ok[0];
            const bool edge = key0 < full_lo || key0 + kUnit > full_hi || !x.ok[0] || !x.ok[1];
            uint32_t bad = 0;  // V groups of the lane's keys that read NaN, a bit a key
            uint32_t kbad[2] = {0, 0};
            if (edge) {
                // V behind the sequence's last key is whatever an earlier owner of the page left
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if (ok && mine0 + t < s.len) continue;
                    if constexpr (D == 128)
                        x.v[t] = 0;
                    else
                        x.v[t / 2] &= t & 1 ? 0xffffu : 0xffff0000u;
                    x.vs[t / 4] = (x.vs[t / 4] & ~(0xffu << (8 * (t & 3)))) | 127u << (8 * (t & 3));
                }
            }
            const uint32_t odd = (x.vs[0] & x.vs[0] << 1) | (x.vs[1] & x.vs[1] << 1);
            const bool nans = __any((odd & 0x80808080u) != 0 || max(x.ks[0], x.ks[1]) >= kKvNanFrom);
            if (nans) {
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const uint32_t byte = (x.vs[t / 4] >> (8 * (t & 3))) & 0xffu;
                    if (byte < kKvNanFrom) continue;
                    bad |= 1u << t;
                    x.vs[t / 4] = (x.vs[t / 4] & ~(0xffu << (8 * (t & 3)))) | 127u << (8 * (t & 3));
                    if constexpr (D == 128)
                        x.v[t] = 0;
                    else
                        x.v[t / 2] &= t & 1 ? 0xffffu : 0xffff0000u;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t w = __ballot(x.ks[h] >= kKvNanFrom);
                    kbad[h] = static_cast<uint32_t>((w | w >> 16 | w >> 32 | w >> 48) & 0xffffu);
                }
            }

            // scores: sc[i][t] is key mine0 + t, row n of the i-th sixteen
            vf4 sc[NQ][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ks = scale_of(x.ks[h]);
                vb8 kf[D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const vu4 w{to_bf16<0>(x.k[h][c], ks), to_bf16<1>(x.k[h][c], ks), to_bf16<2>(x.k[h][c], ks),
                                to_bf16<3>(x.k[h][c], ks)};
                    kf[c] = __builtin_bit_cast(vb8, w);
                }
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    vf4 acc{0.f, 0.f, 0.f, 0.f};
                    // the smallest parts first
#pragma unroll
                    for (int k = kParts - 1; k >= 0; --k)
#pragma unroll
                        for (int c = 0; c < D / 32; ++c)
                            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[c], q[i].q[k][c], acc, 0, 0, 0);
                    sc[i][h] = acc;
                }
            }

            vh8 pf[NQ][kP];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                float x2[8];  // scores in units of log2
#pragma unroll
                for (int t = 0; t < 8; ++t) x2[t] = sc[i][t >> 2][t & 3] * p.scale_log2;
                uint32_t see = 0xff;
                if (nans) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        if (kbad[t >> 2] >> (4 * g + (t & 3)) & 1u) x2[t] = __builtin_nanf("");
                }
                if (edge) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        if (!ok || mine0 + t < lo[i] || mine0 + t >= hi[i]) x2[t] = kNone, see &= ~(1u << t);
                }
                float top = kNone;
#pragma unroll
                for (int t = 0; t < 8; ++t) top = fmaxf(top, x2[t]);
                if (__any(top > m[i] + (kSlack + kLift))) {
                    // the lanes of a row agree on its new reference
                    const float r = fmaxf(across_max(top) - kLift, m[i]);
                    const float f = m[i] == r ? 1.f : __builtin_amdgcn_exp2f(m[i] - r);
                    m[i] = r;
                    sum[i] *= f;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) o[i][j] *= f;
                }
                const float ref = m[i] == kNone ? 0.f : m[i];
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    x2[t] = __builtin_amdgcn_exp2f(x2[t] - ref);
                    sum[i] += x2[t];
                    const _Float16 h = static_cast<_Float16>(x2[t]);
                    pf[i][0][t] = h;
                    if constexpr (kP == 2) pf[i][1][t] = static_cast<_Float16>(x2[t] - static_cast<float>(h));
                }
                if (nans) {
                    // a NaN of V reaches the rows that see its key, and only those
                    uint32_t hit = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t bv = __shfl(static_cast<int>(bad), 16 * k + (D == 128 ? 4 * g : 8 * (g >> 1)), 64);
                        hit |= bv & static_cast<uint32_t>(__shfl(static_cast<int>(see), 16 * k + n, 64));
                    }
                    if (hit)
#pragma unroll
                        for (int j = 0; j < kJ; ++j) o[i][j] = vf4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
                }
            }

            float vs[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) vs[t] = scale_of((x.vs[t / 4] >> (8 * (t & 3))) & 0xffu);
            const auto pv = [&](int j, const uint32_t (&c)[8]) {
                // c: channel pairs 2j, 2j + 1 of the eight keys
                vu4 even, odd_;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    even[t] = __builtin_amdgcn_perm(c[2 * t + 1], c[2 * t], 0x05040100u);
                    odd_[t] = __builtin_amdgcn_perm(c[2 * t + 1], c[2 * t], 0x07060302u);
                }
#pragma unroll
                for (int i = 0; i < NQ; ++i)
#pragma unroll
                    for (int k = kP - 1; k >= 0; --k) {
                        o[i][2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vh8, even), pf[i][k],
                                                                            o[i][2 * j], 0, 0, 0);
                        o[i][2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vh8, odd_),
                                                                                pf[i][k], o[i][2 * j + 1], 0, 0, 0);
                    }
            };
            if constexpr (D == 128) {
                uint32_t c[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = to_f16<0>(x.v[t], vs[t]);
                pv(0, c);
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = to_f16<1>(x.v[t], vs[t]);
                pv(1, c);
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = to_f16<2>(x.v[t], vs[t]);
                pv(2, c);
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = to_f16<3>(x.v[t], vs[t]);
                pv(3, c);
            } else {
                uint32_t c[8];
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    c[t] = t & 1 ? to_f16<2>(x.v[t / 2], vs[t]) : to_f16<0>(x.v[t / 2], vs[t]);
                pv(0, c);
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    c[t] = t & 1 ? to_f16<3>(x.v[t / 2], vs[t]) : to_f16<1>(x.v[t / 2], vs[t]);
                pv(1, c);
            }
        }

        // this segment's results: the whole item, or a part for the second kernel
        const bool whole = a == 0 && z == count;
        float* const part = p.part + (2 * int64_t(me) + (a == 0)) * part_floats<D>(kRows);
        const auto put = [&](int r, int c, float (&v)[8], float top, float l, bool first_piece) {
            // eight channels from c of row r of the item
            const int row = w.tile * kRows + r;
            if (row >= rows) return;
            if (whole) {
                const int token = token_of(p, row), qh = head * p.share + row - token * p.share;
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= inv;
                store_out<T>(row_ptr<T>(p.out, s.q0 + token, qh) + c, v);
                if (p.lse && first_piece)
                    p.lse[int64_t(s.q0 + token) * p.q_heads + qh] =
                        l == 0.f ? kNone : (top + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
            } else {
                float* const y = part + int64_t(r) * (D + 2);
#pragma unroll
                for (int k = 0; k < 8; k += 2) *reinterpret_cast<float2*>(y + c + k) = float2{v[k], v[k + 1]};
                if (first_piece) *reinterpret_cast<float2*>(y + D) = float2{top, l};
            }
        };
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            sum[i] = across_sum(sum[i]);
            if constexpr (!SPLIT) {
                // a lane has D/4 consecutive channels of its row
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = o[i][(8 * c + k) % kJ][(8 * c + k) / kJ];
                    put(wave * 16 * NQ + i * 16 + n, g * (D / 4) + 8 * c, v, m[i], sum[i], g == 0 && c == 0);
                }
            } else {
                __syncthreads();
                float* const y = stage + (wave * 16 + n) * (D + 4) + g * (D / 4);
#pragma unroll
                for (int c = 0; c < D / 4; c += 4)
                    *reinterpret_cast<vf4*>(y + c) = vf4{o[i][c % kJ][c / kJ], o[i][(c + 1) % kJ][(c + 1) / kJ],
                                                         o[i][(c + 2) % kJ][(c + 2) / kJ], o[i][(c + 3) % kJ][(c + 3) / kJ]};
                if (g == 0) stage_m[wave * 16 + n] = m[i], stage_l[wave * 16 + n] = sum[i];
                __syncthreads();
                for (int x = threadIdx.x; x < 16 * (D / 8); x += kThreads) {
                    const int r = x / (D / 8), c = x % (D / 8) * 8;
                    float top = kNone;
#pragma unroll
                    for (int k = 0; k < kWaves; ++k) top = fmaxf(top, stage_m[k * 16 + r]);
                    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
                    for (int k = 0; k < kWaves; ++k) {
                        const float f = stage_m[k * 16 + r] == kNone ? 0.f
                                                                     : __builtin_amdgcn_exp2f(stage_m[k * 16 + r] - top);
                        // a wave without a reference has only zeros, or NaN that must show
                        const float* const y = stage + (k * 16 + r) * (D + 4) + c;
                        l = __builtin_fmaf(stage_l[k * 16 + r], f, l);
#pragma unroll
                        for (int d = 0; d < 8; ++d) v[d] = __builtin_fmaf(y[d], f, v[d]);
                    }
                    put(i * 16 + r, c, v, top, l, c == 0);
                }
            }
        }
        if (threadIdx.x == 0 && a > 0 && z == count) {
            int32_t* const j = p.joins + me * 4;
            j[1] = w.b, j[2] = head, j[3] = w.tile;
            // the workgroup with the item's first unit
            j[0] = static_cast<int32_t>((w.at - count) / w.chunk);
        }

        // on to the next item
        w.rest = 0;
        if (w.at >= w.end) break;
        if (++w.tile >= tiles_of<kRows>(p, s)) {
            w.tile = 0;
            if (++w.head >= p.cache.heads) {
                w.head = 0;
                do s = seq_at(p, ++w.b);  // at < end <= total: another sequence has units
                while (s.nq == 0);
            }
        }
    }
}


// ---- many rows ------------------------------------------------------------------------

typedef float vf16 __attribute__((ext_vector_type(16)));

// Four waves, each with 32 * QB rows of its own, over tiles of 64 keys that all of them
// decode once, into shared memory: K as bf16 [key][channel], V as fp16 [channel][key].
template <typename T, int D, int QB>
struct Wide {
    static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
    static constexpr int kP = sizeof(T) == 4 ? 2 : 1;
    static constexpr int kRows = 32 * QB * kWaves;
    static constexpr int kKeys = 64;
    // with two waves a SIMD the order of reads and products is fixed; three hide it, and lack registers
    static constexpr bool kAhead = D == 128;
#ifndef KR64
#define KR64 3
#endif
    static constexpr int kResident = sizeof(T) == 4 ? 128 / D : D == 64 ? KR64 : 2;  // workgroups of a compute unit
    static constexpr int kPad = 2;
    // K's rows are 16 bytes longer than they need to be: 16 rows then start on different banks
    static constexpr int kKRow = 2 * D + 16;
    static constexpr int kTile = kKeys * kKRow + D * 2 * kKeys;
    // V's rows (a channel's 64 keys) lie two together in 256 bytes, as 16 runs of 8 keys: run q of
    // channel c is number (8 (c & 1) + q) ^ v_turn(c / 2).  Both the 16 consecutive channels that
    // a product reads and the 16 channel pieces that the decoding threads write then lie on
    // different banks.  The turn of c / 2 + x is that of c / 2, ^ x, for x below 4 (2 at 64
    // channels) and c a piece's first.
    __host__ __device__ static constexpr int v_turn(int pair) {
        return D == 128 ? (pair & 7) ^ (pair >> 3 & 3) ^ (pair >> 5 & 1) << 3
                        : (pair & 7) ^ (pair >> 3 & 1) ^ (pair >> 4 & 1) << 3;
    }
    static constexpr int kBytes = 2 * kTile;
};

// A thread's share of a tile: D/4 codes of a key, and four keys of a channel piece.  Its wave's
// threads share 16 keys, and so one page.
template <int D>
struct Share {
    uint32_t k[D / 32], v[D / 32];
    uint32_t ks, vs;  // scale bytes: one, and four
    bool on;          // the keys have a page
};

// The page of a key (the last key's behind it: always inside the cache, and masked later).
// Lanes ask for a tile's four runs of 16 keys, and a wave takes its own: a scalar load, which
// shares its counter with shared memory, would be waited for at the next barrier.
__device__ __forceinline__ int page_at(const AttnArgs& p, const Seq& s, int b, int key0) {
    const int key = key0 + 16 * static_cast<int>(threadIdx.x & 3);
    const int64_t at = int64_t(b) * p.width + (min(key, max(s.len - 1, 0)) >> p.cache.shift);
    return p.table ? p.table[at] : static_cast<int>(at);  // at < pages < 2^31 without a table
}

// Where a thread's share lies in a page's block, from its wave's first key on.
template <int D>
__device__ __forceinline__ Offsets share_offsets(const AttnArgs& p) {
    const int lane = threadIdx.x & 63;
    const KvBlock blk{p.cache.block.page, D};
    Offsets o;
    o.k = blk.k_code(lane / 4) + (lane & 3) * (D / 8);
    o.ks = blk.k_scale(lane / 4, (lane & 3) * (D / 4) / kKvGroup);
    // half a piece: keys 4 h .. of the eight
    const int key = lane / 32 * 8 + (lane & 1) * 4, n = lane / 2 & 15;
    o.v = blk.v_code(key, n);
    o.vs = blk.v_scale(key, n * (D / 16) / kKvGroup);
    return o;
}

// key: the wave's first.
template <int D>
__device__ __forceinline__ void load_share(Share<D>& x, const AttnArgs& p, const Seq& s, int page, const Offsets& o,
                                           int head, int key) {
    x.on = page_on(p, s, page);
    const uint8_t* const base = p.cache.at(x.on ? page : 0, head);
    const int in = key & (p.cache.block.page - 1);
    const uint8_t* const kc = base + in * (D / 2) + o.k;
    const uint8_t* const vc = base + in * (D / 2) + o.v;
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) {
        const vu2 y = *reinterpret_cast<const vu2*>(kc + 4 * i), z = *reinterpret_cast<const vu2*>(vc + 4 * i);
        x.k[i] = y.x, x.k[i + 1] = y.y;
        x.v[i] = z.x, x.v[i + 1] = z.y;
    }
    x.ks = base[in * (D / 32) + o.ks];
    x.vs = *reinterpret_cast<const uint32_t*>(base + in * (D / 32) + o.vs);
}

// Decodes a share into a tile, of whose keys the sequence has the first `left`.  Keys behind them
// become zeros whatever their bytes, and so do groups that read NaN: returns whether the
// wave has any of those, and then k_nan and v_nan, [key][group], say which of its keys' do.
template <int D>
__device__ __forceinline__ bool store_share(Share<D>& x, uint8_t* tile, uint8_t* k_nan, uint8_t* v_nan, int left) {
    using W = Wide<__bf16, D, 1>;
    const int kin = threadIdx.x / 4, vin = threadIdx.x / 32 * 8 + (threadIdx.x & 1) * 4, n = threadIdx.x / 2 & 15;
    uint32_t v[4];  // the channels of a key
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = D == 128 ? x.v[t] : x.v[t / 2] >> (16 * (t & 1));
    bool nan = false;
    if (!x.on || left < W::kKeys || __any(x.ks >= kKvNanFrom || (x.vs & x.vs << 1 & 0x80808080u) != 0)) {
        const bool on = x.on && kin < left, k_bad = x.ks >= kKvNanFrom;
        uint32_t v_bad = 0;
        nan = on && k_bad;
        if (!on || k_bad) {
            x.ks = 127u;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) x.k[i] = 0;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const bool on = x.on && vin + t < left;
            const bool bad = on && (x.vs >> (8 * t) & 0xffu) >= kKvNanFrom;
            nan |= bad;
            v_bad |= static_cast<uint32_t>(bad) << t;
            if (on && !bad) continue;
            x.vs = (x.vs & ~(0xffu << (8 * t))) | 127u << (8 * t);
            v[t] = 0;
        }
        nan = __any(nan);
        if (nan) {
            constexpr int kGroups = D / kKvGroup;
            k_nan[kin * 4 + (threadIdx.x & 3)] = on && k_bad;
#pragma unroll
            for (int t = 0; t < 4; ++t) v_nan[(vin + t) * kGroups + n / (16 / kGroups)] = v_bad >> t & 1;
        }
    }
    {
        const float f = scale_of(x.ks);
        uint8_t* const w = tile + kin * W::kKRow + (threadIdx.x & 3) * (D / 2);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t c = x.k[i];
            *reinterpret_cast<vu4*>(w + 16 * i) = vu4{to_bf16<0>(c, f), to_bf16<1>(c, f), to_bf16<2>(c, f), to_bf16<3>(c, f)};
        }
    }
    {
        float f[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) f[t] = scale_of(x.vs >> (8 * t) & 0xffu);
        const int first = n * (D / 32), turn = W::v_turn(first) ^ vin / 8;  // pair of channels
        uint8_t* const w = tile + W::kKeys * W::kKRow + first * 256 + (vin & 4) * 2;
        const auto pair = [&](int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            *reinterpret_cast<vu2*>(w + 256 * j + 16 * (turn ^ j)) =
                vu2{__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(d, c, 0x05040100u)};
            *reinterpret_cast<vu2*>(w + 256 * j + 16 * (turn ^ j ^ 8)) =
                vu2{__builtin_amdgcn_perm(b, a, 0x07060302u), __builtin_amdgcn_perm(d, c, 0x07060302u)};
        };
        pair(0, to_f16<0>(v[0], f[0]), to_f16<0>(v[1], f[1]), to_f16<0>(v[2], f[2]), to_f16<0>(v[3], f[3]));
        pair(1, to_f16<1>(v[0], f[0]), to_f16<1>(v[1], f[1]), to_f16<1>(v[2], f[2]), to_f16<1>(v[3], f[3]));
        if constexpr (D == 128) {
            pair(2, to_f16<2>(v[0], f[0]), to_f16<2>(v[1], f[1]), to_f16<2>(v[2], f[2]), to_f16<2>(v[3], f[3]));
            pair(3, to_f16<3>(v[0], f[0]), to_f16<3>(v[1], f[1]), to_f16<3>(v[2], f[2]), to_f16<3>(v[3], f[3]));
        }
    }
    return nan;
}

// Nothing moves across: what is read before is in flight while what stands before is worked on.
// Left alone, the compiler reads shared memory one product ahead of nothing, and each waits.
template <bool ON>
__device__ __forceinline__ void stay() {
    if constexpr (ON) __builtin_amdgcn_sched_barrier(0);
}

// A wave's 16 x 16 matrix products of before are 32 x 32 with 16 terms here: lane = 32 h + n
// has row n of a block, and of 32 keys 8 h .. 8 h + 7 and 16 + 8 h .. , K's rows being
// taken in the order that makes it so.
template <typename T, int D, int QB>
__global__ __launch_bounds__(kThreads, (Wide<T, D, QB>::kResident)) void wide_kernel(const AttnArgs p) {
    using W = Wide<T, D, QB>;
    constexpr int kRows = W::kRows, kPad = W::kPad, kParts = W::kParts, kP = W::kP, kKeys = W::kKeys;
    constexpr int kDt = D / 32;
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 31, h = lane >> 5;
    __shared__ __align__(16) uint8_t lds[W::kBytes];
    __shared__ uint32_t flag[2][kWaves];
    __shared__ uint8_t k_nan[2][kKeys * 4], v_nan[2][kKeys * kDt];

    Place w;
    const bool work = place_of<kRows, kKeys, kPad>(p, &w);
    const int me = w.me;
    if (threadIdx.x == 0) p.joins[me * 4] = -1;
    if (!work) return;
    Seq s = seq_at(p, w.b);
    const Offsets offs = share_offsets<D>(p);
    const int v_lane = 8 * (n & 1) ^ h ^ W::v_turn(n / 2);  // v_turn(16 j + x) = v_turn(16 j) ^ v_turn(x)
    // key of row n of K's fragments
    const int k_row = 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);

    while (w.at < w.end) {
        int u0;
        const int count = units_of<kRows, kKeys>(p, s, w.tile, &u0);
        const int64_t take = min(w.end - w.at, count + kPad - w.rest);
        const int a = max(static_cast<int>(w.rest) - kPad, 0), z = static_cast<int>(w.rest + take) - kPad;
        w.at += take;
        if (z <= 0) break;  // the next workgroup begins this item
        const int rows = s.nq * p.share;
        const int row0 = w.tile * kRows + wave * 32 * QB;
        const int head = w.head;

        const int wave_key = 16 * wave;
        Share<D> next;
        int pages = page_at(p, s, w.b, (u0 + a) * kKeys);  // of the tile to load next
        load_share<D>(next, p, s, __builtin_amdgcn_readlane(pages, wave), offs, head, (u0 + a) * kKeys + wave_key);
        pages = page_at(p, s, w.b, (u0 + a + 1) * kKeys);

        vb8 q[QB][kParts][D / 16];
        int lo[QB], hi[QB];
        int full_lo = 0, full_hi = INT32_MAX;
        {
            const int last = min(row0 + 32 * QB, rows) - 1;
            if (last >= row0) {
                full_lo = seen_lo(p, s, token_of(p, last));
                full_hi = seen_hi(p, s, token_of(p, row0));
            }
        }
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const int row = row0 + i * 32 + n;
            const bool on = row < rows;
            const int token = on ? token_of(p, row) : 0;
            const T* const src = row_ptr<T>(p.q, s.q0 + token, head * p.share + (on ? row : 0) - token * p.share);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                float f[8];
                if (on) {
                    Row8<T> r;
                    r.load(src + 16 * c + 8 * h);
                    r.get(f);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float rest = on ? f[j] : 0.f;
#pragma unroll
                    for (int k = 0; k < kParts; ++k) {
                        const __bf16 y = static_cast<__bf16>(rest);
                        q[i][k][c][j] = y;
                        rest -= static_cast<float>(y);
                    }
                }
            }
            lo[i] = on ? seen_lo(p, s, token) : 0;
            hi[i] = on ? seen_hi(p, s, token) : 0;
        }

        vf16 o[QB][kDt];
        float m[QB], sum[QB];
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            m[i] = kNone, sum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < kDt; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k) o[i][j][k] = 0.f;
        }

        __syncthreads();  // the last item's tiles have been read
        {
            const uint32_t nan = store_share<D>(next, lds, k_nan[0], v_nan[0], s.len - (u0 + a) * kKeys);
            if (lane == 0) flag[0][wave] = nan | (next.on ? 0u : 2u);
        }
        const auto load_next = [&](int u) {
            const int page = __builtin_amdgcn_readlane(pages, wave);
            pages = page_at(p, s, w.b, (u0 + u + 1) * kKeys);
            load_share<D>(next, p, s, page, offs, head, (u0 + u) * kKeys + wave_key);
        };
        if (a + 1 < z) load_next(a + 1);
        __syncthreads();

        for (int u = a; u < z; ++u) {
            const int buf = (u - a) & 1;
            const uint8_t* const kt = lds + buf * W::kTile;
            const uint8_t* const vt = kt + kKeys * W::kKRow;
            const int key0 = (u0 + u) * kKeys;
            // what the tile's writers saw in their 16 keys: 1 a group that reads NaN, 2 no page
            const uint32_t f4[4] = {flag[buf][0], flag[buf][1], flag[buf][2], flag[buf][3]};
            const uint32_t seen_by = uniform(static_cast<int>(f4[0] | f4[1] << 2 | f4[2] << 4 | f4[3] << 6));
            const bool edge = key0 < full_lo || key0 + kKeys > full_hi || (seen_by & 0xaa) != 0;
            const bool nans = (seen_by & 0x55) != 0;

            // K's fragments, four ahead of the products: number f is terms 16 (f % (D/16)) of half f / (D/16)
            constexpr int kFrags = 2 * D / 16;
            const uint8_t* const kn = kt + k_row * W::kKRow + 16 * h;
            vf16 sc[2][QB];
            vb8 kf[2][4];
            const auto read_k = [&](int f0) {
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f)
                    kf[f / 4 & 1][f & 3] = *reinterpret_cast<const vb8*>(kn + f / (D / 16) * 32 * W::kKRow + f % (D / 16) * 32);
            };
            read_k(0);
#pragma unroll
            for (int f0 = 0; f0 < kFrags; f0 += 4) {
                if (f0 + 4 < kFrags) read_k(f0 + 4);
                stay<W::kAhead>();
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f)
#pragma unroll
                    for (int i = 0; i < QB; ++i)
#pragma unroll
                        for (int k = kParts - 1; k >= 0; --k) {
                            vf16& x = sc[f / (D / 16)][i];
                            if (f % (D / 16) == 0 && k == kParts - 1)
#pragma unroll
                                for (int r = 0; r < 16; ++r) x[r] = 0.f;
                            x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[f / 4 & 1][f & 3], q[i][k][f % (D / 16)], x, 0, 0, 0);
                        }
                stay<W::kAhead>();
            }
            // score r of half g is of key mine0 + 32 g + 16 * (r / 8) + r % 8
            const int mine0 = key0 + 8 * h;
            if (nans) {
                // a NaN reaches the rows that see its key, and only those
                uint32_t k_bad = 0, v_bad[QB][kDt] = {};
#pragma unroll 1
                for (int r = 0; r < 32; ++r)
                    if (seen_by >> (2 * (r / 8)) & 1u) {
                        const uint8_t* const y = k_nan[buf] + 4 * (8 * h + 16 * (r / 8) + r % 8);
                        k_bad |= static_cast<uint32_t>((y[0] | y[1] | y[2] | y[3]) != 0) << r;
                    }
#pragma unroll 1
                for (int t = 0; t < kKeys; ++t)
                    if (seen_by >> (2 * (t / 16)) & 1u) {
#pragma unroll
                        for (int i = 0; i < QB; ++i)
#pragma unroll
                            for (int j = 0; j < kDt; ++j)
                                v_bad[i][j] |= key0 + t >= lo[i] && key0 + t < hi[i] ? v_nan[buf][t * kDt + j] : 0u;
                    }
#pragma unroll
                for (int i = 0; i < QB; ++i) {
#pragma unroll
                    for (int r = 0; r < 32; ++r)
                        if (k_bad >> r & 1u) sc[r / 16][i][r % 16] = __builtin_nanf("");
#pragma unroll
                    for (int j = 0; j < kDt; ++j)
                        if (v_bad[i][j])
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[i][j][k] = __builtin_nanf("");
                }
            }
            if (edge) {
#pragma unroll
                for (int i = 0; i < QB; ++i)
#pragma unroll
                    for (int r = 0; r < 32; ++r) {
                        const int key = mine0 + 16 * (r / 8) + r % 8;
                        if ((seen_by >> (2 * (r / 8)) & 2u) || key < lo[i] || key >= hi[i]) sc[r / 16][i][r % 16] = kNone;
                    }
            }
            float top[QB];
            bool move = false;
#pragma unroll
            for (int i = 0; i < QB; ++i) {
                top[i] = kNone;
#pragma unroll
                for (int r = 0; r < 32; ++r) top[i] = fmaxf(top[i], sc[r / 16][i][r % 16]);
                top[i] *= p.scale_log2;
                move |= top[i] > m[i] + (kSlack + kLift);
            }
            if (__any(move)) {
#pragma unroll
                for (int i = 0; i < QB; ++i) {
                    const float r = fmaxf(fmaxf(top[i], __shfl_xor(top[i], 32, 64)) - kLift, m[i]);
                    const float f = m[i] == r ? 1.f : __builtin_amdgcn_exp2f(m[i] - r);
                    m[i] = r;
                    sum[i] *= f;
#pragma unroll
                    for (int j = 0; j < kDt; ++j) o[i][j] *= f;
                }
            }
            float ref[QB];
#pragma unroll
            for (int i = 0; i < QB; ++i) ref[i] = m[i] == kNone ? 0.f : -m[i];
            vh8 pf[2][QB][kP][2];
            // probabilities r0 .. r0 + N - 1 of half g
            const auto exps = [&](int g, int r0, int many) {
#pragma unroll
                for (int i = 0; i < QB; ++i)
#pragma unroll
                    for (int r = r0; r < r0 + many; ++r) {
                        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[g][i][r], p.scale_log2, ref[i]));
                        sum[i] += e;
                        const _Float16 y = static_cast<_Float16>(e);
                        pf[g][i][0][r / 8][r % 8] = y;
                        if constexpr (kP == 2) pf[g][i][1][r / 8][r % 8] = static_cast<_Float16>(e - static_cast<float>(y));
                    }
            };
            // V's fragments, likewise: number f is of half f / (2 kDt), terms 16 (f % 2), channels 32 (f / 2 % kDt)
            constexpr int kVFrags = 4 * kDt;
            const uint8_t* const vn = vt + n / 2 * 256;
            vh8 vf[2][4];
            const auto read_v = [&](int f0) {
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f) {
                    const int g = f / (2 * kDt), j = f / 2 % kDt, t = f & 1;
                    vf[f / 4 & 1][f & 3] = *reinterpret_cast<const vh8*>(
                        vn + j * 4096 + 16 * (v_lane ^ (4 * g + 2 * t) ^ W::v_turn(16 * j)));
                }
            };
            read_v(0);
            stay<W::kAhead>();
            exps(0, 0, 16);
#pragma unroll
            for (int f0 = 0; f0 < kVFrags; f0 += 4) {
                if (f0 + 4 < kVFrags) read_v(f0 + 4);
                stay<W::kAhead>();
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f)
#pragma unroll
                    for (int i = 0; i < QB; ++i)
#pragma unroll
                        for (int k = kP - 1; k >= 0; --k) {
                            vf16& x = o[i][f / 2 % kDt];
                            x = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[f / 4 & 1][f & 3], pf[f / (2 * kDt)][i][k][f & 1], x, 0, 0, 0);
                        }
                // the other half's probabilities beside this half's products
                if (f0 < kVFrags / 2) exps(1, f0 * 32 / kVFrags, 4 * 32 / kVFrags);
                stay<W::kAhead>();
            }
            if (u + 1 < z) {
                const uint32_t nan =
                    store_share<D>(next, lds + (buf ^ 1) * W::kTile, k_nan[buf ^ 1], v_nan[buf ^ 1], s.len - key0 - kKeys);
                if (lane == 0) flag[buf ^ 1][wave] = nan | (next.on ? 0u : 2u);
                if (u + 2 < z) load_next(u + 2);
                __syncthreads();
            }
        }

        const bool whole = a == 0 && z == count;
        float* const part = p.part + (2 * int64_t(me) + (a == 0)) * part_floats<D>(kRows);
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const float l = sum[i] + __shfl_xor(sum[i], 32, 64);
            const int r = wave * 32 * QB + i * 32 + n, row = w.tile * kRows + r;
            if (row >= rows) continue;
            const int token = token_of(p, row), qh = head * p.share + row - token * p.share;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T* const dst = row_ptr<T>(p.out, s.q0 + token, qh);
            float* const y = part + int64_t(r) * (D + 2);
            // registers 4 k .. are channels 8 k + 4 h ..
#pragma unroll
            for (int j = 0; j < kDt; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = 32 * j + 8 * k + 4 * h;
                    if (whole) {
                        if constexpr (sizeof(T) == 2) {
                            *reinterpret_cast<vb2*>(dst + c) = vb2{static_cast<__bf16>(o[i][j][4 * k] * inv), static_cast<__bf16>(o[i][j][4 * k + 1] * inv)};
                            *reinterpret_cast<vb2*>(dst + c + 2) = vb2{static_cast<__bf16>(o[i][j][4 * k + 2] * inv), static_cast<__bf16>(o[i][j][4 * k + 3] * inv)};
                        } else {
                            *reinterpret_cast<vf4*>(dst + c) = vf4{o[i][j][4 * k], o[i][j][4 * k + 1], o[i][j][4 * k + 2], o[i][j][4 * k + 3]} * inv;
                        }
                    } else {
                        *reinterpret_cast<float2*>(y + c) = float2{o[i][j][4 * k], o[i][j][4 * k + 1]};
                        *reinterpret_cast<float2*>(y + c + 2) = float2{o[i][j][4 * k + 2], o[i][j][4 * k + 3]};
                    }
                }
            if (h == 0) {
                if (!whole)
                    *reinterpret_cast<float2*>(y + D) = float2{m[i], l};
                else if (p.lse)
                    p.lse[int64_t(s.q0 + token) * p.q_heads + qh] =
                        l == 0.f ? kNone : (m[i] + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
            }
        }
        if (threadIdx.x == 0 && a > 0 && z == count) {
            int32_t* const j = p.joins + me * 4;
            j[1] = w.b, j[2] = head, j[3] = w.tile;
            j[0] = static_cast<int32_t>((w.at - count) / w.chunk);
        }

        w.rest = 0;
        if (w.at >= w.end) break;
        if (++w.tile >= tiles_of<kRows>(p, s)) {
            w.tile = 0;
            if (++w.head >= p.cache.heads) {
                w.head = 0;
                do s = seq_at(p, ++w.b);  // at < end <= total: another sequence has units
                while (s.nq == 0);
            }
        }
    }
}

// Joins the parts of the items that ended up in several workgroups: block (w, y) some rows
// of the item whose last keys were workgroup w's.
template <typename T, int D, int ROWS>
__global__ __launch_bounds__(kThreads) void join_kernel(const AttnArgs p) {
    const int me = blockIdx.x;
    const int first = scalar_load(p.joins + me * 4);
    if (first < 0) return;
    const int b = scalar_load(p.joins + me * 4 + 1), head = scalar_load(p.joins + me * 4 + 2),
              tile = scalar_load(p.joins + me * 4 + 3);
    const Seq s = seq_at(p, b);
    constexpr int kLanes = D / 4, kAtOnce = kThreads / kLanes;
    const int rows = min(ROWS, s.nq * p.share - tile * ROWS);
    const int l0 = threadIdx.x % kLanes, c = 4 * l0, self = threadIdx.x & 63 & ~(kLanes - 1);
    for (int r0 = blockIdx.y * kAtOnce; r0 < rows; r0 += gridDim.y * kAtOnce) {
        const int r = min(r0 + static_cast<int>(threadIdx.x) / kLanes, rows - 1);
        const auto part = [&](int w) {
            return p.part + (2 * int64_t(w) + (w == first)) * part_floats<D>(ROWS) + int64_t(r) * (D + 2);
        };
        // a row's lanes look at a part each
        float top = kNone;
        for (int w = first + l0; w <= me; w += kLanes) top = fmaxf(top, part(w)[D]);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        float v[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
        for (int w0 = first; w0 <= me; w0 += kLanes) {
            const int w = w0 + l0;
            float f = 0.f, lw = 0.f;
            if (w <= me) {
                const float2 ml = *reinterpret_cast<const float2*>(part(w) + D);
                f = ml.x == kNone ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
                lw = ml.y;
            }
            const int many = min(kLanes, me + 1 - w0);
            for (int i = 0; i < many; i += 8) {  // eight parts in flight
                float2 x0[8], x1[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float* const x = part(w0 + min(i + k, many - 1));  // again, for nothing: f is 0
                    x0[k] = *reinterpret_cast<const float2*>(x + c), x1[k] = *reinterpret_cast<const float2*>(x + c + 2);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float fi = __shfl(f, self + i + k, 64);
                    l = __builtin_fmaf(__shfl(lw, self + i + k, 64), fi, l);
                    v[0] = __builtin_fmaf(x0[k].x, fi, v[0]);
                    v[1] = __builtin_fmaf(x0[k].y, fi, v[1]);
                    v[2] = __builtin_fmaf(x1[k].x, fi, v[2]);
                    v[3] = __builtin_fmaf(x1[k].y, fi, v[3]);
                }
            }
        }
        if (r0 + static_cast<int>(threadIdx.x) / kLanes >= rows) continue;
        const int row = tile * ROWS + r, token = token_of(p, row), qh = head * p.share + row - token * p.share;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T* const o = row_ptr<T>(p.out, s.q0 + token, qh) + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = static_cast<T>(v[k] * inv);
        if (p.lse && c == 0)
            p.lse[int64_t(s.q0 + token) * p.q_heads + qh] =
                l == 0.f ? kNone : (top + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
    }
}

struct Plan {
    int rows, groups;
    size_t bytes;
};

constexpr int wide_blocks(int esz, int dim) { return esz == 4 || dim == 128 ? 1 : kWideBlocks; }
constexpr int wide_rows(int a_dtype, int dim) { return 128 * wide_blocks(a_dtype == CF_F32 ? 4 : 2, dim); }

// The kernel for a call: rows is the number of rows that the longest sequence has.
Plan plan_of(int a_dtype, int head_dim, int64_t rows) {
    const int large = wide_rows(a_dtype, head_dim);
    Plan x;
    x.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : large;
    x.groups = x.rows == 16 ? kGroupsSmall : x.rows == 32 ? kGroupsSmall / 2 : (a_dtype == CF_F32 ? 128 / head_dim : head_dim == 64 ? KR64 : 2) * kGroupsLarge;
    const int64_t floats = head_dim == 64 ? part_floats<64>(x.rows) : part_floats<128>(x.rows);
    x.bytes = size_t(x.groups) * (2 * floats * 4 + 16);
    return x;
}

template <typename T, int D, int NQ, bool SPLIT>
hipError_t launch(const AttnArgs& p, int64_t max_rows, hipStream_t stream) {
    constexpr int kRows = Shape<T, D, NQ, SPLIT>::kRows, kJoinRows = kThreads / (D / 4);
    const int join_rows = max_rows < kRows ? static_cast<int>(max_rows) : kRows;
    attn_kernel<T, D, NQ, SPLIT><<<p.groups, kThreads, 0, stream>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<T, D, kRows><<<dim3(p.groups, (join_rows + kJoinRows - 1) / kJoinRows), kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_rows(int rows, const AttnArgs& p, int64_t max_rows, hipStream_t stream) {
    constexpr int kQB = wide_blocks(sizeof(T), D);
    if (rows == 16) return launch<T, D, 1, true>(p, max_rows, stream);
    if (rows == 32) return launch<T, D, 2, true>(p, max_rows, stream);
    constexpr int kRows = Wide<T, D, kQB>::kRows, kJoinRows = kThreads / (D / 4);
    wide_kernel<T, D, kQB><<<p.groups, kThreads, 0, stream>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<T, D, kRows><<<dim3(p.groups, kRows / kJoinRows), kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

size_t kv4_attention_workspace(int a_dtype, int head_dim, int64_t max_rows) {
    return plan_of(a_dtype, head_dim, max_rows).bytes;
}

hipError_t launch_kv4_attention(int a_dtype, const Kv4Attention& c, void* workspace, hipStream_t stream) {
    const int share = c.q_heads / c.cache.heads;
    const int64_t max_rows = c.max_q * share;
    const Plan x = plan_of(a_dtype, c.cache.block.dim, max_rows);
    AttnArgs p{};
    p.q = c.q, p.out = c.out, p.cache = c.cache, p.table = c.table, p.width = c.table_width;
    p.kv_lens = c.kv_lens, p.q_starts = c.q_starts, p.total_q = static_cast<int>(c.total_q);
    p.q_each = c.q_starts ? 0 : static_cast<int>(c.total_q / c.batch);
    p.batch = c.batch, p.q_heads = c.q_heads, p.share = share;
    p.causal = c.causal, p.window = c.window;
    p.scale_log2 = c.scale * 1.44269504088896341f;
    p.lse = c.lse;
    p.groups = x.groups;
    p.joins = static_cast<int32_t*>(workspace);
    p.part = reinterpret_cast<float*>(p.joins + 4 * x.groups);
    const bool d64 = c.cache.block.dim == 64;
    if (a_dtype == CF_BF16)
        return d64 ? launch_rows<__bf16, 64>(x.rows, p, max_rows, stream) : launch_rows<__bf16, 128>(x.rows, p, max_rows, stream);
    return d64 ? launch_rows<float, 64>(x.rows, p, max_rows, stream) : launch_rows<float, 128>(x.rows, p, max_rows, stream);
}

}  // namespace cf
