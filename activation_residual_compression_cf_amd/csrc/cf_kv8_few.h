// The kernel for few rows of the attention over the 8-bit cache (cf_kv8_attn.hip has the method).
#pragma once

#include "cf_attn_few.h"
#include "cf_kv8_codes.h"

namespace cf {
namespace {

// One wave's share of 32 keys, as loaded.
template <int D>
struct Keys8 {
    uint32_t k[2][D / 16];  // two rows of keys, a quarter of the channels each
    uint32_t v[D / 8];      // eight keys of D/16 channels
    uint32_t ks, vs;        // scale bytes
    bool ok[2];             // the first and the last 16 keys have a page
};

// The two pages of a unit's first and last 16 keys (one page, where it has 32 tokens or more).
struct Pages8 {
    int at[2];
};

__device__ __forceinline__ Pages8 pages8_of(const Attn8Args& p, const Seq& s, int b, int unit) {
    Pages8 x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // keys behind the last are read from its page (and masked later): always inside the cache
        const int i = min(unit * kUnit + 16 * h, max(s.len - 1, 0)) >> p.cache.shift;
        const int64_t at = int64_t(b) * p.width + i;
        x.at[h] = p.table ? scalar_load(p.table + at) : static_cast<int>(at);
    }
    return x;
}

// Channel of row `row` of O^T's tile j of 16: a lane's D/16 channels lie in pairs, the pairs of four lanes side by
// side (one load of 16 bytes takes a pair's eight keys), and the four rows that a lane ends up with, over all
// tiles, are D/4 consecutive channels.
template <int D>
__device__ __forceinline__ constexpr int channel8(int j, int row) {
    return (row >> 2) * (D / 4) + 8 * (j >> 1) + 2 * (row & 3) + (j & 1);
}

template <int D>
__device__ __forceinline__ void load_keys8(Keys8<D>& x, const Attn8Args& p, const Seq& s, const Pages8& pages, int head, int unit) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const Kv8Block blk{p.cache.block.page, D};
    const int in = unit * kUnit & (blk.page - 1), mask = min(blk.page, kUnit) - 1;
    const uint8_t* base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        x.ok[h] = page_on(p, s, pages.at[h]);
        base[h] = p.cache.at(x.ok[h] ? pages.at[h] : 0, head);
    }
    const uint8_t* const kb = lane & 8 ? base[1] : base[0];
    const uint8_t* const vb = lane & 32 ? base[1] : base[0];
    const int krow = in + ((8 * (n >> 2) + (n & 3)) & mask), vrow = in + (8 * g & mask);
#pragma unroll
    for (int h = 0; h < 2; ++h)  // four tokens further
#pragma unroll
        for (int i = 0; i < D / 16; i += 4) {
            const vu4 w = *reinterpret_cast<const vu4*>(kb + blk.k_code(krow + 4 * h) + g * (D / 4) + 4 * i);
            x.k[h][i] = w.x, x.k[h][i + 1] = w.y, x.k[h][i + 2] = w.z, x.k[h][i + 3] = w.w;
        }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const vu4 w = *reinterpret_cast<const vu4*>(vb + blk.v_code(vrow, channel8<D>(2 * i, n)));
        x.v[4 * i] = w.x, x.v[4 * i + 1] = w.y, x.v[4 * i + 2] = w.z, x.v[4 * i + 3] = w.w;
    }
    x.ks = kb[blk.k_scale(krow)];
    x.vs = vb[blk.v_scale(vrow)];
}

// The kernel for few rows: its four waves share the item's 16 * NQ rows and take its units in turn.
//
// What a wave does with 32 keys and 16 rows (matrix products of 16 x 16 with 32 terms; lane = 16 g + n):
//   S^T = K Q^T   lane (g, n) holds a quarter of key row n's channels, and the hardware's conversion makes bf16 of
//                 the codes with the scale.  Rows are keys in such an order that lane (g, n) ends up with the
//                 scores of keys 8g .. 8g+7 for row n.
//   O^T = V^T P^T the terms are keys: lane (g, n) needs keys 8g .. 8g+7 of its rows, which it has, and of D/16
//                 channels, whose eight codes lie together in the cache: four conversions of pairs are an
//                 operand, with no exchange between lanes and no permutation.
// So nothing passes through shared memory, and the reference, the sum and the rescaling of O are a lane's own.  The
// next unit's codes, and the page numbers of the one after it, are loaded while one is worked on.
template <typename T, int D, int NQ>
struct Few8 {
    using Type = T;
    static constexpr int kDim = D;
    static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;  // bf16 parts of a query
    static constexpr int kP = Prob<T>::kParts;             // parts of a probability
    static constexpr int kRows = 16 * NQ;
    static constexpr int kGroup = kThreads;
    static constexpr bool kJoins = false;  // by itself
    // What an item costs besides its units, and the shortest run (one of 20 units takes 15.3 us for one token over 4097
    // keys, of 12 13.9, of 8 13.4, of 4 14.7).
    static constexpr int kPad = 12, kLeast = 8;
    // workgroups of a compute unit, by their registers: 64 conversations of 0 to 32768 keys take 89 us with two, 137 with
    // one and 105 with three, which spill
    static constexpr int kResident = NQ == 2 ? (D == 128 ? 1 : 2) : D == 64 ? 3 : 2;
};

template <typename T, int D, int NQ>
__global__ __launch_bounds__(kThreads, (Few8<T, D, NQ>::kResident)) void few8_kernel(const Attn8Args p) {
    using S = Few8<T, D, NQ>;
    constexpr int kRows = S::kRows, kPad = S::kPad, kParts = S::kParts, kP = S::kP;
    constexpr int kJ = D / 16;  // O^T tiles of 16 channels
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 15, g = lane >> 4;

    __shared__ float stage[kWaves * 16 * (D + 4)], stage_m[kWaves * 16], stage_l[kWaves * 16];

    Place w;
    const bool work = place_of<kRows, kUnit, kPad, S::kLeast>(p, &w);
    if (threadIdx.x == 0) p.joins[w.me * kJoin] = -1;
    if (!work) return;
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
        const int row0 = w.tile * kRows;
        const int head = w.head;

        constexpr int kStep = kWaves;
        const int first = a + wave;
        Pages8 pages = pages8_of(p, s, w.b, u0 + first);
        Keys8<D> next;
        if (first < z) load_keys8<D>(next, p, s, pages, head, u0 + first);
        if (first + kStep < z) pages = pages8_of(p, s, w.b, u0 + first + kStep);

        Rows<D, kParts> q[NQ];
        int lo[NQ], hi[NQ];                   // keys that row n of each sixteen sees
        int full_lo = 0, full_hi = INT32_MAX; // keys that all of the item's rows see
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
        uint32_t bad[NQ];                // of the lane's values of O, a bit each: what a NaN of V has reached
        float m[NQ], sum[NQ], high[NQ];  // m: reference in units of log2, lowered by kLift
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            m[i] = high[i] = kNone, sum[i] = 0.f, bad[i] = 0;
#pragma unroll
            for (int j = 0; j < kJ; ++j) o[i][j] = vf4{0.f, 0.f, 0.f, 0.f};
        }

        for (int u = first; u < z; u += kStep) {
            Keys8<D> x = next;
            if (u + kStep < z) load_keys8<D>(next, p, s, pages, head, u0 + u + kStep);
            if (u + 2 * kStep < z) pages = pages8_of(p, s, w.b, u0 + u + 2 * kStep);
            const int key0 = (u0 + u) * kUnit;
            const int mine0 = key0 + 8 * g;  // the lane's own eight keys
            const bool ok = lane & 32 ? x.ok[1] : x.ok[0];
            const bool edge = key0 < full_lo || key0 + kUnit > full_hi || !x.ok[0] || !x.ok[1];
            if (edge) {
                // V behind the sequence's last key is whatever an earlier owner of the page left
                const int valid = ok ? min(max(s.len - mine0, 0), 8) : 0;
                const uint64_t keep = valid == 8 ? ~uint64_t(0) : (uint64_t(1) << (8 * valid)) - 1;
                if (valid == 0) x.vs = 127u;
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    x.v[i] &= static_cast<uint32_t>(i & 1 ? keep >> 32 : keep);
                    any |= nan_codes(x.v[i]);
                }
                if (__any(any != 0)) {
                    // zeros in the products, and NaN of V reaches the rows that see its key, and only those
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const uint32_t l = nan_codes(x.v[2 * j]), h = nan_codes(x.v[2 * j + 1]);
                        x.v[2 * j] &= ~full_bytes(l), x.v[2 * j + 1] &= ~full_bytes(h);
                        const int mine = static_cast<int>(four_bits(l) | four_bits(h) << 4);
#pragma unroll 1
                        for (int k = 0; k < 16; ++k) {
                            const int hit = __shfl(mine, 16 * (k >> 2) + 4 * g + (k & 3), 64);  // row 4 g + k % 4 of the tile, keys 8 (k / 4) ..
#pragma unroll
                            for (int i = 0; i < NQ; ++i) {
                                uint32_t see = 0;
                                for (int t = 0; t < 8; ++t) {
                                    const int key = key0 + 8 * (k >> 2) + t;
                                    see |= static_cast<uint32_t>(key >= lo[i] && key < hi[i]) << t;
                                }
                                if (hit & see) bad[i] |= 1u << (4 * j + (k & 3));
                            }
                        }
                    }
                }
            }

            // scores: sc[i][t] is key mine0 + t, row n of the i-th sixteen
            vf4 sc[NQ][2];
            const float ks = scale_of(x.ks);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                vb8 kf[D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) kf[c] = bf16_codes(x.k[h][2 * c], x.k[h][2 * c + 1], ks);
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

            typename Prob<T>::Frag pf[NQ][kP];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                float x2[8];  // scores in units of log2
#pragma unroll
                for (int t = 0; t < 8; ++t) x2[t] = sc[i][t >> 2][t & 3] * p.scale_log2;
                if (edge) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        if (!ok || mine0 + t < lo[i] || mine0 + t >= hi[i]) x2[t] = kNone;
                }
                float top = kNone;
#pragma unroll
                for (int t = 0; t < 8; ++t) top = fmaxf(top, x2[t]);
                uint64_t low = 0;  // rows whose lanes all lie far below, in the first sixteen bits
                if constexpr (Prob<T>::kFalls) {
                    low = __ballot(top < m[i] - kDrop);
                    low &= low >> 32;
                    low &= low >> 16;
                }
                if (__any(top > m[i] + (kSlack + kLift)) || (low & 0xffffu)) {
                    // the lanes of a row agree on its new reference
                    const float r = next_ref<T>(across_max(top), m[i], &high[i]);
                    const float f = m[i] == r ? 1.f : __builtin_amdgcn_exp2f(m[i] - r);
                    m[i] = r;
                    sum[i] *= f;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) o[i][j] *= f;
                }
                const float ref = m[i] == kNone ? 0.f : m[i];
                float more = 0.f;  // first by itself: one by one, small ones would be lost beside a large sum
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    x2[t] = __builtin_amdgcn_exp2f(x2[t] - ref);
                    more += x2[t];
                    Prob<T>::set(pf[i], t, x2[t]);
                }
                sum[i] += more;
            }

            const float vs = scale_of(x.vs);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const auto f = Codes8<T>::frag(x.v[2 * j], x.v[2 * j + 1], vs);
#pragma unroll
                for (int i = 0; i < NQ; ++i)
#pragma unroll
                    for (int k = kP - 1; k >= 0; --k) o[i][j] = Prob<T>::mul16(f, pf[i][k], o[i][j]);
            }
        }

#pragma unroll
        for (int i = 0; i < NQ; ++i)
            if (__any(bad[i] != 0))
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (bad[i] >> (4 * j + r) & 1u) o[i][j][r] = __builtin_nanf("");
        finish_few<T, D, NQ>(p, w, s, a, z, count, o, m, sum, high, stage, stage_m, stage_l, [&](int i, int c) {
            return o[i][2 * (c >> 3) + (c & 1)][c >> 1 & 3];
        });

        // on to the next item
        w.rest = 0;
        if (w.at >= w.end) break;
        if (++w.tile >= tiles_of<kRows>(p, s)) {
            w.tile = 0;
            if (++w.head >= p.kv_heads) {
                w.head = 0;
                do s = seq_at(p, ++w.b);  // at < end <= total: another sequence has units
                while (s.nq == 0);
            }
        }
    }
}

}  // namespace
}  // namespace cf
