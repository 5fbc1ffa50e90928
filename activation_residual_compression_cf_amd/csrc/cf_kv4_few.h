// The attention kernel for few rows (cf_kv4_attn.hip has the method).
#pragma once

#include "cf_kv4_plan.h"

namespace cf {
namespace {

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
            for (int k = 0; k < PARTS; ++k) x.q[k][i][j] = take_bf16(&rest);
        }
    }
}

// The kernel for few rows: its four waves share the item's 16 * NQ rows and take its units in turn.
//
// What a wave does with 32 keys and 16 rows (matrix products of 16 x 16 with 32 terms; lane =
// 16 g + n):
//   S^T = K Q^T   K rows are keys; lane (g, n) holds a quarter of key row n's channels, which
//                 is one load of codes, and the codes become bf16 by the hardware's
//                 conversion with the group's scale.  Rows are keys in such an order that
//                 lane (g, n) ends up with the scores of keys 8g .. 8g+7 for row n.
//   O^T = V^T P^T the terms are keys: lane (g, n) needs keys 8g .. 8g+7 of its rows, which it
//                 has, and of channel piece n, which is how the cache lays V out: one load.
//                 Conversions give pairs of channels of one key; a byte permutation makes
//                 pairs of keys of them.
// So nothing passes through shared memory, and m, the sum and the rescaling of O are a
// lane's own.  The next unit's codes are loaded, and the page numbers of the one after it, while
// one is worked on (with the numbers loaded beside the codes: 235 us for 64 conversations of 0
// to 32768 keys, 233 MB, where call and join now take 58).  Three contexts of 65537 keys, 642 MB,
// take 140 us with fp32 queries, 4.6 TB/s (129 with two parts of P in place of three).
//
// Workgroups are as many as are resident: with 1024 where 768 fit, the last 256 ran by themselves
// (76 against 66 us), and with two or three rounds of resident ones starts and joins cost more than
// the balance gains (72, 75 us).
template <typename T, int D, int NQ>
struct Few {
    using Type = T;
    static constexpr int kDim = D;
    static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;  // bf16 parts of a query
    static constexpr int kP = Prob<T>::kParts;             // parts of a probability
    static constexpr int kRows = 16 * NQ;
    static constexpr int kPad = 12;  // 8 takes 66 us for the 64 conversations, 12 and 14 59
    // workgroups of a compute unit, by their registers
    static constexpr int kResident = NQ == 2 ? (D == 128 ? 1 : sizeof(T) == 4 ? 2 : 3) : D == 64 ? 4 : sizeof(T) == 4 ? 2 : 3;
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

template <typename T, int D, int NQ>
__global__ __launch_bounds__(kThreads, (Few<T, D, NQ>::kResident)) void few_kernel(const AttnArgs p) {
    using S = Few<T, D, NQ>;
    constexpr int kRows = S::kRows, kPad = S::kPad, kParts = S::kParts, kP = S::kP;
    constexpr int kJ = D / 16;  // O^T tiles of 16 channel pieces
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 15, g = lane >> 4;

    __shared__ float stage[kWaves * 16 * (D + 4)], stage_m[kWaves * 16], stage_l[kWaves * 16];

    Place w;
    const bool work = place_of<kRows, kUnit, kPad>(p, &w);
    const int me = w.me;
    if (threadIdx.x == 0) p.joins[me * kJoin] = -1;
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
        const int row0 = w.tile * kRows;
        const int head = w.head;

        constexpr int kStep = kWaves;
        const int first = a + wave;
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
        float m[NQ], sum[NQ], high[NQ];  // m: reference in units of log2, lowered by kLift
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            m[i] = high[i] = kNone, sum[i] = 0.f;
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

            typename Prob<T>::Frag pf[NQ][kP];
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
                        using Frag = typename Prob<T>::Frag;
                        o[i][2 * j] = Prob<T>::mul16(__builtin_bit_cast(Frag, even), pf[i][k], o[i][2 * j]);
                        o[i][2 * j + 1] = Prob<T>::mul16(__builtin_bit_cast(Frag, odd_), pf[i][k], o[i][2 * j + 1]);
                    }
            };
            if constexpr (D == 128) {
                uint32_t c[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = Prob<T>::template decode<0>(x.v[t], vs[t]);
                pv(0, c);
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = Prob<T>::template decode<1>(x.v[t], vs[t]);
                pv(1, c);
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = Prob<T>::template decode<2>(x.v[t], vs[t]);
                pv(2, c);
#pragma unroll
                for (int t = 0; t < 8; ++t) c[t] = Prob<T>::template decode<3>(x.v[t], vs[t]);
                pv(3, c);
            } else {
                uint32_t c[8];
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    c[t] = t & 1 ? Prob<T>::template decode<2>(x.v[t / 2], vs[t]) : Prob<T>::template decode<0>(x.v[t / 2], vs[t]);
                pv(0, c);
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    c[t] = t & 1 ? Prob<T>::template decode<3>(x.v[t / 2], vs[t]) : Prob<T>::template decode<1>(x.v[t / 2], vs[t]);
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
                        lse_of(top, l);
            } else {
                float* const y = part + int64_t(r) * (D + 2);
#pragma unroll
                for (int k = 0; k < 8; k += 2) *reinterpret_cast<float2*>(y + c + k) = float2{v[k], v[k + 1]};
                if (first_piece) *reinterpret_cast<float2*>(y + D) = float2{top, l};
            }
        };
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if (Prob<T>::kFalls && __any(m[i] != high[i])) {  // lse is more exact from the highest reference
                const float f = m[i] == high[i] ? 1.f : __builtin_amdgcn_exp2f(m[i] - high[i]);
                m[i] = high[i];
                sum[i] *= f;
#pragma unroll
                for (int j = 0; j < kJ; ++j) o[i][j] *= f;
            }
            sum[i] = across_sum(sum[i]);
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
        if (threadIdx.x == 0 && a > 0 && z == count) {
            int32_t* const j = p.joins + me * kJoin;
            j[1] = w.head, j[2] = s.q0, j[3] = w.tile * kRows, j[4] = min(kRows, rows - w.tile * kRows);
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

}  // namespace
}  // namespace cf
