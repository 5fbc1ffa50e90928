// The attention kernel for many rows, over tiles of keys that a workgroup's four waves share through shared memory.
// A source S says where keys come from and how a tile lies in shared memory (cf_attn.hip: rows; cf_kv8_attn.hip: a
// cache's pages).
#pragma once

#include "cf_attn_plan.h"

namespace cf {
namespace {

// Shape of a kernel: source SRC with its types, RB blocks of 32 rows a wave, work-groups of a compute unit.
//
// What a wave does with 32 keys and 32 rows (matrix products of 32 x 32 with 16 terms; lane = 32 h + n):
//   S^T = K Q^T   K's rows are keys, in such an order that lane (h, n) ends up with the scores of keys 8 h .. 8 h + 7
//                 and 16 + 8 h .. for row n
//   O^T = V^T P^T the terms are keys: the lane has them.
// A step multiplies the next 32 keys by the queries and this 32 keys' probabilities by V: the products of the one go
// beside the exponentials of the other, in one wave, so that the matrix units need no second wave to be kept busy.
template <typename SRC, int RB>
struct Tile {
    using Source = SRC;
    using Type = typename SRC::Type;
    static constexpr int kDim = SRC::kDim;
    static constexpr int kRB = RB;
    static constexpr int kRows = 32 * RB * kWaves;
    static constexpr int kKeys = SRC::kKeys;  // of a tile: 32 or 64
    static constexpr int kSub = kKeys / 32;
    static constexpr int kPad = SRC::kPad;
    static constexpr int kResident = SRC::kResident;
    static constexpr int kBuffers = 3;
};

// The reference follows a row's largest score when that has risen by more than 2^kRise.
constexpr float kRise = 8.f;

// Rows of keys, [key][D] bf16 in chunks of 16 bytes that lie turned by their row: the 16 rows that a product's lanes
// read at once, and the consecutive chunks of the rows that are written at once, are then on different banks.
template <int D>
struct KeyRows {
    __host__ __device__ static constexpr uint32_t chunk(int row, int c) {
        return row * (2 * D) + ((c ^ (D == 128 ? row & 15 : row >> 1 & 7)) << 4);
    }
    // key of row n of a product's 32: lane (h, n) gets scores of keys 8 h .. and 16 + 8 h ..
    __device__ static constexpr int key_of(int n) { return 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3); }
};

// The nearest bf16 to a number, which keeps the rest: three in turn are all of it, and the second is at most 2^-8 of
// the whole and the third 2^-17.  Beyond 3.39e38 the nearest is infinite.
__device__ __forceinline__ __bf16 round_bf16(float* rest) {
    const __bf16 b = static_cast<__bf16>(*rest);
    *rest -= static_cast<float>(b);
    return b;
}

// bf16 that is infinite or NaN, in a word of two: its bits all set.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
    const uint32_t lo = (w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u, hi = (w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
    return lo | hi;
}

template <typename K>
__global__ __launch_bounds__(kThreads, K::kResident) void tile_kernel(const typename K::Source::Args p) {
    using S = typename K::Source;
    using T = typename K::Type;
    constexpr int D = K::kDim, RB = K::kRB, kRows = K::kRows, kKeys = K::kKeys, kSub = K::kSub, kPad = K::kPad;
    constexpr int QP = S::kQueryParts, KP = S::kKeyParts, kMost = (QP > KP ? QP : KP) - 1;
    constexpr int kC = D / 16, kDt = D / 32;
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 31, h = lane >> 5;
    __shared__ __align__(256) uint8_t lds[K::kBuffers * S::kBytes];
    __shared__ uint8_t flags[K::kBuffers][4];

    Place w;
    const bool work = place_of<kRows, kKeys, kPad>(p, &w);
    const int me = w.me;
    if (threadIdx.x == 0) p.joins[me * kJoin] = -1;
    if (!work) return;
    Seq s = seq_at(p, w.b);
    S src;
    src.begin(p);

    while (w.at < w.end) {
        int u0;
        const int count = units_of<kRows, kKeys>(p, s, w.tile, &u0);
        const int64_t take = min(w.end - w.at, count + kPad - w.rest);
        const int a = max(static_cast<int>(w.rest) - kPad, 0), z = static_cast<int>(w.rest + take) - kPad;
        w.at += take;
        if (z <= 0) break;  // the next workgroup begins this item
        const int rows = s.nq * p.share;
        const int row0 = w.tile * kRows + wave * 32 * RB;  // the wave's first
        const int tiles = z - a, base = (u0 + a) * kKeys;   // the run's first key

        src.item(p, s, w.b, w.head);
        src.load(p, s, base);

        vb8 q[RB][QP][kC];
        int lo[RB], hi[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int row = row0 + 32 * b + n;
            const bool on = row < rows;
            const int token = on ? token_of(p, row) : 0, q_head = w.head * p.share + (on ? row - token * p.share : 0);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                float f[8];
                if (on) {
                    Row8<T> r;
                    r.load(row_ptr<T>(p.q, s.q0 + token, q_head) + 16 * c + 8 * h);
                    r.get(f);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float rest = on ? f[j] : 0.f;
#pragma unroll
                    for (int k = 0; k < QP; ++k) q[b][k][c][j] = S::part(&rest);
                }
            }
            lo[b] = on ? seen_lo(p, s, token) : 0, hi[b] = on ? seen_hi(p, s, token) : 0;
        }
        int full_lo = 0, full_hi = INT32_MAX;  // keys that all of the wave's rows see
        const int row1 = min(row0 + 32 * RB, rows) - 1;
        if (row1 >= row0) full_lo = seen_lo(p, s, token_of(p, row1)), full_hi = seen_hi(p, s, token_of(p, row0));

        vf16 o[RB][kDt];
        float m[RB], sum[RB];  // m: reference in units of log2
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            m[b] = kNone, sum[b] = 0.f;
#pragma unroll
            for (int j = 0; j < kDt; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k) o[b][j][k] = 0.f;
        }

        vf16 now[RB], next[RB];  // scores
        uint32_t none_now = 0, none_next = 0;  // 16 keys without a page, a bit each

        // scores of keys 32 half .. of the tile in a buffer
        const auto qk = [&](vf16 (&x)[RB], int buf, int half) {
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) x[b][r] = 0.f;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                vb8 kf[KP];
#pragma unroll
                for (int k = 0; k < KP; ++k) kf[k] = src.k_frag(lds, buf, half, k, c);
#pragma unroll
                for (int t = kMost; t >= 0; --t)  // the smallest parts first
#pragma unroll
                    for (int k = 0; k < KP; ++k) {
                        if (t - k < 0 || t - k >= QP) continue;
#pragma unroll
                        for (int b = 0; b < RB; ++b)
                            x[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[k], q[b][t - k][c], x[b], 0, 0, 0);
                    }
            }
        };
        // score r is of key key0 + 8 h + 16 (r / 8) + r % 8
        const auto mask = [&](vf16 (&x)[RB], int key0, uint32_t none) {
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int key = key0 + 8 * h + 16 * (r / 8) + r % 8;
                    if ((none >> (r / 8) & 1u) || key < lo[b] || key >= hi[b]) x[b][r] = kNone;
                }
        };
        const auto on_edge = [&](int key0, uint32_t none) { return key0 < full_lo || key0 + 32 > full_hi || none != 0; };
        // moves the references to new scores
        const auto refer = [&](vf16 (&x)[RB]) {
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                float top = kNone;
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, x[b][r]);
                top *= p.scale_log2;
                if (__any(top > m[b] + kRise)) {
                    const float r = fmaxf(fmaxf(top, __shfl_xor(top, 32, 64)), m[b]);
                    const float f = m[b] == r ? 1.f : __builtin_amdgcn_exp2f(m[b] - r);
                    m[b] = r;
                    sum[b] *= f;
#pragma unroll
                    for (int j = 0; j < kDt; ++j) o[b][j] *= f;
                }
            }
        };
        // probabilities of scores, times V of their keys
        const auto pv = [&](vf16 (&x)[RB], int buf, int half, int key0, bool edge) {
            vb8 pf[RB][2][QP];
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                const float ref = m[b] == kNone ? 0.f : -m[b];
                float more = 0.f;  // first by itself: one by one, small ones would be lost beside a large sum
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b][r], p.scale_log2, ref));
                    more += e;
                    if constexpr (QP == 1)
                        pf[b][r / 8][0][r % 8] = static_cast<__bf16>(e);
                    else
#pragma unroll
                        for (int k = 0; k < QP; ++k) pf[b][r / 8][k][r % 8] = S::part(&e);
                }
                sum[b] += more;
            }
            bool bad = false;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < kDt; ++j) {
                    vb8 vf[KP];
#pragma unroll
                    for (int k = 0; k < KP; ++k) vf[k] = src.v_frag(lds, buf, half, k, t, j);
                    if (edge) {
                        // a probability of zero times an infinity or NaN would be NaN
#pragma unroll
                        for (int k = 0; k < KP; ++k) {
                            vu4 y = __builtin_bit_cast(vu4, vf[k]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t z2 = not_finite2(y[i]);
                                bad |= z2 != 0;
                                y[i] &= ~z2;
                            }
                            vf[k] = __builtin_bit_cast(vb8, y);
                        }
                    }
#pragma unroll
                    for (int i = kMost; i >= 0; --i)
#pragma unroll
                        for (int k = 0; k < KP; ++k) {
                            if (i - k < 0 || i - k >= QP) continue;
#pragma unroll
                            for (int b = 0; b < RB; ++b)
                                o[b][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[k], pf[b][t][i - k], o[b][j], 0, 0, 0);
                        }
                }
            if (edge && __any(bad)) {
                // they reach the rows that see their keys, and only those
#pragma unroll 1
                for (int t = 0; t < 32; ++t) {
                    const int key = key0 + t;
#pragma unroll
                    for (int j = 0; j < kDt; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (src.v_bad(lds, buf, half, t, 32 * j + 8 * (r / 4) + 4 * h + r % 4))
#pragma unroll
                                for (int b = 0; b < RB; ++b)
                                    if (key >= lo[b] && key < hi[b]) o[b][j][r] = __builtin_nanf("");
                }
            }
        };

        // Tile t is read from buffer t % 3, and written there two barriers after the tile before it there was read.
        __syncthreads();  // the last item's tiles have been read
        src.store(p, s, lds, flags[0], 0, base);
        if (tiles > 1) src.load(p, s, base + kKeys);
        int buf = 0, next_buf = 1;  // of tile t, and of the one that is stored
#pragma unroll 1
        for (int t = 0; t <= tiles; ++t) {
            const int key0 = base + t * kKeys;
            const int last_buf = buf == 0 ? 2 : buf - 1;
            if (t < tiles) {
                __syncthreads();
                if (t + 1 < tiles) src.store(p, s, lds, flags[next_buf], next_buf, key0 + kKeys);
                if (t + 2 < tiles) src.load(p, s, key0 + 2 * kKeys);
                none_next = S::none(flags[buf], 0);
                qk(next, buf, 0);
            }
            if (t > 0) pv(now, last_buf, kSub - 1, key0 - 32, on_edge(key0 - 32, none_now));
            if (t == tiles) break;
            if (on_edge(key0, none_next)) mask(next, key0, none_next);
            refer(next);
#pragma unroll
            for (int b = 0; b < RB; ++b) now[b] = next[b];
            none_now = none_next;
            if constexpr (kSub == 2) {
                none_next = S::none(flags[buf], 1);
                qk(next, buf, 1);
                pv(now, buf, 0, key0, on_edge(key0, none_now));
                if (on_edge(key0 + 32, none_next)) mask(next, key0 + 32, none_next);
                refer(next);
#pragma unroll
                for (int b = 0; b < RB; ++b) now[b] = next[b];
                none_now = none_next;
            }
            buf = next_buf;
            next_buf = next_buf == 2 ? 0 : next_buf + 1;
        }

        const bool whole = a == 0 && z == count;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const float l = sum[b] + __shfl_xor(sum[b], 32, 64);
            const int row = row0 + 32 * b + n;
            if (row >= rows) continue;
            const int token = token_of(p, row), q_head = w.head * p.share + row - token * p.share;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T* const dst = row_ptr<T>(p.out, s.q0 + token, q_head);
            float* const y = p.part + (2 * int64_t(me) + (a == 0)) * part_floats<D>(kRows) + int64_t(row - w.tile * kRows) * (D + 2);
            // registers 4 k .. are channels 8 k + 4 h ..
#pragma unroll
            for (int j = 0; j < kDt; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = 32 * j + 8 * k + 4 * h;
                    const vf4 x{o[b][j][4 * k], o[b][j][4 * k + 1], o[b][j][4 * k + 2], o[b][j][4 * k + 3]};
                    if (!whole) {
                        *reinterpret_cast<float2*>(y + c) = float2{x[0], x[1]};
                        *reinterpret_cast<float2*>(y + c + 2) = float2{x[2], x[3]};
                    } else if constexpr (sizeof(T) == 4) {
                        *reinterpret_cast<vf4*>(dst + c) = x * inv;
                    } else {
                        typedef __bf16 vb4 __attribute__((ext_vector_type(4)));
                        *reinterpret_cast<vb4*>(dst + c) = __builtin_convertvector(x * inv, vb4);
                    }
                }
            if (h == 0) {
                if (!whole)
                    *reinterpret_cast<float2*>(y + D) = float2{m[b], l};
                else if (p.lse)
                    p.lse[int64_t(s.q0 + token) * p.q_heads + q_head] = lse_of(m[b], l);
            }
        }
        if (threadIdx.x == 0 && a > 0 && z == count) {
            int32_t* const j = p.joins + me * kJoin;
            j[1] = w.head, j[2] = s.q0, j[3] = w.tile * kRows, j[4] = min(kRows, rows - w.tile * kRows);
            // the workgroup with the item's first unit
            j[0] = static_cast<int32_t>((w.at - count) / w.chunk);
        }

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
