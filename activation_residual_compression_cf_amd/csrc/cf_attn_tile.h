// The attention kernel for many rows, over tiles of keys that a workgroup's waves share through shared memory.
// A source S says where keys come from and how a tile lies in shared memory (cf_attn.hip: rows; cf_kv8_attn.hip: a
// cache's pages).
#pragma once

#include "cf_attn_join.h"

namespace cf {
namespace {

// Shape of a kernel: source SRC with its types, 32 rows a wave.
//
// What a wave does with 32 keys and 32 rows (matrix products of 32 x 32 with 16 terms; lane = 32 h + n):
//   S^T = K Q^T   K's rows are keys, in such an order that lane (h, n) ends up with the scores of keys 8 h .. 8 h + 7
//                 and 16 + 8 h .. for row n
//   O^T = V^T P^T the terms are keys: the lane has them.
template <typename SRC>
struct Tile {
    static constexpr int kGroup = 64 * SRC::kWaves;  // threads
    using Source = SRC;
    using Type = typename SRC::Type;
    static constexpr int kDim = SRC::kDim;
    static constexpr int kRows = 32 * SRC::kWaves;
    static constexpr int kKeys = SRC::kKeys;  // of a tile: 32 or 64
    static constexpr int kSub = kKeys / 32;
    static constexpr int kPad = SRC::kPad;
    static constexpr int kResident = SRC::kResident;
    static constexpr int kBuffers = 3;
    static constexpr bool kJoins = true;  // by itself
};

// A row's reference follows its largest score when that has risen by more than 2^kRiseLog2, or (kSums) when its
// probabilities of a tile add up to more than kRise in a lane: none is larger otherwise.  The sums are there, which
// saves a tenth of the vector instructions at 64 channels, and they are looked at twice a tile.  For rows that pays
// (all tokens of a video 3007 -> 2896 us; 16384 rows over 16384 keys of 128 channels 2043 -> 2008), for the
// 8-bit cache it does not (2925 rows over 17550 keys of 64 channels 541 -> 559, prompts in chunks 170 -> 174).
constexpr float kRise = 256.f, kRiseLog2 = 8.f;

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

// A byte of each wave, about its share of a tile.
typedef uint64_t FlagWord;

// Nothing moves across: what is read before is in flight while what stands before is worked on.
__device__ __forceinline__ void stay() { __builtin_amdgcn_sched_barrier(0); }

// Where values have several parts, a wave has the SIMD for itself and products and vector instructions take equally long:
// each product is followed by some of the others, which run beside it.  Left alone, the compiler puts twenty and more
// in a row (fp32 rows: 1301 us and 1236 so for 4096 over 4608 keys; an image over the 8-bit cache 99.5 and 97.6).
template <int PRODUCTS, int BESIDE>
__device__ __forceinline__ void mix() {
    if constexpr (PRODUCTS > 1) {
#pragma unroll
        for (int i = 0; i < PRODUCTS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);       // a matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x002, BESIDE, 0);  // vector instructions
        }
    }
}

// Keeps the computation of a value where it stands: left alone, the compiler moves it behind the branches to its use, and
// nothing goes beside the products any more.
template <typename V>
__device__ __forceinline__ void here(V& x) {
    asm volatile("" : "+v"(x));
}

// A barrier for what is in shared memory: loads of global memory stay under way.
__device__ __forceinline__ void share_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <typename K>
__global__ __launch_bounds__(K::kGroup, K::kResident * K::Source::kWaves / 4) void tile_kernel(const typename K::Source::Args p) {
    using S = typename K::Source;
    using T = typename K::Type;
    constexpr int D = K::kDim, kRows = K::kRows, kKeys = K::kKeys, kSub = K::kSub, kPad = K::kPad;
    constexpr int QP = S::kQueryParts, KP = S::kKeyParts, kMost = (QP > KP ? QP : KP) - 1;
    constexpr int kC = D / 16, kDt = D / 32;
    constexpr int kProducts = KP == 1 ? QP : QP * (QP + 1) / 2, kBeside = KP == 1 ? 6 : 8;
    static_assert(KP == 1 || KP == QP, "");
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 31, h = lane >> 5;
    __shared__ __align__(256) uint8_t lds[K::kBuffers * S::kBytes];
    // of each buffer's tile: a byte for each wave's share, and which of V's elements are infinite or NaN
    __shared__ __align__(8) uint8_t flags[K::kBuffers][8];
    __shared__ uint8_t bads[K::kBuffers][S::kBad];

    Place w;
    const bool work = place_of<kRows, kKeys, kPad, S::kLeast>(p, &w);
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
        const int row0 = w.tile * kRows + wave * 32;  // the wave's first
        const int tiles = z - a, base = (u0 + a) * kKeys;   // the run's first key

        src.item(p, s, w.b, w.head, base);
        src.next_tile(p, s, base, true);
#pragma unroll
        for (int i = 0; i < S::kPieces; ++i) src.load(i);

        vb8 q[QP][kC];
        int lo, hi;  // keys that the lane's row sees
        {
            const int row = row0 + n;
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
                    for (int k = 0; k < QP; ++k) q[k][c][j] = S::part(&rest);
                }
            }
            lo = on ? seen_lo(p, s, token) : 0, hi = on ? seen_hi(p, s, token) : 0;
        }
        int full_lo = 0, full_hi = INT32_MAX;  // keys that all of the wave's rows see
        const int row1 = min(row0 + 32, rows) - 1;
        if (row1 >= row0) full_lo = seen_lo(p, s, token_of(p, row1)), full_hi = seen_hi(p, s, token_of(p, row0));

        vf16 o[kDt];
        // m: reference in units of log2; rows that see nothing have nothing to follow
        float m = lo < hi ? kNone : 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < kDt; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) o[j][k] = 0.f;

        uint64_t bad = 0;  // the lane's channels (a bit for each of o) that an infinity or NaN of V has reached
        int wg_lo = 0, wg_hi = INT32_MAX;  // keys that all of the item's rows see
        {
            const int r0 = w.tile * kRows, r1 = min(r0 + kRows, rows) - 1;
            if (r1 >= r0) wg_lo = seen_lo(p, s, token_of(p, r1)), wg_hi = seen_hi(p, s, token_of(p, r0));
        }
        // The tile from key0 is all on its way to a buffer.
        const auto stored = [&](int buf, int key0) {
            src.stored(p, s, flags[buf], bads[buf], lds, buf, key0 < wg_lo || key0 + kKeys > wg_hi);
        };
        // The operands of a tile's products, in their order: K's terms 16 (f % kC) of half f / kC of the keys, then V's of half
        // v / (2 kDt), terms 16 (v / kDt % 2), channels 32 (v % kDt), then the next tile's.  They are read kAhead before they
        // are used.
        constexpr int kKs = kSub * kC, kVs = kSub * 2 * kDt, kAhead = KP == 1 ? 4 : 2, kRing = 2 * kAhead;
        static_assert((kKs + kVs) % kRing == 0, "a ring's places are the same in every tile");
        vb8 ring[kRing][KP];
        const auto fetch = [&](int f, int buf, int next_buf) {
            const int v = f - kKs, n = v - kVs;
#pragma unroll
            for (int k = 0; k < KP; ++k)
                ring[f % kRing][k] = f < kKs  ? src.k_frag(lds, buf, f / kC, k, f % kC)
                                     : v < kVs ? src.v_frag(lds, buf, v / (2 * kDt), k, v / kDt % 2, v % kDt)
                                               : src.k_frag(lds, next_buf, n / kC, k, n % kC);
        };

        // Tile t is in buffer t % 3.  One barrier a tile, in its middle: before it waves read K of tile t, write tile t + 1
        // and may still read V of tile t - 1; behind it they read V of tile t and the first of K of tile t + 1.
        share_barrier();  // the last item's tiles have been read
#pragma unroll
        for (int i = 0; i < S::kPieces; ++i) src.store(lds, 0, i);
        stored(0, base);
        src.next_tile(p, s, base + kKeys, tiles > 1);
#pragma unroll
        for (int i = 0; i < S::kPieces; ++i) src.load(i);
        share_barrier();
#pragma unroll
        for (int f = 0; f < kAhead; ++f) fetch(f, 0, 1);
        int buf = 0, next_buf = 1;  // of tiles t and t + 1
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const int key0 = base + t * kKeys;
            FlagWord flag = static_cast<uint32_t>(uniform(static_cast<int>(*reinterpret_cast<const uint32_t*>(flags[buf]))));
            if constexpr (S::kWaves > 4) flag |= static_cast<FlagWord>(static_cast<uint32_t>(uniform(static_cast<int>(*reinterpret_cast<const uint32_t*>(flags[buf] + 4))))) << 32;
            const bool edge = key0 < full_lo || key0 + kKeys > full_hi || S::none(flag) != 0;

            vf16 x[kSub];             // scores: r of half g is of key key0 + 32 g + 8 h + 16 (r / 8) + r % 8
            vu4 pf[kSub][2][QP];      // their probabilities: bf16 in pairs
            float ref, more, before;  // before: of more, what the first half gave
            const auto key_product = [&](int f) {
                if (f % kC == 0)
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[f / kC][r] = 0.f;
                fetch(f + kAhead, buf, next_buf);
#pragma unroll
                for (int i = kMost; i >= 0; --i)  // the smallest parts first
#pragma unroll
                    for (int k = 0; k < KP; ++k) {
                        if (i - k < 0 || i - k >= QP) continue;
                        x[f / kC] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[f % kRing][k], q[i - k][f % kC], x[f / kC], 0, 0, 0);
                    }
            };
            const auto value_product = [&](int v) {
                fetch(kKs + v + kAhead, buf, next_buf);
#pragma unroll
                for (int i = kMost; i >= 0; --i)
#pragma unroll
                    for (int k = 0; k < KP; ++k) {
                        if (i - k < 0 || i - k >= QP) continue;
                        o[v % kDt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            ring[(kKs + v) % kRing][k], __builtin_bit_cast(vb8, pf[v / (2 * kDt)][v / kDt % 2][i - k]), o[v % kDt], 0, 0, 0);
                    }
            };
            // pairs i0 .. i1 - 1 of half g's probabilities
            const auto exps = [&](int g, int i0, int i1) {
#pragma unroll
                for (int i = i0; i < i1; ++i) {
                    float e[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[g][2 * i + j], p.scale_log2, ref));
                        more += e[j];
                    }
                    here(more);
#pragma unroll
                    for (int k = 0; k < QP; ++k) {
                        const vb2 y = QP == 1 ? vb2{static_cast<__bf16>(e[0]), static_cast<__bf16>(e[1])} : vb2{S::part(&e[0]), S::part(&e[1])};
                        uint32_t word = __builtin_bit_cast(uint32_t, y);
                        here(word);
                        pf[g][i / 4][k][i % 4] = word;
                    }
                }
            };
            // hides what rows do not see
            const auto mask = [&](int g) {
                if (!edge) return;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int run = 2 * g + r / 8, key = key0 + 8 * h + 16 * run + r % 8;
                    if ((S::none(flag) >> run & 1u) || key < lo || key >= hi) x[g][r] = kNone;
                }
            };
            // Moves the references up to half g's scores where a row sees its first key, or where its probabilities so far add
            // up to more than kRise: to whole numbers, so that what is moved with them stays as exact.
            // made: the probabilities have been made from the old references.  Nearly always those hold, nothing
            // waits for a decision, and no maximum is taken; else they are made again.
            // Rows decide for themselves, so that none depends on those beside it.
            const auto settle = [&](int g, bool made) {
                float top;
                const auto largest = [&]() {
                    top = kNone;
#pragma unroll
                    for (int r = 0; r < 16; ++r) top = fmaxf(top, x[g][r]);
                    top *= p.scale_log2;
                };
                if (!made) largest();
                const bool rise = made ? m == kNone || more > kRise : top > m + kRiseLog2;
                if (!__any(rise)) return;
                if (made) largest();
                // both lanes of a row, whatever either says
                const int others = __shfl_xor(static_cast<int>(rise), 32, 64);
                const float most = fmaxf(top, __shfl_xor(top, 32, 64));
                const float r = rise | others ? fmaxf(__builtin_ceilf(most), m) : m;
                const float f = m == r ? 1.f : __builtin_amdgcn_exp2f(m - r);
                m = r;
                sum *= f;
                more = before * f;
#pragma unroll
                for (int j = 0; j < kDt; ++j) o[j] *= f;
                ref = m == kNone ? 0.f : -m;
                if (made) exps(g, 0, 8);
            };

            // The same where the maximum is taken, for both halves of a tile at once: the first half's probabilities have been made.
            float most;
            const auto follow = [&](int g, int r0, int r1) {
#pragma unroll
                for (int r = r0; r < r1; ++r) most = fmaxf(most, x[g][r]);
                here(most);
            };
            const auto settle_both = [&]() {
                most *= p.scale_log2;
                if (!__any(most > m + kRiseLog2)) return;
                const float r = fmaxf(__builtin_ceilf(fmaxf(most, __shfl_xor(most, 32, 64))), m);
                const float f = m == r ? 1.f : __builtin_amdgcn_exp2f(m - r);
                m = r;
                sum *= f;
                more = 0.f;
#pragma unroll
                for (int j = 0; j < kDt; ++j) o[j] *= f;
                ref = m == kNone ? 0.f : -m;
                exps(0, 0, 8);
            };

            // the next tile's stores go beside the last of K's products, the loads of the one behind it beside the first of V's
            const auto store_beside = [&](int f) {
#pragma unroll
                for (int i = S::kPieces * f / kC; i < S::kPieces * (f + 1) / kC; ++i) src.store(lds, next_buf, i);
            };
            const auto load_beside = [&](int v) {
#pragma unroll
                for (int i = S::kPieces * v / (2 * kDt); i < S::kPieces * (v + 1) / (2 * kDt); ++i) src.load(i);
            };
#pragma unroll
            for (int f = 0; f < kC; ++f) {
                key_product(f);
                if (f == 0) __builtin_amdgcn_s_setprio(0);
                if constexpr (kSub == 1) store_beside(f);
                mix<kProducts, kBeside>();
                stay();
            }
            more = before = 0.f, most = kNone, ref = m == kNone ? 0.f : -m;
            mask(0);
            if constexpr (kSub == 2) {
                // a half's probabilities beside the other half's products
#pragma unroll
                for (int f = kC; f < 2 * kC; ++f) {
                    key_product(f);
                    exps(0, 8 * (f - kC) / kC, 8 * (f - kC + 1) / kC);
                    if constexpr (!S::kSums) follow(0, 16 * (f - kC) / kC, 16 * (f - kC + 1) / kC);
                    store_beside(f - kC);
                    mix<kProducts, kBeside>();
                    stay();
                }
                mask(1);
                if constexpr (S::kSums) {
                    settle(0, true);
                    before = more;
                } else {
                    follow(1, 0, 16);
                    settle_both();
                }
            } else {
                settle(0, false);
                exps(0, 0, 4);
            }
            // a wave in its second half goes before one in its first: the two of a SIMD drift apart, and one's vector work
            // meets the other's products (1% of 16384 rows over 16384 keys)
            __builtin_amdgcn_s_setprio(1);
            stored(next_buf, key0 + kKeys);
            src.next_tile(p, s, key0 + 2 * kKeys, t + 2 < tiles);
            share_barrier();
#pragma unroll
            for (int v = 0; v < kVs; ++v) {
                value_product(v);
                if (kSub == 2 && v < 2 * kDt) exps(1, 8 * v / (2 * kDt), 8 * (v + 1) / (2 * kDt));
                if (kSub == 1 && v < kDt) exps(0, 4 + 4 * v / kDt, 4 + 4 * (v + 1) / kDt);
                if (v < 2 * kDt) load_beside(v);
                if (S::kSums && kSub == 2 && v == 2 * kDt - 1) settle(1, true);
                mix<kProducts, kBeside>();
                stay();
            }
            sum += more;
            if (S::found(flag)) {
                // infinities and NaN of V, zeros in the products, reach the rows that see their keys, and only those
#pragma unroll 1
                for (int i = 0; i < kKeys; ++i)
#pragma unroll 1
                    for (int c = 0; c < 16 * kDt; ++c)  // register c % 16 of o[c / 16]
                        if (S::bad(flag, bads[buf], i, c / 16 * 32 + c % 16 / 4 * 8 + 4 * h + c % 4) && key0 + i >= lo && key0 + i < hi)
                            bad |= uint64_t(1) << c;
            }
            buf = next_buf;
            next_buf = next_buf == 2 ? 0 : next_buf + 1;
        }
        if (__any(bad != 0))
#pragma unroll
            for (int c = 0; c < 16 * kDt; ++c)
                if (bad >> c & 1) o[c / 16][c % 16] = __builtin_nanf("");

        float l = sum + __shfl_xor(sum, 32, 64);
        // A part: a wave's values in its own order, side by side over the lanes, and behind all waves' each row's m and l.
        const auto part_at = [&](int64_t slot) { return p.part + slot * part_floats<D>(kRows) + int64_t(wave) * (32 * D) + 2 * lane; };
        const auto row_at = [&](int64_t slot) { return p.part + slot * part_floats<D>(kRows) + kRows * D + 2 * (wave * 32 + n); };
        const bool whole = a == 0 && z == count;
        const bool mine = whole || join_parts(p, w, z, count,
            [&](int64_t slot) {
                if (row0 >= rows) return;
                float* const y = part_at(slot);
#pragma unroll
                for (int i = 0; i < 8 * kDt; ++i) store_far(y + 128 * i, o[i / 8][2 * (i % 8)], o[i / 8][2 * (i % 8) + 1]);
                if (h == 0) store_far(row_at(slot), m, l);
            },
            [&](int64_t slot) {
                if (row0 >= rows) return;
                const float* const y = part_at(slot);
                float2 x[8 * kDt];
                const float2 ml = load_far(row_at(slot));
#pragma unroll
                for (int i = 0; i < 8 * kDt; ++i) x[i] = load_far(y + 128 * i);
                const float top = fmaxf(m, ml.x);
                // zeros of a part that saw nothing, or NaN that must show
                const float f = m == kNone ? 0.f : __builtin_amdgcn_exp2f(m - top), g = ml.x == kNone ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
                m = top;
                l = l * f + ml.y * g;
#pragma unroll
                for (int i = 0; i < 8 * kDt; ++i) {
                    o[i / 8][2 * (i % 8)] = o[i / 8][2 * (i % 8)] * f + x[i].x * g;
                    o[i / 8][2 * (i % 8) + 1] = o[i / 8][2 * (i % 8) + 1] * f + x[i].y * g;
                }
            });
        const int row = row0 + n;
        if (mine && row < rows) {
            const int token = token_of(p, row), q_head = w.head * p.share + row - token * p.share;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T* const dst = row_ptr<T>(p.out, s.q0 + token, q_head);
            // registers 4 k .. are channels 8 k + 4 h ..
#pragma unroll
            for (int j = 0; j < kDt; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = 32 * j + 8 * k + 4 * h;
                    const vf4 x{o[j][4 * k], o[j][4 * k + 1], o[j][4 * k + 2], o[j][4 * k + 3]};
                    if constexpr (sizeof(T) == 4) {
                        *reinterpret_cast<vf4*>(dst + c) = x * inv;
                    } else {
                        typedef __bf16 vb4 __attribute__((ext_vector_type(4)));
                        *reinterpret_cast<vb4*>(dst + c) = __builtin_convertvector(x * inv, vb4);
                    }
                }
            if (h == 0 && p.lse) p.lse[int64_t(s.q0 + token) * p.q_heads + q_head] = lse_of(m, l);
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
