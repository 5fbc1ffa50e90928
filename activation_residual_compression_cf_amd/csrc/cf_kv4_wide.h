// The attention kernel for many rows (cf_kv4_attn.hip has the method).
#pragma once

#include "cf_kv4_few.h"

namespace cf {
namespace {

// Four waves, each with 32 rows of its own, over tiles of 64 keys that all of them
// decode once, into shared memory: K as bf16 [key][channel], V as fp16 (bf16 for fp32 queries)
// [channel][key].
// Decoding in registers, as the kernel for few rows does, took a third of the vector units'
// time at 64 rows a wave (165 us for 1024 queries over 4608 keys in 24 heads of 128, where the
// tiles take 88).  64 rows a wave here leave one wave a SIMD, which nothing overlaps: 229 us.
// 4096 queries over 16384 keys run at 911 TFLOP/s at 128 channels and 752 at 64; with fp32 queries,
// whose products are three each, 1024 over 4608 take 187 us.
template <typename T, int D>
struct Wide {
    using Type = T;
    static constexpr int kDim = D;
    static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
    static constexpr int kP = Prob<T>::kParts;
    static constexpr int kRows = 32 * kWaves;
    static constexpr int kKeys = 64;
    // Whether the order of reads and products is fixed, four reads ahead: with two waves a SIMD each
    // product would wait for its read (97 against 99 us for the 1024 queries).  Three waves hide
    // that, and lack the registers (534 against 600 us for 2925 queries over 17550 keys of 64).
    static constexpr bool kAhead = D == 128;
    // workgroups of a compute unit, by their registers; at 64 channels 2 take 597 us and 4, which spill,
    // 591 where 3 take 543
    static constexpr int kResident = sizeof(T) == 4 ? 128 / D : D == 64 ? 3 : 2;
    static constexpr int kPad = 5;  // 2 takes 231 us for the five prompts in chunks, 3 219, 5 216
    // K's rows are 16 bytes longer than they need to be: 16 rows then start on different banks
    static constexpr int kKRow = 2 * D + 16;
    static constexpr int kTile = kKeys * kKRow + D * 2 * kKeys;
    static_assert(kKeys * kKRow % 256 == 0 && kTile % 256 == 0, "V's rows start on 256 bytes");
    // V's rows (a channel's 64 keys) lie two together in 256 bytes, as 16 runs of 8 keys: run q of
    // channel c is number (8 (c & 1) + q) ^ v_turn(c / 2).  Both the 16 consecutive channels that
    // a product reads and the 16 channel pieces that the decoding threads write then lie on
    // different banks (without: half of the LDS cycles were conflicts, 108 against 99 us for the 1024
    // queries).  The turn of c / 2 + x is that of c / 2, ^ x, for x below 4 (2 at 64
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

// Decodes a share into the tile at lds + tile_at, of whose keys the sequence has the first `left`.  Keys behind them
// become zeros whatever their bytes, and so do groups that read NaN: returns whether the
// wave has any of those, and then k_nan and v_nan, [key][group], say which of its keys' do.
template <typename T, int D>
__device__ __forceinline__ bool store_share(Share<D>& x, uint8_t* lds, uint32_t tile_at, uint8_t* k_nan, uint8_t* v_nan, int left) {
    using W = Wide<T, D>;
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
        uint8_t* const w = lds + (tile_at + kin * W::kKRow + (threadIdx.x & 3) * (D / 2));
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
        // a turn of the address: tiles start on 256 bytes
        const uint32_t w = static_cast<uint32_t>(W::kKeys * W::kKRow + first * 256 + (vin & 4) * 2 + 16 * turn) + tile_at;
        using V = Prob<T>;
        const auto pair = [&](int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            *reinterpret_cast<vu2*>(lds + ((w ^ 16 * j) + 256 * j)) =
                vu2{__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(d, c, 0x05040100u)};
            *reinterpret_cast<vu2*>(lds + ((w ^ 16 * (j ^ 8)) + 256 * j)) =
                vu2{__builtin_amdgcn_perm(b, a, 0x07060302u), __builtin_amdgcn_perm(d, c, 0x07060302u)};
        };
        pair(0, V::template decode<0>(v[0], f[0]), V::template decode<0>(v[1], f[1]), V::template decode<0>(v[2], f[2]), V::template decode<0>(v[3], f[3]));
        pair(1, V::template decode<1>(v[0], f[0]), V::template decode<1>(v[1], f[1]), V::template decode<1>(v[2], f[2]), V::template decode<1>(v[3], f[3]));
        if constexpr (D == 128) {
            pair(2, V::template decode<2>(v[0], f[0]), V::template decode<2>(v[1], f[1]), V::template decode<2>(v[2], f[2]), V::template decode<2>(v[3], f[3]));
            pair(3, V::template decode<3>(v[0], f[0]), V::template decode<3>(v[1], f[1]), V::template decode<3>(v[2], f[2]), V::template decode<3>(v[3], f[3]));
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
template <typename T, int D>
__global__ __launch_bounds__(kThreads, (Wide<T, D>::kResident)) void wide_kernel(const AttnArgs p) {
    using W = Wide<T, D>;
    constexpr int kRows = W::kRows, kPad = W::kPad, kParts = W::kParts, kP = W::kP, kKeys = W::kKeys;
    constexpr int kDt = D / 32;
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 31, h = lane >> 5;
    __shared__ __align__(256) uint8_t lds[W::kBytes];
    __shared__ uint32_t flag[2];  // of a tile's 16 keys, a byte for each wave: 1 a group that reads NaN, 2 no page
    __shared__ uint8_t k_nan[2][kKeys * 4], v_nan[2][kKeys * kDt];

    Place w;
    const bool work = place_of<kRows, kKeys, kPad>(p, &w);
    const int me = w.me;
    if (threadIdx.x == 0) p.joins[me * kJoin] = -1;
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
        const int row = w.tile * kRows + wave * 32 + n;  // the lane's
        const bool on = row < rows;
        const int token = on ? token_of(p, row) : 0;
        const int q_head = w.head * p.share + (on ? row - token * p.share : 0);

        const int wave_key = 16 * wave;
        Share<D> next;
        int pages = page_at(p, s, w.b, (u0 + a) * kKeys);  // of the tile to load next
        const auto load_next = [&](int u) {
            const int page = __builtin_amdgcn_readlane(pages, wave);
            pages = page_at(p, s, w.b, (u0 + u + 1) * kKeys);
            load_share<D>(next, p, s, page, offs, w.head, (u0 + u) * kKeys + wave_key);
        };
        load_next(a);

        vb8 q[kParts][D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
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
                for (int k = 0; k < kParts; ++k) q[k][c][j] = take_bf16(&rest);
            }
        }
        const int lo = on ? seen_lo(p, s, token) : 0, hi = on ? seen_hi(p, s, token) : 0;  // keys that the row sees
        int full_lo = 0, full_hi = INT32_MAX;  // keys that all of the wave's rows see
        const int row0 = w.tile * kRows + wave * 32, row1 = min(row0 + 32, rows) - 1;
        if (row1 >= row0) full_lo = seen_lo(p, s, token_of(p, row1)), full_hi = seen_hi(p, s, token_of(p, row0));

        vf16 o[kDt];
        float m = kNone, sum = 0.f, high = kNone;  // m: reference in units of log2, lowered by kLift
#pragma unroll
        for (int j = 0; j < kDt; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) o[j][k] = 0.f;

        const auto store_next = [&](int buf, int key0) {
            const bool nan = store_share<T, D>(next, lds, buf * W::kTile, k_nan[buf], v_nan[buf], s.len - key0);
            if (lane == 0) reinterpret_cast<uint8_t*>(&flag[buf])[wave] = (nan ? 1 : 0) | (next.on ? 0 : 2);
        };
        __syncthreads();  // the last item's tiles have been read
        store_next(0, (u0 + a) * kKeys);
        if (a + 1 < z) load_next(a + 1);
        __syncthreads();

        for (int u = a; u < z; ++u) {
            const int buf = (u - a) & 1;
            const uint8_t* const kt = lds + buf * W::kTile;
            const int key0 = (u0 + u) * kKeys;
            const uint32_t seen_by = uniform(static_cast<int>(flag[buf]));
            const bool edge = key0 < full_lo || key0 + kKeys > full_hi || (seen_by & 0x02020202u) != 0;
            const bool nans = (seen_by & 0x01010101u) != 0;

            // K's fragments: number f is terms 16 (f % (D/16)) of half f / (D/16) of the keys
            constexpr int kFrags = 2 * D / 16;
            const uint8_t* const kn = kt + k_row * W::kKRow + 16 * h;
            vf16 sc[2];
            vb8 kf[2][4];
            const auto read_k = [&](int f0) {
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f)
                    kf[f / 4 & 1][f & 3] = *reinterpret_cast<const vb8*>(kn + f / (D / 16) * 32 * W::kKRow + f % (D / 16) * 32);
            };
            read_k(0);
            // products go before the other waves' probabilities: 2% of the 2925 queries' time
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int f0 = 0; f0 < kFrags; f0 += 4) {
                if (f0 + 4 < kFrags) read_k(f0 + 4);
                stay<W::kAhead>();
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f)
#pragma unroll
                    for (int k = kParts - 1; k >= 0; --k) {  // the smallest parts first
                        vf16& x = sc[f / (D / 16)];
                        if (f % (D / 16) == 0 && k == kParts - 1)
#pragma unroll
                            for (int r = 0; r < 16; ++r) x[r] = 0.f;
                        x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[f / 4 & 1][f & 3], q[k][f % (D / 16)], x, 0, 0, 0);
                    }
                stay<W::kAhead>();
            }
            __builtin_amdgcn_s_setprio(0);
            // score r is of key mine0 + 16 * (r / 8) + r % 8, r in [0, 32)
            const int mine0 = key0 + 8 * h;
            if (nans) {
                // a NaN reaches the rows that see its key, and only those
                uint32_t k_bad = 0, v_bad[kDt] = {};
#pragma unroll 1
                for (int r = 0; r < 32; ++r)
                    if (seen_by >> (8 * (r / 8)) & 1u) {
                        const uint8_t* const y = k_nan[buf] + 4 * (8 * h + 16 * (r / 8) + r % 8);
                        k_bad |= static_cast<uint32_t>((y[0] | y[1] | y[2] | y[3]) != 0) << r;
                    }
#pragma unroll 1
                for (int t = 0; t < kKeys; ++t)
                    if (seen_by >> (8 * (t / 16)) & 1u) {
#pragma unroll
                        for (int j = 0; j < kDt; ++j)
                            v_bad[j] |= key0 + t >= lo && key0 + t < hi ? v_nan[buf][t * kDt + j] : 0u;
                    }
#pragma unroll
                for (int r = 0; r < 32; ++r)
                    if (k_bad >> r & 1u) sc[r / 16][r % 16] = __builtin_nanf("");
#pragma unroll
                for (int j = 0; j < kDt; ++j)
                    if (v_bad[j])
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[j][k] = __builtin_nanf("");
            }
            if (edge) {
#pragma unroll
                for (int r = 0; r < 32; ++r) {
                    const int key = mine0 + 16 * (r / 8) + r % 8;
                    if ((seen_by >> (8 * (r / 8)) & 2u) || key < lo || key >= hi) sc[r / 16][r % 16] = kNone;
                }
            }
            float top = kNone;
#pragma unroll
            for (int r = 0; r < 32; ++r) top = fmaxf(top, sc[r / 16][r % 16]);
            top *= p.scale_log2;
            uint64_t low = 0;  // rows whose two lanes lie far below, in the first 32 bits
            if constexpr (Prob<T>::kFalls) {
                low = __ballot(top < m - kDrop);
                low &= low >> 32;
            }
            if (__any(top > m + (kSlack + kLift)) || low) {
                const float r = next_ref<T>(fmaxf(top, __shfl_xor(top, 32, 64)), m, &high);
                const float f = m == r ? 1.f : __builtin_amdgcn_exp2f(m - r);
                m = r;
                sum *= f;
#pragma unroll
                for (int j = 0; j < kDt; ++j) o[j] *= f;
            }
            const float ref = m == kNone ? 0.f : -m;
            using Frag = typename Prob<T>::Frag;
            Frag pf[2][2][kP];
            // The tile's sum, first by itself: one by one, small probabilities would be lost beside a large
            // sum (2e-4 of it after 16385 keys).
            float more = 0.f;
            // probabilities r0 .. r0 + many - 1 of half g
            const auto exps = [&](int g, int r0, int many) {
#pragma unroll
                for (int r = r0; r < r0 + many; ++r) {
                    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[g][r], p.scale_log2, ref));
                    more += e;
                    Prob<T>::set(pf[g][r / 8], r % 8, e);
                }
            };
            // V's fragments: number f is of half f / (2 kDt), terms 16 (f % 2), channels 32 (f / 2 % kDt)
            constexpr int kVFrags = 4 * kDt;
            const uint32_t vn = buf * W::kTile + kKeys * W::kKRow + n / 2 * 256 + 16 * v_lane;
            Frag vf[2][4];
            const auto read_v = [&](int f0) {
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f) {
                    const int g = f / (2 * kDt), j = f / 2 % kDt, t = f & 1;
                    vf[f / 4 & 1][f & 3] =
                        *reinterpret_cast<const Frag*>(lds + ((vn ^ 16 * (4 * g + 2 * t ^ W::v_turn(16 * j))) + j * 4096));
                }
            };
            read_v(0);
            stay<W::kAhead>();
            exps(0, 0, 16);
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int f0 = 0; f0 < kVFrags; f0 += 4) {
                if (f0 + 4 < kVFrags) read_v(f0 + 4);
                stay<W::kAhead>();
#pragma unroll
                for (int f = f0; f < f0 + 4; ++f)
#pragma unroll
                    for (int k = kP - 1; k >= 0; --k) {
                        vf16& x = o[f / 2 % kDt];
                        x = Prob<T>::mul32(vf[f / 4 & 1][f & 3], pf[f / (2 * kDt)][f & 1][k], x);
                    }
                // the other half's probabilities beside this half's products
                if (f0 < kVFrags / 2) exps(1, f0 * 32 / kVFrags, 4 * 32 / kVFrags);
                stay<W::kAhead>();
            }
            __builtin_amdgcn_s_setprio(0);
            sum += more;
            if (u + 1 < z) {
                store_next(buf ^ 1, key0 + kKeys);
                if (u + 2 < z) load_next(u + 2);
                __syncthreads();
            }
        }

        if (Prob<T>::kFalls && __any(m != high)) {  // lse is more exact from the highest reference
            const float f = m == high ? 1.f : __builtin_amdgcn_exp2f(m - high);
            m = high;
            sum *= f;
#pragma unroll
            for (int j = 0; j < kDt; ++j) o[j] *= f;
        }
        const bool whole = a == 0 && z == count;
        const float l = sum + __shfl_xor(sum, 32, 64);
        if (on) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T* const dst = row_ptr<T>(p.out, s.q0 + token, q_head);
            float* const y = p.part + (2 * int64_t(me) + (a == 0)) * part_floats<D>(kRows) + int64_t(row - w.tile * kRows) * (D + 2);
            // registers 4 k .. are channels 8 k + 4 h ..
#pragma unroll
            for (int j = 0; j < kDt; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = 32 * j + 8 * k + 4 * h;
                    const vf4 x{o[j][4 * k], o[j][4 * k + 1], o[j][4 * k + 2], o[j][4 * k + 3]};
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
                    *reinterpret_cast<float2*>(y + D) = float2{m, l};
                else if (p.lse)
                    p.lse[int64_t(s.q0 + token) * p.q_heads + q_head] = lse_of(m, l);
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
