// cf_kv8_attn.hip - attention over the 8-bit K/V cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i k_j - m_i),  lse_i = m_i + log sum_j p_ij
// over the keys j that row i may see, in one pass over the keys with a running reference m and sum.
//
// Precision.  What the cache holds is exact in bf16, and in fp16 too (the scales' exponents see to that), and so are
// bf16 queries; fp32 queries are split into three bf16 parts that add up to them, and so are their probabilities.
// With bf16 queries probabilities are rounded to fp16 where rows are few (half a step is 2^-11 of each) and to
// bf16 where they are many (2^-8).  bf16 has fp32's range: each keeps its 2^-8 however far below its tile's others it
// lies, where fp16's run out 2^-21 below (beside a key that outweighs the other 63 by e^22 these would be subnormals, by
// e^30 nothing), and no reference has to fall.  Sums, references and O are fp32, and the sum is of unrounded probabilities.
//
// Work is cut as in cf_attn_plan.h.  The kernel for few rows (at most 32: decoding) is bound by the cache's bytes, the
// one for many rows (cf_attn_tile.h) by the matrix and vector units.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf_attn_join.h"
#include "cf_attn_tile.h"
#include "cf_kv8_few.h"

namespace cf {
namespace {

// Tiles of 64 keys of a cache, decoded: K as [key][D], V as [channel][64 keys] in runs of eight keys, which is how the
// cache holds them.  A wave takes 16 or 8 keys of a tile, all of one page and scale.
template <typename T, int D, int WAVES>
struct Kv8Source {
    using Type = T;
    using Args = Attn8Args;
    static constexpr int kDim = D, kWaves = WAVES;
    static constexpr int kQueryParts = sizeof(T) == 4 ? 3 : 1, kKeyParts = 1;
    static constexpr int kKeys = 64;
    static constexpr int kPad = 6, kLeast = 6;  // what an item costs besides its units, and the shortest run (as for rows)
    // workgroups of a compute unit: 1024 fp32 rows of D = 64 over 4608 keys take 102 us with two, 135 with one
    static constexpr int kResident = D == 64 && WAVES == 4 ? 2 : 1;
    static constexpr int kPlane = kKeys * D * 2;
    static constexpr int kBytes = 2 * kPlane;
    // a thread's share: codes of a key, and of eight keys of so many channels; in pieces of 16 or 8 bytes
    static constexpr int kShare = D / WAVES, kChannels = kShare / 8, kPiece = kShare < 16 ? kShare : 16, kPieces = 2 * kShare / kPiece;
    static constexpr int kGroup = 64 * WAVES, kMine = kKeys / WAVES, kLanes = 8 * WAVES;  // keys of a wave; lanes of eight keys
    static constexpr int kBad = kGroup * kChannels;
    static constexpr bool kSums = false;

    int b, head, wave;
    int pages;  // of the four runs of 16 keys of the tile to load next, in lanes 0 .. 3
    uint32_t k_lane, v_lane, k_store, v_store[kChannels];
    const uint8_t *k_at, *v_at, *k_scale, *v_scale;
    vu2 r[kPieces][kPiece / 8];
    uint32_t ks, vs;
    uint64_t keep;  // of V's eight keys: the sequence's
    bool on;

    static __device__ __forceinline__ __bf16 part(float* rest) { return take_bf16(rest); }

    // a channel's eight runs of eight keys lie turned: the 16 channels that a product's lanes read at once, and the
    // channels that are written at once, are on different banks
    static __device__ constexpr uint32_t run(int c, int r) { return c * (2 * kKeys) + ((r ^ ((c >> 1 & 7) ^ (c >> 4 & 1))) << 4); }

    __device__ __forceinline__ void begin(const Attn8Args&) {
        const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
        wave = uniform(static_cast<int>(threadIdx.x) >> 6);
        k_lane = KeyRows<D>::chunk(KeyRows<D>::key_of(n), h);
        v_lane = run(n, h);
        k_store = KeyRows<D>::chunk(kMine * wave + lane / WAVES, lane % WAVES * kChannels);
#pragma unroll
        for (int i = 0; i < kChannels; ++i) v_store[i] = run(lane % kLanes * kChannels + i, kMine / 8 * wave + lane / kLanes);
    }
    // Lanes ask for a tile's four pages, and a wave takes its own: a scalar load, which shares its counter with shared
    // memory, would be waited for at the next barrier.  Keys behind the last are read from its page (and masked later):
    // always inside the cache.
    __device__ __forceinline__ int page_at(const Attn8Args& p, const Seq& s, int key0) const {
        const int key = key0 + 16 * static_cast<int>(threadIdx.x & 3);
        const int64_t at = int64_t(b) * p.width + (min(key, max(s.len - 1, 0)) >> p.cache.shift);
        return p.table ? p.table[at] : static_cast<int>(at);  // at < pages < 2^31 without a table
    }
    __device__ __forceinline__ void item(const Attn8Args& p, const Seq& s, int seq, int kv_head, int key0) {
        b = seq, head = kv_head;
        pages = page_at(p, s, key0);
    }
    __device__ __forceinline__ void next_tile(const Attn8Args& p, const Seq& s, int key0, bool) {
        const int lane = threadIdx.x & 63, key = key0 + kMine * wave;
        const int page = __builtin_amdgcn_readlane(pages, kMine * wave / 16);
        pages = page_at(p, s, key0 + kKeys);
        on = page_on(p, s, page);
        const uint8_t* const base = p.cache.at(on ? page : 0, head);
        const Kv8Block blk{p.cache.block.page, D};
        const int in = key & (blk.page - 1);
        k_at = base + blk.k_code(in + lane / WAVES) + lane % WAVES * kShare;
        v_at = base + blk.v_code(in + 8 * (lane / kLanes), lane % kLanes * kChannels);
        k_scale = base + blk.k_scale(in), v_scale = base + blk.v_scale(in);
        // V behind the sequence's last key is whatever an earlier owner of the page left
        const int valid = on ? min(max(s.len - key - 8 * (lane / kLanes), 0), 8) : 0;
        keep = valid == 8 ? ~uint64_t(0) : (uint64_t(1) << (8 * valid)) - 1;
    }
    __device__ __forceinline__ void load(int i) {
        typedef uint32_t Piece __attribute__((ext_vector_type(kPiece / 4)));
        const Piece x = *reinterpret_cast<const Piece*>(i < kPieces / 2 ? k_at + kPiece * i : v_at + kPiece * (i - kPieces / 2));
#pragma unroll
        for (int j = 0; j < kPiece / 8; ++j) r[i][j] = vu2{x[2 * j], x[2 * j + 1]};
        if (i == 0) ks = *k_scale, vs = *v_scale;
    }
    __device__ __forceinline__ void store(uint8_t* lds, int buf, int i) {
        uint8_t* const at = lds + buf * kBytes;
        const bool is_k = i < kPieces / 2;
        const float f = is_k ? scale_of(ks) : keep ? scale_of(vs) : 1.f;
        const uint32_t lo = static_cast<uint32_t>(keep), hi = static_cast<uint32_t>(keep >> 32);
#pragma unroll
        for (int j = 0; j < kPiece / 8; ++j) {
            const int c = (is_k ? i : i - kPieces / 2) * (kPiece / 8) + j;
            if (is_k)  // chunks of a key are turned by exclusive or
                *reinterpret_cast<vb8*>(at + (k_store ^ 16 * c)) = bf16_codes(r[i][j].x, r[i][j].y, f);
            else
                *reinterpret_cast<vb8*>(at + kPlane + v_store[c]) = bf16_codes(r[i][j].x & lo, r[i][j].y & hi, f);
        }
    }
    // As for rows (cf_attn.hip): a byte for eight keys of a channel.
    __device__ __forceinline__ void stored(const Attn8Args&, const Seq&, uint8_t* flag, uint8_t* bads, uint8_t* lds, int buf, bool part) {
        uint32_t any = 0;
        if (part) {
            const uint32_t lo = static_cast<uint32_t>(keep), hi = static_cast<uint32_t>(keep >> 32);
#pragma unroll
            for (int i = kPieces / 2; i < kPieces; ++i)
#pragma unroll
                for (int j = 0; j < kPiece / 8; ++j) any |= nan_codes(r[i][j].x & lo) | nan_codes(r[i][j].y & hi);
            any = __any(any != 0) ? 2 : 0;
            if (any)
#pragma unroll
                for (int i = kPieces / 2; i < kPieces; ++i) {
#pragma unroll
                    for (int j = 0; j < kPiece / 8; ++j) {
                        const uint32_t x = nan_codes(r[i][j].x & lo), y = nan_codes(r[i][j].y & hi);
                        bads[((i - kPieces / 2) * (kPiece / 8) + j) * kGroup + threadIdx.x] = static_cast<uint8_t>(four_bits(x) | four_bits(y) << 4);
                        r[i][j].x &= ~full_bytes(x), r[i][j].y &= ~full_bytes(y);
                    }
                    store(lds, buf, i);
                }
        }
        if ((threadIdx.x & 63) == 0) flag[wave] = static_cast<uint8_t>(any | (on ? 0 : 1));
    }
    // 16 keys without a page, a bit each
    static __device__ __forceinline__ uint32_t none(FlagWord flag) {
        uint32_t x = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) x |= static_cast<uint32_t>(flag >> (8 * (16 * i / kMine)) & 1) << i;
        return x;
    }
    static __device__ __forceinline__ bool found(FlagWord flag) { return (flag & 0x0202020202020202u) != 0; }
    // whether a channel of a key of a tile is NaN
    static __device__ __forceinline__ bool bad(FlagWord flag, const uint8_t* bads, int key, int c) {
        const int of = key / kMine, lane = key % kMine / 8 * kLanes + c / kChannels;
        return (flag >> (8 * of) & 2u) && (bads[c % kChannels * kGroup + of * 64 + lane] >> (key & 7) & 1u);
    }
    __device__ __forceinline__ vb8 k_frag(const uint8_t* lds, int buf, int half, int, int c) const {
        return *reinterpret_cast<const vb8*>(lds + buf * kBytes + (k_lane ^ 32 * c) + half * 64 * D);
    }
    __device__ __forceinline__ vb8 v_frag(const uint8_t* lds, int buf, int half, int, int t, int j) const {
        // run 4 half + 2 t + h of channel 32 j + n: 32 j turns as 0 does
        return *reinterpret_cast<const vb8*>(lds + buf * kBytes + kPlane + (v_lane ^ 16 * (4 * half + 2 * t)) + j * 64 * kKeys);
    }
};

// Calls f with the kernel's shape and the kernel for a call whose longest sequence has max_rows rows.
template <typename T, int D, typename F>
auto with_kernel(int64_t max_rows, F f) {
    if (max_rows <= 16) return f(Few8<T, D, 1>(), few8_kernel<T, D, 1>);
    if (max_rows <= 32) return f(Few8<T, D, 2>(), few8_kernel<T, D, 2>);
    using K = Tile<Kv8Source<T, D, sizeof(T) == 2 ? 8 : 4>>;
    return f(K(), tile_kernel<K>);
}

template <typename F>
auto with_kernel(int a_dtype, int head_dim, int64_t max_rows, F f) {
    if (a_dtype == CF_BF16)
        return head_dim == 64 ? with_kernel<__bf16, 64>(max_rows, f) : with_kernel<__bf16, 128>(max_rows, f);
    return head_dim == 64 ? with_kernel<float, 64>(max_rows, f) : with_kernel<float, 128>(max_rows, f);
}

}  // namespace

// The largest of what the kernels for up to so many rows use, so that a workspace serves every call with fewer rows too.
size_t kv8_attention_workspace(int a_dtype, int head_dim, int64_t max_rows) {
    size_t most = 0;
    for (const int64_t rows : {1, 17, 33}) {  // the fewest of each kernel
        if (rows > max_rows) break;
        const size_t n = with_kernel(a_dtype, head_dim, rows,
                                     [&](auto shape, auto) { return plan_of<decltype(shape)>(head_dim).bytes(); });
        most = n > most ? n : most;
    }
    return most;
}

hipError_t launch_kv8_attention(int a_dtype, const Kv8Attention& c, void* workspace, hipStream_t stream) {
    Attn8Args p{};
    p.q = c.q, p.out = c.out, p.cache = c.cache, p.table = c.table, p.width = c.table_width;
    p.kv_lens = c.kv_lens, p.q_starts = c.q_starts, p.total_q = static_cast<int>(c.total_q);
    p.q_each = c.q_starts ? 0 : static_cast<int>(c.total_q / c.batch);
    p.batch = c.batch, p.q_heads = c.q_heads, p.kv_heads = c.cache.heads, p.share = c.q_heads / c.cache.heads;
    p.causal = c.causal, p.window = c.window;
    p.scale_log2 = c.scale * 1.44269504088896341f;
    p.lse = c.lse;
    const int64_t max_rows = c.max_q * p.share;
    return with_kernel(a_dtype, c.cache.block.dim, max_rows, [&](auto shape, auto kernel) {
        return launch_attn<decltype(shape)>(p, kernel, max_rows, workspace, stream);
    });
}

}  // namespace cf
