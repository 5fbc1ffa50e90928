// cf_kv8_attn.hip - attention over the 8-bit K/V cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i k_j - m_i),  lse_i = m_i + log sum_j p_ij
// over the keys j that row i may see, in one pass over the keys with a running reference m and sum.
//
// Precision.  What the cache holds is exact in bf16, and in fp16 too (the scales' exponents see to that), and so are
// bf16 queries; fp32 queries are split into three bf16 parts that add up to them, and so are their probabilities.
// With bf16 queries probabilities are rounded to fp16 where rows are few (half a step is 2^-11 of each) and to
// bf16 where they are many (2^-8).  Sums, references and O are fp32, and the sum is of unrounded probabilities.
//
// Work is cut as in cf_attn_plan.h.  The kernel for few rows (at most 32: decoding) is bound by the cache's bytes, the
// one for many rows (cf_attn_tile.h) by the matrix and vector units.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf_attn_tile.h"
#include "cf_kv8_few.h"

namespace cf {
namespace {

// Tiles of 64 keys of a cache, decoded: K as [key][D], V as [channel][64 keys] in runs of eight keys, which is how the
// cache holds them.
template <typename T, int D>
struct Kv8Source {
    using Type = T;
    using Args = Attn8Args;
    static constexpr int kDim = D;
    static constexpr int kQueryParts = sizeof(T) == 4 ? 3 : 1, kKeyParts = 1;
    static constexpr int kKeys = 64;
    static constexpr int kPad = 5;
    static constexpr int kResident = 1;
    static constexpr int kPlane = kKeys * D * 2;
    static constexpr int kBytes = 2 * kPlane;

    int b, head, wave, page;  // page: of the wave's 16 keys of the tile to load next
    uint32_t k_lane, v_lane;
    uint32_t k[D / 16], v[D / 16];
    uint32_t ks, vs;
    bool on;

    static __device__ __forceinline__ __bf16 part(float* rest) { return take_bf16(rest); }

    // a channel's eight runs of eight keys lie turned: the 16 channels that a product's lanes read at once, and the
    // four or two channels apart that are written at once, are on different banks
    static __device__ constexpr uint32_t run(int c, int r) { return c * (2 * kKeys) + ((r ^ ((c >> 1 & 7) ^ (c >> 4 & 1))) << 4); }

    __device__ __forceinline__ void begin(const Attn8Args&) {
        const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
        wave = uniform(static_cast<int>(threadIdx.x) >> 6);
        k_lane = KeyRows<D>::chunk(KeyRows<D>::key_of(n), h);
        v_lane = run(n, h);
    }
    __device__ __forceinline__ void item(const Attn8Args&, const Seq&, int seq, int kv_head) { b = seq, head = kv_head; }
    __device__ __forceinline__ void load(const Attn8Args& p, const Seq& s, int key0) {
        const int lane = threadIdx.x & 63, key = key0 + 16 * wave;
        // keys behind the last are read from its page (and masked later): always inside the cache
        const int64_t at = int64_t(b) * p.width + (min(key, max(s.len - 1, 0)) >> p.cache.shift);
        const int page = p.table ? scalar_load(p.table + at) : static_cast<int>(at);  // at < pages < 2^31 without a table
        on = page_on(p, s, page);
        const uint8_t* const base = p.cache.at(on ? page : 0, head);
        const Kv8Block blk{p.cache.block.page, D};
        const int in = key & (blk.page - 1);
        const uint8_t* const kc = base + blk.k_code(in + lane / 4) + (lane & 3) * (D / 4);
        const uint8_t* const vc = base + blk.v_code(in + 8 * (lane >> 5), (lane & 31) * (D / 32));
#pragma unroll
        for (int i = 0; i < D / 16; i += 4) {
            const vu4 x = *reinterpret_cast<const vu4*>(kc + 4 * i), y = *reinterpret_cast<const vu4*>(vc + 4 * i);
            k[i] = x.x, k[i + 1] = x.y, k[i + 2] = x.z, k[i + 3] = x.w;
            v[i] = y.x, v[i + 1] = y.y, v[i + 2] = y.z, v[i + 3] = y.w;
        }
        ks = base[blk.k_scale(in)], vs = base[blk.v_scale(in)];
    }
    __device__ __forceinline__ void store(const Attn8Args&, const Seq& s, uint8_t* lds, uint8_t* flag, int buf, int key0) {
        const int lane = threadIdx.x & 63, oct = 8 * (lane >> 5), key = 16 * wave + lane / 4;
        if (lane == 0) flag[wave] = on ? 0 : 1;
        if (!on || s.len - key0 < 16 * wave + 16) {
            // V behind the sequence's last key is whatever an earlier owner of the page left
            const int valid = on ? min(max(s.len - key0 - 16 * wave - oct, 0), 8) : 0;
            const uint64_t keep = valid == 8 ? ~uint64_t(0) : (uint64_t(1) << (8 * valid)) - 1;
            if (valid == 0) vs = 127u;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) v[i] &= static_cast<uint32_t>(i & 1 ? keep >> 32 : keep);
        }
        uint8_t* const at = lds + buf * kBytes;
        const float kf = scale_of(ks), vf = scale_of(vs);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            *reinterpret_cast<vb8*>(at + KeyRows<D>::chunk(key, (lane & 3) * (D / 32) + i)) = bf16_codes(k[2 * i], k[2 * i + 1], kf);
            *reinterpret_cast<vb8*>(at + kPlane + run((lane & 31) * (D / 32) + i, 2 * wave + (lane >> 5))) =
                bf16_codes(v[2 * i], v[2 * i + 1], vf);
        }
    }
    static __device__ __forceinline__ uint32_t none(const uint8_t* flag, int half) {
        return uniform(static_cast<int>(flag[2 * half] | flag[2 * half + 1] << 1));
    }
    __device__ __forceinline__ vb8 k_frag(const uint8_t* lds, int buf, int half, int, int c) const {
        return *reinterpret_cast<const vb8*>(lds + buf * kBytes + (k_lane ^ 32 * c) + half * 64 * D);
    }
    __device__ __forceinline__ vb8 v_frag(const uint8_t* lds, int buf, int half, int, int t, int j) const {
        // run 4 half + 2 t + h of channel 32 j + n: 32 j turns as 0 does
        return *reinterpret_cast<const vb8*>(lds + buf * kBytes + kPlane + (v_lane ^ 16 * (4 * half + 2 * t)) + j * 64 * kKeys);
    }
    __device__ __forceinline__ bool v_bad(const uint8_t* lds, int buf, int half, int t, int c) const {
        const uint16_t x = *reinterpret_cast<const uint16_t*>(lds + buf * kBytes + kPlane + run(c, 4 * half + t / 8) + t % 8 * 2);
        return (x & 0x7f80u) == 0x7f80u;
    }
};

// Calls f with the kernel's shape and the kernel for a call whose longest sequence has max_rows rows.
template <typename T, int D, typename F>
auto with_kernel(int64_t max_rows, F f) {
    if (max_rows <= 16) return f(Few8<T, D, 1>(), few8_kernel<T, D, 1>);
    if (max_rows <= 32) return f(Few8<T, D, 2>(), few8_kernel<T, D, 2>);
    using K = Tile<Kv8Source<T, D>, 1>;
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
        using S = decltype(shape);
        p.groups = plan_of<S>(c.cache.block.dim).groups;
        p.joins = static_cast<int32_t*>(workspace);
        p.part = reinterpret_cast<float*>(p.joins + kJoin * p.groups);
        kernel<<<p.groups, kThreads, 0, stream>>>(p);
        if (hipError_t e = hipGetLastError()) return e;
        return launch_join<S>(p, max_rows, stream);
    });
}

}  // namespace cf
