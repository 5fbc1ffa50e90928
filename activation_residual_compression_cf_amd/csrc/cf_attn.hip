// cf_attn.hip - attention over whole prompts: keys and values are rows of heads.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i k_j - m_i),  lse_i = m_i + log sum_j p_ij
// over the keys j that row i may see, in one pass over the keys with a running reference m and sum.  A row is one
// (query token, query head); the rows of the query heads that share a K/V head are worked on together.
//
// Precision.  bf16: queries, keys and values enter the products exactly, probabilities rounded to bf16 (half a step is
// 2^-8 of each; its range is fp32's, so nothing falls out below).  fp32: queries, keys, probabilities and values are
// split into three bf16 parts that add up to them, and of their products those six are taken that can reach 2^-24 of
// the whole.  Sums, references and O are fp32, and the sum is of unrounded probabilities.
//
// Work is cut as for the caches (cf_attn_plan.h): every workgroup takes an equal run of (256 or 128 rows x 64 or 32
// keys) units, whatever items they are of.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf_attn_join.h"
#include "cf_attn_tile.h"

namespace cf {
namespace {

struct RowsArgs : AttnRows {
    RowSet k, v;
    const int32_t* k_starts;  // or null: k_each keys of each sequence
    int total_k, k_each;
};

__device__ __forceinline__ Seq cut_rows(const RowsArgs& p, int q0, int q1, int k0, int k1) {
    Seq s;
    cut_queries(p, &s, q0, q1);
    s.k0 = min(max(k0, 0), p.total_k);
    s.len = min(max(k1, s.k0), p.total_k) - s.k0;
    return s;
}

// b differs from lane to lane.
__device__ __forceinline__ Seq seq_of(const RowsArgs& p, int b) {
    const int q0 = p.q_starts ? p.q_starts[b] : b * p.q_each, q1 = p.q_starts ? p.q_starts[b + 1] : (b + 1) * p.q_each;
    const int k0 = p.k_starts ? p.k_starts[b] : b * p.k_each, k1 = p.k_starts ? p.k_starts[b + 1] : (b + 1) * p.k_each;
    return cut_rows(p, q0, q1, k0, k1);
}

// b is the same in every lane.
__device__ __forceinline__ Seq seq_at(const RowsArgs& p, int b) {
    const int q0 = p.q_starts ? scalar_load(p.q_starts + b) : b * p.q_each;
    const int q1 = p.q_starts ? scalar_load(p.q_starts + b + 1) : (b + 1) * p.q_each;
    const int k0 = p.k_starts ? scalar_load(p.k_starts + b) : b * p.k_each;
    const int k1 = p.k_starts ? scalar_load(p.k_starts + b + 1) : (b + 1) * p.k_each;
    return cut_rows(p, q0, q1, k0, k1);
}

// Tiles of rows: K and V both [key][D] bf16, fp32 as three planes of each.  V is read across its rows by the
// transposing reads of shared memory.
template <typename T, int D, int WAVES>
struct RowSource {
    static constexpr int kWaves = WAVES;
    using Type = T;
    using Args = RowsArgs;
    static constexpr int kDim = D;
    static constexpr int kQueryParts = sizeof(T) == 4 ? 3 : 1, kKeyParts = kQueryParts;
    static constexpr int kKeys = sizeof(T) == 4 ? 32 : 64;
    // What an item costs besides its units, and the shortest run (4 and 4: long causal prompts 3% slower, 3 and 3: 5%; short
    // ones differ by 2% either way).
    static constexpr int kPad = 6, kLeast = 6;
    // Workgroups of a compute unit, by their registers and shared memory.  64 tokens over 4000 keys each, of D = 64: 98 us
    // with two, 150 with one, 110 with three, which spill; 4096 fp32 rows over 4608 keys: 604 with two, 717 with one.
    static constexpr int kResident = D == 64 && WAVES == 4 ? 2 : 1;
    static constexpr int kPlane = kKeys * D * 2;
    static constexpr int kBytes = 2 * kKeyParts * kPlane;
    // a thread's loads: 16 bytes of kPasses rows, kStep apart
    static constexpr int kChunks = D * sizeof(T) / 16, kStep = 64 * WAVES / kChunks, kPasses = kKeys / kStep;

    static constexpr int kGroup = 64 * WAVES, kBad = kGroup * kPasses;
    static constexpr bool kSums = true;
    static constexpr int kPieces = 2 * kPasses;  // of a thread's loads and stores of a tile: K's, and V's

    const char* k;  // the sequence's first key
    const char* v;
    uint32_t k_stride, v_stride, k_off, v_off;
    uint32_t k_lane, v_lane[2], k_store, v_store;
    __amdgpu_buffer_rsrc_t k_tile, v_tile;
    vu4 r[kPieces];

    // rounded parts: what the products leave out is then at most 2^-24 of their factors
    static __device__ __forceinline__ __bf16 part(float* rest) { return round_bf16(rest); }

    // V's channels lie in runs of 16, turned by the row: a transposing read takes four rows of two runs with 32 lanes, which
    // are then all of the banks (turned so that two runs met, LDS was busy a third longer).
    static __device__ constexpr uint32_t run(int row, int r) {
        return row * (2 * D) + ((r ^ (D == 128 ? 2 * (row & 3) : row & 3)) << 5);
    }

    __device__ __forceinline__ void begin(const RowsArgs& p) {
        const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
        k_stride = static_cast<uint32_t>(p.k.token_stride * sizeof(T)), v_stride = static_cast<uint32_t>(p.v.token_stride * sizeof(T));
        const uint32_t row = threadIdx.x / kChunks, c = threadIdx.x % kChunks;
        k_off = row * k_stride + 16 * c, v_off = row * v_stride + 16 * c;
        if constexpr (sizeof(T) == 2)
            k_store = KeyRows<D>::chunk(row, c), v_store = run(row, c >> 1) + (c & 1) * 16;
        else
            k_store = KeyRows<D>::chunk(row, c >> 1) + (c & 1) * 8, v_store = run(row, c >> 2) + (c & 3) * 8;
        k_lane = KeyRows<D>::chunk(KeyRows<D>::key_of(n), h);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v_lane[i] = run(8 * h + 4 * i + ((lane & 15) >> 2), lane >> 4 & 1) + (lane & 3) * 8;
    }
    __device__ __forceinline__ void item(const RowsArgs& p, const Seq& s, int, int head, int) {
        k = reinterpret_cast<const char*>(row_ptr<T>(p.k, s.k0, head));
        v = reinterpret_cast<const char*>(row_ptr<T>(p.v, s.k0, head));
    }
    // Loads are cut off behind the sequence's last row, by the hardware: what lies there reads as zeros.
    __device__ __forceinline__ void next_tile(const RowsArgs&, const Seq& s, int key0, bool on) {
        const int rows = on ? min(s.len - key0, kKeys) : 0;
        const auto tile = [&](const char* first, uint32_t stride) {
            const int64_t at = reinterpret_cast<int64_t>(first) + int64_t(key0) * stride;
            return stream_rsrc(reinterpret_cast<void*>(uniform(at)), rows > 0 ? (rows - 1) * stride + D * sizeof(T) : 0u);
        };
        k_tile = tile(k, k_stride), v_tile = tile(v, v_stride);
    }
    __device__ __forceinline__ void load(int i) {
        r[i] = i < kPasses ? __builtin_amdgcn_raw_buffer_load_b128(k_tile, k_off + i * (kStep * k_stride), 0, 0)
                           : __builtin_amdgcn_raw_buffer_load_b128(v_tile, v_off + (i - kPasses) * (kStep * v_stride), 0, 0);
    }
    __device__ __forceinline__ void store(uint8_t* lds, int buf, int i) {
        const bool is_k = i < kPasses;
        const int further = (is_k ? i : i - kPasses) * kStep;
        // rows 16 further turn as these do, and rows 8 further in one bit
        const uint32_t turn = is_k ? (D == 128 && further & 8 ? 128u : 0u) : 0u;
        static_assert(kStep % 16 == 0 || (D == 128 && kStep == 8), "");
        uint8_t* const at = lds + buf * kBytes + (is_k ? k_store ^ turn : v_store + kKeyParts * kPlane) + further * (2 * D);
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<vu4*>(at) = r[i];
        } else {
            vf4 x = __builtin_bit_cast(vf4, r[i]);
            typedef __bf16 vb4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int k = 0; k < kKeyParts; ++k) {
                vb4 a;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f = x[j];
                    a[j] = part(&f);
                    x[j] = f;
                }
                *reinterpret_cast<vb4*>(at + k * kPlane) = a;
            }
        }
    }
    // Where some of the item's rows do not see all of the tile (part), a probability of zero times an infinity or NaN of V
    // would be NaN: zeros take their place, and bits, a byte for a thread's 16 bytes, say where.
    __device__ __forceinline__ void stored(const RowsArgs&, const Seq&, uint8_t* flag, uint8_t* bads, uint8_t* lds, int buf, bool part) {
        uint32_t any = 0;
        if (part) {
            const auto bits = [&](int i) {
                uint32_t b = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = r[kPasses + i][j];
                    b |= sizeof(T) == 4 ? static_cast<uint32_t>((w & 0x7f800000u) == 0x7f800000u) << j
                                        : static_cast<uint32_t>((w & 0x7f80u) == 0x7f80u) << (2 * j) |
                                              static_cast<uint32_t>((w & 0x7f800000u) == 0x7f800000u) << (2 * j + 1);
                }
                return b;
            };
#pragma unroll
            for (int i = 0; i < kPasses; ++i) any |= bits(i);
            if (__any(any != 0)) {
                any = 1;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const uint32_t b = bits(i);
                    bads[i * kGroup + threadIdx.x] = static_cast<uint8_t>(b);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (sizeof(T) == 4)
                            r[kPasses + i][j] = b >> j & 1u ? 0u : r[kPasses + i][j];
                        else
                            r[kPasses + i][j] &= (b >> (2 * j) & 1u ? 0u : 0xffffu) | (b >> (2 * j + 1) & 1u ? 0u : 0xffff0000u);
                    }
                    store(lds, buf, kPasses + i);
                }
            }
        }
        if ((threadIdx.x & 63) == 0) flag[threadIdx.x >> 6] = static_cast<uint8_t>(any);
    }
    static __device__ __forceinline__ uint32_t none(FlagWord) { return 0; }
    static __device__ __forceinline__ bool found(FlagWord flag) { return flag != 0; }
    // whether a channel of a key of a tile is infinite or NaN
    static __device__ __forceinline__ bool bad(FlagWord flag, const uint8_t* bads, int key, int c) {
        const int thread = key % kStep * kChunks + c / (16 / int(sizeof(T)));
        return (flag >> (8 * (thread >> 6)) & 1u) && (bads[key / kStep * kGroup + thread] >> (c % (16 / int(sizeof(T)))) & 1u);
    }
    // terms 16 c .. of a product's 32 keys
    __device__ __forceinline__ vb8 k_frag(const uint8_t* lds, int buf, int half, int part, int c) const {
        return *reinterpret_cast<const vb8*>(lds + buf * kBytes + (k_lane ^ 32 * c) + part * kPlane + half * 64 * D);
    }
    // channels 32 j .., keys 16 t ..
    __device__ __forceinline__ vb8 v_frag(const uint8_t* lds, int buf, int half, int part, int t, int j) const {
        typedef short vs4 __attribute__((ext_vector_type(4)));
        vs4 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* const at =
                lds + buf * kBytes + (v_lane[i] ^ 64 * j) + (kKeyParts + part) * kPlane + (32 * half + 16 * t) * 2 * D;
            x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) vs4*)at);
        }
        return __builtin_bit_cast(vb8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// Calls f with the kernel's shape and the kernel for a call whose longest sequence has max_rows rows.
template <typename T, int D, typename F>
auto with_kernel(int64_t max_rows, F f) {
    if constexpr (sizeof(T) == 2) {
        if (max_rows > 128) {
            using K = Tile<RowSource<T, D, 8>>;
            return f(K(), tile_kernel<K>);
        }
    }
    using K = Tile<RowSource<T, D, 4>>;
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
size_t attention_workspace(int a_dtype, int head_dim, int64_t max_rows) {
    size_t most = 0;
    for (const int64_t rows : {1, 129}) {  // the fewest of each kernel
        if (rows > max_rows) break;
        const size_t n = with_kernel(a_dtype, head_dim, rows,
                                     [&](auto shape, auto) { return plan_of<decltype(shape)>(head_dim).bytes(); });
        most = n > most ? n : most;
    }
    return most;
}

hipError_t launch_attention(int a_dtype, const RowsAttention& c, void* workspace, hipStream_t stream) {
    const int share = c.q_heads / c.kv_heads;
    RowsArgs p{};
    p.q = c.q, p.out = c.out, p.k = c.k, p.v = c.v, p.q_starts = c.q_starts, p.k_starts = c.k_starts;
    p.total_q = static_cast<int>(c.total_q), p.total_k = static_cast<int>(c.total_k);
    p.q_each = c.q_starts ? 0 : static_cast<int>(c.total_q / c.batch);
    p.k_each = c.k_starts ? 0 : static_cast<int>(c.total_k / c.batch);
    p.batch = c.batch, p.q_heads = c.q_heads, p.kv_heads = c.kv_heads, p.share = share;
    p.causal = c.causal, p.window = c.window;
    p.scale_log2 = c.scale * 1.44269504088896341f;
    p.lse = c.lse;
    const int64_t max_rows = c.max_q * share;
    return with_kernel(a_dtype, c.head_dim, max_rows, [&](auto shape, auto kernel) {
        return launch_attn<decltype(shape)>(p, kernel, max_rows, workspace, stream);
    });
}

}  // namespace cf
