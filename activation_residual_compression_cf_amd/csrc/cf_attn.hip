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
template <typename T, int D>
struct RowSource {
    using Type = T;
    using Args = RowsArgs;
    static constexpr int kDim = D;
    static constexpr int kQueryParts = sizeof(T) == 4 ? 3 : 1, kKeyParts = kQueryParts;
    static constexpr int kKeys = sizeof(T) == 4 ? 32 : 64;
    static constexpr int kPad = 4;
    static constexpr int kResident = 1;
    static constexpr int kPlane = kKeys * D * 2;
    static constexpr int kBytes = 2 * kKeyParts * kPlane;
    // a thread's loads: 16 bytes of kPasses rows, kStep apart
    static constexpr int kChunks = D * sizeof(T) / 16, kStep = kThreads / kChunks, kPasses = kKeys / kStep;
    static constexpr int kTurn = D == 128 ? 7 : 3;

    const char* k;  // the sequence's first key
    const char* v;
    uint32_t k_stride, v_stride, k_off, v_off;
    uint32_t k_lane, v_lane[2];
    vu4 kr[kPasses], vr[kPasses];

    // rounded parts: what the products leave out is then at most 2^-24 of their factors
    static __device__ __forceinline__ __bf16 part(float* rest) { return round_bf16(rest); }

    // V's channels lie in runs of 16, turned by the row: a transposing read takes four rows of one run
    static __device__ constexpr uint32_t run(int row, int r) { return row * (2 * D) + ((r ^ (row & kTurn)) << 5); }

    __device__ __forceinline__ void begin(const RowsArgs& p) {
        const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
        k_stride = static_cast<uint32_t>(p.k.token_stride * sizeof(T)), v_stride = static_cast<uint32_t>(p.v.token_stride * sizeof(T));
        const uint32_t row = threadIdx.x / kChunks, c = threadIdx.x % kChunks * 16;
        k_off = row * k_stride + c, v_off = row * v_stride + c;
        k_lane = KeyRows<D>::chunk(KeyRows<D>::key_of(n), h);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v_lane[i] = run(8 * h + 4 * i + ((lane & 15) >> 2), lane >> 4 & 1) + (lane & 3) * 8;
    }
    __device__ __forceinline__ void item(const RowsArgs& p, const Seq& s, int, int head) {
        k = reinterpret_cast<const char*>(row_ptr<T>(p.k, s.k0, head));
        v = reinterpret_cast<const char*>(row_ptr<T>(p.v, s.k0, head));
    }
    // rows behind the sequence's last are its last again, and masked later
    __device__ __forceinline__ void load(const RowsArgs&, const Seq& s, int key0) {
        const int last = s.len - 1 - key0;
        if (last >= kKeys - 1) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                kr[i] = *reinterpret_cast<const vu4*>(k + int64_t(key0 + i * kStep) * k_stride + k_off);
                vr[i] = *reinterpret_cast<const vu4*>(v + int64_t(key0 + i * kStep) * v_stride + v_off);
            }
            return;
        }
        const int c = threadIdx.x % kChunks * 16;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int row = key0 + min(static_cast<int>(threadIdx.x) / kChunks + i * kStep, last);
            kr[i] = vr[i] = vu4{0, 0, 0, 0};
            if (s.len == 0) continue;  // no row at all
            kr[i] = *reinterpret_cast<const vu4*>(k + int64_t(row) * k_stride + c);
            vr[i] = *reinterpret_cast<const vu4*>(v + int64_t(row) * v_stride + c);
        }
    }
    __device__ __forceinline__ void store(const RowsArgs&, const Seq&, uint8_t* lds, uint8_t*, int buf, int) {
        const int row = threadIdx.x / kChunks, c = threadIdx.x % kChunks;
        uint8_t* const at = lds + buf * kBytes;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = row + i * kStep;
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<vu4*>(at + KeyRows<D>::chunk(r, c)) = kr[i];
                *reinterpret_cast<vu4*>(at + kPlane + run(r, c >> 1) + (c & 1) * 16) = vr[i];
            } else {
                vf4 x = __builtin_bit_cast(vf4, kr[i]), y = __builtin_bit_cast(vf4, vr[i]);
                typedef __bf16 vb4 __attribute__((ext_vector_type(4)));
#pragma unroll
                for (int k = 0; k < kKeyParts; ++k) {
                    vb4 a, b;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float f = x[j], g = y[j];
                        a[j] = part(&f), b[j] = part(&g);
                        x[j] = f, y[j] = g;
                    }
                    *reinterpret_cast<vb4*>(at + k * kPlane + KeyRows<D>::chunk(r, c >> 1) + (c & 1) * 8) = a;
                    *reinterpret_cast<vb4*>(at + (kKeyParts + k) * kPlane + run(r, c >> 2) + (c & 3) * 8) = b;
                }
            }
        }
    }
    static __device__ __forceinline__ uint32_t none(const uint8_t*, int) { return 0; }
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
    // whether a channel of key t of a half is infinite or NaN
    __device__ __forceinline__ bool v_bad(const uint8_t* lds, int buf, int half, int t, int c) const {
        const int r = 32 * half + t;
        const uint16_t x = *reinterpret_cast<const uint16_t*>(lds + buf * kBytes + kKeyParts * kPlane + run(r, c >> 4) + (c & 15) * 2);
        return (x & 0x7f80u) == 0x7f80u;
    }
};

template <typename T, int D, typename F>
auto with_kernel(int64_t, F f) {
    using K = Tile<RowSource<T, D>, 1>;
    return f(K(), tile_kernel<K>);
}

template <typename F>
auto with_kernel(int a_dtype, int head_dim, int64_t max_rows, F f) {
    if (a_dtype == CF_BF16)
        return head_dim == 64 ? with_kernel<__bf16, 64>(max_rows, f) : with_kernel<__bf16, 128>(max_rows, f);
    return head_dim == 64 ? with_kernel<float, 64>(max_rows, f) : with_kernel<float, 128>(max_rows, f);
}

}  // namespace

size_t attention_workspace(int a_dtype, int head_dim, int64_t max_rows) {
    return with_kernel(a_dtype, head_dim, max_rows,
                       [&](auto shape, auto) { return plan_of<decltype(shape)>(head_dim).bytes(); });
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
        using S = decltype(shape);
        p.groups = plan_of<S>(c.head_dim).groups;
        p.joins = static_cast<int32_t*>(workspace);
        p.part = reinterpret_cast<float*>(p.joins + kJoin * p.groups);
        kernel<<<p.groups, kThreads, 0, stream>>>(p);
        if (hipError_t e = hipGetLastError()) return e;
        return launch_join<S>(p, max_rows, stream);
    });
}

}  // namespace cf
