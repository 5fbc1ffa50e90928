// cf_norm.hip - norms of queries and keys for each head, and the position rotation, in one pass.
//
// Row x of D channels (one token, one head):
//   none   n = x
//   RMS    n = x / sqrt(mean(x^2) + eps)
//   layer  n = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps)
//   y = n * w + b, and the first R channels of y turned in pairs (i, j) by the token's angle:
//   y_i' = y_i cos - y_j sin,  y_j' = y_j cos + y_i sin;  pairs (2p, 2p+1) or (p, p + R/2).
// All of it in fp32, rounded once to the rows' type.
//
// Bound by memory: a row is read once and written once.  17550 tokens of 30 + 30 heads of 64 in
// fp32 take 114 us, 4.8 TB/s, where the best copy reaches 6.2 (a lane's eight fp32 channels make its
// 16-byte accesses two-way strided); 1024 tokens of 24 + 24 heads of 128 in bf16 10 us, 16
// tokens 4.0 us (a launch and one round of loads).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf.h"
#include "cf_internal.h"
#include "cf_rows.h"

namespace cf {
namespace {

constexpr int kThreads = 256;
// Rows a slot has in flight: their loads are issued together, before the first is used.
constexpr int kBatch = 4;

struct NormArgs {
    RowSet q, k, qo, ko;
    int64_t tokens;
    int q_heads, heads, dim;  // heads: of q and k together
    int slots;                // slots of a token
    const float *qw, *qb, *kw, *kb;
    float eps;
    const float *cos, *sin;
    const int32_t* positions;
    int64_t n_pos;
    int rot;
};

// Sum over the LPR lanes of a slot, in a fixed order.
template <int LPR>
__device__ __forceinline__ float slot_sum(float v) {
#pragma unroll
    for (int s = 1; s < LPR; s <<= 1) v += __shfl_xor(v, s, 64);
    return v;
}

// A slot of LPR lanes (8 channels a lane) takes the heads s, s + slots, ... of one token, so a
// token's angles are loaded once for all its heads and a wave's loads stay side by side.
template <typename T, int LPR, int NORM, int ROPE>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(const NormArgs p) {
    const int64_t slot = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / LPR;
    const int lane = threadIdx.x % LPR;
    const int64_t t = slot / p.slots;
    if (t >= p.tokens) return;  // whole slots leave together; a slot's shuffles stay inside it
    const int c0 = lane * 8;
    const bool on = c0 < p.dim;

    float cs[8], sn[8];
    bool lost = false;  // a position behind the table: the row becomes NaN
    const int half = p.rot / 2;
    if constexpr (ROPE != CF_ROPE_NONE) {
        const int64_t pos = p.positions ? p.positions[t] : t;
        if (pos < 0) return;  // padding: the token's rows stay as they are
        lost = pos >= p.n_pos;
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
        if (c0 < p.rot && !lost) {
            if constexpr (ROPE == CF_ROPE_HALF) {
                // channels c0 .. of the first half, or their partners of the second
                const int a = c0 < half ? c0 : c0 - half;
                const float* pc = p.cos + pos * half + a;
                const float* ps = p.sin + pos * half + a;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const vf4 c = *reinterpret_cast<const vf4*>(pc + i), s = *reinterpret_cast<const vf4*>(ps + i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) cs[i + j] = c[j], sn[i + j] = c0 < half ? -s[j] : s[j];
                }
            } else {
                const vf4 c = *reinterpret_cast<const vf4*>(p.cos + pos * half + c0 / 2);
                const vf4 s = *reinterpret_cast<const vf4*>(p.sin + pos * half + c0 / 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) cs[2 * j] = cs[2 * j + 1] = c[j], sn[2 * j] = -s[j], sn[2 * j + 1] = s[j];
            }
        }
    }
    // lane that holds this lane's partners (half style); itself where nothing turns
    const int mate = c0 >= p.rot ? lane : c0 < half ? lane + half / 8 : lane - half / 8;
    const float inv_d = 1.f / float(p.dim);

    for (int h0 = int(slot - t * p.slots); h0 < p.heads; h0 += kBatch * p.slots) {
        Row8<T> raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * p.slots;
            if (h < p.heads && on)
                raw[u].load(h < p.q_heads ? row_ptr<T>(p.q, t, h) + c0 : row_ptr<T>(p.k, t, h - p.q_heads) + c0);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * p.slots;
            if (h >= p.heads) break;
            const bool is_q = h < p.q_heads;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
            if (on) raw[u].get(x);
            if constexpr (NORM == CF_NORM_LAYER) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x[i];
                const float mean = slot_sum<LPR>(s) * inv_d;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = on ? x[i] - mean : 0.f;
            }
            if constexpr (NORM != CF_NORM_NONE) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x[i], x[i], s);
                const float r = 1.f / __builtin_sqrtf(slot_sum<LPR>(s) * inv_d + p.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= r;
            }
            const float* w = is_q ? p.qw : p.kw;
            const float* b = is_q ? p.qb : p.kb;
            if (w && on) {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const vf4 v = *reinterpret_cast<const vf4*>(w + c0 + i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[i + j] *= v[j];
                }
            }
            if (b && on) {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const vf4 v = *reinterpret_cast<const vf4*>(b + c0 + i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[i + j] += v[j];
                }
            }
            if constexpr (ROPE != CF_ROPE_NONE) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = ROPE == CF_ROPE_HALF ? __shfl(x[i], (threadIdx.x & 63 & ~(LPR - 1)) | mate, 64) : x[i ^ 1];
                // channels behind the rotated ones stay bit for bit, also where they are infinite
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 < p.rot) x[i] = __builtin_fmaf(o[i], sn[i], x[i] * cs[i]);
                if (lost)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
            }
            if (on) {
                Row8<T> y;
                y.set(x);
                y.store(is_q ? row_ptr<T>(p.qo, t, h) + c0 : row_ptr<T>(p.ko, t, h - p.q_heads) + c0);
            }
        }
    }
}

template <typename T, int LPR, int NORM>
void launch_rope(int rope, uint32_t blocks, hipStream_t stream, const NormArgs& p) {
    switch (rope) {
        case CF_ROPE_NONE:
            norm_rope_kernel<T, LPR, NORM, CF_ROPE_NONE><<<blocks, kThreads, 0, stream>>>(p);
            break;
        case CF_ROPE_INTERLEAVED:
            norm_rope_kernel<T, LPR, NORM, CF_ROPE_INTERLEAVED><<<blocks, kThreads, 0, stream>>>(p);
            break;
        default: norm_rope_kernel<T, LPR, NORM, CF_ROPE_HALF><<<blocks, kThreads, 0, stream>>>(p);
    }
}

template <typename T, int LPR>
void launch_norm(int norm, int rope, uint32_t blocks, hipStream_t stream, const NormArgs& p) {
    switch (norm) {
        case CF_NORM_NONE: launch_rope<T, LPR, CF_NORM_NONE>(rope, blocks, stream, p); break;
        case CF_NORM_RMS: launch_rope<T, LPR, CF_NORM_RMS>(rope, blocks, stream, p); break;
        default: launch_rope<T, LPR, CF_NORM_LAYER>(rope, blocks, stream, p);
    }
}

// Slots of a token: a wave's worth where there are tokens enough to fill the chip, one for
// every head where there are few.
int slots_of(int64_t tokens, int heads, int lpr) {
    const int wave = 64 / lpr;
    int s = wave;
    while (s < heads && tokens * s * lpr < int64_t(256) * 4 * kThreads) s += wave;
    return s < heads ? s : heads;
}

template <typename T>
hipError_t launch(int norm, int rope, NormArgs& p, hipStream_t stream) {
    const int lpr = p.dim <= 64 ? 8 : p.dim <= 128 ? 16 : 32;
    p.slots = slots_of(p.tokens, p.heads, lpr);
    const auto blocks = static_cast<uint32_t>((p.tokens * p.slots * lpr + kThreads - 1) / kThreads);
    if (lpr == 8) launch_norm<T, 8>(norm, rope, blocks, stream, p);
    if (lpr == 16) launch_norm<T, 16>(norm, rope, blocks, stream, p);
    if (lpr == 32) launch_norm<T, 32>(norm, rope, blocks, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(int a_dtype, int64_t tokens, int q_heads, int k_heads, int head_dim, const RowSet& q,
                               const RowSet& k, const RowSet& q_out, const RowSet& k_out, int norm,
                               const float* q_weight, const float* q_bias, const float* k_weight,
                               const float* k_bias, float eps, int rope, const float* cos, const float* sin,
                               int64_t n_pos, int rot_dim, const int32_t* positions, hipStream_t stream) {
    NormArgs p{q, k, q_out, k_out, tokens, q_heads, q_heads + k_heads, head_dim, 0, q_weight, q_bias, k_weight,
               k_bias, eps, cos, sin, positions, n_pos, rope == CF_ROPE_NONE ? 0 : rot_dim};
    return a_dtype == CF_BF16 ? launch<__bf16>(norm, rope, p, stream) : launch<float>(norm, rope, p, stream);
}

}  // namespace cf
