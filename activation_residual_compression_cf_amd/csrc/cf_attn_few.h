// What the attention kernels for few rows share: their queries, and how the waves' results of an item are put
// together.
#pragma once

#include "cf_attn_plan.h"

namespace cf {
namespace {

// Queries of 16 rows: bf16 parts that add up to them, channel order as in K's codes.
template <int D, int PARTS>
struct Rows {
    vb8 q[PARTS][D / 32];
};

template <typename T, int D, int PARTS>
__device__ __forceinline__ void load_rows(Rows<D, PARTS>& x, const AttnRows& p, const Seq& s, int head, int row,
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

template <typename T>
__device__ __forceinline__ void store_out(T* o, const float (&x)[8]) {
    Row8<T> r;
    r.set(x);
    r.store(o);
}

// The results of units [a, z) of an item, which its four waves hold in parts: the whole item, or a part for the
// join.  own(i, c): the lane's value number c of D/4, consecutive channels from g * (D/4) on, of row n of the i-th
// sixteen.
template <typename T, int D, int NQ, typename F>
__device__ __forceinline__ void finish_few(const AttnRows& p, const Place& w, const Seq& s, int a, int z, int count,
                                           vf4 (&o)[NQ][D / 16], float (&m)[NQ], float (&sum)[NQ], float (&high)[NQ],
                                           float* stage, float* stage_m, float* stage_l, F own) {
    constexpr int kRows = 16 * NQ, kJ = D / 16;
    const int me = w.me, rows = s.nq * p.share;
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x) >> 6), n = lane & 15, g = lane >> 4;
    // this segment's results: the whole item, or a part for the second kernel
    const bool whole = a == 0 && z == count;
    float* const part = p.part + (2 * int64_t(me) + (a == 0)) * part_floats<D>(kRows);
    const auto put = [&](int r, int c, float (&v)[8], float top, float l, bool first_piece) {
        // eight channels from c of row r of the item
        const int row = w.tile * kRows + r;
        if (row >= rows) return;
        if (whole) {
            const int token = token_of(p, row), qh = w.head * p.share + row - token * p.share;
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
            *reinterpret_cast<vf4*>(y + c) = vf4{own(i, c), own(i, c + 1), own(i, c + 2), own(i, c + 3)};
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
}

}  // namespace
}  // namespace cf
