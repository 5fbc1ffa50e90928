// cf_kv4_attn.hip - attention over the 4-bit K/V cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i k_j - m_i),  lse_i = m_i + log sum_j p_ij
// over the keys j that row i may see, in one pass over the keys with a running reference m
// and sum.  A row is one (query token, query head); the rows of the query heads that share a
// K/V head are worked on together.
//
// Precision.  K is exact in bf16 and V in fp16 (the cache's exponents see to that) and in bf16, and so are
// bf16 queries; fp32 queries are split into three bf16 parts that add up to them, and so are their
// probabilities.  With bf16 queries P is rounded to fp16 (half a step is 2^-11 of the largest of its tile).  Sums,
// references and O are fp32, and the sum is of unrounded probabilities.
//
// Work.  It is cut into units of 32 (few rows) or 64 keys of one item, an item being up to kRows
// rows of one sequence and K/V head.  Every workgroup takes an equal run of units, whatever
// items they are of: a batch of unequal lengths, and causal rows, leave no workgroup behind.
// Items that end up in several workgroups leave partial results in the workspace, which a second
// kernel joins in the order of the keys.
//
// The kernel for few rows (at most 32: decoding) is bound by the cache's bytes, with fp32 queries by the
// vector units beside them, the one for many rows by the matrix and vector units; measured figures stand
// at each.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf_kv4_few.h"
#include "cf_kv4_wide.h"

namespace cf {
namespace {

// Joins the parts of the items that ended up in several workgroups: block (w, y) some rows
// of the item whose last keys were workgroup w's.  A few microseconds of latency, and with many
// rows the parts' bytes (46 MB, 12 us, for 1024 queries over 4608 keys in 24 heads): eight
// parts are in flight at once (one at a time 12 us where it now takes 4).
template <typename T, int D, int ROWS>
__global__ __launch_bounds__(kThreads) void join_kernel(const AttnArgs p) {
    const int me = blockIdx.x;
    const int32_t* const left = p.joins + me * kJoin;
    const int first = scalar_load(left), head = scalar_load(left + 1), q0 = scalar_load(left + 2),
              row0 = scalar_load(left + 3), rows = scalar_load(left + 4);
    if (first < 0) return;  // and the rest says nothing
    constexpr int kLanes = D / 4, kAtOnce = kThreads / kLanes;
    const int l0 = threadIdx.x % kLanes, c = 4 * l0, self = threadIdx.x & 63 & ~(kLanes - 1);
    for (int r0 = blockIdx.y * kAtOnce; r0 < rows; r0 += gridDim.y * kAtOnce) {
        const int r = min(r0 + static_cast<int>(threadIdx.x) / kLanes, rows - 1);
        const auto part = [&](int w) {
            return p.part + (2 * int64_t(w) + (w == first)) * part_floats<D>(ROWS) + int64_t(r) * (D + 2);
        };
        // a row's lanes look at a part each
        float top = kNone;
        for (int w = first + l0; w <= me; w += kLanes) top = fmaxf(top, part(w)[D]);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        float v[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
        for (int w0 = first; w0 <= me; w0 += kLanes) {
            const int w = w0 + l0;
            float f = 0.f, lw = 0.f;
            if (w <= me) {
                const float2 ml = *reinterpret_cast<const float2*>(part(w) + D);
                f = ml.x == kNone ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
                lw = ml.y;
            }
            const int many = min(kLanes, me + 1 - w0);
            for (int i = 0; i < many; i += 8) {  // eight parts in flight
                float2 x0[8], x1[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float* const x = part(w0 + min(i + k, many - 1));  // again, for nothing: f is 0
                    x0[k] = *reinterpret_cast<const float2*>(x + c), x1[k] = *reinterpret_cast<const float2*>(x + c + 2);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float fi = __shfl(f, self + i + k, 64);
                    l = __builtin_fmaf(__shfl(lw, self + i + k, 64), fi, l);
                    v[0] = __builtin_fmaf(x0[k].x, fi, v[0]);
                    v[1] = __builtin_fmaf(x0[k].y, fi, v[1]);
                    v[2] = __builtin_fmaf(x1[k].x, fi, v[2]);
                    v[3] = __builtin_fmaf(x1[k].y, fi, v[3]);
                }
            }
        }
        if (r0 + static_cast<int>(threadIdx.x) / kLanes >= rows) continue;
        const int row = row0 + r, token = token_of(p, row), qh = head * p.share + row - token * p.share;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T* const o = row_ptr<T>(p.out, q0 + token, qh) + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = static_cast<T>(v[k] * inv);
        if (p.lse && c == 0)
            p.lse[int64_t(q0 + token) * p.q_heads + qh] =
                lse_of(top, l);
    }
}

// A kernel's rows of an item, and its workgroups: as many as are resident at once.
struct Plan {
    int rows, groups, dim;
    size_t bytes() const {
        return size_t(groups) * (2 * (dim == 64 ? part_floats<64>(rows) : part_floats<128>(rows)) * 4 + 4 * kJoin);
    }
};

// Calls f with the kernel's shape and the kernel for a call whose longest sequence has max_rows rows.
template <typename T, int D, typename F>
auto with_kernel(int64_t max_rows, F f) {
    if (max_rows <= 16) return f(Few<T, D, 1>(), few_kernel<T, D, 1>);
    if (max_rows <= 32) return f(Few<T, D, 2>(), few_kernel<T, D, 2>);
    return f(Wide<T, D>(), wide_kernel<T, D>);
}

template <typename F>
auto with_kernel(int a_dtype, int head_dim, int64_t max_rows, F f) {
    if (a_dtype == CF_BF16)
        return head_dim == 64 ? with_kernel<__bf16, 64>(max_rows, f) : with_kernel<__bf16, 128>(max_rows, f);
    return head_dim == 64 ? with_kernel<float, 64>(max_rows, f) : with_kernel<float, 128>(max_rows, f);
}

template <typename S>
Plan plan_of(int head_dim) {
    return {S::kRows, kUnitsOfGpu * S::kResident, head_dim};
}

}  // namespace

// The largest of what the kernels for up to so many rows use: a kernel for more rows may take less (it has
// fewer workgroups resident), and a workspace has to serve every call with fewer rows too.
size_t kv4_attention_workspace(int a_dtype, int head_dim, int64_t max_rows) {
    size_t most = 0;
    for (const int64_t rows : {1, 17, 33}) {  // the fewest of each kernel
        if (rows > max_rows) break;
        const size_t n = with_kernel(a_dtype, head_dim, rows,
                                     [&](auto shape, auto) { return plan_of<decltype(shape)>(head_dim).bytes(); });
        most = n > most ? n : most;
    }
    return most;
}

hipError_t launch_kv4_attention(int a_dtype, const Kv4Attention& c, void* workspace, hipStream_t stream) {
    const int share = c.q_heads / c.cache.heads;
    AttnArgs p{};
    p.q = c.q, p.out = c.out, p.cache = c.cache, p.table = c.table, p.width = c.table_width;
    p.kv_lens = c.kv_lens, p.q_starts = c.q_starts, p.total_q = static_cast<int>(c.total_q);
    p.q_each = c.q_starts ? 0 : static_cast<int>(c.total_q / c.batch);
    p.batch = c.batch, p.q_heads = c.q_heads, p.share = share;
    p.causal = c.causal, p.window = c.window;
    p.scale_log2 = c.scale * 1.44269504088896341f;
    p.lse = c.lse;
    const int64_t max_rows = c.max_q * share;
    return with_kernel(a_dtype, c.cache.block.dim, max_rows, [&](auto shape, auto kernel) {
        using S = decltype(shape);
        p.groups = plan_of<S>(c.cache.block.dim).groups;
        p.joins = static_cast<int32_t*>(workspace);
        p.part = reinterpret_cast<float*>(p.joins + kJoin * p.groups);
        kernel<<<p.groups, kThreads, 0, stream>>>(p);
        if (hipError_t e = hipGetLastError()) return e;
        const int at_once = kThreads / (S::kDim / 4), rows = max_rows < S::kRows ? static_cast<int>(max_rows) : S::kRows;
        join_kernel<typename S::Type, S::kDim, S::kRows>
            <<<dim3(p.groups, (rows + at_once - 1) / at_once), kThreads, 0, stream>>>(p);
        return hipGetLastError();
    });
}

}  // namespace cf
