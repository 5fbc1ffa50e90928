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
    p.batch = c.batch, p.q_heads = c.q_heads, p.kv_heads = c.cache.heads, p.share = share;
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
        return launch_join<S>(p, max_rows, stream);
    });
}

}  // namespace cf
