// Internal launchers of libcf (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf.h"
#include "cf_kv4.h"
#include "cf_kv8.h"

namespace cf {

// Groups of 128 contiguous elements are the unit of every 1/2-bit kernel.
constexpr int kGroup = 128;

// A dispatch counts its work-items per grid dimension in 32 bits.
constexpr int64_t kMaxDispatchItems = (int64_t(1) << 32) - 1;

hipError_t launch_init(int a_dtype, const void* a, float* ahat, float* err, int64_t numel,
                       hipStream_t stream);
hipError_t launch_compress(int bits, int a_dtype, const void* a, float* ahat, float* err,
                           uint8_t* codes, float* scales, int64_t numel, hipStream_t stream);
hipError_t launch_compress_ablation(int mode, int bits, int a_dtype, const void* a, const void* a_prev,
                                    float* ahat, uint8_t* codes, float* scales, int64_t numel,
                                    hipStream_t stream);
// out (bf16 bits of the updated reconstruction) may be null.
hipError_t launch_decompress(int bits, const uint8_t* codes, const float* scales, float* ahat, uint16_t* out,
                             int64_t numel, hipStream_t stream);

// Top-k sparsification of the residual: k of every 128 kept as (index byte, bf16 value).
hipError_t launch_topk_compress(int k, int a_dtype, const void* a, float* ahat, float* err, uint8_t* idx,
                                uint16_t* vals, int64_t numel, hipStream_t stream);
hipError_t launch_topk_decompress(int k, const uint8_t* idx, const uint16_t* vals, float* ahat, int64_t numel,
                                  hipStream_t stream);

// Low-rank workspace regions (carved from one caller buffer).
struct LowrankWorkspace {
    float* r;      // batch x m x n residual
    float* qt;     // batch x kp x n, Q transposed (rank padded to a multiple of 16)
    float* ypart;  // Y partials: batch x segments x m x kp of a projection, or two per strip
                   // range of a fused pass
    float* p;      // batch x m x kp orthonormal factor
    int* alive;    // batch x kp rank-guard flags
    double* gpart; // batch x row blocks x kp x kp Gram partials
    float* cmax;   // batch x row blocks x kp column maxima of the factors
    bool shared;   // one of two halves of a call, run on two streams at once
};

// Largest rank the low-rank kernels accept.
constexpr int kMaxRank = 64;

// Fills the region pointers of one launch sequence over `batch` tensors for `base` (may
// be null) and its size in *bytes; `shared`: the sequence is one of a call's two halves.
LowrankWorkspace carve_lowrank_workspace(void* base, int64_t m, int64_t n, int rank, int64_t batch, bool shared,
                                         size_t* bytes);
// Workspace bytes of a whole call (a large call runs two halves, each with its own regions).
size_t lowrank_workspace_total(int64_t m, int64_t n, int rank, int64_t batch);
// Whether every launch of one low-rank call (or of its receiver) fits a dispatch.
bool lowrank_launches_fit(int64_t m, int64_t n, int rank, int64_t batch);
hipError_t launch_lowrank_compress(int a_dtype, const void* a, float* ahat, float* err, int64_t m,
                                   int64_t n, int rank, int iters, int factor_bits, int64_t batch,
                                   float* q_state, void* u, float* u_scales, void* v, float* v_scales,
                                   void* workspace, hipStream_t stream);
hipError_t launch_lowrank_decompress(int factor_bits, const void* u, const float* u_scales,
                                     const void* v, const float* v_scales, float* ahat, int64_t m,
                                     int64_t n, int rank, int64_t batch, hipStream_t stream);

// Rows of heads: row (t, h) starts at data + t * token_stride + h * head_stride elements.
using RowSet = cf_rows;

hipError_t launch_qk_norm_rope(int a_dtype, int64_t tokens, int q_heads, int k_heads, int head_dim, const RowSet& q,
                               const RowSet& k, const RowSet& q_out, const RowSet& k_out, int norm,
                               const float* q_weight, const float* q_bias, const float* k_weight,
                               const float* k_bias, float eps, int rope, const float* cos, const float* sin,
                               int64_t n_pos, int rot_dim, const int32_t* positions, hipStream_t stream);

hipError_t launch_kv4_append(int a_dtype, const RowSet& k, const RowSet& v, const int64_t* slots, int64_t tokens,
                             const KvCache& cache, hipStream_t stream);
hipError_t launch_kv4_read(int a_dtype, const RowSet& k, const RowSet& v, const int64_t* slots, int64_t tokens,
                           const KvCache& cache, hipStream_t stream);

// One attention call over a paged cache.
template <typename CACHE>
struct PagedAttention {
    RowSet q, out;
    CACHE cache;
    const int32_t* table;     // batch x table_width, or null: sequence b has pages b * table_width ..
    const int32_t* kv_lens;   // batch
    const int32_t* q_starts;  // batch + 1, or null: total_q / batch queries each
    float* lse;               // total_q x q_heads, or null
    int64_t total_q, max_q;
    int batch, table_width, q_heads, causal, window;
    float scale;
};
using Kv4Attention = PagedAttention<KvCache>;
using Kv8Attention = PagedAttention<Kv8Cache>;
// max_rows: the most query tokens of a sequence times the query heads of a K/V head.
size_t kv4_attention_workspace(int a_dtype, int head_dim, int64_t max_rows);
hipError_t launch_kv4_attention(int a_dtype, const Kv4Attention& call, void* workspace, hipStream_t stream);
size_t kv8_attention_workspace(int a_dtype, int head_dim, int64_t max_rows);
hipError_t launch_kv8_attention(int a_dtype, const Kv8Attention& call, void* workspace, hipStream_t stream);

hipError_t launch_kv8_append(int a_dtype, const RowSet& k, const RowSet& v, int64_t tokens, const Kv8Cache& cache,
                             int batch, const int32_t* table, int table_width, const int32_t* kv_lens,
                             const int32_t* starts, hipStream_t stream);
hipError_t launch_kv8_read(int a_dtype, const RowSet& k, const RowSet& v, const int64_t* slots, int64_t tokens,
                           const Kv8Cache& cache, hipStream_t stream);

// One attention call over rows of keys and values.
struct RowsAttention {
    RowSet q, k, v, out;
    const int32_t* q_starts;  // batch + 1, or null: total_q / batch queries each
    const int32_t* k_starts;  // batch + 1, or null: total_k / batch keys each
    float* lse;               // total_q x q_heads, or null
    int64_t total_q, total_k, max_q;
    int batch, q_heads, kv_heads, head_dim, causal, window;
    float scale;
};
size_t attention_workspace(int a_dtype, int head_dim, int64_t max_rows);
hipError_t launch_attention(int a_dtype, const RowsAttention& call, void* workspace, hipStream_t stream);

// One operation on the pages of a cache: sequences in and out (refs, table, lens), and what it reads and says besides.
using Pages = cf_pages;
struct PagesCall {
    Pages in, out;
    int64_t pages;
    int rows, width, page_size;
    const int32_t* want;  // tokens, or parents
    int32_t *src, *dst, *count;
};
size_t pages_workspace(int64_t pages, int rows);
hipError_t launch_pages_resize(const PagesCall& call, void* workspace, hipStream_t stream);
hipError_t launch_pages_fork(const PagesCall& call, bool own, void* workspace, hipStream_t stream);
hipError_t launch_pages_compact(const PagesCall& call, void* workspace, hipStream_t stream);
hipError_t launch_pages_copy(void* data, int64_t pages, int64_t page_bytes, int layers, int64_t layer_stride, const int32_t* src,
                             const int32_t* dst, int64_t n, const int32_t* count, hipStream_t stream);

// A number that no other call of this process has, and hardly anything else that memory may hold; not 0.
uint64_t call_number();

}  // namespace cf
