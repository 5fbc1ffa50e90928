/*
 * cf.h - C ABI of libcf: CompactFusion step-wise activation residual compression
 * with sender-side error feedback, on MI355X (gfx950).
 *
 * Method: "Accelerating Parallel Diffusion Model Serving with Residual
 * Compression" (CompactFusion summary), section Approach; the measured-effects
 * table names the variants built here (Compact-1bit, Compact-2bit,
 * Compact-Lowrank) and the warmup steps.  In short: what crosses the wire at a
 * denoising step is the residual between a layer's activation and the
 * reconstruction both sides already hold, compressed; the sender keeps the part
 * the compression lost and feeds it into the next step's residual; the low-rank
 * variant sends two INT4-quantized factors instead of codes.
 *
 * Conventions shared by every entry point
 *   - Every pointer is a DEVICE pointer on the current HIP device, allocated and
 *     owned by the caller, who keeps it alive until the stream work is done.
 *     The library allocates nothing in these calls and keeps no pointer after
 *     a call returns.
 *   - Calls are stream-ordered and asynchronous: CF_OK means "validated and
 *     enqueued on `stream`" (a hipStream_t; NULL = the null stream).  A fault
 *     inside a kernel surfaces at the caller's next synchronisation.
 *   - Every argument is validated before anything is enqueued, so a call that
 *     returns an error has written nothing (a half-applied state update would
 *     corrupt the error feedback).
 *   - Activations `a` are bf16 (CF_BF16, raw 16-bit storage) or fp32 (CF_F32),
 *     row-major; the reconstruction `ahat` and the error buffer `err` are fp32.
 *   - The error feedback lives in `ahat`: the next step's residual is a - ahat, so
 *     the sender never reads `err`, and resuming needs `ahat` alone.  The senders
 *     therefore take `err = NULL`, which skips writing it (4 bytes per element less;
 *     the low-rank sender also skips re-reading `a`).
 *     State lives only in caller buffers, so a checkpoint is a copy of them.
 *   - A group is CF_GROUP = 128 contiguous elements; `numel` must be a positive
 *     multiple of 128, at most 2^33.  Several tensors laid out back to back may be passed as
 *     one call (one "slab"), since no group straddles two tensors when every
 *     tensor's size is a multiple of 128.
 *   - Every pointer must be 16-byte aligned, except `scales` (one float per
 *     group), which needs 4-byte alignment, and the top-k payload (see there);
 *     input and output ranges must not overlap.
 *   - Results are deterministic: no atomics, fixed reduction orders.
 *   - Calls on different streams with disjoint buffers may run concurrently.
 *   - Non-finite inputs give unspecified (but memory-safe) results.
 */
#ifndef CF_H
#define CF_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes: 0 on success, negative on error. */
enum {
    CF_OK = 0,
    CF_E_NULL = -1,      /* a required pointer is NULL */
    CF_E_SHAPE = -2,     /* numel / m / n / rank / batch out of range */
    CF_E_ALIGN = -3,     /* a pointer is misaligned (16 bytes; scales 4 bytes) */
    CF_E_ARG = -4,       /* bits, k, dtype, factor_bits or iters not supported */
    CF_E_ALIAS = -5,     /* an output range overlaps another operand */
    CF_E_WORKSPACE = -6, /* workspace missing or too small */
    CF_E_DEVICE = -7,    /* current device is not gfx950 */
    CF_E_HIP = -8,       /* the HIP runtime refused a launch; a call that launches several
                            kernels (cf_lowrank_compress) may then have applied part of
                            its update, so treat the state as lost (re-run the warmup) */
    CF_E_SCRATCH = -9    /* cf_lowrank_compress_noalloc: the call needs more scratch than
                            the fixed CF_NOALLOC_SCRATCH_BYTES */
};

enum { CF_BF16 = 0, CF_F32 = 1 };

/* Sender modes of cf_compress_ablation. */
enum { CF_MODE_NOEF = 1, CF_MODE_NAIVE = 2 };

#define CF_GROUP 128

/*
 * Warmup / initialisation (measured-effects table: the rows with one and with two
 * warmup steps).  During the first W steps the activation itself is sent and both
 * sides take it as their reconstruction:  ahat[i] = a[i]  and, when `err` is
 * not NULL (the sender), err[i] = 0.  The receiver passes err = NULL.
 *   a:    numel elements of `a_dtype`
 *   ahat: numel fp32 (out)      err: numel fp32 (out) or NULL
 */
int cf_init_state(int a_dtype, const void* a, float* ahat, float* err, int64_t numel,
                  void* stream);

/*
 * Sender step, Compact-1bit / Compact-2bit (Approach: residual against the
 * previous reconstruction with sender-side error feedback).  Per group g of 128
 * contiguous elements:
 *   r = a - ahat                                         (fp32)
 *   bits = 1: s = mean|r| over the group, taken exactly and rounded once to
 *             fp32 (to nearest, ties to even), so it depends on no summation order;
 *             code = (r < 0);  d = code ? -s : s
 *   bits = 2: s = max|r| / 1.5 (IEEE division);  sign = (r < 0),
 *             mag = (|r| > s);  code = sign | mag << 1;
 *             d = +-(mag ? 1.5*s : 0.5*s)   (levels {-1.5,-0.5,0.5,1.5}*s)
 *   ahat = ahat + d;   err = a - ahat        (each operation rounded once)
 *   codes: numel*bits/8 bytes, LSB first, groups back to back (16*bits bytes
 *          per group); scales: numel/128 fp32, one per group.
 *   a: in; ahat: in/out; err: out or NULL; codes, scales: out.
 */
int cf_compress(int bits, int a_dtype, const void* a, float* ahat, float* err, uint8_t* codes,
                float* scales, int64_t numel, void* stream);

/*
 * Receiver step: decodes codes/scales with exactly the sender's expression for
 * d and applies ahat = ahat + d, so the receiver's reconstruction equals the
 * sender's bit for bit (Approach: the receiver rebuilds the activation from
 * the transmitted residuals).
 *   codes, scales: in (as produced by cf_compress); ahat: in/out.
 */
int cf_decompress(int bits, const uint8_t* codes, const float* scales, float* ahat, int64_t numel,
                  void* stream);

/*
 * Receiver step with a bf16 copy for the consumer (the attention that reads the
 * reconstructed K/V): exactly cf_decompress, and then out[i] = the
 * round-to-nearest-even bf16 of the updated ahat[i].  Decoding several peers'
 * payloads is one call when their codes, scales, mirrors and outputs are laid out
 * back to back (peer p at offset p * numel_per_peer).
 *   out: numel bf16 (raw 16-bit storage), 16-byte aligned, out.
 */
int cf_decompress_bf16(int bits, const uint8_t* codes, const float* scales, float* ahat, uint16_t* out,
                       int64_t numel, void* stream);

/*
 * Ablation modes of the sender, for studies of the method's design (measured-
 * effects table: the row that adds residual compression with error feedback;
 * Surprising findings: 1-bit quantization of whole activations, without residuals,
 * fails).  Same
 * quantizer, codes and scales as cf_compress; per group:
 *   CF_MODE_NOEF:  r = a - a_prev (the raw step delta, no error feedback);
 *                  ahat = ahat + d (the receiver's mirror, which cf_decompress
 *                  reproduces); a_prev: numel of a_dtype, in.
 *   CF_MODE_NAIVE: r = a (the activation itself); ahat = d (its decoded value);
 *                  a_prev unused (may be NULL).
 * No error buffer is kept in either mode.
 */
int cf_compress_ablation(int mode, int bits, int a_dtype, const void* a, const void* a_prev, float* ahat,
                         uint8_t* codes, float* scales, int64_t numel, void* stream);

/*
 * Sender step, top-k sparsification of the residual (Limitations: sparsity is
 * the other fast compressor family beside quantization; the pages give no rule,
 * and the one built here is the following).  Per group g of 128 contiguous
 * elements:
 *   r = a - ahat                                               (fp32)
 *   keep the k elements of largest |r|, ordered by the bit pattern of |r| (the
 *   magnitude order for non-NaN values), equal magnitudes going to the lower
 *   index;  for each kept element i, in increasing i:
 *     idx[g*k + slot] = i (0..127);  vals[g*k + slot] = v = RNE bf16 of r[i];
 *     ahat[i] = ahat[i] + widen(v)
 *   err = a - ahat for all 128 elements (the dropped residuals stay in err).
 *   1 <= k <= 128 (k = 12 spends the 2-bit budget of 36 bytes per group).
 *   idx: numel/128*k bytes, any alignment; vals: numel/128*k bf16 (raw 16-bit),
 *   2-byte aligned; a, ahat, err: 16-byte aligned.
 *   a: in; ahat: in/out; err: out or NULL; idx, vals: out.
 */
int cf_topk_compress(int k, int a_dtype, const void* a, float* ahat, float* err, uint8_t* idx, uint16_t* vals,
                     int64_t numel, void* stream);

/*
 * Receiver step, top-k: ahat[g*128 + (idx[g*k+s] & 127)] += widen(vals[g*k+s]) for
 * every slot s, the sender's own update, so the reconstructions agree bit for bit.
 * Only the low 7 bits of an index byte are used, so any payload stays inside its
 * group; a payload that repeats an index within a group (the sender never does)
 * gives an unspecified value at that element.
 *   idx, vals: in (as produced by cf_topk_compress); ahat: in/out, 16-byte aligned.
 */
int cf_topk_decompress(int k, const uint8_t* idx, const uint16_t* vals, float* ahat, int64_t numel,
                       void* stream);

/*
 * Sender step, Compact-Lowrank (Approach: low-rank compression of the residual
 * with INT4 quantization of the factors; Key results: rank 32 with INT4 factors
 * gives about 100x; measured-effects table: 2 vs 10 subspace iterations;
 * Experimental setup, "Builds on": PowerSGD-style subspace iteration).
 * `batch` tensors of m x n (row-major) laid out back to back.  Per tensor:
 *   r = a - ahat;  Q = q_state;
 *   repeat `iters` times:  Y = r Q;  P = orth(Y);  Q = r^T P
 *     orth: thin QR factor with diag(R) >= 0; a rank-deficient column (|R_jj| <=
 *     1e-5 ||Y||_F) gives a zero column of P;
 *   factor_bits 4:  U = int4(P), V = int4(Q): per column j, s_j = max|x| / 7,
 *     code = rint(x / s_j) clamped to [-7, 7] (0 when s_j = 0), two's-complement
 *     nibbles, row-major rows x rank, low nibble first;  U^ = code * s_j;
 *   factor_bits 16: U, V = the round-to-nearest-even bf16 of P, Q, row-major
 *     (rows x rank) (the table's "Pure Lowrank" variant); scales unused;
 *   factor_bits 32: U = P, V = Q as fp32 row-major (rows x rank); scales unused;
 *   ahat = ahat + U^ V^^T;   err = a - ahat;
 *   q_state = Q (a column zeroed by the rank guard keeps its previous value).
 * Buffers (all device memory):
 *   a: batch*m*n (a_dtype), in; ahat: batch*m*n fp32, in/out; err: out or NULL;
 *   q_state: batch*n*rank fp32, in/out (the start basis; a seeded N(0,1) matrix
 *     before the first compressed step);
 *   u: batch*m*rank*factor_bits/8 bytes, out; v: batch*n*rank*factor_bits/8 bytes,
 *     out; both 4-byte aligned;
 *   u_scales, v_scales: batch*rank fp32, out (may be NULL unless factor_bits = 4);
 *   workspace: ws_bytes >= cf_lowrank_workspace_bytes(m, n, rank, batch), 256-byte
 *     aligned; scratch, its contents are not preserved between calls.
 * Limits: m and n positive multiples of 16; batch*m*n <= 2^33; 1 <= rank <=
 *   min(m, n, 64); rank even when factor_bits = 4; 1 <= iters <= 64; batch >= 1;
 *   every kernel grid within a dispatch's 2^32 - 1 work-items (only extreme shapes,
 *   such as a single row block of 2^28 columns, reach that); CF_E_SHAPE otherwise.
 *   a, ahat, err 16-byte aligned; the other pointers 4-byte aligned.
 * Arithmetic is fp32 (fp64 inside orth).  Results are deterministic for given shapes,
 * rank, iters and batch; a tensor's last bits depend on the batch it is sent in, since
 * the fp32 sums of Y follow the work's split of the whole batch into equal parts.
 */
int cf_lowrank_compress(int a_dtype, const void* a, float* ahat, float* err, int64_t m, int64_t n,
                        int rank, int iters, int factor_bits, int batch, float* q_state, void* u,
                        float* u_scales, void* v, float* v_scales, void* workspace, size_t ws_bytes,
                        void* stream);

/*
 * Receiver step, Compact-Lowrank (Approach: the receiver rebuilds the activation by
 * adding the decoded low-rank residual to its copy of the previous reconstruction;
 * measured-effects table: rank 32 with INT4 factors):  ahat = ahat + U^ V^^T for
 * `batch` tensors, with the sender's dequantization and the sender's reconstruction
 * kernel, so the receiver's ahat equals the sender's bit for bit.  Buffers and limits
 * as in cf_lowrank_compress; u, u_scales, v, v_scales in; ahat in/out.
 */
int cf_lowrank_decompress(int factor_bits, const void* u, const float* u_scales, const void* v,
                          const float* v_scales, float* ahat, int64_t m, int64_t n, int rank,
                          int batch, void* stream);

/*
 * cf_lowrank_compress without a workspace argument, for callers that cannot allocate
 * device memory around the call: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Identical arguments, results and errors to
 * cf_lowrank_compress, except that the workspace is a fixed buffer of
 * CF_NOALLOC_SCRATCH_BYTES that the library holds in each GPU's memory from the first
 * load of its code object until the process ends; the call allocates nothing.
 *   - A call whose cf_lowrank_workspace_bytes(m, n, rank, batch) exceeds
 *     CF_NOALLOC_SCRATCH_BYTES returns CF_E_SCRATCH and writes nothing (64 MiB holds
 *     four 1024 x 3072 tensors at rank 32; split larger batches into several calls).
 *   - Every call on one GPU uses that GPU's one buffer: calls that may overlap in time
 *     on one GPU (different streams, or several host threads) race and give wrong
 *     results.  Order them on one stream, or use cf_lowrank_compress with a workspace
 *     per stream.  Nothing in the buffer needs to start at zero: each call writes every
 *     byte it reads before reading it.
 */
#define CF_NOALLOC_SCRATCH_BYTES (64u << 20)

int cf_lowrank_compress_noalloc(int a_dtype, const void* a, float* ahat, float* err, int64_t m, int64_t n,
                                int rank, int iters, int factor_bits, int batch, float* q_state, void* u,
                                float* u_scales, void* v, float* v_scales, void* stream);

/*
 * Attention operators beside the compressors: what makes the queries and keys (their
 * norms and position rotation), what keeps K and V in 4 bits, and what reads them.
 *
 * Rows of heads.  These entry points take activations of heads as cf_rows: row (t, h) of
 * token t and head h is head_dim consecutive elements from data + t * token_stride +
 * h * head_stride (strides in elements), so slices of a packed projection and head-major
 * layouts pass without a copy.  Every row starts on 16 bytes (CF_E_ALIGN otherwise).
 * Strides are not negative; rows that are written must not overlap each other: either
 * head_stride >= head_dim and token_stride >= the heads' extent, or the reverse
 * (CF_E_SHAPE).  tokens = 0 is a valid call that does nothing.
 */
typedef struct cf_rows {
    void* data;
    int64_t token_stride, head_stride;
} cf_rows;

/* Norms of cf_qk_norm_rope, and its rotation's pairs. */
enum { CF_NORM_NONE = 0, CF_NORM_RMS = 1, CF_NORM_LAYER = 2 };
enum { CF_ROPE_NONE = 0, CF_ROPE_INTERLEAVED = 1, CF_ROPE_HALF = 2 };

/*
 * Norms of queries and keys for each head, with the position rotation in the same pass.
 * Per row x of D = head_dim channels, in fp32, rounded once to a_dtype at the end:
 *   CF_NORM_NONE   n = x
 *   CF_NORM_RMS    n = x / sqrt(mean(x^2) + eps)
 *   CF_NORM_LAYER  n = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps)
 *   y = n * weight + bias  (head_dim fp32 each; NULL = ones / zeros)
 *   the first rot_dim channels of y in pairs (i, j), pair p by the angle whose cosine and
 *   sine are cos[pos * rot_dim/2 + p] and sin[pos * rot_dim/2 + p]:
 *     y_i cos - y_j sin,  y_j cos + y_i sin
 *   CF_ROPE_INTERLEAVED (2p, 2p + 1);  CF_ROPE_HALF (p, p + rot_dim/2);
 *   CF_ROPE_NONE rotates nothing and reads neither tables nor positions.
 *   positions: tokens int32, or NULL = token t has position t (then tokens <= n_pos).  A
 *     token with a negative position is padding: its rows in q_out and k_out stay as they
 *     are.  A position of n_pos or more gives rows of NaN.
 *   cos, sin: n_pos x rot_dim/2 fp32.
 * tokens * heads at most 2^28 rows, times head_dim at most 2^33.  head_dim a multiple of 8, at
 * most 256; rot_dim a multiple of 16, at most head_dim; eps finite and not negative.  q_heads
 * or k_heads may be 0 (that side's pointers are then not used).  In place (q_out the same rows
 * as q, k_out as k) is allowed; any other overlap of an output with another operand is not.
 *   weights, biases, cos, sin: 16-byte aligned; positions 4.
 */
int cf_qk_norm_rope(int a_dtype, int64_t tokens, int q_heads, int k_heads, int head_dim, const cf_rows* q,
                    const cf_rows* k, const cf_rows* q_out, const cf_rows* k_out, int norm,
                    const float* q_weight, const float* q_bias, const float* k_weight, const float* k_bias,
                    float eps, int rope, const float* cos, const float* sin, int64_t n_pos, int rot_dim,
                    const int32_t* positions, void* stream);

/*
 * The 4-bit K/V cache: `pages` pages of `page_size` tokens for each of kv_heads heads, in one
 * buffer of cf_kv4_cache_bytes bytes.  There are fewer than 2^31 pages.  head_dim D is 64 or
 * 128; page_size P is 16, 32, 64, 128 or 256.  The block of page p and head h starts at
 * (p * kv_heads + h) * P * D * 17/16 and holds, in this order:
 *   K codes   [P][D/2]                   low nibble first
 *   V codes   [P/8][16][8 tokens][D/32]  piece n of 16: channels n*D/16 .. of each token
 *   K scales  [P][D/32]                  a byte for each 32 channels
 *   V scales  [P/8][D/32][8 tokens]
 * A code is E2M1: bit 3 the sign, the rest indexes {0, .5, 1, 1.5, 2, 3, 4, 6}; it stands for
 * that times 2^(byte - 127).  The writer takes, for each 32 channels of a row,
 *   e = the least integer with max|x| <= 6 * 2^e, but within [-22, 13]; byte = e + 127;
 *   code = the nearest to x * 2^-e, ties to the even code, 6 above 6
 * (so magnitudes up to 6 * 2^13 are held with an error of at most 2^e, and beyond that they
 * saturate).  A group with a NaN or an infinity gets byte 255 and reads as NaN.  Bytes the
 * writer never makes: 192 and up read as NaN, the others give unspecified values.
 *
 * cf_kv4_append writes row t of k and v (tokens x kv_heads rows) to slot slots[t] = page *
 * page_size + place; a slot that is negative or behind the cache takes nothing (padding).
 * Two tokens with the same slot leave it with unspecified values.  cf_kv4_read reads the rows
 * of slots back into k and v (bf16, rounded, which is exact; or fp32): rows of slots that
 * are not in the cache become zero.
 *   cache: 16-byte aligned; slots: tokens int64, 8-byte aligned.
 */
int64_t cf_kv4_cache_bytes(int64_t pages, int page_size, int kv_heads, int head_dim);

int cf_kv4_append(int a_dtype, const cf_rows* k, const cf_rows* v, const int64_t* slots, int64_t tokens,
                  uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim, void* stream);

int cf_kv4_read(int a_dtype, const uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim,
                const int64_t* slots, int64_t tokens, const cf_rows* k, const cf_rows* v, void* stream);

/*
 * Attention of ragged queries over the cache.  Sequence b has kv_lens[b] keys, token j of
 * it in page table[b * table_width + j / page_size], and the query tokens q_starts[b] ..
 * q_starts[b+1] - 1 of the total_q rows of q.  Query head h reads K/V head
 * h / (q_heads / kv_heads).  Query i of a sequence with n queries and len keys sees key j
 *   CF_ATTN_CAUSAL not set:  j < len
 *   CF_ATTN_CAUSAL set:      j <= at, and with window > 0 also j > at - window,
 *                            at = len - n + i (the queries are the last tokens)
 *   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j),  lse = log sum_j p_j
 * A row that sees no key gives zeros, and lse = -infinity.  What lies in the cache behind a
 * sequence's last key does not matter, whatever its bytes; a NaN reaches only the rows that
 * see it.  A page outside the cache holds no keys.
 *   q, out: total_q x q_heads rows of a_dtype;  lse: total_q x q_heads fp32, or NULL;
 *   table: batch x table_width int32, or NULL: sequence b has the pages b * table_width and
 *     on (batch * table_width <= pages);
 *   kv_lens: batch int32; lengths are cut to [0, table_width * page_size];
 *   q_starts: batch + 1 int32, or NULL: total_q / batch queries each, without a rest.  Rows of
 *     out and lse that belong to no sequence stay as they are.
 *   max_q: the most query tokens of a sequence, a bound that the caller knows, at most total_q
 *     (0: total_q, or total_q / batch where q_starts is NULL).  It chooses the kernel and the
 *     workspace; the results are right for any lengths.  total_q = 0 is a valid call that does
 *     nothing, whatever the bound.
 *   workspace: cf_kv4_attention_workspace_bytes, 256-byte aligned; nothing in it has to be
 *     set before a call, and nothing is kept in it for the next.
 * 0 < scale <= 1e38; window >= 0, and 0 unless causal; q_heads a multiple of kv_heads, at most 65535;
 * total_q * q_heads <= 2^31 - 256, table_width * page_size < 2^31 - 256, 1 <= batch <= 2^24.
 * K and V enter the products exactly.  bf16: queries exactly, probabilities rounded to fp16, off
 * by at most 2^-11 of the largest of the 32 or 64 keys that are taken at once, down to 2^-60 of
 * the row's largest; fp32: queries and probabilities exactly.  Scores, sums and results are fp32 up to
 * the final rounding to a_dtype.  Results are deterministic for given lengths; a row's last
 * bits depend on the batch it is computed in, which is split into equal parts.
 */
enum { CF_ATTN_CAUSAL = 1 };

int cf_kv4_attention(int a_dtype, const cf_rows* q, int64_t total_q, int q_heads, const uint8_t* cache,
                     int64_t pages, int page_size, int kv_heads, int head_dim, int batch, const int32_t* table,
                     int table_width, const int32_t* kv_lens, const int32_t* q_starts, int64_t max_q, int flags,
                     int window, float scale, const cf_rows* out, float* lse, void* workspace, size_t ws_bytes,
                     void* stream);

/* Workspace bytes of cf_kv4_attention (0 for arguments outside the limits): max_q as there; where
 * that is 0, total_q with q_starts and total_q / batch without.  Never less for a larger max_q: a
 * workspace of one call's bytes serves every call with fewer queries. */
size_t cf_kv4_attention_workspace_bytes(int a_dtype, int64_t max_q, int q_heads, int kv_heads, int head_dim);

/*
 * The 8-bit K/V cache: pages, sizes and limits as the 4-bit one's, in a buffer of cf_kv8_cache_bytes bytes.  The
 * block of page p and head h starts at (p * kv_heads + h) * B, B = 2 * P * D + max(16, P / 8), and holds, in this order:
 *   K codes   [P][D]
 *   V codes   [P/8][D][8 tokens]
 *   K scales  [P/16]              a byte for each 16 tokens
 *   V scales  [P/16]
 * A code is E4M3: bit 7 the sign, four exponent bits of bias 7, three of the fraction; magnitudes up to 448, and 127
 * reads NaN.  It stands for that times 2^(byte - 127).
 *
 * cf_kv8_append takes the last tokens of sequences: of sequence b, which has kv_lens[b] tokens with them, rows
 * starts[b] .. starts[b+1] - 1 of k and v (tokens x kv_heads rows).  Token j of it lies in page table[b * table_width +
 * j / page_size], as for cf_kv4_attention, and with 15 others of that page in one block of a scale.  For each block that
 * gets tokens, and each head, for K and for V:
 *   e = the least integer with max|x| <= 448 * 2^e over the finite values that come, but within [-15, 7];
 *   where the block's first token is not among those that come: no less than the block's e before; if that grows, the
 *     codes before those that come are rounded again, from what they stand for, as below;
 *   byte = e + 127;  code = the nearest to x * 2^-e, ties to the even code, 448 above 448; 127 for NaN and infinities
 * So values are held with an error of at most 2^-4 of themselves or 2^(e - 10), e being their block's when they came, and
 * magnitudes beyond 448 * 2^7 saturate.  All that later calls raise a block's scale by costs values that it held at
 * most 2^(e - 9) more, e being the block's then: each raise rounds them again, with an error only where they fall among the
 * scale's smallest.
 * Places of a block behind the tokens that came hold nothing.  Rows with no place (kv_lens[b] is less than their number,
 * a page outside the cache, rows of no sequence) are not kept.  A kv_lens beyond the table's pages is cut to them, and the rows
 * then take their last places.  Sequences of a call must not share a page that gets tokens.
 *   k, v: tokens x kv_heads rows;  table, kv_lens, starts: as in cf_kv4_attention, the rows being the queries there;
 *   tokens <= 2^27, 1 <= batch <= 2^24, table_width * page_size < 2^31 - 256.
 * cf_kv8_read is as cf_kv4_read.
 */
int64_t cf_kv8_cache_bytes(int64_t pages, int page_size, int kv_heads, int head_dim);

int cf_kv8_append(int a_dtype, const cf_rows* k, const cf_rows* v, int64_t tokens, uint8_t* cache, int64_t pages,
                  int page_size, int kv_heads, int head_dim, int batch, const int32_t* table, int table_width,
                  const int32_t* kv_lens, const int32_t* starts, void* stream);

int cf_kv8_read(int a_dtype, const uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim,
                const int64_t* slots, int64_t tokens, const cf_rows* k, const cf_rows* v, void* stream);

/*
 * Attention of ragged queries over the 8-bit cache: arguments, results and limits are cf_kv4_attention's.
 * K and V enter the products exactly.  bf16: queries exactly, probabilities rounded, in calls of at most 32 rows (max_q
 * times the query heads of a K/V head) to fp16 as there, in others to bf16 (2^-8 of each); fp32: queries and
 * probabilities exactly.  A NaN of V reaches its channel in the rows that see it.
 */
int cf_kv8_attention(int a_dtype, const cf_rows* q, int64_t total_q, int q_heads, const uint8_t* cache,
                     int64_t pages, int page_size, int kv_heads, int head_dim, int batch, const int32_t* table,
                     int table_width, const int32_t* kv_lens, const int32_t* q_starts, int64_t max_q, int flags,
                     int window, float scale, const cf_rows* out, float* lse, void* workspace, size_t ws_bytes,
                     void* stream);

size_t cf_kv8_attention_workspace_bytes(int a_dtype, int64_t max_q, int q_heads, int kv_heads, int head_dim);

/*
 * Attention over whole prompts: keys and values are rows of heads, of packed sequences.  Sequence b has the query tokens
 * q_starts[b] .. q_starts[b+1] - 1 of the total_q rows of q and the keys k_starts[b] .. k_starts[b+1] - 1 of the total_k
 * rows of k and v.  Masks, out and lse are as for cf_kv4_attention, with len = the sequence's keys.
 *   q, out: total_q x q_heads rows of a_dtype;  k, v: total_k x kv_heads rows of a_dtype;
 *   q_starts, k_starts: batch + 1 int32, or NULL: total_q / batch queries, total_k / batch keys each, without a rest;
 *   max_q: the most query tokens of a sequence, as there;  lse: total_q x q_heads fp32, or NULL;
 *   workspace: cf_attention_workspace_bytes, 256-byte aligned, as there: calls that may run at once need one each.
 * Rows of out and lse that belong to no sequence stay as they are.  head_dim is 64 or 128;  total_k <= 2^31 - 256, and
 * token strides of k and v are at most 2^26 bytes;  the other limits are cf_kv4_attention's.  total_k = 0 is a call whose rows see no key.
 * bf16: queries, keys and values enter the products exactly, probabilities rounded to bf16, off by at most 2^-8 of
 * each.  fp32 (magnitudes up to 2^127): as six products of bf16 parts, off by at most 2^-24 of their factors.  Scores, sums and results are fp32
 * up to the final rounding to a_dtype.  Magnitudes of V up to 2^100.  An infinity or NaN of a key or value reaches only rows that see
 * it; a NaN gives NaN there, an infinity infinities or NaN, or, of a key, weight 0.  Deterministic as cf_kv4_attention.
 */
int cf_attention(int a_dtype, const cf_rows* q, int64_t total_q, int q_heads, const cf_rows* k, const cf_rows* v,
                 int64_t total_k, int kv_heads, int head_dim, int batch, const int32_t* q_starts,
                 const int32_t* k_starts, int64_t max_q, int flags, int window, float scale, const cf_rows* out,
                 float* lse, void* workspace, size_t ws_bytes, void* stream);

size_t cf_attention_workspace_bytes(int a_dtype, int64_t max_q, int q_heads, int kv_heads, int head_dim);

/*
 * Who holds which page of a cache.  `rows` sequences of up to `width` pages of page_size tokens: row r has lens[r] tokens
 * in pages table[r * width] .. ; refs[p] counts the entries that hold page p, and a page with 0 is free.  The same
 * three arrays serve every cache whose pages they number (4 or 8 bits, each layer's).  The calls below read `in` and write
 * `out`.  Resize and the forks take lens within [0, width * page_size] and write entries behind a row's last page as -1;
 * compact, which has no page size, looks at no length: it hands on lens, and every entry, under its page's new number.
 * Entries that are no page of the cache are handed on and counted nowhere.  refs not less than 0.
 *
 * cf_pages_resize: row r gets want[r] tokens (negative: it stays as it is).  First rows that shrink let go the pages they
 *   no longer need (all of them at 0 tokens); then those that grow, in the order of rows, take free pages in the order of
 *   their numbers.  A row whose pages, behind those of the rows before it, are not all there, or that wants more than
 *   width * page_size, stays as it is.  missing: how many those are.  A row was served exactly if its length is the one
 *   it wanted: one that was not has no places for what is to be appended to it, and cf_kv8_append with its length would
 *   write over its last tokens.  A length of 0 there leaves them as they are and keeps nothing of the new ones.
 * cf_pages_fork: row r becomes a copy of row parents[r] as it was (itself: it stays; outside [0, rows): it becomes empty).
 *   Whole pages are shared.  A last, partly filled page goes on with the parent itself, or else the first of the rows; every
 *   other row, in the order of rows, takes the first free page in its place, src[r] and dst[r] being the pages to copy, for
 *   cf_pages_copy (-1 both where there is nothing to copy).  Pages that no row keeps are let go before that.  A row that
 *   finds no free page ends with its last whole page.  missing: how many those are.
 *   Only rows with the same parent are told apart so.  Rows that have shrunk to inside a page that others hold still share
 *   it, and must not be appended to then: cf_pages_fork_own parts them.
 * cf_pages_fork_own: as cf_pages_fork, but every last, partly filled page is then one row's alone.  Of the rows that would end
 *   in a page, whoever their parents are, the first of those that are their own parent goes on with it, or else the first, or
 *   none where it is a whole page of some row; the others take free pages in its place as above.  With
 *   parents[r] = r it is the call behind a cf_pages_resize that may have shrunk rows so.
 * cf_pages_compact: the pages that are held are made the first ones: the k-th of those behind, page src[k], goes to the
 *   k-th free one before, dst[k], for cf_pages_copy; refs and every table entry follow.  count: how many; src and dst have
 *   pages / 2 places, the rest -1.
 *   out may be in, array by array, for resize and compact; the forks' table and lens must be other arrays.
 *   want, parents: rows int32;  src, dst: rows int32 (fork), pages / 2 (compact);  missing, count: one int32.
 *   workspace: cf_pages_workspace_bytes, 4-byte aligned.
 *   1 <= pages < 2^31, 1 <= rows <= 2^20, width >= 1, rows * width <= 2^30, width * page_size < 2^31 - 256, page_size >= 1.
 *   All arrays 4-byte aligned.
 *
 * cf_pages_copy: page src[i] to page dst[i], in each of `layers` caches that lie layer_stride bytes apart, for i < n and,
 *   where count is not NULL, i < *count.  Pairs of which one is no page, or both the same, copy nothing.  A page
 *   that is copied to must not be in another pair.
 *   page_bytes and layer_stride multiples of 16, layer_stride >= pages * page_bytes (with one layer it does not
 *   matter), data 16-byte aligned; 0 <= n <= 2^30, 1 <= layers <= 65535.
 */
typedef struct cf_pages {
    int32_t* refs;
    int32_t* table;
    int32_t* lens;
} cf_pages;

size_t cf_pages_workspace_bytes(int64_t pages, int rows);

int cf_pages_resize(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size,
                    const int32_t* want, int32_t* missing, void* workspace, size_t ws_bytes, void* stream);

int cf_pages_fork(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size,
                  const int32_t* parents, int32_t* src, int32_t* dst, int32_t* missing, void* workspace, size_t ws_bytes,
                  void* stream);

int cf_pages_fork_own(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size,
                      const int32_t* parents, int32_t* src, int32_t* dst, int32_t* missing, void* workspace, size_t ws_bytes,
                      void* stream);

int cf_pages_compact(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int32_t* src,
                     int32_t* dst, int32_t* count, void* workspace, size_t ws_bytes, void* stream);

int cf_pages_copy(void* data, int64_t pages, int64_t page_bytes, int layers, int64_t layer_stride, const int32_t* src,
                  const int32_t* dst, int64_t n, const int32_t* count, void* stream);

/* Workspace bytes cf_lowrank_compress needs (0 for arguments outside the limits). */
size_t cf_lowrank_workspace_bytes(int64_t m, int64_t n, int rank, int batch);

/* Bytes of packed codes for numel elements at `bits` per element (numel*bits/8),
 * or a negative status for invalid arguments. */
int64_t cf_codes_bytes(int64_t numel, int bits);

/* Human-readable name of a status code (static storage). */
const char* cf_strerror(int status);

/* ABI version of this header: 1. */
int cf_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CF_H */
