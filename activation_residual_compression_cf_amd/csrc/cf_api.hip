// cf_api.hip - the C ABI of libcf: argument validation and kernel launch.
//
// Every entry point validates all arguments before it enqueues anything, so a
// call that fails leaves every buffer untouched.  Validation order: unsupported
// mode (CF_E_ARG), NULL pointers, sizes, alignment, overlapping ranges, device.

#include <hip/hip_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "cf.h"
#include "cf_internal.h"

namespace cf {

uint64_t call_number() {
    static std::atomic<uint64_t> next{static_cast<uint64_t>(std::chrono::system_clock::now().time_since_epoch().count()) ^
                                      reinterpret_cast<uintptr_t>(&next)};
    // a mixing of all 64 bits that can be undone: different counts, different numbers
    uint64_t x = next.fetch_add(1, std::memory_order_relaxed);
    x ^= x >> 32, x *= 0x9e3779b97f4a7c15u;
    x ^= x >> 29, x *= 0xd1342543de82ef95u;
    x ^= x >> 32;
    return x == 0 ? 1 : x;  // 0: of the count 0
}

}  // namespace cf

namespace {

// Largest numel of one call.  The element-wise kernels launch up to one work-item per
// 4 elements (rounded up to whole workgroups), and a dispatch counts at most
// 2^32 - 1 work-items, so 2^33 keeps every grid well inside a dispatch (and every
// byte size far from overflow).
constexpr int64_t kMaxNumel = int64_t(1) << 33;

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

Range range_of(const void* p, int64_t bytes) {
    const auto lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + static_cast<uintptr_t>(bytes)};
}

bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Scales are read and written one float per group: 4-byte alignment suffices, and a
// tensor inside a slab starts its scales at a multiple of 4 bytes only.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Output range `out` must not overlap any other range in `all` (by index).
template <int N>
bool any_alias(const Range (&all)[N], const bool (&is_out)[N]) {
    for (int i = 0; i < N; ++i) {
        if (!is_out[i]) continue;
        for (int j = 0; j < N; ++j)
            if (j != i && all[j].hi > all[j].lo && overlap(all[i], all[j])) return true;
    }
    return false;
}

// Device check: the current device must be gfx950.  Cached per device id.
constexpr int kMaxDevices = 64;
std::once_flag g_dev_once[kMaxDevices];
bool g_dev_ok[kMaxDevices];

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return CF_E_DEVICE;
    std::call_once(g_dev_once[dev], [dev] {
        hipDeviceProp_t prop;
        g_dev_ok[dev] = hipGetDeviceProperties(&prop, dev) == hipSuccess &&
                        std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    });
    return g_dev_ok[dev] ? CF_OK : CF_E_DEVICE;
}

// Fixed scratch of cf_lowrank_compress_noalloc: one copy in every device's memory that
// the library's code object is loaded on, for the life of the process.  Host code must
// not use the array's name as an address (it names a host-side stand-in); it takes the
// device address from hipGetSymbolAddress, once per device, with that device current.
static __device__ __align__(256) unsigned char scratch[CF_NOALLOC_SCRATCH_BYTES];

std::once_flag g_scratch_once[kMaxDevices];
void* g_scratch_ptr[kMaxDevices];

// Device address of the current device's scratch, or nullptr when HIP refuses it.
void* scratch_for_current_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::call_once(g_scratch_once[dev], [dev] {
        void* ptr = nullptr;
        if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) == hipSuccess) g_scratch_ptr[dev] = ptr;
    });
    return g_scratch_ptr[dev];
}

int valid_numel(int64_t numel) {
    return (numel > 0 && numel % CF_GROUP == 0 && numel <= kMaxNumel) ? CF_OK : CF_E_SHAPE;
}

int64_t act_bytes(int a_dtype, int64_t numel) { return numel * (a_dtype == CF_BF16 ? 2 : 4); }

// Checks of cf_lowrank_compress, in the order of the file header: a workspace of
// `ws_bytes` at `workspace` (null for a buffer of the library's own, which then needs no
// NULL or overlap check), `too_small` the status when the call needs more than ws_bytes.
int check_lowrank_compress(int a_dtype, const void* a, float* ahat, float* err, int64_t m, int64_t n, int rank,
                           int iters, int factor_bits, int batch, float* q_state, void* u, float* u_scales,
                           void* v, float* v_scales, const void* workspace, size_t ws_bytes, int too_small) {
    if (a_dtype != CF_BF16 && a_dtype != CF_F32) return CF_E_ARG;
    if (factor_bits != 4 && factor_bits != 16 && factor_bits != 32) return CF_E_ARG;
    if (iters < 1 || iters > 64) return CF_E_ARG;
    if (!a || !ahat || !q_state || !u || !v || (!workspace && too_small == CF_E_WORKSPACE)) return CF_E_NULL;
    if (factor_bits == 4 && (!u_scales || !v_scales)) return CF_E_NULL;
    const size_t need = cf_lowrank_workspace_bytes(m, n, rank, batch);
    if (need == 0 || (factor_bits == 4 && (rank & 1))) return CF_E_SHAPE;
    if (!aligned16(a) || !aligned16(ahat) || (err && !aligned16(err)) || !aligned4(q_state) ||
        !aligned4(u) || !aligned4(v) || (u_scales && !aligned4(u_scales)) ||
        (v_scales && !aligned4(v_scales)) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return CF_E_ALIGN;
    if (ws_bytes < need) return too_small;
    const int64_t numel = m * n * batch;
    const int64_t fsz = factor_bits / 4;  // factor bytes per (row, rank) pair, times 2
    const Range r[8] = {range_of(a, act_bytes(a_dtype, numel)),
                        range_of(ahat, numel * 4),
                        range_of(err, err ? numel * 4 : 0),
                        range_of(q_state, int64_t(batch) * n * rank * 4),
                        range_of(u, int64_t(batch) * m * rank * fsz / 2),
                        range_of(v, int64_t(batch) * n * rank * fsz / 2),
                        range_of(u_scales, factor_bits == 4 ? int64_t(batch) * rank * 4 : 0),
                        range_of(v_scales, factor_bits == 4 ? int64_t(batch) * rank * 4 : 0)};
    const bool out[8] = {false, true, err != nullptr, true, true, true, factor_bits == 4, factor_bits == 4};
    if (any_alias(r, out)) return CF_E_ALIAS;
    if (workspace) {
        const Range wsr = range_of(workspace, static_cast<int64_t>(need));
        for (const Range& x : r)
            if (x.hi > x.lo && overlap(x, wsr)) return CF_E_ALIAS;
    }
    return CF_OK;
}

// ---- rows of heads -------------------------------------------------------------------

typedef __int128 wide;  // extents of rows are formed before they are known to be small

// Rows of a cf_rows: tokens x heads rows of dim elements of esz bytes.
struct RowsOf {
    cf_rows r;
    int64_t tokens, heads, dim, esz;
    bool none() const { return tokens == 0 || heads == 0; }
    wide extent() const {  // elements from the first row's start to the last row's end
        return wide(tokens - 1) * r.token_stride + wide(heads - 1) * r.head_stride + dim;
    }
    Range range() const { return range_of(r.data, none() ? 0 : static_cast<int64_t>(extent() * esz)); }
};

// Rows of one call: a row takes at least 8 work-items, of which a dispatch counts 2^32 - 1.
constexpr int64_t kMaxRows = int64_t(1) << 28;
constexpr wide kMaxExtent = wide(1) << 46;  // bytes: beyond any device's memory
// Sequences of one attention call: every workgroup counts through them, 64 at a time and in 32 bits.
constexpr int kMaxSequences = 1 << 24;
// Query tokens times query heads of one: a tile of up to 256 rows behind the last still counts in 32 bits.
constexpr int64_t kMaxAttnRows = (int64_t(1) << 31) - 256;
// Tokens that cf_kv8_append takes at once: a wave for each in a dispatch of 2^32 - 1 work-items, and head by head.
constexpr int64_t kMaxAppend = int64_t(1) << 27;
// Bytes between the keys of cf_attention: 63 of them in 32 bits.
constexpr int64_t kMaxKeyStride = int64_t(1) << 26;

// NULL, strides, alignment of one operand's rows, in this order.
int check_rows(const cf_rows* r, int64_t tokens, int64_t heads, int64_t dim, int64_t esz, bool written, RowsOf* x) {
    *x = RowsOf{r ? *r : cf_rows{nullptr, 0, 0}, tokens, heads, dim, esz};
    if (x->none()) return CF_OK;
    if (!r || !r->data) return CF_E_NULL;
    if (tokens == 1) x->r.token_stride = 0;  // strides that nothing is multiplied with do not matter
    if (heads == 1) x->r.head_stride = 0;
    const int64_t ts = x->r.token_stride, hs = x->r.head_stride;
    if (ts < 0 || hs < 0 || x->extent() * esz > kMaxExtent) return CF_E_SHAPE;
    if (written) {
        const bool by_token = (heads == 1 || hs >= dim) && (tokens == 1 || ts >= wide(heads - 1) * hs + dim);
        const bool by_head = (tokens == 1 || ts >= dim) && (heads == 1 || hs >= wide(tokens - 1) * ts + dim);
        if (!by_token && !by_head) return CF_E_SHAPE;
    }
    if (!aligned16(r->data) || ts * esz % 16 || hs * esz % 16) return CF_E_ALIGN;
    return CF_OK;
}

// Whether two sets of rows surely share no byte: their ranges are apart, or they are two
// slices of the heads of one packed token-major buffer.
bool apart(const RowsOf& a, const RowsOf& b) {
    if (a.none() || b.none() || !overlap(a.range(), b.range())) return true;
    const int64_t ts = a.r.token_stride;
    if (a.esz != b.esz || ts != b.r.token_stride || ts <= 0) return false;
    const wide wa = wide(a.heads - 1) * a.r.head_stride + a.dim, wb = wide(b.heads - 1) * b.r.head_stride + b.dim;
    if (wa > ts || wb > ts) return false;
    const wide bytes = wide(reinterpret_cast<uintptr_t>(b.r.data)) - wide(reinterpret_cast<uintptr_t>(a.r.data));
    const wide period = wide(ts) * a.esz;
    wide d = bytes % period;
    if (d < 0) d += period;
    return d >= wa * a.esz && d + wb * b.esz <= period;
}

bool same_rows(const RowsOf& a, const RowsOf& b) {
    return a.r.data == b.r.data && a.tokens == b.tokens && a.heads == b.heads && a.esz == b.esz &&
           a.r.token_stride == b.r.token_stride && a.r.head_stride == b.r.head_stride;
}

int64_t elem_bytes(int a_dtype) { return a_dtype == CF_BF16 ? 2 : 4; }

// ---- the 4-bit cache -----------------------------------------------------------------

bool kv4_dims(int page_size, int kv_heads, int head_dim) {
    return (head_dim == 64 || head_dim == 128) && page_size >= 16 && page_size <= 256 &&
           (page_size & (page_size - 1)) == 0 && kv_heads >= 1 && kv_heads <= 65535;
}

cf::KvCache kv4_cache(const uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim) {
    return {const_cast<uint8_t*>(cache), pages, kv_heads, {page_size, head_dim}, __builtin_ctz(page_size)};
}

cf::Kv8Cache kv8_cache(const uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim) {
    return {const_cast<uint8_t*>(cache), pages, kv_heads, {page_size, head_dim}, __builtin_ctz(page_size)};
}

// cf_kv4_append, and the readers, whose rows are written: f is the launch for a checked call.
template <typename F>
int slot_rows(bool read, int a_dtype, const cf_rows* k, const cf_rows* v, const int64_t* slots, int64_t tokens,
              const uint8_t* cache, int64_t bytes, int kv_heads, int head_dim, F f) {
    if (a_dtype != CF_BF16 && a_dtype != CF_F32) return CF_E_ARG;
    if (bytes < 0) return CF_E_SHAPE;
    if (tokens < 0 || tokens > kMaxNumel / head_dim / kv_heads) return CF_E_SHAPE;
    if (tokens == 0) return CF_OK;
    if (!cache || !slots) return CF_E_NULL;
    RowsOf x[2];
    if (int rc = check_rows(k, tokens, kv_heads, head_dim, elem_bytes(a_dtype), read, &x[0])) return rc;
    if (int rc = check_rows(v, tokens, kv_heads, head_dim, elem_bytes(a_dtype), read, &x[1])) return rc;
    if (!aligned16(cache) || (reinterpret_cast<uintptr_t>(slots) & 7u)) return CF_E_ALIGN;
    const Range rc = range_of(cache, bytes), rs = range_of(slots, tokens * 8);
    if (read ? !apart(x[0], x[1]) || overlap(x[0].range(), rs) || overlap(x[1].range(), rs) : overlap(rc, rs))
        return CF_E_ALIAS;
    if (overlap(x[0].range(), rc) || overlap(x[1].range(), rc)) return CF_E_ALIAS;
    if (int e = check_device()) return e;
    return f(x[0].r, x[1].r) == hipSuccess ? CF_OK : CF_E_HIP;
}

// Attention over a paged cache, of `cache_bytes` bytes; f is the launch for a checked call.
template <typename F>
int paged_attention(int a_dtype, const cf_rows* q, int64_t total_q, int q_heads, const uint8_t* cache, int64_t cache_bytes,
                    int64_t pages, int page_size, int kv_heads, int head_dim, int batch, const int32_t* table,
                    int table_width, const int32_t* kv_lens, const int32_t* q_starts, int64_t max_q, int flags,
                    int window, float scale, const cf_rows* out, float* lse, void* workspace, size_t ws_bytes,
                    size_t (*workspace_bytes)(int, int64_t, int, int, int), F f) {
    if (a_dtype != CF_BF16 && a_dtype != CF_F32) return CF_E_ARG;
    if ((flags & ~CF_ATTN_CAUSAL) || window < 0 || (window && !(flags & CF_ATTN_CAUSAL))) return CF_E_ARG;
    if (!(scale > 0.f) || scale > 1e38f) return CF_E_ARG;
    if (cache_bytes < 0) return CF_E_SHAPE;
    if (q_heads < 1 || q_heads > 65535 || q_heads % kv_heads || total_q < 0 || total_q > kMaxAttnRows / q_heads ||
        max_q < 0)
        return CF_E_SHAPE;
    if (total_q == 0) return CF_OK;
    if (max_q > total_q) return CF_E_SHAPE;
    if (batch < 1 || batch > kMaxSequences || table_width < 1 || int64_t(table_width) * page_size > INT32_MAX - 256 ||
        (!table && int64_t(batch) * table_width > pages) || (!q_starts && total_q % batch))
        return CF_E_SHAPE;
    if (!cache || !kv_lens || !workspace) return CF_E_NULL;
    const int64_t esz = elem_bytes(a_dtype);
    RowsOf x[2];
    if (int rc = check_rows(q, total_q, q_heads, head_dim, esz, false, &x[0])) return rc;
    if (int rc = check_rows(out, total_q, q_heads, head_dim, esz, true, &x[1])) return rc;
    if (!aligned16(cache) || !aligned4(table) || !aligned4(kv_lens) || !aligned4(q_starts) || !aligned4(lse) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return CF_E_ALIGN;
    if (max_q == 0) max_q = q_starts ? total_q : total_q / batch;
    const size_t need = workspace_bytes(a_dtype, max_q, q_heads, kv_heads, head_dim);
    if (ws_bytes < need) return CF_E_WORKSPACE;
    if (!apart(x[0], x[1])) return CF_E_ALIAS;
    const Range r[8] = {x[0].range(),
                        range_of(cache, cache_bytes),
                        range_of(table, table ? int64_t(batch) * table_width * 4 : 0),
                        range_of(kv_lens, int64_t(batch) * 4),
                        range_of(q_starts, q_starts ? (int64_t(batch) + 1) * 4 : 0),
                        x[1].range(),
                        range_of(lse, lse ? total_q * q_heads * 4 : 0),
                        range_of(workspace, static_cast<int64_t>(need))};
    for (int i = 5; i < 8; ++i)
        for (int j = i == 5 ? 1 : 0; j < i; ++j)  // q and out were looked at row by row
            if (r[i].hi > r[i].lo && r[j].hi > r[j].lo && overlap(r[i], r[j])) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return f(x[0].r, x[1].r, max_q) == hipSuccess ? CF_OK : CF_E_HIP;
}

// Heads and rows that an attention call's workspace is asked for.
bool attention_dims(int a_dtype, int64_t max_q, int q_heads, int kv_heads, int head_dim) {
    return (a_dtype == CF_BF16 || a_dtype == CF_F32) && kv4_dims(16, kv_heads, head_dim) && q_heads >= 1 &&
           q_heads <= 65535 && q_heads % kv_heads == 0 && max_q >= 1 && max_q <= kMaxAttnRows / q_heads;
}

// ---- pages

constexpr int kMaxPageRows = 1 << 20;

// The three arrays of a call's sequences, in and out, and up to four others of its own: reads, then writes.
int check_pages(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size, bool in_place,
                const void* want, const int32_t* const (&written)[3], const int64_t (&places)[3], const void* workspace,
                size_t ws_bytes) {
    if (pages < 1 || pages > INT32_MAX || rows < 1 || rows > kMaxPageRows || width < 1 || int64_t(rows) * width > (1 << 30) ||
        page_size < 1 || int64_t(width) * page_size > INT32_MAX - 256)
        return CF_E_SHAPE;
    if (!in || !out || !in->refs || !in->table || !in->lens || !out->refs || !out->table || !out->lens || !workspace)
        return CF_E_NULL;
    for (int i = 0; i < 3; ++i)
        if (!written[i] && places[i] > 0) return CF_E_NULL;
    const int64_t entries = int64_t(rows) * width;
    const size_t need = cf_pages_workspace_bytes(pages, rows);
    const Range r[11] = {range_of(in->refs, pages * 4),   range_of(in->table, entries * 4),
                         range_of(in->lens, int64_t(rows) * 4), range_of(want, want ? int64_t(rows) * 4 : 0),
                         range_of(out->refs, pages * 4),  range_of(out->table, entries * 4),
                         range_of(out->lens, int64_t(rows) * 4), range_of(written[0], places[0] * 4),
                         range_of(written[1], places[1] * 4), range_of(written[2], places[2] * 4),
                         range_of(workspace, static_cast<int64_t>(need))};
    for (const Range& x : r)
        if (x.lo & 3u) return CF_E_ALIGN;
    if (ws_bytes < need) return CF_E_WORKSPACE;
    for (int i = 4; i < 11; ++i)
        for (int j = 0; j < i; ++j) {
            if (r[i].hi <= r[i].lo || r[j].hi <= r[j].lo || !overlap(r[i], r[j])) continue;
            if (j == i - 4 && i < 7 && r[i].lo == r[j].lo && (in_place || i == 4)) continue;
            return CF_E_ALIAS;
        }
    return CF_OK;
}

int pages_fork(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size,
               const int32_t* parents, int32_t* src, int32_t* dst, int32_t* missing, bool own, void* workspace,
               size_t ws_bytes, void* stream) {
    if (int rc = check_pages(in, out, pages, rows, width, page_size, false, parents, {src, dst, missing}, {rows, rows, 1}, workspace, ws_bytes))
        return rc;
    if (!parents) return CF_E_NULL;
    if (int rc = check_device()) return rc;
    const cf::PagesCall call{*in, *out, pages, rows, width, page_size, parents, src, dst, missing};
    return cf::launch_pages_fork(call, own, workspace, static_cast<hipStream_t>(stream)) == hipSuccess ? CF_OK : CF_E_HIP;
}

}  // namespace

extern "C" {

int cf_abi_version(void) { return 1; }

const char* cf_strerror(int status) {
    switch (status) {
        case CF_OK: return "ok";
        case CF_E_NULL: return "required pointer is NULL";
        case CF_E_SHAPE: return "size, stride or head count out of range (numel of the 1/2-bit and top-k calls: a positive "
                                "multiple of 128, at most 2^33)";
        case CF_E_ALIGN: return "pointer misaligned (16 bytes; scales 4 bytes)";
        case CF_E_ARG: return "unsupported bits, k, dtype, mode, flag or scale";
        case CF_E_ALIAS: return "output range overlaps another operand";
        case CF_E_WORKSPACE: return "workspace missing or too small";
        case CF_E_DEVICE: return "current device is not gfx950";
        case CF_E_HIP: return "HIP runtime refused the launch";
        case CF_E_SCRATCH:
            return "call needs more scratch than cf_lowrank_compress_noalloc's fixed buffer "
                   "(CF_NOALLOC_SCRATCH_BYTES) holds; pass fewer tensors per call";
        default: return "unknown status";
    }
}

int64_t cf_codes_bytes(int64_t numel, int bits) {
    if (bits != 1 && bits != 2) return CF_E_ARG;
    if (valid_numel(numel) != CF_OK) return CF_E_SHAPE;
    return numel * bits / 8;
}

int cf_init_state(int a_dtype, const void* a, float* ahat, float* err, int64_t numel, void* stream) {
    if (a_dtype != CF_BF16 && a_dtype != CF_F32) return CF_E_ARG;
    if (!a || !ahat) return CF_E_NULL;
    if (int rc = valid_numel(numel)) return rc;
    if (!aligned16(a) || !aligned16(ahat) || (err && !aligned16(err))) return CF_E_ALIGN;
    const Range r[3] = {range_of(a, act_bytes(a_dtype, numel)), range_of(ahat, numel * 4),
                        range_of(err, err ? numel * 4 : 0)};
    const bool out[3] = {false, true, err != nullptr};
    if (any_alias(r, out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_init(a_dtype, a, ahat, err, numel, static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_compress(int bits, int a_dtype, const void* a, float* ahat, float* err, uint8_t* codes,
                float* scales, int64_t numel, void* stream) {
    if ((bits != 1 && bits != 2) || (a_dtype != CF_BF16 && a_dtype != CF_F32)) return CF_E_ARG;
    if (!a || !ahat || !codes || !scales) return CF_E_NULL;
    if (int rc = valid_numel(numel)) return rc;
    if (!aligned16(a) || !aligned16(ahat) || (err && !aligned16(err)) || !aligned16(codes) ||
        !aligned4(scales))
        return CF_E_ALIGN;
    const Range r[5] = {range_of(a, act_bytes(a_dtype, numel)), range_of(ahat, numel * 4),
                        range_of(err, err ? numel * 4 : 0), range_of(codes, numel * bits / 8),
                        range_of(scales, numel / CF_GROUP * 4)};
    const bool out[5] = {false, true, err != nullptr, true, true};
    if (any_alias(r, out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_compress(bits, a_dtype, a, ahat, err, codes, scales, numel,
                               static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_decompress(int bits, const uint8_t* codes, const float* scales, float* ahat, int64_t numel,
                  void* stream) {
    if (bits != 1 && bits != 2) return CF_E_ARG;
    if (!codes || !scales || !ahat) return CF_E_NULL;
    if (int rc = valid_numel(numel)) return rc;
    if (!aligned16(codes) || !aligned4(scales) || !aligned16(ahat)) return CF_E_ALIGN;
    const Range r[3] = {range_of(codes, numel * bits / 8), range_of(scales, numel / CF_GROUP * 4),
                        range_of(ahat, numel * 4)};
    const bool out[3] = {false, false, true};
    if (any_alias(r, out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_decompress(bits, codes, scales, ahat, nullptr, numel, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_decompress_bf16(int bits, const uint8_t* codes, const float* scales, float* ahat, uint16_t* out,
                       int64_t numel, void* stream) {
    if (bits != 1 && bits != 2) return CF_E_ARG;
    if (!codes || !scales || !ahat || !out) return CF_E_NULL;
    if (int rc = valid_numel(numel)) return rc;
    if (!aligned16(codes) || !aligned4(scales) || !aligned16(ahat) || !aligned16(out)) return CF_E_ALIGN;
    const Range r[4] = {range_of(codes, numel * bits / 8), range_of(scales, numel / CF_GROUP * 4),
                        range_of(ahat, numel * 4), range_of(out, numel * 2)};
    const bool is_out[4] = {false, false, true, true};
    if (any_alias(r, is_out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_decompress(bits, codes, scales, ahat, out, numel, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_compress_ablation(int mode, int bits, int a_dtype, const void* a, const void* a_prev, float* ahat,
                         uint8_t* codes, float* scales, int64_t numel, void* stream) {
    if ((mode != CF_MODE_NOEF && mode != CF_MODE_NAIVE) || (bits != 1 && bits != 2) ||
        (a_dtype != CF_BF16 && a_dtype != CF_F32))
        return CF_E_ARG;
    if (!a || !ahat || !codes || !scales || (mode == CF_MODE_NOEF && !a_prev)) return CF_E_NULL;
    if (int rc = valid_numel(numel)) return rc;
    if (!aligned16(a) || (a_prev && !aligned16(a_prev)) || !aligned16(ahat) || !aligned16(codes) ||
        !aligned4(scales))
        return CF_E_ALIGN;
    const Range r[5] = {range_of(a, act_bytes(a_dtype, numel)),
                        range_of(a_prev, mode == CF_MODE_NOEF ? act_bytes(a_dtype, numel) : 0),
                        range_of(ahat, numel * 4), range_of(codes, numel * bits / 8),
                        range_of(scales, numel / CF_GROUP * 4)};
    const bool is_out[5] = {false, false, true, true, true};
    if (any_alias(r, is_out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_compress_ablation(mode, bits, a_dtype, a, a_prev, ahat, codes, scales, numel,
                                        static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_topk_compress(int k, int a_dtype, const void* a, float* ahat, float* err, uint8_t* idx, uint16_t* vals,
                     int64_t numel, void* stream) {
    if (k < 1 || k > CF_GROUP || (a_dtype != CF_BF16 && a_dtype != CF_F32)) return CF_E_ARG;
    if (!a || !ahat || !idx || !vals) return CF_E_NULL;
    if (int rc = valid_numel(numel)) return rc;
    if (!aligned16(a) || !aligned16(ahat) || (err && !aligned16(err)) ||
        (reinterpret_cast<uintptr_t>(vals) & 1u))
        return CF_E_ALIGN;
    const int64_t slots = numel / CF_GROUP * k;
    const Range r[5] = {range_of(a, act_bytes(a_dtype, numel)), range_of(ahat, numel * 4),
                        range_of(err, err ? numel * 4 : 0), range_of(idx, slots), range_of(vals, slots * 2)};
    const bool out[5] = {false, true, err != nullptr, true, true};
    if (any_alias(r, out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_topk_compress(k, a_dtype, a, ahat, err, idx, vals, numel,
                                    static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_topk_decompress(int k, const uint8_t* idx, const uint16_t* vals, float* ahat, int64_t numel,
                       void* stream) {
    if (k < 1 || k > CF_GROUP) return CF_E_ARG;
    if (!idx || !vals || !ahat) return CF_E_NULL;
    if (int rc = valid_numel(numel)) return rc;
    if (!aligned16(ahat) || (reinterpret_cast<uintptr_t>(vals) & 1u)) return CF_E_ALIGN;
    const int64_t slots = numel / CF_GROUP * k;
    const Range r[3] = {range_of(idx, slots), range_of(vals, slots * 2), range_of(ahat, numel * 4)};
    const bool out[3] = {false, false, true};
    if (any_alias(r, out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_topk_decompress(k, idx, vals, ahat, numel, static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

size_t cf_lowrank_workspace_bytes(int64_t m, int64_t n, int rank, int batch) {
    if (m <= 0 || n <= 0 || m % 16 || n % 16 || batch < 1 || rank < 1 || rank > cf::kMaxRank ||
        rank > m || rank > n || m > kMaxNumel / n || m * n > kMaxNumel / batch ||
        !cf::lowrank_launches_fit(m, n, rank, batch))
        return 0;
    return cf::lowrank_workspace_total(m, n, rank, batch);
}

int cf_lowrank_compress(int a_dtype, const void* a, float* ahat, float* err, int64_t m, int64_t n,
                        int rank, int iters, int factor_bits, int batch, float* q_state, void* u,
                        float* u_scales, void* v, float* v_scales, void* workspace, size_t ws_bytes,
                        void* stream) {
    if (int rc = check_lowrank_compress(a_dtype, a, ahat, err, m, n, rank, iters, factor_bits, batch, q_state, u,
                                        u_scales, v, v_scales, workspace, ws_bytes, CF_E_WORKSPACE))
        return rc;
    if (int rc = check_device()) return rc;
    return cf::launch_lowrank_compress(a_dtype, a, ahat, err, m, n, rank, iters, factor_bits, batch,
                                       q_state, u, u_scales, v, v_scales, workspace,
                                       static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_lowrank_compress_noalloc(int a_dtype, const void* a, float* ahat, float* err, int64_t m, int64_t n,
                                int rank, int iters, int factor_bits, int batch, float* q_state, void* u,
                                float* u_scales, void* v, float* v_scales, void* stream) {
    if (int rc = check_lowrank_compress(a_dtype, a, ahat, err, m, n, rank, iters, factor_bits, batch, q_state, u,
                                        u_scales, v, v_scales, nullptr, CF_NOALLOC_SCRATCH_BYTES, CF_E_SCRATCH))
        return rc;
    if (int rc = check_device()) return rc;
    void* ws = scratch_for_current_device();
    if (!ws) return CF_E_HIP;
    return cf::launch_lowrank_compress(a_dtype, a, ahat, err, m, n, rank, iters, factor_bits, batch, q_state,
                                       u, u_scales, v, v_scales, ws, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_lowrank_decompress(int factor_bits, const void* u, const float* u_scales, const void* v,
                          const float* v_scales, float* ahat, int64_t m, int64_t n, int rank,
                          int batch, void* stream) {
    if (factor_bits != 4 && factor_bits != 16 && factor_bits != 32) return CF_E_ARG;
    if (!u || !v || !ahat) return CF_E_NULL;
    if (factor_bits == 4 && (!u_scales || !v_scales)) return CF_E_NULL;
    if (cf_lowrank_workspace_bytes(m, n, rank, batch) == 0 || (factor_bits == 4 && (rank & 1)))
        return CF_E_SHAPE;
    if (!aligned16(ahat) || !aligned4(u) || !aligned4(v) || (u_scales && !aligned4(u_scales)) ||
        (v_scales && !aligned4(v_scales)))
        return CF_E_ALIGN;
    const int64_t numel = m * n * batch;
    const int64_t fsz = factor_bits / 4;
    const Range r[5] = {range_of(ahat, numel * 4),
                        range_of(u, int64_t(batch) * m * rank * fsz / 2),
                        range_of(v, int64_t(batch) * n * rank * fsz / 2),
                        range_of(u_scales, factor_bits == 4 ? int64_t(batch) * rank * 4 : 0),
                        range_of(v_scales, factor_bits == 4 ? int64_t(batch) * rank * 4 : 0)};
    const bool out[5] = {true, false, false, false, false};
    if (any_alias(r, out)) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_lowrank_decompress(factor_bits, u, u_scales, v, v_scales, ahat, m, n, rank, batch,
                                         static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_qk_norm_rope(int a_dtype, int64_t tokens, int q_heads, int k_heads, int head_dim, const cf_rows* q,
                    const cf_rows* k, const cf_rows* q_out, const cf_rows* k_out, int norm,
                    const float* q_weight, const float* q_bias, const float* k_weight, const float* k_bias,
                    float eps, int rope, const float* cos, const float* sin, int64_t n_pos, int rot_dim,
                    const int32_t* positions, void* stream) {
    if (a_dtype != CF_BF16 && a_dtype != CF_F32) return CF_E_ARG;
    if (norm < CF_NORM_NONE || norm > CF_NORM_LAYER || rope < CF_ROPE_NONE || rope > CF_ROPE_HALF) return CF_E_ARG;
    if (!(eps >= 0.f) || eps > 3.4e38f) return CF_E_ARG;
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || q_heads > 65535 || k_heads > 65535 || head_dim <= 0 ||
        head_dim % 8 || head_dim > 256)
        return CF_E_SHAPE;
    const int64_t heads = int64_t(q_heads) + k_heads;
    if (heads == 0 || tokens > kMaxNumel / head_dim / heads || tokens > kMaxRows / heads) return CF_E_SHAPE;
    const bool turn = rope != CF_ROPE_NONE;
    if (turn && (rot_dim <= 0 || rot_dim % 16 || rot_dim > head_dim || n_pos <= 0 || n_pos > kMaxNumel / rot_dim ||
                 (!positions && tokens > n_pos)))
        return CF_E_SHAPE;
    if (tokens == 0) return CF_OK;
    if (turn && (!cos || !sin)) return CF_E_NULL;
    const int64_t esz = elem_bytes(a_dtype);
    RowsOf x[4];
    if (int rc = check_rows(q, tokens, q_heads, head_dim, esz, false, &x[0])) return rc;
    if (int rc = check_rows(k, tokens, k_heads, head_dim, esz, false, &x[1])) return rc;
    if (int rc = check_rows(q_out, tokens, q_heads, head_dim, esz, true, &x[2])) return rc;
    if (int rc = check_rows(k_out, tokens, k_heads, head_dim, esz, true, &x[3])) return rc;
    const float* const par[4] = {q_heads ? q_weight : nullptr, q_heads ? q_bias : nullptr,
                                 k_heads ? k_weight : nullptr, k_heads ? k_bias : nullptr};
    for (const float* w : par)
        if (!aligned16(w)) return CF_E_ALIGN;
    if (turn && (!aligned16(cos) || !aligned16(sin) || !aligned4(positions))) return CF_E_ALIGN;
    if ((!same_rows(x[0], x[2]) && !apart(x[0], x[2])) || (!same_rows(x[1], x[3]) && !apart(x[1], x[3])) ||
        !apart(x[0], x[3]) || !apart(x[1], x[2]) || !apart(x[2], x[3]))
        return CF_E_ALIAS;
    const int64_t table = turn ? n_pos * (rot_dim / 2) * 4 : 0;
    const Range read[7] = {range_of(par[0], par[0] ? head_dim * 4 : 0), range_of(par[1], par[1] ? head_dim * 4 : 0),
                           range_of(par[2], par[2] ? head_dim * 4 : 0), range_of(par[3], par[3] ? head_dim * 4 : 0),
                           range_of(cos, table), range_of(sin, table),
                           range_of(positions, turn && positions ? tokens * 4 : 0)};
    for (const Range& r : read)
        for (const RowsOf* o : {&x[2], &x[3]})
            if (r.hi > r.lo && !o->none() && overlap(r, o->range())) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_qk_norm_rope(a_dtype, tokens, q_heads, k_heads, head_dim, x[0].r, x[1].r, x[2].r, x[3].r, norm,
                                   par[0], par[1], par[2], par[3], eps, rope, cos, sin, n_pos, rot_dim, positions,
                                   static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int64_t cf_kv4_cache_bytes(int64_t pages, int page_size, int kv_heads, int head_dim) {
    if (!kv4_dims(page_size, kv_heads, head_dim) || pages < 1 || pages > INT32_MAX) return CF_E_SHAPE;
    const wide bytes = wide(pages) * kv_heads * page_size * head_dim * 17 / 16;
    return bytes <= kMaxExtent ? static_cast<int64_t>(bytes) : CF_E_SHAPE;
}

int cf_kv4_append(int a_dtype, const cf_rows* k, const cf_rows* v, const int64_t* slots, int64_t tokens,
                  uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim, void* stream) {
    return slot_rows(false, a_dtype, k, v, slots, tokens, cache, cf_kv4_cache_bytes(pages, page_size, kv_heads, head_dim),
                     kv_heads, head_dim, [&](const cf_rows& kr, const cf_rows& vr) {
                         return cf::launch_kv4_append(a_dtype, kr, vr, slots, tokens,
                                                      kv4_cache(cache, pages, page_size, kv_heads, head_dim),
                                                      static_cast<hipStream_t>(stream));
                     });
}

int cf_kv4_read(int a_dtype, const uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim,
                const int64_t* slots, int64_t tokens, const cf_rows* k, const cf_rows* v, void* stream) {
    return slot_rows(true, a_dtype, k, v, slots, tokens, cache, cf_kv4_cache_bytes(pages, page_size, kv_heads, head_dim),
                     kv_heads, head_dim, [&](const cf_rows& kr, const cf_rows& vr) {
                         return cf::launch_kv4_read(a_dtype, kr, vr, slots, tokens,
                                                    kv4_cache(cache, pages, page_size, kv_heads, head_dim),
                                                    static_cast<hipStream_t>(stream));
                     });
}

size_t cf_kv4_attention_workspace_bytes(int a_dtype, int64_t max_q, int q_heads, int kv_heads, int head_dim) {
    return attention_dims(a_dtype, max_q, q_heads, kv_heads, head_dim)
               ? cf::kv4_attention_workspace(a_dtype, head_dim, max_q * (q_heads / kv_heads))
               : 0;
}

int cf_kv4_attention(int a_dtype, const cf_rows* q, int64_t total_q, int q_heads, const uint8_t* cache,
                     int64_t pages, int page_size, int kv_heads, int head_dim, int batch, const int32_t* table,
                     int table_width, const int32_t* kv_lens, const int32_t* q_starts, int64_t max_q, int flags,
                     int window, float scale, const cf_rows* out, float* lse, void* workspace, size_t ws_bytes,
                     void* stream) {
    return paged_attention(a_dtype, q, total_q, q_heads, cache, cf_kv4_cache_bytes(pages, page_size, kv_heads, head_dim), pages,
                           page_size, kv_heads, head_dim, batch, table, table_width, kv_lens, q_starts, max_q, flags,
                           window, scale, out, lse, workspace, ws_bytes, cf_kv4_attention_workspace_bytes,
                           [&](const cf_rows& qr, const cf_rows& outr, int64_t most) {
                               const cf::Kv4Attention call{qr,     outr,  kv4_cache(cache, pages, page_size, kv_heads, head_dim),
                                                           table,  kv_lens, q_starts, lse, total_q, most, batch, table_width, q_heads,
                                                           flags & CF_ATTN_CAUSAL, window, scale};
                               return cf::launch_kv4_attention(a_dtype, call, workspace, static_cast<hipStream_t>(stream));
                           });
}

int64_t cf_kv8_cache_bytes(int64_t pages, int page_size, int kv_heads, int head_dim) {
    if (!kv4_dims(page_size, kv_heads, head_dim) || pages < 1 || pages > INT32_MAX) return CF_E_SHAPE;
    const wide bytes = wide(pages) * kv_heads * cf::Kv8Block{page_size, head_dim}.bytes();
    return bytes <= kMaxExtent ? static_cast<int64_t>(bytes) : CF_E_SHAPE;
}

int cf_kv8_append(int a_dtype, const cf_rows* k, const cf_rows* v, int64_t tokens, uint8_t* cache, int64_t pages,
                  int page_size, int kv_heads, int head_dim, int batch, const int32_t* table, int table_width,
                  const int32_t* kv_lens, const int32_t* starts, void* stream) {
    if (a_dtype != CF_BF16 && a_dtype != CF_F32) return CF_E_ARG;
    const int64_t bytes = cf_kv8_cache_bytes(pages, page_size, kv_heads, head_dim);
    if (bytes < 0) return CF_E_SHAPE;
    if (tokens < 0 || tokens > kMaxAppend || tokens > kMaxNumel / head_dim / kv_heads) return CF_E_SHAPE;
    if (tokens == 0) return CF_OK;
    if (batch < 1 || batch > kMaxSequences || table_width < 1 || int64_t(table_width) * page_size > INT32_MAX - 256 ||
        (!table && int64_t(batch) * table_width > pages) || (!starts && tokens % batch))
        return CF_E_SHAPE;
    if (!cache || !kv_lens) return CF_E_NULL;
    RowsOf x[2];
    if (int rc = check_rows(k, tokens, kv_heads, head_dim, elem_bytes(a_dtype), false, &x[0])) return rc;
    if (int rc = check_rows(v, tokens, kv_heads, head_dim, elem_bytes(a_dtype), false, &x[1])) return rc;
    if (!aligned16(cache) || !aligned4(table) || !aligned4(kv_lens) || !aligned4(starts)) return CF_E_ALIGN;
    const Range rc = range_of(cache, bytes);
    const Range read[5] = {x[0].range(), x[1].range(), range_of(table, table ? int64_t(batch) * table_width * 4 : 0),
                           range_of(kv_lens, int64_t(batch) * 4), range_of(starts, starts ? (int64_t(batch) + 1) * 4 : 0)};
    for (const Range& r : read)
        if (r.hi > r.lo && overlap(r, rc)) return CF_E_ALIAS;
    if (int e = check_device()) return e;
    return cf::launch_kv8_append(a_dtype, x[0].r, x[1].r, tokens, kv8_cache(cache, pages, page_size, kv_heads, head_dim), batch, table,
                                 table_width, kv_lens, starts, static_cast<hipStream_t>(stream)) == hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

int cf_kv8_read(int a_dtype, const uint8_t* cache, int64_t pages, int page_size, int kv_heads, int head_dim,
                const int64_t* slots, int64_t tokens, const cf_rows* k, const cf_rows* v, void* stream) {
    return slot_rows(true, a_dtype, k, v, slots, tokens, cache, cf_kv8_cache_bytes(pages, page_size, kv_heads, head_dim),
                     kv_heads, head_dim, [&](const cf_rows& kr, const cf_rows& vr) {
                         return cf::launch_kv8_read(a_dtype, kr, vr, slots, tokens,
                                                    kv8_cache(cache, pages, page_size, kv_heads, head_dim),
                                                    static_cast<hipStream_t>(stream));
                     });
}

size_t cf_kv8_attention_workspace_bytes(int a_dtype, int64_t max_q, int q_heads, int kv_heads, int head_dim) {
    return attention_dims(a_dtype, max_q, q_heads, kv_heads, head_dim)
               ? cf::kv8_attention_workspace(a_dtype, head_dim, max_q * (q_heads / kv_heads))
               : 0;
}

int cf_kv8_attention(int a_dtype, const cf_rows* q, int64_t total_q, int q_heads, const uint8_t* cache,
                     int64_t pages, int page_size, int kv_heads, int head_dim, int batch, const int32_t* table,
                     int table_width, const int32_t* kv_lens, const int32_t* q_starts, int64_t max_q, int flags,
                     int window, float scale, const cf_rows* out, float* lse, void* workspace, size_t ws_bytes,
                     void* stream) {
    return paged_attention(a_dtype, q, total_q, q_heads, cache, cf_kv8_cache_bytes(pages, page_size, kv_heads, head_dim), pages,
                           page_size, kv_heads, head_dim, batch, table, table_width, kv_lens, q_starts, max_q, flags,
                           window, scale, out, lse, workspace, ws_bytes, cf_kv8_attention_workspace_bytes,
                           [&](const cf_rows& qr, const cf_rows& outr, int64_t most) {
                               const cf::Kv8Attention call{qr,     outr,  kv8_cache(cache, pages, page_size, kv_heads, head_dim),
                                                           table,  kv_lens, q_starts, lse, total_q, most, batch, table_width, q_heads,
                                                           flags & CF_ATTN_CAUSAL, window, scale};
                               return cf::launch_kv8_attention(a_dtype, call, workspace, static_cast<hipStream_t>(stream));
                           });
}

size_t cf_attention_workspace_bytes(int a_dtype, int64_t max_q, int q_heads, int kv_heads, int head_dim) {
    return attention_dims(a_dtype, max_q, q_heads, kv_heads, head_dim)
               ? cf::attention_workspace(a_dtype, head_dim, max_q * (q_heads / kv_heads))
               : 0;
}

int cf_attention(int a_dtype, const cf_rows* q, int64_t total_q, int q_heads, const cf_rows* k, const cf_rows* v,
                 int64_t total_k, int kv_heads, int head_dim, int batch, const int32_t* q_starts,
                 const int32_t* k_starts, int64_t max_q, int flags, int window, float scale, const cf_rows* out,
                 float* lse, void* workspace, size_t ws_bytes, void* stream) {
    if (a_dtype != CF_BF16 && a_dtype != CF_F32) return CF_E_ARG;
    if ((flags & ~CF_ATTN_CAUSAL) || window < 0 || (window && !(flags & CF_ATTN_CAUSAL))) return CF_E_ARG;
    if (!(scale > 0.f) || scale > 1e38f) return CF_E_ARG;
    if (!kv4_dims(16, kv_heads, head_dim) || q_heads < 1 || q_heads > 65535 || q_heads % kv_heads || total_q < 0 ||
        total_q > kMaxAttnRows / q_heads || max_q < 0 || total_k < 0 || total_k > kMaxAttnRows)
        return CF_E_SHAPE;
    if (total_q == 0) return CF_OK;
    if (max_q > total_q || batch < 1 || batch > kMaxSequences || (!q_starts && total_q % batch) || (!k_starts && total_k % batch))
        return CF_E_SHAPE;
    if (!workspace) return CF_E_NULL;
    const int64_t esz = elem_bytes(a_dtype);
    RowsOf x[4];
    if (int rc = check_rows(q, total_q, q_heads, head_dim, esz, false, &x[0])) return rc;
    if (int rc = check_rows(k, total_k, kv_heads, head_dim, esz, false, &x[1])) return rc;
    if (int rc = check_rows(v, total_k, kv_heads, head_dim, esz, false, &x[2])) return rc;
    if (int rc = check_rows(out, total_q, q_heads, head_dim, esz, true, &x[3])) return rc;
    // rows of a tile are reached by 32-bit offsets
    if (total_k && (x[1].r.token_stride > kMaxKeyStride / esz || x[2].r.token_stride > kMaxKeyStride / esz)) return CF_E_SHAPE;
    if (!aligned4(q_starts) || !aligned4(k_starts) || !aligned4(lse) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return CF_E_ALIGN;
    if (max_q == 0) max_q = q_starts ? total_q : total_q / batch;
    const size_t need = cf_attention_workspace_bytes(a_dtype, max_q, q_heads, kv_heads, head_dim);
    if (ws_bytes < need) return CF_E_WORKSPACE;
    for (int i = 0; i < 3; ++i)
        if (!apart(x[i], x[3])) return CF_E_ALIAS;
    const Range r[8] = {x[0].range(),
                        x[1].range(),
                        x[2].range(),
                        range_of(q_starts, q_starts ? (int64_t(batch) + 1) * 4 : 0),
                        range_of(k_starts, k_starts ? (int64_t(batch) + 1) * 4 : 0),
                        x[3].range(),
                        range_of(lse, lse ? total_q * q_heads * 4 : 0),
                        range_of(workspace, static_cast<int64_t>(need))};
    for (int i = 5; i < 8; ++i)
        for (int j = i == 5 ? 3 : 0; j < i; ++j)  // rows and out were looked at row by row
            if (r[i].hi > r[i].lo && r[j].hi > r[j].lo && overlap(r[i], r[j])) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    const cf::RowsAttention call{x[0].r, x[1].r, x[2].r, x[3].r, q_starts, k_starts, lse, total_q, total_k, max_q, batch, q_heads, kv_heads,
                                 head_dim, flags & CF_ATTN_CAUSAL, window, scale};
    return cf::launch_attention(a_dtype, call, workspace, static_cast<hipStream_t>(stream)) == hipSuccess ? CF_OK : CF_E_HIP;
}

size_t cf_pages_workspace_bytes(int64_t pages, int rows) {
    return pages < 1 || pages > INT32_MAX || rows < 1 || rows > kMaxPageRows ? 0 : cf::pages_workspace(pages, rows);
}

int cf_pages_resize(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size,
                    const int32_t* want, int32_t* missing, void* workspace, size_t ws_bytes, void* stream) {
    if (int rc = check_pages(in, out, pages, rows, width, page_size, true, want, {missing, nullptr, nullptr}, {1, 0, 0}, workspace, ws_bytes))
        return rc;
    if (!want) return CF_E_NULL;
    if (int rc = check_device()) return rc;
    const cf::PagesCall call{*in, *out, pages, rows, width, page_size, want, nullptr, nullptr, missing};
    return cf::launch_pages_resize(call, workspace, static_cast<hipStream_t>(stream)) == hipSuccess ? CF_OK : CF_E_HIP;
}

int cf_pages_fork(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size,
                  const int32_t* parents, int32_t* src, int32_t* dst, int32_t* missing, void* workspace, size_t ws_bytes,
                  void* stream) {
    return pages_fork(in, out, pages, rows, width, page_size, parents, src, dst, missing, false, workspace, ws_bytes, stream);
}

int cf_pages_fork_own(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int page_size,
                      const int32_t* parents, int32_t* src, int32_t* dst, int32_t* missing, void* workspace, size_t ws_bytes,
                      void* stream) {
    return pages_fork(in, out, pages, rows, width, page_size, parents, src, dst, missing, true, workspace, ws_bytes, stream);
}

int cf_pages_compact(const cf_pages* in, const cf_pages* out, int64_t pages, int rows, int width, int32_t* src,
                     int32_t* dst, int32_t* count, void* workspace, size_t ws_bytes, void* stream) {
    if (int rc = check_pages(in, out, pages, rows, width, 1, true, nullptr, {src, dst, count}, {pages / 2, pages / 2, 1}, workspace, ws_bytes))
        return rc;
    if (int rc = check_device()) return rc;
    const cf::PagesCall call{*in, *out, pages, rows, width, 1, nullptr, src, dst, count};
    return cf::launch_pages_compact(call, workspace, static_cast<hipStream_t>(stream)) == hipSuccess ? CF_OK : CF_E_HIP;
}

int cf_pages_copy(void* data, int64_t pages, int64_t page_bytes, int layers, int64_t layer_stride, const int32_t* src,
                  const int32_t* dst, int64_t n, const int32_t* count, void* stream) {
    if (pages < 1 || pages > INT32_MAX || page_bytes < 16 || page_bytes % 16 || page_bytes > (int64_t(1) << 40) || layers < 1 ||
        layers > 65535 || n < 0 || n > (1 << 30))
        return CF_E_SHAPE;
    const wide one = wide(pages) * page_bytes;
    if (layers == 1) layer_stride = static_cast<int64_t>(one <= kMaxExtent ? one : 0);
    if (one > kMaxExtent || layer_stride < one || layer_stride % 16 || wide(layers - 1) * layer_stride + one > kMaxExtent ||
        wide(layers) * (page_bytes / 16384 + 1) > INT32_MAX)
        return CF_E_SHAPE;
    if (n == 0) return CF_OK;
    if (!data || !src || !dst) return CF_E_NULL;
    if (!aligned16(data) || !aligned4(src) || !aligned4(dst) || !aligned4(count)) return CF_E_ALIGN;
    const Range d = range_of(data, static_cast<int64_t>(wide(layers - 1) * layer_stride + one));
    if (overlap(d, range_of(src, n * 4)) || overlap(d, range_of(dst, n * 4)) || (count && overlap(d, range_of(count, 4)))) return CF_E_ALIAS;
    if (int rc = check_device()) return rc;
    return cf::launch_pages_copy(data, pages, page_bytes, layers, layer_stride, src, dst, n, count, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? CF_OK
               : CF_E_HIP;
}

}  // extern "C"
