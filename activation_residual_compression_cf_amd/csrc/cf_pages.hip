// cf_pages.hip - who holds which page of a cache: resizing, forking and compacting sequences, and copying pages.
//
// refs[p] counts the rows of a table that hold page p, and a page with none is free.  Free pages are taken in the order
// of their numbers by rows in the order of theirs, so results do not depend on the order in which threads run: counts
// change by integer atomics, whose order does not show, and the rest are sums along the pages and the rows.
//
// Everything but the copy is small: a few words for each page and table entry, bound by latencies.  What fits a
// workgroup's 1024 threads well runs in one launch, phase by phase between barriers; more pages or entries take a
// launch a phase.  The copy is bound by memory.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "cf.h"
#include "cf_internal.h"
#include "cf_vec.h"

namespace cf {
namespace {

constexpr int kBlock = 1024;
constexpr int kBlockWaves = kBlock / 64;
// Up to so many pages and so many table entries are one workgroup's work.  As graphs, in one launch and in several:
// 32000 pages, 1600 entries: resize 22.7 and 23.9 us, fork 25.5 and 26.6, compact 19.6 and 20.8;  500 pages, 2048
// entries: 18.0 and 19.9, 17.1 and 22.3;  2000 pages, 6400 entries: 20.8 and 20.0, 23.3 and 23.1, a fork that
// parts all rows 29.5 and 23.5;  32000 pages, 32000 entries: 37 and 25, 61 and 27, 95 and 28.
constexpr int64_t kSmall = 1 << 15, kSmallEntries = 1 << 12;

// The sum may pass 2^31, where page sizes are no powers of two, but not 2^32: a row has fewer than 2^31 - 256 tokens.
__device__ __forceinline__ int pages_of(int len, int page_size) {
    return static_cast<int>((static_cast<uint32_t>(len) + static_cast<uint32_t>(page_size) - 1) / static_cast<uint32_t>(page_size));
}

// A word that atomics have changed in this launch.
__device__ __forceinline__ int fresh_load(const int32_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Inclusive sums over a workgroup's threads; total: of all.
__device__ int block_scan(int v, int* total) {
    __shared__ int sums[kBlockWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(v, d, 64);
        if (lane >= d) v += x;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 63) sums[wave] = v;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < kBlockWaves; ++i) {
        if (i < wave) before += sums[i];
        all += sums[i];
    }
    *total = all;
    return before + v;
}

struct PagesArgs {
    int32_t *refs_in, *table_in, *lens_in, *refs, *table, *lens;
    int pages, rows, width, page_size;
    const int32_t* want;     // resize: tokens, fork: parents
    int32_t *src, *dst;      // fork, compact
    int32_t* count;          // missing, or moves
    int32_t *first, *offset, *list;  // workspace
    int firsts;                      // how many of `first`
    __device__ __forceinline__ bool named(int page) const { return static_cast<uint32_t>(page) < static_cast<uint32_t>(pages); }
    __device__ __forceinline__ int len_of(int row) const { return min(max(lens_in[row], 0), width * page_size); }
    __device__ __forceinline__ int parent_of(int row) const { return static_cast<uint32_t>(want[row]) < static_cast<uint32_t>(rows) ? want[row] : -1; }
};

// What a row asks for: pages [from, from + need) of it, and its tokens with them and without; or more than it can have.
struct Ask {
    int from, need, size, size_without;
    bool refused;
};

struct Resize {
    static constexpr int kPhases = 1;
    static __device__ __forceinline__ Ask ask(const PagesArgs& p, int row) {
        const int len = p.len_of(row), want = p.want[row];
        if (want < 0) return {0, 0, len, len, false};
        if (want > p.width * p.page_size) return {0, 0, len, len, true};
        const int have = pages_of(len, p.page_size), need = max(pages_of(want, p.page_size) - have, 0);
        return {have, need, want, need ? len : want, false};
    }
    static __device__ __forceinline__ void got(const PagesArgs&, int, int) {}
    static __device__ __forceinline__ void done(const PagesArgs&, int, const Ask&, bool) {}
    static __device__ __forceinline__ void phase(const PagesArgs& p, int, int64_t i, int64_t step) {
        for (; i < int64_t(p.rows) * p.width; i += step) {
            const int row = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.width)), c = static_cast<int>(i) - row * p.width;
            const int len = p.len_of(row), have = pages_of(len, p.page_size);
            const int want = p.want[row];
            const int keep = want < 0 || want > p.width * p.page_size ? have : min(have, pages_of(want, p.page_size));
            const int page = p.table_in[i];
            if (c >= keep && c < have && p.named(page)) atomicSub(p.refs + page, 1);
            p.table[i] = c < keep ? page : -1;
        }
    }
};

// OWN: a row's last, partly filled page is looked at whoever else holds it, not only rows with the same parent.
template <bool OWN>
struct Fork {
    static constexpr int kPhases = 2;
    // A row's claim to go on with a partly filled page: the lowest of a parent's rows, or of a page's, does; the parent
    // itself, or a row that stays, goes first.
    static __device__ __forceinline__ int claim(const PagesArgs& p, int row, int parent) {
        if (OWN) return row == parent ? row : p.rows + row;
        return row == parent ? -1 : row;
    }
    // Whether a row gets a page of its own for its last, partly filled one: all but one of those that claim it do.
    static __device__ __forceinline__ bool fresh(const PagesArgs& p, int row, int parent, int size) {
        if (parent < 0 || size % p.page_size == 0) return false;
        if (!OWN && fresh_load(p.first + parent) == claim(p, row, parent)) return false;
        const int page = p.table_in[int64_t(parent) * p.width + size / p.page_size];
        return p.named(page) && (!OWN || fresh_load(p.first + page) != claim(p, row, parent));
    }
    static __device__ __forceinline__ Ask ask(const PagesArgs& p, int row) {
        const int parent = p.parent_of(row), size = parent < 0 ? 0 : p.len_of(parent), whole = size / p.page_size;
        const bool f = fresh(p, row, parent, size);
        return {whole, f ? 1 : 0, size, f ? whole * p.page_size : size, false};
    }
    static __device__ __forceinline__ void got(const PagesArgs& p, int row, int page) { p.dst[row] = page; }
    static __device__ __forceinline__ void done(const PagesArgs& p, int row, const Ask& a, bool served) {
        const bool copies = a.need && served;
        p.src[row] = copies ? p.table_in[int64_t(p.parent_of(row)) * p.width + a.from] : -1;
        if (!copies) p.dst[row] = -1;
    }
    static __device__ __forceinline__ void phase(const PagesArgs& p, int n, int64_t i, int64_t step) {
        if (n == 0 && !OWN) {
            for (; i < p.rows; i += step) {
                const int row = static_cast<int>(i), parent = p.parent_of(row);
                if (parent >= 0) atomicMin(p.first + parent, claim(p, row, parent));
            }
            return;
        }
        for (; i < int64_t(p.rows) * p.width; i += step) {
            const int row = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.width)), c = static_cast<int>(i) - row * p.width;
            const int parent = p.parent_of(row), size = parent < 0 ? 0 : p.len_of(parent);
            const bool held = c < pages_of(size, p.page_size);
            if (OWN && n == 0) {
                const int page = held ? p.table_in[int64_t(parent) * p.width + c] : -1;
                // nobody goes on with a page that is whole in some row
                if (p.named(page)) atomicMin(p.first + page, c == size / p.page_size ? claim(p, row, parent) : INT32_MIN);
                continue;
            }
            const int old = p.table_in[i];
            if (parent != row && c < pages_of(p.len_of(row), p.page_size) && p.named(old)) atomicSub(p.refs + old, 1);
            int page = -1;
            if (held && !(c == size / p.page_size && fresh(p, row, parent, size))) {
                page = p.table_in[int64_t(parent) * p.width + c];
                if (parent != row && p.named(page)) atomicAdd(p.refs + page, 1);
            } else if (OWN && held && parent == row) {
                atomicSub(p.refs + old, 1);  // a page that is left to those that go on with it
            }
            p.table[i] = page;
        }
    }
};

// What comes before the phases: the counts where they are kept elsewhere, and the workspace's start.
__device__ __forceinline__ void begin(const PagesArgs& p, int64_t i, int64_t step) {
    if (i == 0) *p.count = 0;
    if (p.refs != p.refs_in)
        for (int64_t j = i; j < p.pages; j += step) p.refs[j] = p.refs_in[j];
    if (p.first)
        for (int64_t j = i; j < p.firsts; j += step) p.first[j] = INT32_MAX;
}

// Free pages for the rows that ask, by one workgroup.
template <typename OP>
__device__ void take(const PagesArgs& p) {
    // Up to as many rows as threads are asked once (a row's answer takes four loads that follow each other; 32 rows
    // forked: 11.1 us for 11.8).
    __shared__ int from[kBlock];
    const bool once = p.rows <= kBlock;
    Ask own{};
    // where each row's pages begin in the list of those that are asked for
    int total = 0;
    for (int r0 = 0; r0 < p.rows; r0 += kBlock) {
        const int row = r0 + threadIdx.x;
        if (row < p.rows) own = OP::ask(p, row);
        if (once) from[threadIdx.x] = own.from;
        const int need = row < p.rows ? own.need : 0;
        int all;
        const int upto = block_scan(need, &all);
        if (row < p.rows) p.offset[row] = total + upto - need;
        total += all;
    }
    if (threadIdx.x == 0) p.offset[p.rows] = total;
    // the list: the first free pages, as many as that
    int found = 0;
    constexpr int kEach = 16;
    for (int64_t p0 = 0; p0 < p.pages && found < total; p0 += kBlock * kEach) {
        const int64_t mine = p0 + threadIdx.x * kEach;
        uint32_t free = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (mine + i < p.pages && fresh_load(p.refs + mine + i) == 0) free |= 1u << i;
        int all;
        int at = found + block_scan(__popc(free), &all) - __popc(free);
        for (; free && at < total; free &= free - 1) p.list[at++] = static_cast<int>(mine) + __ffs(static_cast<int>(free)) - 1;
        found += all;
    }
    __syncthreads();
    // a row gets all of its pages or none
    for (int i = threadIdx.x; i < min(total, found); i += kBlock) {
        int row = 0, end = p.rows;  // offset[row] <= i < offset[end]
        while (end - row > 1) {
            const int mid = (row + end) >> 1;
            if (p.offset[mid] <= i)
                row = mid;
            else
                end = mid;
        }
        if (p.offset[row + 1] > found) continue;
        const int page = p.list[i];
        p.table[int64_t(row) * p.width + (once ? from[row] : OP::ask(p, row).from) + i - p.offset[row]] = page;
        p.refs[page] = 1;
        OP::got(p, row, page);
    }
    __syncthreads();  // what is asked for depends on lens, which may be the ones that are written
    int missing = 0;
    for (int row = threadIdx.x; row < p.rows; row += kBlock) {
        const Ask a = once ? own : OP::ask(p, row);
        const bool served = a.need == 0 || p.offset[row + 1] <= found;
        OP::done(p, row, a, served);
        p.lens[row] = served ? a.size : a.size_without;
        missing += !served || a.refused;
    }
    int all;
    block_scan(missing, &all);
    if (threadIdx.x == 0) *p.count = all;
}

template <typename OP>
__global__ __launch_bounds__(kBlock) void small_kernel(const PagesArgs p) {
    begin(p, threadIdx.x, kBlock);
    for (int n = 0; n < OP::kPhases; ++n) {
        __syncthreads();
        OP::phase(p, n, threadIdx.x, kBlock);
    }
    __syncthreads();
    take<OP>(p);
}

__global__ __launch_bounds__(256) void begin_kernel(const PagesArgs p) {
    begin(p, int64_t(blockIdx.x) * 256 + threadIdx.x, int64_t(gridDim.x) * 256);
}

template <typename OP>
__global__ __launch_bounds__(256) void phase_kernel(const PagesArgs p, int n) {
    OP::phase(p, n, int64_t(blockIdx.x) * 256 + threadIdx.x, int64_t(gridDim.x) * 256);
}

template <typename OP>
__global__ __launch_bounds__(kBlock) void take_kernel(const PagesArgs p) {
    take<OP>(p);
}

uint32_t blocks_for(int64_t n) {
    const int64_t b = (n + 255) / 256;
    return static_cast<uint32_t>(b < 1 ? 1 : b > 2048 ? 2048 : b);
}

template <typename OP>
hipError_t run(const PagesArgs& p, hipStream_t stream) {
    const int64_t entries = int64_t(p.rows) * p.width, most = entries > p.pages ? entries : p.pages;
    if (p.pages <= kSmall && entries <= kSmallEntries) {
        small_kernel<OP><<<1, kBlock, 0, stream>>>(p);
        return hipGetLastError();
    }
    begin_kernel<<<blocks_for(most), 256, 0, stream>>>(p);
    for (int n = 0; n < OP::kPhases; ++n) phase_kernel<OP><<<blocks_for(entries), 256, 0, stream>>>(p, n);
    take_kernel<OP><<<1, kBlock, 0, stream>>>(p);
    return hipGetLastError();
}

// ---- compacting

constexpr int kChunk = 4096;  // pages that a workgroup ranks, four a thread
constexpr int kChunkEach = kChunk / kBlock;

struct CompactArgs {
    int32_t *refs_in, *table_in, *lens_in, *refs, *table, *lens;
    int pages, rows, width, chunks;
    int32_t *src, *dst, *count;
    int32_t *used, *to;  // workspace: used pages of each chunk, and where each page goes: a page, or ~ a place in dst
};

__device__ int used_in(const CompactArgs& p, int64_t from, int64_t end) {
    int n = 0;
    for (int64_t i = from + threadIdx.x; i < end; i += kBlock) n += p.refs_in[i] != 0;
    int all;
    block_scan(n, &all);
    return all;
}

__global__ __launch_bounds__(kBlock) void count_kernel(const CompactArgs p) {
    const int64_t from = int64_t(blockIdx.x) * kChunk;
    const int n = used_in(p, from, min(from + kChunk, int64_t(p.pages)));
    if (threadIdx.x == 0) p.used[blockIdx.x] = n;
}

// Pages stay where they are up to as many as are used; the used ones behind go to the free ones before, in order.
// COUNTED: count_kernel has counted each chunk; else every workgroup counts all of the pages itself, a launch less (12000
// pages: 5.9 us for 10.6).
template <bool COUNTED>
__global__ __launch_bounds__(kBlock) void rank_kernel(const CompactArgs p) {
    int before, live, below;  // used pages before the workgroup's, of all, and before page number `live`
    if constexpr (COUNTED) {
        int n = 0, m = 0;
        for (int i = threadIdx.x; i < p.chunks; i += kBlock) {
            const int u = p.used[i];
            n += u;
            if (i < static_cast<int>(blockIdx.x)) m += u;
        }
        block_scan(n, &live);
        block_scan(m, &before);
        const int border = live / kChunk;  // its chunk holds page number `live`
        int b = 0;
        for (int i = threadIdx.x; i < border; i += kBlock) b += p.used[i];
        int whole;
        block_scan(b, &whole);
        below = whole + used_in(p, int64_t(border) * kChunk, live);
    } else {
        int n = 0, m = 0;
        for (int i = threadIdx.x; i < p.pages; i += kBlock) {
            const int u = p.refs_in[i] != 0;
            n += u;
            if (i < static_cast<int>(blockIdx.x) * kChunk) m += u;
        }
        block_scan(n, &live);
        block_scan(m, &before);
        below = used_in(p, 0, live);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.count = live - below, p.used[p.chunks] = live;

    const int64_t mine = int64_t(blockIdx.x) * kChunk + threadIdx.x * kChunkEach;
    uint32_t used = 0;
#pragma unroll
    for (int i = 0; i < kChunkEach; ++i)
        if (mine + i < p.pages && p.refs_in[mine + i] != 0) used |= 1u << i;
    int all;
    int at = before + block_scan(__popc(used), &all) - __popc(used);  // used pages before the page
#pragma unroll
    for (int i = 0; i < kChunkEach; ++i) {
        const int64_t page = mine + i;
        if (page >= p.pages) break;
        const bool on = used >> i & 1u;
        int goes = static_cast<int>(page);
        if (on && page >= live) {
            p.src[at - below] = static_cast<int>(page);
            goes = ~(at - below);
        } else if (!on && page < live) {
            p.dst[page - at] = static_cast<int>(page);
        }
        p.to[page] = goes;
        at += on;
    }
}

__global__ __launch_bounds__(256) void move_kernel(const CompactArgs p) {
    const int64_t i0 = int64_t(blockIdx.x) * 256 + threadIdx.x, step = int64_t(gridDim.x) * 256;
    const int moves = *p.count;
    for (int64_t i = i0; i < int64_t(p.rows) * p.width; i += step) {
        const int page = p.table_in[i];
        const int goes = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pages) ? p.to[page] : page;
        p.table[i] = goes < 0 && goes != page ? p.dst[~goes] : goes;
    }
    // a pair's counts belong to its thread, wherever they are kept
    for (int64_t k = i0; k < p.pages / 2; k += step) {
        if (k >= moves) {
            p.src[k] = p.dst[k] = -1;
            continue;
        }
        const int from = p.src[k], to = p.dst[k];
        p.refs[to] = p.refs_in[from];
        p.refs[from] = 0;
    }
    if (p.refs != p.refs_in) {
        const int live = p.used[p.chunks];
        for (int64_t i = i0; i < p.pages; i += step) {
            const bool on = p.refs_in[i] != 0;
            if (on ? i < live : i >= live) p.refs[i] = p.refs_in[i];
        }
    }
    if (p.lens != p.lens_in)
        for (int64_t i = i0; i < p.rows; i += step) p.lens[i] = p.lens_in[i];
}

// ---- copying

struct CopyArgs {
    uint8_t* data;
    int64_t pages, page_bytes, layer_stride, n;
    int layers, pieces;  // pieces of a page
    const int32_t *src, *dst, *count;
};

constexpr int kPiece = 256 * 16 * 4;  // bytes that a workgroup copies at once

__global__ __launch_bounds__(256) void copy_kernel(const CopyArgs p) {
    const int64_t n = p.count ? min(max(int64_t(*p.count), int64_t(0)), p.n) : p.n;
    const int64_t per = int64_t(p.layers) * p.pieces;
    for (int64_t i = blockIdx.x; i < n * per; i += gridDim.x) {
        const int64_t pair = i / per;
        const int rest = static_cast<int>(i - pair * per), layer = rest / p.pieces, piece = rest - layer * p.pieces;
        const int from = p.src[pair], to = p.dst[pair];
        if (static_cast<uint64_t>(from) >= static_cast<uint64_t>(p.pages) || static_cast<uint64_t>(to) >= static_cast<uint64_t>(p.pages) || from == to)
            continue;
        uint8_t* const base = p.data + layer * p.layer_stride;
        const uint8_t* const a = base + from * p.page_bytes;
        uint8_t* const b = base + to * p.page_bytes;
        vf4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = int64_t(piece) * kPiece + (k * 256 + threadIdx.x) * 16;
            if (at < p.page_bytes) x[k] = ld_nt(reinterpret_cast<const float*>(a + at));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = int64_t(piece) * kPiece + (k * 256 + threadIdx.x) * 16;
            if (at < p.page_bytes) st_nt(reinterpret_cast<float*>(b + at), x[k]);
        }
    }
}

PagesArgs args_of(const PagesCall& c, void* workspace) {
    PagesArgs p{c.in.refs, c.in.table, c.in.lens, c.out.refs, c.out.table, c.out.lens, static_cast<int>(c.pages), c.rows, c.width, c.page_size,
                c.want,    c.src,      c.dst,     c.count,    nullptr,     nullptr,    nullptr,    0};
    p.offset = static_cast<int32_t*>(workspace);
    p.list = p.offset + c.rows + 1;
    return p;
}

}  // namespace

size_t pages_workspace(int64_t pages, int rows) {
    const int64_t chunks = (pages + kChunk - 1) / kChunk;
    return 4 * (2 * static_cast<size_t>(pages) + 2 * static_cast<size_t>(rows) + chunks + 2);
}

hipError_t launch_pages_resize(const PagesCall& c, void* workspace, hipStream_t stream) {
    return run<Resize>(args_of(c, workspace), stream);
}

hipError_t launch_pages_fork(const PagesCall& c, bool own, void* workspace, hipStream_t stream) {
    PagesArgs p = args_of(c, workspace);
    p.first = p.list + c.pages, p.firsts = own ? static_cast<int>(c.pages) : c.rows;
    return own ? run<Fork<true>>(p, stream) : run<Fork<false>>(p, stream);
}

hipError_t launch_pages_compact(const PagesCall& c, void* workspace, hipStream_t stream) {
    const int chunks = static_cast<int>((c.pages + kChunk - 1) / kChunk);
    CompactArgs p{c.in.refs, c.in.table, c.in.lens, c.out.refs, c.out.table, c.out.lens, static_cast<int>(c.pages), c.rows, c.width, chunks,
                  c.src,     c.dst,      c.count,   nullptr,    nullptr};
    p.used = static_cast<int32_t*>(workspace);
    p.to = p.used + chunks + 1;
    if (c.pages <= kSmall) {
        rank_kernel<false><<<chunks, kBlock, 0, stream>>>(p);
    } else {
        count_kernel<<<chunks, kBlock, 0, stream>>>(p);
        rank_kernel<true><<<chunks, kBlock, 0, stream>>>(p);
    }
    const int64_t entries = int64_t(c.rows) * c.width;
    move_kernel<<<blocks_for(entries > c.pages ? entries : c.pages), 256, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_pages_copy(void* data, int64_t pages, int64_t page_bytes, int layers, int64_t layer_stride, const int32_t* src,
                             const int32_t* dst, int64_t n, const int32_t* count, hipStream_t stream) {
    const int pieces = static_cast<int>((page_bytes + kPiece - 1) / kPiece);
    const CopyArgs p{static_cast<uint8_t*>(data), pages, page_bytes, layer_stride, n, layers, pieces, src, dst, count};
    const __int128 items = __int128(n) * layers * pieces;
    const uint32_t grid = items < 256 * 8 ? static_cast<uint32_t>(items) : 256 * 8;
    copy_kernel<<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace cf
