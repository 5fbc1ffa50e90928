// cf_kv8.hip - writer and reader of the 8-bit K/V cache.
//
// Sixteen tokens of a page and head are held as E4M3 codes and the exponent e of one scale, for K and for V:
//   e = the least integer with max|finite x| <= 448 * 2^e, within [-15, 7]
//   code = the nearest E4M3 number to x * 2^-e, ties to the even code; 448 above 448; NaN for NaN and infinities
// x * 2^-e is exact, and so is what a code stands for, so codes are the same for fp32 and bf16 rows of equal
// values.  Tokens that come behind others of the same sixteen keep their scale or raise it; what is held is then
// rounded to the raised one, from the values that it has.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "cf.h"
#include "cf_internal.h"
#include "cf_kv8.h"
#include "cf_rows.h"

namespace cf {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct AppendArgs {
    RowSet k, v;
    int tokens, each;  // each: new tokens of every sequence where starts is null
    Kv8Cache cache;
    int batch, width;
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* starts;
};

// CH consecutive channels of a row, as they lie there: half the registers of fp32, where they are bf16.
template <typename T, int CH>
struct Few {
    typedef T Vec __attribute__((ext_vector_type(CH)));
    typedef uint32_t Words __attribute__((ext_vector_type(CH * sizeof(T) / 4)));
    Words w;
    __device__ __forceinline__ void load(const T* p) { w = __builtin_bit_cast(Words, *reinterpret_cast<const Vec*>(p)); }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
    // the bit patterns of the largest magnitudes so far, whatever they are: one, or of bf16 two
    __device__ __forceinline__ uint32_t largest(uint32_t top) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(CH * sizeof(T) / 4); ++i) {
            if constexpr (sizeof(T) == 2) {
                typedef uint16_t Two __attribute__((ext_vector_type(2)));
                const uint32_t word = w[i] & 0x7fff7fffu;
                top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(Two, word), __builtin_bit_cast(Two, top)));
            } else {
                top = max(top, w[i] & 0x7fffffffu);
            }
        }
        return top;
    }
};

// Bit pattern of the magnitude where it is finite.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))); }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d, 64)));
    return v;
}

// Bit patterns of magnitudes order as the magnitudes do.  top = 1.m * 2^(E - 127); 448 = 1.75 * 2^8.
__device__ __forceinline__ int exponent_of(uint32_t top) {
    const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u);
    return min(max(e, kKv8ExpMin), kKv8ExpMax);
}

__device__ __forceinline__ int held_exponent(uint8_t byte) {
    return min(max(static_cast<int>(byte) - 127, kKv8ExpMin), kKv8ExpMax);
}

__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The largest number of the largest scale.
constexpr uint32_t kLargest = 0x47600000u;  // 448 * 2^kKv8ExpMax

// Codes of two values in the low or high half of c.  The conversion divides by the scale and rounds to nearest
// even; beyond 464 it would give NaN, which infinities are left to become.  CUT: there may be values
// beyond 448 of the scale, or that are not finite.
template <bool HIGH, bool CUT>
__device__ __forceinline__ uint32_t encode2(uint32_t c, float a, float b, float scale) {
    const float lim = 448.f * scale;
    const auto cut = [&](float x) {
        if constexpr (!CUT) return x;
        return (__float_as_uint(x) & 0x7fffffffu) < 0x7f800000u ? __builtin_amdgcn_fmed3f(x, -lim, lim) : __builtin_inff();
    };
    typedef short vs2 __attribute__((ext_vector_type(2)));
    const vs2 r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(__builtin_bit_cast(vs2, c), cut(a), cut(b), scale, HIGH);
    return __builtin_bit_cast(uint32_t, r);
}

typedef float vf2 __attribute__((ext_vector_type(2)));
typedef uint32_t vu4 __attribute__((ext_vector_type(4)));

template <bool HIGH>
__device__ __forceinline__ vf2 decode2(uint32_t c, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, HIGH);
}

// The last sequence whose first token is not behind t, the same in every lane: 64 of them are looked at at a time.
__device__ __forceinline__ int sequence_of(const AppendArgs& p, int t) {
    if (!p.starts) return t / p.each;
    const int lane = threadIdx.x & 63;
    int first = 0;
    for (int n = p.batch; n > 1;) {
        const int step = (n + 63) / 64, i = lane * step;
        const bool before = i < n && p.starts[first + min(i, n - 1)] <= t;
        const int many = static_cast<int>(__popcll(__ballot(before)));
        const int at = many > 0 ? (many - 1) * step : 0;
        first += at;
        n = min(step, n - at);
    }
    return first;
}

// The same for the token of each lane, t0 + lane: the sequences behind b, which is t0's, begin with some of them.
template <int TILE>
__device__ __forceinline__ int sequence_from(const AppendArgs& p, int b, int t0) {
    const int lane = threadIdx.x & 63;
    if (!p.starts) return (t0 + lane) / p.each;
    if constexpr (TILE == 1) return b;
    const bool there = b + 1 + lane < p.batch;
    const int start = p.starts[there ? b + 1 + lane : b];
    int more = 0;
#pragma unroll
    for (int i = 0; i < TILE; ++i) {
        const int n = static_cast<int>(__popcll(__ballot(there && start <= t0 + i)));
        if (lane == i) more = n;
    }
    int of = b + more;
    if (more == 64)  // empty ones, more than were looked at
        while (of + 1 < p.batch && p.starts[of + 1] <= t0 + lane) ++of;
    return of;
}

// A wave writes what a call has of one block (16 tokens of one head).  Lane (o, c) of 2 x 32 holds places 8 o ..
// 8 o + 7 of D/32 channels: V's codes are eight tokens of a channel together, so a lane has its bytes whole, and
// K's leave in runs of a row.  TILE tokens of the call are looked through for first tokens of blocks, each by a
// lane: 16, or one where a call has few tokens of each sequence.
// Bound by instructions and by how many waves hide the loads of starts, lengths, pages and rows that follow each other:
// bf16 rows kept as they came (D = 128: 94 registers, widened 119; fp32 rows 167) and no value cut off that need not be
// took 9180 prompt tokens of 24 heads from 57 to 35 us (169 MB, 4.9 TB/s; 33 to 45 us from box to box), one token each
// of 61 sequences from 6.9 to 5.7.  fp32 rows: 52 us, 5.5 TB/s; D = 64: 22 and 29 us.  Slower: a loop over heads, which
// saves their lookups and takes registers (72 us).
template <typename T, int D, int TILE>
__global__ __launch_bounds__(kThreads) void append_kernel(const AppendArgs p) {
    constexpr int CH = D / 32;
    const int lane = threadIdx.x & 63;
    const int head = blockIdx.y * kWaves + (threadIdx.x >> 6);
    if (head >= p.cache.heads) return;
    const Kv8Block blk{p.cache.block.page, D};
    int place = 0, many = 0, page = -1;  // a first token's place in its page, the block's tokens in this call, the page
    const int mine = blockIdx.x * TILE + lane;
    const int b = sequence_from<TILE>(p, sequence_of(p, blockIdx.x * TILE), blockIdx.x * TILE);
    if (lane < TILE && mine < p.tokens) {
        const int lo = p.starts ? max(p.starts[b], 0) : b * p.each;
        const int hi = p.starts ? min(p.starts[b + 1], p.tokens) : (b + 1) * p.each;
        const int len = min(max(p.kv_lens[b], 0), p.width << p.cache.shift);
        const int64_t pos = int64_t(len) - hi + mine;
        if (mine >= lo && mine < hi && pos >= 0 && ((pos & (kKv8Block - 1)) == 0 || mine == lo)) {
            place = static_cast<int>(pos & (blk.page - 1));
            many = min(kKv8Block - (place & (kKv8Block - 1)), hi - mine);
            const int64_t at = int64_t(b) * p.width + (pos >> p.cache.shift);
            page = p.table ? p.table[at] : static_cast<int>(at);
        }
    }
    const int o = lane >> 5, c0 = (lane & 31) * CH;
    for (uint64_t left = __ballot(many > 0 && page >= 0 && page < p.cache.pages); left; left &= left - 1) {
        const int lead = __builtin_ctzll(left);
        const int t0 = blockIdx.x * TILE + lead;
        const int in = __builtin_amdgcn_readlane(place, lead), n = __builtin_amdgcn_readlane(many, lead);
        uint8_t* const base = p.cache.at(__builtin_amdgcn_readlane(page, lead), head);
        const int from = in & (kKv8Block - 1), first = in - from;  // the block's first place in the page
        Few<T, CH> x[2][8];
        uint32_t top[2] = {0, 0};  // bits of the largest magnitude
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = 8 * o + i - from;
            x[0][i].w = x[1][i].w = 0;
            if (at >= 0 && at < n) {
                x[0][i].load(row_ptr<T>(p.k, t0 + at, head) + c0);
                x[1][i].load(row_ptr<T>(p.v, t0 + at, head) + c0);
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) top[s] = x[s][i].largest(top[s]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if constexpr (sizeof(T) == 2) top[s] = max(top[s] << 16, top[s] & 0xffff0000u);
            top[s] = uniform(wave_max(top[s]));
        }
        // Of finite values up to the largest scale's none needs cutting off: a scale takes its largest value.  So nearly
        // always; doing it for each value took two thirds of the kernel's instructions.
        const bool cut = max(top[0], top[1]) > kLargest;
        if (cut) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (top[s] < 0x7f800000u) continue;
                top[s] = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < CH; ++j) top[s] = max(top[s], finite_bits(x[s][i][j]));
                top[s] = wave_max(top[s]);
            }
        }
        uint8_t* const scales[2] = {base + blk.k_scale(first), base + blk.v_scale(first)};
        int e[2];
        bool raise[2];
        float old[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            e[s] = exponent_of(top[s]);
            const int was = from ? held_exponent(*scales[s]) : e[s];
            raise[s] = was < e[s];
            e[s] = max(e[s], was);
            old[s] = two_to(was);
        }
        const float ks = two_to(e[0]), vs = two_to(e[1]);
        uint8_t* const kc = base + blk.k_code(first + 8 * o) + c0;
        uint8_t* const vc = base + blk.v_code(first + 8 * o, c0);
        const auto fresh = [&](int i) { return 8 * o + i >= from && 8 * o + i < from + n; };
        const auto write = [&](auto cutting) {
            constexpr bool kCut = decltype(cutting)::value;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t c = encode2<false, kCut>(0, x[0][i][0], x[0][i][1], ks);
                if constexpr (CH == 4) c = encode2<true, kCut>(c, x[0][i][2], x[0][i][3], ks);
                if (!fresh(i)) {
                    if (!raise[0] || 8 * o + i >= from) continue;  // places behind the new ones hold nothing
                    if constexpr (CH == 4) {
                        const uint32_t h = *reinterpret_cast<const uint32_t*>(kc + i * D);
                        const vf2 a = decode2<false>(h, old[0]), b = decode2<true>(h, old[0]);
                        c = encode2<true, true>(encode2<false, true>(0, a.x, a.y, ks), b.x, b.y, ks);
                    } else {
                        const vf2 a = decode2<false>(*reinterpret_cast<const uint16_t*>(kc + i * D), old[0]);
                        c = encode2<false, true>(0, a.x, a.y, ks);
                    }
                }
                if constexpr (CH == 4)
                    *reinterpret_cast<uint32_t*>(kc + i * D) = c;
                else
                    *reinterpret_cast<uint16_t*>(kc + i * D) = static_cast<uint16_t>(c);
            }
            const bool whole = from <= 8 * o && from + n >= 8 * o + 8;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                vu2 c;
                c.x = encode2<true, kCut>(encode2<false, kCut>(0, x[1][0][j], x[1][1][j], vs), x[1][2][j], x[1][3][j], vs);
                c.y = encode2<true, kCut>(encode2<false, kCut>(0, x[1][4][j], x[1][5][j], vs), x[1][6][j], x[1][7][j], vs);
                vu2* const to = reinterpret_cast<vu2*>(vc + 8 * j);
                if (whole) {
                    *to = c;
                } else if (raise[1]) {
                    vu2 h = *to;
                    const vf2 a = decode2<false>(h.x, old[1]), b = decode2<true>(h.x, old[1]);
                    const vf2 d = decode2<false>(h.y, old[1]), f = decode2<true>(h.y, old[1]);
                    h.x = encode2<true, true>(encode2<false, true>(0, a.x, a.y, vs), b.x, b.y, vs);
                    h.y = encode2<true, true>(encode2<false, true>(0, d.x, d.y, vs), f.x, f.y, vs);
                    uint64_t keep = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) keep |= fresh(i) ? 0 : uint64_t(0xff) << (8 * i);
                    const uint64_t w = (__builtin_bit_cast(uint64_t, h) & keep) | (__builtin_bit_cast(uint64_t, c) & ~keep);
                    *to = __builtin_bit_cast(vu2, w);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (fresh(i)) vc[8 * j + i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
                }
            }
        };
        if (cut)
            write(std::true_type());
        else
            write(std::false_type());
        if (lane < 2) *(lane ? scales[1] : scales[0]) = static_cast<uint8_t>((lane ? e[1] : e[0]) + 127);
    }
}

struct ReadArgs {
    RowSet k, v;
    const int64_t* slots;
    int64_t tokens;
    Kv8Cache cache;
};

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(const ReadArgs p) {
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int head = blockIdx.y;
    const int64_t t = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes;
    if (t >= p.tokens) return;
    const int64_t slot = p.slots[t];
    const int64_t page = slot >> p.cache.shift;
    float k[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.f;
    if (slot >= 0 && page < p.cache.pages) {
        const int in = static_cast<int>(slot - page * p.cache.block.page);
        const Kv8Block blk{p.cache.block.page, D};
        const uint8_t* const base = p.cache.at(page, head);
        const vu2 kc = *reinterpret_cast<const vu2*>(base + blk.k_code(in) + 8 * lane);
        // V's eight channels lie together with those of seven other tokens, which other lanes read: four loads, and a byte of
        // each eight (9218 tokens of 24 heads of 128 in bf16 28 us, 6.0 TB/s; eight loads of a byte took 59)
        const vu4* const vc = reinterpret_cast<const vu4*>(base + blk.v_code(in & ~7, 8 * lane));
        const uint32_t one = in & 3, low = one | (4 + one) << 8 | 0x0c0c0000u, high = 0x0c0cu | one << 16 | (4 + one) << 24;
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const vu4 x = vc[i];
            c[2 * i] = in & 4 ? x.y : x.x, c[2 * i + 1] = in & 4 ? x.w : x.z;
        }
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __builtin_amdgcn_perm(c[4 * i + 1], c[4 * i], low) | __builtin_amdgcn_perm(c[4 * i + 3], c[4 * i + 2], high);
        const float ks = __uint_as_float(uint32_t(base[blk.k_scale(in)]) << 23), vs = __uint_as_float(uint32_t(base[blk.v_scale(in)]) << 23);
        const auto get = [](uint32_t lo, uint32_t hi, float s, float (&x)[8]) {
            const vf2 a = decode2<false>(lo, s), b = decode2<true>(lo, s), c = decode2<false>(hi, s), d = decode2<true>(hi, s);
            x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
        };
        get(kc.x, kc.y, ks, k);
        get(w[0], w[1], vs, v);
    }
    Row8<T> r;
    r.set(k);
    r.store(row_ptr<T>(p.k, t, head) + lane * 8);
    r.set(v);
    r.store(row_ptr<T>(p.v, t, head) + lane * 8);
}

template <typename T, int D>
void launch_append(const AppendArgs& p, hipStream_t stream) {
    const uint32_t y = (p.cache.heads + kWaves - 1) / kWaves;
    // A wave for each token finds one block or none; for each 16 tokens, those that begin there, one after the other.
    // 64 sequences of 1 to 5 new tokens take 6.7 and 28 us, of 1 to 40 10.5 and 21, of 1 to 100 15 and 15.  (A dispatch
    // counts its work-items in 32 bits.)
    if (p.tokens <= kKv8Block * int64_t(p.batch) && p.tokens <= 1 << 22)
        append_kernel<T, D, 1><<<dim3(p.tokens, y), kThreads, 0, stream>>>(p);
    else
        append_kernel<T, D, 16><<<dim3((p.tokens + 15) / 16, y), kThreads, 0, stream>>>(p);
}

template <typename T, int D>
void launch_read(const ReadArgs& p, hipStream_t stream) {
    constexpr int kRows = kThreads / (D / 8);
    read_kernel<T, D><<<dim3(static_cast<uint32_t>((p.tokens + kRows - 1) / kRows), p.cache.heads), kThreads, 0, stream>>>(p);
}

}  // namespace

hipError_t launch_kv8_append(int a_dtype, const RowSet& k, const RowSet& v, int64_t tokens, const Kv8Cache& cache,
                             int batch, const int32_t* table, int table_width, const int32_t* kv_lens,
                             const int32_t* starts, hipStream_t stream) {
    const AppendArgs p{k,     v,           static_cast<int>(tokens), starts ? 0 : static_cast<int>(tokens / batch), cache, batch,
                       table_width, table, kv_lens,                  starts};
    if (a_dtype == CF_BF16)
        cache.block.dim == 64 ? launch_append<__bf16, 64>(p, stream) : launch_append<__bf16, 128>(p, stream);
    else
        cache.block.dim == 64 ? launch_append<float, 64>(p, stream) : launch_append<float, 128>(p, stream);
    return hipGetLastError();
}

hipError_t launch_kv8_read(int a_dtype, const RowSet& k, const RowSet& v, const int64_t* slots, int64_t tokens,
                           const Kv8Cache& cache, hipStream_t stream) {
    const ReadArgs p{k, v, slots, tokens, cache};
    if (a_dtype == CF_BF16)
        cache.block.dim == 64 ? launch_read<__bf16, 64>(p, stream) : launch_read<__bf16, 128>(p, stream);
    else
        cache.block.dim == 64 ? launch_read<float, 64>(p, stream) : launch_read<float, 128>(p, stream);
    return hipGetLastError();
}

}  // namespace cf
