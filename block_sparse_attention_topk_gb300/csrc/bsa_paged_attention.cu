// bsa_paged_attention.cu -- causal attention of new tokens over everything
// their sequences hold in the paged cache, with an optional sliding window and
// sinks, from a bf16 cache or an 8-bit one.
//
// What it computes, for query head g of KV head h in the row at position p:
//   y_j = log2(e) scale q . k_j,   out = sum_j 2^(y_j - m) v_j / sum_j 2^(y_j - m)
// over the tokens j <= p of the row's sequence, with a window only those with
// j > p - window or j < sinks; in 8 bits k_j and v_j are codes times the scale of
// their page and head.
//
// Both products run on the tensor core.  The 128 rows of an MMA are the G query
// heads of 128 / G tokens (they share the KV head's keys and values); a KV tile is
// one 128-token block of the cache, which lies there as one TMA box.  S = Q K^T
// goes to TMEM, the softmax turns a row a thread (one TMEM lane, so no shuffles)
// into probabilities of 16 bits in the place of the scores, and O += P V takes them
// from there as its A operand.  O stays in TMEM; it is rescaled only when a row's
// maximum has grown by more than 2^8 since the last time.
//  streams    two softmax groups of four warps, each with its own S and O, so that
//             one's products run under the other's exponentials.  An item of more
//             than 128 rows gives each its own 128 rows of the same KV tiles; a
//             smaller one (decode steps, ends of chunks) gives each every other KV
//             tile of the same rows, joined in shared memory.  Heads of more than
//             128 dimensions leave TMEM for one stream, with two S buffers;
//  portions   one warp finds what the CTA does of which item and announces it in
//  and copies shared memory, and copies queries and blocks by TMA into a ring of
//             stages;
//  MMAs       one thread issues them.  The product of half the probabilities
//             starts under the exponentials of the others;
//  values     (bf16) two warps go over the value rows of tiles that some rows do not see
//             in full: 0 * NaN is NaN, so what no row sees (the unused end of a block)
//             is set to zero, and so is what is not finite, which the epilogue gives
//             back to the rows that do see it;
//  widening   (8 bits) two groups of four warps turn codes into 16 bits, exactly, on
//             their way from a ring of codes to the ring, a stage each: keys into halves,
//             values into bf16, where what is not finite comes out as a number and is noted for
//             the epilogue.  Queries become halves too, a row divided by a power of two.
//             A key page's scale multiplies its scores, a value page's its probabilities.
// Rounding: scores, maxima, sums and outputs are fp32.  From a bf16 cache probabilities
// are rounded once, to bf16 (2^-8 of each, as much as the rounding of the output, and
// averaged over tokens).  With 8 bits a token's weight, its probability times its page's
// scale, is two bf16 terms, the second of what the rounding of the first leaves (2^-16 of
// it; with its exponentials and the logarithm of the scale 2^-15).  Both have fp32's range:
// the output may be made of weights far below the row's largest, where that one's value is
// zero (an attention sink, a page of zeros, to which the append gives the scale 1).  One
// half had a fixed step of 2^-24 of the largest there.
// Where the CTAs cut an item depends on the whole batch, so a row's last bit may too; a
// call's bits are the same every time.
//
// The work is cut evenly: the KV steps of all items, in order of (sequence, head,
// rows), are one line of units that the CTAs share in equal parts, wherever in an
// item a part begins or ends.  Lengths are known on the device alone, so each CTA
// finds its part from the lengths at its start.  Parts of an item leave their
// maxima, sums and outputs in the workspace in fp32, and a second launch joins
// them in order.
//
// Measured: two prompts of about 8192 tokens behind up to 8000, 4 x 8 heads of 128, bf16: 1240 us, 1512 TFLOP/s;
// what bounds it is the chain of one stream's softmax (1500 cycles a tile) and products (1024) against the
// other's.  1639 tokens at the end of a context of 114500, 2 x 8 heads of 128, e4m3: 1849 us, 865 TFLOP/s, of which
// second terms are about 100 and values in bf16 in place of half 200; 224 KB go through shared memory a tile (codes in,
// read, widened, read by the products), and the chain through four programs of warps is long.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "bsa_internal.h"
#include "bsa_overlap.h"
#include "bsa_tcgen05.cuh"

namespace bsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 128;               // rows of an MMA, tokens of a KV tile
constexpr int kTile = kPageSize;
constexpr int kAtom = kTile * 128;       // 128 tokens of 64 bf16 dimensions: 16 KB, swizzled by 128 bytes
constexpr int kMaxStages = 12;
constexpr int kInfo = 16;                // tiles whose facts are kept: more than the rings hold, and one
constexpr int kPortions = 4;             // portions announced ahead
constexpr int kWindow = 512;             // sequences whose units a CTA holds at a time while it finds its part
constexpr float kGrow = 8.f;             // log2 of what a maximum may grow by before O is rescaled
constexpr float kLift = 60.f;            // 8 bits: log2 of a row's largest probability and weight in their units
constexpr float kFar = 100.f;            // 8 bits: log2 of how far a page's exponentials may lie below its probabilities
constexpr int kJoinThreads = 256;
constexpr int kMinSteps = 2;             // the least part of a CTA, in steps

struct PagedParams {
    uint16_t* out;
    const uint8_t* v;             // the cache's values, for the epilogue of rows that see infinities
    const float* ks;
    const float* vs;
    const int32_t* table;
    const int32_t* seq_lens;      // decode form
    const int32_t* cu;            // varlen form
    const int32_t* prefix;
    int64_t T;
    int64_t num_pages;
    int32_t dql, num_reqs, max_blocks, H, G, D;
    int32_t tokens;               // of an MMA's rows: 128 / G
    int32_t window, sinks, cache_dtype;
    int32_t min_units;            // the least part of a CTA
    int32_t part_rows;            // rows of a part in the workspace
    float scale_log2e;            // not negative; the scores' instruction negates the queries where the scale is
    uint32_t s_idesc, o_idesc;
    bool wide_out;                // out is 32-byte aligned
    struct PartHead* heads;       // [grid]
    float* parts;                 // [grid][2][part_rows][D]
    float4* sums;                 // [grid][2][part_rows]: maximum, sum, outputs' unit
    uint32_t* status;
    unsigned long long wait_ns;   // a wait's limit
    uint32_t stall;               // stages after which a CTA's copies stop, for tests
};

struct PagedMaps {
    CUtensorMap q, k, v;
};

// The item that a CTA began and left to the next `more` CTAs to finish.
struct PartHead {
    int64_t row0;                 // first token row
    int32_t tokens, h, more;
    int32_t pad;
};

struct alignas(16) Start {
    int64_t lo, hi, first;        // this CTA's units, and the first unit of the item that holds lo
    int64_t U, N;
    int32_t b, h, qt;
};

template <int D_, bool BITS8>
struct Cfg {
    static constexpr int D = D_;                           // dimensions, padded with zeros
    static constexpr int NS = D <= 128 ? 2 : 1;            // streams
    static constexpr int PD = D < 128 ? D : 128;           // dimensions of a panel, a ring stage's
    static constexpr int PANELS = D / PD;
    static constexpr int ATOMS = PD / 64;
    static constexpr int STAGE = ATOMS * kAtom;
    static constexpr int Q_TILE = D / 64 * kAtom;
    static constexpr int CODES = BITS8 ? kTile * PD : 0;   // bytes of a stage of codes
    static constexpr int RING = BITS8 ? 98304 / STAGE : (229376 - NS * Q_TILE) / STAGE;
    static constexpr int CRING = BITS8 ? (229376 - NS * Q_TILE - RING * STAGE) / CODES : 0;
    // warps: softmax, then a group of four with the copies' and the MMAs' and with bf16 two for the
    // values; with 8 bits the values have two groups of their own
    static constexpr int SOFTMAX = NS * 4;
    static constexpr int COPY = SOFTMAX, MMA = SOFTMAX + 1, VALUES = SOFTMAX + (BITS8 ? 4 : 2);
    static constexpr int WARPS = SOFTMAX + (BITS8 ? 12 : 4);
    static constexpr int THREADS = WARPS * 32, VALUE_THREADS = BITS8 ? 128 : 64, VALUE_WARPS = BITS8 ? 8 : 2;
    // registers of a softmax thread and of the others, out of what the launch gives all
    static constexpr int GIVEN = 65536 / THREADS / 8 * 8 < 255 ? 65536 / THREADS / 8 * 8 : 248;
    static constexpr int OTHERS = BITS8 ? 64 : 72;
    static constexpr int MORE = (GIVEN * THREADS - OTHERS * (THREADS - SOFTMAX * 32)) / (SOFTMAX * 32) / 8 * 8;
    static constexpr int MINE = MORE < 255 ? MORE : 248;
    // Units of work: a step in which each stream has its own rows of one tile, one in which both have the
    // same rows of two tiles, and an item's beginning and end.  With 8 bits the second widens twice the codes:
    // 1.25 times as long (without, the CTAs with such steps were last).
    static constexpr int PAIR_UNITS = 4, SPLIT_UNITS = BITS8 && NS == 2 ? 5 : 4, END_UNITS = 4;
    static constexpr uint32_t O_COL = 256;                 // TMEM: scores in columns 0 to 255, outputs behind
    static_assert(RING >= 3 && RING <= kMaxStages && CRING <= kMaxStages && CRING % 2 == 0, "rings; the groups take stages of codes in turn");
};

// The KV tiles that rows at positions [first, last] see: sink tiles [0, st), then
// tiles [wst, ...), nk in all; `end`: the first token that none of them sees any more.
struct Range {
    int nk, st, wst, end;
    __device__ __forceinline__ int tile(int i) const { return i < st ? i : i - st + wst; }
};
// The tiles that rows at positions [first, last] see in full.
struct Whole {
    int end, window, sinks;      // tiles before `end` and from `window` on, or before `sinks`
    __device__ __forceinline__ void set(const PagedParams& A, int64_t first, int64_t last) {
        end = (int)(first < 0 ? 0 : (first + 1) / kTile);
        window = A.window > 0 && last >= A.window ? (int)((last - A.window) / kTile) + 1 : 0;
        sinks = A.sinks / kTile;
    }
    __device__ __forceinline__ bool has(int tile) const { return tile < end && (tile >= window || tile < sinks); }
};

// What a CTA does of one item.  The copies' warp makes it, the others read it from shared memory:
// in registers it cost each of them 40.
struct Portion {
    int64_t row0, pos0;          // first token row, its position
    Range r;
    Whole item, tile[2];         // of all rows, and of each query tile's
    int b, h, tokens;
    int i0, i1;                  // KV tiles of the range
    int number;                  // of the portion, and of those with tiles
    int loads;
    int lo;                      // the first token that the first row's window holds
    int more;                    // CTAs that finish an item begun here
    int split, begins, ends;     // both streams take the same rows; the item's first and last steps are here
    int over;                    // no portion: the end
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], code_full[kMaxStages], code_empty[kMaxStages];
    uint64_t q_full, q_ready, q_empty, s_full[2], p_half[2], p_full[2], o_full[2], portion_full[kPortions], portion_empty[kPortions], to_fix, fixed, drained;
    float scale[kInfo][2][kPagesPerBlock];     // 8 bits: key scales times scale log2 e, log2 of value scales
    int valid[kInfo];                          // tokens of a tile inside the cache
    Portion portion[kPortions];
    int poison[kPortions];                     // 1 + the number of the last portion with values that are not finite
    uint32_t odd_dims[kPortions][2][8];        // 8 bits: dimensions with those in tiles that all rows see: that add infinity, minus infinity (NaN: both)
    uint8_t q_power[2][2][kRows];              // 8 bits: the exponent (by 127) of what a row of queries was divided by, of two portions
    Start start;
    uint32_t tmem_base;
    int gave_up;
};

// ---- the work --------------------------------------------------------------

struct Seq {
    int64_t t0, p0;     // first row, its position
    int n;              // rows
};
__device__ __forceinline__ Seq sequence(const PagedParams& A, int b) {
    Seq s;
    if (A.cu == nullptr) {
        s.t0 = (int64_t)b * A.dql;
        s.n = A.dql;
        s.p0 = (int64_t)__ldg(A.seq_lens + b) - A.dql;
    } else {
        const int64_t a = __ldg(A.cu + b), e = __ldg(A.cu + b + 1);
        s.t0 = a < 0 ? 0 : a < A.T ? a : A.T;
        const int64_t to = e < s.t0 ? s.t0 : e < A.T ? e : A.T;
        s.n = (int)(to - s.t0);
        s.p0 = (int64_t)__ldg(A.prefix + b) + (s.t0 - a);
    }
    return s;
}

__device__ __forceinline__ Range range(const PagedParams& A, int64_t first, int64_t last) {
    Range r;
    const int64_t top = (int64_t)A.max_blocks * kTile;
    r.end = (int)(last + 1 < 0 ? 0 : last + 1 < top ? last + 1 : top);
    const int te = (r.end + kTile - 1) / kTile;
    r.st = r.wst = 0;
    if (A.window > 0) {
        const int64_t lo = (first > 0 ? first : 0) - A.window + 1;
        const int sink_end = A.sinks < r.end ? A.sinks : r.end;
        r.st = (sink_end + kTile - 1) / kTile;
        const int64_t w = lo > 0 ? lo / kTile : 0;
        r.wst = (int)(w < te ? w : te);
        if (r.wst < r.st) r.wst = r.st;
    }
    r.nk = r.st + te - r.wst;
    return r;
}

template <class C>
__device__ __forceinline__ int item_tokens(const PagedParams& A) {
    return C::NS * A.tokens;
}
// KV steps of an item: tiles, or pairs of tiles where both streams take its rows.
template <class C>
__device__ __forceinline__ int item_steps(const PagedParams& A, const Seq& s, int qt, Range* out = nullptr, bool* split = nullptr) {
    const int t = qt * item_tokens<C>(A), n = min(item_tokens<C>(A), s.n - t);
    const Range r = range(A, s.p0 + t, s.p0 + t + n - 1);
    const bool two = C::NS == 2 && n <= A.tokens;
    if (out != nullptr) *out = r;
    if (split != nullptr) *split = two;
    return two ? (r.nk + 1) / 2 : r.nk;
}
// What a step of such an item is worth, and the whole item.
template <class C>
__device__ __forceinline__ int step_units(bool split) {
    return split ? C::SPLIT_UNITS : C::PAIR_UNITS;
}
template <class C>
__device__ __forceinline__ int64_t item_units(const PagedParams& A, const Seq& s, int qt) {
    bool split;
    const int steps = item_steps<C>(A, s, qt, nullptr, &split);
    return (int64_t)steps * step_units<C>(split) + C::END_UNITS;
}
template <class C>
__device__ __forceinline__ int item_count(const PagedParams& A, const Seq& s) {
    return (s.n + item_tokens<C>(A) - 1) / item_tokens<C>(A);
}

// The units of sequences [b0, b0 + n), per head.
template <class C>
__device__ void count_units(const PagedParams& A, long long* units, int b0, int n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i0 = warp * 32; i0 < n; i0 += C::THREADS) {
        const int i = i0 + lane;
        Seq s{};
        int items = 0;
        long long u = 0;
        if (i < n) {
            s = sequence(A, b0 + i);
            items = item_count<C>(A, s);
            if (items <= 4)
                for (int k = 0; k < items; ++k) u += item_units<C>(A, s, k);
        }
        // sequences of many items: the warp together
        for (uint32_t many = __ballot_sync(kFull, items > 4); many != 0; many &= many - 1) {
            const int l = __ffs(many) - 1;
            const Seq x = sequence(A, b0 + i0 + l);
            const int m = item_count<C>(A, x);
            long long v = 0;
            for (int k = lane; k < m; k += 32) v += item_units<C>(A, x, k);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
            if (lane == l) u = v;
        }
        if (i < n) units[i] = u;
    }
    __syncthreads();
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
// Exclusive sum over the lanes.
__device__ __forceinline__ long long warp_before(long long v) {
    const int lane = threadIdx.x & 31;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    return x - v;
}

// x * y / z, of numbers that mostly fit in 32 bits.
__device__ __forceinline__ int64_t mul_div(int64_t x, int64_t y, int64_t z) {
    const int64_t p = x * y;
    return p < INT32_MAX && z < INT32_MAX ? (int32_t)p / (int32_t)z : p / z;
}

// This CTA's part of the units, and the item in which it begins.  `units`: kWindow words.  One
// request on its own waits for this: up to kWindow sequences take two barriers.
template <class C>
__device__ void find_start(const PagedParams& A, Shared& S, long long* units) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int EACH = kWindow / 32;
    long long all = 0;
    for (int b0 = 0; b0 < A.num_reqs; b0 += kWindow) {
        const int n = min(kWindow, A.num_reqs - b0);
        if (b0 > 0) __syncthreads();
        count_units<C>(A, units, b0, n);
        if (warp == 0) {
            long long v = 0;
            for (int i = lane; i < n; i += 32) v += units[i];
            all += warp_sum(v);
        }
    }
    if (warp == 0 && lane == 0) {
        const int64_t U = all * A.H;
        int64_t N = mul_div(U, 1, A.min_units);
        N = N < 1 ? 1 : N < gridDim.x ? N : gridDim.x;
        const int64_t c = blockIdx.x;
        S.start = Start{c < N ? mul_div(c, U, N) : 0, c < N ? mul_div(c + 1, U, N) : 0, 0, U, N, 0, 0, 0};
    }
    if (A.num_reqs > kWindow) __syncthreads();
    else __syncwarp();
    long long before = 0;      // of the sequences so far, all heads
    for (int b0 = 0; b0 < A.num_reqs; b0 += kWindow) {
        const int n = min(kWindow, A.num_reqs - b0);
        if (A.num_reqs > kWindow) {
            __syncthreads();
            count_units<C>(A, units, b0, n);
        }
        if (warp == 0) {
            const int64_t lo = S.start.lo;
            long long mine = 0;
            if (n <= 32) {
                if (lane < n) mine = units[lane];
            } else {
                for (int i = 0; i < EACH; ++i)
                    if (lane * EACH + i < n) mine += units[lane * EACH + i];
            }
            long long at = before + warp_before(mine) * A.H;
            if (lo < S.start.hi && at <= lo && lo < at + mine * A.H) {
                int i = n <= 32 ? lane : lane * EACH;
                while (lo >= at + units[i] * A.H) at += units[i++] * A.H;
                S.start.b = b0 + i;
                S.start.h = (int32_t)mul_div(lo - at, 1, units[i]);
                S.start.first = at + S.start.h * units[i];      // of the head's items
            }
            before += warp_sum(mine) * A.H;
        }
    }
    // the item among the head's
    __syncwarp();
    if (warp == 0 && S.start.lo < S.start.hi) {
        const int64_t lo = S.start.lo;
        const Seq s = sequence(A, S.start.b);
        const int items = item_count<C>(A, s);
        long long at = S.start.first;
        __syncwarp();
        for (int k0 = 0; k0 < items; k0 += 32) {
            const int k = k0 + lane;
            const long long w = k < items ? item_units<C>(A, s, k) : 0;
            const long long mine = at + warp_before(w);
            if (mine <= lo && lo < mine + w) {
                S.start.qt = k;
                S.start.first = mine;
            }
            at += warp_sum(w);
            if (at > lo) break;
        }
    }
}

// The first token in the window of a row at position `first`.
__device__ __forceinline__ int first_seen(const PagedParams& A, int64_t first) {
    const int64_t lo = A.window > 0 ? (first > 0 ? first : 0) - A.window + 1 : 0;
    return (int)(lo < 0 ? 0 : lo < INT32_MAX ? lo : INT32_MAX);
}
// The portions of a CTA in order.
template <class C>
struct Walk {
    int b, h, qt, items, number, loads;
    int64_t at, lo, hi;
    Seq s;
    __device__ __forceinline__ Walk(const PagedParams& A, const Start& st)
        : b(st.b), h(st.h), qt(st.qt), items(0), number(-1), loads(0), at(st.first), lo(st.lo), hi(st.hi) {
        if (lo < hi) {
            s = sequence(A, b);
            items = item_count<C>(A, s);
        }
    }
    // The next one, in *P.
    __device__ bool next(const PagedParams& A, const Start& st, Portion* P) {
        while (at < hi) {
            const int64_t first = at;
            Range r;
            bool split;
            const int steps = item_steps<C>(A, s, qt, &r, &split);
            const int tok0 = qt * item_tokens<C>(A), tokens = min(item_tokens<C>(A), s.n - tok0);
            const int64_t row0 = s.t0 + tok0, pos0 = s.p0 + tok0;
            const int item_b = b, item_h = h;
            const int unit = step_units<C>(split);
            at += (int64_t)steps * unit + C::END_UNITS;
            if (++qt == items) {
                qt = 0;
                if (++h == A.H) {
                    h = 0;
                    while (at < hi) {      // there is a sequence with items behind
                        s = sequence(A, ++b);
                        items = item_count<C>(A, s);
                        if (items > 0) break;
                    }
                }
            }
            // a step is of the part in which its last unit lies
            const int64_t from = lo > first ? (lo - first) / unit : 0, to = (hi - first) / unit;
            const int a = (int)(from < steps ? from : steps), e = (int)(to < steps ? to : steps);
            if (a >= e && !(steps == 0 && first >= lo)) continue;
            P->row0 = row0;
            P->pos0 = pos0;
            P->r = r;
            P->item.set(A, pos0, pos0 + tokens - 1);
            P->tile[0].set(A, pos0, pos0 + min(tokens, A.tokens) - 1);
            P->tile[1].set(A, pos0 + A.tokens, pos0 + tokens - 1);
            P->b = item_b;
            P->h = item_h;
            P->tokens = tokens;
            P->i0 = split ? 2 * a : a;
            P->i1 = split ? min(2 * e, r.nk) : e;
            P->number = ++number;
            P->loads = loads;
            if (P->i1 > P->i0) ++loads;
            P->lo = first_seen(A, pos0);
            // the CTA of the last step's last unit u: lo(c) = c U / N <= u for the c up to ((u + 1) N - 1) / U
            P->more = a == 0 && e < steps ? (int)(((first + (int64_t)steps * unit) * st.N - 1) / st.U - blockIdx.x) : 0;
            P->split = split;
            P->begins = a == 0;
            P->ends = e == steps;
            P->over = 0;
            return true;
        }
        P->over = 1;
        return false;
    }
};

// A role's place among the portions: waits for the next, reads it where it lies, and gives it back.
struct Reader {
    uint32_t number = 0;
    __device__ __forceinline__ const Portion* next(Shared& S, unsigned long long wait_ns);
    __device__ __forceinline__ void done(Shared& S);
};

// The registers of a role's threads; a group of four warps asks as one.
template <int N, bool MORE>
__device__ __forceinline__ void take_registers() {
    if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- small arithmetic ------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void fma2(float& a, float& b, float x0, float x1, float y0, float y1, float z0, float z1) {
    asm("{\n\t.reg .b64 x, y, z, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 r, x, y, z;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(a), "=f"(b)
        : "f"(x0), "f"(x1), "f"(y0), "f"(y1), "f"(z0), "f"(z1));
}
__device__ __forceinline__ void add2(float& a, float& b, float x0, float x1) {
    asm("{\n\t.reg .b64 x, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 r, {%0, %1};\n\t"
        "add.rn.f32x2 r, r, x;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(x0), "f"(x1));
}
__device__ __forceinline__ void mul2(float& a, float& b, float y) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(y));
}
// two values as bf16, a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// four 8-bit codes as bf16, exactly: their bits in place, times what the exponents' biases differ by.
// Codes that are not finite come out as numbers (480; 2^16 and more), which odd_codes tells.
template <bool E4M3>
__device__ __forceinline__ void widen_values(uint32_t w, uint32_t& a, uint32_t& b) {
    const uint32_t hi = (w & 0x80808080u) | (E4M3 ? w >> 4 & 0x07070707u : w >> 3 & 0x0F0F0F0Fu);
    const uint32_t lo = E4M3 ? w << 4 & 0xF0F0F0F0u : w << 5 & 0xE0E0E0E0u;
    constexpr uint32_t UP = E4M3 ? 0x7B807B80u : 0x77807780u;      // 2^120, 2^112
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(__byte_perm(lo, hi, 0x5140)), "r"(UP));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(__byte_perm(lo, hi, 0x7362)), "r"(UP));
}
// `odd` with bit 7 of a byte set whose code is infinite or NaN: all ones from some bit up to bit 6, so that one more carries.  (The
// byte behind such a code may be set with it.)
template <bool E4M3>
__device__ __forceinline__ uint32_t odd_codes(uint32_t w, uint32_t odd) {
    return odd | ((w + (E4M3 ? 0x01010101u : 0x04040404u)) ^ w);
}
// two 8-bit codes as halves, exactly (NaN and infinities too)
template <bool E4M3>
__device__ __forceinline__ uint32_t widen(uint32_t codes) {
    uint32_t h;
    if constexpr (E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}
// Nonzero in bits 15 and 31 where a half of a word of values is infinite or NaN (its exponent all
// ones, so that one more carries); and the word with zeros there.
__device__ __forceinline__ uint32_t odd_word(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t finite_word(uint32_t w) {
    constexpr uint32_t E = 0x7F80u;
    if ((w & E) == E) w &= 0xFFFF0000u;
    if ((w & E << 16) == E << 16) w &= 0x0000FFFFu;
    return w;
}
// 32 bytes, a whole sector, or two halves of it
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool wide) {
    if (wide) {
        int32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (int32_t)w[j];
        st_v8(static_cast<int32_t*>(p), v);
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// bits [0, n) of 32
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// ---- the kernel ------------------------------------------------------------

__device__ __forceinline__ const Portion* Reader::next(Shared& S, unsigned long long wait_ns) {
    int none = 0;
    const uint32_t slot = number % kPortions;
    if (!mbar_wait(&S.portion_full[slot], (number / kPortions) & 1, &none, wait_ns)) {
        S.gave_up = 1;
        return nullptr;
    }
    const Portion* P = &S.portion[slot];
    return P->over ? nullptr : P;
}
// by one thread of a warp, behind the others
__device__ __forceinline__ void Reader::done(Shared& S) { mbar_arrive(&S.portion_empty[number++ % kPortions]); }

// Adds what the values' warps took out to the row's outputs [d0, d0 + 16): values that
// are not finite of tokens that the row sees.  With 8 bits `dims` has those of the tiles that all rows see.
template <class C, bool BITS8>
__device__ __noinline__ void add_odd_values(const PagedParams& A, const Portion& P, const uint32_t (&dims)[2][8], int hi, int lo, int d0, float* o) {
    if constexpr (BITS8) {
        for (int k = 0; k < 16; ++k) {
            if (dims[0][d0 / 32] >> (d0 % 32 + k) & 1) o[k] += INFINITY;
            if (dims[1][d0 / 32] >> (d0 % 32 + k) & 1) o[k] -= INFINITY;
        }
    }
    for (int i = P.i0; i < P.i1; ++i) {
        const int tile = P.r.tile(i);
        if (P.item.has(tile)) continue;      // as the values' warps have it
        const int64_t id = __ldg(A.table + (int64_t)P.b * A.max_blocks + tile);
        for (int c = 0; c < kTile; ++c) {
            const int j = tile * kTile + c;
            const int64_t page = id * kPagesPerBlock + c / kSubPage;
            if (j > hi || (A.window > 0 && j < lo && j >= A.sinks) || page < 0 || page >= A.num_pages) continue;
            const int64_t at = ((page * kSubPage + c % kSubPage) * A.H + P.h) * A.D;
            for (int k = 0; k < 16 && d0 + k < A.D; ++k) {
                float x;
                if constexpr (BITS8) {
                    const uint32_t code = __ldg(A.v + at + d0 + k);
                    const uint32_t w = A.cache_dtype == BSA_DTYPE_E4M3 ? widen<true>(code) : widen<false>(code);
                    x = __low2float(*reinterpret_cast<const __half2*>(&w)) * __ldg(A.vs + page * A.H + P.h);
                } else {
                    x = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(A.v) + at + d0 + k) << 16);
                }
                if (x - x == 0.f) continue;
                o[k] += x;
            }
        }
    }
}

// Where 16 dimensions of a row, a word of codes, go in a stage of bf16: two 16-byte words,
// swizzled.
template <class C>
__device__ __forceinline__ uint8_t* place(uint8_t* to, int k, int half) {
    constexpr int PER_ROW = C::PD / 16;
    const int row = k / PER_ROW, c = k % PER_ROW;
    return to + (c / 4) * kAtom + row * 128 + ((((c % 4) * 2 + half) ^ (row & 7)) << 4);
}

// A stage of key codes widened by 128 threads.
template <class C, bool E4M3>
__device__ __forceinline__ void widen_stage(const uint4* from, uint8_t* to, int me) {
    constexpr int EACH = C::CODES / 16 / 128, BATCH = 2;
#pragma unroll 1
    for (int i = 0; i < EACH; i += BATCH) {
        uint4 x[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) x[j] = from[me + (i + j) * 128];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int k = me + (i + j) * 128;
            const uint32_t in[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = widen<E4M3>(in[e / 2] >> (e % 2 * 16));
            // lanes of the second half of a row store in the other order: no two on one bank
            const int other = k % (C::PD / 16) / 4 & 1;
            const uint4 a = make_uint4(w[0], w[1], w[2], w[3]), b = make_uint4(w[4], w[5], w[6], w[7]);
            *reinterpret_cast<uint4*>(place<C>(to, k, other)) = other ? b : a;
            *reinterpret_cast<uint4*>(place<C>(to, k, 1 - other)) = other ? a : b;
        }
    }
}
// The tokens of a tile that some row of an item sees: rows before `end` that lie at `window` or behind, or before `sinks`.
struct Seen {
    int end, window, sinks;
    __device__ __forceinline__ bool has(int row) const { return row < end && (row >= window || row < sinks); }
};

// What is not finite among a thread's value codes, of tokens that some row sees; whether there was such.  In a tile that all
// rows see (`dims`) it goes down by dimension, from d0 on.
template <class C, bool E4M3>
__device__ __noinline__ bool note_odd_codes(const uint4* from, int me, Seen seen, uint32_t (*dims)[8], int d0, const float* log_scales) {
    constexpr int PER_ROW = C::PD / 16;
    bool any = false;
    for (int k = me; k < C::CODES / 16; k += 128) {
        const int row = k / PER_ROW;
        if (!seen.has(row)) continue;
        const uint4 x = from[k];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        for (int e = 0; e < 16; ++e) {
            const uint32_t code = w[e / 4] >> (e % 4 * 8) & 0xFF, low = code & 0x7F;
            if (E4M3 ? low != 0x7F : low < 0x7C) continue;
            any = true;
            if (dims == nullptr) continue;
            const bool nan = E4M3 || low > 0x7C || log_scales[row / kSubPage] == -INFINITY;      // times a scale of zero
            const int d = d0 + k % PER_ROW * 16 + e;
            for (int sign = 0; sign < 2; ++sign)
                if (nan || (int)(code >> 7) == sign) atomicOr(&dims[sign][d / 32], 1u << (d % 32));
        }
    }
    return any;
}

// A stage of value codes widened by 128 threads; whether some of this thread's may not be finite.  16 codes at a time: with
// 32 the instruction cache makes more of it than the latency (production decode 161 instead of 166 us).
template <class C, bool E4M3>
__device__ __forceinline__ bool widen_value_stage(const uint4* from, uint8_t* to, int me) {
    uint32_t odd = 0;
#pragma unroll 1
    for (int k = me; k < C::CODES / 16; k += 128) {
        const uint4 x = from[k];
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            widen_values<E4M3>(in[e], w[2 * e], w[2 * e + 1]);
            odd = odd_codes<E4M3>(in[e], odd);
        }
        const int other = k % (C::PD / 16) / 4 & 1;
        const uint4 a = make_uint4(w[0], w[1], w[2], w[3]), b = make_uint4(w[4], w[5], w[6], w[7]);
        *reinterpret_cast<uint4*>(place<C>(to, k, other)) = other ? b : a;
        *reinterpret_cast<uint4*>(place<C>(to, k, 1 - other)) = other ? a : b;
    }
    return (odd & 0x80808080u) != 0;
}
// Value rows that no row sees set to zero, and what is not finite in the others; whether there was
// such.
template <class C, class Seen>
__device__ __forceinline__ bool clean_stage(uint8_t* stage, int me, Seen seen) {
    uint4* v = reinterpret_cast<uint4*>(stage);
    uint32_t odd = 0;
    // the search alone is on the way of every such tile (its product waits for it)
#pragma unroll 8
    for (int k = me; k < C::STAGE / 16; k += C::VALUE_THREADS) {
        const uint4 x = v[k];
        if (seen(k % (kAtom / 16) / 8)) odd |= odd_word(x.x) | odd_word(x.y) | odd_word(x.z) | odd_word(x.w);
        else v[k] = make_uint4(0, 0, 0, 0);
    }
    if ((odd & 0x80008000u) == 0) return false;
#pragma unroll 1
    for (int k = me; k < C::STAGE / 16; k += C::VALUE_THREADS) {
        const uint4 x = v[k];
        v[k] = make_uint4(finite_word(x.x), finite_word(x.y), finite_word(x.z), finite_word(x.w));
    }
    return true;
}

// A row of queries from bf16 to half, multiplied by a power of two that takes its largest magnitude
// to [2^14, 2^15): exact down to 2^-28 of that, and off by at most 2^-40 of it below.
// Returns the exponent, by 127, of what the row was divided by.
template <class C>
__device__ __forceinline__ int halve_row(uint8_t* tile, int row) {
    auto word = [&](int c) { return reinterpret_cast<uint4*>(tile + c / 8 * kAtom + row * 128 + ((c % 8 ^ (row & 7)) << 4)); };
    uint32_t most = 0;
#pragma unroll 4
    for (int c = 0; c < C::D / 8; ++c) {
        const uint4 x = *word(c);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) most = max(most, max(w[e] & 0x7FFFu, w[e] >> 16 & 0x7FFFu));
    }
    const int e = min(max((int)(most >> 7) - 127, -112), 126);      // of the largest; NaN and infinities as the largest finite
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
#pragma unroll 4
    for (int c = 0; c < C::D / 8; ++c) {
        uint4* at = word(c);
        const uint4 x = *at;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = pack_half(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up);
        *at = make_uint4(h[0], h[1], h[2], h[3]);
    }
    return 127 - 14 + e;
}

template <int D_, bool BITS8>
__global__ void __launch_bounds__(Cfg<D_, BITS8>::THREADS, 1)
paged_attention_kernel(const __grid_constant__ PagedParams A, const __grid_constant__ PagedMaps M) {
    using C = Cfg<D_, BITS8>;
    constexpr int RING = C::RING, PANELS = C::PANELS, NS = C::NS;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qsm = smem;                             // [NS] query tiles
    uint8_t* ring = qsm + NS * C::Q_TILE;            // [RING] stages of keys and values of 16 bits
    uint8_t* codes = ring + RING * C::STAGE;         // [CRING] stages of codes
    Shared& S = *reinterpret_cast<Shared*>(codes + C::CRING * C::CODES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == C::MMA) tmem_alloc(&S.tmem_base, 512);
    if (tid == 32) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&S.full[i], BITS8 ? 128 : 1);
            mbar_init(&S.empty[i], 1);
            mbar_init(&S.code_full[i], 1);
            mbar_init(&S.code_empty[i], 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_half[i], kRows);
            mbar_init(&S.p_full[i], kRows);
            mbar_init(&S.o_full[i], 1);
        }
        for (int i = 0; i < kPortions; ++i) {
            mbar_init(&S.portion_full[i], 1);
            mbar_init(&S.portion_empty[i], C::SOFTMAX + 1 + C::VALUE_WARPS);
        }
        mbar_init(&S.q_full, 1);
        mbar_init(&S.q_ready, 256);
        mbar_init(&S.q_empty, 2);            // the products, and the join of the streams
        mbar_init(&S.to_fix, 1);
        mbar_init(&S.fixed, 64);
        mbar_init(&S.drained, 1);
        for (int i = 0; i < kPortions; ++i) S.poison[i] = 0;
        S.gave_up = 0;
        mbar_fence_init();
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");
    // rows of no sequence
    if (A.cu != nullptr) {
        const int64_t from = min(max((int64_t)__ldg(A.cu), (int64_t)0), A.T), to = min(max((int64_t)__ldg(A.cu + A.num_reqs), from), A.T);
        const int64_t row = (int64_t)A.H * A.G * A.D / 8, gap = (from + A.T - to) * row;
        for (int64_t i = (int64_t)blockIdx.x * C::THREADS + tid; i < gap; i += (int64_t)gridDim.x * C::THREADS)
            reinterpret_cast<uint4*>(A.out)[i < from * row ? i : to * row + i - from * row] = make_uint4(0, 0, 0, 0);
    }
    find_start<C>(A, S, reinterpret_cast<long long*>(ring));      // the ring is still free
    fence_async_smem();
    __syncthreads();
    const uint32_t tmem = S.tmem_base;
    volatile int* quit = &S.gave_up;
    Reader reader;

    if (warp == C::COPY) {
        take_registers<C::OTHERS, false>();
        // ------------------------------------------------ portions and copies
        Walk<C> walk(A, S.start);
        // the ring that TMA fills: of codes or of bf16
        constexpr int N = BITS8 ? C::CRING : RING;
        uint64_t* const filled = BITS8 ? S.code_full : S.full;
        uint64_t* const drained = BITS8 ? S.code_empty : S.empty;
        uint8_t* const base = BITS8 ? codes : ring;
        constexpr int BYTES = BITS8 ? C::CODES : C::STAGE;
        uint32_t st = 0, use = 0, issued = 0, tiles = 0, loads = 0;
        bool ok = true;
        // past the tensor's end (an empty cache's stands for a page): arrives as zeros
        const int outside = (int)(max(A.num_pages, (int64_t)1) * kSubPage);
        auto copy = [&](const CUtensorMap* map, int token, int h) {
#pragma unroll
            for (int p = 0; p < PANELS; ++p) {
                ok = issued != A.stall && (use == 0 || mbar_wait(&drained[st], (use - 1) & 1, quit, A.wait_ns));
                ok = __all_sync(kFull, ok);
                if (!ok) {
                    S.gave_up = 1;
                    return;
                }
                if (elect_one()) {
                    mbar_expect(&filled[st], BYTES);
                    if constexpr (BITS8) {
                        tma_load_3d(base + st * BYTES, map, p * C::PD, h, token, &filled[st]);
                    } else {
#pragma unroll
                        for (int a = 0; a < C::ATOMS; ++a)
                            tma_load_3d(base + st * BYTES + a * kAtom, map, p * C::PD + a * 64, h, token, &filled[st]);
                    }
                }
                __syncwarp();
                ++issued;
                if (++st == N) {
                    st = 0;
                    ++use;
                }
            }
        };
        for (uint32_t number = 0;; ++number) {
            // also when a wait has run out: the softmax warps fill the rows that are left with NaN
            const uint32_t slot = number % kPortions;
            int none = 0;
            if (number >= kPortions && !mbar_wait(&S.portion_empty[slot], (number / kPortions - 1) & 1, &none, A.wait_ns)) break;
            Portion& P = S.portion[slot];
            bool more = false;
            if (BITS8 && lane < 16) S.odd_dims[slot][lane >> 3][lane & 7] = 0;
            if (lane == 0) more = walk.next(A, S.start, &P);
            more = __shfl_sync(kFull, more, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.portion_full[slot]);
            if (!more) break;
            if (lane == 0 && P.begins) report_status(A.status, P.pos0 + P.tokens > (int64_t)A.max_blocks * kTile, BSA_STATUS_BAD_CONTEXT);
            const int i0 = P.i0, i1 = P.i1, n = i1 - i0, b = P.b, h = P.h;
            if (n == 0 || !ok) continue;
            ok = loads == 0 || mbar_wait(&S.q_empty, (loads - 1) & 1, quit, A.wait_ns);
            ok = __all_sync(kFull, ok);
            if (!ok) continue;
            ++loads;
            const int mtiles = P.tokens > A.tokens ? 2 : 1;
            if (elect_one()) {
                mbar_expect(&S.q_full, mtiles * (C::Q_TILE / kRows) * A.tokens * A.G);
                for (int m = 0; m < mtiles; ++m)
                    for (int a = 0; a < C::D / 64; ++a)
                        tma_load_4d(qsm + m * C::Q_TILE + a * kAtom, &M.q, a * 64, 0, h, (int)(P.row0 + m * A.tokens), &S.q_full);
            }
            __syncwarp();
            const Range r = P.r;
            const int32_t* table = A.table + (int64_t)b * A.max_blocks;
            int32_t ids = 0;      // of 32 tiles
            int before = 0;       // the last tile's token coordinate
            const bool ahead = NS == 1 || P.split;       // keys run one tile ahead of values
            // 8 bits: scales of two tiles, lanes 0 to 15 and 16 to 31, the pages' for keys, then for
            // values; read two tiles ahead, as they may come from DRAM.  A page that no row of the item sees may
            // have any: it counts as one of scale zero.  One that is seen and has a value scale that is not
            // finite or is negative makes the scores of its tokens NaN, so that just the rows that see it are.
            float scale = 0.f;
            const int seen_from = P.lo;
            auto read_scales = [&](int k) {
                const int t = k + (lane >> 4), pg = lane & 7;
                const int id = __shfl_sync(kFull, ids, t & 31);
                scale = lane & 8 ? -INFINITY : 0.f;
                bool odd = false;
                const int token = t < n ? r.tile(i0 + t) * kTile + pg * kSubPage : r.end;
                const bool seen = token < r.end && (token + kSubPage > seen_from || token < A.sinks);
                if (seen && id >= 0 && (int64_t)id * kPagesPerBlock + pg < A.num_pages) {
                    const int64_t where = ((int64_t)id * kPagesPerBlock + pg) * A.H + h;
                    if (lane & 8) {
                        const float x = __ldg(A.vs + where);
                        odd = !(x >= 0.f && x < INFINITY);
                        scale = odd ? -INFINITY : log2f(x);
                    } else {
                        scale = __ldg(A.ks + where) * A.scale_log2e;
                    }
                }
                const uint32_t odds = __ballot_sync(kFull, odd);
                if (odds >> (lane | 8) & 1 && !(lane & 8)) scale = NAN;
            };
            for (int k = 0; ok && k <= n; ++k) {
                int at = 0;
                if (k < n) {
                    if ((k & 31) == 0) {
                        ids = k + lane < n ? __ldg(table + r.tile(i0 + k + lane)) : -1;
                        if constexpr (BITS8) read_scales(k);
                    }
                    const int id = __shfl_sync(kFull, ids, k & 31);
                    const int64_t left = id < 0 ? 0 : (A.num_pages - (int64_t)id * kPagesPerBlock) * kSubPage;
                    const int valid = (int)(left < 0 ? 0 : left < kTile ? left : kTile);
                    at = valid > 0 ? id * kTile : outside;
                    if (lane == 0) {
                        const int t = r.tile(i0 + k), tf = t * kTile;
                        int need = min(kTile, r.end - tf);
                        if (A.window > 0 && t < r.wst) need = min(need, A.sinks - tf);
                        report_status(A.status, valid < need, BSA_STATUS_BAD_BLOCK_ID);
                        S.valid[(tiles + k) % kInfo] = valid;
                    }
                    if constexpr (BITS8) {
                        if ((k & 1) == 0) {
                            if (k + (lane >> 4) < n) S.scale[(tiles + k + (lane >> 4)) % kInfo][lane >> 3 & 1][lane & 7] = scale;
                            if (((k + 2) & 31) != 0) read_scales(k + 2);
                        }
                    }
                    __syncwarp();
                    copy(&M.k, at, h);
                    if (!ahead && ok) copy(&M.v, at, h);
                }
                if (ahead && k > 0 && ok) copy(&M.v, before, h);
                before = at;
            }
            tiles += n;
        }
        // copies in flight land before the CTA's memory goes away, also when nobody waits
        // for them any more
        int none = 0;
        for (uint32_t k = issued > N ? issued - N : 0; k < issued; ++k) mbar_wait(&filled[k % N], (k / N) & 1, &none);
        if (loads > 0) mbar_wait(&S.q_full, (loads - 1) & 1, &none);
    } else if (warp == C::MMA) {
        take_registers<C::OTHERS, false>();
        // ------------------------------------------------ MMAs
        if (elect_one()) {
            // lower halves of operand descriptors; a byte offset adds offset / 16
            const uint32_t q_desc = (uint32_t)smem_desc(smem_addr(qsm), 0, 1024, 2);
            const uint32_t k_desc = (uint32_t)smem_desc(smem_addr(ring), 0, 1024, 2);
            const uint32_t v_desc = (uint32_t)smem_desc(smem_addr(ring), kAtom, 1024, 2);
            const uint32_t upper = (uint32_t)(smem_desc(0, 0, 1024, 2) >> 32);
            uint32_t st = 0, use = 0, p_phase = 0, fixes = 0, nq = 0, loads = 0;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && mbar_wait(bar, parity, quit, A.wait_ns); };
            auto step = [&](uint32_t& s, uint32_t& u) {
                if (++s == RING) {
                    s = 0;
                    ++u;
                }
            };
            auto take = [&](uint32_t s, uint32_t u) {
                wait(&S.full[s], u & 1);
                tc_fence_after();
            };
            // scores of query tile m and one panel of a key stage
            auto scores = [&](int buf, int m, int p, uint32_t s) {
                const uint32_t qd = q_desc + (m * C::Q_TILE + p * C::ATOMS * kAtom) / 16, kd = k_desc + s * (C::STAGE / 16);
#pragma unroll
                for (int k = 0; k < C::PD / 16; ++k) {
                    const int at = (k / 4) * (kAtom / 16) + (k % 4) * 2;
                    mma_f16(tmem + buf * kTile, qd + at, kd + at, upper, A.s_idesc, p + k > 0);
                }
            };
            // outputs of half the probabilities in `buf` (tokens 0 to 63, or 64 to 127) and a value stage; with
            // 8 bits of both terms
            auto outputs = [&](int half, int buf, int o, int p, uint32_t s, bool more) {
                const uint32_t vd = v_desc + s * (C::STAGE / 16);
                constexpr int TERMS = BITS8 ? 2 : 1;
#pragma unroll
                for (int k = half * 4; k < half * 4 + 4; ++k)
#pragma unroll
                    for (int t = 0; t < TERMS; ++t)
                        mma_f16_ts(tmem + C::O_COL + o * C::D + p * C::PD, tmem + buf * kTile + (k * TERMS + t) * 8, vd + k * 128, upper,
                                   A.o_idesc, more || k > 0 || t > 0);
            };
            auto probabilities = [&](uint64_t* bar, int buf) {
                wait(&bar[buf], (p_phase >> buf) & 1);
                tc_fence_after();
            };
            while (const Portion* at = reader.next(S, A.wait_ns)) {
                const Portion& P = *at;
                const int n = P.i1 - P.i0, i0 = P.i0;
                // bf16: tiles that some rows do not see in full pass through the values' warps,
                // while their probabilities are formed
                auto partly = [&](int k) { return !BITS8 && !P.item.has(P.r.tile(i0 + k)); };
                auto fixed = [&]() {
                    wait(&S.fixed, fixes & 1);
                    ++fixes;
                };
                if (ok && n > 0) {
                    wait(BITS8 ? &S.q_ready : &S.q_full, loads & 1);
                    tc_fence_after();
                    ++loads;
                }
                if (n == 0 || !ok) {
                    // nothing to do
                } else if (NS == 2 && !P.split) {
                    take(st, use);
                    if (ok) {
                        for (int s = 0; s < 2; ++s) {
                            scores(s, s, 0, st);
                            tc_commit(&S.s_full[s]);
                        }
                        tc_commit(&S.empty[st]);
                        if (n == 1) tc_commit(&S.q_empty);
                        step(st, use);
                    }
                    for (int k = 0; ok && k < n; ++k) {
                        const bool next = k + 1 < n, fix = partly(k);
                        uint32_t ks = st, ku = use;
                        step(ks, ku);
                        take(st, use);
                        if (ok && fix) mbar_arrive(&S.to_fix);
#pragma unroll 1
                        for (int s = 0; s < 2; ++s) {
                            probabilities(S.p_half, s);
                            if (fix && s == 0) fixed();
                            if (!ok) break;
                            outputs(0, s, s, 0, st, k > 0);
                            probabilities(S.p_full, s);
                            if (!ok) break;
                            p_phase ^= 1u << s;
                            outputs(1, s, s, 0, st, true);
                            if (s == 1) tc_commit(&S.empty[st]);
                            if (next) {
                                if (s == 0) take(ks, ku);
                                if (!ok) break;
                                scores(s, s, 0, ks);
                                tc_commit(&S.s_full[s]);
                                if (s == 1) {
                                    tc_commit(&S.empty[ks]);
                                    if (k + 2 == n) tc_commit(&S.q_empty);
                                }
                            } else {
                                tc_commit(&S.o_full[s]);
                            }
                        }
                        step(st, use);
                        if (next) step(st, use);
                    }
                } else {
                    // Keys one tile ahead (with two streams: of each stream).  With one stream the buffer of
                    // tile k + 1 was read by the product of tile k - 1, issued before.
                    auto keys = [&](int k) {
                        const int buf = NS == 2 ? k & 1 : (nq + k) & 1;
#pragma unroll
                        for (int p = 0; p < PANELS; ++p) {
                            take(st, use);
                            if (!ok) return;
                            scores(buf, 0, p, st);
                            tc_commit(&S.empty[st]);
                            step(st, use);
                        }
                        tc_commit(&S.s_full[buf]);
                        if (k + 1 == n) tc_commit(&S.q_empty);
                    };
                    int asked = 0;      // tiles whose scores are issued
#pragma unroll 1
                    for (int k = 0; ok && k < n; ++k) {
#pragma unroll 1
                        for (; ok && asked < n && asked <= k + 1; ++asked) keys(asked);
                        if (!ok) break;
                        const int buf = NS == 2 ? k & 1 : (nq + k) & 1;
                        const bool fix = partly(k);
                        uint32_t vs = st, vu = use;
                        for (int p = 0; p < PANELS; ++p) {
                            take(vs, vu);
                            step(vs, vu);
                        }
                        if (ok && fix) mbar_arrive(&S.to_fix);
#pragma unroll 1
                        for (int half = 0; ok && half < 2; ++half) {
                            probabilities(half == 0 ? S.p_half : S.p_full, buf);
                            if (fix && half == 0) fixed();
                            if (!ok) break;
                            vs = st;
                            vu = use;
#pragma unroll
                            for (int p = 0; p < PANELS; ++p) {
                                outputs(half, buf, NS == 2 ? buf : 0, p, vs, k >= NS || half > 0);
                                if (half == 1) tc_commit(&S.empty[vs]);
                                step(vs, vu);
                            }
                        }
                        if (!ok) break;
                        p_phase ^= 1u << buf;
                        st = vs;
                        use = vu;
                        if (NS == 1) tc_commit(&S.o_full[0]);
                        else if (k + 2 >= n) tc_commit(&S.o_full[buf]);
                    }
                    if (NS == 1) nq += n;
                }
                reader.done(S);
            }
            // no MMA runs on into the release of its memory
            int none = 0;
            tc_commit(&S.drained);
            mbar_wait(&S.drained, 0, &none);
        }
        __syncwarp();
    } else if (warp >= C::VALUES) {
        take_registers<C::OTHERS, false>();
        // ------------------------------------------------ values, and codes to 16 bits
        const int me = (tid - C::VALUES * 32) % C::VALUE_THREADS, group = (warp - C::VALUES) / 4;
        bool ok = true;
        uint32_t st = group, use = 0, cst = group, cuse = 0, stages = 0, fixes = 0, loads = 0, tiles = 0;
        while (const Portion* at = reader.next(S, A.wait_ns)) {
            const Portion& P = *at;
            const int n = P.i1 - P.i0;
            const bool ahead = NS == 1 || P.split;
            auto seen = [&](int tile) { return Seen{P.r.end - tile * kTile, P.lo - tile * kTile, A.sinks - tile * kTile}; };
            auto poison = [&]() { *(volatile int*)&S.poison[P.number % kPortions] = P.number + 1; };
            if constexpr (!BITS8) {
                for (int i = 0; ok && i < n; ++i) {
                    const int tile = P.r.tile(P.i0 + i);
                    if (P.item.has(tile)) continue;
                    // K and V stages in the copies' order: those before this tile's values
                    const Seen rows = seen(tile);
                    const uint32_t s0 = st + (ahead ? min(i + 2, n) + i : 2 * i + 1) * PANELS;
                    // the MMAs' thread has them in the ring, and waits
                    ok = mbar_wait(&S.to_fix, fixes & 1, quit, A.wait_ns);
                    ++fixes;
                    for (int p = 0; p < PANELS; ++p) {
                        const uint32_t s = (s0 + p) % RING, u = use + (s0 + p) / RING;
                        ok = ok && mbar_wait(&S.full[s], u & 1, quit, A.wait_ns);
                        ok = __all_sync(kFull, ok);
                        if (ok && clean_stage<C>(ring + s * C::STAGE, me, [&](int row) { return rows.has(row); })) poison();
                    }
                    if (!ok) break;
                    fence_async_smem();
                    mbar_arrive(&S.fixed);
                }
                const uint32_t total = st + 2 * n * PANELS;
                use += total / RING;
                st = total % RING;
            } else {
                // the two groups take stages in turn, each the ring's every other
                bool queries = false;
#pragma unroll 1
                for (int q = (stages & 1) != group; ok && q < 2 * n * PANELS; q += 2) {
                    // the copies' order: K V K V ..., or K K V K V ... V V
                    const int i = q / PANELS;
                    const bool value = ahead ? (i > 0 && (i % 2 == 0 || i == 2 * n - 1)) : (i & 1);
                    const int k = ahead ? (value ? (i == 2 * n - 1 ? n - 1 : i / 2 - 1) : (i + 1) / 2) : i / 2;
                    ok = mbar_wait(&S.code_full[cst], cuse & 1, quit, A.wait_ns) &&
                         (use == 0 || mbar_wait(&S.empty[st], (use - 1) & 1, quit, A.wait_ns));
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    const uint4* from = reinterpret_cast<const uint4*>(codes + cst * C::CODES);
                    uint8_t* to = ring + st * C::STAGE;
                    if (value) {
                        const bool e4m3 = A.cache_dtype == BSA_DTYPE_E4M3;
                        const bool odd = e4m3 ? widen_value_stage<C, true>(from, to, me) : widen_value_stage<C, false>(from, to, me);
                        if (odd) {
                            const int tile = P.r.tile(P.i0 + k), d0 = q % PANELS * C::PD;
                            uint32_t(*dims)[8] = P.item.has(tile) ? S.odd_dims[P.number % kPortions] : nullptr;
                            const float* log_scales = S.scale[(tiles + k) % kInfo][1];
                            if (e4m3 ? note_odd_codes<C, true>(from, me, seen(tile), dims, d0, log_scales)
                                     : note_odd_codes<C, false>(from, me, seen(tile), dims, d0, log_scales))
                                poison();
                        }
                    } else if (A.cache_dtype == BSA_DTYPE_E4M3) {
                        widen_stage<C, true>(from, to, me);
                    } else {
                        widen_stage<C, false>(from, to, me);
                    }
                    mbar_arrive(&S.code_empty[cst]);
                    fence_async_smem();
                    mbar_arrive(&S.full[st]);
                    cst += 2;
                    if (cst >= C::CRING) {
                        cst -= C::CRING;
                        ++cuse;
                    }
                    st += 2;
                    if (st >= RING) {
                        st -= RING;
                        ++use;
                    }
                    if (!queries) {
                        // each group a query tile, the first group the only one
                        queries = true;
                        ok = mbar_wait(&S.q_full, loads & 1, quit, A.wait_ns);
                        ok = __all_sync(kFull, ok);
                        if (!ok) break;
                        const int m = P.tokens > A.tokens ? group : 0;
                        const int rows = min(A.tokens, P.tokens - m * A.tokens) * A.G;
                        if (me < rows && (m == group || group == 0)) S.q_power[loads & 1][m][me] = (uint8_t)halve_row<C>(qsm + m * C::Q_TILE, me);
                        fence_async_smem();
                        mbar_arrive(&S.q_ready);
                        ++loads;
                    }
                }
                stages += 2 * n * PANELS;
                tiles += n;
            }
            __syncwarp();
            if (lane == 0) reader.done(S);
            else ++reader.number;
        }
    } else if (warp >= C::SOFTMAX) {
        take_registers<C::OTHERS, false>();      // warps without work, of a group of four
    } else {
        take_registers<C::MINE, true>();
        // ------------------------------------------------ softmax and output
        const int stream = warp >> 2, row = tid & 127, token = row / A.G;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t o_addr = lanes + C::O_COL + stream * C::D;
        uint32_t s_phase = 0, o_phase = 0, tiles = 0, nq = 0;
        bool ok = true, left_head = false;
        while (const Portion* at = reader.next(S, A.wait_ns)) {
            const Portion& P = *at;
            const int n = P.i1 - P.i0;
            const int m = NS == 2 && !P.split ? stream : 0;              // its query tile
            const int mine = min(A.tokens, P.tokens - m * A.tokens);     // tokens of it
            const bool valid = row < A.tokens * A.G && token < mine;
            const bool live = __any_sync(kFull, valid);
            int hi, lo;                                                  // the last token that the row sees, its window's first
            {
                const int64_t first = P.pos0 + m * A.tokens, pos = valid ? first + token : first + mine - 1;   // rows beyond do as the last
                const int64_t top = (int64_t)A.max_blocks * kTile;
                hi = (int)(pos < 0 ? -1 : pos < top ? pos : top - 1);
                lo = A.window > 0 ? (int)(pos - A.window + 1 < 0 ? 0 : pos - A.window + 1 < top ? pos - A.window + 1 : top) : 0;
            }
            // The row's sums are in units of 2^mx and its outputs in units of 2^mo: with bf16 the same; with 8
            // bits mo goes by the largest weight, a probability times its page's scale.  Both units lie 2^kLift below
            // the largest: a weight may fall 2^178 below it before its second term is lost, and a probability 2^86
            // (126 + kLift - kFar; its page's weights are then 2^186 below theirs).
            float mx = -INFINITY, mo = -INFINITY, l[4] = {};
            bool written = false;                                        // O holds something
            const int stride = P.split ? 2 : 1;
            for (int k = P.split ? stream : 0; ok && k < n; k += stride) {
                const int buf = NS == 2 ? stream : (nq + k) & 1;
                ok = mbar_wait(&S.s_full[buf], (s_phase >> buf) & 1, quit, A.wait_ns);
                s_phase ^= 1u << buf;
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                tc_fence_after();
                if (!P.split && tid == 0 && k == 0) mbar_arrive(&S.q_empty);
                bool settled = NS == 2 || k == 0;      // the last values' product is done
                // one stream: it may still run under this tile's scores
                auto settle = [&]() {
                    if (settled) return;
                    ok = ok && mbar_wait(&S.o_full[0], o_phase ^ 1, quit, A.wait_ns);
                    ok = __all_sync(kFull, ok);
                    tc_fence_after();
                    settled = true;
                };
                bool halved = false;      // the product of the first 64 tokens may start
                if (live) {
                    const int tile = P.r.tile(P.i0 + k), slot = (tiles + k) % kInfo;
                    const int inside = S.valid[slot];
                    const bool whole = inside == kTile && P.tile[m].has(tile);
                    const uint32_t s_addr = lanes + buf * kTile;
                    constexpr int N = BITS8 ? 1 : 4;      // chunks of 32 columns in registers
                    using One = std::integral_constant<int, 1>;
                    using All = std::integral_constant<int, N>;
                    float x[N][32];
                    const float qs = BITS8 ? __uint_as_float((uint32_t)S.q_power[P.loads & 1][m][row] << 23) : 1.f;
                    // 8 bits: what the scores of a chunk's two pages are multiplied by, and log2 of their value
                    // scales; read before the chunk is waited for (shared memory is busy: a read takes long)
                    float2 ks = make_float2(1.f, 1.f), lv = ks;
                    // chunk c of the row's scores: hidden ones are -inf (with 8 bits after their scale, as that
                    // may be zero)
                    auto hide = [&](int c, float (&v)[32]) {
                        const int from = tile * kTile + 32 * c;
                        uint32_t seen = low_bits(min(hi + 1 - from, inside - 32 * c));
                        if (A.window > 0) seen &= ~low_bits(lo - from) | low_bits(A.sinks - from);
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if constexpr (BITS8) v[j] *= j < 16 ? ks.x : ks.y;
                            v[j] = seen >> j & 1 ? v[j] : -INFINITY;
                        }
                        if constexpr (BITS8) ks = make_float2(1.f, 1.f);
                    };
                    auto fetch = [&](auto count, int c0) {
#pragma unroll
                        for (int c = 0; c < count.value; ++c) tmem_ld32(s_addr + 32 * (c0 + c), x[c]);
                        if constexpr (BITS8) {
                            ks = *reinterpret_cast<const float2*>(&S.scale[slot][0][2 * c0]);
                            lv = *reinterpret_cast<const float2*>(&S.scale[slot][1][2 * c0]);
                            ks.x *= qs;
                            ks.y *= qs;
                        }
#pragma unroll
                        for (int c = 0; c < count.value; ++c) tmem_wait32(x[c]);
                        if (!whole) {
#pragma unroll
                            for (int c = 0; c < count.value; ++c) hide(c0 + c, x[c]);
                        }
                    };
                    // maxima of 16 columns, the largest in `top_s`, with their pages' value scales in `top_o`
                    float top_s = -INFINITY, top_o = -INFINITY;
                    auto maxima = [&](auto count) {
                        constexpr int STRANDS = 4 * count.value;
                        float m8[STRANDS];      // of 8 columns, side by side
#pragma unroll
                        for (int p = 0; p < STRANDS; ++p) m8[p] = x[p / 4][p % 4 * 8];
#pragma unroll
                        for (int j = 1; j < 7; j += 2)
#pragma unroll
                            for (int p = 0; p < STRANDS; ++p) m8[p] = fmaxf(fmaxf(m8[p], x[p / 4][p % 4 * 8 + j]), x[p / 4][p % 4 * 8 + j + 1]);
#pragma unroll
                        for (int p = 0; p < STRANDS; p += 2) {
                            m8[p] = fmaxf(fmaxf(m8[p], x[p / 4][p % 4 * 8 + 7]), fmaxf(m8[p + 1], x[p / 4][p % 4 * 8 + 15]));
                            if constexpr (BITS8) {
                                m8[p] *= p == 0 ? ks.x : ks.y;
                                top_o = fmaxf(top_o, m8[p] + (p == 0 ? lv.x : lv.y));
                            }
                            top_s = fmaxf(top_s, m8[p]);
                        }
                    };
                    if constexpr (!BITS8) {
                        fetch(All{}, 0);
                        maxima(All{});
                        top_s *= A.scale_log2e;
                        top_o = top_s;
                    } else {
                        // The loops over chunks stay loops: the SM's warps run five programs with 8 bits, and
                        // waited for instructions for 2.7 of 11 cycles an issue with this one unrolled.
#pragma unroll 1
                        for (int c = 3; c >= 0; --c) {
                            fetch(One{}, c);
                            maxima(One{});
                        }
                    }
                    // a row whose maximum has grown by more than 2^kGrow takes it over
                    constexpr float LIFT = BITS8 ? kLift : 0.f;
                    top_s -= LIFT;
                    top_o -= LIFT;
                    const bool grow = valid && top_s > mx + kGrow, grow_o = BITS8 ? valid && top_o > mo + kGrow : grow;
                    if (__any_sync(kFull, grow || grow_o)) {
                        // in two factors with 8 bits, as units may lie further apart than fp32's range
                        constexpr float PART = BITS8 ? 0.5f : 1.f;
                        const float keep = grow ? ex2(PART * (mx - top_s)) : 1.f, keep_o = grow_o ? ex2(PART * (mo - top_o)) : 1.f;
                        if (grow) mx = top_s;
                        if (grow_o) mo = top_o;
#pragma unroll
                        for (int i = 0; i < 4; ++i) l[i] = BITS8 ? l[i] * keep * keep : l[i] * keep;
                        if (written) {
                            settle();
#pragma unroll 1
                            for (int c = 0; c < C::D / 16; ++c) {
                                float o[16];
                                tmem_ld16(o_addr + 16 * c, o);
                                uint32_t w[16];
#pragma unroll
                                for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(BITS8 ? o[j] * keep_o * keep_o : o[j] * keep_o);
                                tmem_st16(o_addr + 16 * c, w);
                            }
                        }
                    }
                    const float base = mx == -INFINITY ? 0.f : -mx;
                    const float base_o = mo == -INFINITY ? 0.f : -mo;
                    // the probabilities of chunk c, in v, to the scores' place: 16 columns of 32 tokens' or, with 8
                    // bits, 8 of a page's first terms and 8 of its second
                    auto turn = [&](int c, const float (&v)[32]) {
                        if constexpr (!BITS8) {
                            uint32_t w[16];
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                float a, b;
                                fma2(a, b, v[j], v[j + 1], A.scale_log2e, A.scale_log2e, base, base);
                                a = ex2(a);
                                b = ex2(b);
                                add2(l[j / 2 % 2 * 2], l[j / 2 % 2 * 2 + 1], a, b);
                                w[j / 2] = pack_bf16(a, b);
                            }
                            tmem_st16(s_addr + 16 * c, w);
                        } else {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                // A page's weights are 2^x of its probabilities, in these units, for any x: its exponentials take
                                // 2^h of that, all of it unless the scale is zero or far below those that count, the sum of the
                                // probabilities gives it back, and f is the rest.
                                const float k = g == 0 ? ks.x : ks.y, x = (g == 0 ? lv.x : lv.y) + (base_o - base);
                                const float h = fmaxf(x, -kFar), from = base + h, u = ex2(-h), f = ex2(x - h);
                                uint32_t w[16];
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    float a, b;
                                    fma2(a, b, v[16 * g + j], v[16 * g + j + 1], k, k, from, from);
                                    a = ex2(a);
                                    b = ex2(b);
                                    float& l0 = l[j / 2 % 2 * 2];
                                    float& l1 = l[j / 2 % 2 * 2 + 1];
                                    fma2(l0, l1, a, b, u, u, l0, l1);
                                    mul2(a, b, f);
                                    w[j / 2] = pack_bf16(a, b);
                                    fma2(a, b, __uint_as_float(w[j / 2] << 16), __uint_as_float(w[j / 2] & 0xFFFF0000u), -1.f, -1.f, a, b);
                                    w[8 + j / 2] = pack_bf16(a, b);
                                }
                                tmem_st16(s_addr + 32 * c + 16 * g, w);
                            }
                        }
                    };
                    auto half_done = [&]() {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&S.p_half[buf]);
                        halved = true;
                    };
                    if constexpr (!BITS8) {
                        turn(0, x[0]);
                        turn(1, x[1]);
                        half_done();
                        turn(2, x[2]);
                        turn(3, x[3]);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            // the first chunk is there; the others were not touched by its probabilities
                            if (c > 0) fetch(One{}, c);
                            turn(c, x[0]);
                            if (c == 1) half_done();
                        }
                    }
                    tmem_wait_st();
                    written = true;
                }
                tc_fence_before();
                if (!halved) mbar_arrive(&S.p_half[buf]);
                settle();
                if (NS == 1) o_phase ^= 1;      // as many products as tiles
                tc_fence_before();
                mbar_arrive(&S.p_full[buf]);
            }
            if (NS == 1) nq += n;
            tiles += n;
            // ---- the portion's result
            const bool any = n > (P.split ? stream : 0);
            if (NS == 1) {
                if (n > 0) ok = ok && mbar_wait(&S.o_full[0], o_phase ^ 1, quit, A.wait_ns);
            } else if (any) {
                ok = ok && mbar_wait(&S.o_full[stream], o_phase, quit, A.wait_ns);
                o_phase ^= 1;
            }
            ok = __all_sync(kFull, ok);
            tc_fence_after();
            float sum = (l[0] + l[1]) + (l[2] + l[3]);
            if constexpr (!BITS8) mo = mx;
            if (!ok) mx = mo = sum = NAN;
            // 16 of the row's outputs, not yet divided by the sum
            auto result = [&](int c, float (&o)[16]) {
                if (ok && any && live) {
                    tmem_ld16(o_addr + 16 * c, o);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = ok ? 0.f : NAN;
                }
            };
            const bool join = P.split && n > 1;      // both streams have a part of the rows
            float f0 = 1.f, f1 = 0.f;
            // the second stream's maxima, sums and units, and half of its outputs, in the queries' place: its
            // last product is behind all scores
            float4* other = reinterpret_cast<float4*>(qsm);
            float* xch = reinterpret_cast<float*>(qsm + C::Q_TILE);      // [D / 2][128]
            if (NS == 2 && join) {
                if (stream == 1) other[row] = make_float4(mx, sum, mo, 0.f);
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (stream == 0) {
                    const float4 y = other[row];
                    const float m2 = fmaxf(mx, y.x), o2 = fmaxf(mo, y.z);
                    constexpr float PART = BITS8 ? 0.5f : 1.f;
                    auto times = [](float x, float f) { return BITS8 ? x * f * f : x * f; };
                    f0 = mo == -INFINITY ? 0.f : ex2(PART * (mo - o2));
                    f1 = y.z == -INFINITY ? 0.f : ex2(PART * (y.z - o2));
                    sum = (mx == -INFINITY ? 0.f : times(sum, ex2(PART * (mx - m2)))) + (y.x == -INFINITY ? 0.f : times(y.y, ex2(PART * (y.x - m2))));
                    mx = m2;
                    mo = o2;
                    if (!(y.y == y.y)) sum = NAN;
                }
            }
            // behind the join: the other stream's tiles have been gone over too
            const bool odd = any && *(volatile int*)&S.poison[P.number % kPortions] == P.number + 1;
            const bool whole_item = P.begins && P.ends;
            // from the outputs' unit to the sums', in two factors where it may pass the range of one
            const float back = BITS8 && whole_item && mo > -INFINITY ? ex2(0.5f * (mo - mx)) : 1.f;
            const float scale = whole_item ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            const int64_t t = P.row0 + m * A.tokens + token;
            uint16_t* out = A.out + ((t * A.H + P.h) * A.G + row % A.G) * A.D;
            const int64_t part_row = ((int64_t)blockIdx.x * 2 + (P.begins ? 1 : 0)) * A.part_rows + m * kRows + row;
            const bool writes = valid && (stream == 0 || !P.split);
            if (!whole_item && writes) A.sums[part_row] = make_float4(mx, sum, mo, 0.f);
            float* part = A.parts + part_row * A.D;
            if (P.more > 0 && tid == 0) {
                A.heads[blockIdx.x] = PartHead{P.row0, P.tokens, P.h, P.more, 0};
                left_head = true;
            }
#pragma unroll 1
            for (int half = 0; half < (NS == 2 ? 2 : 1); ++half) {
                constexpr int CH = C::D / 16 / (NS == 2 ? 2 : 1);      // chunks of 16 a half
                if (NS == 2 && join) {
                    if (stream == 1) {
#pragma unroll 1
                        for (int c = 0; c < CH; ++c) {
                            float o[16];
                            result(half * CH + c, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) xch[(c * 16 + j) * kRows + row] = o[j];
                        }
                    }
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                }
                if (live && (stream == 0 || !P.split)) {
#pragma unroll 1
                    for (int c = 0; c < CH; ++c) {
                        const int d0 = (half * CH + c) * 16;
                        float o[16];
                        result(half * CH + c, o);
                        if (NS == 2 && join) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float y = xch[(c * 16 + j) * kRows + row];
                                o[j] = BITS8 ? o[j] * f0 * f0 + y * f1 * f1 : o[j] * f0 + y * f1;
                            }
                        }
                        // behind the join, whose factors may be zero
                        if (odd && valid) {
                            float x[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[j] = 0.f;
                            add_odd_values<C, BITS8>(A, P, S.odd_dims[P.number % kPortions], hi, lo, d0, x);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] += x[j];
                        }
                        if (!writes || d0 >= A.D) continue;
                        if (whole_item) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float b = BITS8 ? back : 1.f;
                                w[j] = pack_bf16(o[2 * j] * scale * b * b, o[2 * j + 1] * scale * b * b);
                            }
                            store32(out + d0, w, A.wide_out);
                        } else {
                            store32(part + d0, reinterpret_cast<const uint32_t*>(o), true);
                            store32(part + d0 + 8, reinterpret_cast<const uint32_t*>(o + 8), true);
                        }
                    }
                }
                if (NS == 2 && join) {
                    fence_async_smem();      // queries of the next item come to this place by TMA
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                }
            }
            tc_fence_before();
            if (P.split && tid == 0 && n > 0) mbar_arrive(&S.q_empty);
            __syncwarp();
            if (lane == 0) reader.done(S);
            else ++reader.number;
        }
        if (tid == 0 && !left_head) A.heads[blockIdx.x].more = 0;
        if (tid == 0) report_status(A.status, S.gave_up != 0, BSA_STATUS_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA) tmem_free(tmem, 512);
}

// Joins the parts of items that CTAs left to one another: block x takes the item that
// CTA x began, a slice of its rows.  A thread takes 8 dimensions of a row; of many
// parts (one request on its own has one in each of dozens of CTAs, each a read from L2
// or beyond) four lanes take every fourth, then join theirs, always in the same order.
template <bool BITS8>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedParams A) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PartHead head = A.heads[blockIdx.x];
    if (head.more <= 0) return;
    struct Sum {
        float m, mo, l, o[8];
        // another's maximum, sum, unit and outputs; a part without tokens has -inf for its maximum, one that is not
        // finished NaN
        __device__ __forceinline__ void add(float ym, float yl, float yo, const float (&v)[8]) {
            const float m2 = fmaxf(m, ym), o2 = fmaxf(mo, yo);
            // 8 bits: in two factors, as units may lie further apart than fp32's range; outputs that are not finite stay
            constexpr float PART = BITS8 ? 0.5f : 1.f;
            auto times = [](float x, float f) {
                if constexpr (BITS8) return x - x == 0.f ? x * f * f : x;
                else return x * f;
            };
            l = (m == -INFINITY ? 0.f : times(l, ex2(PART * (m - m2)))) +
                (ym == -INFINITY ? 0.f : times(yl, ex2(ym != ym ? NAN : PART * (ym - m2))));
            const float f0 = mo == -INFINITY ? 0.f : ex2(PART * (mo - o2)), f1 = yo == -INFINITY ? 0.f : ex2(yo != yo ? NAN : PART * (yo - o2));
            m = m2;
            mo = o2;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = times(o[j], f0) + times(v[j], f1);
        }
    };
    const int words = A.D / 8, rows = head.tokens * A.G;
    const int lanes = head.more >= 4 ? 4 : 1, lane = threadIdx.x % lanes, each = kJoinThreads / lanes;
    for (int i0 = blockIdx.y * each; i0 < rows * words; i0 += gridDim.y * each) {
        const int i = i0 + (int)threadIdx.x / lanes;
        const bool here = i < rows * words;
        const int r = here ? i / words : 0, d = here ? i - r * words : 0;
        const int token = r / A.G, g = r - token * A.G, tile = token / A.tokens;
        const int64_t part_row = tile * kRows + (token - tile * A.tokens) * A.G + g;
        Sum t{-INFINITY, -INFINITY, 0.f, {}};
        constexpr int AHEAD = 4;
        for (int k0 = lane; k0 <= head.more; k0 += lanes * AHEAD) {
            float4 s[AHEAD], x[AHEAD], y[AHEAD];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                const int k = k0 + lanes * e;
                if (k > head.more) continue;
                const int64_t at = ((int64_t)(blockIdx.x + k) * 2 + (k == 0)) * A.part_rows + part_row;
                const float4* p = reinterpret_cast<const float4*>(A.parts + at * A.D + d * 8);
                s[e] = A.sums[at];
                x[e] = p[0];
                y[e] = p[1];
            }
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                if (k0 + lanes * e > head.more) continue;
                const float v[8] = {x[e].x, x[e].y, x[e].z, x[e].w, y[e].x, y[e].y, y[e].z, y[e].w};
                t.add(s[e].x, s[e].y, s[e].z, v);
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            if (o >= lanes) break;
            float v[8];
            const float ym = __shfl_down_sync(kFull, t.m, o, 4), yl = __shfl_down_sync(kFull, t.l, o, 4), yo = __shfl_down_sync(kFull, t.mo, o, 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __shfl_down_sync(kFull, t.o[j], o, 4);
            t.add(ym, yl, yo, v);      // of use in the lanes that have a partner
        }
        if (!here || lane != 0) continue;
        const float back = BITS8 && t.mo > -INFINITY ? ex2(0.5f * (t.mo - t.m)) : 1.f;
        const float inv = t.l == 0.f ? 0.f : 1.f / t.l;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = BITS8 ? pack_bf16(t.o[2 * j] * inv * back * back, t.o[2 * j + 1] * inv * back * back) : pack_bf16(t.o[2 * j] * inv, t.o[2 * j + 1] * inv);
        const int64_t row = ((head.row0 + token) * A.H + head.h) * A.G + g;
        *reinterpret_cast<uint4*>(A.out + row * A.D + d * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ---- host ------------------------------------------------------------------

std::atomic<unsigned long long> g_paged_wait_ns{kWaitNs};
std::atomic<uint32_t> g_paged_stall{UINT32_MAX};

using EncodeFn = decltype(&cuTensorMapEncodeTiled);
EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// The cache as a tensor of (dimension, head, token), read in boxes of a block of one
// head: bf16 64 dimensions at a time, swizzled as the tensor core reads them; codes a
// panel at a time, as they are.
bool encode_cache(CUtensorMap* map, const void* base, int64_t tokens, int64_t H, int64_t D, bool bits8) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t size = bits8 ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {D * size, H * D * size};
    const cuuint32_t box[3] = {(cuuint32_t)(bits8 && D > 64 ? 128 : 64), 1, (cuuint32_t)kTile};
    const cuuint32_t unit[3] = {1, 1, 1};
    return fn(map, bits8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
              box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, bits8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              bits8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as a tensor of (dimension, query head of a KV head, KV head, token), read in
// boxes of `tokens` tokens' heads: the rows of an MMA.
bool encode_queries(CUtensorMap* map, const void* base, int64_t T, int64_t H, int64_t G, int64_t D, int tokens) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)(G * D) * 2, (cuuint64_t)(H * G * D) * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)tokens};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool paged_sizes_ok(int64_t T, int64_t H, int64_t G, int64_t D) {
    return T >= 0 && T <= INT32_MAX && H >= 1 && H <= 65536 && G >= 1 && G <= BSA_MAX_PAGED_GROUP && T * H * G <= INT32_MAX &&
           D >= 16 && D <= BSA_MAX_CACHE_DIM && D % 16 == 0;
}

// Whether a call's inputs share memory with `x`; `ints`: the form's own index tensors.
bool meets_inputs(const Rows& x, const bsa_paged_attention_args_t& a, const Rows (&ints)[2]) {
    const bool bits8 = a.cache_dtype != BSA_DTYPE_BF16;
    const int64_t cache = a.num_pages * kSubPage * a.H * a.D * (bits8 ? 1 : 2), scales = bits8 ? a.num_pages * a.H * 4 : 0;
    const Rows in[8] = {whole_rows(a.q, a.T * a.H * a.G * a.D * 2), whole_rows(a.k_cache, cache), whole_rows(a.v_cache, cache),
                        whole_rows(a.k_scale, scales), whole_rows(a.v_scale, scales),
                        whole_rows(a.block_table, a.num_reqs * a.max_blocks * 4), ints[0], ints[1]};
    for (const Rows& r : in)
        if (rows_overlap(x, r)) return true;
    return false;
}

// The checks that both forms share.
int check_paged(const bsa_paged_attention_args_t& a, const Rows (&ints)[2]) {
    if (a.cache_dtype != BSA_DTYPE_BF16 && a.cache_dtype != BSA_DTYPE_E4M3 && a.cache_dtype != BSA_DTYPE_E5M2) return BSA_ERR_DTYPE;
    if (!paged_sizes_ok(a.T, a.H, a.G, a.D) || a.num_pages < 0 || a.num_pages >= (1ll << 27) || a.num_reqs < 0 ||
        a.num_reqs > (1 << 24) || a.max_blocks < 0 || a.max_blocks >= (1 << 24) || a.window < 0 || a.sinks < 0)
        return BSA_ERR_SHAPE;
    if (a.T == 0) return BSA_OK;
    const bool bits8 = a.cache_dtype != BSA_DTYPE_BF16;
    if (a.q == nullptr || a.out == nullptr || (a.num_reqs > 0 && a.max_blocks > 0 && a.block_table == nullptr)) return BSA_ERR_NULL;
    if (a.num_pages > 0 && (a.k_cache == nullptr || a.v_cache == nullptr || (bits8 && (a.k_scale == nullptr || a.v_scale == nullptr))))
        return BSA_ERR_NULL;
    const void* wide[4] = {a.q, a.out, a.k_cache, a.v_cache};
    for (const void* p : wide)
        if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return BSA_ERR_ALIGN;
    return meets_inputs(whole_rows(a.out, a.T * a.H * a.G * a.D * 2), a, ints) ? BSA_ERR_SHAPE : BSA_OK;
}

// Rows of an item's part in the workspace.
int part_rows(int64_t T, int64_t G, int64_t D) {
    const int64_t tokens = kRows / G;
    return (int)(T <= tokens ? T * G : D <= 128 ? 2 * kRows : kRows);
}

struct Parts {
    size_t heads, sums, bytes;      // offsets, and all of it
};
Parts place_parts(int64_t T, int64_t G, int64_t D, int grid) {
    const size_t rows = (size_t)grid * 2 * part_rows(T, G, D);
    Parts p;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    p.heads = up(rows * D * sizeof(float));
    p.sums = p.heads + up((size_t)grid * sizeof(PartHead));
    p.bytes = p.sums + up(rows * sizeof(float4));
    return p;
}

template <int D, bool BITS8>
cudaError_t launch_kernel(const PagedParams& A, const PagedMaps& M, int grid, cudaStream_t st) {
    using C = Cfg<D, BITS8>;
    constexpr int SMEM = C::NS * C::Q_TILE + C::RING * C::STAGE + C::CRING * C::CODES + (int)sizeof(Shared);
    static_assert(SMEM <= 232448, "a CTA's shared memory");
    static_assert(kWindow * 8 <= C::RING * C::STAGE, "units fit in the ring");
    auto kern = paged_attention_kernel<D, BITS8>;
    static FuncOnce once;
    const cudaError_t e = once.smem(reinterpret_cast<const void*>(kern), SMEM);
    if (e != cudaSuccess) return e;
    kern<<<grid, C::THREADS, SMEM, st>>>(A, M);
    return cudaGetLastError();
}

int launch_paged(const bsa_paged_attention_args_t& a, const Rows (&ints)[2], PagedParams& A, cudaStream_t st) {
    const int grid = device_sm_count();
    const Parts parts = place_parts(a.T, a.G, a.D, grid);
    if (a.workspace == nullptr || a.workspace_bytes < parts.bytes || (reinterpret_cast<uintptr_t>(a.workspace) & 255) != 0)
        return BSA_ERR_WORKSPACE;
    const Rows scratch = whole_rows(a.workspace, (int64_t)parts.bytes);
    if (rows_overlap(scratch, whole_rows(a.out, a.T * a.H * a.G * a.D * 2)) || meets_inputs(scratch, a, ints)) return BSA_ERR_SHAPE;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const bool bits8 = a.cache_dtype != BSA_DTYPE_BF16;
    A.out = static_cast<uint16_t*>(a.out);
    A.v = static_cast<const uint8_t*>(a.v_cache);
    A.ks = a.k_scale;
    A.vs = a.v_scale;
    A.table = a.block_table;
    A.T = a.T;
    A.num_pages = a.num_pages;
    A.num_reqs = (int32_t)a.num_reqs;
    A.max_blocks = (int32_t)a.max_blocks;
    A.H = (int32_t)a.H;
    A.G = (int32_t)a.G;
    A.D = (int32_t)a.D;
    A.tokens = kRows / A.G;
    A.window = a.window;
    A.sinks = a.sinks;
    A.cache_dtype = a.cache_dtype;
    A.min_units = kMinSteps * (bits8 ? Cfg<128, true>::SPLIT_UNITS : Cfg<128, false>::SPLIT_UNITS);
    A.part_rows = part_rows(a.T, a.G, a.D);
    // a scale of zero must not meet the -inf of hidden scores; the least one has its result: times the largest
    // score it is 2^-21
    const float scale = fabsf(a.scale) * 1.44269504f;
    A.scale_log2e = scale == 0.f ? 0x1p-149f : scale;
    A.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    A.s_idesc = f16_idesc(!bits8, a.scale < 0.f, false, kRows, kTile);
    A.o_idesc = f16_idesc(true, false, true, kRows, a.D <= 64 ? 64 : 128);
    A.parts = reinterpret_cast<float*>(ws);
    A.heads = reinterpret_cast<PartHead*>(ws + parts.heads);
    A.sums = reinterpret_cast<float4*>(ws + parts.sums);
    A.status = current_status_word();
    A.wait_ns = g_paged_wait_ns.load(std::memory_order_relaxed);
    A.stall = g_paged_stall.load(std::memory_order_relaxed);
    PagedMaps M;
    // an empty cache: no box lies inside, any address serves
    const int64_t tokens = (a.num_pages > 0 ? a.num_pages : 1) * kSubPage;
    if (!encode_queries(&M.q, a.q, a.T, a.H, a.G, a.D, A.tokens) ||
        !encode_cache(&M.k, a.num_pages > 0 ? a.k_cache : a.q, tokens, a.H, a.D, bits8) ||
        !encode_cache(&M.v, a.num_pages > 0 ? a.v_cache : a.q, tokens, a.H, a.D, bits8))
        return (int)cudaErrorInvalidValue;
    cudaError_t e;
    if (a.D <= 64) e = bits8 ? launch_kernel<64, true>(A, M, grid, st) : launch_kernel<64, false>(A, M, grid, st);
    else if (a.D <= 128) e = bits8 ? launch_kernel<128, true>(A, M, grid, st) : launch_kernel<128, false>(A, M, grid, st);
    else e = bits8 ? launch_kernel<256, true>(A, M, grid, st) : launch_kernel<256, false>(A, M, grid, st);
    if (e != cudaSuccess) return (int)e;
    cudaLaunchConfig_t cfg{};
    const int slices = (A.part_rows * A.D / 8 * 4 + kJoinThreads - 1) / kJoinThreads;
    cfg.gridDim = dim3((unsigned)grid, (unsigned)(slices < 8 ? slices : 8));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = bits8 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<true>, (const PagedParams)A) : cudaLaunchKernelEx(&cfg, paged_join_kernel<false>, (const PagedParams)A);
    return e == cudaSuccess ? BSA_OK : (int)e;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

// For tests, not part of the ABI: in later calls each CTA's copies stop after `stages`
// stages (UINT32_MAX: never) and waits give up after `wait_ns` (0: the usual four seconds).
extern "C" void bsa_paged_attention_stall(uint32_t stages, uint64_t wait_ns) {
    g_paged_stall.store(stages, std::memory_order_relaxed);
    g_paged_wait_ns.store(wait_ns == 0 ? kWaitNs : wait_ns, std::memory_order_relaxed);
}

extern "C" size_t bsa_paged_attention_workspace_bytes(int64_t T, int64_t H, int64_t G, int64_t D) {
    if (!paged_sizes_ok(T, H, G, D) || T == 0) return 0;
    return place_parts(T, G, D, device_sm_count()).bytes;
}

extern "C" int bsa_paged_attention_decode(const bsa_paged_attention_args_t* args, const int32_t* seq_lens, int32_t decode_query_len,
                                          void* stream) {
    if (args == nullptr) return BSA_ERR_NULL;
    const bsa_paged_attention_args_t& a = *args;
    const Rows ints[2] = {whole_rows(seq_lens, a.num_reqs * 4), whole_rows(nullptr, 0)};
    const int rc = check_paged(a, ints);
    if (rc != BSA_OK) return rc;
    if (decode_query_len < 1) return BSA_ERR_SHAPE;
    if (a.T != a.num_reqs * decode_query_len) return BSA_ERR_ROWS;
    if (a.T == 0) return BSA_OK;
    if (seq_lens == nullptr) return BSA_ERR_NULL;
    PagedParams A{};
    A.seq_lens = seq_lens;
    A.dql = decode_query_len;
    return launch_paged(a, ints, A, static_cast<cudaStream_t>(stream));
}

extern "C" int bsa_paged_attention_varlen(const bsa_paged_attention_args_t* args, const int32_t* cu_seqlens_q,
                                          const int32_t* prefix_lens, void* stream) {
    if (args == nullptr) return BSA_ERR_NULL;
    const bsa_paged_attention_args_t& a = *args;
    const Rows ints[2] = {whole_rows(cu_seqlens_q, (a.num_reqs + 1) * 4), whole_rows(prefix_lens, a.num_reqs * 4)};
    const int rc = check_paged(a, ints);
    if (rc != BSA_OK) return rc;
    if (a.T == 0) return BSA_OK;
    if (cu_seqlens_q == nullptr || (a.num_reqs > 0 && prefix_lens == nullptr)) return BSA_ERR_NULL;
    PagedParams A{};
    A.cu = cu_seqlens_q;
    A.prefix = prefix_lens;
    return launch_paged(a, ints, A, static_cast<cudaStream_t>(stream));
}
