// paged_attn.cu -- the new tokens of a packed ragged batch attend over a paged cache.
//
// No counterpart on the pages: a server's batch holds sequences that decode one token, verify a
// block of drafts and run a chunk of their prompt. Row b has n new tokens, the last n of len
// positions; query head hq of token j sees position t <= len - n + j of KV head hq / g:
//   out[j, hq] = sum_t softmax_t(scale * q[j, hq] . K_t) V_t
// One pass over the tiles with a running reference m and sum l per query: p_t = 2^(s_t - m),
// O += p V, l += p (for binary16 all times 2^7); m moves only when a row's maximum exceeds it by
// more than 2^8 (O and l are then scaled).
//
// Design.
//  * A unit is one row, KV head and block of up to 128 query vectors: 128 / g tokens times the g
//    query heads that share the KV head, so K and V are read once for all of them. Its products
//    run on the fifth-generation tensor cores: S = Q.K^T (M 128, N 128, K 64) and O += P.V
//    (M 128, N 64, K 128); scores, outputs and P (as the A operand) in tensor memory, Q, K and V in
//    128-byte-swizzled shared memory. Tiles are 128 positions: with 64, and so twice the hand-offs
//    between the roles, a chunk of 512 tokens over 16384 took 104 us instead of 98 (measured before
//    the loop lost its spilled registers, which brought the latter to 73).
//  * Six warps: four hold the rows (thread t: tensor-memory lane t), one issues the products, one
//    copies K and V through two and three slots. A page that holds less than a tile is a TMA box of
//    its own, a lane of the copying warp per page; page numbers are read a tile ahead. Boxes from
//    the unit's last visible position on are not read. The scores of the next tile are issued as
//    soon as these are in registers. Two blocks per SM: while one waits, the other computes.
//  * Units of at most 32 vectors (16 in short ones) hold them four times, in lanes 32 apart, and
//    each copy takes the softmax of a quarter of a tile's positions, with P zero elsewhere: a
//    decoding sequence, with 4 query vectors, uses all four warps. The copies are joined at the
//    unit's end. (Held once, one row of 8192 takes 2 % longer, 32 rows to 16384 2 %, 8 rows of 5
//    tokens 5 %.)
//  * Work. The tiles of all units form one list, by weight, and every CTA of one wave takes an
//    equal stretch of it; units cut by a stretch's end merge through the workspace, the last CTA
//    to arrive in the order of the list. So neither one long row nor few rows leave SMs idle, and
//    the tiles of decoding rows (HBM) and of prompt chunks (softmax) run at the same time. The
//    copying warp runs ahead into the CTA's next unit. The list is not made by the host, as lengths
//    lie on the device: every CTA sums the rows' weights (about 2 us).
//
// Measured (in a graph, caches warm where they fit; a copy runs at 6.8 TB/s, a large product at
// 1928 TFLOP/s):
//   1 row x 8192 positions, 32/8 heads         12.3 us   the launch, the list and the merge; 64
//                                                        tiles: 13.9 at 61, 62 and 63, see kUnit
//   32 rows to 16384, 32/8 heads                126 us   6.4 TB/s
//   8 rows x 5 tokens over up to 4095            32 us   4.0 TB/s
//   a chunk of 512 over 16384, 32/8 heads        72 us   940 TFLOP/s: the row warps' chain of
//                                                        loads, maxima, exponentials and
//                                                        hand-offs, 2200 cycles a tile
//   30 rows, two with chunks of 1000 at 8000     98 us   the same
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "kvd_paged.cuh"
#include "kvd_tc.cuh"

namespace kvd {
namespace {

constexpr int kRowThreads = 128;               // the softmax warps
constexpr int kPgThreads = kRowThreads + 64;   // + the MMA warp and the copying warp
constexpr int kPgRows = 128;                   // query vectors per unit
constexpr int kStep = 128;                     // positions per tile: two TMA boxes or more
constexpr int kStepBytes = kStep * kRowBytes;  // of K (or V)
constexpr int kSlotsK = 2, kSlotsV = 3;        // K and V tiles in flight: K is read first
constexpr int kPgMinBlocks = 2;                // blocks per SM the sizes below are chosen for
// tensor memory: scores (128 fp32 columns), output (64), weights (64 columns of two)
constexpr uint32_t kPgColsO = kStep;
constexpr uint32_t kPgColsP = kPgColsO + kHeadDim;
constexpr uint32_t kPgCols = 256;
static_assert(kPgCols >= kPgColsP + kStep / 2 && kPgMinBlocks * kPgCols <= 512,
              "the resident blocks' tensor memory");
constexpr uint32_t kPgQBytes = kPgRows * kRowBytes;
constexpr uint32_t kOddOffset = 256 + kPgRows * 8 + kRowThreads * 16;  // behind the barriers
constexpr int kOddWords = 3 * kHeadDim;        // see scan_hidden
// shared memory: K slots | V slots | Q | barriers | rows' references and sums | merge | odd
constexpr uint32_t kPgSmem = (kSlotsK + kSlotsV) * kStepBytes + kPgQBytes + 256 + kPgRows * 8 +
                             kRowThreads * 16 + kOddWords * 4 + 16 + 1024;
constexpr int kTable = kPgQBytes / 4;  // entries of the rows' prefix sums, in Q's place at first
constexpr float kPgGrow = 8.f;  // a row's reference moves for maxima above it by 2^this
// Weights, sums and outputs are held times 2^this (it cancels in the end). binary16's steps end at
// 2^-24 and its range at 2^16: with 7, weights reach 2^15 at most, and those down to 2^-32 of the
// reference's are kept. (With 0 it was 2^-25: 131072 positions of that weight beside one of the
// reference's lost 0.4 % of the output.) bfloat16 has fp32's range.
template <typename T>
constexpr float kPgLift = std::is_same<T, __half>::value ? 7.f : 0.f;
static_assert(kPgGrow + kPgLift<__half> < 16.f, "binary16's range");

// The list's weights: of a tile, and what a unit costs besides (its start, end and merge).
// Measured on one row of 61, 62, 63 and 64 tiles x 8 heads and on a mixed batch: 13.9, 13.9, 13.9,
// 12.5 us and 98.2 (shares of 20 fit units of 4 n tiles, and no block has more than 4 then; of
// other units some block has 6). A unit as 3, 5 and 6 tiles instead of 4: 12.7, 13.7, 13.9, 14.2
// and 98.1; 13.9, 13.9, 12.2, 14.0 and 98.6; 13.8, 13.9, 13.8, 14.1 and 98.8. A cut at least 20
// from a unit's ends: 15.5, 15.8, 15.7, 16.3 and 98.4; at least 5: 12.7, 12.0, 12.5, 12.5 and 98.2.
// A least share of 15, 25, 30: 13.9, 13.3, 14.0, 14.5; 13.7, 14.4, 15.1, 13.9; 15.6, 15.6, 16.3,
// 15.9 (the mixed batch 98.2 with each).
constexpr uint32_t kWeight = 5, kUnit = 20;
constexpr int kShort = 2;           // see copies_of
constexpr uint32_t kSnap = 12;      // no cut this close to a unit's ends
constexpr uint32_t kLeast = 20;     // a CTA's least share
// A unit of more than 32 vectors and T tiles, cut into n pieces, takes T / n tiles and n joins of
// 128 rows, one after the other, which cost half a tile each: about 1.4 sqrt(T) pieces are best, so
// a least share of kShare sqrt(T) for calls with few units. (16 tokens x 8 heads at 20000: 29 us
// with it, 34.5 without; at 100000 46 and 143; two rows of 211 tokens at 11523 29 and 33.)
constexpr float kShare = 4.f;
constexpr int kMaxCtas = 512;

struct PagedParams {
    const uint8_t* q;
    int64_t q_st, q_sh;       // bytes
    void* out;                // [n_tokens, n_q_heads, 64]
    const int32_t* starts;
    const int32_t* lens;
    const int32_t* table;
    int64_t table_stride;
    const uint8_t* v;         // the pool, byte strides: see odd_of_copies
    int64_t v_sp, v_sh, v_st;
    int32_t batch, n_tokens, max_new, capacity;
    int32_t n_q_heads, n_kv_heads, group, tq;  // tq: tokens per unit
    int32_t n_pages, page_log2, box_rows, boxes;  // boxes per tile
    float scale_log2;         // above 0; the scale's sign goes into the queries
    int32_t scale_sign;
    float4* ws_part;          // [2 CTAs][16][slot_rows]: 4 dims of a row
    float2* ws_ml;            // [2 CTAs][slot_rows]: reference, sum
    int32_t* ws_cnt;          // a ticket per CTA that holds the first piece of a cut unit
    int32_t slot_rows;
    int32_t* dev_err;
    int32_t test_stall;
};

// ---------------------------------------------------------------- the list of tiles --
struct Row {
    int s, n, len;  // first packed token, new tokens (0: nothing to do), positions
};
__device__ __forceinline__ Row row_of(const PagedParams& p, int b, bool& bad) {
    Row r;
    r.len = p.lens[b];
    bad = !row_tokens(p.starts, b, p.n_tokens, r.s, r.n);
    if (r.n > 0 && (r.n > p.max_new || r.len < r.n || r.len > p.capacity)) {
        bad = true;
        r.n = 0;
    }
    return r;
}

// sum_{i < n} floor((a i + b) / 128), by the Euclidean recursion on (a, 128). The sum is below
// 2^32.
__device__ __forceinline__ uint32_t floor_sum(uint32_t n, uint32_t a, uint32_t b) {
    auto pairs = [](uint32_t n) { return (uint32_t)((uint64_t)n * (n - 1) / 2); };
    // (the first step by hand: divisions by a constant)
    uint32_t sum = pairs(n) * (a / kStep) + n * (b / kStep);
    a %= kStep;
    b %= kStep;
    uint32_t top = a * n + b, m = a;
    n = top / kStep;
    b = top % kStep;
    a = kStep;
    while (n > 0) {
        sum += pairs(n) * (a / m);
        a %= m;
        if (b >= m) {
            sum += n * (b / m);
            b %= m;
        }
        top = a * n + b;
        if (top < m) break;
        n = top / m;
        b = top % m;
        const uint32_t x = m;
        m = a;
        a = x;
    }
    return sum;
}

struct Shape {  // of a row's units
    Row r;
    int nmb;     // blocks of tq tokens
    __device__ __forceinline__ int s0() const { return r.len - r.n; }
};
__device__ __forceinline__ Shape shape_of(const PagedParams& p, const Row& r) {
    Shape s;
    s.r = r;
    s.nmb = r.n <= p.tq ? (r.n > 0) : (r.n + p.tq - 1) / p.tq;
    return s;
}
// Vectors, tiles and weight of block mb.
__device__ __forceinline__ int live_rows(const PagedParams& p, const Shape& s, int mb) {
    return min(p.tq, s.r.n - mb * p.tq) * p.group;
}
__device__ __forceinline__ int kv_end(const PagedParams& p, const Shape& s, int mb) {
    return s.s0() + min(s.r.n, (mb + 1) * p.tq);
}
__device__ __forceinline__ int tiles_of(const PagedParams& p, const Shape& s, int mb) {
    return (kv_end(p, s, mb) + kStep - 1) / kStep;
}
// Units of at most 32 vectors hold them four times; those of more than 16 only if they have more
// than kShort tiles, as the join of their copies takes as long as two tiles (106 rows of 5 tokens x
// 80/20 heads and one tile: 50 us with it, 42 without; 64 of 5 x 32/8 at 700, five tiles: 24.8 and
// 28.6).
__device__ __forceinline__ int copies_of(int live, int tiles) {
    return live > 32 || (live > 16 && tiles <= kShort) ? 1 : 4;
}
__device__ __forceinline__ uint32_t unit_weight(const PagedParams& p, const Shape& s, int mb) {
    return tiles_of(p, s, mb) * kWeight + kUnit;
}
// Weight of the first k blocks of one head, 0 <= k < nmb (they are full).
__device__ __forceinline__ uint32_t full_blocks(const PagedParams& p, const Shape& s, int k) {
    if (k == 0) return 0;
    return kWeight * floor_sum((uint32_t)k, (uint32_t)p.tq,
                                (uint32_t)(s.s0() + p.tq + kStep - 1)) + (uint32_t)k * kUnit;
}
__device__ __forceinline__ uint32_t row_weight(const PagedParams& p, const Row& r) {
    if (r.n == 0) return 0;
    const Shape s = shape_of(p, r);
    return p.n_kv_heads * (full_blocks(p, s, s.nmb - 1) + unit_weight(p, s, s.nmb - 1));
}

// Tiles of a row's longest unit, where that has more than 32 vectors.
__device__ __forceinline__ int heavy_tiles(const PagedParams& p, const Row& r) {
    return min(r.n, p.tq) * p.group > 32 ? r.len / kStep : 0;
}

// Prefix sums over the rows' weights: tab[e] is the list's length up to and with the rows of entry
// e, `each` rows an entry. The host has bounded the length that distinct rows can give; sums that
// leave 32 bits all the same (stretches of tokens that overlap) stay at kTooLong.
constexpr uint32_t kTooLong = 0xffffffffu;
__device__ __forceinline__ uint32_t add_length(uint32_t a, uint32_t b) {
    const uint32_t s = a + b;
    return s < a ? kTooLong : s;
}
struct Table {
    uint32_t* tab;
    int each, n;
};
// All threads; the sums are whole behind a barrier and finish_table (one warp).
__device__ __forceinline__ Table fill_table(const PagedParams& p, uint32_t* tab, int& longest) {
    Table t;
    longest = 0;
    t.tab = tab;
    t.each = (p.batch + kTable - 1) / kTable;
    t.n = t.each == 1 ? p.batch : (p.batch + t.each - 1) / t.each;
    for (int e = threadIdx.x; e < t.n; e += kPgThreads) {
        uint32_t w = 0;
        for (int b = e * t.each; b < min((e + 1) * t.each, p.batch); ++b) {
            bool bad;
            const Row r = row_of(p, b, bad);
            w = add_length(w, row_weight(p, r));
            longest = max(longest, heavy_tiles(p, r));
            if (bad && blockIdx.x == 0) flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
        }
        tab[e] = w;
    }
    return t;
}
// Sums of the warp's values up to and with each lane's.
__device__ __forceinline__ uint32_t scan_rows(uint32_t inc) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc = add_length(inc, o);
    }
    return inc;
}
__device__ __forceinline__ uint32_t finish_table(const Table& t) {
    const int lane = threadIdx.x & 31;
    uint32_t before = 0;
    for (int e0 = 0; e0 < t.n; e0 += 32) {
        const uint32_t inc =
            add_length(scan_rows(e0 + lane < t.n ? t.tab[e0 + lane] : 0), before);
        if (e0 + lane < t.n) t.tab[e0 + lane] = inc;
        before = __shfl_sync(0xffffffffu, inc, 31);
    }
    __syncwarp();
    return before;
}
// The row that holds place `at`, which is below the list's length, and the list's length before
// it. One warp.
__device__ __forceinline__ int find_row(const PagedParams& p, const Table& t, uint32_t at,
                                        uint32_t& before) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = t.n;  // the first entry above `at`: 32 probes a step
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int e = lo + (lane + 1) * step;
        lo += __popc(__ballot_sync(0xffffffffu, e < hi && t.tab[e - 1] <= at)) * step;
        hi = min(lo + step, hi);
    }
    before = lo > 0 ? t.tab[lo - 1] : 0;
    int b = lo * t.each;
    for (const int last = min(b + t.each, p.batch) - 1; b < last; ++b) {
        bool bad;
        const uint32_t w = row_weight(p, row_of(p, b, bad));
        if (before + w > at) break;
        before += w;
    }
    return b;
}

struct Place {  // of a unit
    Row r;
    int b, mb, h;
    uint32_t w;
    uint32_t u0;  // where it starts in the list
};
// The unit of u's row at place `at`, which the row holds; the list's length before the row. One
// warp.
__device__ __forceinline__ void find_unit(const PagedParams& p, Place& u, uint32_t at,
                                          uint32_t before) {
    const Shape s = shape_of(p, u.r);
    const uint32_t in = at - before;
    // the last block that starts at or before `at`: 32 probes a step
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = s.nmb;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int k = lo + (lane + 1) * step;
        const unsigned le =
            __ballot_sync(0xffffffffu, k < hi && p.n_kv_heads * full_blocks(p, s, k) <= in);
        lo += __popc(le) * step;
        hi = min(lo + step, hi);
    }
    u.mb = lo;
    const uint32_t pre = p.n_kv_heads * full_blocks(p, s, lo);
    u.w = unit_weight(p, s, lo);
    u.h = (int)((in - pre) / u.w);
    u.u0 = before + pre + (uint32_t)u.h * u.w;
}

// Stretches of the list: CTA i's share starts at floor(i total / ctas), the quotient in 16.16 bits.
struct Shares {
    uint32_t total, ctas;
    uint64_t each;  // floor(2^16 total / ctas)
    __device__ __forceinline__ uint32_t start(uint32_t i) const {
        return i < ctas ? (uint32_t)(i * each >> 16) : total;
    }
    __device__ __forceinline__ uint32_t holder(uint32_t at) const {  // whose share has place `at`
        uint32_t i = min((uint32_t)__fdividef((float)at * (float)ctas, (float)total), ctas - 1);
        while (start(i) > at) --i;
        while (i + 1 < ctas && start(i + 1) <= at) ++i;
        return i;
    }
};
__device__ __forceinline__ Shares shares(uint32_t total, uint32_t least) {
    Shares s;
    s.total = total;
    s.ctas = max(1u, min(gridDim.x, total / least));
    const uint32_t per = total / s.ctas;
    s.each = ((uint64_t)per << 16) + ((total - per * s.ctas) << 16) / s.ctas;
    return s;
}
// Where the stretch really starts whose share starts inside a unit of weight w: there from keep_lo
// to keep_hi - 1, else at the nearer end of the unit, as a cut costs more than some tiles. (Units
// too small for that are not cut.)
__device__ __forceinline__ bool cuttable(uint32_t w) { return w >= kUnit + 2 * kSnap; }
__device__ __forceinline__ uint32_t keep_lo(uint32_t w) {
    return cuttable(w) ? kUnit + kSnap : (w + 1) / 2;
}
__device__ __forceinline__ uint32_t keep_hi(uint32_t w) {
    return cuttable(w) ? w - kSnap : keep_lo(w);
}
__device__ __forceinline__ uint32_t cut(const Place& u, uint32_t at) {
    const uint32_t in = at - u.u0;
    return in < keep_lo(u.w) ? u.u0 : in >= keep_hi(u.w) ? u.u0 + u.w : at;
}

// A walk through the units of the CTA's stretch [cur, end); every role warp has its own.
struct Walk {
    uint32_t cur, end, u0;
    int b, mb, h;
    Shape s;
    // of the unit
    int live, kvend, tiles, v0, v1;
    uint32_t w;
    // The first position that some token of the unit does not see, and whether the stretch has it.
    __device__ __forceinline__ int hidden(const PagedParams& p) const {
        return s.s0() + mb * p.tq + 1;
    }
    __device__ __forceinline__ bool hides(const PagedParams& p) const {
        const int at = hidden(p);
        return at < kvend && at < v1 * kStep;
    }
    __device__ __forceinline__ void unit(const PagedParams& p) {
        live = live_rows(p, s, mb);
        kvend = kv_end(p, s, mb);
        tiles = tiles_of(p, s, mb);
        w = tiles * kWeight + kUnit;
        const uint32_t in = cur - u0, out = min(w, end - u0);
        v0 = in > kUnit ? (in - kUnit) / kWeight : 0;
        v1 = out == w ? tiles : (out - kUnit) / kWeight;
    }
    // From the unit that holds `from` or ends there; false if there is nothing before `to`.
    __device__ __forceinline__ bool start(const PagedParams& p, const Place& u, uint32_t from,
                                          uint32_t to) {
        cur = from;
        end = to;
        u0 = u.u0;
        b = u.b;
        mb = u.mb;
        h = u.h;
        s = shape_of(p, u.r);
        w = u.w;
        if (from >= to) return false;
        if (from >= u0 + w) return next(p);
        unit(p);
        return true;
    }
    // The next unit; false at the stretch's end.
    __device__ __forceinline__ bool next(const PagedParams& p) {
        u0 += w;
        cur = u0;
        if (cur >= end) return false;
        if (++h == p.n_kv_heads) {
            h = 0;
            if (++mb == s.nmb) {
                mb = 0;
                Row r;
                bool bad;
                do r = row_of(p, ++b, bad);
                while (r.n == 0 && b + 1 < p.batch);
                s = shape_of(p, r);
            }
        }
        unit(p);
        return true;
    }
};

enum PgBar {
    kBarFullK = 0,                      // K of slot s landed (TMA bytes)
    kBarFreeK = kBarFullK + kSlotsK,    // the products that read it are done (MMA commit)
    kBarFullV = kBarFreeK + kSlotsK,    // the same for V
    kBarFreeV = kBarFullV + kSlotsV,
    kBarS = kBarFreeV + kSlotsV,        // scores written (MMA commit)
    kBarRead = kBarS + 1,               // scores read by every row (an arrival per warp)
    kBarP = kBarRead + 1,               // weights written by every row (an arrival per warp)
    kBarO = kBarP + 1,                  // the products with V done (MMA commit)
    kBarQ = kBarO + 1,                  // the unit's rows staged (an arrival per warp)
    kBarScan = kBarQ + 1,               // the unit's hidden rows of V looked through (an arrival)
    kBarDrain = kBarScan + 1,           // every MMA issued so far done (after a failure)
    kBarCount = kBarDrain + 1
};

__device__ __forceinline__ void rows_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kRowThreads) : "memory");
}
// Whether `x` holds in any of the row threads.
__device__ __forceinline__ bool rows_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(kRowThreads)
        : "memory");
    return r != 0;
}
// Whether phase `parity` of the barrier is complete, without waiting. Asked for ahead of the use:
// an answer takes about a hundred cycles.
__device__ __forceinline__ bool mbar_done(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The warp's wait for a phase, of which `done` may tell that it is complete.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, bool done = false) {
    if (__all_sync(0xffffffffu, done)) return true;
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}
// One arrival for the warp, behind what its lanes did.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

struct Smem {
    uint8_t *k, *v, *q;
    uint64_t* bars;
    float2* ml;      // [128]
    float4* part;    // [128]
    int32_t* odd;    // [3][64], see scan_hidden
    __device__ __forceinline__ uint32_t bar(int i) const { return smem_u32(&bars[i]); }
};

__device__ __forceinline__ Smem smem_at(uint8_t* base) {
    Smem sm;
    sm.k = base;
    sm.v = sm.k + kSlotsK * kStepBytes;
    sm.q = sm.v + kSlotsV * kStepBytes;
    sm.bars = reinterpret_cast<uint64_t*>(sm.q + kPgQBytes);
    sm.ml = reinterpret_cast<float2*>(sm.q + kPgQBytes + 256);
    sm.part = reinterpret_cast<float4*>(sm.ml + kPgRows);
    sm.odd = reinterpret_cast<int32_t*>(sm.part + kRowThreads);
    return sm;
}

// The loop over a unit's tiles takes all registers that a thread has. So what the row warps need
// before and behind it is not kept meanwhile: the walk lies in shared memory, a copy per warp,
// written by every lane alike; addresses and the thread's number are formed anew (these forms keep
// the compiler from saving them). With 25 registers spilled around the loop a chunk of 512 tokens
// over 16384 positions took 94 us, without 75.
template <typename S> __device__ __forceinline__ void put_away(uint32_t* to, const S& s) {
    uint32_t w[sizeof(S) / 4];
    memcpy(w, &s, sizeof(S));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < (int)sizeof(S) / 4; ++i) reinterpret_cast<volatile uint32_t*>(to)[i] = w[i];
    __syncwarp();
}
template <typename S> __device__ __forceinline__ S take_back(const uint32_t* from) {
    uint32_t w[sizeof(S) / 4];
#pragma unroll
    for (int i = 0; i < (int)sizeof(S) / 4; ++i)
        w[i] = reinterpret_cast<const volatile uint32_t*>(from)[i];
    S s;
    memcpy(&s, w, sizeof(S));
    return s;
}
__device__ __forceinline__ uint8_t* smem_base(uint8_t* raw) {
    asm volatile("" : "+l"(raw));
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
}
// 16 bytes into shared memory, the first n of them from `from`, the others zeros.
__device__ __forceinline__ void cp_async16_part(uint32_t to, const void* from, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n)
                 : "memory");
}
__device__ __forceinline__ int row_thread() {
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    return t;
}

// ------------------------------------------------- infinities and NaN behind the mask --
// Positions that only some tokens of a unit see have weight 0 for the others, and 0 * inf is NaN.
// So what is not finite in those rows of V is taken out before the product, and noted: the first
// position of each dim with +inf, -inf and NaN. It is added to the outputs of the tokens that see
// it (repair). One warp, behind the copy of the tile at `base` and before the product that reads
// it; positions lo .. hi - 1. Returns whether there was any.
template <typename T>
__device__ __forceinline__ bool scan_hidden(uint32_t tile, int base, int lo, int hi, int32_t* odd) {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    bool any = false;
    for (int x = threadIdx.x & 31; x < (hi - lo) * 8; x += 32) {
        const int pos = lo + (x >> 3);
        const uint32_t at = tile + swz(pos - base, x & 7);
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at)
                     : "memory");
        bool here = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) here |= ((w[i >> 1] >> (16 * (i & 1))) & kExp) == kExp;
        if (!here) continue;
        any = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
            if ((v & kExp) != kExp) continue;
            const int kind = (v & 0x7fffu) != kExp ? 2 : (int)(v >> 15);
            atomicMin(odd + kind * kHeadDim + (x & 7) * 8 + i, pos);
            w[i >> 1] &= i & 1 ? 0xffffu : 0xffff0000u;
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3])
                     : "memory");
    }
    any = __any_sync(0xffffffffu, any);
    if (any) fence_proxy_async();
    __syncwarp();
    return any;
}
__device__ __forceinline__ int lds_s32(uint32_t at) {
    int v;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
// A lane's outputs, with what scan_hidden took out at positions before `lim`; of a copy of the row,
// with those of its W positions of a tile from `base` on.
__device__ __forceinline__ void repair(uint32_t t_o, uint32_t odd, int lim, int base, int W) {
#pragma unroll 1
    for (int h = 0; h < kHeadDim; h += 16) {
        float o[16];
        uint32_t w[16];
        tc_ld16(t_o + h, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int kind = 0; kind < 3; ++kind) {
                const int pos = lds_s32(odd + 4 * (kind * kHeadDim + h + i));
                if (pos < lim && (uint32_t)(pos % kStep - base) < (uint32_t)W)
                    o[i] += __uint_as_float(kind == 0 ? 0x7f800000u
                                                      : kind == 1 ? 0xff800000u : 0x7fffffffu);
            }
            w[i] = __float_as_uint(o[i]);
        }
        tc_st16_u(t_o + h, w);
    }
}

// ---------------------------------------------------------------- the rows ----------
// Tiles of a unit from v0 on, with numbers it .. end - 1 in the CTA: scores into weights, one row
// per thread. REP copies of the rows, each with W = 128 / REP positions of a tile. Keys t < lim are
// visible, and t < kvend to any row. scan: -1, or the phase of kBarScan. (A function of its own, so
// that what the caller keeps takes no registers from the loop.)
struct RowsEnd {
    float m, l;  // this thread's reference (log2 units) and sum
    bool ok;     // every wait ended
};
template <typename T, int REP>
__device__ __noinline__ RowsEnd run_rows(float scale_log2, uint32_t bars, uint32_t tmem, int v0,
                                         uint32_t it, uint32_t end, int kvend, int lim, int scan) {
    static_assert(REP == 1 || REP == 4, "W is 128 or 32");
    constexpr int W = kStep / REP;
    const int tid = threadIdx.x;
    const int base = REP == 1 ? 0 : tid / (kPgRows / REP) * W;  // of the copy's positions in a tile
    const uint32_t lanes = tmem + ((uint32_t)(tid & ~31) << 16);
    const uint32_t t_s = lanes + base, t_o = lanes + kPgColsO, t_p = lanes + kPgColsP;
    bool first_tile = true;
    float m = -INFINITY, l = 0.f;
    if (REP > 1) {
        // what the other copies hold stays zero in this lane
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0u;
        tc_st32_u(t_p, z);
        tc_st32_u(t_p + 32, z);
    }
    int t0 = v0 * kStep + base;  // of this thread's positions
    bool s_done = false;
    for (; it != end; ++it, t0 += kStep, first_tile = false) {
        if (!warp_wait(bars + 8 * kBarS, it & 1, s_done)) return {m, l, false};
        tc_fence_after();
        bool p_free = false;
        uint32_t w[W / 2];
        if (__builtin_expect(__all_sync(0xffffffffu, t0 >= lim), 0)) {
            // the warp sees nothing of it
            tc_fence_before();
            warp_arrive(bars + 8 * kBarRead);
#pragma unroll
            for (int i = 0; i < W / 2; ++i) w[i] = 0u;
        } else {
            float s[W];
            if constexpr (W == 128) tc_ld128(t_s, s);
            else tc_ld32(t_s, s);
            tc_fence_before();
            warp_arrive(bars + 8 * kBarRead);
            if (__builtin_expect(__any_sync(0xffffffffu, t0 + W > lim), 0)) {
#pragma unroll
                for (int i = 0; i < W; ++i) s[i] = t0 + i < lim ? s[i] : -INFINITY;
            }
            float pm[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                pm[e] = s[e];
#pragma unroll
                for (int i = e + 8; i + 8 < W; i += 16) pm[e] = max3(pm[e], s[i], s[i + 8]);
                pm[e] = fmaxf(pm[e], s[W - 8 + e]);
            }
            const float tmax = max3(max3(pm[0], pm[1], pm[2]), max3(pm[3], pm[4], pm[5]),
                                    fmaxf(pm[6], pm[7])) * scale_log2;
            const bool grow = tmax > m + kPgGrow;
            if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
                float factor = 1.f;
                if (grow) {
                    factor = exp2f(m - tmax);  // 0 on the first tile
                    m = tmax;
                }
                l *= factor;
                if (!first_tile) {
                    // O is rescaled once P.V of the tile before is done
                    if (!warp_wait(bars + 8 * kBarO, (it - 1) & 1)) return {m, l, false};
                    tc_fence_after();
                    float ov[16];
                    uint32_t ow[16];
#pragma unroll 1
                    for (int h = 0; h < kHeadDim; h += 16) {
                        tc_ld16(t_o + h, ov);
#pragma unroll
                        for (int i = 0; i < 16; ++i) ow[i] = __float_as_uint(ov[i] * factor);
                        tc_st16_u(t_o + h, ow);
                    }
                }
            }
            // the weights, rounded to the storage type; their sum is taken before that (rounding
            // to nearest leaves no bias, but where binary16 has no values any more: see kPgLift)
            if (!first_tile) p_free = mbar_done(bars + 8 * kBarO, (it - 1) & 1);
            const float nref = m == -INFINITY ? 0.f : kPgLift<T> - m;
            const Pair cs2(scale_log2, scale_log2), ref2(nref, nref);
            Pair sum[4] = {Pair(0.f, 0.f), Pair(0.f, 0.f), Pair(0.f, 0.f), Pair(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                const float2 x = fma2(Pair(s[2 * i], s[2 * i + 1]), cs2, ref2).get();
                const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                sum[i & 3] = add2(sum[i & 3], Pair(e.x, e.y));
                w[i] = Half16<T>::from_f2(e.x, e.y);
            }
            const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])).get();
            l += all.x + all.y;
        }
        // the weights' last reader is P.V of the tile before
        if (!first_tile && !warp_wait(bars + 8 * kBarO, (it - 1) & 1, p_free)) return {m, l, false};
        tc_fence_after();
        s_done = it + 1 != end && mbar_done(bars + 8 * kBarS, (it + 1) & 1);
        if constexpr (W == 128) {
            tc_st32_u(t_p, w);
            tc_st32_u(t_p + 32, w + 32);
        } else {
            tc_st16_u(t_p + base / 2, w);
        }
        const int first = kvend - (t0 - base);
        if (__builtin_expect(first < kStep, 0)) {
            // Positions past the last visible one hold other data (or nothing): P is 0 there, but
            // 0 * NaN would still poison P.V, so those V rows are cleared once the copy landed.
            const uint32_t slot = it % kSlotsV;
            if (!warp_wait(bars + 8 * (kBarFullV + slot), (it / kSlotsV) & 1))
                return {m, l, false};
            const uint32_t vt = bars - kPgQBytes - (kSlotsV - slot) * kStepBytes;
            for (int x = tid; x < (kStep - first) * 8; x += kRowThreads)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 vt + swz(first + (x >> 3), x & 7)),
                             "r"(0u)
                             : "memory");
            fence_proxy_async();
        }
        tc_fence_before();
        warp_arrive(bars + 8 * kBarP);
    }
    if (scan >= 0) {
        if (!warp_wait(bars + 8 * kBarO, (end - 1) & 1) || !warp_wait(bars + 8 * kBarScan, scan))
            return {m, l, false};
        tc_fence_after();
        const uint32_t odd = bars + kOddOffset;
        if (lds_s32(odd + 4 * kOddWords)) repair(t_o, odd, lim, base, W);
    }
    return {m, l, true};
}

// Where 4 dims of vector r of a unit go.
template <typename T>
__device__ __forceinline__ T* out_row(const PagedParams& p, const Walk& u, int r) {
    const int tok = r / p.group, hg = r - tok * p.group;
    const int64_t t = u.s.r.s + (int64_t)u.mb * p.tq + tok;
    return static_cast<T*>(p.out) + (t * p.n_q_heads + u.h * p.group + hg) * kHeadDim;
}
// 0 * x of eight values.
template <typename T>
__device__ __forceinline__ uint4 times_zero(const uint4& x) {
    float f[8];
    unpack8<T>(x, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= 0.f;
    return make_uint4(Half16<T>::from_f2(f[0], f[1]), Half16<T>::from_f2(f[2], f[3]),
                      Half16<T>::from_f2(f[4], f[5]), Half16<T>::from_f2(f[6], f[7]));
}
template <typename T>
__device__ __forceinline__ uint2 pack4(const float4& o, float inv) {
    return make_uint2(Half16<T>::from_f2(o.x * inv, o.y * inv),
                      Half16<T>::from_f2(o.z * inv, o.w * inv));
}

// Of a unit held several times: a copy has weight 0 at the other copies' positions, so an infinity
// in a row of V that all its tokens see (scan_hidden takes out the others) has made that dim NaN in
// the joined outputs. Its rows of V, positions lo .. hi - 1, are then read again, and outputs that
// have an infinity or NaN among the positions that they see become what the sum with it is. Row y
// sees positions below lim0 + y / group; ml: the copies' sums; to: the partial of a piece, or null.
// The row threads, behind a barrier; ends before one. (To look through every tile of V before its
// product, as scan_hidden does, took 2 % more for 32 rows to 16384, 9 % for 8 rows of 5 tokens and
// 30 % for the mixed batch; this nothing, and 4.2 times as long for 32 rows with infinities.) The
// copying and the MMA warp wait meanwhile, for a second at most; it takes 40 ns a position, and a
// pool of 280 GB gives a block pieces of 4 million positions.
template <typename T, int REP>
__device__ __noinline__ void odd_of_copies(const PagedParams& p, int32_t* odd, const float2* ml,
                                           int b, int h, int live, int lo, int hi, int lim0,
                                           int64_t first, float* to) {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    const int tid = threadIdx.x;
    for (int i = tid; i < kOddWords; i += kRowThreads) odd[i] = INT_MAX;
    rows_sync();
    const int32_t* pages = p.table + b * p.table_stride;
    const uint8_t* v = p.v + h * p.v_sh + (tid & 7) * 16;
    constexpr int kAhead = 2;
#pragma unroll 1
    for (int at = lo + (tid >> 3); at < hi; at += kAhead * (kRowThreads / 8)) {
        int page[kAhead];
        uint4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int pos = at + k * (kRowThreads / 8);
            page[k] = pos < hi ? __ldg(pages + (pos >> p.page_log2)) : -1;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int slot = (at + k * (kRowThreads / 8)) & ((1 << p.page_log2) - 1);
            x[k] = make_uint4(0u, 0u, 0u, 0u);  // (as pages outside the pool count)
            if (page[k] >= 0 && page[k] < p.n_pages)
                x[k] = __ldg(reinterpret_cast<const uint4*>(v + page[k] * p.v_sp + slot * p.v_st));
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t e = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
                if ((e & kExp) != kExp) continue;
                const int kind = (e & 0x7fffu) != kExp ? 2 : (int)(e >> 15);
                atomicMin(odd + kind * kHeadDim + (tid & 7) * 8 + i, at + k * (kRowThreads / 8));
            }
        }
    }
    rows_sync();
#pragma unroll 1
    for (int x = tid; x < live * kHeadDim; x += kRowThreads) {
        const int y = x / kHeadDim, d = x % kHeadDim, tok = y / p.group;
        const int lim = lim0 + tok;
        const bool above = odd[d] < lim, below = odd[kHeadDim + d] < lim;
        const bool none = odd[2 * kHeadDim + d] < lim;
        float l = 0.f;
        for (int k = 0; k < REP; ++k) l += ml[y + k * (kPgRows / REP)].y;
        if (!(above || below || none) || l != l) continue;  // (a weight is NaN: so are the outputs)
        const float o = none || (above && below) ? __uint_as_float(0x7fffffffu)
                                                 : above ? INFINITY : -INFINITY;
        if (to)
            to[((d / 4) * p.slot_rows + y) * 4 + d % 4] = o;
        else
            static_cast<T*>(p.out)[((first + tok) * p.n_q_heads + h * p.group + y -
                                    tok * p.group) * kHeadDim + d] = Half16<T>::from_f(o);
    }
    rows_sync();
    for (int i = tid; i < kOddWords; i += kRowThreads) odd[i] = INT_MAX;  // (as scan_hidden does)
}

// The unit's outputs from tensor memory: written, or (a piece of the unit) left in the workspace.
// Every product of the unit is done.
template <typename T, int REP>
__device__ __forceinline__ void finish_rows(const PagedParams& p, const Smem& sm, uint32_t tmem,
                                            const Walk& u, bool whole, int slot, float m,
                                            float l) {
    const int tid = threadIdx.x;
    constexpr int R = kPgRows / REP;
    const int r = tid & (R - 1);
    const uint32_t t_o = tmem + ((uint32_t)(tid & ~31) << 16) + kPgColsO;
    float4* wsp = p.ws_part + (int64_t)slot * 16 * p.slot_rows;  // + 4 dims * slot_rows + row
    float2* wsm = p.ws_ml + (int64_t)slot * p.slot_rows;
    if constexpr (REP == 1) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float o[32];
            tc_ld32(t_o + half * 32, o);
            if (r < u.live) {
                if (whole) {
                    uint4* dst = reinterpret_cast<uint4*>(out_row<T>(p, u, r) + half * 32);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint2 a = pack4<T>(make_float4(o[8 * c], o[8 * c + 1], o[8 * c + 2],
                                                             o[8 * c + 3]), inv);
                        const uint2 b = pack4<T>(make_float4(o[8 * c + 4], o[8 * c + 5],
                                                             o[8 * c + 6], o[8 * c + 7]), inv);
                        dst[c] = make_uint4(a.x, a.y, b.x, b.y);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        wsp[(half * 8 + c) * p.slot_rows + r] =
                            make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                }
            }
        }
        if (!whole && r < u.live) wsm[r] = make_float2(m, l);
    } else {
        // the copies' partials meet in the rows' shared memory (every S is done), 32 dims at a
        // time where all 64 do not fit
        sm.ml[tid] = make_float2(m, l);
        float o[64];
        tc_ld64(t_o, o);
        float4* buf = reinterpret_cast<float4*>(sm.q);
        // (places for 4, 16 or 32 rows: with 16 for the 4 of a decoding row most threads idle)
        const int phases = u.live > 16 ? 2 : 1, quads = 16 / phases;
        const int log_rows = u.live > 16 ? 5 : u.live > 4 ? 4 : 2, rows = 1 << log_rows;
        bool finite = true;
#pragma unroll 1
        for (int h = 0; h < phases; ++h) {
            if (r < u.live) {  // [quad][copy][row]
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    buf[(c * REP + tid / R) * rows + r] =
                        make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                if (phases == 1) {
#pragma unroll
                    for (int c = 8; c < 16; ++c)
                        buf[(c * REP + tid / R) * rows + r] =
                            make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                }
            }
            rows_sync();
            for (int x = tid; x < quads * rows; x += kRowThreads) {
                const int y = x & (rows - 1), c = x >> log_rows;
                if (y >= u.live) continue;
                float top = -INFINITY, all = 0.f;
#pragma unroll
                for (int k = 0; k < REP; ++k) top = fmaxf(top, sm.ml[y + k * R].x);
                const float ref = top == -INFINITY ? 0.f : top;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < REP; ++k) {
                    const float2 ml = sm.ml[y + k * R];
                    const float4 b = buf[(c * REP + k) * rows + y];
                    const float f = ex2_approx(ml.x - ref);
                    all = fmaf(ml.y, f, all);
                    a.x = fmaf(b.x, f, a.x);
                    a.y = fmaf(b.y, f, a.y);
                    a.z = fmaf(b.z, f, a.z);
                    a.w = fmaf(b.w, f, a.w);
                }
                const int d4 = h * 8 + c;
                finite = finite && fabsf((a.x + a.y) + (a.z + a.w)) < INFINITY;
                if (whole) {
                    *reinterpret_cast<uint2*>(out_row<T>(p, u, y) + d4 * 4) =
                        pack4<T>(a, all > 0.f ? 1.f / all : 0.f);
                } else {
                    wsp[d4 * p.slot_rows + y] = a;
                    if (d4 == 0) wsm[y] = make_float2(top, all);
                }
            }
            if (phases == 2) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = o[32 + i];
            }
            // read before the second half, or the next unit's rows, are written
            finite = !rows_any(!finite);
        }
        if (__builtin_expect(!finite, 0)) {
            const int t0 = u.mb * p.tq;  // of the row's new tokens
            odd_of_copies<T, REP>(p, sm.odd, sm.ml, u.b, u.h, u.live, u.v0 * kStep,
                                  min(u.kvend, u.v1 * kStep), u.s.s0() + t0 + 1,
                                  (int64_t)u.s.r.s + t0,
                                  whole ? nullptr : reinterpret_cast<float*>(wsp));
        }
    }
}

// Partials (reference, sum, Q quads of dims) joined, N at a time.
template <int Q>
struct Joined {
    float top, l;
    float4 o[Q];
    __device__ __forceinline__ void clear() {
        top = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int c = 0; c < Q; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // The first n of them.
    template <int N>
    __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N][Q], int n) {
        float t = top;
#pragma unroll
        for (int k = 0; k < N; ++k) t = fmaxf(t, k < n ? ml[k].x : t);
        const float ref = t == -INFINITY ? 0.f : t, f0 = ex2_approx(top - ref);
        top = t;
        l *= f0;
#pragma unroll
        for (int c = 0; c < Q; ++c) {
            o[c].x *= f0;
            o[c].y *= f0;
            o[c].z *= f0;
            o[c].w *= f0;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (k >= n) break;
            const float f = ex2_approx(ml[k].x - ref);
            l = fmaf(ml[k].y, f, l);
#pragma unroll
            for (int c = 0; c < Q; ++c) {
                o[c].x = fmaf(v[k][c].x, f, o[c].x);
                o[c].y = fmaf(v[k][c].y, f, o[c].y);
                o[c].z = fmaf(v[k][c].z, f, o[c].z);
                o[c].w = fmaf(v[k][c].w, f, o[c].w);
            }
        }
    }
    __device__ __forceinline__ float inv() const { return l > 0.f ? 1.f / l : 0.f; }
};

// Loads that are issued where they stand. (The compiler would put them behind the tests for which
// piece is there, one round trip after the other.)
__device__ __forceinline__ float4 load_now(const float4* at) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 load_now(const float2* at) {
    float2 v;
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(at) : "memory");
    return v;
}

// Pieces i .. last - 1 of row r, quads c .. c + Q - 1, N pieces in flight. (The first CTA's lies
// one slot further.) One warp runs on each scheduler here, so every instruction counts: an address
// worked out per piece instead of a step cost one row of 8192 positions 1.2 us.
template <int Q, int N>
__device__ __forceinline__ Joined<Q> join_pieces(const PagedParams& p, int i0, int i, int last,
                                                 int r, int c) {
    Joined<Q> a;
    a.clear();
    const int S = p.slot_rows;
#pragma unroll 1
    for (; i < last; i += N) {
        // (2 x 512 slots of 16 x 128 places: indexes of 32 bits)
        const int slot = (2 * (i0 + i) + (i == 0)) * S, back = i == 0 ? S : 0;
        const float2* at_ml = p.ws_ml + (slot + r);
        const float4* at_v = p.ws_part + (slot * 16 + c * S + r);
        float2 ml[N];
        float4 v[N][Q];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (k > 0 && i + k < last) {
                at_ml += 2 * S - (k == 1 ? back : 0);
                at_v += (2 * S - (k == 1 ? back : 0)) * 16;
            }
            ml[k] = load_now(at_ml);
#pragma unroll
            for (int q = 0; q < Q; ++q) v[k][q] = load_now(at_v + q * S);
        }
        a.add(ml, v, last - i);
    }
    return a;
}

// A cut unit's pieces, which lie in the workspace: CTAs i0 .. i0 + n - 1, the last to arrive merges
// them in that order.
template <typename T>
__device__ __forceinline__ void merge_pieces(const PagedParams& p, const Smem& sm, const Walk& u,
                                             int i0, int n, int* s_last) {
    const int tid = threadIdx.x;
    rows_sync();
    if (tid == 0) {
        // (released and acquired for the other threads of the block by the barriers around it)
        int old;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                     : "=r"(old)
                     : "l"(p.ws_cnt + i0)
                     : "memory");
        *s_last = old == n - 1;
    }
    rows_sync();
    if (!*s_last) return;
    if (tid == 0) p.ws_cnt[i0] = 0;
    // (two rows of 211 tokens at 11523, 24 pieces of 128 rows a unit: 34 us; a thread per 4 dims of
    // a row, 16 turns of it, 60)
    if (u.live > 32) {
        // a thread per row
        if (tid >= u.live) return;
        const Joined<16> a = join_pieces<16, 1>(p, i0, 0, n, tid, 0);
        const float inv = a.inv();
        uint4* dst = reinterpret_cast<uint4*>(out_row<T>(p, u, tid));
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint2 x = pack4<T>(a.o[2 * c], inv), y = pack4<T>(a.o[2 * c + 1], inv);
            dst[c] = make_uint4(x.x, x.y, y.x, y.y);
        }
    } else if (u.live > 8) {
        // a lane per row, a quarter of the dims per warp
        const int r = tid & 31, c = tid / 32 * 4;
        if (r >= u.live) return;
        const Joined<4> a = join_pieces<4, 4>(p, i0, 0, n, r, c);
        const float inv = a.inv();
        uint4* dst = reinterpret_cast<uint4*>(out_row<T>(p, u, r) + c * 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint2 x = pack4<T>(a.o[2 * k], inv), y = pack4<T>(a.o[2 * k + 1], inv);
            dst[k] = make_uint4(x.x, x.y, y.x, y.y);
        }
    } else {
        // a thread per row, 4 dims and, of at most 4 rows, share of the pieces, joined in order
        const int items = u.live * 16, shares = kRowThreads / items;
        const int share = (int)((unsigned)tid / (unsigned)items);  // (of the last threads: none)
        const int y = tid - share * items, c = y & 15, r = y >> 4;
        auto store = [&](const Joined<1>& a) {
            *reinterpret_cast<uint2*>(out_row<T>(p, u, r) + c * 4) = pack4<T>(a.o[0], a.inv());
        };
        Joined<1> a;
        if (share < shares) {
            a = join_pieces<1, 8>(p, i0, n * share / shares, n * (share + 1) / shares, r, c);
            if (shares == 1) {
                store(a);
            } else {
                sm.part[tid] = a.o[0];
                sm.ml[tid] = make_float2(a.top, a.l);
            }
        }
        if (shares > 1) {
            rows_sync();
            if (tid < items) {
                a.clear();
                for (int k = 0; k < shares; ++k) {
                    const float2 ml[1] = {sm.ml[k * items + tid]};
                    const float4 v[1][1] = {{sm.part[k * items + tid]}};
                    a.add(ml, v, 1);
                }
                store(a);
            }
            rows_sync();  // read before the next unit's sums are written
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kPgThreads, kPgMinBlocks)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ PagedParams p) {
    extern __shared__ uint8_t smem_raw[];
    const Smem sm = smem_at(smem_base(smem_raw));
    static_assert(kBarCount * 8 <= 256, "the barriers' place");
    __shared__ Place s_place;
    __shared__ uint32_t s_total, s_least, s_from, s_to, s_tmem;
    __shared__ uint32_t s_walk[kRowThreads / 32][sizeof(Walk) / 4];
    __shared__ int s_last, s_longest[kPgThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool mma_warp = warp == kRowThreads / 32, copy_warp = warp == kRowThreads / 32 + 1;
    if (copy_warp && lane == 0) {
        for (int i = 0; i < kBarCount; ++i)
            mbar_init(sm.bar(i),
                      i == kBarRead || i == kBarP || i == kBarQ ? kRowThreads / 32 : 1);
        fence_barrier_init();
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    pdl_wait();
    pdl_trigger();
    if (mma_warp) {
        tc_alloc(smem_u32(&s_tmem), kPgCols);
        tc_relinquish();
        tc_fence_before();
    }
    // Warp 0 finds where the stretch starts, warp 1 where it ends: each from a list of its own of
    // at most 32 rows, or from the block's table (1 row x 8192 that way: 12.6 us instead of 12.2).
    const bool few = p.batch <= 32;
    Table tab;
    uint32_t total = 0, sum = 0;
    int longest = 0;
    if (!few) {
        tab = fill_table(p, reinterpret_cast<uint32_t*>(sm.q), longest);
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 0) s_longest[warp] = longest;
        __syncthreads();
        if (warp == 0) {
            total = finish_table(tab);
            if (lane == 0) s_total = total;
        }
        __syncthreads();
        total = s_total;
    }
    if (warp < 2) {
        Row mine = {0, 0, 0};
        uint32_t least = kLeast;
        if (few) {
            bool bad = false;
            if (lane < p.batch) mine = row_of(p, lane, bad);
            if (bad && blockIdx.x == 0 && warp == 0) flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
            sum = scan_rows(row_weight(p, mine));
            total = __shfl_sync(0xffffffffu, sum, 31);
            longest = __reduce_max_sync(0xffffffffu, heavy_tiles(p, mine));
        } else {
            longest = __reduce_max_sync(0xffffffffu, lane < kPgThreads / 32 ? s_longest[lane] : 0);
        }
        least = max(least, (uint32_t)(kShare * sqrtf((float)longest)));
        if (total == kTooLong) {
            if (lane == 0 && warp == 0 && blockIdx.x == 0)
                flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
            total = 0;
        }
        const Shares sh = shares(total, least);
        const uint32_t at = sh.start(blockIdx.x + warp);
        if (blockIdx.x >= sh.ctas || at >= total) {
            if (lane == 0) *(warp ? &s_to : &s_from) = warp ? total : 0xffffffffu;
        } else {
            Place u;
            uint32_t before;
            bool bad;
            if (few) {
                u.b = __popc(__ballot_sync(0xffffffffu, sum <= at));
                before = __shfl_sync(0xffffffffu, sum, max(u.b - 1, 0));
                if (u.b == 0) before = 0;
                u.r.s = __shfl_sync(0xffffffffu, mine.s, u.b);
                u.r.n = __shfl_sync(0xffffffffu, mine.n, u.b);
                u.r.len = __shfl_sync(0xffffffffu, mine.len, u.b);
            } else {
                u.b = find_row(p, tab, at, before);
                u.r = row_of(p, u.b, bad);
            }
            find_unit(p, u, at, before);
            if (lane == 0) {
                if (warp == 0) s_place = u;
                *(warp ? &s_to : &s_from) = cut(u, at);
            }
        }
        if (tid == 0) {
            s_total = total;
            s_least = least;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    Walk u;
    bool ok = u.start(p, s_place, s_from, s_to);
    if (!ok) {
        if (mma_warp) tc_dealloc(tmem, kPgCols);
        return;
    }

    if (copy_warp) {
        // ---- K/V tiles, a slot each ----
        uint32_t it = 0, it_k = 0;  // tiles of V and K copied
        const int in_page = (1 << p.page_log2) - 1;
        do {
            // lane i: box i of K, lane 16 + i: box i of V
            const int box = lane & 15;
            const bool mine = box < p.boxes, is_v = lane >= 16;
            const int32_t* row = p.table + u.b * p.table_stride;
            auto page_of = [&](int v) {
                const int pos = v * kStep + box * p.box_rows;
                return mine && v < u.v1 && pos < u.kvend ? __ldg(row + (pos >> p.page_log2)) : 0;
            };
            int page = page_of(u.v0);
            for (int v = u.v0; ok && v < u.v1; ++v, ++it) {
                const int pos = v * kStep + box * p.box_rows;
                const bool on = mine && pos < u.kvend;
                int pg = page;
                page = page_of(v + 1);
                if (on && (pg < 0 || pg >= p.n_pages)) {
                    flag_error(p.dev_err, KVD_ERR_BAD_INDEX);
                    pg = p.n_pages;  // outside the tensor: zeros
                }
                const uint32_t bytes =
                    __popc(__ballot_sync(0xffffffffu, on)) / 2 * p.box_rows * kRowBytes;
                auto copy = [&](int slots, int full, int free, const uint8_t* to,
                                const CUtensorMap* map, bool half) {
                    const uint32_t slot = it % slots, turn = it / slots;
                    if (turn > 0 && !warp_wait(sm.bar(free + slot), (turn - 1) & 1)) return false;
                    const uint32_t bar = sm.bar(full + slot);
                    if (lane == 0) {
                        // test only: 16 bytes more than the copies bring
                        if (p.test_stall && it == 0) mbar_expect_tx_only(bar, 16);
                        mbar_expect_tx(bar, bytes);
                    }
                    __syncwarp();
                    if (on && half)
                        tma_load_4d(smem_u32(to + slot * kStepBytes) + box * p.box_rows * kRowBytes,
                                    map, bar, 0, pos & in_page, u.h, pg);
                    __syncwarp();
                    return true;
                };
                if (!(ok = copy(kSlotsK, kBarFullK, kBarFreeK, sm.k, &tmk, !is_v))) break;
                ++it_k;
                if (!(ok = copy(kSlotsV, kBarFullV, kBarFreeV, sm.v, &tmv, is_v))) break;
            }
        } while (ok && u.next(p));
        if (!ok) {
            if (lane == 0) flag_error(p.dev_err, KVD_ERR_TIMEOUT);
            // the copies in flight land before the block leaves
            for (uint32_t i = it_k > kSlotsK ? it_k - kSlotsK : 0; i < it_k; ++i)
                mbar_wait_bounded(sm.bar(kBarFullK + i % kSlotsK), (i / kSlotsK) & 1);
            for (uint32_t i = it > kSlotsV ? it - kSlotsV : 0; i < it; ++i)
                mbar_wait_bounded(sm.bar(kBarFullV + i % kSlotsV), (i / kSlotsV) & 1);
        }
    } else if (mma_warp) {
        // ---- the products: the whole warp runs the loop, one elected lane issues ----
        constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
        constexpr uint32_t kIdS = tc_idesc_f16(kBf16, kPgRows, kStep, false);
        constexpr uint32_t kIdO = tc_idesc_f16(kBf16, kPgRows, kHeadDim, true);
        const uint64_t qdesc = tc_desc_sw128(smem_u32(sm.q));
        const uint64_t kdesc = tc_desc_sw128(smem_u32(sm.k)), vdesc = tc_desc_sw128(smem_u32(sm.v));
        constexpr uint64_t kStepDesc = kStepBytes / 16;  // a descriptor's addresses: 16 bytes
        const uint32_t lead = elect_one();
        auto issue_s = [&](uint32_t it) -> bool {
            const uint32_t slot = it % kSlotsK;
            if (!warp_wait(sm.bar(kBarFullK + slot), (it / kSlotsK) & 1)) return false;
            tc_fence_after();
            const uint64_t kd = kdesc + slot * kStepDesc;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                tc_mma_f16_if(lead, tmem, qdesc + kk * 2, kd + kk * 2, kIdS, kk > 0);
            tc_commit_if(lead, sm.bar(kBarS));
            tc_commit_if(lead, sm.bar(kBarFreeK + slot));
            return true;
        };
        uint32_t it = 0, units = 0;
        bool odd = true;  // (at first: what the table holds is not known)
        do {
            if (!(ok = warp_wait(sm.bar(kBarQ), units & 1))) break;
            tc_fence_after();
            // (the rows are done with the last unit's)
            const bool hides = u.hides(p);
            const int hidden = u.hidden(p);
            if (hides && odd) {
                for (int i = lane; i < kOddWords; i += 32) sm.odd[i] = INT_MAX;
                __syncwarp();
                odd = false;
            }
            const int nt = u.v1 - u.v0;
            ok = issue_s(it);
            auto tile = [&](int j, bool scan) {
                // the next scores as soon as the rows have read these, while they form the weights
                if (!warp_wait(sm.bar(kBarRead), it & 1)) return false;
                if (j + 1 < nt && !issue_s(it + 1)) return false;
                const uint32_t slot = it % kSlotsV;
                if (!warp_wait(sm.bar(kBarFullV + slot), (it / kSlotsV) & 1)) return false;
                if (scan) {
                    const int base = (u.v0 + j) * kStep;
                    odd |= scan_hidden<T>(smem_u32(sm.v) + slot * kStepBytes, base,
                                          max(hidden, base), min(u.kvend, base + kStep), sm.odd);
                }
                if (!warp_wait(sm.bar(kBarP), it & 1)) return false;
                tc_fence_after();
                const uint64_t vd = vdesc + slot * kStepDesc;
                tc_mma_f16_tmem_a_if(lead, tmem + kPgColsO, tmem + kPgColsP, vd, kIdO, j > 0);
#pragma unroll
                for (int kk = 1; kk < kStep / 16; ++kk)
                    tc_mma_f16_tmem_a_if(lead, tmem + kPgColsO, tmem + kPgColsP + kk * 8,
                                         vd + kk * (16 * kRowBytes / 16), kIdO, 1);
                tc_commit_if(lead, sm.bar(kBarO));
                tc_commit_if(lead, sm.bar(kBarFreeV + slot));
                ++it;
                return true;
            };
            const int seen = hides ? max(hidden / kStep - u.v0, 0) : nt;  // tiles that all see
            int j = 0;
            for (; ok && j < seen; ++j) ok = tile(j, false);
#pragma unroll 1
            for (; ok && j < nt; ++j) ok = tile(j, true);
            ++units;
            if (ok && hides) {
                if (lane == 0) sm.odd[kOddWords] = odd;
                warp_arrive(sm.bar(kBarScan));
            }
        } while (ok && u.next(p));
        if (!ok) {
            if (lead) {
                flag_error(p.dev_err, KVD_ERR_TIMEOUT);
                tc_commit(sm.bar(kBarDrain));
                mbar_wait_bounded(sm.bar(kBarDrain), 0);
            }
            __syncwarp();
        }
    } else {
        // ---- the rows ----
        uint32_t it0 = 0, scans = 0;
        auto walk = [&]() { return s_walk[row_thread() / 32]; };
        // this thread's query row (zeros past the unit's) on its way into the swizzled A operand,
        // and handed over
        auto fetch_q = [&](const Walk& u) {
            const uint32_t to = smem_u32(smem_at(smem_base(smem_raw)).q);
            const int r = row_thread() & (kPgRows / copies_of(u.live, u.tiles) - 1);
            const int from = r < u.live ? r : 0, tok = from / p.group, hg = from - tok * p.group;
            const int64_t t = u.s.r.s + (int64_t)u.mb * p.tq + tok;
            const uint8_t* src = p.q + t * p.q_st + (int64_t)(u.h * p.group + hg) * p.q_sh;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                cp_async16_part(to + swz(row_thread(), c), src + c * 16, r < u.live ? 16 : 0);
            cp_async_commit();
        };
        auto stage_q = [&]() {
            const Smem sm = smem_at(smem_base(smem_raw));
            cp_async_wait_all();
            if (p.scale_sign <= 0) {
                // (the loop over the tiles knows positive scales only)
                const uint32_t flip = p.scale_sign < 0 ? 0x80008000u : 0u;
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint4* at = reinterpret_cast<uint4*>(sm.q + swz(row_thread(), c));
                    const uint4 v = *at;
                    *at = flip ? make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip)
                               : times_zero<T>(v);
                }
            }
            fence_proxy_async();
            warp_arrive(sm.bar(kBarQ));
        };
        // the tiles of the unit that is put away
        auto weigh = [&]() {
            const Walk u = take_back<Walk>(walk());
            const uint32_t bars = smem_at(smem_base(smem_raw)).bar(0), end = it0 + u.v1 - u.v0;
            const int rep = copies_of(u.live, u.tiles), r = row_thread() & (kPgRows / rep - 1);
            // keys t < lim are visible; rows past the unit's see all of it (and are not written)
            const int lim = r < u.live ? u.s.s0() + u.mb * p.tq + r / p.group + 1 : u.kvend;
            const int scan = u.hides(p) ? (int)(scans & 1) : -1;
            if (rep == 1)
                return run_rows<T, 1>(p.scale_log2, bars, tmem, u.v0, it0, end, u.kvend, lim, scan);
            return run_rows<T, 4>(p.scale_log2, bars, tmem, u.v0, it0, end, u.kvend, lim, scan);
        };
        put_away(walk(), u);
        fetch_q(u);
        stage_q();
        for (bool more = true; more;) {
            const RowsEnd e = weigh();
            const Walk done = take_back<Walk>(walk());
            u = done;
            more = u.next(p);
            put_away(walk(), u);
            // (every score of the unit is done, so Q's place is free, but for the join of copies)
            const bool early = copies_of(done.live, done.tiles) == 1;
            if (more && early) fetch_q(u);
            const Smem sm = smem_at(smem_base(smem_raw));
            it0 += done.v1 - done.v0;
            scans += done.hides(p);
            ok = e.ok && mbar_wait_bounded(sm.bar(kBarO), (it0 - 1) & 1);
            if (rows_any(!ok)) {
                if (row_thread() == 0) flag_error(p.dev_err, KVD_ERR_TIMEOUT);
                cp_async_wait_all();
                break;
            }
            tc_fence_after();
            const bool whole = done.v0 == 0 && done.v1 == done.tiles;
            const int slot = 2 * (int)blockIdx.x + (done.v0 == 0);
            if (copies_of(done.live, done.tiles) == 1)
                finish_rows<T, 1>(p, sm, tmem, done, whole, slot, e.m, e.l);
            else
                finish_rows<T, 4>(p, sm, tmem, done, whole, slot, e.m, e.l);
            tc_fence_before();  // O is read before the next unit's products
            if (more) {
                if (!early) fetch_q(take_back<Walk>(walk()));
                stage_q();
            }
            if (!whole) {
                const Shares sh = shares(s_total, s_least);
                // (the last share that starts before the unit's first cut, and before its last)
                const uint32_t i0 = sh.holder(done.u0 + keep_lo(done.w) - 1);
                const uint32_t i1 = sh.holder(done.u0 + keep_hi(done.w) - 1);
                merge_pieces<T>(p, sm, done, (int)i0, (int)(i1 - i0) + 1, &s_last);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (mma_warp) {
        tc_fence_after();
        tc_dealloc(tmem, kPgCols);
    }
}

constexpr int kMaxDevP = 64;

// Once per kernel and device: its shared memory.
template <typename T>
bool prepare_paged() {
    static std::once_flag once[kMaxDevP];
    static bool ok[kMaxDevP];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevP) return false;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(paged_attn_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kPgSmem) == cudaSuccess;
        cudaGetLastError();
    });
    return ok[dev];
}

template <typename T>
kvd_status run_paged(PagedParams& p, int nsm, const CUtensorMap& mk, const CUtensorMap& mv,
                     uint8_t* ws, bool pdl, cudaStream_t st) {
    if (!prepare_paged<T>()) return KVD_ERR_CUDA;
    const int blocks = std::min(kMaxCtas, nsm * kPgMinBlocks);
    p.ws_cnt = reinterpret_cast<int32_t*>(ws);
    p.ws_part = reinterpret_cast<float4*>(ws + KVD_WS_COUNTER_BYTES);
    p.ws_ml = reinterpret_cast<float2*>(p.ws_part + (size_t)2 * blocks * 16 * p.slot_rows);
    return launch(paged_attn_kernel<T>, dim3((unsigned)blocks), dim3(kPgThreads), kPgSmem, st,
                  pdl, mk, mv, p);
}

// Query vectors of the largest unit.
int unit_rows(int group, int max_new) {
    return (int)std::min<int64_t>(kPgRows / group, max_new) * group;
}

}  // namespace

size_t paged_workspace_bytes(int n_q_heads, int n_kv_heads, int max_new) {
    return KVD_WS_COUNTER_BYTES + (size_t)2 * kMaxCtas * (kHeadDim + 2) * sizeof(float) *
                                      unit_rows(n_q_heads / n_kv_heads, max_new);
}

}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_paged_attn(kvd_dtype dtype, const kvd_paged_cache* cache,
                                     int32_t n_tokens, int32_t max_new, const kvd_token_rows* q,
                                     const int32_t* starts, const int32_t* lens, float scale,
                                     void* workspace, size_t workspace_bytes, uint32_t flags,
                                     int32_t* dev_err, kvd_stream_t stream) {
    if (dtype != KVD_F16 && dtype != KVD_BF16) return KVD_ERR_INVALID_ARG;
    if (kvd_status s = validate_paged_cache(cache)) return s;
    if (n_tokens < 0 || max_new < 1 || !starts || !lens) return KVD_ERR_INVALID_ARG;
    if (!(scale < INFINITY) || !(scale > -INFINITY)) return KVD_ERR_INVALID_ARG;
    if (n_tokens == 0) return KVD_OK;
    if (kvd_status s = validate_token_rows(q)) return s;
    if (!q->out || q->out == q->x || q->n_heads % cache->n_kv_heads) return KVD_ERR_INVALID_ARG;
    const int group = q->n_heads / cache->n_kv_heads;
    if (group > KVD_MAX_GROUP) return KVD_ERR_UNSUPPORTED;
    max_new = std::min(max_new, n_tokens);
    const size_t need = paged_workspace_bytes(q->n_heads, cache->n_kv_heads, max_new);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need)
        return KVD_ERR_WORKSPACE;
    // the list of tiles, at its longest, is counted in 32 bits
    const int tq = kPgRows / group;
    const double blocks = (double)cache->n_kv_heads * ((double)n_tokens / tq + cache->batch);
    const double longest = kWeight * ((double)cache->table_width * cache->page_size / kStep + 1.);
    if (blocks * (longest + kUnit) > 4e9) return KVD_ERR_UNSUPPORTED;
    const int nsm = sm_count();
    if (nsm <= 0) return KVD_ERR_CUDA;
    CUtensorMap mk, mv;
    if (kvd_status s = encode_pool_map(&mk, dtype, cache->k, cache)) return s;
    if (kvd_status s = encode_pool_map(&mv, dtype, cache->v, cache)) return s;
    PagedParams p = {};
    p.q = static_cast<const uint8_t*>(q->x);
    p.q_st = q->stride_t * 2;
    p.q_sh = q->stride_h * 2;
    p.out = q->out;
    p.starts = starts;
    p.lens = lens;
    p.table = cache->table;
    p.table_stride = cache->table_stride;
    p.v = static_cast<const uint8_t*>(cache->v);
    p.v_sp = cache->stride_p * 2;
    p.v_sh = cache->stride_h * 2;
    p.v_st = cache->stride_t * 2;
    p.batch = cache->batch;
    p.n_tokens = n_tokens;
    p.max_new = max_new;
    p.capacity = cache->table_width * cache->page_size;
    p.n_q_heads = q->n_heads;
    p.n_kv_heads = cache->n_kv_heads;
    p.group = group;
    p.tq = tq;
    p.n_pages = cache->n_pages;
    while ((1 << p.page_log2) < cache->page_size) ++p.page_log2;
    p.box_rows = std::min(kTile, cache->page_size);
    p.boxes = kStep / p.box_rows;
    const float scale_log2 = scale * kLog2e;
    p.scale_sign = (scale_log2 > 0.f) - (scale_log2 < 0.f);
    p.scale_log2 = p.scale_sign ? std::fabs(scale_log2) : 1.f;
    p.slot_rows = unit_rows(group, max_new);
    p.dev_err = dev_err;
    p.test_stall = (flags & KVD_FLAG_TEST_STALL) ? 1 : 0;
    const bool pdl = (flags & (KVD_FLAG_PDL | KVD_FLAG_EARLY_KV)) != 0;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    return dtype == KVD_BF16 ? run_paged<__nv_bfloat16>(p, nsm, mk, mv, ws, pdl, st)
                             : run_paged<__half>(p, nsm, mk, mv, ws, pdl, st);
}
