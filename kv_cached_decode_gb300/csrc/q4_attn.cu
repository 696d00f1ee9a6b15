// q4_attn.cu -- attention of 1..16 query tokens per row over a cache held in 4 bits, with an
// optional sliding window and sinks.
//
// No counterpart on the pages. For query i of a block at position p_i = len - qlen + i and
// K, V rows stored as n in 0..15 with a step s and a zero point z (value s * (n - z)):
//   score_t = scale * sK_t * (q . nK_t - zK_t * sum(q))
//   out     = sum_t w_t sV_t (nV_t - zV_t) / sum_t w_t,   w_t = exp(score_t - max)
// so the products run on the stored integers and steps and zero points enter once per row
// and position.
//
// Design.
//  * Products are mma.sync m16n8k16 in fp16 with fp32 accumulation. A nibble masked out of a
//    word with 0x000F000F IS a pair of binary16 subnormals n * 2^-24 (0x00F000F0: n * 2^-20):
//    one AND per two values instead of a conversion. The products are exact; q is scaled by a
//    power of two per row, the powers are undone in fp32. Their sums are cut: 16 products are
//    aligned by their factors' exponents, and a subnormal counts as 2^-14, so every product is
//    cut at 2^-15 of the largest q (or weight times step) among them, in units of n. (Measured
//    with one such factor 2^10 times the others: off by 3.4e-4 of it, 3.6e-6 with n itself. 16
//    times closer with n * 2^-20 throughout, for two more shifts a word.)
//  * The cache is the 16-row operand of both products (16 positions x dims for the scores, 16
//    dims x positions for the output) and the queries are the 8 columns: half the products of
//    the other way round, and a lane prepares the parameters of 4 positions per tile instead
//    of 8. The weights turn from score to operand layout with one movmatrix per 8 positions.
//  * A byte holds consecutive dims. The contraction order of q.K is free, so lane c of a
//    quad takes dims 16c..16c+15 of a K row (8 consecutive bytes) and q is loaded in the
//    same order; the row order of the output product is free, so lane g takes word g of a V
//    row, dims 8g..8g+7. Row g of 8 positions is position g / 2 + 4 (g % 2), which keeps both
//    reads free of bank conflicts. Pairs of positions are two words merged with PRMT.
//  * One reference C per query and warp (log2 units, a whole number) serves softmax and V alike:
//    w = 2^(score - C), summed unrounded in fp32, and w * sV, rounded to binary16, multiplies
//    nV. C is set so that the largest w * sV of the rows the query sees is 2^7.5 or more and
//    moves only when one nears 2^15 (or a w 2^96). So what a product loses below binary16's
//    normal range is 2^-32 of the largest product, and neither rows the query does not see nor
//    rows of little weight, whatever their steps, cost the others bits. Rows of zeros (n = z =
//    0) add nothing and do not set C: their step is 1 however small V is. (Products below 2^-82
//    of the largest w lose more: w is 2^90 at most when C is set.) The zero points multiply the
//    same rounded products, so their rounding is not amplified by n - z cancelling. Whether any
//    may have to move is one vote per tile: the usual tile has no reduction across lanes at all.
//    Each query then moves by what it sees itself, so its bits do not depend on others.
//  * Each warp streams its own tiles of 32 positions (2304 bytes with the parameters)
//    through a ring of cp.async stages: no block barrier in the loop, and rows at or past
//    the length are filled with zeros and never read.
//  * Work. A unit is a (row, KV head, block of <= 16 query vectors). Little work in all: every
//    unit is cut into splits of equal tile counts of the row's own length, which form a
//    thread-block cluster and merge through distributed shared memory, every CTA a share of
//    the outputs. Much work (STREAM): the tiles of all units form one list, every CTA of one
//    wave takes an equal stretch of it, and units cut by a stretch's end merge through the
//    workspace (last arrival): the longest row does not set the time.
//
// Measured: 16 rows x 8 heads (4 queries each), ragged to 32768 positions, 227 MB: 49.0 to 49.6 us,
// 4.6 TB/s, bound by the chain of a tile (about 300 instructions, four warps per scheduler: issue on
// half of the cycles, DRAM 57 %, tensor cores 24 %); 16 rows of 65536 positions 112 us, 5.4 TB/s.
// 1 row x 8 heads x 8192: 8.2 to 8.4 us, the chain of launch, first tile and merge.
// Tried: 10 or 12 warps 59 and 57 us, 16 warps and one CTA per SM 52.7, three CTAs at 80
// registers 57.3, 4-warp CTAs 58 to 64, 3 or 5 stages 51.1 and 52.0 (then 51.2); the next unit's
// first tiles fetched before the last one's merge 52.5.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {
namespace {

constexpr int kWarpsQ = 8;
constexpr int kThreadsQ = kWarpsQ * 32;
constexpr int kT = 32;                       // positions per tile
constexpr int kStagesQ = 4;                  // cp.async stages per warp
constexpr int kStageBytes = kT * (32 + 32 + 8);
constexpr int kMaxClusterQ = 16;
constexpr int kMaxStream = 512;              // CTAs of a STREAM launch
// STREAM: a unit counts as its tiles and kUnitCost more, for the time that a CTA needs for any
// unit at all (loads that nothing hides, the merge). 37 rows x 16 heads, lengths in equal steps up
// to 32768: 179 us without it, 160, 142, 134 us with 8, 16, 24; up to 8192: 102, 70, 57, 50 us.
constexpr uint32_t kUnitCost = 24;
// No cut this close to a unit's ends (20.8 -> 15.3 us: 37 x 16, up to 2048, before kUnitCost).
constexpr uint32_t kSnap = 8;
// Lists this short per CTA (in weight) are cut evenly among units; see shares().
constexpr uint32_t kAlignFew = 64, kAlignMost = 128;
// Powers of two of a query's largest product w * sV and of its largest w, when C is set; C moves
// when one is kSlackLog2 more. (A product's exponent is that of w plus that of sV, or one more:
// below 2^16. A lane's 2^24 rows with w of 2^96 add up to 2^120.)
constexpr float kSetLog2 = 8.f, kSetWeightLog2 = 90.f, kSlackLog2 = 6.f;
constexpr int kPart = kHeadDim + 4;          // floats per partial: o[64], max, sum, 2 pad

struct Q4AttnParams {
    const void* q;
    void* out;
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* par;
    int64_t sb, sh;          // rows
    const int32_t* lens;
    int32_t fixed_len, capacity, batch;
    int32_t n_q_heads, n_kv_heads, group, qlen;
    int32_t M, msub, nsub;   // query vectors per (row, KV head), per block; blocks
    int32_t splits;          // cluster launches: splits per unit
    int32_t causal, window, n_sinks;
    float scale_log2;
    float* ws_part;          // STREAM: [2 * CTAs][msub][kPart]
    int32_t* ws_cnt;         // [units]
    int32_t* dev_err;
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async8_zfill(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 8 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// All threads of all CTAs of the cluster: writes before are visible to reads after.
__device__ __forceinline__ void cluster_sync_q4() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Transpose of an 8 x 8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ float half_bits(uint32_t b) {
    return __half2float(__ushort_as_half((uint16_t)b));
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    return Half16<__half>::from_f2(a, b);
}
// The exponent of x >= 0 (-127 for 0 and subnormals).
__device__ __forceinline__ float power_of(float x) {
    return __uint_as_float(0x4B400000u + (__float_as_uint(x) >> 23)) - (0x1.8p23f + 127.f);
}

// The tiles a unit reads, numbered 0 .. total-1: with a window, the tiles of the sinks, then
// those from the first tile of the window on.
struct TileMap {
    int head, gap, total;  // tiles < head as they are; the others are `gap` further on
    __device__ __forceinline__ int pos(int v) const { return (v < head ? v : v + gap) * kT; }
};
__device__ __forceinline__ TileMap tile_map(const Q4AttnParams& p, int len) {
    TileMap m;
    const int all = (len + kT - 1) / kT;
    m.head = 0;
    m.gap = 0;
    if (p.window > 0) {
        // query 0 sees positions > len - qlen - window
        const int64_t lo = (int64_t)len - p.qlen - p.window + 1;
        const int first = lo > 0 ? (int)(lo / kT) : 0;
        const int sinks = (min(p.n_sinks, len) + kT - 1) / kT;
        if (sinks < first) {
            m.head = sinks;
            m.gap = first - sinks;
        }
    }
    m.total = all - m.gap;
    return m;
}
__device__ __forceinline__ int row_len(const Q4AttnParams& p, int b) {
    return p.lens ? p.lens[b] : p.fixed_len;
}

// STREAM: what a unit counts in the list.
__device__ __forceinline__ uint32_t weight(const TileMap& m) {
    return m.total ? m.total + kUnitCost : 0;
}

// STREAM: the list has the units of rows 0 .. batch-1 (a row's: KV heads x blocks), by weight.
// The row that holds place `at` of the list, and the list's length before that row; with at past
// the end, `before` is the length of the list. One warp, the same in all of them.
__device__ __forceinline__ int find_row(const Q4AttnParams& p, uint32_t at, uint32_t& before) {
    const int lane = threadIdx.x & 31;
    const uint32_t units = (uint32_t)(p.n_kv_heads * p.nsub);
    before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        uint32_t n = 0;
        if (b0 + lane < p.batch) {
            const int len = row_len(p, b0 + lane);
            if (len >= 0 && len <= p.capacity) n = weight(tile_map(p, len)) * units;
        }
        uint32_t inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            before += __shfl_sync(0xffffffffu, inc - n, l);
            return b0 + l;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return p.batch;
}

// STREAM: stretches of the list, CTA i's from floor(total i / ctas) on.
struct Shares {
    uint32_t total, ctas, per, rest;  // total = per ctas + rest
    __device__ __forceinline__ uint32_t start(uint32_t i) const {
        return i * per + i * rest / ctas;  // (rest < ctas <= 512)
    }
    __device__ __forceinline__ uint32_t holder(uint32_t at) const {  // whose share has place `at`
        uint32_t i = (uint32_t)((float)at * ((float)ctas / (float)total));
        i = min(i, ctas - 1);
        while (start(i) > at) --i;
        while (start(i + 1) <= at) ++i;
        return i;
    }
};
// How many CTAs share a list of weight `total`: a tile per warp at least, but not fewer CTAs than
// units. Short lists: a number of CTAs per unit, or of units per CTA, so that equal lengths are
// cut at the ends of units and a CTA meets no more of them than it must (37 rows x 16 heads of
// 1024: 22.8 -> 16.1 us; 16 x 8 of 2048: 15.9 -> 11.9 us). With long ones the idle CTAs cost more
// (16 x 8 of 16384: 38.5 -> 40.6 us).
__device__ __forceinline__ Shares shares(const Q4AttnParams& p, uint32_t total) {
    const uint32_t units = (uint32_t)(p.batch * p.n_kv_heads * p.nsub);
    uint32_t n = min((uint32_t)gridDim.x, max((total + kWarpsQ - 1) / kWarpsQ, units));
    uint32_t even = n / units * units;
    if (even == 0) {
        const uint32_t least = (units + n - 1) / n;
        for (uint32_t k = least; k < 2 * least && even == 0; ++k)
            if (units % k == 0) even = units / k;
    }
    if (even > 0 && total < gridDim.x * (4 * even >= 3 * n ? kAlignMost : kAlignFew)) n = even;
    n = max(1u, min(n, total));
    Shares s;
    s.total = total;
    s.ctas = n;
    s.per = total / n;
    s.rest = total - s.per * n;
    return s;
}

// Where the stretch really starts whose share starts at `at`: inside a unit of weight w from
// keep_lo to keep_hi - 1, else at the nearer end of the unit, as a cut costs more than some tiles.
// (Units too small for that are not cut.)
__device__ __forceinline__ bool cuttable(uint32_t w) { return w >= kUnitCost + 2 * kSnap; }
__device__ __forceinline__ uint32_t keep_lo(uint32_t w) {
    return cuttable(w) ? kUnitCost + kSnap : (w + 1) / 2;
}
__device__ __forceinline__ uint32_t keep_hi(uint32_t w) {
    return cuttable(w) ? w - kSnap : keep_lo(w);
}
__device__ __forceinline__ uint32_t cut(const Q4AttnParams& p, uint32_t total, uint32_t at) {
    if (at >= total) return total;
    uint32_t before;
    const int b = find_row(p, at, before);
    const uint32_t w = weight(tile_map(p, row_len(p, b))), in = (at - before) % w;
    return in < keep_lo(w) ? at - in : in >= keep_hi(w) ? at - in + w : at;
}

// NT: blocks of 8 query vectors.
template <typename T, int NT, bool STREAM>
__global__ void __launch_bounds__(kThreadsQ, 2) q4_attn_kernel(const Q4AttnParams p) {
    constexpr int RM = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    float* red = reinterpret_cast<float*>(smem);  // after a unit's tiles: [warp][RM][kPart]
    float* part = red + kWarpsQ * RM * kPart;     // this CTA's partial [msub][kPart]

    pdl_wait();
    pdl_trigger();

    // ---- the stretch of the tile list, or the split of the unit ----
    uint32_t cur = 0, end = 0;
    Shares sh = {};
    if (STREAM) {
        uint32_t total;
        find_row(p, 0xffffffffu, total);
        sh = shares(p, total);
        const uint32_t i = blockIdx.x;
        cur = cut(p, total, i < sh.ctas ? sh.start(i) : total);
        end = cut(p, total, i < sh.ctas ? sh.start(i + 1) : total);
        // rows without a tile: flagged, or (length 0) zeros
        for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
            const int len = row_len(p, b);
            if (len < 0 || len > p.capacity) {
                if (tid == 0) flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
            } else if (len == 0) {
                const int64_t n = (int64_t)p.n_q_heads * p.qlen * (kHeadDim / 8);
                uint4* o = static_cast<uint4*>(p.out) + b * n;
                for (int64_t x = tid; x < n; x += kThreadsQ) o[x] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    do {
        int b, uh, v0, v1, len;  // uh: unit within the row
        uint32_t u0 = 0;         // STREAM: where the unit starts in the list
        TileMap tm;
        if (STREAM) {
            if (cur >= end) break;
            uint32_t before;
            b = find_row(p, cur, before);
            len = row_len(p, b);
            tm = tile_map(p, len);
            const uint32_t w = weight(tm);
            uh = (int)((cur - before) / w);
            u0 = before + uh * w;
            v0 = max((int)(cur - u0) - (int)kUnitCost, 0);
            cur = min(u0 + w, end);
            v1 = (int)(cur - u0 - kUnitCost);
        } else {
            b = blockIdx.z;
            uh = blockIdx.y;
            len = row_len(p, b);
            if (len < 0 || len > p.capacity) {  // the same in every CTA of a cluster
                if (tid == 0 && blockIdx.x == 0 && uh == 0)
                    flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
                return;
            }
            tm = tile_map(p, len);
            v0 = (int)((int64_t)tm.total * blockIdx.x / p.splits);
            v1 = (int)((int64_t)tm.total * (blockIdx.x + 1) / p.splits);
        }
        const int h = uh / p.nsub, m0 = uh % p.nsub * p.msub;
        const int mcount = min(p.msub, p.M - m0);

        // ---- the warp's ring ----
        uint8_t* ring = smem + warp * (kStagesQ * kStageBytes);
        const int64_t row0 = b * p.sb + h * p.sh;
        const uint8_t* kbase = p.k + row0 * 32 + lane * 16;
        const uint8_t* vbase = p.v + row0 * 32 + lane * 16;
        const uint8_t* pbase = p.par + row0 * 8 + lane * 8;
        auto fetch = [&](int v, int stage) {
            if (v < v1) {
                const int t0 = tm.pos(v);
                const uint32_t dst = smem_u32(ring + stage * kStageBytes) + lane * 16;
                const int64_t off = (int64_t)t0 * 32;
                if (t0 + kT <= len) {
                    cp_async16(dst, kbase + off);
                    cp_async16(dst + 512, kbase + off + 512);
                    cp_async16(dst + kT * 32, vbase + off);
                    cp_async16(dst + kT * 32 + 512, vbase + off + 512);
                    cp_async8(dst + kT * 64 - lane * 8, pbase + (int64_t)t0 * 8);
                } else {  // zeros from the length on
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool on = t0 + 16 * i + (lane >> 1) < len;
                        const int64_t o = on ? off + 512 * i : 0;
                        cp_async16_zfill(dst + 512 * i, kbase + o, on);
                        cp_async16_zfill(dst + kT * 32 + 512 * i, vbase + o, on);
                    }
                    const bool on = t0 + lane < len;
                    cp_async8_zfill(dst + kT * 64 - lane * 8, pbase + (on ? (int64_t)t0 * 8 : 0),
                                    on);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStagesQ - 1; ++i) fetch(v0 + warp + i * kWarpsQ, i);

        // ---- the queries: lane (g, c) has dims 16c..16c+15 of query g of every block of 8,
        // fp16, scaled by 2^e so that a row's largest value lies in [2^14, 2^15) ----
        uint32_t qb[NT][4][2];
        // of the queries 2c, 2c + 1 of a block: score factor (log2 units), sum of the scaled
        // q * 2^-24, and the limit: a query sees t < lim
        float rs[NT][2], qs[NT][2];
        int lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int m = 8 * nt + g;
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
            if (m < mcount) {
                const int i = (m0 + m) % p.qlen, hq = h * p.group + (m0 + m) / p.qlen;
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const T*>(p.q) +
                    (((int64_t)b * p.n_q_heads + hq) * p.qlen + i) * kHeadDim + 16 * c);
                unpack8<T>(src[0], x);
                unpack8<T>(src[1], x + 8);
            }
            float big = 0.f;
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                big = fmaxf(big, fabsf(x[e]));
                odd |= !(fabsf(x[e]) < INFINITY);
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // a row with an infinity or a NaN keeps its values (its outputs are not finite)
            const bool any_odd =
                ((__ballot_sync(0xffffffffu, odd) >> (lane & 28)) & 15u) != 0;
            int e2 = 0;
            if (big > 0.f && !any_odd) {
                frexpf(big, &e2);  // big = f * 2^e2, f in [0.5, 1)
                e2 = min(15 - e2, 120);
            }
            const float up = p.scale_log2 < 0.f ? -1.f : 1.f;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[e] = __half2float(__float2half_rn(up * ldexpf(x[e], e2)));
                sum += x[e];
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const float f = ldexpf(fabsf(p.scale_log2), 24 - e2);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int mq = 8 * nt + 2 * c + e;
                rs[nt][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + e));
                qs[nt][e] = __shfl_sync(0xffffffffu, sum, 4 * (2 * c + e)) * 0x1p-24f;
                const int pos1 = len - p.qlen + (m0 + mq) % p.qlen + 1;
                lim[nt][e] = mq < mcount ? (p.causal ? max(pos1, 0) : len) : 0;
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    // nibbles n and n + 4 of word kk / 2; the odd ones come times 16
                    const int n = 8 * (kk >> 1) + 2 * (kk & 1) + w;
                    const float s = w ? 0.0625f : 1.f;
                    qb[nt][kk][w] = pack_half(x[n] * s, x[n + 4] * s);
                }
        }

        float acc[4][NT][4];  // dims 8g + 2j (and + 1, times 16) of queries 2c, 2c + 1
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][nt][e] = 0.f;
        // -C, and this lane's share of the normalisers and of the zero points' sums
        float ref[NT][2], l[NT][2], zs[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ref[nt][e] = INFINITY;  // (the first row seen moves it)
                l[nt][e] = zs[nt][e] = 0.f;
            }

        // positions every query of the block sees wholly: t < seen_hi, and with a window
        // t >= seen_lo or t < n_sinks
        const int seen_hi = p.causal ? len - p.qlen + 1 : len;
        const int seen_lo = p.window > 0 ? (int)max((int64_t)len - p.window, (int64_t)0) : 0;

        auto tile = [&](const uint8_t* st, int t0, auto masked_) {
            constexpr bool kMasked = decltype(masked_)::value;
            const int krow = (g >> 1) + 4 * (g & 1);  // this lane's position of every 8
            const uint8_t* sK = st + krow * 32 + c * 8;
            const uint8_t* sV = st + kT * 32 + c * 32 + g * 4;
            const uint8_t* sP = st + kT * 64 + krow * 8;
            float sc[2][NT][4];  // positions 16 t + krow and + 8 of queries 2c, 2c + 1
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[t][nt][e] = 0.f;
                const uint2 a = *reinterpret_cast<const uint2*>(sK + t * 512);
                const uint2 d = *reinterpret_cast<const uint2*>(sK + t * 512 + 256);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t wa = (kk < 2 ? a.x : a.y) >> (8 * (kk & 1));
                    const uint32_t wd = (kk < 2 ? d.x : d.y) >> (8 * (kk & 1));
                    const uint32_t f[4] = {wa & 0x000F000Fu, wd & 0x000F000Fu, wa & 0x00F000F0u,
                                           wd & 0x00F000F0u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        Mma<__half>::run(sc[t][nt], f, qb[nt][kk][0], qb[nt][kk][1]);
                }
            }
            float vs[2][2], vz[2][2];  // V steps and zero points of the positions
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint2 pr = *reinterpret_cast<const uint2*>(sP + (16 * t + 8 * hh) * 8);
                    // an infinite zero point must not reach rows that do not see it
                    if (kMasked && ((pr.y >> 16) & 0x7C00u) == 0x7C00u) pr.y = 0x7FC0u;
                    const float ks = __uint_as_float(pr.x << 16), kz = half_bits(pr.x >> 16);
                    vs[t][hh] = __uint_as_float(pr.y << 16);
                    vz[t][hh] = half_bits(pr.y >> 16);
                    const int pos = t0 + 16 * t + 8 * hh + krow;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float* s2 = &sc[t][nt][2 * hh];
                        const float2 x2 = mul2(fma2(Pair(-kz, -kz), Pair(qs[nt][0], qs[nt][1]),
                                                    Pair(s2[0], s2[1])),
                                               Pair(ks, ks)).get();
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = e ? x2.y : x2.x;
                            if (kMasked) {
                                const int lm = lim[nt][e];
                                if (!(pos < lm && (p.window == 0 || pos >= lm - p.window ||
                                                   pos < p.n_sinks)))
                                    x = -INFINITY;
                            }
                            s2[e] = x;
                        }
                    }
                }
            // One vote: may a query's reference have to move? By the largest score and the largest
            // step of a lane's rows, seen or not; what moves is decided by the rows themselves.
            {
                const float big = max3(max3(vs[0][0], vs[0][1], vs[1][0]), vs[1][1], 0.f);
                const float over = fmaxf(power_of(big) - kSetLog2, -kSetWeightLog2) - kSlackLog2;
                bool move = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float top = max3(max3(sc[0][nt][e], sc[0][nt][2 + e], sc[1][nt][e]),
                                               sc[1][nt][2 + e], -INFINITY);
                        move |= fmaf(top, rs[nt][e], over) > -ref[nt][e];
                    }
                if (__any_sync(0xffffffffu, move)) {
                    if (vz[0][0] * vz[0][1] * vz[1][0] * vz[1][1] == 0.f) {  // rows of zeros?
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4* v = reinterpret_cast<const uint4*>(
                                st + kT * 32 + (8 * i + krow) * 32);
                            const uint4 u = v[0], w = v[1];
                            if (vz[i >> 1][i & 1] == 0.f &&
                                (u.x | u.y | u.z | u.w | w.x | w.y | w.z | w.w) == 0u)
                                vs[i >> 1][i & 1] = 0.f;
                        }
                    }
                    float lv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // (a step of 0 or an infinity: by w alone)
                        const float s = vs[i >> 1][i & 1];
                        lv[i] = fmaxf(s > 0.f && s < INFINITY ? power_of(s) - kSetLog2 : -INFINITY,
                                      -kSetWeightLog2);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float to = -INFINITY;  // where C has to be
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float x = sc[i >> 1][nt][2 * (i & 1) + e];
                                if (kMasked && x == -INFINITY) continue;
                                to = fmaxf(to, fmaf(x, rs[nt][e], lv[i]));
                            }
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1)
                                to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, off));
                            if (to - kSlackLog2 > -ref[nt][e]) {
                                to = rintf(to);
                                const float f = exp2f(-to - ref[nt][e]);  // (from INFINITY: 0)
                                ref[nt][e] = -to;
                                l[nt][e] *= f;
                                zs[nt][e] *= f;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    acc[j][nt][e] *= f;
                                    acc[j][nt][2 + e] *= f;
                                }
                            }
                        }
                }
            }
            // the weights times the steps, as the output product's operand
            uint32_t pw[2][2][NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const float* x = &sc[t][nt][2 * hh];
                        const float2 a = fma2(Pair(x[0], x[1]), Pair(rs[nt][0], rs[nt][1]),
                                              Pair(ref[nt][0], ref[nt][1])).get();
                        float2 w = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                        if (kMasked) {
                            if (x[0] == -INFINITY) w.x = 0.f;
                            if (x[1] == -INFINITY) w.y = 0.f;
                        }
                        const Pair w2(w.x, w.y);
                        float2 f = mul2(w2, Pair(vs[t][hh], vs[t][hh])).get();
                        if (kMasked) {  // (an infinite step)
                            if (x[0] == -INFINITY) f.x = 0.f;
                            if (x[1] == -INFINITY) f.y = 0.f;
                        }
                        const float2 l2 = add2(Pair(l[nt][0], l[nt][1]), w2).get();
                        l[nt][0] = l2.x;
                        l[nt][1] = l2.y;
                        const uint32_t pk = pack_half(f.x, f.y);
                        const float2 r = Half16<__half>::to_f2(pk);
                        const float2 z2 = fma2(Pair(r.x, r.y), Pair(vz[t][hh], vz[t][hh]),
                                               Pair(zs[nt][0], zs[nt][1])).get();
                        zs[nt][0] = z2.x;
                        zs[nt][1] = z2.y;
                        pw[t][hh][nt] = transpose8(pk);
                    }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t w[4];  // positions c, c + 4, c + 8, c + 12
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = *reinterpret_cast<const uint32_t*>(sV + t * 512 + i * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t sel = j < 2 ? 0x5410 : 0x7632;
                    const uint32_t a = __byte_perm(w[0], w[1], sel) >> (8 * (j & 1));
                    const uint32_t d = __byte_perm(w[2], w[3], sel) >> (8 * (j & 1));
                    const uint32_t f[4] = {a & 0x000F000Fu, a & 0x00F000F0u, d & 0x000F000Fu,
                                           d & 0x00F000F0u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        Mma<__half>::run(acc[j][nt], f, pw[t][0][nt], pw[t][1][nt]);
                }
            }
        };

        int stage = 0;
        for (int v = v0 + warp; v < v1; v += kWarpsQ) {
            cp_async_wait<kStagesQ - 2>();
            __syncwarp();
            const int t0 = tm.pos(v);
            const uint8_t* st = ring + stage * kStageBytes;
            // refill the stage read in the previous iteration
            fetch(v + (kStagesQ - 1) * kWarpsQ, stage == 0 ? kStagesQ - 1 : stage - 1);
            if (t0 + kT <= seen_hi && (t0 >= seen_lo || t0 + kT <= p.n_sinks))
                tile(st, t0, std::false_type{});
            else
                tile(st, t0, std::true_type{});
            stage = stage + 1 == kStagesQ ? 0 : stage + 1;
            __syncwarp();  // the tile is read before its stage is refilled
        }
        cp_async_wait_all();
        __syncthreads();

        // ---- merge the warps: red[warp][query][kPart] over the ring ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = l[nt][e], z = zs[nt][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    t += __shfl_xor_sync(0xffffffffu, t, off);
                    z += __shfl_xor_sync(0xffffffffu, z, off);
                }
                const int m = 8 * nt + 2 * c + e;
                if (m < mcount) {
                    // partials of different C meet: the sum's power of two goes into it
                    const int up = min(max((int)(__float_as_uint(t) >> 23), 1), 253) - 127;
                    const float down = __uint_as_float((uint32_t)(127 - up) << 23);
                    float* o = red + (warp * RM + m) * kPart;
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[2 * j] = fmaf(acc[j][nt][e], 0x1p24f, -z) * down;
                        x[2 * j + 1] = fmaf(acc[j][nt][2 + e], 0x1p20f, -z) * down;
                    }
                    float4* d = reinterpret_cast<float4*>(o + 8 * g);
                    d[0] = make_float4(x[0], x[1], x[2], x[3]);
                    d[1] = make_float4(x[4], x[5], x[6], x[7]);
                    if (g == 0) {
                        o[kHeadDim] = (float)up - ref[nt][e];
                        o[kHeadDim + 1] = t * down;
                    }
                }
            }
        __syncthreads();
        const int items = mcount * (kHeadDim / 4);  // (query vector, 4 dims)
        auto store = [&](int it, const float4& o, float sum) {
            const int m = it >> 4, d = (it & 15) * 4;
            const int i = (m0 + m) % p.qlen, hq = h * p.group + (m0 + m) / p.qlen;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint2 w;
            w.x = Half16<T>::from_f2(o.x * inv, o.y * inv);
            w.y = Half16<T>::from_f2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(static_cast<T*>(p.out) +
                                      (((int64_t)b * p.n_q_heads + hq) * p.qlen + i) * kHeadDim +
                                      d) = w;
        };
        // (max, sum, o) of n partials, load(i, quad) the i-th's float4 (quad 16: max, sum), in
        // order
        auto combine = [&](int n, auto&& load, int q4, float& mx, float& sum) -> float4 {
            mx = -INFINITY;
#pragma unroll 4
            for (int i = 0; i < n; ++i) mx = fmaxf(mx, load(i, kHeadDim / 4).x);
            const float rf = mx == -INFINITY ? 0.f : mx;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            sum = 0.f;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float4 ml = load(i, kHeadDim / 4), x = load(i, q4);
                const float a = exp2f(ml.x - rf);
                sum = fmaf(ml.y, a, sum);
                o.x = fmaf(x.x, a, o.x);
                o.y = fmaf(x.y, a, o.y);
                o.z = fmaf(x.z, a, o.z);
                o.w = fmaf(x.w, a, o.w);
            }
            return o;
        };
        const bool whole = STREAM ? v0 == 0 && v1 == tm.total : p.splits == 1;
        float* mine = part;  // where this CTA's partial goes, when the unit is not whole
        if (STREAM) mine = p.ws_part + (2 * (int64_t)blockIdx.x + (v0 == 0)) * p.msub * kPart;
        for (int it = tid; it < items; it += kThreadsQ) {
            const float4* r0 = reinterpret_cast<const float4*>(red + (it >> 4) * kPart);
            float mx, sum;
            const float4 o = combine(
                kWarpsQ, [&](int i, int q4) { return r0[i * (RM * kPart / 4) + q4]; }, it & 15, mx,
                sum);
            if (whole) {
                store(it, o, sum);
            } else {
                float* d = mine + (it >> 4) * kPart;
                reinterpret_cast<float4*>(d)[it & 15] = o;
                if ((it & 15) == 0)
                    *reinterpret_cast<float4*>(d + kHeadDim) = make_float4(mx, sum, 0.f, 0.f);
            }
        }
        if (!STREAM) {
            if (whole) return;
            // every CTA merges a share of the outputs out of all CTAs' partials
            cluster_sync_q4();
            const uint32_t base = smem_u32(part);
            for (int it = blockIdx.x + p.splits * tid; it < items; it += p.splits * kThreadsQ) {
                const uint32_t off = base + (it >> 4) * (kPart * 4);
                float mx, sum;
                const float4 o = combine(
                    p.splits,
                    [&](int i, int q4) { return ld_cluster4(map_shared(off + q4 * 16, i)); },
                    it & 15, mx, sum);
                store(it, o, sum);
            }
            cluster_sync_q4();  // no CTA leaves while another may still read its partial
            return;
        }
        if (!whole) {
            // the CTAs whose stretches meet the unit; the last to arrive merges their partials
            // in the order of the list
            // (the last whose share starts before the unit's first, and before its last cut)
            const uint32_t w = weight(tm);
            const uint32_t i0 = sh.holder(u0 + keep_lo(w) - 1);
            const uint32_t i1 = sh.holder(u0 + keep_hi(w) - 1);
            const int n = (int)(i1 - i0) + 1;
            const int unit = b * p.n_kv_heads * p.nsub + uh;
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(&p.ws_cnt[unit], 1) == n - 1;
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int it = tid; it < items; it += kThreadsQ) {
                    float mx, sum;
                    const float4 o = combine(
                        n,
                        [&](int i, int q4) {
                            const int64_t slot = 2 * (int64_t)(i0 + i) + (i == 0);
                            return __ldcg(reinterpret_cast<const float4*>(
                                              p.ws_part + (slot * p.msub + (it >> 4)) * kPart) +
                                          q4);
                        },
                        it & 15, mx, sum);
                    store(it, o, sum);
                }
                if (tid == 0) p.ws_cnt[unit] = 0;
            }
        }
        __syncthreads();  // the ring is free for the next unit
    } while (STREAM);
}

// Ring of all warps, reused for the warps' partials; the CTA's partial follows them.
constexpr uint32_t q4_smem(int rm) {
    const uint32_t ring = kWarpsQ * kStagesQ * kStageBytes;
    const uint32_t red = (kWarpsQ + 1) * rm * kPart * 4;
    return ring > red ? ring : red;
}

constexpr int kMaxDevQ = 64;

// Once per kernel and device: shared memory, clusters of 16. Returns the largest cluster
// (0 on error).
template <auto Kern>
int prepare_q4(size_t smem) {
    static std::once_flag once[kMaxDevQ];
    static int result[kMaxDevQ];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevQ) return 0;
    std::call_once(once[dev], [&] {
        if (cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess) {
            cudaGetLastError();
            return;
        }
        const bool big = cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                              1) == cudaSuccess;
        cudaGetLastError();
        result[dev] = big ? kMaxClusterQ : 8;
    });
    return result[dev];
}

// Blocks (cluster == 1) or clusters of `cluster` blocks resident at once on the device, which
// prepare_q4 has found in range.
template <auto Kern>
int resident_q4(int dev, size_t smem, int cluster, int nsm) {
    static std::atomic<int> cache[kMaxDevQ][kMaxClusterQ + 1];  // value + 1
    std::atomic<int>& v = cache[dev][cluster];
    if (const int have = v.load(std::memory_order_relaxed)) return have - 1;
    int n = 0;
    if (cluster <= 1) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kern, kThreadsQ, smem) !=
            cudaSuccess)
            n = 0;
        n *= nsm;
    } else {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)cluster);
        cfg.blockDim = dim3(kThreadsQ);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute a;
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = (unsigned)cluster;
        a.val.clusterDim.y = 1;
        a.val.clusterDim.z = 1;
        cfg.attrs = &a;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, Kern, &cfg) != cudaSuccess) n = 0;
    }
    cudaGetLastError();
    v.store(n + 1, std::memory_order_relaxed);
    return n;
}

struct Q4Shape {
    int group, M, nsub, msub;
    int64_t units;
};
Q4Shape q4_shape(int batch, int n_q_heads, int n_kv_heads, int qlen) {
    Q4Shape s;
    s.group = n_q_heads / n_kv_heads;
    s.M = s.group * qlen;
    s.nsub = (s.M + 15) / 16;
    s.msub = (s.M + s.nsub - 1) / s.nsub;
    s.units = (int64_t)batch * n_kv_heads * s.nsub;
    return s;
}

// Most tiles a unit reads when its length is at most `bound`.
int64_t q4_tiles(int64_t bound, int qlen, int window, int n_sinks) {
    const int64_t all = (bound + kT - 1) / kT;
    if (window <= 0) return all;
    const int64_t near = ((int64_t)window + qlen - 1 + 2 * (kT - 1)) / kT;
    return std::min(all, near + ((int64_t)n_sinks + kT - 1) / kT);
}

// A launch streams the list of tiles when a split could have this many of them. The host knows
// the bound of the lengths only, and streaming pays where they differ or the units fill a wave
// badly (splits | stream, us, lengths equal / in equal steps):
//   16 rows x 8 heads, to 32768 (512 tiles a split):  64.7 / 50.9 | 63.1 / 41.3
//   24 x 8 (1 split each), to 8192 (256):             34.2 / 29.9 | 33.0 / 23.0
//   24 x 8, to 2048 (64):                             11.9 / 11.1 | 13.9 / 16.8
//   40 x 8, to 32768 (1024):                         179.6 /  102 |  137 / 78.9
// one row of 32768 among 40 of 2048: 78.7 | 34.4; all of 600 in a cache of 32768: 10.2 | 15.0.
constexpr int64_t kStreamTiles = 256;
constexpr int64_t kStreamLeast = 152 * 2 * 64;  // and in all: 8 per warp of a wave
// With more units than this (two waves) the block scheduler spreads whole units better: 128 rows x
// 8 heads, to 8192: 112 / 68.8 | 125 / 76.0; 64 x 8: 66.1 / 42.0 | 68.4 / 43.5, one long row 26.7
// | 20.4.
constexpr int64_t kStreamUnits = 640;
static_assert(kStreamUnits * sizeof(int32_t) <= KVD_WS_COUNTER_BYTES, "a counter per unit");
bool q4_streams(const Q4Shape& sh, int64_t tiles) {
    return tiles >= kStreamTiles && sh.units * tiles >= kStreamLeast &&
           sh.units <= kStreamUnits &&
           sh.units * (tiles + kUnitCost) < (INT64_C(1) << 31);
}

template <typename T, int NT>
kvd_status run_q4(Q4AttnParams& p, const Q4Shape& sh, int64_t tiles, int nsm, void* ws,
                  size_t ws_bytes, bool pdl, cudaStream_t st) {
    constexpr size_t smem = q4_smem(8 * NT);
    constexpr auto kern = q4_attn_kernel<T, NT, false>;
    const int mc = prepare_q4<kern>(smem);
    int dev = 0;
    if (mc <= 0 || cudaGetDevice(&dev) != cudaSuccess) return KVD_ERR_CUDA;
    // the most splits (a tile per warp at least) whose clusters are all resident at once
    int64_t want = std::min<int64_t>(std::max<int64_t>(1, (tiles + kWarpsQ - 1) / kWarpsQ), mc);
    for (; want > 1; --want)
        if (resident_q4<kern>(dev, smem, (int)want, nsm) >= sh.units) break;
    if (tiles >= want * kStreamTiles && q4_streams(sh, tiles)) {
        constexpr auto stream = q4_attn_kernel<T, NT, true>;
        if (prepare_q4<stream>(smem) <= 0) return KVD_ERR_CUDA;
        const int slots = std::min(kMaxStream, resident_q4<stream>(dev, smem, 1, nsm));
        if (slots <= 0) return KVD_ERR_CUDA;
        const size_t need =
            KVD_WS_COUNTER_BYTES + (size_t)2 * slots * sh.msub * kPart * sizeof(float);
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < need)
            return KVD_ERR_WORKSPACE;
        p.ws_cnt = static_cast<int32_t*>(ws);
        p.ws_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + KVD_WS_COUNTER_BYTES);
        return launch(stream, dim3((unsigned)slots), dim3(kThreadsQ), smem, st, pdl, p);
    }
    p.splits = (int)want;
    const dim3 grid((unsigned)p.splits, (unsigned)(p.n_kv_heads * sh.nsub), (unsigned)p.batch);
    return launch_ex(kern, grid, dim3(kThreadsQ), smem, st, pdl, (unsigned)p.splits, p);
}

}  // namespace

size_t q4_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int qlen, int max_len) {
    const Q4Shape sh = q4_shape(batch, n_q_heads, n_kv_heads, qlen);
    // (max_len may be any bound: beyond the longest range that streams, shorter ones still do)
    const int64_t most = INT64_C(0x7fffffff) / std::max<int64_t>(sh.units, 1) - kUnitCost;
    if (!q4_streams(sh, std::min(q4_tiles(max_len, qlen, 0, 0), most))) return KVD_WS_COUNTER_BYTES;
    return KVD_WS_COUNTER_BYTES + (size_t)2 * kMaxStream * sh.msub * kPart * sizeof(float);
}

}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_q4_attn(kvd_dtype dtype, int32_t batch, int32_t n_q_heads,
                                  int32_t qlen, const void* q, const kvd_q4_cache* cache,
                                  const int32_t* lens, int32_t fixed_len, int32_t causal,
                                  int32_t window, int32_t n_sinks, float scale, void* out,
                                  void* workspace, size_t workspace_bytes, uint32_t flags,
                                  int32_t* dev_err, kvd_stream_t stream) {
    if (dtype != KVD_F16 && dtype != KVD_BF16) return KVD_ERR_INVALID_ARG;
    if (kvd_status s = validate_q4_cache(cache)) return s;
    if (batch < 0 || n_q_heads <= 0) return KVD_ERR_INVALID_ARG;
    if (qlen < 1 || qlen > KVD_MAX_QLEN) return KVD_ERR_UNSUPPORTED;
    if (n_q_heads % cache->n_kv_heads || batch > cache->batch) return KVD_ERR_INVALID_ARG;
    if (window < 0 || n_sinks < 0 || (window > 0 && !causal)) return KVD_ERR_INVALID_ARG;
    if (!(scale < INFINITY) || !(scale > -INFINITY)) return KVD_ERR_INVALID_ARG;
    if (batch == 0) return KVD_OK;
    if (!q || !out || q == out || !aligned16(q) || !aligned16(out)) return KVD_ERR_INVALID_ARG;
    if (!lens && (fixed_len < 0 || fixed_len > cache->capacity)) return KVD_ERR_INVALID_ARG;
    const Q4Shape sh = q4_shape(batch, n_q_heads, cache->n_kv_heads, qlen);
    if (batch > 65535 || (int64_t)cache->n_kv_heads * sh.nsub > 65535 || sh.units > 0x7fffffff)
        return KVD_ERR_UNSUPPORTED;
    const int nsm = sm_count();
    if (nsm <= 0) return KVD_ERR_CUDA;
    Q4AttnParams p = {};
    p.q = q;
    p.out = out;
    p.k = static_cast<const uint8_t*>(cache->k);
    p.v = static_cast<const uint8_t*>(cache->v);
    p.par = static_cast<const uint8_t*>(cache->params);
    p.sb = cache->stride_b;
    p.sh = cache->stride_h;
    p.lens = lens;
    p.fixed_len = fixed_len;
    p.capacity = cache->capacity;
    p.batch = batch;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = cache->n_kv_heads;
    p.group = sh.group;
    p.qlen = qlen;
    p.M = sh.M;
    p.msub = sh.msub;
    p.nsub = sh.nsub;
    p.causal = causal != 0;
    // more than the cache holds sees the whole cache: the kernel's sums stay small
    p.window = window = std::min(window, cache->capacity);
    p.n_sinks = window > 0 ? std::min(n_sinks, cache->capacity) : 0;
    p.scale_log2 = scale * kLog2e;
    p.dev_err = dev_err;
    const int64_t tiles =
        q4_tiles(lens ? cache->capacity : fixed_len, qlen, window, p.n_sinks);
    const bool pdl = (flags & (KVD_FLAG_PDL | KVD_FLAG_EARLY_KV)) != 0;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool one = sh.msub <= 8;
    if (dtype == KVD_BF16)
        return one ? run_q4<__nv_bfloat16, 1>(p, sh, tiles, nsm, workspace, workspace_bytes, pdl,
                                              st)
                   : run_q4<__nv_bfloat16, 2>(p, sh, tiles, nsm, workspace, workspace_bytes, pdl,
                                              st);
    return one ? run_q4<__half, 1>(p, sh, tiles, nsm, workspace, workspace_bytes, pdl, st)
               : run_q4<__half, 2>(p, sh, tiles, nsm, workspace, workspace_bytes, pdl, st);
}
