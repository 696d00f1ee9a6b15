// sample_filtered.cu -- one token per row after temperature, top-k, top-p and min-p.
//
// "Inference 抽象と KV キャッシュ" of "Whisper のデコーダー内部" samples from
// Categorical(logits / T); the filters have no counterpart on the pages. With the ids of a
// row in order (logit descending, then id ascending) and w = exp((x - max) / T), every
// filter keeps a prefix of that order, so together they keep the shortest of three:
//   top-k: the first k;  top-p: up to the id at which the mass reaches top_p * (mass of the
//   top-k);  min-p: while w >= min_p.  Then token = the smallest id whose running mass of kept
//   ids, in id order, exceeds u * total.
//
// Masses. A draw moves to another id when a running sum moves across u * total, so fp32
// sums in whatever order would give other tokens run by run. Here w is an integer in units
// of 2^-44 and sums are integers: the same on every run and for every split of the row. What
// counts is the sum of all errors against the spacing of the running sums, so w has no bias:
// w = 2^-y, y = (max - x) * log2(e) / T carried in two floats. For y < 16 (heavy ids) y is
// taken apart as n + j/256 + r: a table, a cubic in r, a relative 2^-29, about 30 instructions.
// Below (light ids), fp32 rounding of y (unbiased, its constant in two floats: 2^-24 y) and the
// hardware's 2^x, whose measured mean error of 3.47e-8 is taken off, come to 2^-36 absolute at
// a third of the price. Below 2^-45.5 w is 0. (Double precision would be 30 times slower here.)
// Where min-p drops all ids from some y below 14.5 on, the light form starts at 8 or 1.5 above
// that y: the weights of dropped ids only add up to the mass that top-p is a share of, and 2^-21
// of one, unbiased, is enough there (64 rows x 128000 ids, top-p 0.95, min-p 0.02: 63.6 ->
// 37.5 us, as none of them is listed either).
//
// Design. Bound by the chain of passes and exchanges for few rows, by instruction issue (the
// weights) for many. One thread-block cluster per row; CTA c has the ids [c * slice, (c + 1) *
// slice), each warp a segment of them. Slices of at most kKeep logits stay in shared memory;
// longer ones (many rows: fewer CTAs per row, one wave) are read again from L2, where a whole
// batch fits, so that two CTAs fit on an SM.
//  1. Read, largest logit (lowest id first), number of logits above -inf: one exchange.
//  2. Every warp lists the places of the heavy ids of its segment (eight ids per lane and one
//     warp scan: no atomics) and sums the mass of the light ones. What follows works on the
//     lists (half of flat, a few of peaked logits), unless a cut lies among the light ids: then
//     it takes all ids.
//  3. select(): the k-th id (counts) or the id at which the mass reaches its target. A
//     histogram of 1024 bins over y (bins fall with x, so they are intervals of the order;
//     counts, or 64-bit masses as two 32-bit additions: a 64-bit one in shared memory is a
//     loop of exchanges, measured several times slower) and the sums of every 32 bins; through
//     distributed shared memory every CTA finds the group, then the bin (reading all bins of
//     all CTAs instead takes longer than both). If at most kList ids are in it, every CTA
//     gathers them and ranks them all against all; else the interval of their bit patterns is
//     cut into 1024 again, until few are left or all are equal, when the cut falls by id.
//     A prefix of at most kFewList ids (the usual top-k) is gathered whole and finished there.
//  4. The kept mass per warp segment; one exchange; the CTA that holds u * total scans that
//     segment and writes the row's outputs. The others have exited.
// Exchanges are one cluster barrier each: 2, and 2 more for each of top-k and top-p. One more,
// arrived at before the read and waited for after it, tells that all CTAs have started.
//
// Measured (logits normal, sigma 2.5 or 3): 1 row x 51865 ids, top-k 50 and top-p 12 us; 64
// rows x 128000: min-p 21 us, top-p and min-p 38 us (of 70000 cycles 9500 read, 14500 weigh,
// 13000 cut, the rest draws and waits), top-k 50 and top-p 39.5 us, no filter 42 us, top-p 0.95
// alone 56 to 79 us (half of the ids are listed and weighed as heavy ones, up to four times),
// where more than 256 ids share a row's last bin another round of bins: up to 115, at top-p 0.99
// 129 to 142. Reading them once takes 4.8 us. Ranking by one 64-bit key, a warp's neighbours
// sharing an entry, and up to 256 ids: top-p 0.95 alone 97.7 -> 76.5 us on one set of logits.
#include <algorithm>
#include <climits>
#include <cstddef>
#include <mutex>

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {
namespace {

constexpr int kSfThreads = 512;
constexpr int kSfWarps = kSfThreads / 32;
constexpr int kSfMaxCluster = 16;
constexpr int kGroup = 32;                           // bins per group: a lane each
constexpr int kGroups = 32;
constexpr int kBins = kGroup * kGroups;
constexpr int kList = 256;                           // ids ranked all against all
constexpr int kFewList = 128;                        // the longest prefix finished that way
static_assert(kList <= kSfThreads && kFewList <= kList, "a thread per entry at least");
constexpr int kKeep = 8192;                          // logits of a slice kept in shared memory
constexpr int kMaxSlice = KVD_MAX_VOCAB / kSfMaxCluster;
constexpr float kYMax = 45.5f;                       // 2^-y below this is 0
constexpr float kHeavy = 16.f;                       // y of the heavy ids is below this,
constexpr float kHeavyFew = 8.f;                     // where min-p drops the light ones this
constexpr unsigned long long kOne = 1ull << 44;      // w = 1
constexpr uint32_t kMeanError = 149;                 // of ex2.approx, in 2^-32: 3.47e-8

// 2^(-j/256) in units of 2^-30, j < 256, from repeated products of 2^(-1/256).
struct PowTable {
    uint32_t t[256];
};
constexpr PowTable make_pow_table() {
    PowTable p = {};
    double v = 1073741824.0;  // 2^30
    for (int j = 0; j < 256; ++j) {
        p.t[j] = (uint32_t)(v + 0.5);
        v *= 0.99729605608547012625;  // 2^(-1/256)
    }
    return p;
}
__device__ const PowTable g_pow = make_pow_table();

struct FilterParams {
    const float* logits;
    int64_t row_stride;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* token;
    float* logprob;
    int32_t* n_kept;
    int32_t* dev_err;
    int32_t vocab, cluster, slice;  // slice: ids per CTA, a multiple of kSfThreads
};

// An id and its weight; keys fall with the order of the ids.
struct Entry {
    unsigned long long key, w;
};

struct alignas(16) FilterShared {
    uint32_t pow[256];
    // one bin: its mass (or its count), low and high half. Cleared after every use.
    uint2 hist[kBins];
    unsigned long long group[kSfMaxCluster][kGroups];   // sums of kGroup bins, of every CTA
    unsigned long long part[kSfMaxCluster][kGroup];     // one row per CTA of the cluster
    Entry list[kList];                   // this CTA's members
    Entry all[kList];                    // the cluster's
    // exchanged: written by CTA c into slot c of every CTA, each once per use below
    unsigned long long ex_best[kSfMaxCluster], ex_sum[kSfMaxCluster], ex_light[kSfMaxCluster],
        ex_key[kSfMaxCluster];
    uint32_t ex_fin[kSfMaxCluster], ex_cnt[kSfMaxCluster], ex_tie[kSfMaxCluster],
        ex_n[kSfMaxCluster];
    unsigned long long red[kSfWarps];
    uint32_t red32[kSfWarps], red_b[kSfWarps];
    uint32_t n_list, n_all;
    float cut_x, min_x;
    int32_t cut_id;
    int32_t found;
    // places of the listed ids in their warp's segment, a segment's length apart
    alignas(16) uint16_t lists[kMaxSlice];
    // (a slice of at most kKeep logits: lists in the first quarter, logits behind it)
};
static_assert(kKeep * 6 <= kMaxSlice * 2 && offsetof(FilterShared, lists) % 16 == 0,
              "kept logits, in 16-byte stores");
static_assert(kMaxSlice / kSfWarps <= 65536, "places in a segment are 16 bits");

// Total order of finite floats and infinities as unsigned integers (no -0 reaches it).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Logit descending, then id ascending.
__device__ __forceinline__ unsigned long long key_of(float x, int id) {
    return ((unsigned long long)ordered(x) << 32) | ~(uint32_t)id;
}
__device__ __forceinline__ float key_x(unsigned long long k) {
    return unordered((uint32_t)(k >> 32));
}
__device__ __forceinline__ int key_id(unsigned long long k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ void st_cluster_u64(void* local, int rank, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                     map_shared(smem_u32(local), (uint32_t)rank)),
                 "l"(v)
                 : "memory");
}
__device__ __forceinline__ void st_cluster_u32(void* local, int rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                     map_shared(smem_u32(local), (uint32_t)rank)),
                 "r"(v)
                 : "memory");
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(const void* local, int rank) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];"
                 : "=l"(v)
                 : "r"(map_shared(smem_u32(local), (uint32_t)rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ ulonglong2 ld_cluster_2u64(const void* local, int rank) {
    ulonglong2 v;
    asm volatile("ld.shared::cluster.v2.u64 {%0, %1}, [%2];"
                 : "=l"(v.x), "=l"(v.y)
                 : "r"(map_shared(smem_u32(local), (uint32_t)rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const void* local, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                 : "=r"(v)
                 : "r"(map_shared(smem_u32(local), (uint32_t)rank))
                 : "memory");
    return v;
}
// All threads of the cluster (of the block, when it is alone): writes before are visible to
// reads after.
__device__ __forceinline__ void sync_row(int cluster) {
    if (cluster > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
}

// The row's weights, in units of 2^-44.
struct Weights {
    float m, ch, cl;  // largest logit; log2(e) / T in two floats
    float split;      // heavy ids: y below this
    const uint32_t* pow;

    // y's leading part, monotone in x; 0 at the largest (which may be infinite)
    __device__ __forceinline__ float lead(float x) const {
        return (x == m ? 0.f : m - x) * ch;
    }
    // y = p + e
    __device__ __forceinline__ void exact(float x, float& p, float& e) const {
        const float d = x == m ? 0.f : m - x;
        p = d * ch;
        // m - x = d + dl exactly
        const float bb = d - m;
        const float dl = x == m ? 0.f : (m - (d - bb)) - (x + bb);
        e = fmaf(d, ch, -p) + fmaf(d, cl, dl * ch);
    }
    // (m - x) / T
    __device__ __forceinline__ float nats(float x) const {
        float p, e;
        exact(x, p, e);
        return fmaf(e, 0.693147181f, p * 0.693147181f);
    }
    // y < split
    __device__ __forceinline__ unsigned long long heavy(float x) const {
        float p, e;
        exact(x, p, e);
        // k = p * 256 rounded, in the low bits of kf + 1.5 * 2^23
        const float ks = fmaf(p, 256.f, 12582912.f), kf = ks - 12582912.f;
        const float r = fmaf(kf, -0.00390625f, p) + e;  // the first part is exact; |r| <= 2^-9
        // (2^-r - 1) * 2^32: -r ln 2 + (r ln 2)^2 / 2 - (r ln 2)^3 / 6
        const float q = r * fmaf(r, fmaf(r, -238388331.5f, 1031764992.f), -2977044471.8f);
        const int k = __float_as_int(ks) & 0x3FFF, n = k >> 8;  // n <= 16
        const int t = (int)pow[k & 255];
        // * 2^(14 - n), as a 32 x 32 -> 64 bit product
        return (unsigned long long)(uint32_t)(t + __mulhi(t, __float2int_rn(q))) *
                   (65536u >> n) >> 2;
    }
    // w * 2^13 * unit, with the mean error of the hardware's 2^x; 0 for -inf and NaN (a sum that
    // overflows is -inf or NaN, too)
    __device__ __forceinline__ uint32_t raw(float x, float unit) const {
        const float d = m - x;
        // 13 - y: a small number where the weight is not, so hardly rounded there
        const float a = fmaf(-d, cl, fmaf(-d, ch, 13.f));
        return __float2uint_rn(ex2_approx(a) * unit);
    }
    // y >= split = kHeavy
    __device__ __forceinline__ uint32_t light(float x) const {
        const uint32_t w = raw(x, 0x1p31f);
        return w - __umulhi(w, kMeanError);
    }
    __device__ __forceinline__ unsigned long long of(float x) const {
        return lead(x) < split ? heavy(x) : (unsigned long long)light(x);
    }
};

// floor(f * s) for 0 <= f < 1, exactly; `rest`: whether f * s is above it. Integers: double
// precision arithmetic of a whole block would cost microseconds here.
__device__ __forceinline__ unsigned long long mul_floor(float f, unsigned long long s,
                                                        bool& rest) {
    const uint32_t b = __float_as_uint(f);
    const int ex = (int)(b >> 23);  // f = mant * 2^-k
    const unsigned long long mant = (b & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const int k = 150 - max(ex, 1);  // 24 .. 149
    const unsigned long long hi = __umul64hi(mant, s), lo = mant * s;
    if (k < 64) {
        rest = (lo << (64 - k)) != 0;
        return (hi << (64 - k)) | (lo >> k);
    }
    // hi < 2^24: nothing is left of it from k = 88 on
    const int j = min(k - 64, 63);
    rest = lo != 0 || (hi & ((1ull << j) - 1)) != 0;
    return hi >> j;
}

// A prefix of the order: ids with x > cut_x, or x == cut_x and id <= cut_id.
struct Cut {
    float x;
    int32_t id;
    __device__ __forceinline__ bool keeps(float v, int i) const {
        return v > x || (v == x && i <= id);
    }
};

// Sum over the warp, to every lane (of values whose sum is below 2^64).
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
    const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x3FFFFFu);
    const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 22) & 0x3FFFFFu);
    const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 44));
    return a + ((unsigned long long)b << 22) + ((unsigned long long)c << 44);
}
__device__ __forceinline__ unsigned long long warp_incl(unsigned long long v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}
// Exclusive prefix over the block (thread order) of v, and the block's total. `red` is free
// for reuse only after the next block barrier.
__device__ __forceinline__ unsigned long long block_excl(FilterShared& S, unsigned long long v,
                                                         unsigned long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned long long inc = warp_incl(v);
    if (lane == 31) S.red[warp] = inc;
    __syncthreads();
    const unsigned long long w = lane < kSfWarps ? S.red[lane] : 0ull;
    total = warp_sum(w);
    return warp_sum(lane < warp ? w : 0ull) + inc - v;
}

struct Row {
    const float* x;  // this CTA's logits: in shared memory, or where they were given
    int n, lo, seg;  // logits here, the first one's id, logits per warp segment
    int rank, cluster;
    int w0, wn, wl;  // this warp's segment: first logit, logits, listed ones
    uint16_t* lj;    // the slice's lists, warp w's from w0 on

    __device__ __forceinline__ float at(int i) const {
        const float v = x[i];
        return isnan(v) ? -INFINITY : v + 0.f;  // -0 and +0 are one value
    }
};
// f(x, i) for the logits of this warp's segment: the listed ones, or all. The loads of several
// go first (f's atomics would hold later ones back).
template <typename F>
__device__ __forceinline__ void for_ids(const Row& R, bool full, F&& f) {
    const int lane = threadIdx.x & 31;
    if (full) {
        constexpr int G = 8;
#pragma unroll 1
        for (int j0 = lane; j0 < R.wn; j0 += 32 * G) {
            float v[G];
#pragma unroll
            for (int g = 0; g < G; ++g) v[g] = R.at(R.w0 + min(j0 + 32 * g, R.wn - 1));
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (j0 + 32 * g < R.wn) f(v[g], R.w0 + j0 + 32 * g);
        }
    } else {
        constexpr int G = 8;
        const uint16_t* lj = R.lj + R.w0;
#pragma unroll 1
        for (int j0 = lane; j0 < R.wl; j0 += 32 * G) {
            float v[G];
            int i[G];
#pragma unroll
            for (int g = 0; g < G; ++g) i[g] = R.w0 + lj[min(j0 + 32 * g, R.wl - 1)];
#pragma unroll
            for (int g = 0; g < G; ++g) v[g] = R.x[i[g]] + 0.f;  // (never a NaN)
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (j0 + 32 * g < R.wl) f(v[g], i[g]);
        }
    }
}

// The block's threads over n <= kSfThreads entries: `parts` neighbours (a power of two, at most a
// warp) share an entry, part p taking every parts-th of the others.
struct Share {
    int entry, part, parts;
};
__device__ __forceinline__ Share share_of(int n) {
    int lg = 0;
    while (lg < 5 && (n << (lg + 1)) <= kSfThreads) ++lg;
    return Share{(int)threadIdx.x >> lg, (int)threadIdx.x & ((1 << lg) - 1), 1 << lg};
}
__device__ __forceinline__ unsigned long long join(unsigned long long v, int parts) {
    for (int off = 1; off < parts; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

enum SelectResult { kCutHere, kBeyond, kAll, kFew };

// The last id of the shortest prefix (within `kept`) that holds `k` ids (MASS false) or whose
// mass reaches frac * (mass of `kept`) (MASS true; frac < 1; `light`: this CTA's light mass, 0
// when none of it is kept; only ids of weight w_min or more can be cut at, the others just add
// to the mass). Over the listed ids, or with `full` over all. Returns kBeyond, leaving `kept`,
// when the cut is not among the listed ids (of that weight); kAll when it is among none; kFew
// (counts only) with the whole prefix, and the rest of its last bin, in S.all of every CTA
// (S.n_all entries, in no order). Every thread of the cluster calls it; the histogram is clear
// before and after.
template <bool MASS>
__device__ SelectResult select(FilterShared& S, const Row& R, const Weights& W, bool full,
                               Cut& kept, unsigned long long k, float frac,
                               unsigned long long light, unsigned long long w_min) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto clear_hist = [&]() {
        for (int i = tid; i < kBins; i += kSfThreads) S.hist[i] = make_uint2(0u, 0u);
        __syncthreads();
    };
    // members of the current interval: all, then ordered keys in [klo, khi]
    bool first = true;
    uint32_t klo = 0, khi = 0;
    int shift = 0;
    unsigned long long before = 0;   // count or mass before the interval
    unsigned long long target = k;   // the prefix is complete once its count or mass is this
    const float scale = kBins / (full ? kYMax : W.split);
    auto bin_of = [&](float x, bool& in) -> int {
        if (first) {
            const float y = W.lead(x);
            in = y < kYMax;  // (the listed ones are below W.split)
            return min((int)(y * scale), kBins - 1);
        }
        const uint32_t key = ordered(x);
        in = key >= klo && key <= khi;
        return (int)((khi - key) >> shift);
    };
    for (;;) {
        // ---- histogram of the members over the bins ----
        unsigned long long mass = 0;
        for_ids(R, full, [&](float x, int i) {
            bool in;
            const int bin = bin_of(x, in);
            if (in && kept.keeps(x, R.lo + i)) {
                if (MASS) {
                    const unsigned long long w = full ? W.of(x) : W.heavy(x);
                    mass += w;
                    if (w < w_min) return;
                    const uint32_t lo = (uint32_t)w;
                    const uint32_t old = atomicAdd(&S.hist[bin].x, lo);
                    const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
                    if (hi) atomicAdd(&S.hist[bin].y, hi);
                } else {
                    atomicAdd(&S.hist[bin].x, 1u);
                }
            }
        });
        if (MASS && first) {
            mass = warp_sum(mass);
            if (lane == 0) S.red[warp] = mass;
        }
        __syncthreads();
        if (MASS && first) {  // this CTA's share of the mass that frac is of
            mass = light + warp_sum(lane < kSfWarps ? S.red[lane] : 0ull);
            if (R.cluster > 1) {
                if (tid < R.cluster) st_cluster_u64(&S.ex_light[R.rank], tid, mass);
            } else if (tid == 0) {
                S.ex_light[0] = mass;
            }
        }
#pragma unroll
        for (int h = 0; h < kGroups / kSfWarps; ++h) {
            const int g = warp * (kGroups / kSfWarps) + h;
            const uint2 v = S.hist[g * kGroup + lane];
            const unsigned long long sum = warp_sum(((unsigned long long)v.y << 32) | v.x);
            if (lane < R.cluster) {  // into every CTA
                if (R.cluster > 1) st_cluster_u64(&S.group[R.rank][g], lane, sum);
                else S.group[0][g] = sum;
            }
        }
        sync_row(R.cluster);
        // ---- the group, then the bin in which the prefix becomes complete ----
        // lane l gets the cluster's l-th of 32 sums in every CTA
        auto over_ctas = [&](const unsigned long long (*from)[kGroup]) -> unsigned long long {
            unsigned long long v = 0;
#pragma unroll 4
            for (int r = 0; r < R.cluster; ++r) v += from[r][lane];
            return v;
        };
        auto bins_of = [&](int g) -> unsigned long long {
            const unsigned long long* mine =
                reinterpret_cast<const unsigned long long*>(S.hist) + g * kGroup + lane;
            if (R.cluster == 1) return *mine;
            if (warp < R.cluster) S.part[warp][lane] = ld_cluster_u64(mine, warp);
            __syncthreads();
            return over_ctas(S.part);
        };
        if (tid == 0) S.n_list = 0;  // (every CTA has read the last list: it has arrived above)
        unsigned long long v = over_ctas(S.group);
        unsigned long long inc = before + warp_incl(v);
        if (first) {
            const unsigned long long total = __shfl_sync(0xffffffffu, inc, 31);
            if (MASS) {
                bool rest = false;
                const unsigned long long all =
                    warp_sum(lane < R.cluster ? S.ex_light[lane] : 0ull);
                target = frac > 0.f ? mul_floor(frac, all, rest) : 0ull;
                target += rest ? 1 : 0;  // a mass reaches frac * all when it is >= this
                if (target == 0) target = 1;
            }
            if (total < target) {  // the same in every CTA
                sync_row(R.cluster);  // all have read the sums
                clear_hist();
                return full ? kAll : kBeyond;
            }
        }
        uint32_t hit = __ballot_sync(0xffffffffu, inc >= target);
        const int grp = hit ? __ffs(hit) - 1 : 0;
        before = __shfl_sync(0xffffffffu, inc - v, grp);
        v = bins_of(grp);
        inc = before + warp_incl(v);
        hit = __ballot_sync(0xffffffffu, inc >= target);
        const int in_grp = hit ? __ffs(hit) - 1 : 0;
        before = __shfl_sync(0xffffffffu, inc - v, in_grp);
        const int bin = grp * kGroup + in_grp;
        // a short prefix is gathered whole: what follows needs no exchange then
        const bool few =
            !MASS && first && __shfl_sync(0xffffffffu, inc, in_grp) <=
                                  (unsigned long long)kFewList;
        __syncthreads();  // n_list is 0

        // ---- gather its members ----
        for_ids(R, full, [&](float x, int i) {
            bool in;
            const int mine = bin_of(x, in);
            if (in && (mine == bin || (few && mine < bin)) && kept.keeps(x, R.lo + i)) {
                const unsigned long long w = MASS || few ? W.of(x) : 1ull;
                if (MASS && w < w_min) return;
                const uint32_t at = atomicAdd(&S.n_list, 1u);
                if (at < kList) S.list[at] = Entry{key_of(x, R.lo + i), w};
            }
        });
        __syncthreads();
        if (tid < R.cluster) {
            if (R.cluster > 1) st_cluster_u32(&S.ex_n[R.rank], tid, S.n_list);
            else S.ex_n[0] = S.n_list;
        }
        sync_row(R.cluster);
        if (!few) clear_hist();  // all have read them (and after `few` no one does)
        const uint32_t nr = lane < R.cluster ? S.ex_n[lane] : 0u;
        const uint32_t n = __reduce_add_sync(0xffffffffu, nr);

        // ---- few: rank them all against all ----
        if (n <= kList) {
            // thread t: member t of the concatenated lists
            if (tid < kList) {  // whole warps
                uint32_t base = 0, off = 0;
                int from = 0;
                for (int r = 0; r < R.cluster; ++r) {
                    const uint32_t c = __shfl_sync(0xffffffffu, nr, r);
                    if ((uint32_t)tid >= base) {
                        from = r;
                        off = tid - base;
                    }
                    base += c;
                }
                if (tid < (int)n)
                    *reinterpret_cast<ulonglong2*>(&S.all[tid]) =
                        R.cluster > 1 ? ld_cluster_2u64(&S.list[off], from)
                                      : *reinterpret_cast<const ulonglong2*>(&S.list[off]);
            }
            if (tid == 0) S.n_all = n;
            __syncthreads();
            if (few) return kFew;
            const Share sh = share_of((int)n);
            const Entry me = S.all[min(sh.entry, max((int)n - 1, 0))];
            unsigned long long sum = 0;
#pragma unroll 4
            for (int k = sh.part; k < (int)n; k += sh.parts) {
                const Entry o = S.all[k];
                sum += o.key > me.key ? o.w : 0ull;
            }
            sum = before + join(sum, sh.parts);
            if (sh.entry < (int)n && sh.part == 0 && sum < target && sum + me.w >= target) {
                S.cut_x = key_x(me.key);
                S.cut_id = key_id(me.key);
            }
            __syncthreads();
            kept.x = S.cut_x;
            kept.id = S.cut_id;
            // (every CTA has read the others' lists before it arrives at the next exchange)
            return kCutHere;
        }

        // ---- many: the interval of their bit patterns ----
        uint32_t lo = 0xffffffffu, hi = 0;
        for_ids(R, full, [&](float x, int i) {
            bool in;
            const int mine = bin_of(x, in);
            if (in && mine == bin && kept.keeps(x, R.lo + i)) {
                const uint32_t key = ordered(x);
                lo = min(lo, key);
                hi = max(hi, key);
            }
        });
        __syncwarp();
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            S.red32[tid >> 5] = lo;
            S.red_b[tid >> 5] = hi;
        }
        __syncthreads();
        lo = __reduce_min_sync(0xffffffffu, S.red32[lane & (kSfWarps - 1)]);
        hi = __reduce_max_sync(0xffffffffu, S.red_b[lane & (kSfWarps - 1)]);
        if (R.cluster > 1) {
            if (tid < R.cluster)
                st_cluster_u64(&S.ex_key[R.rank], tid, ((unsigned long long)lo << 32) | hi);
            sync_row(R.cluster);
            const unsigned long long v = S.ex_key[lane & (R.cluster - 1)];
            lo = __reduce_min_sync(0xffffffffu, (uint32_t)(v >> 32));
            hi = __reduce_max_sync(0xffffffffu, (uint32_t)v);
        }
        first = false;
        klo = lo;
        khi = hi;
        if (klo < khi) {
            // cut (khi - klo + 1) patterns into at most kBins intervals
            static_assert(kBins == 1024, "the shift below");
            shift = max(0, 32 - __clz(khi - klo) - 10);
            continue;
        }

        // ---- all equal: the cut falls by id; the take-th of them is the last to stay ----
        const float xv = unordered(klo);
        unsigned long long take = target - before;
        if (MASS) {
            const unsigned long long w = W.of(xv);
            take = (take + w - 1) / w;  // the least number with enough mass; w > 0
        }
        auto member = [&](int i) {
            const float x = R.at(i);
            return ordered(x) == klo && kept.keeps(x, R.lo + i);
        };
        uint32_t c = 0;
        for (int i = tid; i < R.n; i += kSfThreads) c += member(i);
        c = __reduce_add_sync(0xffffffffu, c);
        __syncthreads();
        if (lane == 0) S.red32[tid >> 5] = c;
        __syncthreads();
        c = __reduce_add_sync(0xffffffffu, lane < kSfWarps ? S.red32[lane] : 0u);
        if (R.cluster > 1) {
            if (tid < R.cluster) st_cluster_u32(&S.ex_tie[R.rank], tid, c);
            sync_row(R.cluster);
        } else {
            if (tid == 0) S.ex_tie[0] = c;
            __syncthreads();
        }
        unsigned long long run = 0;
        int owner = 0;
        for (int r = 0; r < R.cluster; ++r) {
            if (run + S.ex_tie[r] >= take) {
                owner = r;
                break;
            }
            run += S.ex_tie[r];
        }
        take -= run;  // the take-th member of the owner's, in id order
        if (owner == R.rank) {
            // 512 ids at a time (a block-uniform loop)
            unsigned long long seen = 0;
            for (int i0 = 0; i0 < R.n; i0 += kSfThreads) {
                const int i = i0 + tid;
                const bool mine = i < R.n && member(i);
                unsigned long long all;
                const unsigned long long ex = block_excl(S, mine ? 1ull : 0ull, all);
                if (mine && seen + ex + 1 == take) {
                    if (R.cluster > 1)
                        for (int r = 0; r < R.cluster; ++r)
                            st_cluster_u32(&S.cut_id, r, (uint32_t)(R.lo + i));
                    else
                        S.cut_id = R.lo + i;
                }
                __syncthreads();
                seen += all;
                if (seen >= take) break;
            }
        }
        sync_row(R.cluster);
        kept.x = xv;
        kept.id = S.cut_id;
        return kCutHere;
    }
}

__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

// log of the share that the id with logit x and weight w has of `total`.
__device__ __forceinline__ float log_share(const Weights& W, float x, unsigned long long w,
                                           unsigned long long total) {
    // near 1 from what is left over, which the integers know exactly; for a light id from its
    // logit, as its weight is a number of few bits
    const float tf = (float)total;
    if (w > total / 2) return log1pf(-((float)(total - w) / tf));
    if (W.lead(x) < kHeavy) return logf((float)w / tf);
    return -W.nats(x) - logf(tf * 0x1p-44f);
}

// A short prefix, all in S.all: top-k, top-p, min-p and the draw by ranking every entry against
// every other.
__device__ void draw_few(FilterShared& S, const Weights& W, const FilterParams& p, int b,
                         int top_k, float top_p, unsigned long long w_min, float min_x, float y_max,
                         float u) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = (int)S.n_all;
    const Share sh = share_of(n);
    const bool mine = sh.entry < n;  // (its other threads know the same of the entry)
    const Entry me = S.all[min(sh.entry, max(n - 1, 0))];
    auto sum_all = [&](unsigned long long v) {  // over the entries
        v = warp_sum(mine && sh.part == 0 ? v : 0ull);
        __syncthreads();
        if (lane == 0) S.red[warp] = v;
        __syncthreads();
        return warp_sum(lane < kSfWarps ? S.red[lane] : 0ull);
    };
    unsigned long long before = 0, mass = 0;
#pragma unroll 4
    for (int i = sh.part; i < n; i += sh.parts) {
        const Entry o = S.all[i];
        const bool ahead = o.key > me.key;
        before += ahead;
        mass += ahead ? o.w : 0ull;
    }
    before = join(before, sh.parts);
    mass = join(mass, sh.parts);
    bool in = mine && before < (unsigned long long)top_k;
    if (top_p < 1.f) {  // (uniform)
        const unsigned long long all = sum_all(in ? me.w : 0ull);
        bool rest = false;
        unsigned long long target = top_p > 0.f ? mul_floor(top_p, all, rest) : 0ull;
        target += rest ? 1 : 0;
        if (target == 0) target = 1;
        in = in && mass < target;
    }
    in = in && me.w >= w_min && W.lead(key_x(me.key)) <= y_max && key_x(me.key) >= min_x;
    const unsigned long long w = in ? me.w : 0ull;
    if (tid == 0) S.n_list = 0;  // (the entries are in S.all: it counts the kept ones)
    __syncthreads();
    if (in && sh.part == 0) atomicAdd(&S.n_list, 1u);
    const unsigned long long total = sum_all(w);
    const uint32_t cnt = S.n_list;
    // (all have read the entries before the sums)
    if (mine && sh.part == 0) S.all[sh.entry].w = w;
    if (tid == 0) S.found = -1;
    __syncthreads();
    // the draw, in id order
    const bool lost = u >= 1.f;
    bool rest;
    const unsigned long long t = lost ? ~0ull : mul_floor(fmaxf(u, 0.f), total, rest) + 1;
    unsigned long long run = 0;
#pragma unroll 4
    for (int i = sh.part; i < n; i += sh.parts) {
        const Entry o = S.all[i];
        run += (uint32_t)o.key > (uint32_t)me.key ? o.w : 0ull;  // (a smaller id)
    }
    run = join(run, sh.parts);
    const int id = key_id(me.key);
    if (lost) {
        if (w > 0) atomicMax(&S.found, id);
        __syncthreads();
    }
    if (w > 0 && sh.part == 0 && (lost ? id == S.found : run < t && run + w >= t)) {
        p.token[b] = id;
        if (p.logprob) p.logprob[b] = log_share(W, key_x(me.key), w, total);
        if (p.n_kept) p.n_kept[b] = (int32_t)cnt;
    }
}

__global__ void __launch_bounds__(kSfThreads, 2) sample_filtered_kernel(const FilterParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    FilterShared& S = *reinterpret_cast<FilterShared*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Row R;
    R.cluster = p.cluster;
    R.rank = (int)(blockIdx.x % (unsigned)p.cluster);
    const int b = (int)(blockIdx.x / (unsigned)p.cluster);
    R.lo = R.rank * p.slice;
    R.n = max(0, min(p.slice, p.vocab - R.lo));
    R.seg = p.slice / kSfWarps;
    R.w0 = warp * R.seg;
    R.wn = max(0, min(R.seg, R.n - R.w0));
    if (tid < 256) S.pow[tid] = g_pow.t[tid];
    for (int i = tid; i < kBins; i += kSfThreads) S.hist[i] = make_uint2(0u, 0u);
    pdl_wait();
    pdl_trigger();
    const float T = p.temperature ? p.temperature[b] : 1.f;
    const float top_p = p.top_p ? p.top_p[b] : 1.f;
    const float min_p = p.min_p ? p.min_p[b] : 0.f;
    const int top_k = p.top_k ? p.top_k[b] : 0;
    const float u = p.u[b];
    // the same in every CTA of the row: all of them leave
    if (!(T >= 0.f) || !(T < INFINITY) || isnan(top_p) || isnan(min_p) || isnan(u)) {
        if (tid == 0 && R.rank == 0) flag_error(p.dev_err, KVD_ERR_BAD_PARAM);
        return;
    }

    // (every CTA of the row comes here or none: the first exchange waits until all have, as
    // nothing may be written into a CTA that has not started)
    if (R.cluster > 1) cluster_arrive_relaxed();

    // ---- 1. read; the largest logit, lowest id first; how many are above -inf ----
    const float* src = p.logits + (int64_t)b * p.row_stride + R.lo;
    const bool keep = p.slice <= kKeep;
    R.lj = S.lists;
    float* xs = reinterpret_cast<float*>(S.lists + kKeep);  // (keep)
    R.x = keep ? xs : src;
    // 16-byte loads where the row allows (segments start at multiples of 32 ids)
    const bool wide = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
    const int whole = wide ? R.wn & ~3 : 0;
    float top = -INFINITY;
    int top_i = 0;
    uint32_t n_fin = 0;
    bool nan = false;
    auto take = [&](float x, int i) -> float {  // ids ascend within a thread
        nan |= isnan(x);
        n_fin += x > -INFINITY;
        if (x > top) {
            top = x;
            top_i = i;
        }
        return x;
    };
    for (int j0 = lane * 4; j0 < whole; j0 += 512) {
        float4 v[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
            v[g] = __ldg(
                reinterpret_cast<const float4*>(src + R.w0 + min(j0 + g * 128, whole - 4)));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int i = R.w0 + j0 + g * 128;
            if (j0 + g * 128 < whole) {
                take(v[g].x, i);
                take(v[g].y, i + 1);
                take(v[g].z, i + 2);
                take(v[g].w, i + 3);
                if (keep) *reinterpret_cast<float4*>(xs + i) = v[g];
            }
        }
    }
    for (int j = whole + lane; j < R.wn; j += 256) {
        float v[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) v[g] = __ldg(src + R.w0 + min(j + 32 * g, R.wn - 1));
#pragma unroll
        for (int g = 0; g < 8; ++g)
            if (j + 32 * g < R.wn) {
                take(v[g], R.w0 + j + 32 * g);
                if (keep) xs[R.w0 + j + 32 * g] = v[g];
            }
    }
    const uint32_t fin_w = __reduce_add_sync(0xffffffffu, n_fin);
    {
        // the warp's largest, then the lowest id that has it (0: nothing above -inf)
        const uint32_t key = top > -INFINITY ? ordered(top + 0.f) : 0u;
        const uint32_t mk = __reduce_max_sync(0xffffffffu, key);
        const uint32_t mi =
            __reduce_min_sync(0xffffffffu, key == mk ? (uint32_t)(R.lo + top_i) : 0xffffffffu);
        if (lane == 0) {
            S.red[warp] = mk ? ((unsigned long long)mk << 32) | (uint32_t)~mi : 0ull;
            S.red32[warp] = fin_w;
        }
    }
    if (__syncthreads_or(nan) && tid == 0) flag_error(p.dev_err, KVD_ERR_NAN);
    auto best_of = [&](unsigned long long v) {  // the largest of the warp's
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
        const uint32_t lo =
            __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
        return ((unsigned long long)hi << 32) | lo;
    };
    unsigned long long best = best_of(lane < kSfWarps ? S.red[lane] : 0ull);
    uint32_t fin = __reduce_add_sync(0xffffffffu, lane < kSfWarps ? S.red32[lane] : 0u);
    if (R.cluster > 1) {
        __syncwarp();
        cluster_wait();  // every CTA has started: its shared memory can be written
        if (tid < R.cluster) {
            st_cluster_u64(&S.ex_best[R.rank], tid, best);
            st_cluster_u32(&S.ex_fin[R.rank], tid, fin);
        }
        sync_row(R.cluster);
        best = best_of(lane < R.cluster ? S.ex_best[lane] : 0ull);
        fin = __reduce_add_sync(0xffffffffu, lane < R.cluster ? S.ex_fin[lane] : 0u);
    }
    if (fin == 0) {
        if (tid == 0 && R.rank == 0) {
            p.token[b] = -1;
            if (p.logprob) p.logprob[b] = -INFINITY;
            if (p.n_kept) p.n_kept[b] = 0;
        }
        // (no CTA reads another's memory after the exchange)
        return;
    }
    // (no weight is above 1)
    if (T == 0.f || top_k == 1 || min_p > 1.f) {
        if (tid == 0 && R.rank == 0) {
            p.token[b] = (int32_t)~(uint32_t)best;
            if (p.logprob) p.logprob[b] = 0.f;
            if (p.n_kept) p.n_kept[b] = 1;
        }
        return;
    }
    Weights W;
    W.m = unordered((uint32_t)(best >> 32));
    W.pow = S.pow;
    {
        // log2(e) = 0x1.715476p0 + 0x1.4ae0cp-26, over T
        const float h = 0x1.715476p0f, l = 0x1.4ae0cp-26f;
        const float q = __fdiv_rn(h, T);
        W.ch = fminf(q, 3e38f);
        W.cl = q < 3e38f ? __fdiv_rn(fmaf(-q, T, h) + l, T) : 0.f;
    }

    // min-p: by the weight of heavy ids, else (weights of fewer bits) by the least logit that
    // passes, which one thread works out in 64 bits. Past y_max no id is kept (with room for y's
    // rounding)
    const bool by_w = !(min_p > 0.f && min_p < 0x1p-14f);
    if (!by_w && tid == 0)
        S.min_x = __double2float_ru((double)W.m + (double)T * log((double)min_p));
    unsigned long long w_min = 0;
    if (by_w && min_p > 0.f) {
        bool rest = false;
        w_min = min_p < 1.f ? mul_floor(min_p, kOne, rest) : kOne;
        w_min += rest ? 1 : 0;
    }
    const float y_max = min_p > 0.f ? fmaf(-log2f(min_p), 1.00001f, 1e-4f) : INFINITY;

    // ---- 2. the heavy ids of this warp's segment; the light ones' mass ----
    // (a top-k that cuts leaves no light id, or all ids are looked at)
    const bool cuts = top_k > 0 && (uint32_t)top_k < fin;
    // without masses to add up, the ids that min-p drops need not be listed either
    const bool masses = top_p < 1.f;
    // Where min-p drops an id, its weight is only added up: fp32's 2^-22 of it is enough.
    W.split = cuts ? kHeavy : fminf(kHeavy, fmaxf(kHeavyFew, y_max + 1.5f));
    const float y_list = cuts ? kHeavy : fminf(W.split, y_max);
    unsigned long long light_w = 0, light_40 = 0;  // (the second in units of 2^-40)
    R.wl = 0;
    const bool finite = W.m < INFINITY;
    if (finite) {
        const bool quads = keep || wide;
        // eight logits per lane of the 256 from jb on; place e of them
        auto place = [&](int jb, int e, bool q) {
            return q ? jb + lane * 4 + (e & 3) + 128 * (e >> 2) : jb + lane + 32 * e;
        };
        auto load8 = [&](int jb, float (&x)[8]) {
            if (quads && jb + 256 <= R.wn) {
                const float4 a = *reinterpret_cast<const float4*>(R.x + R.w0 + jb + lane * 4);
                const float4 c =
                    *reinterpret_cast<const float4*>(R.x + R.w0 + jb + lane * 4 + 128);
                x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
                x[4] = c.x; x[5] = c.y; x[6] = c.z; x[7] = c.w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = jb + lane + 32 * e;
                    x[e] = j < R.wn ? R.x[R.w0 + j] : -INFINITY;
                }
            }
        };
        uint16_t* lj = R.lj + R.w0;
        float next[8];
        load8(0, next);
        for (int jb = 0; jb < R.wn; jb += 256) {
            const bool q = quads && jb + 256 <= R.wn;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = next[e];
            load8(jb + 256, next);
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)  // (a NaN is neither: its lead is NaN, its weight 0)
                mine |= (W.m - x[e]) * W.ch < y_list ? 1u << e : 0u;
            if (masses && y_list < W.split) {
                uint32_t some = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool heavy = (W.m - x[e]) * W.ch < W.split;
                    some |= heavy ? 1u << e : 0u;
                    light_40 += heavy ? 0u : W.raw(x[e], 0x1p27f);
                }
                // few: read again rather than a branch for each of the eight
                for (some &= ~mine; some; some &= some - 1)
                    light_w += W.heavy(R.x[R.w0 + place(jb, __ffs(some) - 1, q)]);
            } else if (!cuts && y_list == W.split) {
#pragma unroll
                for (int e = 0; e < 8; ++e) light_w += mine >> e & 1 ? 0u : W.light(x[e]);
            }
            if (!__any_sync(0xffffffffu, mine != 0)) continue;
            uint32_t inc = __popc(mine);
            const uint32_t own = inc;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += o;
            }
            int at = R.wl + (int)(inc - own);
            R.wl += (int)__shfl_sync(0xffffffffu, inc, 31);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (mine >> e & 1) lj[at++] = (uint16_t)place(jb, e, q);
        }
    }
    light_w = warp_sum(light_w + ((light_40 - (light_40 * kMeanError >> 32)) << 4));
    __syncthreads();  // S.red is free
    if (lane == 0) S.red[warp] = light_w;
    __syncthreads();
    const unsigned long long light_cta = warp_sum(lane < kSfWarps ? S.red[lane] : 0ull);
    __syncthreads();  // S.red is free
    const bool plain = !cuts && !(top_p < 1.f) && !(min_p > 0.f);  // every id above -inf stays

    // ---- 3. the filters ----
    // light: what of the light ids is kept: all, none, or (all ids are to be looked at) some
    enum { kNone, kLightAll, kSome };
    int light = finite ? kLightAll : kSome;
    Cut kept = {-INFINITY, -1};
    if (cuts) {
        SelectResult r = kBeyond;
        if (light != kSome) {
            r = select<false>(S, R, W, false, kept, (unsigned long long)top_k, 0.f, 0ull, 0ull);
        }
        light = kNone;
        if (r == kBeyond) {
            r = select<false>(S, R, W, true, kept, (unsigned long long)top_k, 0.f, 0ull, 0ull);
            light = kSome;
        }
        if (r == kFew) {
            if (R.cluster > 1) cluster_arrive();  // this CTA has read the others' lists
            if (R.rank == 0)
                draw_few(S, W, p, b, top_k, top_p, w_min, by_w ? -INFINITY : S.min_x, y_max, u);
            if (R.cluster > 1) cluster_wait();  // the others have read this one's
            return;
        }
    }
    if (masses) {
        SelectResult r = kBeyond;
        if (light != kSome) {
            r = select<true>(S, R, W, false, kept, 0ull, top_p,
                             light == kLightAll ? light_cta : 0ull, w_min);
            if (r == kCutHere) light = kNone;
            // (where min-p keeps no light id, its prefix ends before top-p's)
            if (y_max < W.split - 1.f) r = kCutHere;
        }
        if (r == kBeyond &&
            select<true>(S, R, W, true, kept, 0ull, top_p, 0ull, w_min) == kCutHere)
            light = kSome;
    }
    if (!by_w && S.min_x > kept.x) kept = Cut{S.min_x, INT_MAX};
    if (light == kLightAll && min_p > 0.f) light = y_max < W.split - 1.f ? kNone : kSome;

    // ---- 4. the kept ids' mass, per warp segment ----
    unsigned long long sum = 0;
    uint32_t count = 0;
    auto weigh = [&](float x, int i, bool listed) -> unsigned long long {
        if (!kept.keeps(x, R.lo + i) || !(W.lead(x) <= y_max)) return 0ull;
        const unsigned long long w = listed ? W.heavy(x) : W.of(x);
        if (w < w_min) return 0ull;
        ++count;
        return w;
    };
    if (light == kSome) for_ids(R, true, [&](float x, int i) { sum += weigh(x, i, false); });
    else for_ids(R, false, [&](float x, int i) { sum += weigh(x, i, true); });
    __syncwarp();
    sum = warp_sum(sum);
    count = __reduce_add_sync(0xffffffffu, count);
    if (light == kLightAll) {  // every id above -inf is kept
        sum += light_w;
        count = 0;
    }
    __syncthreads();
    if (lane == 0) {
        S.red[warp] = sum;
        S.red32[warp] = count;
    }
    if (tid == 0) S.found = -1;
    __syncthreads();
    const unsigned long long seg_sum = lane < kSfWarps ? S.red[lane] : 0ull;
    const unsigned long long cta_sum = warp_sum(seg_sum);
    const uint32_t cta_cnt =
        __reduce_add_sync(0xffffffffu, lane < kSfWarps ? S.red32[lane] : 0u);
    unsigned long long ex_sum = lane == 0 ? cta_sum : 0ull;
    uint32_t cnt = cta_cnt;
    if (R.cluster > 1) {
        if (tid < R.cluster) {
            st_cluster_u64(&S.ex_sum[R.rank], tid, cta_sum);
            st_cluster_u32(&S.ex_cnt[R.rank], tid, cta_cnt);
        }
        sync_row(R.cluster);  // nothing is read from another CTA after this
        ex_sum = lane < R.cluster ? S.ex_sum[lane] : 0ull;
        cnt = __reduce_add_sync(0xffffffffu, lane < R.cluster ? S.ex_cnt[lane] : 0u);
    }
    if (plain || light == kLightAll) cnt = fin;
    const unsigned long long total = warp_sum(ex_sum);
    // the draw: the first id whose running mass exceeds u * total, i.e. is at least t (else the
    // last kept id of mass: u >= 1)
    bool rest;
    const bool lost = u >= 1.f;
    const unsigned long long t = lost ? ~0ull : mul_floor(fmaxf(u, 0.f), total, rest) + 1;
    // the first entry of v (one per lane) at which `from` + the running sum reaches t (lost:
    // the last one with any), and the sum before it
    auto find = [&](unsigned long long v, unsigned long long from,
                    unsigned long long& before) -> int {
        const unsigned long long inc = from + warp_incl(v);
        const uint32_t hit = __ballot_sync(0xffffffffu, lost ? v > 0 : inc >= t);
        const int l = hit ? (lost ? 31 - __clz(hit) : __ffs(hit) - 1) : 0;
        before = __shfl_sync(0xffffffffu, inc - v, l);
        return l;
    };
    unsigned long long run;
    if (find(ex_sum, 0ull, run) != R.rank) return;
    const int ow = find(seg_sum, run, run);
    // thread t of the block: ids [t * q, (t + 1) * q) of the segment
    const int w0 = ow * R.seg;
    const int len = max(0, min(R.seg, R.n - w0));
    const int q = (len + kSfThreads - 1) / kSfThreads;
    const int i0 = w0 + min(len, tid * q), i1 = w0 + min(len, (tid + 1) * q);
    unsigned long long part = 0;
    int last_i = -1;
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
        const unsigned long long w = weigh(R.at(i), i, false);
        part += w;
        if (w > 0) last_i = i;
    }
    __syncthreads();  // S.red is free
    unsigned long long dummy;
    const unsigned long long ex = run + block_excl(S, part, dummy);
    int token = -1;
    if (lost) {
        if (last_i >= 0) atomicMax(&S.found, last_i);
        __syncthreads();
        if (tid == 0) token = S.found;
    } else if (ex < t && ex + part >= t) {
        unsigned long long at = ex;
        for (int i = i0; i < i1; ++i) {
            at += weigh(R.at(i), i, false);
            if (at >= t) {
                token = i;
                break;
            }
        }
    }
    if (token >= 0) {
        p.token[b] = R.lo + token;
        if (p.logprob) p.logprob[b] = log_share(W, R.at(token), W.of(R.at(token)), total);
        if (p.n_kept) p.n_kept[b] = (int32_t)(top_k > 0 ? min((uint32_t)top_k, cnt) : cnt);
    }
}

constexpr int kMaxDevF = 64;
constexpr size_t kSfSmem = sizeof(FilterShared);
static_assert(2 * (kSfSmem + 1024) <= 227 * 1024, "two CTAs per SM");

// Once per device: shared memory and clusters of 16; the largest usable cluster.
int prepare_filtered() {
    static std::once_flag once[kMaxDevF];
    static int result[kMaxDevF];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevF) return 0;
    std::call_once(once[dev], [&] {
        if (cudaFuncSetAttribute(sample_filtered_kernel,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSfSmem) != cudaSuccess) {
            cudaGetLastError();
            return;
        }
        const bool big = cudaFuncSetAttribute(sample_filtered_kernel,
                                              cudaFuncAttributeNonPortableClusterSizeAllowed,
                                              1) == cudaSuccess;
        cudaGetLastError();
        int n = 0;
        if (big) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kSfMaxCluster);
            cfg.blockDim = dim3(kSfThreads);
            cfg.dynamicSmemBytes = kSfSmem;
            cudaLaunchAttribute a;
            a.id = cudaLaunchAttributeClusterDimension;
            a.val.clusterDim.x = kSfMaxCluster;
            a.val.clusterDim.y = 1;
            a.val.clusterDim.z = 1;
            cfg.attrs = &a;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, sample_filtered_kernel, &cfg) != cudaSuccess)
                n = 0;
            cudaGetLastError();
        }
        result[dev] = n > 0 ? kSfMaxCluster : 8;
    });
    return result[dev];
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_sample_filtered(const float* logits, int64_t row_stride, int32_t batch,
                                          int32_t vocab, const float* temperature,
                                          const int32_t* top_k, const float* top_p,
                                          const float* min_p, const float* u, int32_t* token,
                                          float* logprob, int32_t* n_kept, uint32_t flags,
                                          int32_t* dev_err, kvd_stream_t stream) {
    if (batch < 0 || vocab <= 0 || row_stride < vocab) return KVD_ERR_INVALID_ARG;
    if (vocab > KVD_MAX_VOCAB || batch > 65535) return KVD_ERR_UNSUPPORTED;
    if (batch == 0) return KVD_OK;
    if (!logits || !u || !token) return KVD_ERR_INVALID_ARG;
    const int nsm = sm_count();
    const int mc = prepare_filtered();
    if (nsm <= 0 || mc <= 0) return KVD_ERR_CUDA;
    // CTAs per row, a power of two: enough for the longest slice; then more while slices stay
    // long and all rows' CTAs are resident at once: two per SM, but one on every other SM where
    // 16 form a cluster, which fewer places fit (128000 ids, top-p and min-p, with 16, 8, 4: 1 row
    // 11.9, 15.1, 20.0 us, 4 rows 12.2, 15.4, 21.3, 8 rows 15.5, 16.3, 22.5, 16 rows 24.3, 20.0,
    // 21.9, 64 rows 69, 43.7, 34.0; 51865 ids, 8 rows: 13.6, 12.4, 16.6)
    int c = 1;
    while (c < mc && ((int64_t)c * kMaxSlice < vocab ||
                      (2ll * c * batch <= (c < 8 ? 2 * nsm : nsm / 2) &&
                       (int64_t)c * 2048 < vocab)))
        c *= 2;
    FilterParams p;
    p.slice = ((vocab + c - 1) / c + kSfThreads - 1) / kSfThreads * kSfThreads;
    p.cluster = c;
    p.logits = logits;
    p.row_stride = row_stride;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.u = u;
    p.token = token;
    p.logprob = logprob;
    p.n_kept = n_kept;
    p.dev_err = dev_err;
    p.vocab = vocab;
    if (p.slice > kMaxSlice) return KVD_ERR_UNSUPPORTED;  // (a device without clusters of 16)
    return launch_ex(sample_filtered_kernel, dim3((unsigned)(batch * c)), dim3(kSfThreads), kSfSmem,
                     reinterpret_cast<cudaStream_t>(stream), (flags & KVD_FLAG_PDL) != 0,
                     (unsigned)c, p);
}
