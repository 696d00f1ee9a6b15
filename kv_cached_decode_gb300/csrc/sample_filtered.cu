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
// of 2^-44 and sums are integers: the same on every run and for every split of the row. w
// itself is 2^-y with y = (max - x) * log2(e) / T carried in two floats, taken apart as
// 2^-n * 2^(-j/256) (a table) * 2^-r, |r| <= 2^-9 (a cubic): relative error below 2^-31, at
// about thirty fp32/integer instructions -- double precision would be 30 times slower here.
// Where w is below 2^-45.5 it is 0.
//
// Design. Bound by the chain of passes and exchanges for few rows, by instruction issue (the
// weights) for many; the logits are read from HBM once. One thread-block cluster per row;
// CTA c keeps the ids [c * slice, (c + 1) * slice) in shared memory.
//  1. Load, largest logit (lowest id first), number of logits above -inf: one exchange.
//  2. select(): the k-th id (counts) or the id at which the mass reaches its target. A
//     histogram of 2048 bins over y (bins fall with x, so they are intervals of the order;
//     counts, and 64-bit masses in the second case), summed over the cluster through
//     distributed shared memory (each CTA a share of the bins), names the bin. If at most
//     kList ids are in it, every CTA gathers them and ranks them all against all; else the
//     interval of their bit patterns is cut into 2048 again, until few are left or all are
//     equal, when the cut falls by id.
//  3. The kept ids' mass per 512-thread segment of the slice; one exchange; the CTA that holds
//     u * total scans that segment and writes the row's outputs. The others have exited.
#include <algorithm>
#include <mutex>

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {
namespace {

constexpr int kSfThreads = 512;
constexpr int kSfWarps = kSfThreads / 32;
constexpr int kSfMaxCluster = 16;
constexpr int kBins = 2048;
constexpr int kList = 128;
constexpr float kYMax = 45.5f;                       // 2^-y below this is 0
constexpr float kBinScale = (kBins - 1) / kYMax;     // the last bin: weight 0
constexpr unsigned long long kOne = 1ull << 44;      // w = 1

// 2^(-j/256) in units of 2^-44, j < 256, from repeated products of 2^(-1/256).
struct PowTable {
    unsigned long long t[256];
};
constexpr PowTable make_pow_table() {
    PowTable p = {};
    double v = 17592186044416.0;  // 2^44
    for (int j = 0; j < 256; ++j) {
        p.t[j] = (unsigned long long)(v + 0.5);
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

struct Entry {
    float x;
    int32_t id;
    unsigned long long w;
};

struct FilterShared {
    unsigned long long pow[256];
    unsigned long long mass[kBins];
    uint32_t cnt[kBins];
    // exchanged: written by CTA c into slot c of every CTA
    unsigned long long ex_best[kSfMaxCluster], ex_fin[kSfMaxCluster];
    unsigned long long ex_a[kSfMaxCluster], ex_b[kSfMaxCluster];
    unsigned long long res_mass;         // select's result, written by one CTA into all
    uint32_t res_cnt, res_n;
    int32_t res_bin;
    uint32_t n_list;
    Entry list[kList];                   // this CTA's members
    Entry all[kList];                    // the cluster's
    unsigned long long red[kSfWarps], red2[kSfWarps];
    float cut_x;
    int32_t cut_id;
    int32_t found;
};

// Total order of floats as unsigned integers (-0 below +0; both compare equal as floats, so
// callers order by the float first).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

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

// The row's weights. y in two floats (p, e).
struct Weights {
    float m, ch, cl;  // largest logit; log2(e) / T in two floats
    const unsigned long long* pow;

    // y's leading part, monotone in x; 0 at the largest, inf where the weight is 0 anyway
    __device__ __forceinline__ float lead(float x) const {
        return x == m ? 0.f : (m - x) * ch;
    }
    __device__ __forceinline__ unsigned long long of(float x) const {
        if (x == m) return kOne;
        const float d = m - x;
        const float p = d * ch;
        if (!(p < kYMax)) return 0ull;
        // m - x = d + dl exactly
        const float bb = d - m;
        const float dl = (m - (d - bb)) - (x + bb);
        const float e = fmaf(d, ch, -p) + fmaf(d, cl, dl * ch);
        const int k = __float2int_rn(p * 256.f);
        const float r = fmaf((float)k, -0.00390625f, p) + e;  // the first part is exact
        const float z = r * -0.693147180559945f;
        const float q = fmaf(z * z, fmaf(z, 0.16666667f, 0.5f), z);  // 2^-r - 1
        const unsigned long long t = pow[k & 255];
        const int n = k >> 8;
        const long long w =
            (long long)t +
            (((long long)(int32_t)(t >> 14) * (long long)__float2int_rn(q * 0x1p40f)) >> 26);
        return ((unsigned long long)w + ((1ull << n) >> 1)) >> n;
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

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
// Sum over the block of two values, to every thread. Ends with the arrays free for reuse.
__device__ __forceinline__ void block_sum2(FilterShared& S, unsigned long long& a,
                                           unsigned long long& b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) {
        S.red[warp] = a;
        S.red2[warp] = b;
    }
    __syncthreads();
    a = b = 0;
#pragma unroll
    for (int w = 0; w < kSfWarps; ++w) {
        a += S.red[w];
        b += S.red2[w];
    }
    __syncthreads();
}
// Exclusive prefix over the block (thread order) of v.
__device__ __forceinline__ unsigned long long block_excl(FilterShared& S, unsigned long long v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
    }
    if (lane == 31) S.red[warp] = inc;
    __syncthreads();
    unsigned long long base = 0;
#pragma unroll
    for (int w = 0; w < kSfWarps; ++w) base += w < warp ? S.red[w] : 0ull;
    __syncthreads();
    return base + inc - v;
}

struct Row {
    const float* x;  // this CTA's logits in shared memory (NaN replaced by -inf)
    int n, lo;       // how many, and the first one's id
    int rank, cluster;
};

// The last id of the shortest prefix (within `kept`) that holds `k` ids (MASS false) or whose
// mass reaches frac * (mass of `kept`) (MASS true; frac < 1). Returns false, leaving `kept`, when the
// prefix ends among ids of weight 0. Every thread of the cluster calls it.
template <bool MASS>
__device__ bool select(FilterShared& S, const Row& R, const Weights& W, Cut& kept,
                       unsigned long long k, float frac) {
    const int tid = threadIdx.x;
    // members of the current interval: all, then ordered keys in [klo, khi]
    bool first = true;
    uint32_t klo = 0, khi = 0;
    int shift = 0;
    unsigned long long before_c = 0, before_m = 0;
    unsigned long long target = k;  // the prefix is complete once its count or mass is this
    auto bin_of = [&](float x, bool& in) -> int {
        if (first) {
            const float y = W.lead(x);
            in = y < kYMax;
            return in ? (int)(y * kBinScale) : kBins - 1;
        }
        const uint32_t key = ordered(x);
        in = key >= klo && key <= khi;
        return (int)((khi - key) >> shift);
    };
    for (;;) {
        // ---- histogram of the members over the bins ----
        for (int i = tid; i < kBins; i += kSfThreads) {
            S.cnt[i] = 0;
            if (MASS) S.mass[i] = 0;
        }
        __syncthreads();
        for (int i = tid; i < R.n; i += kSfThreads) {
            const float x = R.x[i];
            bool in;
            const int bin = bin_of(x, in);
            if (in && kept.keeps(x, R.lo + i)) {
                atomicAdd(&S.cnt[bin], 1u);
                if (MASS) atomicAdd(&S.mass[bin], W.of(x));
            }
        }
        sync_row(R.cluster);
        // ---- this CTA's share of the bins, summed over the cluster ----
        const int share = kBins / R.cluster;  // a power of two of CTAs
        const int per = (share + kSfThreads - 1) / kSfThreads;  // at most 4
        unsigned long long c4[4], m4[4], cs = 0, ms = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c4[j] = m4[j] = 0;
            const int i = tid * per + j;
            if (j < per && i < share) {
                const int bin = R.rank * share + i;
                for (int r = 0; r < R.cluster; ++r) {
                    c4[j] += R.cluster > 1 ? ld_cluster_u32(&S.cnt[bin], r) : S.cnt[bin];
                    if (MASS)
                        m4[j] += R.cluster > 1 ? ld_cluster_u64(&S.mass[bin], r) : S.mass[bin];
                }
                cs += c4[j];
                ms += m4[j];
            }
        }
        unsigned long long pc = block_excl(S, cs), pm = MASS ? block_excl(S, ms) : 0ull;
        if (tid == kSfThreads - 1) {  // the share's totals
            S.red[0] = pc + cs;
            S.red[1] = pm + ms;
        }
        __syncthreads();
        if (tid < R.cluster) {
            if (R.cluster > 1) {
                st_cluster_u64(&S.ex_a[R.rank], tid, S.red[0]);
                st_cluster_u64(&S.ex_b[R.rank], tid, S.red[1]);
            } else {
                S.ex_a[0] = S.red[0];
                S.ex_b[0] = S.red[1];
            }
        }
        if (tid == 0) {
            S.n_list = 0;  // (every CTA has read the last list: it has arrived above)
            S.res_bin = -1;
        }
        sync_row(R.cluster);
        unsigned long long tc = 0, tmass = 0;
        for (int r = 0; r < R.cluster; ++r) {
            if (r == R.rank) {
                pc += tc;
                pm += tmass;
            }
            tc += S.ex_a[r];
            tmass += S.ex_b[r];
        }
        if (MASS && first) {
            bool rest = false;
            target = frac > 0.f ? mul_floor(frac, tmass, rest) : 0ull;
            target = target + (rest ? 1 : 0);  // a mass reaches frac * tmass when it is >= this
            if (target == 0) target = 1;
        }
        // ---- the bin at whose end the prefix is complete: one thread of the cluster has it ----
        pc += before_c;
        pm += before_m;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j >= per) break;
            const bool here = MASS ? pm < target && pm + m4[j] >= target
                                   : pc < target && pc + c4[j] >= target;
            if (here && c4[j] > 0 && tid * per + j < share) {
                for (int r = 0; r < R.cluster; ++r) {
                    const int bin = R.rank * share + tid * per + j;
                    if (R.cluster > 1) {
                        st_cluster_u64(&S.res_mass, r, pm);
                        st_cluster_u32(&S.res_cnt, r, (uint32_t)pc);
                        st_cluster_u32(&S.res_n, r, (uint32_t)c4[j]);
                        st_cluster_u32(&S.res_bin, r, (uint32_t)bin);
                    } else {
                        S.res_mass = pm;
                        S.res_cnt = (uint32_t)pc;
                        S.res_n = (uint32_t)c4[j];
                        S.res_bin = bin;
                    }
                }
            }
            pc += c4[j];
            pm += m4[j];
        }
        sync_row(R.cluster);
        const int bin = S.res_bin;
        if (bin < 0) return false;  // it ends among ids of weight 0: nothing to cut
        before_c = S.res_cnt;
        before_m = S.res_mass;
        const uint32_t n = S.res_n;

        // ---- few members: gather and rank them ----
        if (n <= kList) {
            for (int i = tid; i < R.n; i += kSfThreads) {
                const float x = R.x[i];
                bool in;
                const int mine = bin_of(x, in);
                if (in && mine == bin && kept.keeps(x, R.lo + i)) {
                    const uint32_t at = atomicAdd(&S.n_list, 1u);
                    if (at < kList) {
                        S.list[at].x = x;
                        S.list[at].id = R.lo + i;
                        S.list[at].w = MASS ? W.of(x) : 0ull;
                    }
                }
            }
            sync_row(R.cluster);
            if (R.cluster > 1) {
                int base = 0;
                for (int r = 0; r < R.cluster; ++r) {
                    const int nr = (int)ld_cluster_u32(&S.n_list, r);
                    if (tid < nr && base + tid < kList) {
                        const unsigned long long xi = ld_cluster_u64(&S.list[tid], r);
                        S.all[base + tid].x = __uint_as_float((uint32_t)xi);
                        S.all[base + tid].id = (int32_t)(xi >> 32);
                        S.all[base + tid].w = ld_cluster_u64(&S.list[tid].w, r);
                    }
                    base += nr;
                }
            } else if (tid < (int)n) {
                S.all[tid] = S.list[tid];
            }
            __syncthreads();
            if (tid < (int)n) {
                const Entry me = S.all[tid];
                unsigned long long c = before_c, mm = before_m;
                for (uint32_t i = 0; i < n; ++i) {
                    const Entry o = S.all[i];
                    if (o.x > me.x || (o.x == me.x && o.id < me.id)) {
                        ++c;
                        mm += o.w;
                    }
                }
                if (MASS ? mm < target && mm + me.w >= target : c + 1 == target) {
                    S.cut_x = me.x;
                    S.cut_id = me.id;
                }
            }
            __syncthreads();
            kept.x = S.cut_x;
            kept.id = S.cut_id;
            // (every CTA has read the others' lists before the next exchange completes)
            return true;
        }

        // ---- many: the interval of their bit patterns ----
        uint32_t lo = 0xffffffffu, hi = 0;
        for (int i = tid; i < R.n; i += kSfThreads) {
            const float x = R.x[i];
            bool in;
            const int mine = bin_of(x, in);
            if (in && mine == bin && kept.keeps(x, R.lo + i)) {
                const uint32_t key = ordered(x);
                lo = min(lo, key);
                hi = max(hi, key);
            }
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if ((tid & 31) == 0) S.red[tid >> 5] = ((unsigned long long)lo << 32) | hi;
        __syncthreads();
        lo = 0xffffffffu;
        hi = 0;
        for (int w = 0; w < kSfWarps; ++w) {
            lo = min(lo, (uint32_t)(S.red[w] >> 32));
            hi = max(hi, (uint32_t)S.red[w]);
        }
        if (R.cluster > 1) {
            if (tid < R.cluster)
                st_cluster_u64(&S.ex_a[R.rank], tid, ((unsigned long long)lo << 32) | hi);
            sync_row(R.cluster);
            for (int r = 0; r < R.cluster; ++r) {
                lo = min(lo, (uint32_t)(S.ex_a[r] >> 32));
                hi = max(hi, (uint32_t)S.ex_a[r]);
            }
        }
        __syncthreads();
        first = false;
        klo = lo;
        khi = hi;
        if (klo < khi) {
            // cut (khi - klo + 1) patterns into at most kBins intervals
            shift = max(0, 32 - __clz(khi - klo) - 11);
            continue;
        }

        // ---- all equal: the cut falls by id. r: how many of them stay ----
        unsigned long long take;
        if (MASS) {
            const float xv = __uint_as_float(klo & 0x80000000u ? klo & 0x7fffffffu : ~klo);
            const unsigned long long w = W.of(xv);
            take = (target - before_m + w - 1) / w;  // the least r with r * w enough; w > 0
        } else {
            take = target - before_c;
        }
        auto member = [&](int i) {
            return ordered(R.x[i]) == klo && kept.keeps(R.x[i], R.lo + i);
        };
        unsigned long long c = 0, none = 0;
        for (int i = tid; i < R.n; i += kSfThreads) c += member(i);
        block_sum2(S, c, none);
        if (R.cluster > 1) {
            if (tid < R.cluster) st_cluster_u64(&S.ex_b[R.rank], tid, c);
            sync_row(R.cluster);
        } else {
            if (tid == 0) S.ex_b[0] = c;
            __syncthreads();
        }
        unsigned long long run = 0;
        int owner = 0;
        for (int r = 0; r < R.cluster; ++r) {
            if (run + S.ex_b[r] >= take) {
                owner = r;
                break;
            }
            run += S.ex_b[r];
        }
        take -= run;  // the take-th member of the owner's, in id order
        if (owner == R.rank) {
            // 512 ids at a time (a block-uniform loop)
            unsigned long long seen = 0;
            for (int i0 = 0; i0 < R.n; i0 += kSfThreads) {
                const int i = i0 + tid;
                const bool mine = i < R.n && member(i);
                const unsigned long long ex = block_excl(S, mine ? 1ull : 0ull);
                if (mine && seen + ex + 1 == take) {
                    if (R.cluster > 1)
                        for (int r = 0; r < R.cluster; ++r)
                            st_cluster_u32(&S.cut_id, r, (uint32_t)(R.lo + i));
                    else
                        S.cut_id = R.lo + i;
                }
                unsigned long long all = mine ? 1ull : 0ull, none2 = 0;
                block_sum2(S, all, none2);
                seen += all;
                if (seen >= take) break;
            }
        }
        sync_row(R.cluster);
        kept.x = __uint_as_float(klo & 0x80000000u ? klo & 0x7fffffffu : ~klo);
        kept.id = S.cut_id;
        return true;
    }
}

__global__ void __launch_bounds__(kSfThreads, 2) sample_filtered_kernel(const FilterParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    FilterShared& S = *reinterpret_cast<FilterShared*>(smem_raw);
    float* xs = reinterpret_cast<float*>(smem_raw + sizeof(FilterShared));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Row R;
    R.cluster = p.cluster;
    R.rank = (int)(blockIdx.x % (unsigned)p.cluster);
    const int b = (int)(blockIdx.x / (unsigned)p.cluster);
    R.lo = R.rank * p.slice;
    R.n = max(0, min(p.slice, p.vocab - R.lo));
    R.x = xs;
    if (tid < 256) S.pow[tid] = g_pow.t[tid];
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

    // ---- 1. load; the largest logit, lowest id first; how many are above -inf ----
    const float* src = p.logits + (int64_t)b * p.row_stride + R.lo;
    unsigned long long best = 0;  // (ordered x, ~id)
    uint32_t n_fin = 0;
    bool nan = false;
    constexpr int G = 8;
    for (int i0 = tid; i0 < R.n; i0 += G * kSfThreads) {
        float v[G];
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const int i = i0 + j * kSfThreads;
            v[j] = i < R.n ? __ldcs(src + i) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const int i = i0 + j * kSfThreads;
            if (i >= R.n) break;
            float x = v[j];
            if (isnan(x)) {
                nan = true;
                x = -INFINITY;
            }
            x = x == 0.f ? 0.f : x;  // -0 and +0 are one value
            xs[i] = x;
            n_fin += x > -INFINITY;
            const unsigned long long key =
                ((unsigned long long)ordered(x) << 32) | (uint32_t)~(R.lo + i);
            best = key > best ? key : best;
        }
    }
    if (__syncthreads_or(nan) && tid == 0) flag_error(p.dev_err, KVD_ERR_NAN);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
        best = o > best ? o : best;
    }
    n_fin = __reduce_add_sync(0xffffffffu, n_fin);
    if (lane == 0) {
        S.red[warp] = best;
        S.red2[warp] = n_fin;
    }
    __syncthreads();
    unsigned long long fin = 0;
    for (int w = 0; w < kSfWarps; ++w) {
        best = S.red[w] > best ? S.red[w] : best;
        fin += S.red2[w];
    }
    if (R.cluster > 1) {
        if (tid < R.cluster) {
            st_cluster_u64(&S.ex_best[R.rank], tid, best);
            st_cluster_u64(&S.ex_fin[R.rank], tid, fin);
        }
        sync_row(R.cluster);
        best = fin = 0;
        for (int r = 0; r < R.cluster; ++r) {
            best = S.ex_best[r] > best ? S.ex_best[r] : best;
            fin += S.ex_fin[r];
        }
    }
    __syncthreads();
    if (fin == 0) {
        if (tid == 0 && R.rank == 0) {
            p.token[b] = -1;
            if (p.logprob) p.logprob[b] = -INFINITY;
            if (p.n_kept) p.n_kept[b] = 0;
        }
        // (no CTA reads another's memory after the exchange)
        return;
    }
    if (T == 0.f || top_k == 1) {
        if (tid == 0 && R.rank == 0) {
            p.token[b] = (int32_t)~(uint32_t)best;
            if (p.logprob) p.logprob[b] = 0.f;
            if (p.n_kept) p.n_kept[b] = 1;
        }
        return;
    }
    Weights W;
    const uint32_t mk = (uint32_t)(best >> 32);
    W.m = __uint_as_float(mk & 0x80000000u ? mk & 0x7fffffffu : ~mk);
    W.pow = S.pow;
    {
        // log2(e) = 0x1.715476p0 + 0x1.4ae0cp-26, over T
        const float h = 0x1.715476p0f, l = 0x1.4ae0cp-26f;
        const float q = __fdiv_rn(h, T);
        W.ch = fminf(q, 3e38f);
        W.cl = q < 3e38f ? __fdiv_rn(fmaf(-q, T, h) + l, T) : 0.f;
    }

    // ---- 2. the filters ----
    Cut kept = {-INFINITY, -1};
    if (top_k > 0 && (unsigned long long)top_k < fin)
        select<false>(S, R, W, kept, (unsigned long long)top_k, 0.f);
    if (top_p < 1.f) select<true>(S, R, W, kept, 0ull, top_p);
    // min-p by the weight, or (where it is too small for the weight's unit) by y
    const bool by_w = min_p >= 0x1p-40f;
    unsigned long long w_min = 0;
    if (by_w) {
        bool rest = false;
        w_min = min_p < 1.f ? mul_floor(min_p, kOne, rest) : kOne;
        w_min += rest ? 1 : 0;
    }
    const float y_max = min_p > 0.f && !by_w ? -log2f(min_p) : INFINITY;

    // ---- 3. the kept ids' mass, per segment of kSfThreads * q ids of this CTA ----
    // warp w: segment w of the slice
    const int seg = (p.slice / kSfThreads) * 32;  // ids per warp
    unsigned long long sum = 0, count = 0;
    auto weigh = [&](int i, unsigned long long& c) -> unsigned long long {
        const float x = xs[i];
        if (!kept.keeps(x, R.lo + i) || !(W.lead(x) <= y_max)) return 0ull;
        const unsigned long long w = W.of(x);
        if (w < w_min) return 0ull;
        c += 1;
        return w;
    };
    for (int i = warp * seg + lane; i < min(R.n, (warp + 1) * seg); i += 32) sum += weigh(i, count);
    sum = warp_sum(sum);
    count = warp_sum(count);
    __syncthreads();
    if (lane == 0) {
        S.red[warp] = sum;
        S.red2[warp] = count;
    }
    __syncthreads();
    unsigned long long mine = 0, cnt = 0;
    for (int w = 0; w < kSfWarps; ++w) {
        mine += S.red[w];
        cnt += S.red2[w];
    }
    if (R.cluster > 1) {
        if (tid < R.cluster) {
            st_cluster_u64(&S.ex_a[R.rank], tid, mine);
            st_cluster_u64(&S.ex_b[R.rank], tid, cnt);
        }
        sync_row(R.cluster);  // nothing is read from another CTA after this
    } else {
        if (tid == 0) {
            S.ex_a[0] = mine;
            S.ex_b[0] = cnt;
        }
        __syncthreads();
    }
    unsigned long long total = 0;
    cnt = 0;
    for (int r = 0; r < R.cluster; ++r) {
        total += S.ex_a[r];
        cnt += S.ex_b[r];
    }
    // the draw: the first id whose running mass exceeds u * total, i.e. is at least t (else the
    // last kept id of mass: u >= 1)
    bool rest;
    const unsigned long long t = u >= 1.f ? ~0ull : mul_floor(fmaxf(u, 0.f), total, rest) + 1;
    unsigned long long run = 0, run_owner = 0;
    int owner = -1, last = 0;
    for (int r = 0; r < R.cluster; ++r) {
        if (owner < 0 && run + S.ex_a[r] >= t) {
            owner = r;
            run_owner = run;
        }
        if (S.ex_a[r] > 0) last = r;
        run += S.ex_a[r];
    }
    const bool lost = owner < 0;  // u >= 1
    if (lost) owner = last;
    if (owner != R.rank) return;
    // the warp segment of this CTA
    int ow = -1, lw = 0;
    run = run_owner;
    unsigned long long run_w = run;
    for (int w = 0; w < kSfWarps; ++w) {
        if (!lost && ow < 0 && run + S.red[w] >= t) {
            ow = w;
            run_w = run;
        }
        if (S.red[w] > 0) lw = w;
        run += S.red[w];
    }
    if (lost) ow = lw;
    __syncthreads();
    if (tid == 0) S.found = -1;
    // thread t of the block: ids [t * q, (t + 1) * q) of the segment
    const int q = (seg + kSfThreads - 1) / kSfThreads;
    const int s0 = ow * seg, s1 = min(R.n, s0 + seg);
    const int i0 = min(s1, s0 + tid * q), i1 = min(s1, i0 + q);
    unsigned long long part = 0, dummy = 0;
    int last_i = -1;
    for (int i = i0; i < i1; ++i) {
        const unsigned long long w = weigh(i, dummy);
        part += w;
        if (w > 0) last_i = i;
    }
    const unsigned long long ex = run_w + block_excl(S, part);
    int token = -1;
    if (lost) {
        if (last_i >= 0) atomicMax(&S.found, last_i);
    } else if (ex < t && ex + part >= t) {
        unsigned long long at = ex;
        for (int i = i0; i < i1; ++i) {
            at += weigh(i, dummy);
            if (at >= t) {
                token = i;
                break;
            }
        }
    }
    if (lost) {
        __syncthreads();
        if (tid == 0) token = S.found;
    }
    if (token >= 0) {
        p.token[b] = R.lo + token;
        if (p.logprob) {
            // near 1 from what is left over, which the integers know exactly
            const unsigned long long w = W.of(xs[token]);
            const float tf = (float)total;
            p.logprob[b] = w > total / 2 ? log1pf(-((float)(total - w) / tf)) : logf((float)w / tf);
        }
        if (p.n_kept)
            p.n_kept[b] = (int32_t)(top_k > 0 && (unsigned long long)top_k < cnt ? top_k : cnt);
    }
}

constexpr int kMaxDevF = 64;

// Once per device: shared memory and clusters of 16; the largest usable cluster.
int prepare_filtered(size_t smem) {
    static std::once_flag once[kMaxDevF];
    static int result[kMaxDevF];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevF) return 0;
    std::call_once(once[dev], [&] {
        if (cudaFuncSetAttribute(sample_filtered_kernel,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess) {
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
            cfg.dynamicSmemBytes = smem;
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
    constexpr int kMaxSlice = KVD_MAX_VOCAB / kSfMaxCluster;  // 128 KiB of logits
    constexpr size_t kMost = sizeof(FilterShared) + (size_t)kMaxSlice * sizeof(float);
    static_assert(kMost <= 227 * 1024, "shared memory");
    const int mc = prepare_filtered(kMost);
    if (mc <= 0) return KVD_ERR_CUDA;
    // the fewest CTAs (a power of two) whose slices hold the row
    int c = 1;
    while (c < mc && (int64_t)c * kSfThreads * 16 < vocab) c *= 2;
    FilterParams p;
    p.slice = ((vocab + c - 1) / c + kSfThreads - 1) / kSfThreads * kSfThreads;
    if (p.slice > kMaxSlice) return KVD_ERR_UNSUPPORTED;  // (clusters of 8 only)
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
    const size_t smem = sizeof(FilterShared) + (size_t)p.slice * sizeof(float);
    return launch_ex(sample_filtered_kernel, dim3((unsigned)(batch * c)), dim3(kSfThreads), smem,
                     reinterpret_cast<cudaStream_t>(stream), (flags & KVD_FLAG_PDL) != 0,
                     (unsigned)c, p);
}
