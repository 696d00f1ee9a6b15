// token_logprobs.cu -- log probabilities of given tokens, their ranks, the row's entropy and its
// best alternatives, in one pass over the logits.
//
// "Inference 抽象と KV キャッシュ" of "Whisper のデコーダー内部": the decoder sums the chosen
// tokens' log probabilities; the rest has no counterpart on the pages. For a row x, temperature T,
// largest logit M, held by n ids, and d_v = x_v - M:
//   S = n + R,  R = sum over the others of exp(d_v / T)        (n is counted, not summed)
//   lse = M / T + log S,   log p_t = d_t / T - log S           (log1p(R) where n is 1)
//   entropy = log S - (sum exp(d_v / T) d_v) / (T S)           (both terms >= 0)
// so a log probability near 0 keeps its relative precision.
//
// Design. One read of the row bounds many rows (HBM), the chain of a pass few.
//  * A row is one block, or for few rows one cluster of blocks with a slice each, merged in the
//    first block's shared memory. A block takes rounds of 4096 logits, 16 per thread, which bulk
//    copies bring into a ring in shared memory.
//  * Per logit: y = x c - M c in one FMA (c = log2 e / T), its power of two, two sums, in two-lane
//    fp32: 2.5 instructions. M is the block's largest of the first round, and a warp's own from
//    where that is exceeded; only a warp whose chunk holds M itself tells it apart from the rest.
//    What rounding M c shifts every y by is known and undone in the sums.
//  * Ranks: a compare and half an add per logit and token, only for chunks that reach the token's
//    logit; ids below the token count equal logits, ids above do not, so the threshold is set per
//    vector of consecutive ids.
//  * Alternatives: an id is one 64-bit key (order of the logit, then lower id). After the first
//    round the n-th largest of 64 groups' maxima is a bound that at least n ids reach; from then
//    on a thread whose chunk exceeds it notes the chunk, one compare per 16 logits. Noted chunks
//    are read again, their keys that reach the bound listed, and the same step over the list
//    raises the bound: it leaves at most half of it, whatever the order of the row, and in the end
//    at most 128 keys, ranked by counting.
//  * A chunk with a logit of -inf has no finite sum of exponents: it is added logit by logit. Rows
//    with masks scattered over them so take longer.
//
// Measured (in a graph): 1 x 51865 fp32, 5 alternatives 9.0 us, a chain of barriers; 64 x 128000
// bf16, a rank, 20 alternatives 21.2 us (half of the ids masked, scattered: 23.5; the first half:
// 21.0); 2000 x 51865 fp32, a rank, one alternative 90.5 us, 4.6 TB/s (masked so: 107 and 88),
// issue on 59 % of the cycles. Registers are spilled in every build (bytes stored and loaded per
// thread): 20 to 30 and 32 to 36 without ranks, 130 to 142 and 140 to 152 for one given token, both
// in 64 registers; 18 to 34 and 12 to 108 for more, in 80 and 128.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kPer = 16;                          // logits per thread and round
constexpr int kRound = kLpThreads * kPer;
constexpr int kStageBytes = kRound * 4;           // a round of fp32, two of 16-bit logits
constexpr int kStages = 2;                        // of the ring
constexpr int kGroups = 64;
constexpr int kRanked = 128;                      // keys ranked by counting
constexpr int kNotedSoft = 64;                    // noted chunks from which they are looked into
constexpr int kNotedCap = kNotedSoft + 2 * kLpThreads;  // (a round notes one per thread at most)
constexpr int kPass = 64;                         // noted chunks per pass
constexpr int kListSoft = 256;                    // keys from which the list is cut
constexpr int kListCap = kListSoft + kPass * kPer + 32;  // (and 2 x 7 from the row's ends)
constexpr int kLpMaxCluster = 16;
constexpr float kFar = -3.402823466e38f;          // for -inf in weight * exponent (0 * -inf is NaN)
// Blocks a launch should have before rows are no longer split (64 x 128000 bf16 at 1, 2, 3, 4 per
// SM: 27.8, 21.4, 21.4, 21.5 us; 256 x 32000: 20.0, 19.9, 20.0, 21.5).
constexpr int64_t kLpManyBlocks = 152 * 2;

// Tokens per row that a build of three blocks per SM holds (771 rows of 102542 fp32 logits with 2
// given tokens: 78 us, 95 with the build for 16; 1514 of 18529 f16 with 4: 53 and 62).
constexpr int kFewGiven = 4;

constexpr float kLn2 = 0.69314718056f;

typedef unsigned long long Key;

struct LogprobParams {
    const void* x;
    int64_t stride;           // elements
    int32_t rows, vocab, cluster, slice;
    const float* temperature;
    const int32_t* tokens;
    int32_t given;
    float* logprob;
    int32_t* rank;
    float* entropy;
    float* lse;
    int32_t top;
    int32_t* top_id;
    float* top_logprob;
    int32_t* dev_err;
    int32_t test_stall;
};

// Sums of a part of a row: largest logit (-inf: none), how many have it, the others' weights
// relative to it and their sum of weight * exponent (log2 units).
struct Part {
    float m, n, rest, ent;
};
struct __align__(128) LpShared {
    uint8_t ring[kStages * kStageBytes];
    Key list[kListCap];
    Key group[kLpThreads];
    int32_t noted[kNotedCap];                       // round * kLpThreads + thread
    Part part[kLpWarps];
    float first[kLpWarps];                          // largest logits of the first round
    int32_t count[KVD_MAX_GIVEN];
    // of every CTA of the cluster, in the first one's: nothing else lies there, as the others
    // write it while the first may still be at its own slice
    Key ex_key[kLpMaxCluster * KVD_MAX_TOP];
    Part ex_part[kLpMaxCluster];
    int32_t ex_count[kLpMaxCluster][KVD_MAX_GIVEN];
    int32_t ex_lost[kLpMaxCluster];                 // whether one's wait ran out
    int32_t token[KVD_MAX_GIVEN];
    float value[KVD_MAX_GIVEN];                     // the tokens' logits
    int32_t place[kGroups];
    uint64_t bars[kStages];
    Key bound;
    int32_t n_list, n_noted, lost;
};

// Order-preserving image of a logit (not NaN, -0 as +0) above the complement of the id.
__device__ __forceinline__ Key make_key(float v, int id) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return ((Key)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32) | (uint32_t)~(uint32_t)id;
}
__device__ __forceinline__ float key_value(Key k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_id(Key k) { return (int)~(uint32_t)k; }

// The largest key of a warp: the high words first, then the low ones of the lanes that have it.
__device__ __forceinline__ Key warp_max_key(Key k) {
    const uint32_t hi = (uint32_t)(k >> 32), top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? (uint32_t)k : 0u);
    return ((Key)top << 32) | lo;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// -1 if v >= at, else 0 (one compare, and half a three-input add).
__device__ __forceinline__ int at_least(float v, float at) {
    int d;
    asm("set.ge.s32.f32 %0, %1, %2;" : "=r"(d) : "f"(v), "f"(at));
    return d;
}
// The next fp32 above v; NaN, which nothing reaches, above +inf.
__device__ __forceinline__ float next_up(float v) {
    if (!(v < INFINITY)) return __uint_as_float(0x7fffffffu);
    if (v == 0.f) return __uint_as_float(1u);
    const uint32_t u = __float_as_uint(v);
    return __uint_as_float(u & 0x80000000u ? u - 1 : u + 1);
}

__device__ __forceinline__ Part join(const Part& a, const Part& b, float c) {
    Part r;
    r.m = fmaxf(a.m, b.m);
    if (r.m == -INFINITY) return a;
    r.n = r.rest = r.ent = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const Part& x = k ? b : a;
        if (x.m == r.m) {
            r.n += x.n;
            r.rest += x.rest;
            r.ent += x.ent;
        } else if (x.m > -INFINITY) {
            const float y = (x.m - r.m) * c, f = exp2f(y), s = x.n + x.rest;
            if (f > 0.f) {
                r.rest = fmaf(s, f, r.rest);
                r.ent = fmaf(f, fmaf(y, s, x.ent), r.ent);
            }
        }
    }
    return r;
}
__device__ __forceinline__ Part shfl_part(const Part& a, int off) {
    Part r;
    r.m = __shfl_xor_sync(0xffffffffu, a.m, off);
    r.n = __shfl_xor_sync(0xffffffffu, a.n, off);
    r.rest = __shfl_xor_sync(0xffffffffu, a.rest, off);
    r.ent = __shfl_xor_sync(0xffffffffu, a.ent, off);
    return r;
}

// n parts, at most N of them (a power of two), joined by a warp; every lane gets the result.
template <int N>
__device__ __forceinline__ Part join_few(const Part* parts, int n, float c) {
    const int lane = threadIdx.x & 31;
    Part a = {-INFINITY, 0.f, 0.f, 0.f};
    if (lane < n) a = parts[lane];
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) a = join(a, shfl_part(a, o), c);
    return a;
}

// The largest of the warp's values (none is NaN).
__device__ __forceinline__ float warp_max(float v) {
    float d;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}
// A thread's running sums: exponents are x c + mc, mc = -m c rounded, and lo what that lacks. Where
// |m c| is so large (2^25 on, past fp32, or NaN) that lo may be more than 1, 2^lo may leave fp32.
// mc is NaN then, which sends every chunk to add_one and its exponents (x - m) c.
struct Sums {
    Part a;
    float c, mc, lo;
    __device__ __forceinline__ void set_reference(float m) {
        a.m = m;
        mc = -(m * c);
        lo = -fmaf(m, c, mc);
        if (!(fabsf(lo) <= 1.f)) {
            lo = 0.f;
            mc = __uint_as_float(0x7fffffffu);
        }
    }
    // lo goes into the sums.
    __device__ __forceinline__ void settle() {
        const float f = exp2f(lo);
        a.ent = f * fmaf(lo, a.rest, a.ent);
        a.rest *= f;
    }
    __device__ __forceinline__ void raise_to(float m) {
        if (!(m > a.m)) return;
        settle();
        // (as add_one: sums by a reference lack its lo; y is -inf where there are none yet)
        float y = (a.m - m) * c;
        const float s = a.n + a.rest;
        set_reference(m);
        y -= lo;
        const float f = exp2f(y);
        a.rest = s * f;
        a.ent = f > 0.f ? f * fmaf(y, s, a.ent) : 0.f;
        a.n = 0.f;
    }
    __device__ __forceinline__ void add_one(float x) {
        if (x == a.m) {
            a.n += 1.f;
        } else {
            const float y = (x - a.m) * c - lo, e = ex2_approx(y);
            a.rest += e;
            a.ent = fmaf(e, fmaxf(y, kFar), a.ent);
        }
    }
    // None of the logits is above a.m, which is above -inf. top: whether any of the warp's is a.m.
    template <int N>
    __device__ __forceinline__ void add_chunk(const float (&x)[N], bool top) {
        if (!top) {
            Pair r[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)}, t[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
            const Pair cc(c, c), mm(mc, mc);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const Pair y = fma2(Pair(x[i], x[i + 1]), cc, mm);
                const float2 z = y.get();
                const Pair e(ex2_approx(z.x), ex2_approx(z.y));
                r[(i >> 1) & 1] = add2(r[(i >> 1) & 1], e);
                t[(i >> 1) & 1] = fma2(e, y, t[(i >> 1) & 1]);
            }
            const float2 rs = add2(r[0], r[1]).get(), ts = add2(t[0], t[1]).get();
            const float ent = ts.x + ts.y;
            if (ent == ent) {  // (a logit of -inf: 0 * -inf is NaN; and see mc)
                a.rest += rs.x + rs.y;
                a.ent += ent;
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) add_one(x[i]);
    }
};

template <typename T> struct Vec;  // 16 bytes of logits
template <> struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void get(const uint4& u, float* x) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ float one(float v) { return v; }
};
template <> struct Vec<__half> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void get(const uint4& u, float* x) { unpack8<__half>(u, x); }
    static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void get(const uint4& u, float* x) {
        unpack8<__nv_bfloat16>(u, x);
    }
    static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
};
// S.bound: the n-th largest of 64 groups' largest keys, out of S.group[t], a key per thread
// (thread t's group is t % 64). All threads; the caller has not synchronised since its write.
__device__ __forceinline__ void set_bound(LpShared& S, int n) {
    const int tid = threadIdx.x;
    __syncthreads();
    Key g = 0;
    if (tid < kGroups) {
#pragma unroll
        for (int k = 0; k < kLpThreads / kGroups; ++k) g = max(g, S.group[tid + k * kGroups]);
        S.group[tid] = g;
        S.place[tid] = 0;
    }
    const int some = __syncthreads_count(g != 0);
    {
        const Key mine = S.group[tid % kGroups];
        int above = 0;
        constexpr int each = kGroups * kGroups / kLpThreads;
        const int k0 = tid / kGroups * each;
#pragma unroll
        for (int k = 0; k < each; ++k) above += S.group[k0 + k] > mine;
        if (above) atomicAdd(&S.place[tid % kGroups], above);
    }
    __syncthreads();
    // (groups without an id share the key 0 and the first place behind the others)
    if (tid < kGroups) {
        const Key mine = S.group[tid];
        if (S.place[tid] == n - 1 && mine != 0) S.bound = mine;
    }
    if (tid == 0 && some < n) S.bound = 1;  // every id
    __syncthreads();
}

// Cuts the list down to the entries that reach a bound at least n of them reach: at most n *
// ceil(entries / 64). All threads, after a barrier.
__device__ __noinline__ void cut_list(LpShared& S, int n) {
    const int tid = threadIdx.x, have = S.n_list;
    constexpr int kMost = (kListCap + kLpThreads - 1) / kLpThreads;
    Key best = 0;
    for (int i = tid; i < have; i += kLpThreads) best = max(best, S.list[i]);
    S.group[tid] = best;
    set_bound(S, n);
    const Key bound = S.bound;
    Key own[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int i = tid + k * kLpThreads;
        own[k] = i < have ? S.list[i] : 0;
    }
    __syncthreads();
    if (tid == 0) S.n_list = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMost; ++k)
        if (own[k] >= bound && own[k] != 0) S.list[atomicAdd(&S.n_list, 1)] = own[k];
    __syncthreads();
}

// The list's n largest keys in order, into out (0 where there are fewer). All threads, after a
// barrier; out is not in the list's place.
__device__ __forceinline__ void rank_list(LpShared& S, int n, Key* out) {
    const int tid = threadIdx.x;
    while (S.n_list > kRanked) cut_list(S, n);  // (uniform)
    const int have = S.n_list, whole = (have + 3) & ~3;
    if (tid < n) out[tid] = 0;
    if (tid >= have && tid < whole) S.list[tid] = 0;
    __syncthreads();
    if (tid < have) {
        const Key mine = S.list[tid];
        const ulonglong2* list = reinterpret_cast<const ulonglong2*>(S.list);
        int above = 0;
        for (int i = 0; i < whole / 2; i += 2) {
            const ulonglong2 a = list[i], b = list[i + 1];
            above += (a.x > mine) + (a.y > mine) + (b.x > mine) + (b.y > mine);
        }
        if (above < n) out[above] = mine;
    }
    __syncthreads();
}

__device__ __forceinline__ void push(LpShared& S, Key k) { S.list[atomicAdd(&S.n_list, 1)] = k; }

// The noted chunks' keys that reach the bound go to the list, which is cut as it grows. x: the
// row's first whole vector, of id `id0`; `vecs` of them. All threads, after a barrier; ends with
// one.
template <typename T>
__device__ __noinline__ void look_into(LpShared& S, const T* x, int id0, int vecs, int n) {
    constexpr int VN = Vec<T>::n, NV = kPer / VN;
    const int tid = threadIdx.x, have = S.n_noted;
    for (int c0 = 0; c0 < have; c0 += kPass) {
        const int n_vec = min(kPass, have - c0) * NV;
        constexpr int kEach = (kPass * NV + kLpThreads - 1) / kLpThreads;  // vectors per thread
        uint4 raw[kEach];
        int at[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = tid + k * kLpThreads;
            at[k] = vecs;
            if (i < n_vec) {
                const int chunk = S.noted[c0 + i / NV];
                at[k] = (chunk / kLpThreads * NV + i % NV) * kLpThreads + chunk % kLpThreads;
                if (at[k] < vecs) raw[k] = __ldg(reinterpret_cast<const uint4*>(x) + at[k]);
            }
        }
        const Key bound = S.bound;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (at[k] >= vecs) continue;
            float f[VN];
            Vec<T>::get(raw[k], f);
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                const Key key = make_key(f[e], id0 + at[k] * VN + e);
                if (key >= bound && f[e] > -INFINITY) push(S, key);  // (not NaN)
            }
        }
        __syncthreads();
        if (S.n_list > kListSoft) {
            while (S.n_list > kRanked) cut_list(S, n);
        }
        __syncthreads();  // nobody adds before all have seen the count
    }
    if (S.n_list > kGroups) cut_list(S, n);  // a higher bound for what comes
    if (tid == 0) S.n_noted = 0;
    __syncthreads();
}

__device__ __forceinline__ void st_cluster_key(void* local, int rank, Key v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                     map_shared(smem_u32(local), (uint32_t)rank)),
                 "l"(v)
                 : "memory");
}
__device__ __forceinline__ void st_cluster_word(void* local, int rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                     map_shared(smem_u32(local), (uint32_t)rank)),
                 "r"(v)
                 : "memory");
}

// GIVEN: the most tokens per row whose ranks are counted.
template <typename T, int GIVEN>
__global__ void __launch_bounds__(kLpThreads, GIVEN > 4 ? 2 : GIVEN > 1 ? 3 : 4)
    token_logprobs_kernel(const LogprobParams p) {
    extern __shared__ uint8_t lp_smem[];
    LpShared& S = *reinterpret_cast<LpShared*>(
        (reinterpret_cast<uintptr_t>(lp_smem) + 127) & ~uintptr_t(127));
    constexpr int VN = Vec<T>::n, NV = kPer / VN;
    constexpr int kSub = 4 / (int)sizeof(T);  // rounds per stage
    static_assert(kSub <= 2, "the noted chunks' place");
    constexpr int kTok = GIVEN > 1 ? GIVEN : 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)(blockIdx.x % (unsigned)p.cluster);
    const int row = (int)(blockIdx.x / (unsigned)p.cluster);
    if (p.cluster > 1) cluster_arrive_relaxed();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&S.bars[i]), 1);
        fence_barrier_init();
        S.n_list = S.n_noted = 0;
    }
    pdl_wait();
    pdl_trigger();
    const T* x = static_cast<const T*>(p.x) + row * p.stride;
    const int lo = min(rank * p.slice, p.vocab), hi = min(lo + p.slice, p.vocab);
    // [lo, hi): up to VN - 1 logits, then whole 16-byte vectors, then up to VN - 1
    const int off = (int)((reinterpret_cast<uintptr_t>(x + lo) / sizeof(T)) % VN);
    const int body = min(hi, lo + (off ? VN - off : 0));
    const int vecs = (hi - body) / VN, tail = body + vecs * VN;
    const int rounds = (vecs + NV * kLpThreads - 1) / (NV * kLpThreads);
    const int stages = (rounds + kSub - 1) / kSub;
    auto copy = [&](int g) {  // one thread
        const int at = g * kStageBytes, bytes = min(kStageBytes, vecs * 16 - at);
        const uint32_t bar = smem_u32(&S.bars[g % kStages]);
        mbar_expect_tx(bar, bytes);
        bulk_load(smem_u32(S.ring + g % kStages * kStageBytes),
                  reinterpret_cast<const uint8_t*>(x + body) + at, bytes, bar);
    };
    if (tid == 0) {
        // test only: 16 bytes more than the first copy brings
        if (p.test_stall && stages > 0 && rank == row % p.cluster)
            mbar_expect_tx_only(smem_u32(&S.bars[0]), 16);
        for (int g = 0; g < min(kStages, stages); ++g) copy(g);
    }
    const float T_ = p.temperature ? p.temperature[row] : 1.f;
    const bool bad_t = !(T_ > 0.f) || !(T_ < INFINITY);
    if (tid < p.given) {
        const int t = p.tokens[(int64_t)row * p.given + tid];
        const bool in = t >= 0 && t < p.vocab;
        S.token[tid] = in ? t : -1;
        S.value[tid] = in ? fmaxf(Vec<T>::one(x[t]), -INFINITY) : 0.f;
        S.count[tid] = 0;
        if (!in && t != -1 && rank == 0) flag_error(p.dev_err, KVD_ERR_BAD_TOKEN);
    }
    // the ends that are not whole vectors: one logit of a thread
    float end_v = -INFINITY;
    int end_id = -1;
    bool nan = false;
    if (tid < body - lo) end_id = lo + tid;
    else if (tid >= 32 && tid - 32 < hi - tail) end_id = tail + tid - 32;
    if (end_id >= 0) {
        const float one = Vec<T>::one(x[end_id]);
        nan = one != one;
        end_v = fmaxf(one, -INFINITY);
    }
    __syncthreads();
    int tok[kTok], cnt[kTok];
    float val[kTok], val_up[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        cnt[i] = 0;
        if (GIVEN && i < p.given) {
            tok[i] = S.token[i];
            val[i] = S.value[i];
            val_up[i] = next_up(val[i]);
            if (end_id >= 0)
                cnt[i] -= end_v > val[i] || (end_v == val[i] && end_id < tok[i]);
        }
    }

    Sums sum;
    sum.a = {-INFINITY, 0.f, 0.f, 0.f};
    sum.c = kLog2e / T_;
    sum.mc = sum.lo = 0.f;
    // alternatives: one is the largest key seen, several take a bound and a list
    const bool single = p.top == 1, several = p.top > 1;
    float bound_v = -INFINITY;  // of S.bound; of a single one, the warp's largest so far
    int best_id = -1;
    // The first round's largest logits and bound. cm: the thread's largest, of id `id`.
    auto begin = [&](float cm, int id) {
        const float w = warp_max(fmaxf(cm, end_v));
        if (lane == 0) S.first[warp] = w;
        if (several) {
            const bool head = end_v > -INFINITY && end_id < body;
            const Key mine = head ? make_key(end_v, end_id) : 0;
            S.group[tid] = max(mine, cm > -INFINITY ? make_key(cm, id) : 0);
            set_bound(S, p.top);
            const Key bound = S.bound;
            bound_v = bound == 1 ? -INFINITY : key_value(bound);
            if (head && mine >= bound) push(S, mine);
        } else {
            __syncthreads();
        }
        float m = S.first[0];
#pragma unroll
        for (int k = 1; k < kLpWarps; ++k) m = fmaxf(m, S.first[k]);
        if (m > -INFINITY) {
            sum.set_reference(m);
            if (end_v > -INFINITY) sum.add_one(end_v);
        }
    };
    bool dead = false, full = false;
    // One round; MASKED: the first, or one with vectors that lie behind the slice.
    auto round = [&](int r, auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
        const int g = r / kSub, sub = r % kSub;
        if (sub == 0)
            dead = dead || !mbar_wait_bounded(smem_u32(&S.bars[g % kStages]), (g / kStages) & 1);
        const uint4* st = reinterpret_cast<const uint4*>(S.ring + g % kStages * kStageBytes) +
                          sub * NV * kLpThreads + tid;
        // the thread's first vector; kLpThreads apart
        const int v0 = r * NV * kLpThreads + tid;
        float v[kPer];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!MASKED || v0 + k * kLpThreads < vecs) {
                Vec<T>::get(st[k * kLpThreads], v + k * VN);
            } else {
#pragma unroll
                for (int i = 0; i < VN; ++i) v[k * VN + i] = -INFINITY;
            }
        }
        auto largest = [&]() {
            float q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = max_nan(max3_nan(v[e], v[e + 4], v[e + 8]), v[e + 12]);
            return max_nan(max3_nan(q[0], q[1], q[2]), q[3]);
        };
        float cm = largest();
        if (cm != cm) {
            nan = true;
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = fmaxf(v[i], -INFINITY);
            cm = largest();
        }
        auto id_of_largest = [&]() {
            int id = 0;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i)
                if (v[i] == cm) id = body + (v0 + i / VN * kLpThreads) * VN + i % VN;
            return id;
        };
        if (MASKED && r == 0) begin(cm, several ? id_of_largest() : 0);
        const float top_of = warp_max(cm);
        if (single && top_of > bound_v) {  // (the same in the whole warp)
            bound_v = top_of;
            best_id = cm == top_of ? id_of_largest() : -1;
        }
        if (top_of > -INFINITY) {  // (the same in the whole warp, like the reference)
            sum.raise_to(top_of);
            if (!MASKED || cm > -INFINITY) sum.add_chunk(v, top_of == sum.a.m);
        }
        if (GIVEN) {
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                if (GIVEN > 1 && i >= p.given) break;
                if (cm < val[i]) continue;
                // all of a round before the token, or behind it
                const int from = body + r * NV * kLpThreads * VN;  // the round's first id
                const bool before = tok[i] >= from + NV * kLpThreads * VN;
                if (!MASKED && (before || tok[i] < from)) {
                    const float at = before ? val[i] : val_up[i];
#pragma unroll
                    for (int e = 0; e < kPer; ++e) cnt[i] += at_least(v[e], at);
                    continue;
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    if (MASKED && v0 + k * kLpThreads >= vecs) break;
                    // ids below the token's count equal logits
                    const int id0 = body + (v0 + k * kLpThreads) * VN;
                    const float at = id0 < tok[i] ? val[i] : val_up[i];
#pragma unroll
                    for (int e = 0; e < VN; ++e) cnt[i] += at_least(v[k * VN + e], at);
                    // (of the vector that holds the token, those from it on do not)
                    if ((unsigned)(tok[i] - id0 - 1) < (unsigned)(VN - 1)) {
#pragma unroll
                        for (int e = 0; e < VN; ++e)
                            cnt[i] += id0 + e >= tok[i] && v[k * VN + e] == val[i];
                    }
                }
            }
        }
        // (later ids need more than the bound's logit)
        const bool note = several && cm > -INFINITY &&
                          (MASKED && r == 0 ? cm >= bound_v : cm > bound_v);
        if (note) {
            const int at = atomicAdd(&S.n_noted, 1);
            S.noted[at] = r * kLpThreads + tid;
            full |= at >= kNotedSoft;
        }
        if (MASKED && rounds == 1 && several) {
            // a short slice: straight to the list, while the logits are at hand
            __syncthreads();
            const int noted = S.n_noted;
            __syncthreads();
            if (noted <= kPass) {
                if (tid == 0) S.n_noted = 0;
                if (note) {
                    const Key bound = S.bound;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const Key k =
                            make_key(v[i], body + (v0 + i / VN * kLpThreads) * VN + i % VN);
                        if (k >= bound && v[i] > -INFINITY) push(S, k);
                    }
                }
            }
        }
    };
    int issued = min(kStages, stages);
    bool lost = false;
    if (rounds == 0) begin(-INFINITY, 0);
    for (int g = 0; g < stages; ++g) {
        full = false;
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
            const int r = g * kSub + sub;
            if (r >= rounds) break;
            if (r > 0 && (r + 1) * NV * kLpThreads <= vecs) round(r, std::false_type{});
            else round(r, std::true_type{});
        }
        if (g + 1 == stages) break;
        // the stage is read; (nobody notes a chunk while they are looked into)
        if (__syncthreads_or(dead || full)) {
            if ((lost = __syncthreads_or(dead))) break;
            look_into<T>(S, x + body, body, vecs, p.top);
            const Key bound = S.bound;
            bound_v = bound == 1 ? -INFINITY : key_value(bound);
        }
        if (issued < stages) {
            if (tid == 0) {
                fence_proxy_async();
                copy(issued);
            }
            ++issued;
        }
    }

    // ---- the block's sums and counts ----
    if (nan && !dead) flag_error(p.dev_err, KVD_ERR_NAN);
    if (sum.a.m > -INFINITY) sum.settle();
    Part a = sum.a;
    const float c = sum.c;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {  // (the warp shares its reference)
        a.n += __shfl_xor_sync(0xffffffffu, a.n, o);
        a.rest += __shfl_xor_sync(0xffffffffu, a.rest, o);
        a.ent += __shfl_xor_sync(0xffffffffu, a.ent, o);
    }
    if (lane == 0) S.part[warp] = a;
    if (single) {
        Key k = best_id >= 0 ? make_key(bound_v, best_id) : 0;
        if (end_v > -INFINITY) k = max(k, make_key(end_v, end_id));
        k = warp_max_key(k);
        if (lane == 0) S.group[warp] = k;
    }
    if (GIVEN) {
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (GIVEN > 1 && i >= p.given) break;
            const int n = __reduce_add_sync(0xffffffffu, cnt[i]);
            if (lane == 0) atomicSub(&S.count[i], n);
        }
    }
    // (a wait that ran out: the copies in flight land before the block leaves, and the row is not
    // written; a cluster's blocks all pass its barriers)
    if (__syncthreads_or(dead)) lost = true;
    if (lost && tid == 0) {
        flag_error(p.dev_err, KVD_ERR_TIMEOUT);
        for (int g = max(0, issued - kStages); g < issued; ++g)
            mbar_wait_bounded(smem_u32(&S.bars[g % kStages]), (g / kStages) & 1);
    }
    if (warp == 0) a = join_few<kLpWarps>(S.part, kLpWarps, c);
    Key* best = S.group;  // [top]
    if (single) {
        if (warp == 0) {
            const Key k = warp_max_key(lane < kLpWarps ? S.group[lane] : 0);
            if (lane == 0) best[0] = k;
        }
    } else if (several) {
        if (S.n_noted > 0 && !lost) look_into<T>(S, x + body, body, vecs, p.top);
        if (end_id >= body && end_v > -INFINITY) {
            const Key k = make_key(end_v, end_id);
            if (k >= S.bound) push(S, k);
        }
        __syncthreads();
        rank_list(S, p.top, best);
    }
    // ---- the cluster's, in its first block ----
    if (p.cluster > 1) {
        cluster_wait();  // every block has started: its shared memory can be written
        if (tid < p.top) st_cluster_key(&S.ex_key[rank * p.top + tid], 0, best[tid]);
        if (tid == 0) {
            st_cluster_word(&S.ex_part[rank].m, 0, __float_as_uint(a.m));
            st_cluster_word(&S.ex_part[rank].n, 0, __float_as_uint(a.n));
            st_cluster_word(&S.ex_part[rank].rest, 0, __float_as_uint(a.rest));
            st_cluster_word(&S.ex_part[rank].ent, 0, __float_as_uint(a.ent));
            st_cluster_word(&S.ex_lost[rank], 0, lost);
        }
        if (GIVEN && tid < p.given)
            st_cluster_word(&S.ex_count[rank][tid], 0, (uint32_t)S.count[tid]);
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank != 0) return;
        if (warp == 0) {
            a = join_few<kLpMaxCluster>(S.ex_part, p.cluster, c);
            lost = __any_sync(0xffffffffu, lane < p.cluster && S.ex_lost[lane]);
        }
        if (tid == 0) S.n_list = p.cluster * p.top;
        if (GIVEN && tid < p.given) {
            int n = 0;
            for (int k = 0; k < p.cluster; ++k) n += S.ex_count[k][tid];
            S.count[tid] = n;
        }
        if (single) {
            if (warp == 0) {
                const Key k = warp_max_key(lane < p.cluster ? S.ex_key[lane] : 0);
                if (lane == 0) best[0] = k;
            }
        } else if (several) {
            for (int i = tid; i < p.cluster * p.top; i += kLpThreads) S.list[i] = S.ex_key[i];
            __syncthreads();
            rank_list(S, p.top, best);
        }
    }
    // ---- the outputs ----
    __syncthreads();
    if (tid == 0) {
        S.part[0] = a;
        S.lost = lost;
    }
    __syncthreads();
    if (bad_t || S.lost) {
        if (bad_t && tid == 0) flag_error(p.dev_err, KVD_ERR_BAD_PARAM);
        return;
    }
    a = S.part[0];
    const bool none = a.m == -INFINITY;
    const float log_s = none ? -INFINITY : a.n == 1.f ? log1pf(a.rest) : logf(a.n + a.rest);
    auto logprob = [&](float v) {
        if (none || v == -INFINITY) return -INFINITY;
        return v == a.m ? -log_s : (v - a.m) / T_ - log_s;
    };
    if (tid < p.given) {
        const int t = S.token[tid];
        const int64_t o = (int64_t)row * p.given + tid;
        if (p.logprob) p.logprob[o] = t < 0 ? 0.f : logprob(S.value[tid]);
        if (GIVEN && p.rank) p.rank[o] = t < 0 ? -1 : S.count[tid];
    }
    if (tid < p.top) {
        const Key k = best[tid];
        const int64_t o = (int64_t)row * p.top + tid;
        if (p.top_id) p.top_id[o] = k ? key_id(k) : -1;
        if (p.top_logprob) p.top_logprob[o] = k ? logprob(key_value(k)) : -INFINITY;
    }
    if (tid == 0) {
        if (p.lse) p.lse[row] = none ? -INFINITY : a.m / T_ + log_s;
        if (p.entropy)
            p.entropy[row] = none ? 0.f : log_s - a.ent * kLn2 / (a.n + a.rest);
    }
}

constexpr size_t kLpSmem = sizeof(LpShared) + 128;
constexpr int kMaxDevL = 64;

// Once per kernel and device: shared memory, clusters of 16.
template <auto Kern>
bool prepare_logprobs() {
    static std::once_flag once[kMaxDevL];
    static bool ok[kMaxDevL];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevL) return false;
    std::call_once(once[dev], [&] {
        ok[dev] = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kLpSmem) == cudaSuccess &&
                  cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                      cudaSuccess;
        cudaGetLastError();
    });
    return ok[dev];
}

template <typename T, int GIVEN>
kvd_status run(const LogprobParams& p, bool pdl, cudaStream_t st) {
    constexpr auto kern = token_logprobs_kernel<T, GIVEN>;
    if (!prepare_logprobs<kern>()) return KVD_ERR_CUDA;
    return launch_ex(kern, dim3((unsigned)p.rows * (unsigned)p.cluster), dim3(kLpThreads),
                     kLpSmem, st, pdl, (unsigned)p.cluster, p);
}
template <typename T>
kvd_status run_type(const LogprobParams& p, bool pdl, cudaStream_t st) {
    if (!p.rank || p.given == 0) return run<T, 0>(p, pdl, st);
    if (p.given == 1) return run<T, 1>(p, pdl, st);
    return p.given <= kFewGiven ? run<T, kFewGiven>(p, pdl, st)
                                : run<T, KVD_MAX_GIVEN>(p, pdl, st);
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_token_logprobs(kvd_dtype dtype, const void* logits, int64_t row_stride,
                                         int32_t rows, int32_t vocab, const float* temperature,
                                         const int32_t* tokens, int32_t n_given, float* logprob,
                                         int32_t* rank, float* entropy, float* lse, int32_t n_top,
                                         int32_t* top_id, float* top_logprob, uint32_t flags,
                                         int32_t* dev_err, kvd_stream_t stream) {
    if (dtype != KVD_F16 && dtype != KVD_BF16 && dtype != KVD_F32) return KVD_ERR_INVALID_ARG;
    if (rows < 0 || vocab <= 0 || row_stride < vocab || n_given < 0 || n_top < 0)
        return KVD_ERR_INVALID_ARG;
    if (n_given > KVD_MAX_GIVEN || n_top > KVD_MAX_TOP || vocab > KVD_MAX_VOCAB)
        return KVD_ERR_UNSUPPORTED;
    if (rows == 0) return KVD_OK;
    if (n_given > 0 && !tokens) return KVD_ERR_INVALID_ARG;
    const uintptr_t size = dtype == KVD_F32 ? 4 : 2;
    if (!logits || (reinterpret_cast<uintptr_t>(logits) & (size - 1))) return KVD_ERR_INVALID_ARG;
    if (rows > 0x7fffffff / kLpMaxCluster) return KVD_ERR_UNSUPPORTED;
    LogprobParams p = {};
    p.x = logits;
    p.stride = row_stride;
    p.rows = rows;
    p.vocab = vocab;
    p.temperature = temperature;
    p.tokens = tokens;
    p.given = n_given;
    p.logprob = logprob;
    p.rank = rank;
    p.entropy = entropy;
    p.lse = lse;
    p.top = top_id || top_logprob ? n_top : 0;
    p.top_id = top_id;
    p.top_logprob = top_logprob;
    p.dev_err = dev_err;
    p.test_stall = (flags & KVD_FLAG_TEST_STALL) ? 1 : 0;
    // split a row while the launch has few blocks and a block keeps half a round of logits
    int cluster = 1;
    while (2 * cluster <= kLpMaxCluster && (int64_t)rows * cluster * 2 <= kLpManyBlocks &&
           (vocab + 2 * cluster - 1) / (2 * cluster) >= kRound / 2)
        cluster *= 2;
    p.cluster = cluster;
    p.slice = (vocab + cluster - 1) / cluster;
    const bool pdl = (flags & KVD_FLAG_PDL) != 0;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KVD_F32) return run_type<float>(p, pdl, st);
    return dtype == KVD_F16 ? run_type<__half>(p, pdl, st) : run_type<__nv_bfloat16>(p, pdl, st);
}
