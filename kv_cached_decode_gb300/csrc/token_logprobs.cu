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
//    first block's shared memory. A block takes rounds of 4096 logits, 16 per thread, the next
//    round's loads in flight. The chunk's maximum decides once per 16 logits whether the running
//    maximum moves; sums are two-lane fp32.
//  * Ranks: a compare and an add per logit and token; ids below the token count equal logits, ids
//    above do not, so the threshold is set per vector of consecutive ids.
//  * Alternatives: an id is one 64-bit key (order of the logit, then lower id). After the first
//    round the n-th largest of 64 groups' maxima is a bound that at least n ids reach; from then
//    on only ids that reach it go to a list, one compare per 16 logits. When the list grows the
//    same step over its entries raises the bound, at least halving it whatever the order of the
//    row, and at the end it leaves at most 128, ranked by counting.
#include <algorithm>
#include <mutex>

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kPer = 16;                          // logits per thread and round
constexpr int kRound = kLpThreads * kPer;
constexpr int kListSoft = 1000;                   // entries from which the list is cut down
constexpr int kListCap = kListSoft + kRound + 32; // (a round adds kRound at most, the first 2 x 7)
constexpr int kGroups = 64;
constexpr int kRanked = 128;                      // entries ranked by counting
constexpr int kLpMaxCluster = 16;
constexpr float kFar = -3.402823466e38f;          // for the distance to a logit of -inf in weight *
                                                  // distance (0 * -inf is NaN)
// Blocks a launch should have before rows are no longer split.
constexpr int64_t kLpManyBlocks = 152 * 3;

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
};

// Sums of a part of a row: largest logit (-inf: none), how many have it, the others' weights
// relative to it and their sum of weight * distance.
struct Part {
    float m, n, rest, ent;
};
struct __align__(16) LpShared {
    Key list[kListCap];
    Key group[kLpThreads];
    Part part[kLpWarps];
    int32_t count[KVD_MAX_GIVEN];
    // of every CTA of the cluster, in the first one's: nothing else lies there, as the others
    // write it while the first may still be at its own slice
    Key ex_key[kLpMaxCluster * KVD_MAX_TOP];
    Part ex_part[kLpMaxCluster];
    int32_t ex_count[kLpMaxCluster][KVD_MAX_GIVEN];
    int32_t token[KVD_MAX_GIVEN];
    float value[KVD_MAX_GIVEN];                     // the tokens' logits
    int32_t place[kGroups];
    Key bound;
    int32_t n_list;
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
            const float d = x.m - r.m, f = exp2f(d * c), s = x.n + x.rest;
            if (f > 0.f) {
                r.rest = fmaf(s, f, r.rest);
                r.ent = fmaf(f, fmaf(d, s, x.ent), r.ent);
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

// One thread's chunk of a round joins its sums; cm: the chunk's largest, above -inf.
template <int N>
__device__ __forceinline__ void add_chunk(Part& a, const float (&x)[N], float cm, float c) {
    if (cm > a.m) {
        if (a.m > -INFINITY) {
            const float d = a.m - cm, f = exp2f(d * c), s = a.n + a.rest;
            a.rest = s * f;
            a.ent = f > 0.f ? f * fmaf(d, s, a.ent) : 0.f;
        }
        a.n = 0.f;
        a.m = cm;
    }
    if (cm == a.m) {  // (rarely: the row's maximum moves a few times per thread)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (x[i] == a.m) {
                a.n += 1.f;
            } else {
                const float d = x[i] - a.m, e = ex2_approx(d * c);
                a.rest += e;
                a.ent = fmaf(e, fmaxf(d, kFar), a.ent);
            }
        }
        return;
    }
    Pair r[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)}, t[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
    const Pair neg(-a.m, -a.m), cc(c, c);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const Pair dd = add2(Pair(x[i], x[i + 1]), neg);
        const float2 d = dd.get(), y = mul2(dd, cc).get();
        const Pair e(ex2_approx(y.x), ex2_approx(y.y));
        r[(i >> 1) & 1] = add2(r[(i >> 1) & 1], e);
        t[(i >> 1) & 1] =
            fma2(e, Pair(fmaxf(d.x, kFar), fmaxf(d.y, kFar)), t[(i >> 1) & 1]);
    }
    const float2 rs = add2(r[0], r[1]).get(), ts = add2(t[0], t[1]).get();
    a.rest += rs.x + rs.y;
    a.ent += ts.x + ts.y;
}

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
__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

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
    const int have = S.n_list;
    if (tid < n) out[tid] = 0;
    __syncthreads();
    if (tid < have) {
        const Key mine = S.list[tid];
        int above = 0;
        for (int i = 0; i < have; ++i) above += S.list[i] > mine;
        if (above < n) out[above] = mine;
    }
    __syncthreads();
}

__device__ __forceinline__ void push(LpShared& S, Key k) { S.list[atomicAdd(&S.n_list, 1)] = k; }

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

// GIVEN: 0 no ranks; 1 one token per row; 2 up to KVD_MAX_GIVEN.
template <typename T, int GIVEN>
__global__ void __launch_bounds__(kLpThreads, GIVEN == 2 ? 2 : 4)
    token_logprobs_kernel(const LogprobParams p) {
    extern __shared__ __align__(16) uint8_t lp_smem[];
    LpShared& S = *reinterpret_cast<LpShared*>(lp_smem);
    constexpr int VN = Vec<T>::n, NV = kPer / VN;
    constexpr int kTok = GIVEN == 2 ? KVD_MAX_GIVEN : 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)(blockIdx.x % (unsigned)p.cluster);
    const int row = (int)(blockIdx.x / (unsigned)p.cluster);
    if (p.cluster > 1) cluster_arrive_relaxed();
    pdl_wait();
    pdl_trigger();
    const T* x = static_cast<const T*>(p.x) + row * p.stride;
    const int lo = min(rank * p.slice, p.vocab), hi = min(lo + p.slice, p.vocab);
    // [lo, hi): up to VN - 1 logits, then whole 16-byte vectors, then up to VN - 1
    const int off = (int)((reinterpret_cast<uintptr_t>(x + lo) / sizeof(T)) % VN);
    const int body = min(hi, lo + (off ? VN - off : 0));
    const int vecs = (hi - body) / VN, tail = body + vecs * VN;
    uint4 buf[NV];
    auto fetch = [&](int r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = (r * NV + k) * kLpThreads + tid;
            if (v < vecs) buf[k] = load_stream(x + body + v * VN);
        }
    };
    fetch(0);
    const float T_ = p.temperature ? p.temperature[row] : 1.f;
    const bool bad_t = !(T_ > 0.f) || !(T_ < INFINITY);
    const float c = kLog2e / T_;
    if (tid < p.given) {
        const int t = p.tokens[(int64_t)row * p.given + tid];
        const bool in = t >= 0 && t < p.vocab;
        S.token[tid] = in ? t : -1;
        S.value[tid] = in ? fmaxf(Vec<T>::one(x[t]), -INFINITY) : 0.f;
        S.count[tid] = 0;
        if (!in && t != -1 && rank == 0) flag_error(p.dev_err, KVD_ERR_BAD_TOKEN);
    }
    if (tid == 0) S.n_list = 0;
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
        }
    }
    // before[i] += 1 for a logit v of id `id` ahead of token i
    auto count_one = [&](float v, int id) {
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (GIVEN && (GIVEN == 1 || i < p.given))
                cnt[i] += v > val[i] || (v == val[i] && id < tok[i]);
    };

    Part a = {-INFINITY, 0.f, 0.f, 0.f};
    bool nan = false;
    // the ends that are not whole vectors: one logit of a thread
    float end_v = -INFINITY;
    int end_id = 0;
    if (tid < body - lo) end_id = lo + tid;
    else if (tid >= 32 && tid - 32 < hi - tail) end_id = tail + tid - 32;
    else end_id = -1;
    if (end_id >= 0) {
        const float one[1] = {Vec<T>::one(x[end_id])};
        nan = one[0] != one[0];
        end_v = fmaxf(one[0], -INFINITY);
        if (end_v > -INFINITY) {
            a.m = end_v;
            a.n = 1.f;
        }
        if (GIVEN) count_one(end_v, end_id);
    }

    const int rounds = max(1, (vecs + NV * kLpThreads - 1) / (NV * kLpThreads));
    float bound_v = -INFINITY;  // of S.bound
    for (int r = 0; r < rounds; ++r) {
        float v[kPer];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            Vec<T>::get(buf[k], v + k * VN);
            if ((r * NV + k) * kLpThreads + tid >= vecs) {
#pragma unroll
                for (int i = 0; i < VN; ++i) v[k * VN + i] = -INFINITY;
            }
        }
        if (r + 1 < rounds) fetch(r + 1);
        auto id_of = [&](int i) {
            return body + ((r * NV + i / VN) * kLpThreads + tid) * VN + i % VN;
        };
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
        if (cm > -INFINITY) add_chunk(a, v, cm, c);
        if (GIVEN) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int id0 = id_of(k * VN);
                if (id0 >= tail) break;
#pragma unroll
                for (int i = 0; i < kTok; ++i) {
                    if (GIVEN == 2 && i >= p.given) break;
                    // ids below the token's count equal logits
                    const float at = id0 < tok[i] ? val[i] : val_up[i];
                    if (tok[i] - id0 < VN && tok[i] > id0) {
#pragma unroll
                        for (int e = 0; e < VN; ++e)
                            cnt[i] += v[k * VN + e] > val[i] ||
                                      (v[k * VN + e] == val[i] && id0 + e < tok[i]);
                    } else {
#pragma unroll
                        for (int e = 0; e < VN; ++e) cnt[i] += v[k * VN + e] >= at;
                    }
                }
            }
        }
        if (p.top > 0) {
            if (r == 0) {
                // a bound that at least `top` ids of the round reach
                Key best = end_v > -INFINITY ? make_key(end_v, end_id) : 0;
                if (cm > -INFINITY) {
                    int id = 0;
#pragma unroll
                    for (int i = kPer - 1; i >= 0; --i)
                        if (v[i] == cm) id = id_of(i);
                    best = max(best, make_key(cm, id));
                }
                S.group[tid] = best;
                set_bound(S, p.top);
                const Key bound = S.bound;
                bound_v = bound == 1 ? -INFINITY : key_value(bound);
                if (end_v > -INFINITY && make_key(end_v, end_id) >= bound)
                    push(S, make_key(end_v, end_id));
            }
            if (cm >= bound_v && cm > -INFINITY) {
                const Key bound = S.bound;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (v[i] >= bound_v && v[i] > -INFINITY) {
                        const Key k = make_key(v[i], id_of(i));
                        if (k >= bound) push(S, k);
                    }
            }
            if (r + 1 < rounds) {
                __syncthreads();
                if (S.n_list > kListSoft) {  // uniform: nobody adds before the next barrier
                    while (S.n_list > kListSoft / 4) cut_list(S, p.top);
                    const Key bound = S.bound;
                    bound_v = bound == 1 ? -INFINITY : key_value(bound);
                }
                __syncthreads();
            }
        }
    }

    // ---- the block's sums and counts ----
    if (nan) flag_error(p.dev_err, KVD_ERR_NAN);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = join(a, shfl_part(a, o), c);
    if (lane == 0) S.part[warp] = a;
    if (GIVEN) {
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (GIVEN == 2 && i >= p.given) break;
            const int n = __reduce_add_sync(0xffffffffu, cnt[i]);
            if (lane == 0) atomicAdd(&S.count[i], n);
        }
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll 1
        for (int w = 1; w < kLpWarps; ++w) a = join(a, S.part[w], c);
    }
    // ---- the cluster's, in its first block ----
    Key* best = S.group;  // [top]
    if (p.top > 0) rank_list(S, p.top, best);
    if (p.cluster > 1) {
        cluster_wait();  // every block has started: its shared memory can be written
        if (tid < p.top) st_cluster_key(&S.ex_key[rank * p.top + tid], 0, best[tid]);
        if (tid == 0) {
            st_cluster_word(&S.ex_part[rank].m, 0, __float_as_uint(a.m));
            st_cluster_word(&S.ex_part[rank].n, 0, __float_as_uint(a.n));
            st_cluster_word(&S.ex_part[rank].rest, 0, __float_as_uint(a.rest));
            st_cluster_word(&S.ex_part[rank].ent, 0, __float_as_uint(a.ent));
        }
        if (GIVEN && tid < p.given)
            st_cluster_word(&S.ex_count[rank][tid], 0, (uint32_t)S.count[tid]);
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank != 0) return;
        if (tid == 0) {
            a = S.ex_part[0];
#pragma unroll 1
            for (int k = 1; k < p.cluster; ++k) a = join(a, S.ex_part[k], c);
            S.n_list = p.cluster * p.top;
        }
        if (GIVEN && tid < p.given) {
            int n = 0;
            for (int k = 0; k < p.cluster; ++k) n += S.ex_count[k][tid];
            S.count[tid] = n;
        }
        for (int i = tid; i < p.cluster * p.top; i += kLpThreads) S.list[i] = S.ex_key[i];
        __syncthreads();
        if (p.top > 0) rank_list(S, p.top, best);
    }
    if (bad_t) {
        if (tid == 0) flag_error(p.dev_err, KVD_ERR_BAD_PARAM);
        return;
    }
    // ---- the outputs ----
    __syncthreads();
    if (tid == 0) S.part[0] = a;
    __syncthreads();
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
            p.entropy[row] = none ? 0.f : log_s - a.ent / T_ / (a.n + a.rest);
    }
}

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
                                       (int)sizeof(LpShared)) == cudaSuccess &&
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
                     sizeof(LpShared), st, pdl, (unsigned)p.cluster, p);
}
template <typename T>
kvd_status run_type(const LogprobParams& p, bool pdl, cudaStream_t st) {
    if (!p.rank || p.given == 0) return run<T, 0>(p, pdl, st);
    return p.given == 1 ? run<T, 1>(p, pdl, st) : run<T, 2>(p, pdl, st);
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
    // split a row while the launch has few blocks and a block keeps a round of logits at least
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
