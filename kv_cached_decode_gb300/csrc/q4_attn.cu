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
//    one AND per two values instead of a conversion. Exact: the tensor cores take
//    subnormals, q is scaled by a power of two per row, the powers are undone in fp32.
//  * A byte holds consecutive dims. The contraction order of q.K is free, so lane c of a
//    quad takes dims 16c..16c+15 of a K row (8 consecutive bytes) and q is loaded in the
//    same order; in P.V the n-block of an output column is free, so lane g takes word g of
//    a V row, dims 8g..8g+7, one per n-block. Columns 2c and 2c+1 of a score fragment are
//    rows c and c+4, which keeps both reads free of bank conflicts. Pairs of positions for
//    the V operand are two words merged with PRMT.
//  * The weights that multiply V are fp16(w * sV / 2^E), E a per-warp exponent that follows
//    the largest step; the zero points are one more n-block of the same product, so the same
//    rounded weights multiply n and z and their rounding is not amplified by n - z
//    cancelling. The normaliser sums w unrounded in fp32.
//  * Rows' references move only when a score exceeds them by 2^8, decided by one vote per
//    tile: the usual tile has no reduction across lanes at all.
//  * Each warp streams its own tiles of 32 positions (2304 bytes with the parameters)
//    through a ring of cp.async stages: no block barrier in the loop, and rows at or past
//    the length are filled with zeros and never read.
//  * A (row, KV head, block of <= 16 query vectors) unit is cut into splits of equal tile
//    counts of the row's own length. Splits of a unit form a thread-block cluster and merge
//    through distributed shared memory, every CTA a share of the outputs; for a few long
//    units, more splits than a cluster holds merge through the workspace (last arrival).
#include <algorithm>
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
constexpr int kMaxSplitsQ = 128;
constexpr float kGrowLog2 = 8.f;
constexpr int kPart = kHeadDim + 4;          // floats per partial: o[64], max, sum, 2 pad

struct Q4AttnParams {
    const void* q;
    void* out;
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* par;
    int64_t sb, sh;          // rows
    const int32_t* lens;
    int32_t fixed_len, capacity;
    int32_t n_q_heads, n_kv_heads, group, qlen;
    int32_t M, msub, nsub;   // query vectors per (row, KV head), per block; blocks
    int32_t splits, cluster; // splits per unit; 1: they form a cluster, 0: workspace
    int32_t causal, window, n_sinks;
    float scale_log2;
    float* ws_part;          // [units][splits][msub][kPart]
    int32_t* ws_cnt;
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
__device__ __forceinline__ float half_bits(uint32_t b) {
    return __half2float(__ushort_as_half((uint16_t)b));
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    return Half16<__half>::from_f2(a, b);
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

template <typename T, int RM>
__global__ void __launch_bounds__(kThreadsQ, 2) q4_attn_kernel(const Q4AttnParams p) {
    constexpr bool kFull = RM == 16;
    constexpr int kAcc = kFull ? 4 : 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int s = blockIdx.x, h = blockIdx.y / p.nsub, sub = blockIdx.y % p.nsub, b = blockIdx.z;
    const int m0 = sub * p.msub, mcount = min(p.msub, p.M - m0);

    pdl_wait();
    pdl_trigger();
    const int len = p.lens ? p.lens[b] : p.fixed_len;
    const bool bad = len < 0 || len > p.capacity;  // the same in every CTA of a cluster
    if (bad) {
        if (tid == 0 && s == 0 && blockIdx.y == 0) flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
        return;
    }
    const TileMap tm = tile_map(p, len);
    const int v0 = (int)((int64_t)tm.total * s / p.splits);
    const int v1 = (int)((int64_t)tm.total * (s + 1) / p.splits);

    // ---- the warp's ring ----
    uint8_t* ring = smem + warp * (kStagesQ * kStageBytes);
    const int64_t row0 = b * p.sb + h * p.sh;
    const uint8_t* kbase = p.k + row0 * 32;
    const uint8_t* vbase = p.v + row0 * 32;
    const uint8_t* pbase = p.par + row0 * 8;
    auto fetch = [&](int v, int stage) {
        if (v < v1) {
            const int t0 = tm.pos(v);
            const uint32_t dst = smem_u32(ring + stage * kStageBytes);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = lane + 32 * i;
                const bool on = t0 + (x >> 1) < len;
                const int64_t off = on ? (int64_t)t0 * 32 + x * 16 : 0;
                cp_async16_zfill(dst + x * 16, kbase + off, on);
                cp_async16_zfill(dst + kT * 32 + x * 16, vbase + off, on);
            }
            const bool on = t0 + lane < len;
            cp_async8_zfill(dst + kT * 64 + lane * 8, pbase + (on ? (int64_t)(t0 + lane) * 8 : 0),
                            on);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStagesQ - 1; ++i) fetch(v0 + warp + i * kWarpsQ, i);

    // ---- the query rows g (A) and g + 8 (B) of the block: 16 dims per lane ----
    // fp16, scaled by 2^e so that a row's largest value lies in [2^14, 2^15)
    uint32_t qa[4][4];
    float rs[2], qs[2];  // score factor (log2 units) and sum of the scaled q, * 2^-24
    int lim[2], wlo[2];  // the row sees t < lim with t >= wlo or t < n_sinks
#pragma unroll
    for (int r = 0; r < (kFull ? 2 : 1); ++r) {
        const int m = g + 8 * r;
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.f;
        lim[r] = 0;
        wlo[r] = 0;
        if (m < mcount) {
            const int i = (m0 + m) % p.qlen, hq = h * p.group + (m0 + m) / p.qlen;
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(p.q) +
                (((int64_t)b * p.n_q_heads + hq) * p.qlen + i) * kHeadDim + 16 * c);
            unpack8<T>(src[0], x);
            unpack8<T>(src[1], x + 8);
            const int pos = len - p.qlen + i;
            lim[r] = p.causal ? max(pos + 1, 0) : len;
            if (p.window > 0) wlo[r] = (int)max((int64_t)pos - p.window + 1, (int64_t)0);
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
        const bool any_odd = ((__ballot_sync(0xffffffffu, odd) >> (lane & 28)) & 15u) != 0;
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
        qs[r] = sum * 0x1p-24f;
        rs[r] = ldexpf(fabsf(p.scale_log2), 24 - e2);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                // nibbles n and n + 4 of word kk / 2; the odd ones come times 16
                const int n = 8 * (kk >> 1) + 2 * (kk & 1) + w;
                const float f = w ? 0.0625f : 1.f;
                qa[kk][2 * w + r] = pack_half(x[n] * f, x[n + 4] * f);
            }
    }
    if (!kFull) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) qa[kk][1] = qa[kk][3] = 0u;
        rs[1] = qs[1] = 0.f;
        lim[1] = wlo[1] = 0;
    }
    auto mma = [&](float* acc, const uint32_t* a, uint32_t b0, uint32_t b1) {
        if (kFull) Mma<__half>::run(acc, a, b0, b1);
        else Mma<__half>::run_top(acc, a[0], a[2], b0, b1);
    };

    float acc[9][kAcc];  // n-blocks 0..7: the output dims; 8: the zero points
#pragma unroll
    for (int n = 0; n < 9; ++n)
#pragma unroll
        for (int e = 0; e < kAcc; ++e) acc[n][e] = 0.f;
    float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float vref = 0.f, vinv = 0.f;  // 2^E and 2^-E of the V steps (0: none seen yet)

    // positions every row of the block sees wholly: t < seen_hi, and with a window
    // t >= seen_lo or t < n_sinks
    const int seen_hi = p.causal ? len - p.qlen + 1 : len;
    const int seen_lo = p.window > 0 ? (int)max((int64_t)len - p.window, (int64_t)0) : 0;

    auto tile = [&](const uint8_t* st, int t0, auto masked_) {
        constexpr bool kMasked = decltype(masked_)::value;
        const uint8_t* sK = st;
        const uint8_t* sV = st + kT * 32;
        const uint2* sP = reinterpret_cast<const uint2*>(st + kT * 64);
        // the lane's positions: 8 nb + 4 e + c, nb 0..3, e 0..1
        float sc[4][kAcc];
        const int krow = (g >> 1) + 4 * (g & 1);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
            for (int e = 0; e < kAcc; ++e) sc[nb][e] = 0.f;
            const uint2 w = *reinterpret_cast<const uint2*>(sK + (8 * nb + krow) * 32 + c * 8);
            mma(sc[nb], qa[0], w.x & 0x000F000Fu, w.x & 0x00F000F0u);
            mma(sc[nb], qa[1], (w.x >> 8) & 0x000F000Fu, (w.x >> 8) & 0x00F000F0u);
            mma(sc[nb], qa[2], w.y & 0x000F000Fu, w.y & 0x00F000F0u);
            mma(sc[nb], qa[3], (w.y >> 8) & 0x000F000Fu, (w.y >> 8) & 0x00F000F0u);
        }
        float vs[4][2];     // V steps of the lane's positions
        uint32_t vz[4];     // zero points of V: pair (row c, row c + 4)
        float top[2] = {-INFINITY, -INFINITY}, vtop = 0.f;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            uint2 pr[2] = {sP[8 * nb + c], sP[8 * nb + 4 + c]};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (kMasked) {
                    // an infinite zero point must not reach rows that do not see it
                    if (((pr[e].y >> 16) & 0x7C00u) == 0x7C00u) pr[e].y = 0x7FC0u;
                }
                const float ks = __uint_as_float(pr[e].x << 16), kz = half_bits(pr[e].x >> 16);
                vs[nb][e] = __uint_as_float(pr[e].y << 16);
                vtop = fmaxf(vtop, vs[nb][e] < INFINITY ? vs[nb][e] : 0.f);
#pragma unroll
                for (int r = 0; r < kAcc / 2; ++r) {
                    float x = fmaf(-kz, qs[r], sc[nb][2 * r + e]) * ks;
                    if (kMasked) {
                        const int t = t0 + 8 * nb + 4 * e + c;
                        if (!(t < lim[r] && (t >= wlo[r] || t < p.n_sinks))) x = -INFINITY;
                    }
                    sc[nb][2 * r + e] = x;
                    top[r] = fmaxf(top[r], x);
                }
            }
            vz[nb] = __byte_perm(pr[0].y, pr[1].y, 0x7632);
        }
        // One vote: does a row's reference or the step exponent have to move?
        bool move = vtop > 16.f * vref;
#pragma unroll
        for (int r = 0; r < kAcc / 2; ++r) move |= top[r] * rs[r] > ref[r] + kGrowLog2;
        if (__any_sync(0xffffffffu, move)) {
            const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(vtop));
            float fv = 1.f;
            if (__uint_as_float(vb) > vref) {
                // 2^E: the largest step's power of two (at least the smallest normal)
                const float nv = __uint_as_float(max(vb & 0x7F800000u, 0x00800000u));
                fv = vref * (1.f / nv);
                vref = nv;
                vinv = 1.f / nv;
            }
#pragma unroll
            for (int r = 0; r < kAcc / 2; ++r) {
                float t = top[r];
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                t = t == -INFINITY ? t : t * rs[r];
                const float nref = fmaxf(ref[r], t);
                const float f = nref == -INFINITY ? 1.f : exp2f(ref[r] - nref);
                ref[r] = nref;
                l[r] *= f;
#pragma unroll
                for (int n = 0; n < 9; ++n) {
                    acc[n][2 * r] *= f * fv;
                    acc[n][2 * r + 1] *= f * fv;
                }
            }
        }
        // weights, in pairs of positions (row c, row c + 4) of each n-block
        uint32_t pw[4][2];
        const float nr[2] = {ref[0] == -INFINITY ? 0.f : -ref[0],
                             ref[1] == -INFINITY ? 0.f : -ref[1]};
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float y[2] = {vs[nb][0] * vinv, vs[nb][1] * vinv};
#pragma unroll
            for (int r = 0; r < kAcc / 2; ++r) {
                float w[2], f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = sc[nb][2 * r + e];
                    w[e] = ex2_approx(fmaf(x, rs[r], nr[r]));
                    f[e] = w[e] * y[e];
                    if (kMasked && x == -INFINITY) w[e] = f[e] = 0.f;
                }
                l[r] += w[0] + w[1];
                pw[nb][r] = pack_half(f[0], f[1]);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t pa[4] = {pw[2 * half][0], 0u, pw[2 * half + 1][0], 0u};
            if (kFull) {
                pa[1] = pw[2 * half][1];
                pa[3] = pw[2 * half + 1][1];
            }
            const uint8_t* vr = sV + (16 * half + c) * 32 + g * 4;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint32_t*>(vr + j * 128);
            const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), b0 = __byte_perm(w[2], w[3], 0x5410);
            const uint32_t a1 = __byte_perm(w[0], w[1], 0x7632), b1 = __byte_perm(w[2], w[3], 0x7632);
            mma(acc[0], pa, a0 & 0x000F000Fu, b0 & 0x000F000Fu);
            mma(acc[1], pa, a0 & 0x00F000F0u, b0 & 0x00F000F0u);
            mma(acc[2], pa, (a0 >> 8) & 0x000F000Fu, (b0 >> 8) & 0x000F000Fu);
            mma(acc[3], pa, (a0 >> 8) & 0x00F000F0u, (b0 >> 8) & 0x00F000F0u);
            mma(acc[4], pa, a1 & 0x000F000Fu, b1 & 0x000F000Fu);
            mma(acc[5], pa, a1 & 0x00F000F0u, b1 & 0x00F000F0u);
            mma(acc[6], pa, (a1 >> 8) & 0x000F000Fu, (b1 >> 8) & 0x000F000Fu);
            mma(acc[7], pa, (a1 >> 8) & 0x00F000F0u, (b1 >> 8) & 0x00F000F0u);
            mma(acc[8], pa, vz[2 * half], vz[2 * half + 1]);
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

    // ---- merge the warps: red[warp][row][kPart] over the ring ----
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int r = 0; r < kAcc / 2; ++r) {
        float t = l[r];
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        const int m = g + 8 * r;
        if (m < mcount) {
            float* o = red + (warp * RM + m) * kPart;
            // columns 2c, 2c + 1 are dims 16c + n and 16c + 8 + n; the odd n-blocks are
            // times 16
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float z = acc[8][2 * r + e];
                float x[8];
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    x[n] = fmaf(acc[n][2 * r + e], n & 1 ? 0x1p20f : 0x1p24f, -z) * vref;
                float4* d = reinterpret_cast<float4*>(o + 16 * c + 8 * e);
                d[0] = make_float4(x[0], x[1], x[2], x[3]);
                d[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
            if (c == 0) {
                o[kHeadDim] = ref[r];
                o[kHeadDim + 1] = t;
            }
        }
    }
    __syncthreads();
    const int items = mcount * (kHeadDim / 4);  // (query vector, 4 dims)
    float* part = red + kWarpsQ * RM * kPart;   // this CTA's partial [msub][kPart]
    auto store = [&](int it, const float4& o, float sum) {
        const int m = it >> 4, d = (it & 15) * 4;
        const int i = (m0 + m) % p.qlen, hq = h * p.group + (m0 + m) / p.qlen;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint2 w;
        w.x = Half16<T>::from_f2(o.x * inv, o.y * inv);
        w.y = Half16<T>::from_f2(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) +
                                  (((int64_t)b * p.n_q_heads + hq) * p.qlen + i) * kHeadDim + d) = w;
    };
    const int unit = (b * p.n_kv_heads + h) * p.nsub + sub;
    float* wp = p.splits > 1 && !p.cluster
                    ? p.ws_part + ((int64_t)unit * p.splits + s) * p.msub * kPart
                    : nullptr;
    for (int it = tid; it < items; it += kThreadsQ) {
        const float* r0 = red + (it >> 4) * kPart;
        const int q4 = it & 15;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarpsQ; ++w) mx = fmaxf(mx, r0[w * RM * kPart + kHeadDim]);
        const float rf = mx == -INFINITY ? 0.f : mx;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarpsQ; ++w) {
            const float* pw = r0 + w * RM * kPart;
            const float a = exp2f(pw[kHeadDim] - rf);
            const float4 x = reinterpret_cast<const float4*>(pw)[q4];
            sum = fmaf(pw[kHeadDim + 1], a, sum);
            o.x = fmaf(x.x, a, o.x);
            o.y = fmaf(x.y, a, o.y);
            o.z = fmaf(x.z, a, o.z);
            o.w = fmaf(x.w, a, o.w);
        }
        if (p.splits == 1) {
            store(it, o, sum);
        } else {
            float* d = (wp ? wp : part) + (it >> 4) * kPart;
            reinterpret_cast<float4*>(d)[q4] = o;
            if (q4 == 0) *reinterpret_cast<float4*>(d + kHeadDim) = make_float4(mx, sum, 0.f, 0.f);
        }
    }
    if (p.splits == 1) return;

    if (p.cluster) {
        // every CTA merges a share of the outputs out of all CTAs' partials, in split order
        cluster_sync_q4();
        const uint32_t base = smem_u32(part);
        for (int it = s + p.splits * tid; it < items; it += p.splits * kThreadsQ) {
            const uint32_t off = base + (it >> 4) * (kPart * 4);
            float mx = -INFINITY;
            for (int i = 0; i < p.splits; ++i)
                mx = fmaxf(mx, ld_cluster4(map_shared(off + kHeadDim * 4, i)).x);
            const float rf = mx == -INFINITY ? 0.f : mx;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll 4
            for (int i = 0; i < p.splits; ++i) {
                const float4 ml = ld_cluster4(map_shared(off + kHeadDim * 4, i));
                const float4 x = ld_cluster4(map_shared(off + (it & 15) * 16, i));
                const float a = exp2f(ml.x - rf);
                sum = fmaf(ml.y, a, sum);
                o.x = fmaf(x.x, a, o.x);
                o.y = fmaf(x.y, a, o.y);
                o.z = fmaf(x.z, a, o.z);
                o.w = fmaf(x.w, a, o.w);
            }
            store(it, o, sum);
        }
        cluster_sync_q4();  // no CTA leaves while another may still read its partial
        return;
    }

    // ---- the last split of the unit to arrive merges all of them, in split order ----
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(&p.ws_cnt[unit], 1) == p.splits - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const float* up = p.ws_part + (int64_t)unit * p.splits * p.msub * kPart;
    float* wt = red;  // the splits' maxima, [mcount][splits]
    for (int x = tid; x < mcount * p.splits; x += kThreadsQ)
        wt[x] = __ldcg(up + ((int64_t)(x % p.splits) * p.msub + x / p.splits) * kPart + kHeadDim);
    __syncthreads();
    for (int it = tid; it < items; it += kThreadsQ) {
        const int m = it >> 4, q4 = it & 15;
        float mx = -INFINITY;
        for (int i = 0; i < p.splits; ++i) mx = fmaxf(mx, wt[m * p.splits + i]);
        const float rf = mx == -INFINITY ? 0.f : mx;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 8
        for (int i = 0; i < p.splits; ++i) {
            const float* src = up + ((int64_t)i * p.msub + m) * kPart;
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src) + q4);
            const float li = __ldcg(src + kHeadDim + 1);
            const float a = exp2f(wt[m * p.splits + i] - rf);
            sum = fmaf(li, a, sum);
            o.x = fmaf(x.x, a, o.x);
            o.y = fmaf(x.y, a, o.y);
            o.z = fmaf(x.z, a, o.z);
            o.w = fmaf(x.w, a, o.w);
        }
        store(it, o, sum);
    }
    if (tid == 0) p.ws_cnt[unit] = 0;
}

// Ring of all warps, reused for the warps' partials; the CTA's partial follows them.
constexpr uint32_t q4_smem(int rm) {
    const uint32_t ring = kWarpsQ * kStagesQ * kStageBytes;
    const uint32_t red = (kWarpsQ + 1) * rm * kPart * 4;
    return ring > red ? ring : red;
}
// the workspace merge's maxima [rm][kMaxSplitsQ] reuse the same bytes
static_assert(16 * kMaxSplitsQ * 4 <= q4_smem(16) && 8 * kMaxSplitsQ * 4 <= q4_smem(8), "maxima");

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

// Blocks (cluster == 1) or clusters of `cluster` blocks resident at once on the device.
template <auto Kern>
int resident_q4(size_t smem, int cluster, int nsm) {
    static std::mutex mu;
    static int cache[kMaxDevQ][kMaxClusterQ + 1];  // value + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevQ) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int& v = cache[dev][cluster];
    if (v) return v - 1;
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
    v = n + 1;
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

// A workspace merge is considered for at most this many units, when a cluster's CTAs would
// each read more than this many tiles per warp.
constexpr int kWsUnitsQ = 8;
constexpr int kWsTilesQ = 4;
bool q4_ws_pays(int64_t units, int64_t tiles) {
    return units <= kWsUnitsQ && tiles > (int64_t)kMaxClusterQ * kWarpsQ * kWsTilesQ;
}

template <typename T, int RM>
kvd_status run_q4(Q4AttnParams& p, const Q4Shape& sh, int batch, int64_t tiles, int nsm,
                  void* ws, size_t ws_bytes, bool pdl, cudaStream_t st) {
    constexpr auto kern = q4_attn_kernel<T, RM>;
    constexpr size_t smem = q4_smem(RM);
    const int mc = prepare_q4<kern>(smem);
    if (mc <= 0) return KVD_ERR_CUDA;
    const int64_t most = std::max<int64_t>(1, (tiles + kWarpsQ - 1) / kWarpsQ);
    const int64_t slots = resident_q4<kern>(smem, 1, nsm);
    p.splits = 1;
    p.cluster = 0;
    if (q4_ws_pays(sh.units, tiles)) {
        p.splits =
            (int)std::min<int64_t>({most, kMaxSplitsQ, std::max<int64_t>(1, slots / sh.units)});
    } else {
        int64_t want = std::min<int64_t>(most, mc);
        for (; want > 1; --want)
            if (resident_q4<kern>(smem, (int)want, nsm) >= sh.units) break;
        p.splits = (int)std::max<int64_t>(1, want);
        p.cluster = p.splits > 1;
    }
    if (p.splits > 1 && !p.cluster) {
        const size_t need = KVD_WS_COUNTER_BYTES +
                            (size_t)sh.units * p.splits * sh.msub * kPart * sizeof(float);
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < need)
            return KVD_ERR_WORKSPACE;
        p.ws_cnt = static_cast<int32_t*>(ws);
        p.ws_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + KVD_WS_COUNTER_BYTES);
    }
    const dim3 grid((unsigned)p.splits, (unsigned)(p.n_kv_heads * sh.nsub), (unsigned)batch);
    return launch_ex(kern, grid, dim3(kThreadsQ), smem, st, pdl,
                     p.cluster ? (unsigned)p.splits : 1u, p);
}

}  // namespace

size_t q4_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int qlen, int max_len) {
    const Q4Shape sh = q4_shape(batch, n_q_heads, n_kv_heads, qlen);
    const int64_t tiles = q4_tiles(max_len, qlen, 0, 0);
    if (!q4_ws_pays(sh.units, tiles)) return KVD_WS_COUNTER_BYTES;
    const size_t part = (size_t)sh.units * kMaxSplitsQ * sh.msub * kPart * sizeof(float);
    return KVD_WS_COUNTER_BYTES + (part + 255) / 256 * 256;
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
    if (!q || !out || !aligned16(q) || !aligned16(out)) return KVD_ERR_INVALID_ARG;
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
    if (dtype == KVD_BF16)
        return sh.msub <= 8 ? run_q4<__nv_bfloat16, 8>(p, sh, batch, tiles, nsm, workspace,
                                                       workspace_bytes, pdl, st)
                            : run_q4<__nv_bfloat16, 16>(p, sh, batch, tiles, nsm, workspace,
                                                        workspace_bytes, pdl, st);
    return sh.msub <= 8 ? run_q4<__half, 8>(p, sh, batch, tiles, nsm, workspace, workspace_bytes,
                                            pdl, st)
                        : run_q4<__half, 16>(p, sh, batch, tiles, nsm, workspace,
                                             workspace_bytes, pdl, st);
}
