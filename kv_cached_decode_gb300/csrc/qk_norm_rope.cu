// qk_norm_rope.cu -- RMS norm of every query and key head and the position rotation, in
// one pass.
//
// No counterpart on the pages: decoder-only models that normalise queries and keys per
// head do it between the QKV projection and the attention. For a head row x of 64 values
// at position p (w: the head norm's weight, 1 without one):
//   y = x * w / sqrt(sum(x^2) / 64 + eps)
//   out[i] = y[i] cos a - y[i+32] sin a,  out[i+32] = y[i+32] cos a + y[i] sin a,
//   a = p * base^(-i/32), i < 32
// all in fp32, rounded to the storage type once, at the end. The input is read in place
// from the projection's output (any strides); the output has the [batch, heads, n, 64]
// layout of the attention calls.
//
// The angle. p * theta rounded to fp32 is off by up to p * theta * 2^-24 radians, 4e-3 at
// p = 65536: more than a 16-bit rounding. Here the host gives theta / 2 pi modulo 1 as a
// 64-bit fixed-point fraction of a turn; p times it, modulo 2^64, is the angle in turns
// with the whole turns already dropped, exact to p * 2^-53. Its top 32 bits go to
// sincospif. One 64-bit integer multiply instead of a long argument reduction.
//
// Design. Bound by HBM (each row read and written once, 256 bytes) when there are many
// rows, by the launch when there are few. Four lanes own a row (lane l: dims 8l..8l+7 and
// 32+8l..32+8l+7, i.e. whole rotation pairs), so the sum of squares takes two shuffles and
// a warp covers eight heads of one token. Each lane computes one of the token's 32 cos/sin
// pairs and gets its eight by shuffles; multiplied with the weights they become the four
// coefficients of each pair, used for every further group of eight heads the warp takes:
//   out[i] = inv (x[i] w[i] cos - x[i+32] w[i+32] sin), out[i+32] likewise
// at three operations a value. A warp takes more than one group only while the launch still
// has many warps; the loads of four groups are in flight at a time, and as soon as one is stored
// the next is loaded.
//
// Measured: 4 x 4096 tokens x 40 heads of fp16, 168 MB, 30.5 us, 5.5 TB/s (a plain copy of as many
// bytes takes 26 us, a transposing one 104 us); 16 tokens 2.6 us. Eight sincospi per lane and
// weights applied per row were 359 instructions per eight heads, bound by their issue; now the
// loads in flight bound it: cos and sin kept in registers, pointers kept with the data and batches
// of loads instead of the rolling ones 34.4; two, three or five groups ahead 30.4 to 32.3 with the
// registers cut to fit, 31.2 and more without; four tokens per warp 44.5.
#include <cmath>
#include <cstring>

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {
namespace {

constexpr int kNrThreads = 128;
// Warps a launch should have before a warp takes more than one group of heads: 152
// SMs x 16 warps keep enough 16-byte loads in flight.
constexpr int64_t kNrManyWarps = 152 * 16;
constexpr int kAhead = 4;  // groups of heads whose loads a warp has in flight

struct NormRopeParams {
    const uint8_t* x[2];   // q, k
    uint8_t* y[2];
    const uint8_t* w[2];   // [64] of the storage type, or null
    int64_t sb[2], sh[2], st[2];  // input strides, bytes
    int32_t heads[2];
    const int32_t* pos0;   // [batch] or null
    int32_t n;
    uint32_t tokens, hgroups, iters;  // tokens; warps per token; groups of 8 heads per warp
    int32_t rotate;
    float eps;
    uint64_t freq[32];     // base^(-i/32) / (2 pi) modulo 1, in units of 2^-64 turns
};

// The coefficients of this lane's eight pairs: w[i] cos, w[i+32] sin, w[i+32] cos, w[i] sin; lane i
// of the warp has the cos and sin of pair i in `mine`.
struct Coef {
    float a[8], b[8], c[8], d[8];
};
template <typename T>
__device__ __forceinline__ void make_coef(Coef& k, float2 mine, const uint8_t* w, int l) {
    float wa[8], wb[8];
    if (w) {
        unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w) + l), wa);
        unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w) + 4 + l), wb);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float cos = __shfl_sync(0xffffffffu, mine.x, 8 * l + e);
        const float sin = __shfl_sync(0xffffffffu, mine.y, 8 * l + e);
        k.a[e] = wa[e] * cos;
        k.b[e] = wb[e] * sin;
        k.c[e] = wb[e] * cos;
        k.d[e] = wa[e] * sin;
    }
}

// One row's 16 values of this lane: norm, weight, rotation, rounding.
template <typename T>
__device__ __forceinline__ void norm_rotate(uint4& lo, uint4& hi, const Coef& k, float eps) {
    float x[8], y[8];
    unpack8<T>(lo, x);
    unpack8<T>(hi, y);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    const float inv = rsqrtf(ss * (1.f / 64.f) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float u = fmaf(x[e], k.a[e], -(y[e] * k.b[e])) * inv;
        const float v = fmaf(y[e], k.c[e], x[e] * k.d[e]) * inv;
        x[e] = u;
        y[e] = v;
    }
    uint32_t* pl = reinterpret_cast<uint32_t*>(&lo);
    uint32_t* ph = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        pl[e] = Half16<T>::from_f2(x[2 * e], x[2 * e + 1]);
        ph[e] = Half16<T>::from_f2(y[2 * e], y[2 * e + 1]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kNrThreads, 5) qk_norm_rope_kernel(const NormRopeParams p) {
    __shared__ uint64_t s_freq[32];
    if (threadIdx.x < 32) s_freq[threadIdx.x] = p.freq[threadIdx.x];
    pdl_wait();
    __syncthreads();
    const uint32_t wid = blockIdx.x * (kNrThreads / 32) + (threadIdx.x >> 5);
    const uint32_t token = wid / p.hgroups, hg = wid % p.hgroups;
    const int b = (int)(token / (uint32_t)p.n), j = (int)(token % (uint32_t)p.n);
    const int lane = threadIdx.x & 31, l = lane & 3;
    const int total = p.heads[0] + p.heads[1];
    // this lane's row of group `it` of the token
    struct Item {
        uint4 lo, hi;
    };
    auto head = [&](uint32_t it) { return (int)(hg * p.iters + it) * 8 + (lane >> 2); };
    auto load = [&](uint32_t it) {
        Item r;
        r.lo = r.hi = make_uint4(0u, 0u, 0u, 0u);
        const int h0 = head(it);
        if (it < p.iters && h0 < total) {
            // (selects: an index known only at run time would put the parameters on the stack)
            const bool k = h0 >= p.heads[0];
            const int h = k ? h0 - p.heads[0] : h0;
            const uint8_t* src = (k ? p.x[1] : p.x[0]) + b * (k ? p.sb[1] : p.sb[0]) +
                                 h * (k ? p.sh[1] : p.sh[0]) + j * (k ? p.st[1] : p.st[0]);
            r.lo = *reinterpret_cast<const uint4*>(src + l * 16);
            r.hi = *reinterpret_cast<const uint4*>(src + 64 + l * 16);
        }
        return r;
    };
    if (token < p.tokens) {  // warp-uniform
        // kAhead groups' loads in flight, the first ones before the token's cos/sin
        Item item[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) item[u] = load(u);
        // cos/sin of pair `lane`
        float2 mine = make_float2(1.f, 0.f);
        if (p.rotate) {
            const int64_t pos = (int64_t)(p.pos0 ? p.pos0[b] : 0) + j;
            const uint64_t turn = (uint64_t)pos * s_freq[lane];
            // half turns in [-1, 1]
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &mine.y, &mine.x);
        }
        Coef coef;
        int have = -1;  // which weights the coefficients hold
        for (uint32_t it = 0; it < p.iters; it += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (it + u >= p.iters) break;
                Item& cur = item[u];
                const int h0 = head(it + u);
                const bool k = h0 >= p.heads[0];
                if (__any_sync(0xffffffffu, have != (int)k)) {
                    have = k;
                    make_coef<T>(coef, mine, k ? p.w[1] : p.w[0], l);
                }
                norm_rotate<T>(cur.lo, cur.hi, coef, p.eps);
                if (h0 < total) {
                    const int h = k ? h0 - p.heads[0] : h0;
                    uint8_t* dst = (k ? p.y[1] : p.y[0]) +
                                   (((int64_t)b * (k ? p.heads[1] : p.heads[0]) + h) * p.n + j) *
                                       kRowBytes;
                    *reinterpret_cast<uint4*>(dst + l * 16) = cur.lo;
                    *reinterpret_cast<uint4*>(dst + 64 + l * 16) = cur.hi;
                }
                if (it + u + kAhead < p.iters) cur = load(it + u + kAhead);
            }
        }
    }
    pdl_trigger();
}

// theta_i / (2 pi) modulo 1 for the 32 pairs. A thread that keeps calling with one base
// computes them once.
const uint64_t* turn_table(float base) {
    thread_local float have = 0.f;
    thread_local uint64_t t[32];
    if (have != base) {
        for (int i = 0; i < 32; ++i) {
            const double turns = std::pow((double)base, -i / 32.0) * 0.15915494309189533577;
            t[i] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);
        }
        have = base;
    }
    return t;
}

kvd_status check_rows(const kvd_head_rows* r, int32_t batch, int32_t n) {
    if (!r) return KVD_OK;
    if (r->n_heads <= 0 || !r->x || !r->out) return KVD_ERR_INVALID_ARG;
    if (!aligned16(r->x) || !aligned16(r->out) || !aligned16(r->weight))
        return KVD_ERR_INVALID_ARG;
    if (r->stride_b < 0 || r->stride_h < 0 || r->stride_t < 0 ||
        ((r->stride_b | r->stride_h | r->stride_t) & 7))
        return KVD_ERR_INVALID_ARG;
    if (r->out == r->x) {  // in place: the input has the output's layout
        const int64_t row = KVD_HEAD_DIM;
        if ((n > 1 && r->stride_t != row) || (r->n_heads > 1 && r->stride_h != n * row) ||
            (batch > 1 && r->stride_b != r->n_heads * (n * row)))
            return KVD_ERR_INVALID_ARG;
    }
    return KVD_OK;
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_qk_norm_rope(kvd_dtype dtype, int32_t batch, int32_t n,
                                       const kvd_head_rows* q, const kvd_head_rows* k,
                                       const int32_t* pos0, float eps, float base,
                                       uint32_t flags, int32_t* dev_err, kvd_stream_t stream) {
    (void)dev_err;
    if (dtype != KVD_F16 && dtype != KVD_BF16) return KVD_ERR_INVALID_ARG;
    if (batch < 0 || n < 0 || !(eps >= 0.f) || !(eps < INFINITY)) return KVD_ERR_INVALID_ARG;
    if (!(base >= 0.f) || !(base < INFINITY)) return KVD_ERR_INVALID_ARG;
    if (batch == 0 || n == 0 || (!q && !k)) return KVD_OK;
    if (kvd_status s = check_rows(q, batch, n)) return s;
    if (kvd_status s = check_rows(k, batch, n)) return s;
    NormRopeParams p = {};
    const kvd_head_rows* rows[2] = {q, k};
    int64_t heads = 0;
    for (int t = 0; t < 2; ++t) {
        if (!rows[t]) continue;
        p.x[t] = static_cast<const uint8_t*>(rows[t]->x);
        p.y[t] = static_cast<uint8_t*>(rows[t]->out);
        p.w[t] = static_cast<const uint8_t*>(rows[t]->weight);
        p.sb[t] = rows[t]->stride_b * 2;
        p.sh[t] = rows[t]->stride_h * 2;
        p.st[t] = rows[t]->stride_t * 2;
        p.heads[t] = rows[t]->n_heads;
        heads += rows[t]->n_heads;
    }
    const int64_t tokens = (int64_t)batch * n, groups = (heads + 7) / 8;
    // fewest warps that still fill the GPU: a warp's cos/sin then serve more heads
    int64_t iters = 1;
    while (iters < groups && tokens * ((groups + iters) / (iters + 1)) >= kNrManyWarps) ++iters;
    const int64_t hgroups = (groups + iters - 1) / iters;
    const int64_t warps = tokens * hgroups;
    if (heads > 0x3fffffff || warps > 0x7fffffff) return KVD_ERR_UNSUPPORTED;
    p.pos0 = pos0;
    p.n = n;
    p.tokens = (uint32_t)tokens;
    p.hgroups = (uint32_t)hgroups;
    p.iters = (uint32_t)iters;
    p.rotate = base > 0.f;
    p.eps = eps;
    if (p.rotate) std::memcpy(p.freq, turn_table(base), sizeof(p.freq));
    constexpr int kWarpsPerBlock = kNrThreads / 32;
    const dim3 grid((unsigned)((warps + kWarpsPerBlock - 1) / kWarpsPerBlock));
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool pdl = (flags & KVD_FLAG_PDL) != 0;
    if (dtype == KVD_BF16)
        return launch(qk_norm_rope_kernel<__nv_bfloat16>, grid, dim3(kNrThreads), 0, st, pdl, p);
    return launch(qk_norm_rope_kernel<__half>, grid, dim3(kNrThreads), 0, st, pdl, p);
}
