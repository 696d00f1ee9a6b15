// rope_scaled.cu -- rotary positions with pairs of halves or interleaved, in a part of the head,
// with frequencies scaled for contexts longer than the trained one.
//
// No counterpart on the pages: kvd_rope has one form (halves, the whole head, base^(-i/32)). With
// pairs (a, b) = (i, i + rot/2) or (2i, 2i+1), i < rot/2, at position p:
//   y[a] = m (x[a] cos(p t_i) - x[b] sin(p t_i)),  y[b] = m (x[b] cos(p t_i) + x[a] sin(p t_i))
// t_i the scaled frequencies of kvd_rope_spec, formed on the host in 64 bits and given as
// fractions of a turn in 64-bit fixed point (see kvd_rotate.cuh); dims from rot on are copied.
// fp32 products, one rounding to the storage type.
//
// Design. Every row of 128 bytes is read and written once: HBM bounds many rows, the launch few.
// A warp takes the heads of one token, four at a time, so that cos and sin are formed once per
// token and lane; several groups of heads are in flight, and the next is loaded as soon as one is
// stored. A launch with few tokens spreads a token's heads over several warps.
//
// Measured (in a graph): 16 tokens x 24 heads 2.5 us, a launch's time; 4 x 4096 tokens x 24 heads
// 18.3 us from cold buffers, 5.5 TB/s of what is read and written (a copy: 6.8), 15.6 with buffers
// that the second-level cache holds in part. Addresses are formed once per token: with all of a
// row's strides multiplied for each row the latter was 18.7 us, bound by instructions.
#include <cmath>
#include <cstring>

#include "kvd_rotate.cuh"

namespace kvd {
namespace {

constexpr int kRsThreads = 128;
// Warps that a launch should have before a warp takes more heads (4 x 4096 tokens x 24 heads: the
// same time at 1 to 64 per SM; a warp per four heads and token takes twice as long).
constexpr int64_t kRsManyWarps = 152 * 16;
constexpr int kRsAhead = 4;                 // groups of four heads whose loads are in flight

struct RopeScaledParams {
    const uint8_t* x[2];          // q, k
    uint8_t* y[2];
    int64_t sb[2], sh[2], st[2];  // input strides, bytes
    int32_t heads[2];
    const int32_t* pos0;          // [batch] or null
    const int32_t* positions;     // [batch, n] or null
    int32_t n;
    uint32_t tokens, hgroups, iters;  // tokens; warps per token; groups of 4 heads per warp
    RopeTurns turns;
};

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRsThreads) rope_scaled_kernel(const RopeScaledParams p) {
    __shared__ uint64_t s_freq[32];
    if (threadIdx.x < 32) s_freq[threadIdx.x] = p.turns.freq[threadIdx.x];
    pdl_wait();
    __syncthreads();
    const uint32_t wid = blockIdx.x * (kRsThreads / 32) + (threadIdx.x >> 5);
    const uint32_t token = wid / p.hgroups, hg = wid % p.hgroups;
    const int b = (int)(token / (uint32_t)p.n), j = (int)(token % (uint32_t)p.n);
    const int lane = threadIdx.x & 31, ch = lane & 7;
    // this lane's heads are h0, h0 + 4, ..: those of q, then those of k
    const int h0 = (int)(hg * p.iters) * 4 + (lane >> 3), total = p.heads[0] + p.heads[1];
    const int last = min(total, (int)((hg + 1) * p.iters) * 4);
    // the token's rows of q's (k's) first head
    const uint8_t* xq = p.x[0] + b * p.sb[0] + j * p.st[0] + ch * 16;
    const uint8_t* xk = p.x[1] + b * p.sb[1] + j * p.st[1] + ch * 16;
    uint8_t* yq = p.y[0] + ((int64_t)b * p.heads[0] * p.n + j) * kRowBytes + ch * 16;
    uint8_t* yk = p.y[1] + ((int64_t)b * p.heads[1] * p.n + j) * kRowBytes + ch * 16;
    const int64_t to_head = (int64_t)p.n * kRowBytes;
    auto load = [&](int h) {
        if (h >= last) return make_uint4(0u, 0u, 0u, 0u);
        const int hk = h - p.heads[0];
        return *reinterpret_cast<const uint4*>(hk >= 0 ? xk + hk * p.sh[1] : xq + h * p.sh[0]);
    };
    if (token < p.tokens) {  // warp-uniform
        uint4 item[kRsAhead];
#pragma unroll
        for (int u = 0; u < kRsAhead; ++u) item[u] = load(h0 + 4 * u);
        const int64_t pos =
            p.positions ? p.positions[token] : (int64_t)(p.pos0 ? p.pos0[b] : 0) + j;
        Turn t;
        make_turn<INTER>(t, s_freq[lane], pos, p.turns.rot, p.turns.mag);
        for (int g = h0; g - (lane >> 3) < last; g += 4 * kRsAhead) {  // (the warp's bound)
#pragma unroll
            for (int u = 0; u < kRsAhead; ++u) {
                const int h = g + 4 * u, hk = h - p.heads[0];
                if (h - (lane >> 3) >= last) break;
                const uint4 v = rotate_chunk<T, INTER>(item[u], t, p.turns.rot);
                if (h < last)
                    *reinterpret_cast<uint4*>(hk >= 0 ? yk + hk * to_head : yq + h * to_head) = v;
                item[u] = load(h + 4 * kRsAhead);
            }
        }
    }
    pdl_trigger();
}

kvd_status check_rows(const kvd_head_rows* r, int32_t batch, int32_t n) {
    if (!r) return KVD_OK;
    if (r->n_heads <= 0 || !r->x || !r->out || r->weight) return KVD_ERR_INVALID_ARG;
    if (!aligned16(r->x) || !aligned16(r->out)) return KVD_ERR_INVALID_ARG;
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

template <typename T>
kvd_status run(const RopeScaledParams& p, dim3 grid, cudaStream_t st, bool pdl) {
    return p.turns.inter
               ? launch(rope_scaled_kernel<T, true>, grid, dim3(kRsThreads), 0, st, pdl, p)
               : launch(rope_scaled_kernel<T, false>, grid, dim3(kRsThreads), 0, st, pdl, p);
}

}  // namespace

// The last spec of a thread is kept with its frequencies: a program has one per model, and 32
// powers cost as much as the launch.
kvd_status rope_turns(const kvd_rope_spec* s, RopeTurns* t) {
    thread_local kvd_rope_spec have = {};  // base 0: none
    thread_local RopeTurns last;
    if (!s) return KVD_ERR_INVALID_ARG;
    if (have.base == s->base && have.rot_dim == s->rot_dim && have.interleaved == s->interleaved &&
        have.scaling == s->scaling && have.factor == s->factor && have.low == s->low &&
        have.high == s->high && have.original_len == s->original_len &&
        have.magnitude == s->magnitude && s->base > 0.f) {
        *t = last;
        return KVD_OK;
    }
    if (!(s->base > 0.f) || !(s->base < INFINITY)) return KVD_ERR_INVALID_ARG;
    if (!(s->magnitude > -INFINITY) || !(s->magnitude < INFINITY)) return KVD_ERR_INVALID_ARG;
    if (s->rot_dim < 16 || s->rot_dim > KVD_HEAD_DIM || s->rot_dim % 16) return KVD_ERR_UNSUPPORTED;
    if (s->interleaved != 0 && s->interleaved != 1) return KVD_ERR_INVALID_ARG;
    if (s->scaling < KVD_ROPE_NONE || s->scaling > KVD_ROPE_RAMP) return KVD_ERR_INVALID_ARG;
    const bool parts = s->scaling == KVD_ROPE_BANDS || s->scaling == KVD_ROPE_RAMP;
    if (s->scaling != KVD_ROPE_NONE && (!(s->factor > 0.f) || !(s->factor < INFINITY)))
        return KVD_ERR_INVALID_ARG;
    if (parts && (s->original_len < 1 || !(s->low > 0.f) || !(s->high > s->low) ||
                  !(s->high < INFINITY)))
        return KVD_ERR_INVALID_ARG;
    if (s->scaling == KVD_ROPE_RAMP && !(s->base > 1.f)) return KVD_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586477, base = s->base, rot = s->rot_dim;
    const double len = s->original_len, factor = s->factor;
    double lo = 0., hi = 0.;
    if (s->scaling == KVD_ROPE_RAMP) {
        // the pair that turns r times over the trained length
        auto pair = [&](double r) {
            return rot * std::log(len / (two_pi * r)) / (2. * std::log(base));
        };
        lo = std::fmax(std::floor(pair(s->high)), 0.);
        hi = std::fmin(std::ceil(pair(s->low)), rot - 1.);
    }
    for (int i = 0; i < 32; ++i) {
        if (2 * i >= s->rot_dim) {
            t->freq[i] = 0;
            continue;
        }
        const double theta = std::pow(base, -2. * i / rot);
        double keep = 1.;  // how much of the pair keeps its frequency
        if (s->scaling == KVD_ROPE_LINEAR) keep = 0.;
        if (s->scaling == KVD_ROPE_BANDS)
            keep = (len * theta / two_pi - s->low) / ((double)s->high - s->low);
        if (s->scaling == KVD_ROPE_RAMP) keep = 1. - (i - lo) / std::fmax(hi - lo, 0.001);
        keep = std::fmin(std::fmax(keep, 0.), 1.);
        const double scaled = s->scaling == KVD_ROPE_NONE ? theta
                                                          : theta * (keep + (1. - keep) / factor);
        const double turns = scaled / two_pi, part = turns - std::floor(turns);
        t->freq[i] = (uint64_t)std::ldexp(part, 64);  // (part < 1: below 2^64)
    }
    t->rot = s->rot_dim;
    t->inter = s->interleaved;
    t->mag = s->magnitude;
    last = *t;
    have = *s;
    return KVD_OK;
}

}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_rope_scaled(kvd_dtype dtype, int32_t batch, int32_t n,
                                      const kvd_head_rows* q, const kvd_head_rows* k,
                                      const int32_t* pos0, const int32_t* positions,
                                      const kvd_rope_spec* spec, uint32_t flags, int32_t* dev_err,
                                      kvd_stream_t stream) {
    (void)dev_err;
    if (dtype != KVD_F16 && dtype != KVD_BF16) return KVD_ERR_INVALID_ARG;
    if (batch < 0 || n < 0 || (pos0 && positions)) return KVD_ERR_INVALID_ARG;
    RopeScaledParams p = {};
    if (kvd_status s = rope_turns(spec, &p.turns)) return s;
    if (batch == 0 || n == 0 || (!q && !k)) return KVD_OK;
    if (kvd_status s = check_rows(q, batch, n)) return s;
    if (kvd_status s = check_rows(k, batch, n)) return s;
    const kvd_head_rows* rows[2] = {q, k};
    int64_t heads = 0;
    for (int t = 0; t < 2; ++t) {
        if (!rows[t]) continue;
        p.x[t] = static_cast<const uint8_t*>(rows[t]->x);
        p.y[t] = static_cast<uint8_t*>(rows[t]->out);
        p.sb[t] = rows[t]->stride_b * 2;
        p.sh[t] = rows[t]->stride_h * 2;
        p.st[t] = rows[t]->stride_t * 2;
        p.heads[t] = rows[t]->n_heads;
        heads += rows[t]->n_heads;
    }
    const int64_t tokens = (int64_t)batch * n, groups = (heads + 3) / 4;
    // fewest warps that still fill the GPU: a warp's cos and sin then serve more heads
    int64_t iters = 1;
    while (iters < groups && tokens * ((groups + iters) / (iters + 1)) >= kRsManyWarps) ++iters;
    const int64_t hgroups = (groups + iters - 1) / iters;
    if (heads > 0x3fffffff || tokens > 0x7fffffff || tokens * hgroups > 0x7fffffff)
        return KVD_ERR_UNSUPPORTED;
    p.pos0 = pos0;
    p.positions = positions;
    p.n = n;
    p.tokens = (uint32_t)tokens;
    p.hgroups = (uint32_t)hgroups;
    p.iters = (uint32_t)iters;
    constexpr int kWarpsPerBlock = kRsThreads / 32;
    const dim3 grid((unsigned)((tokens * hgroups + kWarpsPerBlock - 1) / kWarpsPerBlock));
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool pdl = (flags & KVD_FLAG_PDL) != 0;
    return dtype == KVD_BF16 ? run<__nv_bfloat16>(p, grid, st, pdl) : run<__half>(p, grid, st, pdl);
}
