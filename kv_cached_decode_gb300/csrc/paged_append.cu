// paged_append.cu -- new tokens of a packed ragged batch, rotated and written to the pages that a
// table gives.
//
// No counterpart on the pages: a server that runs many sequences keeps their caches in pages of
// one pool. Token j of row b stands at position s = lens_in[b] + j; its K and V rows go to slot
// s % page_size of page table[b, s / page_size], K (and the queries, if given) rotated by a
// kvd_rope_spec at s.
//
// Design. Rows of 128 bytes are read and written once: HBM bounds prompts, the launch single
// tokens. A warp takes the heads of one token (or a share of them when tokens are few), four rows
// at a time, eight lanes a row, so a token's row, page and angles are found once. Its rows are on
// their way meanwhile, if some row of the batch holds the token. Which one comes from a search over
// `starts`, 32 probes a step; rows, lengths and pages that do not fit are flagged and skipped.
//
// Measured (in a graph): 64 tokens x 40 heads 3.5 us, a launch and four loads that need one
// another (row, length, page, rows); 6 rows of up to 2000 tokens x 28 heads 16.6 us from cold
// buffers, 3.9 TB/s of what is read and written (14.3 with buffers that the second-level cache
// holds in part): one wave of warps, so the loads and the stores hardly overlap.
#include <algorithm>

#include "kvd_paged.cuh"
#include "kvd_rotate.cuh"

namespace kvd {

kvd_status validate_paged_cache(const kvd_paged_cache* c) {
    if (!c || !c->k || !c->v || !c->table) return KVD_ERR_INVALID_ARG;
    if (c->head_dim != KVD_HEAD_DIM) return KVD_ERR_UNSUPPORTED;
    if (c->n_pages <= 0 || c->n_kv_heads <= 0 || c->batch <= 0 || c->table_width <= 0 ||
        c->page_size <= 0)
        return KVD_ERR_INVALID_ARG;
    if (c->page_size < KVD_MIN_PAGE || c->page_size > KVD_MAX_PAGE ||
        (c->page_size & (c->page_size - 1)))
        return KVD_ERR_UNSUPPORTED;
    if ((int64_t)c->table_width * c->page_size > kPagedMaxLen) return KVD_ERR_UNSUPPORTED;
    if (c->table_stride < c->table_width) return KVD_ERR_INVALID_ARG;
    if (c->stride_t < KVD_HEAD_DIM || c->stride_h < KVD_HEAD_DIM || c->stride_p < KVD_HEAD_DIM ||
        ((c->stride_t | c->stride_h | c->stride_p) & 7))
        return KVD_ERR_INVALID_ARG;
    // what a tensor map of 16-bit values can hold
    const int64_t most = INT64_C(1) << 38;
    if (c->stride_t > most || c->stride_h > most || c->stride_p > most) return KVD_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->table) & 3))
        return KVD_ERR_INVALID_ARG;
    return KVD_OK;
}

kvd_status validate_token_rows(const kvd_token_rows* r) {
    if (!r || !r->x || r->n_heads <= 0) return KVD_ERR_INVALID_ARG;
    if (!aligned16(r->x) || !aligned16(r->out)) return KVD_ERR_INVALID_ARG;
    if (r->stride_t < 0 || r->stride_h < 0 || ((r->stride_t | r->stride_h) & 7))
        return KVD_ERR_INVALID_ARG;
    return KVD_OK;
}

namespace {

constexpr int kPaThreads = 128;
// Warps that a launch should have before a warp takes more heads (64 tokens x 40 heads: 4.4 us at 1
// per SM, 3.5 from 4 on; 6 x 2000 tokens x 28 heads: the same time at 1 to 64 per SM, a warp per
// four heads and token takes twice as long).
constexpr int64_t kPaManyWarps = 152 * 16;
constexpr int kPaAhead = 4;                 // groups of four heads whose loads are in flight

struct PagedAppendParams {
    const uint8_t* x[3];        // k, v, q
    int64_t st[3], sh[3];       // strides, bytes
    uint8_t* kc;                // the pools, byte strides
    uint8_t* vc;
    int64_t sp, ch, ct;
    uint8_t* q_out;             // [n_tokens, n_q_heads, 64]
    const int32_t* table;
    int64_t table_stride;
    const int32_t* starts;
    const int32_t* lens_in;
    int32_t* lens_out;
    int32_t* dev_err;
    int32_t batch, n_tokens, n_pages, page_log2, capacity;
    int32_t hk, hq;
    uint32_t hgroups, iters;    // warps per token; groups of 4 heads per warp
    int32_t rotate;
    RopeTurns turns;
};

template <typename T, bool INTER>
__global__ void __launch_bounds__(kPaThreads) paged_append_kernel(const PagedAppendParams p) {
    __shared__ uint64_t s_freq[32];
    if (threadIdx.x < 32) s_freq[threadIdx.x] = p.turns.freq[threadIdx.x];
    pdl_wait();
    const int first = p.starts[0], end = min(p.starts[p.batch], p.n_tokens);
    __syncthreads();
    // lengths after the call, and the rows that do not fit
    for (int64_t b = (int64_t)blockIdx.x * kPaThreads + threadIdx.x; b < p.batch;
         b += (int64_t)gridDim.x * kPaThreads) {
        int s, n;
        const int len = p.lens_in[b];
        const bool ok = row_tokens(p.starts, (int)b, p.n_tokens, s, n) && len >= 0 &&
                        (int64_t)len + n <= p.capacity;
        if (!ok) flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
        if (p.lens_out) p.lens_out[b] = ok ? len + n : len;
    }
    const int64_t wid = (int64_t)blockIdx.x * (kPaThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(wid / p.hgroups);
    const uint32_t hg = (uint32_t)(wid % p.hgroups);
    const int lane = threadIdx.x & 31, ch = lane & 7;
    if (t >= first && t < end) {  // (warp-uniform; tokens of no row are not read)
        // this lane's heads are h0, h0 + 4, ..: those of K, of V and of q
        const int hk = p.hk, h0 = (int)(hg * p.iters) * 4 + (lane >> 3);
        const int last = min(2 * p.hk + p.hq, (int)((hg + 1) * p.iters) * 4);
        // the token's rows, as if each tensor's heads were numbered so
        const uint8_t* xk = p.x[0] + t * p.st[0] + ch * 16;
        const uint8_t* xv = p.x[1] + t * p.st[1] - hk * p.sh[1] + ch * 16;
        const uint8_t* xq = p.x[2] + t * p.st[2] - 2 * hk * p.sh[2] + ch * 16;
        auto load = [&](int h) {
            if (h >= last) return make_uint4(0u, 0u, 0u, 0u);
            return *reinterpret_cast<const uint4*>(h < hk       ? xk + h * p.sh[0]
                                                   : h < 2 * hk ? xv + h * p.sh[1]
                                                                : xq + h * p.sh[2]);
        };
        // (the rows do not depend on where they go)
        uint4 item[kPaAhead];
#pragma unroll
        for (int u = 0; u < kPaAhead; ++u) item[u] = load(h0 + 4 * u);
        const int b = find_token_row(p.starts, p.batch, t);
        int s, n;
        const bool in_row = row_tokens(p.starts, b, p.n_tokens, s, n) && t >= s && t < s + n;
        const int len = p.lens_in[b];
        if (in_row && len >= 0 && (int64_t)len + n <= p.capacity) {
            const int pos = len + (t - s);
            const int page = p.table[b * p.table_stride + (pos >> p.page_log2)];
            const bool page_ok = page >= 0 && page < p.n_pages;
            if (!page_ok && hg == 0 && lane == 0) flag_error(p.dev_err, KVD_ERR_BAD_INDEX);
            const int64_t slot =
                page * p.sp + (int64_t)(pos & ((1 << p.page_log2) - 1)) * p.ct + ch * 16;
            uint8_t* yk = p.kc + slot;
            uint8_t* yv = p.vc + slot - hk * p.ch;
            uint8_t* yq = p.q_out + ((int64_t)t * p.hq - 2 * hk) * kRowBytes + ch * 16;
            Turn turn;
            if (p.rotate)
                make_turn<INTER>(turn, s_freq[lane], pos, p.turns.rot, p.turns.mag);
            for (int g = h0; g - (lane >> 3) < last; g += 4 * kPaAhead) {  // (the warp's bound)
#pragma unroll
                for (int u = 0; u < kPaAhead; ++u) {
                    const int h = g + 4 * u;
                    if (h - (lane >> 3) >= last) break;
                    const bool k = h < hk, q = h >= 2 * hk;
                    uint4 v = item[u];
                    if (p.rotate) {
                        const uint4 r = rotate_chunk<T, INTER>(v, turn, p.turns.rot);
                        if (k || q) v = r;
                    }
                    if (h < last && (page_ok || q))
                        *reinterpret_cast<uint4*>(q   ? yq + (int64_t)h * kRowBytes
                                                  : k ? yk + h * p.ch
                                                      : yv + h * p.ch) = v;
                    item[u] = load(h + 4 * kPaAhead);
                }
            }
        }
    }
    pdl_trigger();
}

template <typename T>
kvd_status run(const PagedAppendParams& p, dim3 grid, cudaStream_t st, bool pdl) {
    return p.rotate && p.turns.inter
               ? launch(paged_append_kernel<T, true>, grid, dim3(kPaThreads), 0, st, pdl, p)
               : launch(paged_append_kernel<T, false>, grid, dim3(kPaThreads), 0, st, pdl, p);
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_paged_append(kvd_dtype dtype, const kvd_paged_cache* cache,
                                       int32_t n_tokens, const kvd_token_rows* k_new,
                                       const kvd_token_rows* v_new, const kvd_token_rows* q,
                                       const int32_t* starts, const int32_t* lens_in,
                                       int32_t* lens_out, const kvd_rope_spec* spec,
                                       uint32_t flags, int32_t* dev_err, kvd_stream_t stream) {
    if (dtype != KVD_F16 && dtype != KVD_BF16) return KVD_ERR_INVALID_ARG;
    if (kvd_status s = validate_paged_cache(cache)) return s;
    if (n_tokens < 0) return KVD_ERR_INVALID_ARG;
    PagedAppendParams p = {};
    if (spec) {
        if (kvd_status s = rope_turns(spec, &p.turns)) return s;
        p.rotate = 1;
    }
    if (!starts || !lens_in || (lens_out && lens_out == lens_in)) return KVD_ERR_INVALID_ARG;
    const kvd_token_rows* rows[3] = {k_new, v_new, q};
    if (n_tokens > 0) {
        if (!k_new || !v_new) return KVD_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i) {
            if (!rows[i]) continue;
            if (kvd_status s = validate_token_rows(rows[i])) return s;
            if (i < 2 && (rows[i]->n_heads != cache->n_kv_heads || rows[i]->out))
                return KVD_ERR_INVALID_ARG;
            p.x[i] = static_cast<const uint8_t*>(rows[i]->x);
            p.st[i] = rows[i]->stride_t * 2;
            p.sh[i] = rows[i]->stride_h * 2;
        }
        if (q) {
            if (!q->out) return KVD_ERR_INVALID_ARG;
            if (q->out == q->x && ((n_tokens > 1 && q->stride_t != (int64_t)q->n_heads * 64) ||
                                   (q->n_heads > 1 && q->stride_h != 64)))
                return KVD_ERR_INVALID_ARG;  // in place: the input has the output's layout
            p.hq = q->n_heads;
            p.q_out = static_cast<uint8_t*>(q->out);
        }
    }
    p.kc = static_cast<uint8_t*>(cache->k);
    p.vc = static_cast<uint8_t*>(cache->v);
    p.sp = cache->stride_p * 2;
    p.ch = cache->stride_h * 2;
    p.ct = cache->stride_t * 2;
    p.table = cache->table;
    p.table_stride = cache->table_stride;
    p.starts = starts;
    p.lens_in = lens_in;
    p.lens_out = lens_out;
    p.dev_err = dev_err;
    p.batch = cache->batch;
    p.n_tokens = n_tokens;
    p.n_pages = cache->n_pages;
    while ((1 << p.page_log2) < cache->page_size) ++p.page_log2;
    p.capacity = cache->table_width * cache->page_size;
    p.hk = cache->n_kv_heads;
    const int64_t heads = 2 * (int64_t)p.hk + p.hq, groups = (heads + 3) / 4;
    if (heads > 0x1fffffff) return KVD_ERR_UNSUPPORTED;
    // fewest warps that still fill the GPU: what a token needs is then found for more heads
    int64_t iters = 1;
    while (iters < groups && n_tokens * ((groups + iters) / (iters + 1)) >= kPaManyWarps) ++iters;
    const int64_t hgroups = (groups + iters - 1) / iters;
    constexpr int kWarpsPerBlock = kPaThreads / 32;
    const int64_t blocks =
        std::max<int64_t>(1, (n_tokens * hgroups + kWarpsPerBlock - 1) / kWarpsPerBlock);
    if (blocks > 0x7fffffff) return KVD_ERR_UNSUPPORTED;
    p.hgroups = (uint32_t)hgroups;
    p.iters = (uint32_t)iters;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool pdl = (flags & KVD_FLAG_PDL) != 0;
    const dim3 grid((unsigned)blocks);
    return dtype == KVD_BF16 ? run<__nv_bfloat16>(p, grid, st, pdl) : run<__half>(p, grid, st, pdl);
}
