// q4_cache.cu -- the 4-bit cache's rows: quantise and append, and read back in 16 bits.
//
// A row is 64 values of one head at one position: n in 0..15 (32 bytes), a bfloat16 step
// and a binary16 zero point z, value = step * (n - z). The step has bfloat16's exponent
// range (any input range fits), the zero point binary16's 11 bits (|z| <= 15 * 2^11 for
// inputs of 11 bits). Both are rounded BEFORE n is formed, so their rounding moves the
// grid and is not an error of every value.
//
// Design. On a prompt HBM bounds the read-back (36 bytes read, 128 written per row: 16 rows x 8
// heads x 4096 of K and V in 32.6 us, 5.3 TB/s), HBM and the issue of instructions the append
// (36.6 us, 4.7 TB/s); on a step the launch (1.9 and 2.2 us). Four lanes own a row, 16 values
// (two 16-byte accesses) each; minimum and maximum are taken on the 16-bit values, two at a
// time, and over the row with two shuffles. x / step rounded correctly, for every value of a
// row by the same step, is a product with the rounded reciprocal and one remainder step
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990: exact when the reciprocal is rounded to nearest and nothing leaves the normal range),
// a fifth of the instructions of a division; rows whose step is near the ends of the range
// divide. Two values share an instruction (fp32 pairs, rounded each by itself). Everything else
// is the IEEE operation in one fixed order, so that the stored bits follow from the definition
// on any machine.
#include <algorithm>

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {
namespace {

constexpr int kQ4Threads = 256;

struct Q4RowsParams {
    uint8_t* data[2];     // K, V rows of the cache
    uint8_t* params;
    const uint8_t* in[2];  // append: the new K, V
    uint8_t* out[2];       // read-back
    int64_t sb, sh;        // rows
    const int32_t* pos0;   // lens_in of the append
    const int32_t* counts;
    int32_t* lens_out;
    int32_t* dev_err;
    int32_t capacity, heads, n;
};

__device__ __forceinline__ float bf16_up(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f2bf(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

__device__ __forceinline__ __half2 as_pair(uint32_t v, __half) {
    return *reinterpret_cast<__half2*>(&v);
}
__device__ __forceinline__ __nv_bfloat162 as_pair(uint32_t v, __nv_bfloat16) {
    return *reinterpret_cast<__nv_bfloat162*>(&v);
}

// n = clamp(rint(x / step + z), 0, 15) of the 16 values in the words v, packed.
// FAST: rcp is step's rounded reciprocal.
template <typename T, bool FAST>
__device__ __forceinline__ uint2 pack16(const uint32_t* v, float step, float rcp, float z) {
    // the words, less what the sums below add to them besides n
    constexpr uint32_t kMagic = 0x4B400000u;  // 1.5 * 2^23
    constexpr uint32_t kRest = kMagic * 0x11111111u;
    uint32_t w[2] = {0u - kRest, 0u - kRest};
    const Pair rcp2(rcp, rcp), neg(-step, -step), z2(z, z), magic(12582912.f, 12582912.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 xf = Half16<T>::to_f2(v[e]);
        const Pair x(xf.x, xf.y);
        Pair q = x;
        if (FAST) {
            q = mul2(x, rcp2);
            q = fma2(fma2(q, neg, x), rcp2, q);
        } else {
            q = Pair(__fdiv_rn(xf.x, step), __fdiv_rn(xf.y, step));
        }
        // clamped, then rounded to even by adding 1.5 * 2^23: n in the low bits
        float2 t = add2(q, z2).get();
        t.x = fminf(fmaxf(t.x, 0.f), 15.f);
        t.y = fminf(fmaxf(t.y, 0.f), 15.f);
        const float2 n = add2(Pair(t.x, t.y), magic).get();
        w[e >> 2] += __float_as_uint(n.x) << (8 * (e & 3));
        w[e >> 2] += __float_as_uint(n.y) << (8 * (e & 3) + 4);
    }
    return make_uint2(w[0], w[1]);
}

// a / b, correctly rounded: see above. b has at most 8 significant bits (bfloat16, or 7.5), so the
// remainder is exact and no quotient is closer than 2^-9 of a step to where rounding turns, far
// more than the last product's error. b within (kQuickMin, kQuickMax): nothing that matters
// leaves the normal range (|a / b| <= 2^15 or so; one below 2^-60 rounds away in what follows).
constexpr float kQuickMin = 0x1p-50f, kQuickMax = 0x1p90f;
__device__ __forceinline__ float quotient(float a, float b, float rcp) {
    const float q = __fmul_rn(a, rcp);
    return __fmaf_rn(__fmaf_rn(-q, b, a), rcp, q);
}
// a / b for a >= 0 and a constant b. (A division of 0 would take its slow path: a warp with one
// row of zeros, or one past its prompt, took 8 us.)
__device__ __forceinline__ float by_const(float a, float b, float rcp) {
    return a == 0.f ? 0.f : a > kQuickMin && a < kQuickMax ? quotient(a, b, rcp) : __fdiv_rn(a, b);
}

// Quantise the 16 values (eight words) of this lane, a quarter of a row; the row's lanes are
// lane ^ 1, ^ 2, ^ 3: packed nibbles and the row's (step | zero point << 16). bad: the row
// holds an infinity or a NaN.
template <typename T>
__device__ __forceinline__ uint2 quantise16(const uint32_t* v, uint32_t& par, bool& bad) {
    auto l2 = as_pair(v[0], T()), h2 = l2;  // (NaN stays)
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        l2 = __hmin2_nan(l2, as_pair(v[e], T()));
        h2 = __hmax2_nan(h2, as_pair(v[e], T()));
    }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
        l2 = __hmin2_nan(l2, __shfl_xor_sync(0xffffffffu, l2, off));
        h2 = __hmax2_nan(h2, __shfl_xor_sync(0xffffffffu, h2, off));
    }
    const float2 lf = Half16<T>::to_f2(*reinterpret_cast<const uint32_t*>(&l2));
    const float2 hf = Half16<T>::to_f2(*reinterpret_cast<const uint32_t*>(&h2));
    const float lo = fminf(lf.x, lf.y), hi = fmaxf(hf.x, hf.y);
    // (0 * finite is 0)
    bad = !(lf.x * 0.f + lf.y * 0.f + hf.x * 0.f + hf.y * 0.f == 0.f);
    // halves: no finite range overflows
    const float d = __fsub_rn(__fmul_rn(0.5f, hi), __fmul_rn(0.5f, lo));
    uint16_t sbits = f2bf(by_const(d, 7.5f, 1.f / 7.5f));
    float step = bf16_up(sbits);
    const bool flat = step == 0.f;
    if (flat) {
        sbits = f2bf(by_const(fabsf(lo), 15.f, 1.f / 15.f));
        if (sbits == 0) sbits = f2bf(1.f);
        step = bf16_up(sbits);
    }
    const bool quick = step > kQuickMin && step < kQuickMax;
    const float rcp = quick ? __frcp_rn(step) : 0.f;
    float z = lo < 0.f ? 15.f : 0.f;
    if (!flat) {
        const float q = quick ? quotient(-lo, step, rcp) : __fdiv_rn(-lo, step);
        z = __half2float(__float2half_rn(q)) + 0.f;  // (no -0)
    }
    par = (uint32_t)sbits | ((uint32_t)__half_as_ushort(__float2half_rn(z)) << 16);
    if (bad) {
        par = 0x7FC0u;
        return make_uint2(0u, 0u);
    }
    return quick ? pack16<T, true>(v, step, rcp, z) : pack16<T, false>(v, step, rcp, z);
}

// Block (x, y, z): rows 64 x on of a head of batch row z; no index needs a division.
// BOTH: four lanes do K's row and V's of a head (y) and position (twice the loads in flight,
// parameters stored together): prompts. Else K's only or V's only (y: 2 head + tensor): the chain
// of a step is shorter.
template <typename T, bool BOTH>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(const Q4RowsParams p) {
    constexpr int N = BOTH ? 2 : 1;
    pdl_wait();
    const int b = blockIdx.z, h = BOTH ? blockIdx.y : blockIdx.y >> 1;
    const int t0 = BOTH ? 0 : (int)(blockIdx.y & 1);
    const int l = (int)(threadIdx.x & 3);
    const int j = (int)(blockIdx.x * (kQ4Threads / 4) + threadIdx.x / 4);
    const int64_t row = ((int64_t)b * p.heads + h) * p.n + j;
    uint4 in[N][2] = {};
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint8_t* base = BOTH ? p.in[k] : t0 ? p.in[1] : p.in[0];
            const uint4* src = reinterpret_cast<const uint4*>(base + row * kRowBytes + l * 32);
            in[k][0] = src[0];
            in[k][1] = src[1];
        }
    };
    if (!p.counts && j < p.n) load();  // before the row's length is known
    const int len = p.pos0 ? p.pos0[b] : 0;
    const int cnt = p.counts ? p.counts[b] : p.n;
    const bool first = t0 == 0 && h == 0 && j == 0 && l == 0;
    const bool wrong = len < 0 || cnt < 0 || cnt > p.n || (int64_t)len + cnt > p.capacity;
    if (first && wrong) flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
    if (first && p.lens_out) p.lens_out[b] = wrong ? len : len + cnt;
    const bool live = !wrong && j < cnt;
    if (!__any_sync(0xffffffffu, live)) {  // (rows past their prompts)
        pdl_trigger();
        return;
    }
    if (live && p.counts) load();
    const int64_t at = b * p.sb + h * p.sh + len + j;
    uint32_t par[N];
    bool any_bad = false;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint4 a = in[k][0], d = in[k][1];
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
        bool bad;
        // every lane: the shuffles need whole rows
        const uint2 w = quantise16<T>(v, par[k], bad);
        any_bad |= bad;
        uint8_t* base = BOTH ? p.data[k] : t0 ? p.data[1] : p.data[0];
        if (live) *reinterpret_cast<uint2*>(base + at * 32 + l * 8) = w;
    }
    if (live && l == 0) {
        if (BOTH)
            *reinterpret_cast<uint2*>(p.params + at * 8) = make_uint2(par[0], par[N - 1]);
        else
            *reinterpret_cast<uint32_t*>(p.params + at * 8 + t0 * 4) = par[0];
        if (any_bad) flag_error(p.dev_err, KVD_ERR_NAN);
    }
    pdl_trigger();
}

// Blocks as the append's, K or V (both by one group of lanes: 33.2 -> 36.2 us for 16 rows x 8
// heads x 4096).
template <typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_dequant_kernel(const Q4RowsParams p) {
    pdl_wait();
    const bool two = p.out[0] && p.out[1];
    const int b = blockIdx.z, h = two ? blockIdx.y >> 1 : blockIdx.y;
    const int t = two ? (int)(blockIdx.y & 1) : p.out[0] ? 0 : 1;
    const int l = (int)(threadIdx.x & 3);
    const int j = (int)(blockIdx.x * (kQ4Threads / 4) + threadIdx.x / 4);
    const int pos = p.pos0 ? p.pos0[b] : 0;
    if (pos < 0 || (int64_t)pos + p.n > p.capacity) {
        if (h == 0 && j == 0 && l == 0) flag_error(p.dev_err, KVD_ERR_LEN_OVERFLOW);
    } else if (j < p.n) {
        const int64_t at = b * p.sb + h * p.sh + pos + j;
        const uint8_t* from = (t ? p.data[1] : p.data[0]) + at * 32 + l * 8;
        const uint2 w = *reinterpret_cast<const uint2*>(from);
        const uint32_t par = *reinterpret_cast<const uint32_t*>(p.params + at * 8 + t * 4);
        const float step = bf16_up((uint16_t)par);
        const float z = __half2float(__ushort_as_half((uint16_t)(par >> 16)));
        const Pair step2(step, step), z2(-z, -z), base(-8388608.f, -8388608.f);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t v = (e < 4 ? w.x : w.y) >> (8 * (e & 3));
            // n as 2^23 + n (no conversion), exactly
            const Pair n(__uint_as_float(0x4B000000u | (v & 15u)),
                         __uint_as_float(0x4B000000u | (v >> 4 & 15u)));
            const float2 x = mul2(step2, add2(add2(n, base), z2)).get();
            o[e] = Half16<T>::from_f2(x.x, x.y);
        }
        const int64_t row = ((int64_t)b * p.heads + h) * p.n + j;
        uint4* dst =
            reinterpret_cast<uint4*>((t ? p.out[1] : p.out[0]) + row * kRowBytes + l * 32);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    pdl_trigger();
}

// Rows (of K) from which four lanes do K's and V's: 16 rows x 8 heads x 4096 47.7 -> 38.7 us, 1 x
// 8 x 2048 3.32 -> 3.21 us, but 16 x 8 x 1 2.20 -> 2.67 us.
constexpr int64_t kBothRows = 8192;

// per_head: blocks' y per head
dim3 rows_grid(const Q4RowsParams& p, int32_t batch, int per_head) {
    return dim3((unsigned)((p.n + kQ4Threads / 4 - 1) / (kQ4Threads / 4)),
                (unsigned)(p.heads * per_head), (unsigned)batch);
}
// Whole warps for the rows there are.
dim3 rows_block(const Q4RowsParams& p) {
    return dim3((unsigned)std::min<int64_t>(kQ4Threads, ((int64_t)p.n * 4 + 31) / 32 * 32));
}

template <typename T>
kvd_status run_append(const Q4RowsParams& p, int32_t batch, cudaStream_t st, bool pdl) {
    if ((int64_t)batch * p.heads * p.n >= kBothRows)
        return launch(q4_append_kernel<T, true>, rows_grid(p, batch, 1), rows_block(p), 0, st, pdl,
                      p);
    return launch(q4_append_kernel<T, false>, rows_grid(p, batch, 2), rows_block(p), 0, st, pdl, p);
}
template <typename T>
kvd_status run_dequant(const Q4RowsParams& p, int32_t batch, cudaStream_t st, bool pdl) {
    return launch(q4_dequant_kernel<T>, rows_grid(p, batch, p.out[0] && p.out[1] ? 2 : 1),
                  rows_block(p), 0, st, pdl, p);
}

kvd_status rows_params(Q4RowsParams& p, const kvd_q4_cache* c, int32_t batch, int32_t n) {
    p.data[0] = static_cast<uint8_t*>(c->k);
    p.data[1] = static_cast<uint8_t*>(c->v);
    p.params = static_cast<uint8_t*>(c->params);
    p.sb = c->stride_b;
    p.sh = c->stride_h;
    p.capacity = c->capacity;
    p.heads = c->n_kv_heads;
    p.n = n;
    return batch > 65535 || c->n_kv_heads > 32767 ? KVD_ERR_UNSUPPORTED : KVD_OK;  // the grid's
}

}  // namespace

kvd_status validate_q4_cache(const kvd_q4_cache* c) {
    if (!c || !c->k || !c->v || !c->params) return KVD_ERR_INVALID_ARG;
    if (c->head_dim != KVD_HEAD_DIM) return KVD_ERR_UNSUPPORTED;
    if (c->batch <= 0 || c->n_kv_heads <= 0 || c->capacity <= 0) return KVD_ERR_INVALID_ARG;
    if (c->capacity > (1 << 30)) return KVD_ERR_UNSUPPORTED;  // positions + a tile fit an int
    if ((c->batch > 1 && c->stride_b < c->capacity) || c->stride_b < 0 ||
        (c->n_kv_heads > 1 && c->stride_h < c->capacity) || c->stride_h < 0)
        return KVD_ERR_INVALID_ARG;  // a head's positions are consecutive rows
    if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->params) & 7))
        return KVD_ERR_INVALID_ARG;
    return KVD_OK;
}

}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kvd_q4_append(kvd_dtype dtype, const kvd_q4_cache* cache, int32_t batch,
                                    int32_t q, const void* k_new, const void* v_new,
                                    const int32_t* lens_in, const int32_t* counts,
                                    int32_t* lens_out, uint32_t flags, int32_t* dev_err,
                                    kvd_stream_t stream) {
    if (dtype != KVD_F16 && dtype != KVD_BF16) return KVD_ERR_INVALID_ARG;
    if (kvd_status s = validate_q4_cache(cache)) return s;
    if (batch < 0 || q < 0 || batch > cache->batch) return KVD_ERR_INVALID_ARG;
    if (batch == 0 || q == 0) return KVD_OK;
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return KVD_ERR_INVALID_ARG;
    if (lens_out && (lens_out == lens_in || lens_out == counts)) return KVD_ERR_INVALID_ARG;
    Q4RowsParams p = {};
    if (kvd_status s = rows_params(p, cache, batch, q)) return s;
    p.in[0] = static_cast<const uint8_t*>(k_new);
    p.in[1] = static_cast<const uint8_t*>(v_new);
    p.pos0 = lens_in;
    p.counts = counts;
    p.lens_out = lens_out;
    p.dev_err = dev_err;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool pdl = (flags & KVD_FLAG_PDL) != 0;
    return dtype == KVD_BF16 ? run_append<__nv_bfloat16>(p, batch, st, pdl)
                             : run_append<__half>(p, batch, st, pdl);
}

extern "C" kvd_status kvd_q4_dequant(kvd_dtype dtype, const kvd_q4_cache* cache, int32_t batch,
                                     int32_t n, void* k_out, void* v_out, const int32_t* pos0,
                                     uint32_t flags, int32_t* dev_err, kvd_stream_t stream) {
    if (dtype != KVD_F16 && dtype != KVD_BF16) return KVD_ERR_INVALID_ARG;
    if (kvd_status s = validate_q4_cache(cache)) return s;
    if (batch < 0 || n < 0 || batch > cache->batch) return KVD_ERR_INVALID_ARG;
    if (batch == 0 || n == 0 || (!k_out && !v_out)) return KVD_OK;
    if (!aligned16(k_out) || !aligned16(v_out)) return KVD_ERR_INVALID_ARG;
    Q4RowsParams p = {};
    if (kvd_status s = rows_params(p, cache, batch, n)) return s;
    p.out[0] = static_cast<uint8_t*>(k_out);
    p.out[1] = static_cast<uint8_t*>(v_out);
    p.pos0 = pos0;
    p.dev_err = dev_err;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool pdl = (flags & KVD_FLAG_PDL) != 0;
    return dtype == KVD_BF16 ? run_dequant<__nv_bfloat16>(p, batch, st, pdl)
                             : run_dequant<__half>(p, batch, st, pdl);
}
