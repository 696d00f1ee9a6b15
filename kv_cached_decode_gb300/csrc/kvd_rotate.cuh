// kvd_rotate.cuh -- rotation of head rows by a kvd_rope_spec, for the kernels that read rows of
// 64 values, rotate them and write them somewhere else (rope_scaled.cu, paged_append.cu).
//
// A row is held by eight lanes, lane c with dims 8c..8c+7, so a warp has four rows of one token.
// Pair i of rot/2 pairs turns by pos * freq[i]; freq is a 64-bit fixed-point fraction of a turn, so
// pos * freq modulo 2^64 is the angle with the whole turns dropped, exact to pos * 2^-53. Lane i
// forms cos and sin of pair i once per token, and each lane takes the eight it needs by shuffles:
//   y[e] = x[e] C[e] + p[e] S[e],  p the other value of the pair
// interleaved pairs lie in one lane, halves rot/16 lanes apart (rot is a multiple of 16).
#pragma once

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {

// Of the calling lane, for one token.
struct Turn {
    float c[8], s[8];
    bool turns;  // whether the lane's dims do
};

template <bool INTER>
__device__ __forceinline__ void make_turn(Turn& t, uint64_t freq, int64_t pos, int rot, float mag) {
    const int lane = threadIdx.x & 31, ch = lane & 7;
    t.turns = 8 * ch < rot;
    float sn, cs;
    // half turns in [-1, 1)
    sincospif((float)(int32_t)((uint64_t)pos * freq >> 32) * 0x1p-31f, &sn, &cs);
    sn *= mag;
    cs *= mag;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // (rot/2 is a power of two or 24: a subtraction, not a remainder)
        int i = INTER ? 4 * ch + e / 2 : 8 * ch + e;
        if (!INTER && i >= rot / 2) i -= rot / 2;
        const float c = __shfl_sync(0xffffffffu, cs, i & 31);
        const float s = __shfl_sync(0xffffffffu, sn, i & 31);
        t.c[e] = c;
        t.s[e] = (INTER ? (e & 1) != 0 : 8 * ch >= rot / 2) ? s : -s;
    }
}

// This lane's chunk of a row, rotated; all lanes of the warp call it. Dims from rot on keep their
// bits.
template <typename T, bool INTER>
__device__ __forceinline__ uint4 rotate_chunk(const uint4& x, const Turn& t, int rot) {
    const int lane = threadIdx.x & 31, ch = lane & 7;
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[4];
    // the lane with the other halves (chunks not rotated read their own)
    const int far = rot >> 4;
    const int from = 8 * ch >= rot ? lane : ch < far ? lane + far : lane - far;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float2 a = Half16<T>::to_f2(in[w]);
        float2 y;
        if (INTER) {
            y = make_float2(fmaf(a.x, t.c[2 * w], a.y * t.s[2 * w]),
                            fmaf(a.y, t.c[2 * w + 1], a.x * t.s[2 * w + 1]));
        } else {
            const float2 b = Half16<T>::to_f2(__shfl_sync(0xffffffffu, in[w], from));
            const Pair p = mul2(Pair(b.x, b.y), Pair(t.s[2 * w], t.s[2 * w + 1]));
            y = fma2(Pair(a.x, a.y), Pair(t.c[2 * w], t.c[2 * w + 1]), p).get();
        }
        out[w] = Half16<T>::from_f2(y.x, y.y);
    }
    return t.turns ? make_uint4(out[0], out[1], out[2], out[3]) : x;
}

// Host: the scaled frequencies of a spec as fractions of a turn, in units of 2^-64 turns
// (rope_scaled.cu). false: out of range.
struct RopeTurns {
    uint64_t freq[32];
    int32_t rot, inter;
    float mag;
};
kvd_status rope_turns(const kvd_rope_spec* spec, RopeTurns* t);

}  // namespace kvd
