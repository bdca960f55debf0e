// kv4_attention.cuh -- what the attention kernels over the 4-bit cache share:
// their parameters, the split of the work and the softmax's scale.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "kv4.cuh"

namespace sk {
namespace attn {

constexpr int WARPS = 4;
constexpr int CT = WARPS * 32;         // threads of the register kernels' CTAs
constexpr int STEP = 32;               // positions per warp step: two records
constexpr int TILE = WARPS * STEP;     // positions per CTA step, the unit of the work split
constexpr int NROW = 8;                // query rows per n8 tile
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// Each row's weights are taken against a reference r, p = 2^(z - r + P_SHIFT):
// any r gives the same quotient, so r is a maximum the row had earlier and is
// moved only when a score passes it by more than SLACK (then the sums so far
// are scaled).  Most steps need neither the row's maximum across lanes nor a
// rescaling.  The p go to the second product in FP16, at most 2^(P_SHIFT +
// SLACK) = 2^15 and normal down to 2^-21 of r's (2^-32 is the rounding of the
// smaller ones).  Their rounding (2^-11 relative at most, independent from
// position to position) is of the size of the output's own rounding to FP16;
// the sum of the weights is taken from the unrounded FP32 values.
constexpr float P_SHIFT = 7.f, SLACK = 8.f;

struct AttnParams {
    const __half *q;
    long long q_stride;        // elements between query rows
    const uint8_t *cache;
    const int32_t *table, *lens;
    __half *out;
    float *lse;
    const float *acc_in;
    float *acc_out;
    float *part_o, *part_ml;   // per partial slot: [ROWS][D] sums, [ROWS][2] (maximum, sum)
    int2 *seg;                 // per segment: first CTA, partial slots (0: written whole)
    unsigned int *err;
    int pages, heads, recs, width, cap;   // recs: records per page; cap: positions the table can hold
    int B, M, G, RT, ctas;     // G: query heads per kv head; RT: row tiles
    float scale2, vg;          // scale * key scale * log2 e; value scale
    sk::Div by_recs;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two scale codes -> f16x2.  Scales are written non-negative; a NaN code (only
// memory that no position was written to can hold one) becomes zero, so that a
// weight of zero times what lies there is zero.
__device__ __forceinline__ uint32_t scale_pair(uint32_t codes) {
    const uint32_t s = sk::e4m3x2_h_to_f16x2(uint16_t(codes));
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(s), "r"(0u));
    return d;
}

__device__ __forceinline__ int length_of(const AttnParams &p, int b) { return min(max(p.lens[b], 0), p.cap); }
__device__ __forceinline__ int tiles_of(int len) { return (len + TILE - 1) / TILE; }

// The CTA's share of all (sequence, head, row tile, position tile) in that
// order: tiles [T c / P, T (c + 1) / P) of T for CTA c of P = min(ctas, T),
// so every CTA reads the same number of positions whatever the lengths.
struct Share {
    long long total, t, end;   // tiles in all, this CTA's next and end
    int parts, b;              // P; the sequence of tile t
    long long off;             // tile t's index among the tiles of sequence b
};

__device__ __forceinline__ Share share_of(const AttnParams &p, int per_len, long long *sm /* CT / 32 + 4 */) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nw = blockDim.x >> 5;
    const int each = (p.B + int(blockDim.x) - 1) / int(blockDim.x);
    const int lo = min(p.B, tid * each), hi = min(p.B, lo + each);
    long long mine = 0;
    for (int b = lo; b < hi; ++b) mine += (long long)tiles_of(length_of(p, b)) * per_len;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sm[wid] = x;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < wid) before += sm[w];
        total += sm[w];
    }
    __syncthreads();
    Share s;
    s.total = total;
    s.parts = int(total < p.ctas ? total : p.ctas);
    const bool in = int(blockIdx.x) < s.parts;
    s.t = in ? total * blockIdx.x / s.parts : 0;
    s.end = in ? total * (blockIdx.x + 1) / s.parts : 0;
    before += x - mine;
    if (in && s.t >= before && s.t < before + mine) {
        int b = lo;
        long long left = s.t - before;
        for (; b + 1 < hi; ++b) {
            const long long n = (long long)tiles_of(length_of(p, b)) * per_len;
            if (left < n) break;
            left -= n;
        }
        sm[0] = b;
        sm[1] = left;
    }
    __syncthreads();
    s.b = int(sm[0]);
    s.off = sm[1];
    return s;
}

// The tensor-core kernel for many rows (kv4_attention_tc.cu): head size 128, up
// to TC_MOST query rows of a kv head at a time, two CTAs per SM.
constexpr int TC_MOST = 96, TC_CTAS = 2;
// Rows per tile it takes `rows` in, and how many tiles.
int tc_rows(int rows, int *tiles);
cudaError_t launch_tc(AttnParams &p, int rows_per_tile, cudaStream_t s);

}  // namespace attn
}  // namespace sk
