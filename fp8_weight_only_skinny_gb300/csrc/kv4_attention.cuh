// kv4_attention.cuh -- what the attention kernels over the 4-bit cache share:
// their parameters, the split of the work and the softmax's scale.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/skinny.h"
#include "cluster.cuh"
#include "kv4.cuh"

namespace sk {
namespace attn {

constexpr int WARPS = 4;
constexpr int CT = WARPS * 32;         // threads of the register kernels' CTAs
constexpr int STEP = 32;               // positions per warp step: two records
// Positions per CTA step, the unit of the work split.  (Split by single steps
// the CTAs' shares are more even, but more of them take parts of two segments:
// 52 -> 69 us on 23 ragged sequences of 8 heads.)
constexpr int TILE = WARPS * STEP;
constexpr int NROW = 8;                // query rows per n8 tile
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// Each row's weights are taken against a base, a score in the units of q . k:
// p = 2^((s - base) c) with c = scale * key scale * log2 e.  Any base gives the
// same quotient, so it is P_SHIFT / c below a maximum the row had earlier and is
// moved only when a score passes that maximum by more than SLACK / c (then the
// sums so far are scaled).  Most steps need neither the row's maximum across
// lanes nor a rescaling.  The base is subtracted before anything is scaled: the
// difference of neighbouring numbers is exact, so that weights near the maximum
// are right whatever the scores' size (c s - c base, each rounded by itself, is
// off by up to 2^5 where the scores are 2^28, and the FP16 weights overflow or
// vanish); two scores at a time, an add and a multiply of f32x2, that costs about
// what an fma each did (0.96 to 1.02 of the call, over seventeen shapes).  A base is rounded
// such that (s - base) c is between 0 and P_SHIFT for the maximum, and moves when
// that exceeds P_SHIFT + SLACK.  The p go to the second product in FP16, at most
// 2^15 and normal down to 2^-21 of the maximum's (2^-32 is the rounding of the
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
    float2 *norm;              // per row, where weights are accumulated: minus its base, log2 of the sum under it
    unsigned int *err;
    int stall;                 // issue no copies (sk_inject_wait_timeout)
    int pages, heads, recs, width, cap;   // recs: records per page; cap: positions the table can hold
    int limit, window, sinks;  // of a window: positions the table can hold (cap: that are looked at), see Seen
    int B, M, G, RT, ctas;     // G: query heads per kv head; RT: row tiles
    float c, shift, reach, vg; // scale * key scale * log2 e; P_SHIFT / c; (P_SHIFT + SLACK) / c; value scale
    sk::Div by_recs;
};

// Rows keep minus their base.  NO_BASE: no score seen yet; any score passes it,
// and the sums under it are zero.
constexpr float NO_BASE = 3.402823466e38f;
// Minus the base for a maximum of m, rounded so that the base is at or above
// P_SHIFT / c below m (and at most m: m itself is among the numbers rounded to).
__device__ __forceinline__ float neg_base(const AttnParams &p, float m) { return __fadd_rd(p.shift, -m); }
// Whether the score s makes its row's base move.
__device__ __forceinline__ bool passes(const AttnParams &p, float s, float neg) { return s + neg > p.reach; }
// A weight of the score s.
__device__ __forceinline__ float weight(const AttnParams &p, float s, float neg) { return ex2((s + neg) * p.c); }
// Two weights at a time, and two with a factor of 2^-g each.
__device__ __forceinline__ float2 weights2(const AttnParams &p, float s0, float s1, float n0, float n1) {
    float2 d;
    asm("{ .reg .b64 s, n, c; mov.b64 s, {%2, %3}; mov.b64 n, {%4, %5}; mov.b64 c, {%6, %6};\n\t"
        "add.rn.f32x2 s, s, n; mul.rn.f32x2 s, s, c; mov.b64 {%0, %1}, s; }"
        : "=f"(d.x), "=f"(d.y) : "f"(s0), "f"(s1), "f"(n0), "f"(n1), "f"(p.c));
    return make_float2(ex2(d.x), ex2(d.y));
}
__device__ __forceinline__ float2 weights2(const AttnParams &p, float s0, float s1, const float2 &n, const float2 &neg_g) {
    float2 d;
    asm("{ .reg .b64 s, n, c, g; mov.b64 s, {%2, %3}; mov.b64 n, {%4, %5}; mov.b64 c, {%6, %6}; mov.b64 g, {%7, %8};\n\t"
        "add.rn.f32x2 s, s, n; fma.rn.f32x2 s, s, c, g; mov.b64 {%0, %1}, s; }"
        : "=f"(d.x), "=f"(d.y) : "f"(s0), "f"(s1), "f"(n.x), "f"(n.y), "f"(p.c), "f"(neg_g.x), "f"(neg_g.y));
    return make_float2(ex2(d.x), ex2(d.y));
}
// What sums under one base are multiplied by to stand under another.
__device__ __forceinline__ float rebase(const AttnParams &p, float from, float to) { return ex2((from - to) * p.c); }
// What a row's statistics, the sum l of its weights under a base, are needed
// for later: the natural log of the sum, and for the accumulated weights base
// and sum apart (the log holds no fraction where it is large).
__device__ __forceinline__ void write_stats(const AttnParams &p, long long row, float base, float l) {
    const float lg = __log2f(l);
    if (p.lse) p.lse[row] = l == 0.f ? NEG_INF : fmaf(base, p.c, lg) * LN2;
    if (p.norm) p.norm[row] = l == 0.f ? make_float2(0.f, -NEG_INF) : make_float2(-base, lg);
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

// The positions of a sequence that its rows look at.  With a window: those before
// `sinks` and those from the first row's window on, numbered without the whole
// records in between: records from `gap` on lie `skip` records further.  Row m
// sees the number j if j < lim and (j < sinks or j >= lim - window), where lim =
// len - (M - 1 - m); a gap's ends lie at or below every row's lim - window.
template <bool WIN>
struct Seen {
    int len, gap, skip;
    __device__ __forceinline__ Seen(const AttnParams &p, int b) : gap(0), skip(0) {
        if constexpr (WIN) {
            len = min(max(p.lens[b], 0), p.limit);
            gap = (min(p.sinks, len) + sk::KV4_REC - 1) / sk::KV4_REC;
            skip = max(0, max(0, len - (p.M - 1) - p.window) / sk::KV4_REC - gap);
            len -= skip * sk::KV4_REC;
        } else {
            len = length_of(p, b);
        }
    }
    __device__ __forceinline__ int record(int r) const { return WIN && r >= gap ? r + skip : r; }
};
__device__ __forceinline__ int tiles_of(int len) { return (len + TILE - 1) / TILE; }

// The CTA's share of all (sequence, head, row tile, position tile) in that
// order: the T tiles go to P = min(ctas, T) CTAs, T / P each and one more to the
// first T mod P, so every CTA reads the same number of positions whatever the
// lengths.  (The caller has checked that T fits 31 bits.)
struct Share {
    int t, end;                // this CTA's next tile and the end of its share
    int parts, base, extra;    // P, T / P, T mod P
    int b, off;                // the sequence of tile t; its index among that sequence's tiles
};
__device__ __forceinline__ int first_tile(const Share &s, int cta) { return cta * s.base + min(cta, s.extra); }
__device__ __forceinline__ int cta_of(const Share &s, int tile) {
    const int large = s.extra * (s.base + 1);
    return tile < large ? tile / (s.base + 1) : s.extra + (tile - large) / s.base;
}

template <typename T>
__device__ __forceinline__ T inclusive_scan(T x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// per_len: segments of a sequence; sm: a word per warp and two more.
template <bool WIN = false>
__device__ __forceinline__ Share share_of(const AttnParams &p, int per_len, int *sm) {
    auto length = [&](int b) { return Seen<WIN>(p, b).len; };
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nw = blockDim.x >> 5, c = blockIdx.x;
    Share s;
    auto split = [&](int total) {
        s.parts = min(total, p.ctas);
        s.base = s.parts ? total / s.parts : 0;
        s.extra = total - s.base * s.parts;
        const bool in = c < s.parts;
        s.t = in ? first_tile(s, c) : 0;
        s.end = in ? first_tile(s, c + 1) : 0;
    };
    if (p.B <= 32) {
        // every warp by itself, a lane a sequence
        const int mine = lane < p.B ? tiles_of(length(lane)) * per_len : 0;
        const int x = inclusive_scan(mine, lane);
        split(__shfl_sync(0xffffffffu, x, 31));
        const unsigned int past = __ballot_sync(0xffffffffu, x > s.t);
        s.b = past ? __ffs(past) - 1 : 0;
        s.off = s.t - __shfl_sync(0xffffffffu, x - mine, s.b);
        return s;
    }
    const int each = (p.B + int(blockDim.x) - 1) / int(blockDim.x);
    const int lo = min(p.B, tid * each), hi = min(p.B, lo + each);
    int mine = 0;
    for (int b = lo; b < hi; ++b) mine += tiles_of(length(b)) * per_len;
    const int x = inclusive_scan(mine, lane);
    if (lane == 31) sm[wid] = x;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < wid) before += sm[w];
        total += sm[w];
    }
    split(total);
    before += x - mine;
    if (s.t < s.end && s.t >= before && s.t < before + mine) {
        int b = lo, left = s.t - before;
        for (; b + 1 < hi; ++b) {
            const int n = tiles_of(length(b)) * per_len;
            if (left < n) break;
            left -= n;
        }
        sm[nw] = b;
        sm[nw + 1] = left;
    }
    __syncthreads();
    s.b = sm[nw];
    s.off = sm[nw + 1];
    return s;
}

// The tensor-core kernel for many rows (kv4_attention_tc.cu): head size 128, up
// to TC_MOST query rows of a kv head at a time, two CTAs per SM.
constexpr int TC_MOST = 96, TC_CTAS = 2;
// Rows per tile it takes `rows` in, and how many tiles.
int tc_rows(int rows, int *tiles);
cudaError_t launch_tc(AttnParams &p, int rows_per_tile, cudaStream_t s);

// The kernel for chunks of any length (kv4_chunk.cu), for M rows of every sequence
// with `limit`, `window` and `sinks` set; up to CHUNK_SEQS sequences.
constexpr int CHUNK_SEQS = 16383;
sk_status chunk_rows(const AttnParams &a, int head_dim, unsigned char *scratch, int sms, cudaStream_t s);

}  // namespace attn
}  // namespace sk
