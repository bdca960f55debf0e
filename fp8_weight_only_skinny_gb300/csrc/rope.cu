// rope.cu -- what lies between the fused qkv projection and the attention: the
// norm of each query and key head, its rotation by position, and (kv4_append_rope)
// the keys' and values' way into the 4-bit cache, in one pass.
//
// For a head x of D components, with r = 1 / sqrt(mean x^2 + eps):
//     y_i = x_i r w_i                                   (without weights: y = x)
// and for each of the R / 2 pairs (a, b) of the first R components
//     (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t),
//     t = 2 pi frac(position F / 2^64),
// F the pair's frequency as a fraction of a turn in units of 2^-64: the product
// modulo 2^64 is exact, so that the angle is right at any position.
//
// Bound by DRAM and instructions together: 8191 tokens of 32 + 8 heads of 128, interleaved
// and normed, 31 us (168 MB, 5.4 TB/s); 16387 tokens of 24 + 2 + 2 heads of 256 to the
// cache 99 us (446 MB, 4.5 TB/s; issue 64 %, DRAM 52 %). One token 2.9 us.
// Two components an instruction, f32x2, gained nothing: 99 -> 105 us, 31 -> 31. At 64
// registers a thread the append's kernels spill 28 to 56 bytes, the rotation's none.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/skinny.h"
#include "internal.h"
#include "kv4.cuh"
#include "launch_util.cuh"
#include "quant.cuh"

namespace {

constexpr int RT = 128;        // threads per CTA
constexpr int MIN_CTAS = 8;    // per SM (64 registers a thread)
// Units whose loads are in flight, and the most a warp takes: as many as keep
// every SM full once, since a warp forms its angles once (8191 tokens, 32 + 8 heads
// of 128: up to 32 units 33 us, 8 37, 4 45). Three units ahead and eight CTAs: 16387
// tokens of 24 + 2 + 2 heads of 256 to the cache 99 us; four and eight 106, four and
// seven 104, three and ten (48 registers) 119, two units of keys a warp 110.
constexpr int AHEAD = 3, MOST_UNITS = 32;

struct RopeParams {
    const __half *q, *k, *v;
    long long q_stride, k_stride, v_stride;      // elements between tokens
    __half *q_out, *k_out;
    long long qo_stride, ko_stride;
    const int32_t *positions;
    const uint64_t *freqs;
    const float *qw, *kw;                        // null: no norm
    double eps, amplitude;
    int tokens, hq, hk, R;
    int uq, uk;                                  // units (a warp's heads) of the queries and of the keys
    int per, chunks, kper, kchunks;              // units per warp and warps per token, for each
    unsigned int ratio;                          // CTAs of keys among all, in units of 2^-32 (without a cache: of queries)
    // kv4_append_rope
    const int32_t *slots;
    uint8_t *cache;
    float gk, gv;
    int pages, recs, page;
};

// A number of 24 bits that rounds to a format of fewer bits as v does: v cut,
// its last bit set where something was cut off.
__device__ __forceinline__ float odd_float(double v) {
    const float f = __double2float_rz(v);
    return double(f) == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The fraction of a turn at a position, in units of 2^-64 from -1/2 to 1/2.
__device__ __forceinline__ long long turn_of(int position, uint64_t f) {
    return (long long)(uint64_t(int64_t(position)) * f);
}

// A lane holds eight neighbouring components of a head, L = D / 8 lanes hold a
// head, a warp 32 / L heads (a unit). In the half layout a component's partner is
// R / 2 further or back: lane +- R / 16; interleaved pairs are a lane's own.
template <int D, bool INTER>
struct Lane {
    static constexpr int L = D / 8, HW = 32 / L;
    static constexpr int NP = INTER ? 4 : 8;             // angles of a lane
    int l, head, c0, partner;                            // lane in the head, head in the unit, first component, partner lane
    int away;                                            // from a component to its partner (half layout)
    bool rotated, upper;
    __device__ Lane(int lane, int R) {
        l = lane % L;
        head = lane / L;
        c0 = 8 * l;
        rotated = c0 < R;
        upper = !INTER && rotated && c0 >= R / 2;
        away = !rotated ? 0 : upper ? -(R / 2) : R / 2;
        partner = INTER ? lane : lane + away / 8;
    }
    // of component e of the lane: its pair, its partner, and whether it is the pair's second
    __device__ int pair(int e, int R) const { return INTER ? (c0 + e) / 2 : c0 + e - (upper ? R / 2 : 0); }
    __device__ int other(int e) const { return INTER ? (rotated ? (c0 + e) ^ 1 : c0 + e) : c0 + e + away; }
    __device__ bool second(int e) const { return INTER ? (e & 1) : upper; }
};

// Cosines and sines of a lane's angles, times the amplitude.
template <int D, bool INTER>
__device__ __forceinline__ void angles(const RopeParams &p, const Lane<D, INTER> &ln, int position,
                                       float (&c)[Lane<D, INTER>::NP], float (&s)[Lane<D, INTER>::NP]) {
    const float amplitude = float(p.amplitude);
    // Half layout: the two lanes of a pair of components need the same eight angles and form four each.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float cj = 1.f, sj = 0.f;
        if (ln.rotated) {
            // the upper 32 bits: off by 2^-32 of a turn
            const int e = INTER ? 2 * j : j + (ln.upper ? 4 : 0);
            sincospif(float(int(turn_of(position, p.freqs[ln.pair(e, p.R)]) >> 32)) * 0x1p-31f, &sj, &cj);
            cj *= amplitude;
            sj *= amplitude;
        }
        if constexpr (INTER) {
            c[j] = cj;
            s[j] = sj;
        } else {
            const float co = __shfl_sync(0xffffffffu, cj, ln.partner), so = __shfl_sync(0xffffffffu, sj, ln.partner);
            c[j] = ln.upper ? co : cj;
            s[j] = ln.upper ? so : sj;
            c[j + 4] = ln.upper ? cj : co;
            s[j + 4] = ln.upper ? sj : so;
        }
    }
}

// Cosines and signed sines with the weights of the component and of its partner:
// a component becomes (x cw + partner sw) r.
template <int D, bool INTER>
__device__ __forceinline__ void weigh(const Lane<D, INTER> &ln, const float *weight, const float (&c)[Lane<D, INTER>::NP],
                                      const float (&s)[Lane<D, INTER>::NP], float (&cw)[8], float (&sw)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int j = INTER ? e / 2 : e;
        cw[e] = c[j] * (weight ? weight[ln.c0 + e] : 1.f);
        sw[e] = (ln.second(e) ? s[j] : -s[j]) * (weight ? weight[ln.other(e)] : 1.f);
    }
}

// The norm's factor of a head.
template <int L>
__device__ __forceinline__ float norm_of(const RopeParams &p, const float (&x)[8]) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return rsqrtf(ss * (1.f / (8 * L)) + float(p.eps));
}

// The partners of a lane's components.
template <int D, bool INTER>
__device__ __forceinline__ void partners(const Lane<D, INTER> &ln, const uint4 &mine, const float (&x)[8], float (&xp)[8]) {
    if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = x[e ^ 1];
    } else {
        sk::unpack8(make_uint4(__shfl_sync(0xffffffffu, mine.x, ln.partner), __shfl_sync(0xffffffffu, mine.y, ln.partner),
                               __shfl_sync(0xffffffffu, mine.z, ln.partner), __shfl_sync(0xffffffffu, mine.w, ln.partner)),
                    xp);
    }
}

// ------------------------------------------------------------- the keys ----

// The norm's factor in 64 bits.
template <int L>
__device__ __noinline__ double norm64(double eps, const uint4 raw) {
    float x[8];
    sk::unpack8(raw, x);
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += double(x[e]) * double(x[e]);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return 1.0 / sqrt(ss / (8 * L) + eps);
}

// A component in 64 bits, without the norm's factor: a and b are the component
// and its partner with their weights.
__device__ __noinline__ double turned64(double a, double b, long long turn, double amplitude, bool rotated, bool second) {
    if (!rotated) return a;
    double s, c;
    sincospi(double(turn) * 0x1p-63, &s, &c);
    return (second ? a * c + b * s : a * c - b * s) * amplitude;
}

// The codes of a key's eight components and its block's scale, from y, of which
// component e is off by at most err[e]; the quotients add less than |y| 2^-21.
// Where both ends of every interval have one code, that is the code of exact
// arithmetic. Otherwise the components in doubt alone are taken in 64 bits: those
// that may be the block's largest, if the scale is open, then those whose codes
// are (one component in 10^5: the 64-bit unit has a 64th of the rate). All lanes of
// a warp come here.
template <int D, bool INTER>
__device__ __forceinline__ void key_codes(const RopeParams &p, const Lane<D, INTER> &ln, const uint4 &raw, int position,
                                          const float (&x)[8], const float (&xp)[8], const float (&y)[8],
                                          const float (&err)[8], uint32_t &codes, uint32_t &sc) {
    const float G = p.gk;
    float b = 0.f, w = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        b = fmaxf(b, fabsf(y[e]));
        w = fmaxf(w, err[e]);
    }
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 1));
    w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 1));
    w = fmaf(b, 0x1p-21f, w);
    const uint32_t ends = sk::e4m3x2_rn(__fdiv_rn(__fdiv_rn(b - w, 6.f), G), __fdiv_rn(__fdiv_rn(b + w, 6.f), G));
    sc = ends & 0xFFu;
    const bool open = sc != ends >> 8;
    auto quotients = [&](uint32_t &lo, uint32_t &hi) {
        const float S = sk::e4m3_value(sc);
        const float r = S == 0.f ? 0.f : __frcp_rn(__fmul_rn(S, G));
        lo = hi = 0u;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float w0 = fmaf(fabsf(y[e]), 0x1p-21f, err[e]), w1 = fmaf(fabsf(y[e + 1]), 0x1p-21f, err[e + 1]);
            lo |= sk::e2m1x2_rn((y[e] - w0) * r, (y[e + 1] - w1) * r) << (4 * e);
            hi |= sk::e2m1x2_rn((y[e] + w0) * r, (y[e + 1] + w1) * r) << (4 * e);
        }
    };
    uint32_t hi;
    quotients(codes, hi);
    if (__all_sync(0xffffffffu, !open && codes == hi)) return;

    const float *wt = p.kw;
    const double r64 = wt ? norm64<Lane<D, INTER>::L>(p.eps, raw) : 1.0;
    auto exact = [&](int e) {          // component e, a number that differs from lane to lane
        float a = 0.f, o = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i == e) {
                a = x[i];
                o = xp[i];
            }
        const double wa = wt ? double(wt[ln.c0 + e]) : 1.0, wo = wt ? double(wt[ln.other(e)]) : 1.0;
        const long long turn = ln.rotated ? turn_of(position, p.freqs[ln.pair(e, p.R)]) : 0;
        return turned64(a * wa, o * wo, turn, p.amplitude, ln.rotated, ln.second(e)) * r64;
    };
    if (__any_sync(0xffffffffu, open)) {
        unsigned int todo = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (open && fabsf(y[e]) + err[e] >= b - w) todo |= 1u << e;
        double top = 0.0;
        while (__any_sync(0xffffffffu, todo)) {
            const double v = exact(todo ? __ffs(todo) - 1 : 0);
            if (todo) top = fmax(top, fabs(v));
            todo &= todo - 1u;
        }
        top = fmax(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (open) sc = sk::e4m3x2_rn(odd_float(top / (6.0 * double(G))), 0.f) & 0xFFu;
        quotients(codes, hi);
    }
    unsigned int todo = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (((codes ^ hi) >> (4 * e)) & 15u) todo |= 1u << e;
    const double unit = double(sk::e4m3_value(sc)) * double(G);
    while (__any_sync(0xffffffffu, todo)) {
        const int e = todo ? __ffs(todo) - 1 : 0;
        const double v = exact(e);
        const float f = unit == 0.0 ? copysignf(0.f, float(v)) : odd_float(v / unit);
        if (todo) codes = (codes & ~(15u << (4 * e))) | ((sk::e2m1x2_rn(f, 0.f) & 15u) << (4 * e));
        todo &= todo - 1u;
    }
}

// A value's block: the steps of kv4_append.
__device__ __forceinline__ void value_codes(const float (&x)[8], float G, uint32_t &codes, uint32_t &sc) {
    float b = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) b = fmaxf(b, fabsf(x[e]));
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 1));
    sc = sk::e4m3x2_rn(__fdiv_rn(__fdiv_rn(b, 6.f), G), 0.f) & 0xFFu;
    const float S = sk::e4m3_value(sc);
    codes = 0u;
    if (S == 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (__float_as_uint(x[e]) >> 31) codes |= 0x8u << (4 * e);
    } else {
        const float unit = __fmul_rn(S, G), r = __frcp_rn(unit);
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            codes |= sk::quotient_codes<0x1FFFFFu>(x[e], x[e + 1], unit, r, sk::e2m1x2_rn) << (4 * e);
    }
}

// One token's units u0 .. u1 of x: normed, rotated, to `out`. AHEAD units' loads
// are in flight, two of them worked on at a time.
template <int D, bool INTER>
__device__ __forceinline__ void rotate(const RopeParams &p, const Lane<D, INTER> &ln, int position, const __half *x,
                                       __half *out, const float *weight, int heads, int u0, int u1) {
    using LN = Lane<D, INTER>;
    constexpr int HW = LN::HW;
    auto fetch = [&](int u) {
        const int h = u * HW + ln.head;
        return u < u1 && h < heads ? *reinterpret_cast<const uint4 *>(x + h * D + ln.c0) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 raw[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) raw[j] = fetch(u0 + j);
    float cw[8], sw[8];
    {
        float c[LN::NP], s[LN::NP];
        angles<D, INTER>(p, ln, position, c, s);
        weigh<D, INTER>(ln, weight, c, s, cw, sw);
    }
#pragma unroll 1
    for (int i = u0; i < u1; i += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (i + j >= u1) break;
            const uint4 mine = raw[j];
            raw[j] = fetch(i + j + AHEAD);
            float v[8], vp[8];
            sk::unpack8(mine, v);
            const float r = weight ? norm_of<LN::L>(p, v) : 1.f;
            partners<D, INTER>(ln, mine, v, vp);
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const __half2 z = __floats2half2_rn(fmaf(v[e], cw[e], vp[e] * sw[e]) * r,
                                                    fmaf(v[e + 1], cw[e + 1], vp[e + 1] * sw[e + 1]) * r);
                y[e / 2] = *reinterpret_cast<const uint32_t *>(&z);
            }
            const int h = (i + j) * HW + ln.head;
            if (h < heads) *reinterpret_cast<uint4 *>(out + h * D + ln.c0) = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
}

// One token's keys and values of a unit of heads, to the cache.
template <int D, bool INTER>
__device__ __forceinline__ void append(const RopeParams &p, const Lane<D, INTER> &ln, int token, int unit) {
    using LN = Lane<D, INTER>;
    const int h = unit * LN::HW + ln.head;
    uint4 key = make_uint4(0u, 0u, 0u, 0u), value = key;
    if (h < p.hk) {
        key = *reinterpret_cast<const uint4 *>(p.k + token * p.k_stride + h * D + ln.c0);
        value = *reinterpret_cast<const uint4 *>(p.v + token * p.v_stride + h * D + ln.c0);
    }
    const int slot = p.slots[token], position = p.positions ? p.positions[token] : 0;
    const int page = slot / p.page, at = slot - page * p.page, b = ln.l >> 1, pos = at & 15;
    const bool kept = h < p.hk && slot >= 0 && page < p.pages;
    uint8_t *const rec = p.cache + (kept ? ((size_t(page) * p.hk + h) * p.recs + (at >> 4)) * sk::kv4_rec_bytes(D) : 0);
    float cw[8], sw[8], wm[8], wo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        wm[e] = p.kw ? p.kw[ln.c0 + e] : 1.f;
        wo[e] = p.kw ? p.kw[ln.other(e)] : 1.f;
    }
    {
        float c[LN::NP], s[LN::NP];
        angles<D, INTER>(p, ln, position, c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int j = INTER ? e / 2 : e;
            cw[e] = c[j] * wm[e];
            sw[e] = (ln.second(e) ? s[j] : -s[j]) * wo[e];
            wm[e] = fabsf(wm[e]);
            wo[e] = ln.rotated ? fabsf(wo[e]) : 0.f;
        }
    }
    uint32_t codes, sc;
    float x[8];
    sk::unpack8(value, x);
    value_codes(x, p.gv, codes, sc);
    if (kept) {
        *reinterpret_cast<uint32_t *>(rec + sk::kv4_code_at<true>(D, pos, b) + 4 * (ln.l & 1)) = codes;
        if (!(ln.l & 1)) rec[sk::kv4_scale_at<true>(D, pos, b)] = uint8_t(sc);
    }
    sk::unpack8(key, x);
    float xp[8], y[8], err[8];
    const float r = p.kw ? norm_of<LN::L>(p, x) : 1.f;
    partners<D, INTER>(ln, key, x, xp);
    // In units of u = 2^-24 of the two terms a cosine or sine of one would leave: the norm's sum of 13 roundings and
    // eps's 2, halved by the root, and 4 of rsqrtf's two last places, 11.5; an angle's 3.2 (pi times its rounding), one
    // of sincospif's last places, amplitude's 2, the weight's 1; products, sum and factor 3: 21.7, of 24 (without a
    // norm 10.2, of 12).
    const float u = (p.kw ? 24.f : 12.f) * 0x1p-24f * r * fmaxf(1.f, fabsf(float(p.amplitude)));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // (a component that is not turned keeps the sign of its zero)
        y[e] = (ln.rotated ? fmaf(x[e], cw[e], xp[e] * sw[e]) : x[e] * cw[e]) * r;
        err[e] = fmaf(fabsf(x[e]), wm[e], fabsf(xp[e]) * wo[e]) * u;
    }
    key_codes<D, INTER>(p, ln, key, position, x, xp, y, err, codes, sc);
    if (kept) {
        *reinterpret_cast<uint32_t *>(rec + sk::kv4_code_at<false>(D, pos, b) + 4 * (ln.l & 1)) = codes;
        if (!(ln.l & 1)) rec[sk::kv4_scale_at<false>(D, pos, b)] = uint8_t(sc);
    }
}

// A warp takes up to `per` units of one token's queries, so that the angles are
// formed once for all of them, or up to `kper` of its keys (with APPEND one, and its
// values). The CTAs
// of keys are spread evenly among those of queries: the ones wait for memory, the
// others compute (16387 tokens of 24 + 2 + 2 heads of 256: one kind after the other
// 132 us, mixed 111).
template <int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(RT, MIN_CTAS) rope_kernel(const __grid_constant__ RopeParams p) {
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    // of the first i CTAs, floor(i ratio / 2^32) are of keys
    const unsigned int before = APPEND ? (unsigned long long)blockIdx.x * p.ratio >> 32
                                       : blockIdx.x < p.ratio ? 0 : blockIdx.x - p.ratio,
                       upto = ((unsigned long long)blockIdx.x + 1) * p.ratio >> 32;
    const bool keys = APPEND ? upto != before : blockIdx.x >= p.ratio;
    const unsigned int w = (keys ? before : APPEND ? blockIdx.x - before : blockIdx.x) * (RT / 32) + (threadIdx.x >> 5),
                       chunks = keys ? p.kchunks : p.chunks;
    const unsigned int token = w / chunks, chunk = w - token * chunks;
    if (token >= unsigned(p.tokens)) return;
    const Lane<D, INTER> ln(lane, p.R);
    const int per = keys ? p.kper : p.per, u0 = chunk * per, u1 = min(keys ? p.uk : p.uq, u0 + per);
    if (APPEND && keys) {
        append<D, INTER>(p, ln, token, u0);
        return;
    }
    rotate<D, INTER>(p, ln, p.positions ? p.positions[token] : 0, keys ? p.k + token * p.k_stride : p.q + token * p.q_stride,
                     keys ? p.k_out + token * p.ko_stride : p.q_out + token * p.qo_stride, keys ? p.kw : p.qw,
                     keys ? p.hk : p.hq, u0, u1);
}

template <int D, bool INTER, bool APPEND>
sk_status launch(RopeParams &p, int sms, cudaStream_t s) {
    constexpr int HW = Lane<D, INTER>::HW;
    p.uq = (p.hq + HW - 1) / HW;
    p.uk = (p.hk + HW - 1) / HW;
    const long long held = (long long)sms * MIN_CTAS * (RT / 32);
    auto share = [&](int units, int most) {
        const long long per = (long long)p.tokens * units / held;
        return int(per < 1 ? 1 : per > most ? most : per);
    };
    p.per = share(p.uq, MOST_UNITS);
    p.kper = share(p.uk, APPEND ? 1 : MOST_UNITS);
    p.chunks = (p.uq + p.per - 1) / p.per;
    p.kchunks = (p.uk + p.kper - 1) / p.kper;
    auto ctas = [&](int chunks) { return ((long long)p.tokens * chunks + RT / 32 - 1) / (RT / 32); };
    const long long kctas = ctas(p.kchunks), all = ctas(p.chunks) + kctas;
    if (all * (RT / 32) > 0x7FFFFFFFLL) return SK_ERR_UNSUPPORTED_SHAPE;
    p.ratio = (unsigned int)(APPEND ? (((unsigned long long)kctas << 32) + all - 1) / all : all - kctas);      // (kctas < all)
    return sk::launch_pdl(rope_kernel<D, INTER, APPEND>, dim3(unsigned(all)), dim3(RT), 0, s, p) == cudaSuccess ? SK_OK
                                                                                                               : SK_ERR_CUDA;
}

template <bool APPEND>
sk_status run(RopeParams &p, int dim, bool inter, cudaStream_t s) {
    const int sms = sk::device_sm_count();
    if (sms < 1) return SK_ERR_CUDA;
    switch (dim) {
        case 64: return inter ? launch<64, true, APPEND>(p, sms, s) : launch<64, false, APPEND>(p, sms, s);
        case 128: return inter ? launch<128, true, APPEND>(p, sms, s) : launch<128, false, APPEND>(p, sms, s);
        default: return inter ? launch<256, true, APPEND>(p, sms, s) : launch<256, false, APPEND>(p, sms, s);
    }
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// What both calls ask of their arguments (SK_OK: go on).
sk_status check_rope(const RopeParams &p, int dim, int interleaved) {
    if (p.tokens < 0 || p.hq < 1 || p.hk < 1 || p.R < 0) return SK_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return SK_ERR_INVALID_ARG;
    if (!(p.eps >= 0.0 && p.eps <= 1.0) || !(std::fabs(p.amplitude) >= 1e-3 && std::fabs(p.amplitude) <= 1e3))
        return SK_ERR_INVALID_ARG;
    if ((dim != 64 && dim != 128 && dim != 256) || p.R % 16 || p.R > dim || p.hq > 4096 || p.hk > 4096)
        return SK_ERR_UNSUPPORTED_SHAPE;
    if (!p.qw != !p.kw) return SK_ERR_INVALID_ARG;
    return SK_OK;
}

}  // namespace

extern "C" sk_status rope_frequencies(uint64_t *freqs, int rot_dim, int scaling, double base, double factor, double original,
                                      double low, double high) {
    if (!freqs || rot_dim < 0 || rot_dim % 2 || scaling < SK_ROPE_PLAIN || scaling > SK_ROPE_INDEX) return SK_ERR_INVALID_ARG;
    if (!(base > 1.0 && base <= 1e12)) return SK_ERR_INVALID_ARG;
    if (scaling != SK_ROPE_PLAIN && !(factor >= 1.0 && factor <= 1e6)) return SK_ERR_INVALID_ARG;
    const bool bands = scaling == SK_ROPE_TURNS || scaling == SK_ROPE_INDEX;
    if (bands && !(original >= 1.0 && original <= 1e12 && low > 0.0 && high > low && high <= 1e6)) return SK_ERR_INVALID_ARG;
    if (scaling == SK_ROPE_BASE && rot_dim == 2) return SK_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559, r = rot_dim;
    if (scaling == SK_ROPE_BASE && rot_dim) base *= std::pow(factor, r / (r - 2));
    // the index at which a frequency turns `t` times within the original context
    auto at = [&](double t) { return r * std::log(original / (t * two_pi)) / (2 * std::log(base)); };
    const double first = std::fmax(0.0, std::floor(at(high))), last = std::fmin(r - 1, std::ceil(at(low)));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        double keep = 1.0;
        if (scaling == SK_ROPE_LINEAR) keep = 0.0;
        if (scaling == SK_ROPE_TURNS) keep = (original * f / two_pi - low) / (high - low);
        if (scaling == SK_ROPE_INDEX) keep = 1.0 - (i - first) / std::fmax(1e-3, last - first);
        keep = std::fmin(1.0, std::fmax(0.0, keep));
        if (scaling != SK_ROPE_PLAIN && scaling != SK_ROPE_BASE) f *= keep + (1.0 - keep) / factor;
        freqs[i] = uint64_t(f / two_pi * 0x1p64);
    }
    return SK_OK;
}

extern "C" sk_status qk_norm_rope(const void *q, long long q_stride, const void *k, long long k_stride,
                                  const int32_t *positions, const uint64_t *freqs, const float *q_weight,
                                  const float *k_weight, double eps, double amplitude, void *q_out, long long q_out_stride,
                                  void *k_out, long long k_out_stride, int tokens, int q_heads, int kv_heads, int head_dim,
                                  int rot_dim, int interleaved, void *stream) {
    RopeParams p = {};
    p.q = static_cast<const __half *>(q);
    p.k = static_cast<const __half *>(k);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out = static_cast<__half *>(q_out);
    p.k_out = static_cast<__half *>(k_out);
    p.qo_stride = q_out_stride;
    p.ko_stride = k_out_stride;
    p.positions = positions;
    p.freqs = freqs;
    p.qw = q_weight;
    p.kw = k_weight;
    p.eps = eps;
    p.amplitude = amplitude;
    p.tokens = tokens;
    p.hq = q_heads;
    p.hk = kv_heads;
    p.R = rot_dim;
    const sk_status st = check_rope(p, head_dim, interleaved);
    if (st != SK_OK || tokens == 0) return st;
    if (!q || !k || !q_out || !k_out || (rot_dim && (!positions || !freqs))) return SK_ERR_INVALID_ARG;
    const long long qrow = (long long)q_heads * head_dim, krow = (long long)kv_heads * head_dim;
    if (q_stride < qrow || k_stride < krow || q_out_stride < qrow || k_out_stride < krow) return SK_ERR_INVALID_ARG;
    if (q_stride % 8 || k_stride % 8 || q_out_stride % 8 || k_out_stride % 8 || !aligned(q, 16) || !aligned(k, 16) ||
        !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(positions, 4) || !aligned(freqs, 8) ||
        !aligned(q_weight, 4) || !aligned(k_weight, 4))
        return SK_ERR_MISALIGNED;
    return run<false>(p, head_dim, interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" sk_status kv4_append_rope(const void *q, long long q_stride, const void *k, long long k_stride, const void *v,
                                     long long v_stride, const int32_t *slots, const int32_t *positions,
                                     const uint64_t *freqs, const float *q_weight, const float *k_weight, double eps,
                                     double amplitude, void *q_out, long long q_out_stride, uint8_t *cache, float k_scale,
                                     float v_scale, int tokens, int pages, int q_heads, int kv_heads, int head_dim,
                                     int page_size, int rot_dim, int interleaved, void *stream) {
    RopeParams p = {};
    p.q = static_cast<const __half *>(q);
    p.k = static_cast<const __half *>(k);
    p.v = static_cast<const __half *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<__half *>(q_out);
    p.qo_stride = q_out_stride;
    p.positions = positions;
    p.freqs = freqs;
    p.qw = q_weight;
    p.kw = k_weight;
    p.eps = eps;
    p.amplitude = amplitude;
    p.tokens = tokens;
    p.hq = q_heads;
    p.hk = kv_heads;
    p.R = rot_dim;
    p.slots = slots;
    p.cache = cache;
    p.gk = k_scale;
    p.gv = v_scale;
    p.pages = pages;
    p.page = page_size;
    p.recs = page_size / sk::KV4_REC;
    sk_status st = check_rope(p, head_dim, interleaved);
    if (st != SK_OK) return st;
    if (pages < 1 || page_size < 1 || !sk::kv4_scale_ok(k_scale) || !sk::kv4_scale_ok(v_scale)) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_shape_ok(pages, kv_heads, head_dim, page_size)) return SK_ERR_UNSUPPORTED_SHAPE;
    if (tokens == 0) return SK_OK;
    if (!q || !k || !v || !slots || !q_out || !cache || (rot_dim && (!positions || !freqs))) return SK_ERR_INVALID_ARG;
    const long long qrow = (long long)q_heads * head_dim, krow = (long long)kv_heads * head_dim;
    if (q_stride < qrow || k_stride < krow || v_stride < krow || q_out_stride < qrow) return SK_ERR_INVALID_ARG;
    if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_out_stride % 8 || !aligned(q, 16) || !aligned(k, 16) ||
        !aligned(v, 16) || !aligned(q_out, 16) || !aligned(slots, 4) || !aligned(positions, 4) || !aligned(freqs, 8) ||
        !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(cache, 16))
        return SK_ERR_MISALIGNED;
    return run<true>(p, head_dim, interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
}
