// kv4_attention.cu -- attention of 1..8 query rows per sequence over the paged
// 4-bit cache (kv4.cuh), and the sum of the weights each position received.
//
// For row m of sequence b and query head x, over positions j < lens[b] - (M-1-m):
//     z_j = scale * q . k_j,   p_j = exp(z_j - max z),   out = sum p_j v_j / sum p_j
// in one pass over the cache with a running maximum and sum (FP32).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/skinny.h"
#include "internal.h"
#include "kv4.cuh"
#include "launch_util.cuh"

namespace {

constexpr int WARPS = 4;
constexpr int CT = WARPS * 32;
constexpr int STEP = 32;               // positions per warp step: two records
constexpr int TILE = WARPS * STEP;     // positions per CTA step, the unit of the work split
constexpr int ROWS = 16;               // query rows per tile (one m16 operand)
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// The weights p go to the second product in FP16, scaled by 2^P_SHIFT: at most
// 2^15, and normal FP16 numbers down to 2^-29 of the row's largest.  Their
// rounding (2^-12 relative at most, independent from position to position) is
// of the size of the output's own rounding to FP16; the sum of the weights is
// taken from the unrounded FP32 values.
constexpr float P_SHIFT = 15.f;
constexpr uint64_t WAIT_NS = 1000000000ull;

template <int D>
struct Cfg {
    static constexpr int REC = sk::kv4_rec_bytes(D);
    static constexpr int STAGE = 2 * REC;
    static constexpr int STAGES = D == 64 ? 4 : D == 128 ? 3 : 2;
    static constexpr int KSTEPS = D / 16;
    static constexpr int QBYTES = KSTEPS * 512;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int CTAS = D == 256 ? 2 : 3;
    static constexpr int OSTRIDE = D + 4;        // floats between rows of a warp's sums at the merge
    static constexpr size_t SMEM = RING + QBYTES + WARPS * STAGES * 8 + WARPS * ROWS * 8;
    static_assert(WARPS * ROWS * OSTRIDE * 4 <= RING, "the merge reuses the ring");
};

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

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// Untiled bulk copy into this CTA's shared memory (16-byte aligned, bytes a
// multiple of 16), completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
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

// Query rows [rt * 16, rt * 16 + 16) of (b, h) as A operands of the k16 steps:
// step s of lane (g = lane / 4, t = lane % 4) takes components c..c+3 of rows g
// and g + 8, where c = 128 (s / 8) + 32 t + 4 (s % 8) (D = 64: 16 t + 4 s):
// the same order in which a lane's key bytes decode.  Rows past the last are zero.
template <int D>
__device__ __forceinline__ void load_q(const AttnParams &p, int b, int h, int rt, uint32_t qs) {
    for (int i = threadIdx.x; i < Cfg<D>::KSTEPS * 32; i += blockDim.x) {
        const int s = i >> 5, l = i & 31, g = l >> 2, t = l & 3;
        const int c = D == 64 ? 16 * t + 4 * s : 128 * (s >> 3) + 32 * t + 4 * (s & 7);
        uint2 v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = rt * ROWS + g + 8 * k, m = r / p.G;
            v[k] = make_uint2(0u, 0u);
            if (m < p.M)
                v[k] = *reinterpret_cast<const uint2 *>(p.q + ((long long)b * p.M + m) * p.q_stride +
                                                         (long long)(h * p.G + r - m * p.G) * D + c);
        }
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(qs + i * 16), "r"(v[0].x), "r"(v[1].x),
                     "r"(v[0].y), "r"(v[1].y) : "memory");
    }
}

// Key bytes of one n8 tile's row for this lane, as loaded from a record at
// `rec` (shared memory), row i = position in the record.
template <int D>
struct Keys {
    static constexpr int PIECES = D == 256 ? 2 : 1, WP = D == 64 ? 2 : 4;
    uint32_t w[PIECES * WP];
    uint32_t s[PIECES];        // scales of the lane's blocks, f16x2 (D = 64: the one scale, twice)
};

template <int D>
__device__ __forceinline__ void load_keys(uint32_t rec, int i, int t, Keys<D> &k) {
    if constexpr (D == 64) {
        const uint2 v = ld_shared_v2(rec + i * 32 + t * 8);
        k.w[0] = v.x;
        k.w[1] = v.y;
        k.s[0] = sk::bcast_lo(scale_pair(ld_shared_u8(rec + 8 * D + i * 4 + t)));
    } else {
#pragma unroll
        for (int c = 0; c < Keys<D>::PIECES; ++c) {
            const uint4 v = sk::ld_shared_v4(rec + i * (D / 2) + c * 64 + t * 16);
            k.w[4 * c] = v.x;
            k.w[4 * c + 1] = v.y;
            k.w[4 * c + 2] = v.z;
            k.w[4 * c + 3] = v.w;
            k.s[c] = scale_pair(sk::ld_shared_u16(rec + 8 * D + i * (D / 16) + c * 8 + t * 2));
        }
    }
}

// s[j] += q . k over all D components for NT tiles of eight positions: each
// key byte pair decodes to the B operand, scaled in FP16 first (exact: 2 x 4
// significant bits, inside the FP16 normal range).
template <int D, int NT>
__device__ __forceinline__ void qk(const Keys<D> (&k)[NT], uint32_t qs, int lane, float (&s)[NT][4]) {
#pragma unroll
    for (int w = 0; w < Keys<D>::PIECES * Keys<D>::WP; ++w) {
        const uint4 a = sk::ld_shared_v4(qs + ((2 * w) * 32 + lane) * 16);
        const uint4 c = sk::ld_shared_v4(qs + ((2 * w + 1) * 32 + lane) * 16);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint32_t d[4];
            sk::e2m1x8_to_f16x2x4(k[j].w[w], d);
            const uint32_t sc = D == 64 ? k[j].s[0] : (w & 2) ? sk::bcast_hi(k[j].s[w / 4]) : sk::bcast_lo(k[j].s[w / 4]);
#pragma unroll
            for (int x = 0; x < 4; ++x) d[x] = sk::hmul2(d[x], sc);
            sk::mma_16816(s[j], a.x, a.y, a.z, a.w, d[0], d[1]);
            sk::mma_16816(s[j], c.x, c.y, c.z, c.w, d[2], d[3]);
        }
    }
}

// Codes of two neighbouring positions a, b (eight components each) -> f16x2
// pairs {a_c, b_c}: their nibbles are interleaved first, so that one convert
// yields both.
__device__ __forceinline__ void decode_pair(uint32_t a, uint32_t b, uint32_t (&d)[8]) {
    const uint32_t lo = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
    const uint32_t hi = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
    uint32_t e[4], o[4];
    sk::e2m1x8_to_f16x2x4(lo, e);
    sk::e2m1x8_to_f16x2x4(hi, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d[2 * i] = e[i];
        d[2 * i + 1] = o[i];
    }
}

// o += p . v over the 16 positions of the record at `rec`; a[4] is the A
// operand of p.
template <int D>
__device__ __forceinline__ void pv(uint32_t rec, const uint32_t (&a)[4], int g, int t, float (&o)[D / 8][4]) {
    constexpr int NB = D == 64 ? 1 : D / 128, PER = D == 64 ? 8 : 16;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int blk = D == 64 ? g >> 1 : g + 8 * nb;
        uint32_t b[2][PER];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 v = sk::ld_shared_v4(rec + 9 * D + j * 4 * D + blk * 64 + t * 16);
            const uint32_t sc = scale_pair(sk::ld_shared_u16(rec + 17 * D + blk * 16 + 8 * j + 2 * t));
            uint32_t d[8];
            if constexpr (D == 64) {
                decode_pair((g & 1) ? v.y : v.x, (g & 1) ? v.w : v.z, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) b[j][i] = sk::hmul2(d[i], sc);
            } else {
                decode_pair(v.x, v.z, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) b[j][i] = sk::hmul2(d[i], sc);
                decode_pair(v.y, v.w, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) b[j][8 + i] = sk::hmul2(d[i], sc);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) sk::mma_16816(o[nb * PER + i], a[0], a[1], a[2], a[3], b[0][i], b[1][i]);
    }
}

__device__ __forceinline__ void wait_full(uint32_t bar, uint32_t parity, unsigned int *err, bool &dead) {
    if (dead) return;
    if (sk::mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = sk::globaltimer_ns();
    while (!sk::mbar_try_wait(bar, parity)) {
        if (sk::globaltimer_ns() - t0 > WAIT_NS) {
            dead = true;
            atomicOr(err, 1u);
            return;
        }
    }
}

// Few query rows per kv head: each warp streams its own steps of 32 positions
// (bulk copies into a ring of its own, issued by one lane two or three steps
// ahead) and keeps 16 query rows' maxima, sums and outputs in registers; the
// four warps meet only at the end of a segment (sequence, head, row tile).
template <int D>
__global__ void __launch_bounds__(CT, Cfg<D>::CTAS) kv4_attention_kernel(const __grid_constant__ AttnParams p) {
    using C = Cfg<D>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long sm_share[WARPS + 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t base = sk::smem_u32(smem);
    const uint32_t qs = base + C::RING, bars = qs + C::QBYTES;
    const uint32_t ring = base + warp * C::STAGES * C::STAGE, bar = bars + warp * C::STAGES * 8;
    float *const obuf = reinterpret_cast<float *>(smem);
    float2 *const mlbuf = reinterpret_cast<float2 *>(smem + C::RING + C::QBYTES + WARPS * C::STAGES * 8);
    if (lane == 0)
        for (int s = 0; s < C::STAGES; ++s) sk::mbar_init(bar + s * 8, 1);
    sk::fence_barrier_init();
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    Share sh = share_of(p, p.heads * p.RT, sm_share);
    uint32_t it = 0;           // steps this warp has consumed: ring position and parity
    bool dead = false;

    while (sh.t < sh.end && sh.b < p.B) {
        const int len = length_of(p, sh.b), nt = tiles_of(len);
        if (nt == 0) {
            ++sh.b;
            continue;
        }
        const int hr = int(sh.off / nt), t_lo = int(sh.off - (long long)hr * nt);
        const int t_hi = int(min((long long)nt, t_lo + sh.end - sh.t));
        const int h = hr / p.RT, rt = hr - h * p.RT, b = sh.b;
        const int32_t *table = p.table + (long long)b * p.width;
        const int nrec = (len + 15) / 16;
        load_q<D>(p, b, h, rt, qs);

        // this warp's steps: st = st_lo + warp, + WARPS, ... below st_hi
        const int st_hi = min(t_hi * WARPS, (len + STEP - 1) / STEP);
        int st = t_lo * WARPS + warp;
        const int n = st < st_hi ? (st_hi - st + WARPS - 1) / WARPS : 0;
        auto record = [&](int rec) { return sk::kv4_record(table, min(rec, nrec - 1), p.recs, p.pages, p.heads, h); };
        auto issue = [&](uint32_t slot, int step, size_t r0, size_t r1) {
            const uint32_t dst = ring + (slot % C::STAGES) * C::STAGE, fb = bar + (slot % C::STAGES) * 8;
            const bool two = 2 * step + 1 < nrec;
            sk::mbar_arrive_expect_tx(fb, two ? 2 * C::REC : C::REC);
            bulk_load(dst, p.cache + r0 * C::REC, C::REC, fb);
            if (two) bulk_load(dst + C::REC, p.cache + r1 * C::REC, C::REC, fb);
        };
        for (int i = 0; i < C::STAGES; ++i)
            if (i < n && lane == 0) {
                const int step = st + i * WARPS;
                issue(it + i, step, record(2 * step), record(2 * step + 1));
            }
        // the records of the next step to issue, looked up one step ahead
        size_t r0 = 0, r1 = 0;
        if (C::STAGES < n) {
            const int step = st + C::STAGES * WARPS;
            r0 = record(2 * step);
            r1 = record(2 * step + 1);
        }
        __syncthreads();       // the query rows are in shared memory

        float o[D / 8][4], mx[2] = {NEG_INF, NEG_INF}, sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
        // rows g and g + 8 of the tile see positions below lim
        int lim[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) lim[k] = len - (p.M - 1 - min((rt * ROWS + g + 8 * k) / p.G, p.M - 1));

        for (int i = 0; i < n; ++i, ++it, st += WARPS) {
            const uint32_t stage = ring + (it % C::STAGES) * C::STAGE;
            wait_full(bar + (it % C::STAGES) * 8, (it / C::STAGES) & 1, p.err, dead);
            float s[4][4];
            {
                Keys<D> k[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    load_keys<D>(stage + (j >> 1) * C::REC, (j & 1) * 8 + g, t, k[j]);
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[j][x] = 0.f;
                }
                qk<D, 4>(k, qs, lane, s);
            }
            const int pos = st * STEP;
            const bool edge = pos + STEP > len - (p.M - 1);
            if (edge) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (pos + j * 8 + 2 * t + (x & 1) >= lim[x >> 1]) s[j][x] = NEG_INF;
            }
            float off[2];
            bool grown = false;
            float alpha[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float m = s[0][2 * k];
#pragma unroll
                for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(s[j][2 * k], s[j][2 * k + 1]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const float now = fmaxf(mx[k], m * p.scale2);
                alpha[k] = mx[k] == now ? 1.f : ex2(mx[k] - now);
                grown |= mx[k] != now;
                mx[k] = now;
                off[k] = now == NEG_INF ? 0.f : P_SHIFT - now;
            }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int x = 0; x < D / 8; ++x) {
                    o[x][0] *= alpha[0];
                    o[x][1] *= alpha[0];
                    o[x][2] *= alpha[1];
                    o[x][3] *= alpha[1];
                }
                sum[0] *= alpha[0];
                sum[1] *= alpha[1];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[j][x] = ex2(fmaf(s[j][x], p.scale2, off[x >> 1]));
                    sum[x >> 1] += s[j][x];
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t a[4] = {pack_f16(s[2 * r][0], s[2 * r][1]), pack_f16(s[2 * r][2], s[2 * r][3]),
                                       pack_f16(s[2 * r + 1][0], s[2 * r + 1][1]),
                                       pack_f16(s[2 * r + 1][2], s[2 * r + 1][3])};
                pv<D>(stage + r * C::REC, a, g, t, o);
            }
            __syncwarp();      // every lane has read the stage
            if (i + C::STAGES < n) {
                if (lane == 0) issue(it + C::STAGES, st + C::STAGES * WARPS, r0, r1);
                if (i + C::STAGES + 1 < n) {
                    const int step = st + (C::STAGES + 1) * WARPS;
                    r0 = record(2 * step);
                    r1 = record(2 * step + 1);
                }
            }
        }

        // ---- the four warps' sums, in warp order
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
            if (t == 0) mlbuf[warp * ROWS + g + 8 * k] = make_float2(mx[k], sum[k]);
        }
        __syncthreads();       // every warp is done with its ring
        {
            float *dst = obuf + warp * ROWS * C::OSTRIDE;
#pragma unroll
            for (int x = 0; x < D / 8; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int nn = 2 * t + (e & 1), row = g + 8 * (e >> 1);
                    const int d = D == 64 ? 8 * nn + x : 16 * (nn + 8 * (x >> 4)) + (x & 15);
                    dst[row * C::OSTRIDE + d] = o[x][e];
                }
        }
        __syncthreads();
        const bool whole = t_lo == 0 && t_hi == nt;
        const int rows = min(ROWS, p.M * p.G - rt * ROWS);
        const size_t slot = size_t(blockIdx.x) * 2 + (t_lo == 0 ? 1 : 0);
        for (int i = tid; i < rows * (D / 4); i += CT) {
            const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
            float2 ml[WARPS];
            float top = NEG_INF, l = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                ml[w] = mlbuf[w * ROWS + r];
                top = fmaxf(top, ml[w].x);
            }
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float f = ml[w].x == NEG_INF ? 0.f : ex2(ml[w].x - top);
                const float4 x = *reinterpret_cast<const float4 *>(obuf + (w * ROWS + r) * C::OSTRIDE + d);
                l += ml[w].y * f;
                v.x += x.x * f;
                v.y += x.y * f;
                v.z += x.z * f;
                v.w += x.w * f;
            }
            if (whole) {
                const int row = rt * ROWS + r, m = row / p.G;
                const long long at = ((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G;
                const float f = l == 0.f ? 0.f : p.vg / l;
                const __half2 y0 = __floats2half2_rn(v.x * f, v.y * f), y1 = __floats2half2_rn(v.z * f, v.w * f);
                uint2 y = make_uint2(*reinterpret_cast<const uint32_t *>(&y0), *reinterpret_cast<const uint32_t *>(&y1));
                *reinterpret_cast<uint2 *>(p.out + at * D + d) = y;
                if (d == 0 && p.lse) p.lse[at] = l == 0.f ? NEG_INF : (top + __log2f(l) - P_SHIFT) * LN2;
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (slot * ROWS + r) * D + d) = v;
                if (d == 0) *reinterpret_cast<float2 *>(p.part_ml + (slot * ROWS + r) * 2) = make_float2(top, l);
            }
        }
        if (tid == 0 && t_lo == 0) {
            const long long last = sh.t + nt - 1;     // the segment's last tile
            const int c1 = int(((last + 1) * sh.parts - 1) / sh.total);
            p.seg[((long long)b * p.heads + h) * p.RT + rt] = make_int2(int(blockIdx.x), whole ? 0 : c1 - int(blockIdx.x) + 1);
        }
        // the ring's next copies come after these reads and writes of it
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        sh.t += t_hi - t_lo;
        sh.off += t_hi - t_lo;
        if (sh.off == (long long)nt * p.heads * p.RT) {
            ++sh.b;
            sh.off = 0;
        }
    }
}

// One CTA per query row: the partial sums of its segment, in the order of the
// CTAs that wrote them, joined under the common maximum.  Rows of an empty
// sequence are written here too (zero, with a log sum of minus infinity).
constexpr int JT = 256;

template <int D>
__global__ void __launch_bounds__(JT) kv4_join_kernel(const __grid_constant__ AttnParams p, int max_parts) {
    extern __shared__ float wgt[];                 // one weight per partial
    __shared__ float red[JT / 32], red_l[JT / 32];
    __shared__ float part[JT / 32][D];
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    const int rows = p.M * p.G, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int bh = blockIdx.x / rows, row = blockIdx.x - bh * rows, b = bh / p.heads, h = bh - b * p.heads;
    const int rt = row / ROWS, r = row - rt * ROWS, m = row / p.G;
    const long long at = ((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G;
    const bool empty = length_of(p, b) == 0;
    if (empty) {
        for (int d = tid; d < D; d += JT) p.out[at * D + d] = __float2half_rn(0.f);
        if (tid == 0 && p.lse) p.lse[at] = NEG_INF;
        return;
    }
    const int2 seg = p.seg[(long long)bh * p.RT + rt];
    if (seg.y == 0) return;
    const int n = min(seg.y, max_parts);
    // slot of partial i: the first CTA's second slot, the first slot of the others
    auto slot = [&](int i) { return (size_t(seg.x) + i) * 2 + (i == 0 ? 1 : 0); };
    float top = NEG_INF;
    for (int i = tid; i < n; i += JT) top = fmaxf(top, p.part_ml[(slot(i) * ROWS + r) * 2]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[wid] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < JT / 32; ++w) top = fmaxf(top, red[w]);
    float l = 0.f;
    for (int i = tid; i < n; i += JT) {
        const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + (slot(i) * ROWS + r) * 2);
        const float f = ml.x == NEG_INF ? 0.f : ex2(ml.x - top);
        wgt[i] = f;
        l += ml.y * f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red_l[wid] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < JT / 32; ++w) l += red_l[w];
    constexpr int PER = D / 32;
    float v[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) v[x] = 0.f;
#pragma unroll 8
    for (int i = wid; i < n; i += JT / 32) {
        const float *src = p.part_o + (slot(i) * ROWS + r) * D + lane * 2;
        const float f = wgt[i];
#pragma unroll
        for (int x = 0; x < PER; x += 2) {
            const float2 y = *reinterpret_cast<const float2 *>(src + x * 32);
            v[x] += y.x * f;
            v[x + 1] += y.y * f;
        }
    }
#pragma unroll
    for (int x = 0; x < PER; x += 2) *reinterpret_cast<float2 *>(&part[wid][x * 32 + lane * 2]) = make_float2(v[x], v[x + 1]);
    __syncthreads();
    for (int d = tid; d < D; d += JT) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < JT / 32; ++w) y += part[w][d];
        p.out[at * D + d] = __float2half_rn(l == 0.f ? 0.f : y * (p.vg / l));
    }
    if (tid == 0 && p.lse) p.lse[at] = l == 0.f ? NEG_INF : (top + __log2f(l) - P_SHIFT) * LN2;
}

// acc_out = acc_in + the weights of all query rows, per position and kv head:
// the scores once more (the keys alone are read), against the rows' final log
// sums.  Each warp owns its positions, so the sum over rows has one order.
constexpr int WT_WARPS = 8;
constexpr int WT_TILES = 8;            // row tiles held in shared memory at a time

template <int D>
__global__ void __launch_bounds__(WT_WARPS * 32) kv4_weights_kernel(const __grid_constant__ AttnParams p, int held) {
    using C = Cfg<D>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long sm_share[WT_WARPS + 4];
    __shared__ float lse2[WT_TILES * ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t qs = sk::smem_u32(smem);
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    Share sh = share_of(p, p.heads, sm_share);
    while (sh.t < sh.end && sh.b < p.B) {
        const int len = length_of(p, sh.b), nt = tiles_of(len);
        if (nt == 0) {
            ++sh.b;
            continue;
        }
        const int h = int(sh.off / nt), t_lo = int(sh.off - (long long)h * nt), b = sh.b;
        const int t_hi = int(min((long long)nt, t_lo + sh.end - sh.t));
        const int32_t *table = p.table + (long long)b * p.width;
        const int rows = p.M * p.G;
        for (int rt0 = 0; rt0 < p.RT; rt0 += held) {
            const int nr = min(held, p.RT - rt0);
            __syncthreads();
            for (int x = 0; x < nr; ++x) load_q<D>(p, b, h, rt0 + x, qs + x * C::QBYTES);
            for (int x = tid; x < nr * ROWS; x += WT_WARPS * 32) {
                const int row = rt0 * ROWS + x, m = row / p.G;
                float v = NEG_INF;
                if (row < rows) v = p.lse[((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G];
                lse2[x] = v == NEG_INF ? -NEG_INF : v * LOG2E;     // no weight from rows that see nothing
            }
            __syncthreads();
            const int rec_hi = min(t_hi * (TILE / 16), (len + 15) / 16);
            for (int rec = t_lo * (TILE / 16) + warp; rec < rec_hi; rec += WT_WARPS) {
                const uint8_t *src = p.cache + sk::kv4_record(table, rec, p.recs, p.pages, p.heads, h) * C::REC;
                Keys<D> k[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i = j * 8 + g;
                    if constexpr (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(src + i * 32 + t * 8);
                        k[j].w[0] = v.x;
                        k[j].w[1] = v.y;
                        k[j].s[0] = sk::bcast_lo(scale_pair(src[8 * D + i * 4 + t]));
                    } else {
#pragma unroll
                        for (int c = 0; c < Keys<D>::PIECES; ++c) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(src + i * (D / 2) + c * 64 + t * 16);
                            k[j].w[4 * c] = v.x;
                            k[j].w[4 * c + 1] = v.y;
                            k[j].w[4 * c + 2] = v.z;
                            k[j].w[4 * c + 3] = v.w;
                            k[j].s[c] =
                                scale_pair(*reinterpret_cast<const uint16_t *>(src + 8 * D + i * (D / 16) + c * 8 + t * 2));
                        }
                    }
                }
                float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
                for (int x = 0; x < nr; ++x) {
                    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                    qk<D, 2>(k, qs + x * C::QBYTES, lane, s);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int row = x * ROWS + g + 8 * y;
                        const float neg = -lse2[row];
                        const int lim = len - (p.M - 1 - min((rt0 * ROWS + row) / p.G, p.M - 1));
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float z = fmaf(s[j][2 * y + e], p.scale2, neg);
                                if (rec * 16 + j * 8 + 2 * t + e < lim) w[j][e] += neg == NEG_INF ? 0.f : ex2(z);
                            }
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w[j][e] += __shfl_xor_sync(0xffffffffu, w[j][e], 4);
                        w[j][e] += __shfl_xor_sync(0xffffffffu, w[j][e], 8);
                        w[j][e] += __shfl_xor_sync(0xffffffffu, w[j][e], 16);
                    }
                // lane g = 0..3 of each t writes one of the four positions
                if (g < 4) {
                    const int pos = rec * 16 + (g >> 1) * 8 + 2 * t + (g & 1);
                    const float mine = (g >> 1) ? ((g & 1) ? w[1][1] : w[1][0]) : ((g & 1) ? w[0][1] : w[0][0]);
                    if (pos < len) {
                        const size_t at = (size_t(b) * p.heads + h) * size_t(p.cap) + pos;
                        const float *old = rt0 == 0 ? p.acc_in : p.acc_out;
                        p.acc_out[at] = (old ? old[at] : 0.f) + mine;
                    }
                }
            }
        }
        sh.t += t_hi - t_lo;
        sh.off += t_hi - t_lo;
        if (sh.off == (long long)nt * p.heads) {
            ++sh.b;
            sh.off = 0;
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int MAX_SEGMENTS = 131072;

template <int D>
sk_status run(AttnParams &p, unsigned char *scratch, int sms, cudaStream_t s) {
    using C = Cfg<D>;
    p.ctas = sms * C::CTAS;
    p.seg = reinterpret_cast<int2 *>(scratch);
    p.part_ml = reinterpret_cast<float *>(scratch + size_t(MAX_SEGMENTS) * sizeof(int2));
    p.part_o = p.part_ml + size_t(p.ctas) * 2 * ROWS * 2;
    if (size_t(reinterpret_cast<unsigned char *>(p.part_o + size_t(p.ctas) * 2 * ROWS * D) - scratch) > sk::SCRATCH_BYTES)
        return SK_ERR_WORKSPACE;
    if (sk::prepare_kernel<kv4_attention_kernel<D>>(C::SMEM) != cudaSuccess) return SK_ERR_CUDA;
    if (sk::launch_pdl(kv4_attention_kernel<D>, dim3(p.ctas), dim3(CT), C::SMEM, s, p) != cudaSuccess) return SK_ERR_CUDA;
    const long long rows = (long long)p.B * p.heads * p.M * p.G;
    if (sk::launch_pdl(kv4_join_kernel<D>, dim3(unsigned(rows)), dim3(JT), size_t(p.ctas) * 4, s, p, p.ctas) != cudaSuccess)
        return SK_ERR_CUDA;
    if (p.acc_out) {
        const int held = p.RT < WT_TILES ? p.RT : WT_TILES;
        const size_t bytes = size_t(held) * C::QBYTES;
        p.ctas = sms * 4;
        if (sk::prepare_kernel<kv4_weights_kernel<D>>(WT_TILES * C::QBYTES) != cudaSuccess) return SK_ERR_CUDA;
        if (sk::launch_pdl(kv4_weights_kernel<D>, dim3(p.ctas), dim3(WT_WARPS * 32), bytes, s, p, held) != cudaSuccess)
            return SK_ERR_CUDA;
    }
    return SK_OK;
}

}  // namespace

extern "C" sk_status kv4_attention(const void *q, long long q_stride, const uint8_t *cache, const int32_t *table,
                                   const int32_t *lens, float k_scale, float v_scale, float scale, void *out,
                                   float *lse, const float *acc_in, float *acc_out, int seqs, int rows, int q_heads,
                                   int kv_heads, int head_dim, int pages, int page_size, int table_width,
                                   void *stream) {
    if (seqs < 0 || rows < 1 || rows > 8 || q_heads < 1 || kv_heads < 1 || pages < 1 || page_size < 1 ||
        table_width < 1)
        return SK_ERR_INVALID_ARG;
    if (q_heads % kv_heads) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_scale_ok(k_scale) || !sk::kv4_scale_ok(v_scale) || !(scale > 0.f && scale < 1e20f)) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_shape_ok(pages, kv_heads, head_dim, page_size)) return SK_ERR_UNSUPPORTED_SHAPE;
    if ((long long)table_width * page_size > 0x7FFFFF00LL) return SK_ERR_UNSUPPORTED_SHAPE;
    if (seqs == 0) return SK_OK;
    if (!q || !cache || !table || !lens || !out) return SK_ERR_INVALID_ARG;
    if ((acc_out && !lse) || (acc_in && !acc_out)) return SK_ERR_INVALID_ARG;
    if (q_stride < (long long)q_heads * head_dim) return SK_ERR_INVALID_ARG;
    if (q_stride % 8 || !aligned(q, 16) || !aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(out, 16) || !aligned(lse, 4) || !aligned(acc_in, 4) || !aligned(acc_out, 4))
        return SK_ERR_MISALIGNED;
    AttnParams p = {};
    p.B = seqs;
    p.M = rows;
    p.heads = kv_heads;
    p.G = q_heads / kv_heads;
    p.RT = (rows * p.G + ROWS - 1) / ROWS;
    if ((long long)seqs * kv_heads * p.RT > MAX_SEGMENTS || (long long)seqs * q_heads * rows > 0x7FFFFFFFLL)
        return SK_ERR_UNSUPPORTED_SHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    sk::Scratch sc;
    if (!sk::scratch_for(s, &sc)) return SK_ERR_NOT_INITIALIZED;
    p.q = static_cast<const __half *>(q);
    p.q_stride = q_stride;
    p.cache = cache;
    p.table = table;
    p.lens = lens;
    p.out = static_cast<__half *>(out);
    p.lse = lse;
    p.acc_in = acc_in;
    p.acc_out = acc_out;
    p.err = sc.err;
    p.pages = pages;
    p.recs = page_size / sk::KV4_REC;
    p.width = table_width;
    p.cap = table_width * page_size;
    p.scale2 = scale * k_scale * LOG2E;
    p.vg = v_scale;
    switch (head_dim) {
        case 64: return run<64>(p, sc.base, sc.num_sms, s);
        case 128: return run<128>(p, sc.base, sc.num_sms, s);
        default: return run<256>(p, sc.base, sc.num_sms, s);
    }
}
