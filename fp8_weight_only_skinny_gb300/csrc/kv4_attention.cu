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
#include "kv4_attention.cuh"
#include "launch_util.cuh"

namespace {

using namespace sk::attn;

// NR tiles of eight query rows are taken together: positions (q . k) and
// components (p . v) are the 16-wide operand, query rows the 8-wide one, so
// that few rows cost few multiplications and the decoded codes serve 8 NR rows.
template <int D, int NR>
struct Cfg {
    static constexpr int ROWS = NROW * NR;
    static constexpr int REC = sk::kv4_rec_bytes(D);
    static constexpr int STAGE = 2 * REC;
    static constexpr int KPAIRS = D / 32;            // pairs of k16 steps
    static constexpr int QTILE = KPAIRS * 512;       // bytes of eight query rows
    // accumulators are D / 4 NR registers a thread: CTAs per SM by what is left
    // (six of D = 64, NR = 1: 8 sequences of 30000, 8 heads, one row 46 -> 43 us;
    // five of 32 accumulators spill: 33 -> 37 us at D = 128)
    static constexpr int ACC = D / 4 * NR;
    static constexpr int CTAS = ACC >= 96 ? 2 : ACC >= 64 ? 3 : ACC <= 16 ? 6 : 4;
    static constexpr int STAGES = D == 64 ? (CTAS == 6 ? 3 : 4) : D == 128 ? (CTAS == 4 ? 2 : 3) : 2;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int OSTRIDE = D == 256 ? D + 8 : D;          // floats between rows of a warp's sums at the merge
    static constexpr int MERGE = WARPS * ROWS * OSTRIDE * 4;
    static constexpr int BODY = RING > MERGE ? RING : MERGE;      // the merge reuses the ring
    static constexpr size_t SMEM = BODY + NR * QTILE + WARPS * STAGES * 8 + WARPS * ROWS * 8;
};

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

// Query rows [row0, row0 + 8 n) of (b, h) as B operands, two k16 steps in one
// 16-byte word: word i (pair w, tile r) of lane (g = lane / 4, t = lane % 4) holds
// components c .. c + 7 of row row0 + 8 r + g, c = 128 (w / 4) + 32 t + 8 (w % 4)
// (D = 64: 16 t + 8 w): the order in which a lane's key bytes decode.  Rows
// past the last are zero.
template <int D>
__device__ __forceinline__ uint4 fetch_q(const AttnParams &p, int b, int h, int row0, int i) {
    constexpr int KPAIRS = D / 32;
    const int l = i & 31, w = (i >> 5) % KPAIRS, r = (i >> 5) / KPAIRS, g = l >> 2, t = l & 3;
    const int c = D == 64 ? 16 * t + 8 * w : 128 * (w >> 2) + 32 * t + 8 * (w & 3);
    const int row = row0 + 8 * r + g, m = row / p.G;
    if (m >= p.M) return make_uint4(0u, 0u, 0u, 0u);
    return *reinterpret_cast<const uint4 *>(p.q + ((long long)b * p.M + m) * p.q_stride +
                                             (long long)(h * p.G + row - m * p.G) * D + c);
}
__device__ __forceinline__ void store_q(uint32_t qs, int i, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(qs + i * 16), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Key bytes of one position for this lane, as loaded from a record at
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

// s[x][r] = q . k over all D components for NX records (16 positions each; the
// lane holds positions g and g + 8 as k[2 x] and k[2 x + 1]) and NR tiles of
// query rows: each key byte pair decodes to a pair of A elements, scaled in
// FP16 first (exact: 2 x 4 significant bits, inside the FP16 normal range).
// s[x][r] holds (g, 2 t), (g, 2 t + 1), (g + 8, 2 t), (g + 8, 2 t + 1) as
// (position, row).
template <int D, int NX, int NR>
__device__ __forceinline__ void qk(const Keys<D> (&k)[2 * NX], uint32_t qs, int lane, float (&s)[NX][NR][4]) {
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[x][r][e] = 0.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        uint4 q[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) q[r] = sk::ld_shared_v4(qs + ((r * (D / 32) + w) * 32 + lane) * 16);
#pragma unroll
        for (int x = 0; x < NX; ++x) {
            uint32_t d[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const Keys<D> &kk = k[2 * x + y];
                sk::e2m1x8_to_f16x2x4(kk.w[w], d[y]);
                const uint32_t sc = D == 64 ? kk.s[0] : (w & 2) ? sk::bcast_hi(kk.s[w / 4]) : sk::bcast_lo(kk.s[w / 4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[y][e] = sk::hmul2(d[y][e], sc);
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                sk::mma_16816(s[x][r], d[0][0], d[1][0], d[0][1], d[1][1], q[r].x, q[r].y);
                sk::mma_16816(s[x][r], d[0][2], d[1][2], d[0][3], d[1][3], q[r].z, q[r].w);
            }
        }
    }
}

// An 8 x 8 tile of f16 pairs, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
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

// o += v^T . p^T over the 16 positions of the record at `rec`: b[r] is the B
// operand of the weights of row tile r.  Lane g of a quad column decodes one
// block (D = 64: half of one) of two neighbouring positions at a time; tile i
// takes its components 2 i (rows g of the tile) and 2 i + 1 (rows g + 8).
template <int D, int NR>
__device__ __forceinline__ void pv(uint32_t rec, const uint32_t (&b)[NR][2], int g, int t, float (&o)[D / 16][NR][4]) {
    constexpr int NB = D == 64 ? 1 : D / 128, PER = D == 64 ? 8 : 16;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int blk = D == 64 ? g >> 1 : g + 8 * nb;
        uint32_t a[2][PER];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 v = sk::ld_shared_v4(rec + 9 * D + j * 4 * D + blk * 64 + t * 16);
            const uint32_t sc = scale_pair(sk::ld_shared_u16(rec + 17 * D + blk * 16 + 8 * j + 2 * t));
            uint32_t d[8];
            if constexpr (D == 64) {
                decode_pair((g & 1) ? v.y : v.x, (g & 1) ? v.w : v.z, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) a[j][i] = sk::hmul2(d[i], sc);
            } else {
                decode_pair(v.x, v.z, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) a[j][i] = sk::hmul2(d[i], sc);
                decode_pair(v.y, v.w, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) a[j][8 + i] = sk::hmul2(d[i], sc);
            }
        }
#pragma unroll
        for (int i = 0; i < PER / 2; ++i)
#pragma unroll
            for (int r = 0; r < NR; ++r)
                sk::mma_16816(o[nb * (PER / 2) + i][r], a[0][2 * i], a[0][2 * i + 1], a[1][2 * i], a[1][2 * i + 1],
                              b[r][0], b[r][1]);
    }
}

// Where a warp's sums lie at the merge: component pairs of a row are permuted
// so that the 16 lanes of a store (four rows, four groups of components) meet 16
// different pairs of banks (one sequence of 60000, 12 rows a head of 128: 18.8 ->
// 17.7 us).  With the accumulators of D = 256 the permutation's registers cost
// more than the conflicts of padded rows (64 sequences to 16411: 78.6 -> 79.7 us).
template <int D>
__device__ __forceinline__ int merge_swizzle(int row, int d) {
    const int t = (row >> 1) & 3;
    return D == 256 ? 0 : D == 64 ? t : 2 * t | ((d >> 5) & 1);
}

constexpr int MAX_CLUSTER = 16;

// Four components of query row r of a segment, and its statistics, from the sums
// under the base `top`.
template <int D>
__device__ __forceinline__ void write_row(const AttnParams &p, int b, int h, int row, int d, const float4 &v, float top, float l) {
    const int m = row / p.G;
    const long long to = ((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G;
    const float f = l == 0.f ? 0.f : p.vg / l;
    const __half2 y0 = __floats2half2_rn(v.x * f, v.y * f), y1 = __floats2half2_rn(v.z * f, v.w * f);
    uint2 y = make_uint2(*reinterpret_cast<const uint32_t *>(&y0), *reinterpret_cast<const uint32_t *>(&y1));
    *reinterpret_cast<uint2 *>(p.out + to * D + d) = y;
    if (d == 0) write_stats(p, to, top, l);
}

// Each warp streams its own steps of 32 positions (bulk copies into a ring of
// its own, issued by one lane a ring's length ahead) and keeps 8 NR query rows'
// bases, sums and outputs in registers; the four warps meet only at the
// end of a segment (sequence, head, row tile).
//
// SHORT: a cluster per segment, each CTA the same number of the table's tiles,
// joined through distributed shared memory.  Otherwise the CTAs share all tiles
// evenly, and kv4_join_kernel joins what they leave in the scratch memory.
//
// Bound by fixed latencies where registers leave two warps a scheduler: 64
// sequences of up to 16411 positions, 24 query over 2 kv heads of 256, the call
// 80 us (281 MB, 3.5 TB/s) with issue slots 44 % used, tensor pipe 40 %, DRAM 47
// %, and most of a warp's time between dependent instructions.  One sequence of
// 1031 positions, 48 over 4 heads of 128: 5.2 us, all of it latency.
template <int D, int NR, bool SHORT>
__global__ void __launch_bounds__(CT, (Cfg<D, NR>::CTAS)) kv4_attention_kernel(const __grid_constant__ AttnParams p) {
    using C = Cfg<D, NR>;
    constexpr int ROWS = C::ROWS, NX = C::ACC >= 64 || NR > 2 ? 1 : 2;       // records scored together
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int sm_share[WARPS + 2];
    __shared__ __align__(16) float2 all_ml[SHORT ? ROWS : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t base = sk::smem_u32(smem);
    const uint32_t qs = base + C::BODY, bars = qs + NR * C::QTILE;
    const uint32_t ring = base + warp * C::STAGES * C::STAGE, bar = bars + warp * C::STAGES * 8;
    float *const obuf = reinterpret_cast<float *>(smem);
    float2 *const mlbuf = reinterpret_cast<float2 *>(smem + C::BODY + NR * C::QTILE + WARPS * C::STAGES * 8);
    if (lane == 0)
        for (int s = 0; s < C::STAGES; ++s) sk::mbar_init(bar + s * 8, 1);
    sk::fence_barrier_init();
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    Share sh;
    if constexpr (!SHORT) sh = share_of(p, p.heads * p.RT, sm_share);
    const uint32_t CL = SHORT ? sk::cluster_size() : 1u;
    uint32_t at = 0, parity = 0;   // this warp's ring position
    const bool issuer = lane == 0 && !p.stall;
    bool dead = false;

    for (;;) {
        int b, hr, len, nt, t_lo, t_hi;
        if constexpr (SHORT) {
            const int which = int(blockIdx.x / CL), rank = int(blockIdx.x % CL);
            b = which / (p.heads * p.RT);
            hr = which - b * (p.heads * p.RT);
            len = length_of(p, b);
            nt = tiles_of(len);
            const int each = (nt + int(CL) - 1) / int(CL);
            t_lo = min(nt, rank * each);
            t_hi = min(nt, t_lo + each);
        } else {
            if (sh.t >= sh.end || sh.b >= p.B) break;
            b = sh.b;
            len = length_of(p, b);
            nt = tiles_of(len);
            if (nt == 0) {
                ++sh.b;
                continue;
            }
            hr = sh.off / nt;
            t_lo = sh.off - hr * nt;
            t_hi = min(nt, t_lo + sh.end - sh.t);
        }
        const int h = hr / p.RT, rt = hr - h * p.RT;
        const int32_t *table = p.table + (long long)b * p.width;
        const int nrec = (len + 15) / 16;

        // this warp's steps: st0, st0 + WARPS, ... (n of them)
        const int st0 = t_lo * WARPS + warp, st_hi = min(t_hi * WARPS, (len + STEP - 1) / STEP);
        const int n = st0 < st_hi ? (st_hi - st0 + WARPS - 1) / WARPS : 0;
        // Record lookups, 16 steps at a time: lane l holds record l % 2 of step
        // 16 k + l / 2; the next batch is fetched a whole batch early.
        auto lookup = [&](int k) {
            const int rec = 2 * (st0 + (16 * k + (lane >> 1)) * WARPS) + (lane & 1);
            return sk::kv4_record(table, min(rec, nrec - 1), p.recs, p.by_recs, p.pages, p.heads, h);
        };
        uint32_t now = 0, soon = 0;
        // copy step i of this warp into stage `slot`
        auto issue = [&](int i, uint32_t slot) {
            if ((i & 15) == 0) {
                now = i == 0 ? lookup(0) : soon;
                if (i + 16 < n) soon = lookup((i >> 4) + 1);
            }
            const uint32_t r0 = __shfl_sync(0xffffffffu, now, (2 * i) & 31), r1 = __shfl_sync(0xffffffffu, now, (2 * i + 1) & 31);
            if (issuer && !dead) {
                const uint32_t dst = ring + slot * C::STAGE, fb = bar + slot * 8;
                const bool two = 2 * (st0 + i * WARPS) + 1 < nrec, one_copy = two && r1 == r0 + 1;
                sk::mbar_arrive_expect_tx(fb, two ? 2 * C::REC : C::REC);
                sk::bulk_load(dst, p.cache + size_t(r0) * C::REC, one_copy ? 2 * C::REC : C::REC, fb);
                if (two && !one_copy) sk::bulk_load(dst + C::REC, p.cache + size_t(r1) * C::REC, C::REC, fb);
            }
        };
        // The query rows are asked for before the first copies: behind those of
        // all CTAs they arrive microseconds later (64 sequences of up to 16411, 24
        // over 2 heads of 256: the call 82 us, 78.4 this way).
        constexpr int QPER = (NR * C::KPAIRS * 32 + CT - 1) / CT;
        uint4 qv[QPER];
#pragma unroll
        for (int x = 0; x < QPER; ++x) qv[x] = fetch_q<D>(p, b, h, rt * ROWS, x * CT + tid);
        for (int i = 0; i < min(n, C::STAGES); ++i) {
            uint32_t slot = at + i;
            if (slot >= C::STAGES) slot -= C::STAGES;
            issue(i, slot);
        }
#pragma unroll
        for (int x = 0; x < QPER; ++x)
            if (x * CT + tid < NR * C::KPAIRS * 32) store_q(qs, x * CT + tid, qv[x]);
        __syncthreads();       // the query rows are in shared memory

        float o[D / 16][NR][4];
        float neg[NR][2], sum[NR][2];              // per row 2 t + e of tile r: minus the base, the sum
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                neg[r][e] = NO_BASE;
                sum[r][e] = 0.f;
            }
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][r][e] = 0.f;
        }
        const int all_see = len - (p.M - 1);       // positions below it are seen by every row

        for (int i = 0; i < n; ++i) {
            const uint32_t stage = ring + at * C::STAGE;
            sk::wait_ring<C::STAGES>(bar, at, parity, p.err, dead);
#pragma unroll
            for (int x0 = 0; x0 < 2; x0 += NX) {
                float s[NX][NR][4];
                {
                    Keys<D> k[2 * NX];
#pragma unroll
                    for (int j = 0; j < 2 * NX; ++j)
                        load_keys<D>(stage + (x0 + (j >> 1)) * C::REC, (j & 1) * 8 + g, t, k[j]);
                    qk<D, NX, NR>(k, qs, lane, s);
                }
                const int pos = (st0 + i * WARPS) * STEP + 16 * x0;
                if (pos + 16 * NX > all_see) {
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = rt * ROWS + 8 * r + 2 * t + e;
                            const int lim = len - (p.M - 1 - min(row / p.G, p.M - 1));
#pragma unroll
                            for (int x = 0; x < NX; ++x)
#pragma unroll
                                for (int y = 0; y < 2; ++y)
                                    if (pos + 16 * x + 8 * y + g >= lim) s[x][r][2 * y + e] = NEG_INF;
                        }
                }
                float top[NR][2];
                bool rise = false;
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[r][e] = fmaxf(s[0][r][e], s[0][r][2 + e]);
                        if constexpr (NX == 2) top[r][e] = fmaxf(top[r][e], fmaxf(s[1][r][e], s[1][r][2 + e]));
                        rise |= passes(p, top[r][e], neg[r][e]);
                    }
                if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = top[r][e];
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            const float had = neg[r][e];
                            neg[r][e] = fminf(had, neg_base(p, m));
                            const float f = rebase(p, neg[r][e], had);
                            sum[r][e] *= f;
#pragma unroll
                            for (int x = 0; x < D / 16; ++x) {
                                o[x][r][e] *= f;
                                o[x][r][2 + e] *= f;
                            }
                        }
                }
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    uint32_t w[NR][2];
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float2 w2 = weights2(p, s[x][r][2 * y], s[x][r][2 * y + 1], neg[r][0], neg[r][1]);
                            const float p0 = w2.x, p1 = w2.y;
                            sum[r][0] += p0;
                            sum[r][1] += p1;
                            w[r][y] = transpose8(pack_f16(p0, p1));
                        }
                    pv<D, NR>(stage + (x0 + x) * C::REC, w, g, t, o);
                }
            }
            __syncwarp();      // every lane has read the stage
            if (i + C::STAGES < n) issue(i + C::STAGES, at);
            if (++at == C::STAGES) {
                at = 0;
                parity ^= 1;
            }
        }

        // ---- the four warps' sums, in warp order
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[r][e] += __shfl_xor_sync(0xffffffffu, sum[r][e], 4);
                sum[r][e] += __shfl_xor_sync(0xffffffffu, sum[r][e], 8);
                sum[r][e] += __shfl_xor_sync(0xffffffffu, sum[r][e], 16);
                if (g == 0) mlbuf[warp * ROWS + 8 * r + 2 * t + e] = make_float2(-neg[r][e], sum[r][e]);
            }
        __syncthreads();       // every warp is done with its ring
        {
            float *dst = obuf + warp * ROWS * C::OSTRIDE;
            constexpr int PER = D == 64 ? 8 : 16;
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = PER * (g + 8 * (x / (PER / 2))) + 2 * (x % (PER / 2)), row = 8 * r + 2 * t + e;
                        *reinterpret_cast<float2 *>(dst + row * C::OSTRIDE + (d ^ (2 * merge_swizzle<D>(row, d)))) =
                            make_float2(o[x][r][e], o[x][r][2 + e]);
                    }
        }
        __syncthreads();
        const bool whole = SHORT ? CL == 1u : t_lo == 0 && t_hi == nt;
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
            const int sw = merge_swizzle<D>(r, d), at_r = d ^ (2 * (sw & ~1));     // the four of d: pairs change places if sw is odd
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float f = rebase(p, ml[w].x, top);
                const float4 x = *reinterpret_cast<const float4 *>(obuf + (w * ROWS + r) * C::OSTRIDE + at_r);
                l += ml[w].y * f;
                v.x += x.x * f;
                v.y += x.y * f;
                v.z += x.z * f;
                v.w += x.w * f;
            }
            if (sw & 1) v = make_float4(v.z, v.w, v.x, v.y);
            if (whole) {
                write_row<D>(p, b, h, rt * ROWS + r, d, v, top, l);
            } else if constexpr (SHORT) {
                // in warp 0's place: no other thread reads it
                *reinterpret_cast<float4 *>(obuf + r * C::OSTRIDE + at_r) = v;
                if (d == 0) all_ml[r] = make_float2(top, l);
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (slot * ROWS + r) * D + d) = v;
                if (d == 0) *reinterpret_cast<float2 *>(p.part_ml + (slot * ROWS + r) * 2) = make_float2(top, l);
            }
        }
        if constexpr (SHORT) {
            if (CL == 1u) break;
            sk::cluster_sync();
            // the cluster's, in its order, every CTA a part of the rows and components
            const uint32_t ml_at = sk::smem_u32(all_ml);
            for (int i = int(blockIdx.x % CL) * CT + tid; i < rows * (D / 4); i += int(CL) * CT) {
                const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
                float2 ml[MAX_CLUSTER];
                float4 x[MAX_CLUSTER];
#pragma unroll
                for (uint32_t k = 0; k < MAX_CLUSTER; ++k) {
                    ml[k] = make_float2(NEG_INF, 0.f);
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < CL) {
                        ml[k] = sk::ld_peer_v2(sk::peer(ml_at + r * 8, k));
                        x[k] = sk::ld_peer_v4(sk::peer(base + (r * C::OSTRIDE + (d ^ (2 * (merge_swizzle<D>(r, d) & ~1)))) * 4, k));
                    }
                }
                float top = NEG_INF, l = 0.f;
#pragma unroll
                for (int k = 0; k < MAX_CLUSTER; ++k) top = fmaxf(top, ml[k].x);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < MAX_CLUSTER; ++k) {
                    const float f = rebase(p, ml[k].x, top);
                    l += ml[k].y * f;
                    v.x += x[k].x * f;
                    v.y += x[k].y * f;
                    v.z += x[k].z * f;
                    v.w += x[k].w * f;
                }
                write_row<D>(p, b, h, rt * ROWS + r, d, v, top, l);
            }
            sk::cluster_sync();                      // no CTA leaves while its sums are read
            break;
        } else {
        if (tid == 0 && t_lo == 0) {
            const int c1 = cta_of(sh, sh.t + nt - 1);     // of the segment's last tile
            p.seg[(b * p.heads + h) * p.RT + rt] = make_int2(int(blockIdx.x), whole ? 0 : c1 - int(blockIdx.x) + 1);
        }
        // the ring's next copies come after these reads and writes of it
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        sh.t += t_hi - t_lo;
        sh.off += t_hi - t_lo;
        if (sh.off == nt * p.heads * p.RT) {
            ++sh.b;
            sh.off = 0;
        }
        }
    }
}

// DC components of a query row per CTA: the partial sums of its segment, in the
// order of the CTAs that wrote them, joined under the largest base.  DC / 4
// threads take a part at a time, 1024 / DC parts together.  Rows of an empty
// sequence are written here too (zero, with a log sum of minus infinity).
constexpr int JT = 256;

template <int D, int DC>
__global__ void __launch_bounds__(JT) kv4_join_kernel(const __grid_constant__ AttnParams p, int tile_rows) {
    constexpr int COLS = DC / 4, GROUPS = JT / COLS, CHUNKS = D / DC;
    extern __shared__ float2 ml[];                 // (base, sum) of each part, then (factor, -)
    __shared__ float red[JT / 32], red_l[JT / 32];
    __shared__ float4 part[GROUPS][COLS];
    // (Here and in the weights' kernel nothing is let in early.  The kernel after
    // it fills an SM's registers to the last block, and CTAs of it placed around
    // this kernel's leave a hole that is too small for the last one, which then
    // runs after the others: 64 sequences of 3000, 48 query over 4 heads of 128,
    // calls in a row 58 us each, 42 without, with the weights 90 and 62.)
    sk::pdl_wait_primary();
    const int rows = p.M * p.G, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int which = blockIdx.x / CHUNKS, d0 = (blockIdx.x - which * CHUNKS) * DC;
    const int bh = which / rows, row = which - bh * rows, b = bh / p.heads, h = bh - b * p.heads;
    const int rt = row / tile_rows, r = row - rt * tile_rows, m = row / p.G;
    const int2 seg = p.seg[bh * p.RT + rt];        // of an earlier call where the sequence is empty
    const bool empty = length_of(p, b) == 0;
    if (!empty && seg.y == 0) return;
    const long long at = ((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G;
    if (empty) {
        for (int d = tid; d < DC; d += JT) p.out[at * D + d0 + d] = __float2half_rn(0.f);
        if (tid == 0 && d0 == 0 && p.lse) p.lse[at] = NEG_INF;
        return;
    }
    const int n = seg.y;
    // slot of part i: the first CTA's second slot, the first slot of the others
    auto slot = [&](int i) { return (size_t(seg.x) + i) * 2 + (i == 0 ? 1 : 0); };
    float top = NEG_INF;
    for (int i = tid; i < n; i += JT) {
        const float2 v = *reinterpret_cast<const float2 *>(p.part_ml + (slot(i) * tile_rows + r) * 2);
        ml[i] = v;
        top = fmaxf(top, v.x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[wid] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < JT / 32; ++w) top = fmaxf(top, red[w]);
    float l = 0.f;
    for (int i = tid; i < n; i += JT) {
        const float f = rebase(p, ml[i].x, top);
        l += ml[i].y * f;
        ml[i].x = f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red_l[wid] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < JT / 32; ++w) l += red_l[w];
    const int grp = tid / COLS, col = tid - grp * COLS;
    const float *src = p.part_o + size_t(r) * D + d0 + col * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = grp; i < n; i += GROUPS) {
        const float4 y = *reinterpret_cast<const float4 *>(src + slot(i) * tile_rows * D);
        const float f = ml[i].x;
        v.x += y.x * f;
        v.y += y.y * f;
        v.z += y.z * f;
        v.w += y.w * f;
    }
    part[grp][col] = v;
    __syncthreads();
    for (int d = tid; d < DC; d += JT) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < GROUPS; ++w) y += reinterpret_cast<const float *>(part[w])[d];
        p.out[at * D + d0 + d] = __float2half_rn(l == 0.f ? 0.f : y * (p.vg / l));
    }
    if (tid == 0 && d0 == 0) write_stats(p, at, top, l);
}

// The same with a warp per row, for segments of few parts: no barriers.
template <int D>
__global__ void __launch_bounds__(JT) kv4_join_rows_kernel(const __grid_constant__ AttnParams p, int tile_rows) {
    constexpr int PER = D / 32;                    // components per lane: two neighbouring ones, 64 apart
    sk::pdl_wait_primary();
    const int rows = p.M * p.G, lane = threadIdx.x & 31;
    const int which = blockIdx.x * (JT / 32) + (threadIdx.x >> 5);
    const int bh = which / rows, row = which - bh * rows, b = bh / p.heads, h = bh - b * p.heads;
    if (b >= p.B) return;
    const int rt = row / tile_rows, r = row - rt * tile_rows, m = row / p.G;
    const int2 seg = p.seg[bh * p.RT + rt];        // of an earlier call where the sequence is empty
    const bool empty = length_of(p, b) == 0;
    if (!empty && seg.y == 0) return;
    const long long at = ((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G;
    __half2 *const out = reinterpret_cast<__half2 *>(p.out + at * D) + lane;
    if (empty) {
#pragma unroll
        for (int x = 0; x < PER / 2; ++x) out[32 * x] = __floats2half2_rn(0.f, 0.f);
        if (lane == 0 && p.lse) p.lse[at] = NEG_INF;
        return;
    }
    const int n = seg.y;
    auto slot = [&](int i) { return (size_t(seg.x) + i) * 2 + (i == 0 ? 1 : 0); };
    float top = NEG_INF, l = 0.f, v[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) v[x] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {           // 32 parts at a time, under the largest base so far
        float2 ml = make_float2(NEG_INF, 0.f);
        if (i0 + lane < n) ml = *reinterpret_cast<const float2 *>(p.part_ml + (slot(i0 + lane) * tile_rows + r) * 2);
        float now = ml.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
        now = fmaxf(now, top);
        const float old = rebase(p, top, now), f = rebase(p, ml.x, now);
        top = now;
        float add = ml.y * f;
#pragma unroll
        for (int o = 16; o; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
        l = l * old + add;
#pragma unroll
        for (int x = 0; x < PER; ++x) v[x] *= old;
        const int k = min(32, n - i0);
#pragma unroll 4
        for (int i = 0; i < k; ++i) {
            const float w = __shfl_sync(0xffffffffu, f, i);
            const float2 *src = reinterpret_cast<const float2 *>(p.part_o + (slot(i0 + i) * tile_rows + r) * D) + lane;
#pragma unroll
            for (int x = 0; x < PER / 2; ++x) {
                const float2 y = src[32 * x];
                v[2 * x] += y.x * w;
                v[2 * x + 1] += y.y * w;
            }
        }
    }
    const float f = l == 0.f ? 0.f : p.vg / l;
#pragma unroll
    for (int x = 0; x < PER / 2; ++x) out[32 * x] = __floats2half2_rn(v[2 * x] * f, v[2 * x + 1] * f);
    if (lane == 0) write_stats(p, at, top, l);
}

// acc_out = acc_in + the weights of all query rows, per position and kv head:
// the scores once more (the keys alone are read), against the rows' final bases
// and sums.  A warp owns the 32 positions of a step, whose sum over the rows is
// taken in one order; the next step's keys are on their way meanwhile.  (Taken
// during the attention the weights would need each row's final sum, which is
// not known until its last position.)  23 sequences of up to 9001 positions, 2
// rows, 32 over 8 heads of 64: the whole call 41 us, this pass about 20 of it,
// issue slots half used.  (Scores kept by the first pass would be 4 bytes per
// position and row each way: 25 MB twice in this case, 7.5 us at the copy rate.
// Not built.)
constexpr int WT_TILES = 16;           // tiles of eight rows held in shared memory at a time
constexpr int WT_STAGES = 4;
constexpr int ACC_STEPS = 4;           // steps whose accumulated weights are on their way

template <int D>
struct WeightsCfg {
    static constexpr int KEY = 9 * D;                // the keys' part of a record
    static constexpr int STAGE = 2 * KEY;
    static constexpr int RING = WARPS * WT_STAGES * STAGE;
    static constexpr int QTILE = D / 32 * 512;
    static constexpr int FIXED = RING + WARPS * WT_STAGES * 8;
    static constexpr int CTAS = D == 256 ? 2 : 4;
};

template <int D>
__global__ void __launch_bounds__(CT, WeightsCfg<D>::CTAS)
    kv4_weights_kernel(const __grid_constant__ AttnParams p, int tiles) {
    using C = WeightsCfg<D>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int sm_share[WARPS + 2];
    // minus each row's base, and minus log2 of its sum
    __shared__ __align__(8) float neg[WT_TILES * NROW], neg_g[WT_TILES * NROW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t base = sk::smem_u32(smem), qs = base + C::FIXED;
    const uint32_t ring = base + warp * WT_STAGES * C::STAGE, bar = base + C::RING + warp * WT_STAGES * 8;
    if (lane == 0)
        for (int s = 0; s < WT_STAGES; ++s) sk::mbar_init(bar + s * 8, 1);
    sk::fence_barrier_init();
    sk::pdl_wait_primary();
    Share sh = share_of(p, p.heads, sm_share);
    uint32_t it = 0;               // steps this warp has consumed
    const bool issuer = lane == 0 && !p.stall;
    bool dead = false;
    // this lane's position in a step once the sums are spread: record t / 2, half t % 2, position g
    const int mine = (t >> 1) * 16 + (t & 1) * 8 + g;
    while (sh.t < sh.end && sh.b < p.B) {
        const int len = length_of(p, sh.b), nt = tiles_of(len);
        if (nt == 0) {
            ++sh.b;
            continue;
        }
        const int h = sh.off / nt, t_lo = sh.off - h * nt, b = sh.b;
        const int t_hi = min(nt, t_lo + sh.end - sh.t);
        const int32_t *table = p.table + (long long)b * p.width;
        const int rows = p.M * p.G, nrec = (len + 15) / 16;
        const size_t acc_at = (size_t(b) * p.heads + h) * size_t(p.cap);
        const int st0 = t_lo * WARPS + warp, st_hi = min(t_hi * WARPS, (len + STEP - 1) / STEP);
        const int n = st0 < st_hi ? (st_hi - st0 + WARPS - 1) / WARPS : 0;
        for (int r0 = 0; r0 < tiles; r0 += WT_TILES) {
            const int nr = min(WT_TILES, tiles - r0);
            auto lookup = [&](int k) {
                const int rec = 2 * (st0 + (16 * k + (lane >> 1)) * WARPS) + (lane & 1);
                return sk::kv4_record(table, min(rec, nrec - 1), p.recs, p.by_recs, p.pages, p.heads, h);
            };
            uint32_t now = 0, soon = 0;
            auto issue = [&](int i, uint32_t slot) {
                if ((i & 15) == 0) {
                    now = i == 0 ? lookup(0) : soon;
                    if (i + 16 < n) soon = lookup((i >> 4) + 1);
                }
                const uint32_t a = __shfl_sync(0xffffffffu, now, (2 * i) & 31), c = __shfl_sync(0xffffffffu, now, (2 * i + 1) & 31);
                if (issuer && !dead) {
                    const uint32_t dst = ring + slot * C::STAGE, fb = bar + slot * 8;
                    const bool two = 2 * (st0 + i * WARPS) + 1 < nrec;
                    sk::mbar_arrive_expect_tx(fb, two ? 2 * C::KEY : C::KEY);
                    sk::bulk_load(dst, p.cache + size_t(a) * sk::kv4_rec_bytes(D), C::KEY, fb);
                    if (two) sk::bulk_load(dst + C::KEY, p.cache + size_t(c) * sk::kv4_rec_bytes(D), C::KEY, fb);
                }
            };
            for (int i = 0; i < min(n, WT_STAGES); ++i) issue(i, (it + i) % WT_STAGES);
            __syncthreads();
            for (int x = tid; x < nr * (D / 32) * 32; x += CT) store_q(qs, x, fetch_q<D>(p, b, h, r0 * NROW, x));
            for (int x = tid; x < nr * NROW; x += CT) {
                const int row = r0 * NROW + x, m = row / p.G;
                // a row that sees nothing (or does not exist) gives no weight: 2^-inf
                float2 v = make_float2(0.f, -NEG_INF);
                if (row < rows) v = p.norm[((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G];
                neg[x] = v.x;
                neg_g[x] = -v.y;
            }
            __syncthreads();
            const float *old = r0 == 0 ? p.acc_in : p.acc_out;
            auto fetch = [&](int i) {      // what the lane's position of step i had
                const int pos = (st0 + i * WARPS) * STEP + mine;
                return old && i < n && pos < len ? old[acc_at + pos] : 0.f;
            };
            float had[ACC_STEPS];              // (a rotation through moves would wait for each)
#pragma unroll
            for (int j = 0; j < ACC_STEPS; ++j) had[j] = fetch(j);
            for (int i0 = 0; i0 < n; i0 += ACC_STEPS) {
#pragma unroll
                for (int j = 0; j < ACC_STEPS; ++j) {
                    const int i = i0 + j;
                    if (i >= n) break;
                    const uint32_t slot = it % WT_STAGES, stage = ring + slot * C::STAGE;
                    sk::wait_ring<WT_STAGES>(bar, slot, (it / WT_STAGES) & 1, p.err, dead);
                    Keys<D> k[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) load_keys<D>(stage + (x >> 1) * C::KEY, (x & 1) * 8 + g, t, k[x]);
                    const int pos = (st0 + i * WARPS) * STEP;
                    const bool edge = pos + STEP > len - (p.M - 1);
                    float w[4] = {0.f, 0.f, 0.f, 0.f};     // record x, half y: w[2 x + y], of position g
                    for (int r = 0; r < nr; ++r) {
                        float s[2][1][4];
                        qk<D, 2, 1>(k, qs + r * C::QTILE, lane, s);
                        const float2 n = *reinterpret_cast<const float2 *>(&neg[r * NROW + 2 * t]);
                        const float2 ng = *reinterpret_cast<const float2 *>(&neg_g[r * NROW + 2 * t]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float *v = s[x >> 1][0] + 2 * (x & 1);
                            const float2 y = weights2(p, v[0], v[1], n, ng);
                            v[0] = y.x;
                            v[1] = y.y;
                        }
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int lim = len - (p.M - 1 - min(((r0 + r) * NROW + 2 * t + e) / p.G, p.M - 1));
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    if (pos + 8 * x + g >= lim) s[x >> 1][0][2 * (x & 1) + e] = 0.f;
                            }
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) w[x] += s[x >> 1][0][2 * (x & 1)] + s[x >> 1][0][2 * (x & 1) + 1];
                    }
                    __syncwarp();
                    if (i + WT_STAGES < n) issue(i + WT_STAGES, slot);
                    // sums over the four t, halving what a lane keeps
#pragma unroll
                    for (int half = 2; half >= 1; half >>= 1) {
                        const bool up = t & half;
#pragma unroll
                        for (int x = 0; x < half; ++x) {
                            const float give = up ? w[x] : w[x + half], keep = up ? w[x + half] : w[x];
                            w[x] = keep + __shfl_xor_sync(0xffffffffu, give, half);
                        }
                    }
                    if (pos + mine < len) p.acc_out[acc_at + pos + mine] = had[j] + w[0];
                    had[j] = fetch(i + ACC_STEPS);
                    ++it;
                }
            }
        }
        sh.t += t_hi - t_lo;
        sh.off += t_hi - t_lo;
        if (sh.off == nt * p.heads) {
            ++sh.b;
            sh.off = 0;
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int MAX_SEGMENTS = 131072;
// More query rows of a kv head than these go to the tensor-core kernel, which
// decodes a tile once for up to 96 rows where the registers hold 24 to 32:
// 60000 positions, 4 heads of 128, 96 rows 36 us against 52, 36 rows 26.6
// against 30.3, 24 rows 24.2 against 21.4; 8 heads, 28 rows, 64 sequences of 300
// 28 against 30 and 16 of 20000 139 against 153, 24 rows 27 against 25 and 139
// against 118.
constexpr int TC_ABOVE = 24;

// The scratch memory: the segment list, the rows' statistics where weights are
// accumulated (16 MiB at most: MAX_SEGMENTS tiles of 16 rows), and in the rest
// the partial sums for `rows` per tile.
unsigned char *place_rows(AttnParams &p, unsigned char *scratch) {
    p.seg = reinterpret_cast<int2 *>(scratch);
    scratch += size_t(MAX_SEGMENTS) * sizeof(int2);
    if (!p.acc_out) return scratch;
    p.norm = reinterpret_cast<float2 *>(scratch);
    return scratch + (size_t(p.B) * p.heads * p.M * p.G * sizeof(float2) + 255) / 256 * 256;
}
bool place_partials(AttnParams &p, unsigned char *rest, int rows, int D) {
    p.part_ml = reinterpret_cast<float *>(rest);
    p.part_o = p.part_ml + size_t(p.ctas) * 2 * rows * 2;
    return size_t(reinterpret_cast<unsigned char *>(p.part_o + size_t(p.ctas) * 2 * rows * D) -
                  reinterpret_cast<unsigned char *>(p.seg)) <= sk::SCRATCH_BYTES;
}

template <int D>
sk_status join(const AttnParams &p, int tile_rows, int sms, cudaStream_t s) {
    // By how many parts a segment has on average: few, a warp per row (64
    // sequences of 2 heads, 3 parts: the call 84 -> 82 us); many, a CTA per row, and
    // where the rows are few as well, each split over CTAs of 32 components, so
    // that a thread's parts are all in flight (ten rows of 456 parts: the call
    // 24 -> 15 us).
    const long long rows = (long long)p.B * p.heads * p.M * p.G, segments = (long long)p.B * p.heads * p.RT;
    const size_t smem = size_t(p.ctas) * sizeof(float2);
    cudaError_t e;
    if (p.ctas <= 8 * segments)
        e = sk::launch_pdl(kv4_join_rows_kernel<D>, dim3(unsigned((rows + JT / 32 - 1) / (JT / 32))), dim3(JT), 0, s, p,
                           tile_rows);
    else if (rows <= sms)
        e = sk::launch_pdl(kv4_join_kernel<D, 32>, dim3(unsigned(rows) * (D / 32)), dim3(JT), smem, s, p, tile_rows);
    else
        e = sk::launch_pdl(kv4_join_kernel<D, D>, dim3(unsigned(rows)), dim3(JT), smem, s, p, tile_rows);
    return e == cudaSuccess ? SK_OK : SK_ERR_CUDA;
}

// CTAs per segment with which all segments run at a time, each CTA with few of
// the table's tiles; 0 where there is no such number.
// Few: one launch then takes less than two and the scratch memory's round trip
// (48 query over 4 heads of 128, one sequence of 1031 positions 5.4 us against
// 7.7, of 7900 8.4 against 9.5; 50 of up to 500 9.5 against 11.5); with eight
// tiles each one of 16000 takes 12.5 against 11.3.  In place of the tensor cores
// (rows above TC_ABOVE) half as many: 32 rows, one of 4000 10.1 against 12.5.
constexpr int SHORT_TILES = 4;
template <int D, int NR>
int short_cluster(const AttnParams &p, int few) {
    using C = Cfg<D, NR>;
    constexpr auto kernel = kv4_attention_kernel<D, NR, true>;
    if (sk::prepare_kernel<kernel>(C::SMEM, true) != cudaSuccess) return 0;
    const long long segments = (long long)p.B * p.heads * p.RT, tiles = ((long long)p.cap + TILE - 1) / TILE;
    int c = 1;
    while (c < MAX_CLUSTER && c < tiles && segments <= sk::resident_clusters<kernel>(c * 2, CT, C::SMEM)) c *= 2;
    return tiles <= (long long)c * few && segments <= sk::resident_clusters<kernel>(c, CT, C::SMEM) ? c : 0;
}

// The launch of that form, where there is one.
template <int D, int NR>
bool attend_short(const AttnParams &p, int few, cudaStream_t s, sk_status *st) {
    const int cluster = short_cluster<D, NR>(p, few);
    if (!cluster) return false;
    const dim3 grid(unsigned(cluster) * unsigned(p.B * p.heads * p.RT));
    *st = sk::launch_pdl_cluster(kv4_attention_kernel<D, NR, true>, cluster, grid, dim3(CT), Cfg<D, NR>::SMEM, s, p) ==
                  cudaSuccess
              ? SK_OK
              : SK_ERR_CUDA;
    return true;
}

template <int D, int NR>
sk_status attend(AttnParams &p, unsigned char *rest, int sms, cudaStream_t s) {
    using C = Cfg<D, NR>;
    sk_status st;
    if (attend_short<D, NR>(p, SHORT_TILES, s, &st)) return st;
    p.ctas = sms * C::CTAS;
    if (!place_partials(p, rest, C::ROWS, D)) return SK_ERR_WORKSPACE;
    if (sk::prepare_kernel<kv4_attention_kernel<D, NR, false>>(C::SMEM) != cudaSuccess) return SK_ERR_CUDA;
    if (sk::launch_pdl(kv4_attention_kernel<D, NR, false>, dim3(p.ctas), dim3(CT), C::SMEM, s, p) != cudaSuccess)
        return SK_ERR_CUDA;
    return join<D>(p, C::ROWS, sms, s);
}

sk_status attend_tc(AttnParams &p, unsigned char *rest, int sms, cudaStream_t s) {
    const int rows = tc_rows(p.M * p.G, &p.RT);
    p.ctas = sms * TC_CTAS;
    if (!place_partials(p, rest, rows, 128)) return SK_ERR_WORKSPACE;
    if (launch_tc(p, rows, s) != cudaSuccess) return SK_ERR_CUDA;
    return join<128>(p, rows, sms, s);
}

template <int D>
sk_status run(AttnParams &p, unsigned char *scratch, int sms, cudaStream_t s) {
    // Query rows of a kv head in tiles of 8 NR rows, as even as they can be: NR
    // up to 4 (the outputs are D / 4 NR registers a thread; D = 256: up to 2;
    // D = 128: up to 3, more rows go to the tensor cores).
    constexpr int MOST = D == 256 ? 2 : D == 128 ? TC_ABOVE / NROW : 4;
    const int tiles = (p.M * p.G + NROW - 1) / NROW;       // of eight rows
    p.RT = (tiles + MOST - 1) / MOST;
    const int nr = (tiles + p.RT - 1) / p.RT;
    unsigned char *const rest = place_rows(p, scratch);
    sk_status st;
    if (D == 128 && p.M * p.G > TC_ABOVE) {
        const bool done = nr == 3 ? attend_short<128, 3>(p, SHORT_TILES / 2, s, &st)
                                  : attend_short<128, 2>(p, SHORT_TILES / 2, s, &st);
        if (!done) st = attend_tc(p, rest, sms, s);
    } else if (nr == 1) st = attend<D, 1>(p, rest, sms, s);
    else if (nr == 2) st = attend<D, 2>(p, rest, sms, s);
    else if constexpr (MOST == 4) st = nr == 3 ? attend<D, 3>(p, rest, sms, s) : attend<D, 4>(p, rest, sms, s);
    else if constexpr (MOST == 3) st = attend<D, 3>(p, rest, sms, s);
    else return SK_ERR_UNSUPPORTED_SHAPE;
    if (st != SK_OK || !p.acc_out) return st;
    const int held = tiles < WT_TILES ? tiles : WT_TILES;
    using W = WeightsCfg<D>;
    p.ctas = sms * W::CTAS;
    if (sk::prepare_kernel<kv4_weights_kernel<D>>(W::FIXED + WT_TILES * W::QTILE) != cudaSuccess) return SK_ERR_CUDA;
    return sk::launch_pdl(kv4_weights_kernel<D>, dim3(p.ctas), dim3(CT), size_t(W::FIXED) + size_t(held) * W::QTILE, s, p,
                          tiles) == cudaSuccess
               ? SK_OK
               : SK_ERR_CUDA;
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
    // The kernels use the product: it neither vanishes nor is infinite, nor is
    // the largest score (256 65504 2688) times it, nor P_SHIFT + SLACK divided by
    // it; and it takes NO_BASE far enough from any base that a sum under NO_BASE
    // counts for nothing (2^-64).
    const double product = double(scale) * double(k_scale);
    if (!(product >= 5e-37 && product <= 1e27)) return SK_ERR_INVALID_ARG;
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
    // (sequence, kv head, tile of 16 rows) fit the segment list, whatever tiles the head size gets
    if ((long long)seqs * kv_heads * ((rows * p.G + 15) / 16) > MAX_SEGMENTS ||
        (long long)seqs * q_heads * rows > 0x7FFFFFFLL)
        return SK_ERR_UNSUPPORTED_SHAPE;
    // tiles of positions, over all segments, fit 31 bits
    if ((long long)seqs * kv_heads * ((rows * p.G + 7) / 8) * (((long long)table_width * page_size + TILE - 1) / TILE) > 0x7FFFFFFFLL)
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
    p.by_recs = sk::Div(p.recs);
    p.width = table_width;
    p.cap = table_width * page_size;
    p.c = float(product * double(LOG2E));
    p.shift = P_SHIFT / p.c;
    p.reach = (P_SHIFT + SLACK) / p.c;
    p.vg = v_scale;
    p.stall = sk::take_inject_stall();
    switch (head_dim) {
        case 64: return run<64>(p, sc.base, sc.num_sms, s);
        case 128: return run<128>(p, sc.base, sc.num_sms, s);
        default: return run<256>(p, sc.base, sc.num_sms, s);
    }
}
