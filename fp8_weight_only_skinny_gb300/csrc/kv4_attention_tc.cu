// kv4_attention_tc.cu -- the attention over the 4-bit cache for many query rows
// per kv head (verify rounds over grouped heads), on the fifth-generation
// tensor cores.  Head size 128.
//
// With the positions as the 128-wide operand and the N query rows as the
// narrow one, a tile of 128 positions is two products:
//     S (128 x N, TMEM)  = K (128 x 128) . q^T       A: keys decoded into TMEM
//     O (128 x N, TMEM) += V^T (128 x 128) . p^T     A: values decoded into
//                                                    shared memory, read along d
// so decoded keys never pass through shared memory, and both accumulators are
// N columns.  A thread of the softmax holds one position: the row bases
// are the same for all threads and move rarely (kv4_attention.cuh), and the sums
// of the weights are added up across positions once per segment.  Two CTAs
// share an SM: one's decoding covers the other's products and softmax.
//
// Bound by the softmax's and the decoding's instructions between barriers, not
// by the products: 100003 positions of 4 heads, 8 rows of 48 query heads (96
// rows a kv head), 46 us with the join, 420 TFLOP/s (58 MB read); with 24-row
// tiles in registers 79 us.  The scores of a position are read from TMEM a few
// rows at a time: all 48 at once leave the sums no registers (52 us).  (A ninth
// warp for products and copies leaves 96 registers a thread: spills, 62 us.)
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/skinny.h"
#include "internal.h"
#include "kv4_attention.cuh"
#include "launch_util.cuh"

namespace {

using namespace sk::attn;

constexpr int D = 128;
static_assert(TILE == 128, "positions per tile");
constexpr int TT = 256;                // threads: eight warps
constexpr int REC = sk::kv4_rec_bytes(D);
constexpr int PART = REC / 2;          // the keys' or the values' half of a record
constexpr int UNIT = 8 * PART;         // of a tile's eight records: the unit of the ring
constexpr float MOST_WEIGHT = 32768.f; // 2^(P_SHIFT + SLACK): a larger weight moves its row's base
static_assert(P_SHIFT + SLACK == 15.f, "MOST_WEIGHT");

template <int N>
struct Tc {
    static constexpr int UNITS = N <= 64 ? 4 : 3;
    static constexpr int V = 0, Q = V + 128 * D * 2, P = Q + N * D * 2, RAW = P + N * 128 * 2, SMALL = RAW + UNITS * UNIT;
    // per row: minus its base, that before it moved, a factor, the first unseen position; four warps' values of each
    // row; barriers of the ring, of the two products and of the end; the TMEM
    // address
    static constexpr int NEG = SMALL, OLD = NEG + 4 * N, FAC = OLD + 4 * N, LIM = FAC + 4 * N,
                         WARP = LIM + 4 * N, BARS = WARP + 16 * N, TMEM = BARS + 8 * (UNITS + 3);
    static constexpr size_t SMEM = 1024 + TMEM + 16;
    static constexpr int S_COL = 64, O_COL = 64 + N;         // TMEM columns: keys 0..63, S, O
    static_assert(O_COL + N <= 256, "half of the TMEM");
};

// ------------------------------------------------------- tcgen05 ----------

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory operand: start address, the two strides, swizzle (0 none, 2 of
// 128 bytes).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride, uint64_t swizzle) {
    return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t((lead >> 4) & 0x3FFFu) << 16) |
           (uint64_t((stride >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (swizzle << 61);
}
// D (FP32) of M = 128, N columns, FP16 operands; bits 15 and 16: A and B stored
// along M and N.
__host__ __device__ constexpr uint32_t shape(int n, bool a_along_m, bool b_along_n) {
    return (1u << 4) | (uint32_t(a_along_m) << 15) | (uint32_t(b_along_n) << 16) | (uint32_t(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void mma_smem_a(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
// Arrive on `bar` when the products issued so far by this thread are done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// NH columns of this warp's 32 lanes, all loads in flight together.
template <int NH>
__device__ __forceinline__ void ld_row(uint32_t addr, float (&v)[NH]) {
#pragma unroll
    for (int c = 0; c < NH; c += 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[c]), "=f"(v[c + 1]), "=f"(v[c + 2]), "=f"(v[c + 3]), "=f"(v[c + 4]), "=f"(v[c + 5]),
                       "=f"(v[c + 6]), "=f"(v[c + 7])
                     : "r"(addr + c) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // no use of the values is moved ahead of the wait
#pragma unroll
    for (int c = 0; c < NH; c += 8)
        asm volatile("" : "+f"(v[c]), "+f"(v[c + 1]), "+f"(v[c + 2]), "+f"(v[c + 3]), "+f"(v[c + 4]), "+f"(v[c + 5]),
                          "+f"(v[c + 6]), "+f"(v[c + 7]));
}
// Eight columns of this warp's 32 lanes.
__device__ __forceinline__ void ld8(uint32_t addr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr) : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void st8(uint32_t addr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "r"(addr)
                 : "memory");
}
// Sixteen lanes x 32 columns: lane (g, t) of the warp gives columns 8 j + 2 t and
// 8 j + 2 t + 1 of rows g (v[4 j], v[4 j + 1]) and g + 8 (v[4 j + 2], v[4 j + 3]).
__device__ __forceinline__ void st_16x32(uint32_t addr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(addr) : "memory");
}

// Eight rows' numbers from shared memory.
__device__ __forceinline__ void row8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Keys of the record at `rec` (shared memory) into 16 lanes of TMEM.  A lane
// decodes 32 components of positions g and g + 8 (components 32 t on); column
// 8 j + 2 t + x takes components 32 t + 4 j + 2 x and the next, the order in
// which load_q places the query rows.
__device__ __forceinline__ void decode_keys(uint32_t rec, uint32_t tmem, int g, int t) {
    uint4 k[2];
    uint32_t sc[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int i = g + 8 * y;
        k[y] = sk::ld_shared_v4(rec + i * 64 + t * 16);
        sc[y] = scale_pair(sk::ld_shared_u16(rec + 8 * D + i * 8 + t * 2));
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {                         // a block of 16 components: 32 columns
        uint32_t v[16];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t w[2] = {hf ? k[y].z : k[y].x, hf ? k[y].w : k[y].y};
            const uint32_t s = hf ? sk::bcast_hi(sc[y]) : sk::bcast_lo(sc[y]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t d[4];
                sk::e2m1x8_to_f16x2x4(w[q], d);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int pair = 4 * q + e;              // = 2 j + x
                    v[4 * (pair >> 1) + 2 * y + (pair & 1)] = sk::hmul2(d[e], s);
                }
            }
        }
        st_16x32(tmem + 32 * hf, v);
    }
}

// Values of a record (their half of it; positions pos0 .. pos0 + 15 of the tile) to the operand
// of the second product: 64 components (128 bytes) of a position in a row, eight
// positions an atom of 1024 bytes whose 16-byte pieces are swizzled, the upper
// 64 components 16 KB further.
__device__ __forceinline__ void decode_values(uint32_t rec, uint32_t vbase, int pos0, int lane) {
    const int blk = lane >> 2, pair = (lane & 3) * 2;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const uint4 c = sk::ld_shared_v4(rec + hf * 4 * D + lane * 16);
        const uint32_t s = scale_pair(sk::ld_shared_u16(rec + 8 * D + blk * 16 + hf * 8 + pair));
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int y = 0; y < 2; ++y) {                        // the two positions
            const uint32_t sc = y ? sk::bcast_hi(s) : sk::bcast_lo(s);
            const int row = pair + y;
            const uint32_t at = vbase + (blk >> 2) * 16384 + ((pos0 >> 3) + hf) * 1024 + row * 128;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                uint32_t d[4];
                sk::e2m1x8_to_f16x2x4(w[2 * y + z], d);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] = sk::hmul2(d[e], sc);
                st_shared_v4(at + ((((blk & 3) * 2 + z) ^ row) << 4), d[0], d[1], d[2], d[3]);
            }
        }
    }
}

template <int N>
__global__ void __launch_bounds__(TT, 2) kv4_attention_tc_kernel(const __grid_constant__ AttnParams p) {
    using C = Tc<N>;
    constexpr int NH = N / 2, UNITS = C::UNITS;              // columns per thread; units in the ring
    extern __shared__ unsigned char dyn[];
    __shared__ int sm_share[TT / 32 + 2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int quad = warp & 3, side = warp >> 2;             // this warp's TMEM lanes and its half of the columns
    const uint32_t base = (sk::smem_u32(dyn) + 1023u) & ~1023u;
    unsigned char *const smem = dyn + (base - sk::smem_u32(dyn));
    float *const neg = reinterpret_cast<float *>(smem + C::NEG);
    float *const old = reinterpret_cast<float *>(smem + C::OLD), *const fac = reinterpret_cast<float *>(smem + C::FAC);
    int *const lim = reinterpret_cast<int *>(smem + C::LIM);
    float *const of_warp = reinterpret_cast<float *>(smem + C::WARP);
    const uint32_t bars = base + C::BARS, bar_s = bars + 8 * UNITS, bar_o = bar_s + 8, bar_end = bar_o + 8;

    if (warp == 0) tmem_alloc(base + C::TMEM, 256);
    if (tid == 0) {
        for (int i = 0; i < UNITS + 3; ++i) sk::mbar_init(bars + 8 * i, 1);
        sk::fence_barrier_init();
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::TMEM);
    const uint32_t my_lanes = tmem + (uint32_t(quad * 32) << 16);
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    Share sh = share_of(p, p.heads * p.RT, sm_share);
    // the products' shared-memory operands at their first k16 step
    const uint64_t q_op = operand(base + C::Q, 16, 1024, 2), v_op = operand(base + C::V, 16384, 1024, 2),
                   p_op = operand(base + C::P, 128, 2048, 0);
    uint32_t unit0 = 0, ph_s = 0, ph_o = 0;                  // units consumed; parities of the two products' barriers
    bool dead = false;
    // Copies of unit u (counted from the kernel's start), and a product beside which the units from u on are in flight.
    auto wait_unit = [&](uint32_t u) { sk::wait_ring<UNITS>(bars, u % UNITS, (u / UNITS) & 1, p.err, dead); };
    auto wait_product = [&](uint32_t bar, uint32_t parity, uint32_t u) {
        if (dead || sk::wait_limited(bar, parity)) return;
        dead = true;
        if (p.err) atomicOr(p.err, 1u);
        sk::drain_ring<UNITS>(bars, u % UNITS, (u / UNITS) & 1);
    };

    while (sh.t < sh.end && sh.b < p.B) {
        const int len = length_of(p, sh.b), nt = tiles_of(len);
        if (nt == 0) {
            ++sh.b;
            continue;
        }
        const int hr = sh.off / nt, t_lo = sh.off - hr * nt;
        const int t_hi = min(nt, t_lo + sh.end - sh.t);
        const int h = hr / p.RT, rt = hr - h * p.RT, b = sh.b, tiles = t_hi - t_lo;
        const int32_t *table = p.table + (long long)b * p.width;
        const int nrec = (len + 15) / 16, rec0 = t_lo * 8;

        // Unit u is the keys (even) or the values (odd) of tile u / 2, whose slot
        // is free again after the barrier that ends their decoding: every copy
        // has a tile's time to arrive.  Warp 1 issues them, a lane a record.
        auto lookup = [&](int tile) {
            const int rec = rec0 + 8 * tile + (lane & 7);
            return sk::kv4_record(table, min(rec, nrec - 1), p.recs, p.by_recs, p.pages, p.heads, h);
        };
        auto issue = [&](int u, uint32_t idx) {              // idx: the tile's records
            if (u >= 2 * tiles || p.stall || __any_sync(0xffffffffu, dead)) return;
            const bool load = lane < 8 && rec0 + 8 * (u >> 1) + lane < nrec;
            const uint32_t slot = (unit0 + uint32_t(u)) % UNITS, bar = bars + 8 * slot;
            const unsigned int mask = __ballot_sync(0xffffffffu, load);
            if (lane == 0) sk::mbar_arrive_expect_tx(bar, __popc(mask) * PART);
            __syncwarp();
            if (load)
                sk::bulk_load(base + C::RAW + slot * UNIT + lane * PART, p.cache + size_t(idx) * REC + (u & 1) * PART, PART, bar);
        };
        // rows: query, base, first unseen position
        uint2 qv[N / 8];                                     // on their way before the first copies
        const int qc = tid & 31;                             // eight bytes: j = c / 4, t = c % 4
#pragma unroll
        for (int x = 0; x < N / 8; ++x) {
            const int row = rt * N + 8 * x + (tid >> 5), m = row / p.G;
            qv[x] = make_uint2(0u, 0u);
            if (m < p.M)
                qv[x] = *reinterpret_cast<const uint2 *>(p.q + ((long long)b * p.M + m) * p.q_stride +
                                                        (long long)(h * p.G + row - m * p.G) * D + 32 * (qc & 3) + 4 * (qc >> 2));
        }
        uint32_t idx1 = 0, idx2 = 0, idx3 = 0;               // records of the next three tiles
        if (warp == 1) {
            const uint32_t idx0 = lookup(0);
            idx1 = lookup(1);
            idx2 = lookup(2);
            issue(0, idx0);
            issue(1, idx0);
            issue(2, idx1);
            if (UNITS == 4) issue(3, idx1);
        }
        static_assert(TT == 256, "eight rows at a time");
        const int q_at = (qc >> 4) * (N * 128) + warp * 128 + (((((8 * qc & 127) >> 4) ^ warp) << 4) | (8 * qc & 15));
#pragma unroll
        for (int x = 0; x < N / 8; ++x)
            *reinterpret_cast<uint2 *>(smem + C::Q + q_at + x * 1024) = qv[x];
        for (int n = tid; n < N; n += TT) {
            neg[n] = NO_BASE;
            lim[n] = len - (p.M - 1 - min((rt * N + n) / p.G, p.M - 1));
        }
        float l[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) l[i] = 0.f;
        fence_async_smem();
        __syncthreads();

        for (int i = 0; i < tiles; ++i) {
            const uint32_t uk = unit0 + 2 * i, uv = uk + 1;
            const uint32_t keys = base + C::RAW + (uk % UNITS) * UNIT, vals = base + C::RAW + (uv % UNITS) * UNIT;
            // ---- S = K . q^T
            wait_unit(uk);
            {
                const int r = 2 * quad + side;               // record, in this warp's lanes
                decode_keys(keys + r * PART, tmem + (uint32_t(16 * r) << 16), g, t);
                wait_st();
            }
            fence_before();
            __syncthreads();
            if (tid == 0) {
                fence_after();
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_tmem_a(tmem + C::S_COL, tmem + 8 * s, q_op + ((s >> 2) * (N * 128) + (s & 3) * 32) / 16,
                               shape(N, false, false), s > 0);
                commit(bar_s);
            }
            if (warp == 1) {
                idx3 = lookup(i + 3);
                issue(2 * i + UNITS, UNITS == 4 ? idx2 : idx1);
            }
            // ---- V, once the last tile's second product has read its own
            if (i > 0) {
                wait_product(bar_o, ph_o, uv);
                ph_o ^= 1;
                fence_after();
            }
            wait_unit(uv);
            decode_values(vals + warp * PART, base + C::V, warp * 16, lane);
            // ---- the weights, to the operand of the second product: eight rows
            // of a position in 16 bytes, positions 16 bytes apart
            wait_product(bar_s, ph_s, uv + 1);
            ph_s ^= 1;
            fence_after();
            const int at = quad * 32 + lane, pos = (t_lo + i) * TILE + at;
            const bool edge = (t_lo + i + 1) * TILE > len - (p.M - 1);
            // CH scores of this position, rows side * NH + c and on
            constexpr int CH = NH % 24 == 0 ? 24 : NH % 16 == 0 ? 16 : 8;
            auto scores = [&](int c, float (&s)[CH]) {
                ld_row<CH>(my_lanes + C::S_COL + side * NH + c, s);
                if (edge) {
                    // the tile's end: scores that their rows do not see
#pragma unroll
                    for (int e = 0; e < CH; ++e)
                        if (pos >= lim[side * NH + c + e]) s[e] = NEG_INF;
                }
            };
            auto store_weights = [&](int c, const float (&s)[CH]) {
#pragma unroll
                for (int x = 0; x < CH; x += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack_f16(s[x + 2 * e], s[x + 2 * e + 1]);
                    st_shared_v4(base + C::P + (side * NH + c + x) / 8 * 2048 + at * 16, w[0], w[1], w[2], w[3]);
                }
            };
            bool rise = i == 0;                              // whether a score has passed its row's base
            if (i > 0) {
#pragma unroll
                for (int c = 0; c < NH; c += CH) {
                    float s[CH];
                    scores(c, s);
#pragma unroll
                    for (int x = 0; x < CH; x += 8) {
                        float m[8];
                        row8(neg + side * NH + c + x, m);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float2 y = weights2(p, s[x + e], s[x + e + 1], m[e], m[e + 1]);
                            rise |= y.x > MOST_WEIGHT || y.y > MOST_WEIGHT;
                            l[c + x + e] += y.x;
                            l[c + x + e + 1] += y.y;
                            s[x + e] = y.x;
                            s[x + e + 1] = y.y;
                        }
                    }
                    store_weights(c, s);
                }
                fence_async_smem();
                fence_before();
            }
            const bool any = __syncthreads_or(rise);         // the ring's records are decoded, too
            if (warp == 1) {
                issue(2 * i + 1 + UNITS, idx2);
                idx1 = idx2;
                idx2 = idx3;
            }
            if (any) {
                // move the bases: each row's maximum over this warp's
                // positions first, eight rows at a time, halving what a lane
                // keeps (lanes 4 i .. 4 i + 3 end with row i)
                fence_after();
#pragma unroll
                for (int c = 0; c < NH; c += CH) {
                    float s[CH];
                    scores(c, s);
#pragma unroll
                    for (int x = 0; x < CH; x += 8) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = s[x + e];
#pragma unroll
                        for (int half = 4, o = 16; half >= 1; half >>= 1, o >>= 1) {
                            const bool up = lane & o;
#pragma unroll
                            for (int e = 0; e < half; ++e) {
                                const float give = up ? v[e] : v[e + half], keep = up ? v[e + half] : v[e];
                                v[e] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
                            }
                        }
                        v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
                        v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
                        if ((lane & 3) == 0) of_warp[quad * N + side * NH + c + x + (lane >> 2)] = v[0];
                    }
                }
                __syncthreads();
                for (int n = tid; n < N; n += TT) {
                    const float m = fmaxf(fmaxf(of_warp[n], of_warp[N + n]), fmaxf(of_warp[2 * N + n], of_warp[3 * N + n]));
                    const float had = neg[n], now = passes(p, m, had) ? fminf(had, neg_base(p, m)) : had;
                    fac[n] = rebase(p, now, had);
                    old[n] = had;
                    neg[n] = now;
                }
                __syncthreads();
                // The weights again.  A sum already holds this tile's weight
                // under the old base: it is taken out (the rounding that
                // leaves is of the size of the new weight's own) unless the
                // base rose so far that what was summed before vanishes
                // beside the position it rose to.
#pragma unroll
                for (int c = 0; c < NH; c += CH) {
                    float s[CH];
                    scores(c, s);
#pragma unroll
                    for (int e = 0; e < CH; ++e) {
                        const int n = side * NH + c + e;
                        const float f = fac[n], y = weight(p, s[e], neg[n]);
                        const float both = (l[c + e] - weight(p, s[e], old[n])) * f + y;
                        l[c + e] = f < 0x1p-64f ? y : f == 1.f && i > 0 ? l[c + e] : both;
                        s[e] = y;
                    }
                    store_weights(c, s);
                }
                if (i > 0) {
#pragma unroll 1
                    for (int c = 0; c < NH; c += 8) {
                        float o[8];
                        ld8(my_lanes + C::O_COL + side * NH + c, o);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] *= fac[side * NH + c + e];
                        st8(my_lanes + C::O_COL + side * NH + c, o);
                    }
                    wait_st();
                }
                fence_async_smem();
                fence_before();
                __syncthreads();
            }
            if (tid == 0) {
                fence_after();
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_smem_a(tmem + C::O_COL, v_op + s * 2048 / 16, p_op + s * 256 / 16, shape(N, true, true),
                               i > 0 || s > 0);
                commit(bar_o);
            }
        }
        unit0 += 2 * tiles;

        // ---- the rows' sums over the positions, then the outputs
        // (a warp's 32 positions, eight rows at a time, halving what a lane
        // keeps: lanes 4 i .. 4 i + 3 end with row i)
#pragma unroll
        for (int c = 0; c < NH; c += 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = l[c + e];
#pragma unroll
            for (int half = 4, o = 16; half >= 1; half >>= 1, o >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int e = 0; e < half; ++e) {
                    const float give = up ? v[e] : v[e + half], keep = up ? v[e + half] : v[e];
                    v[e] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
            if ((lane & 3) == 0) of_warp[quad * N + side * NH + c + (lane >> 2)] = v[0];
        }
        wait_product(bar_o, ph_o, unit0);
        ph_o ^= 1;
        fence_after();
        __syncthreads();
        const bool whole = t_lo == 0 && t_hi == nt;
        const int rows = min(N, p.M * p.G - rt * N), d = quad * 32 + lane;
        const size_t slot = size_t(blockIdx.x) * 2 + (t_lo == 0 ? 1 : 0);
        // row n's sum, and what its output is multiplied by
        for (int n = tid; n < rows; n += TT) {
            const float sum = (of_warp[n] + of_warp[N + n]) + (of_warp[2 * N + n] + of_warp[3 * N + n]);
            fac[n] = sum == 0.f ? 0.f : p.vg / sum;
            if (whole) {
                const int row = rt * N + n, m = row / p.G;
                const long long to = ((long long)b * p.M + m) * (p.heads * p.G) + h * p.G + row - m * p.G;
                lim[n] = int(to - ((long long)b * p.M * p.heads * p.G));       // the row within its sequence
                write_stats(p, to, -neg[n], sum);
            } else {
                *reinterpret_cast<float2 *>(p.part_ml + (slot * N + n) * 2) = make_float2(-neg[n], sum);
            }
        }
        __syncthreads();
        __half *const out = p.out + (long long)b * p.M * p.heads * p.G * D + d;
        float *const part = p.part_o + slot * N * D + d;
#pragma unroll 1
        for (int c = 0; c < NH; c += 8) {
            float o[8];
            ld8(my_lanes + C::O_COL + side * NH + c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int n = side * NH + c + e;
                if (n >= rows) break;
                if (whole) out[(long long)lim[n] * D] = __float2half_rn(o[e] * fac[n]);
                else part[n * D] = o[e];
            }
        }
        if (tid == 0 && t_lo == 0) {
            const int c1 = cta_of(sh, sh.t + nt - 1);     // of the segment's last tile
            p.seg[(b * p.heads + h) * p.RT + rt] = make_int2(int(blockIdx.x), whole ? 0 : c1 - int(blockIdx.x) + 1);
        }
        fence_before();
        __syncthreads();
        fence_after();
        sh.t += t_hi - t_lo;
        sh.off += t_hi - t_lo;
        if (sh.off == nt * p.heads * p.RT) {
            ++sh.b;
            sh.off = 0;
        }
    }
    if (__syncthreads_or(dead)) {
        // a product may still be under way: its end, too, is waited for
        if (tid == 0) commit(bar_end);
        sk::wait_limited(bar_end, 0);
        fence_after();
        __syncthreads();
    }
    if (warp == 0) tmem_free(tmem, 256);
}

template <int N>
cudaError_t launch(AttnParams &p, cudaStream_t s) {
    const cudaError_t e = sk::prepare_kernel<kv4_attention_tc_kernel<N>>(Tc<N>::SMEM);
    if (e != cudaSuccess) return e;
    return sk::launch_pdl(kv4_attention_tc_kernel<N>, dim3(p.ctas), dim3(TT), Tc<N>::SMEM, s, p);
}

}  // namespace

namespace sk {
namespace attn {

int tc_rows(int rows, int *tiles) {
    *tiles = (rows + TC_MOST - 1) / TC_MOST;
    const int each = (rows + *tiles - 1) / *tiles;
    return (each + 15) / 16 * 16;
}

cudaError_t launch_tc(AttnParams &p, int n, cudaStream_t s) {
    switch (n) {
        case 32: return launch<32>(p, s);
        case 48: return launch<48>(p, s);
        case 64: return launch<64>(p, s);
        case 80: return launch<80>(p, s);
        default: return launch<96>(p, s);
    }
}

}  // namespace attn
}  // namespace sk
