// kv4_chunk.cu -- attention of chunks of new tokens, any number per sequence, over
// the paged 4-bit cache (kv4.cuh), on the fifth-generation tensor cores.
//
// Query row i of sequence b (n rows, the last of len positions) and query head x,
// over the positions j <= at = len - n + i with j > at - window or j < sinks:
//     z_j = scale * q . k_j,   p_j = exp(z_j - max z),   out = sum p_j v_j / sum p_j
//
// The rows of a kv head's G query heads are one list (row i, head g: i G + g), cut
// into tiles of 128, a row a TMEM lane. For 64 positions at a time
//     S (128 x 64, TMEM)  = Q (128 x D, TMEM; D = 128: shared memory) . K^T      K: decoded into shared memory
//     O (128 x D, TMEM)  += P (128 x 64, TMEM) . V       V: the same; P over S's own columns
// so that a softmax thread owns a row: its maximum, base and sum need no other
// thread, and shared memory carries only the decoded keys and values. Roles: four
// warps of softmax per tile, warps that decode keys and warps that decode values, one
// thread that issues the products, one warp that lists the work. At head size 256 a
// pair of CTAs takes two tiles and decodes each block once for both: decoding alone
// bounds a single CTA there (2048 rows over 61003 positions, 24 over 2 heads: 2346 us
// against 1684, when the pairs were new).
//
// At head size 256 bound by the products: that case 1699 to 1765 us over several runs of
// calls, 1710 to 1777 TFLOP/s. At 128 and 64 by the softmax's chain from a
// product to the next (1900 and 1520 clocks a block of two tiles, whose products take
// 1280 and 512): 2048 rows over 16384 positions, 48 over 4 heads of 128, 590 us, 1310
// TFLOP/s; issue slots, ALU and XU are below half of their rates. 128 registers a thread,
// of which 44, 72 and 60 bytes are spilled at head sizes 256, 128 and 64 (92 bytes loaded
// again at most). Twenty warps at 128, with registers moved to the softmax's, spilled far
// more and took longer (644 -> 763). Calls of a row over 24 to 4096 positions: 6 to 18 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstddef>
#include <cstdint>

#include "../../include/skinny.h"
#include "internal.h"
#include "kv4_attention.cuh"
#include "launch_util.cuh"
#include "tcgen05.cuh"

namespace {

using namespace sk::attn;
using sk::ex2;
namespace t5 = sk::t5;

constexpr int KB = 64;                 // positions per block
constexpr int MOST_SEQS = CHUNK_SEQS;
// What a tile costs beside its blocks, in blocks (4099 rows over themselves, heads of
// 256: 4 207 us, 8 169, 12 173; 8195 rows in windows of 1024, heads of 128: 284, 255, 259).
constexpr int SETUP = 8;
constexpr int WHOLE_BLOCKS = 12;       // tables of no more blocks are not worth a second kernel where each tile has a CTA
constexpr int MIN_SHARE = 40;          // least cost a CTA takes, above that of one block: no part of a tile is empty

// T tiles of 128 rows share what a CTA decodes; NB buffers of S per tile; HW warps
// decode keys and as many values; ST stages of each. PAIR: two CTAs, each with a tile
// of its own, share what is decoded, each decoding half the keys of a block and half
// the components of its values; the first one issues the products of both.
template <int D>
struct Cc {
    static constexpr bool PAIR = D == 256;
    static constexpr int T = D == 256 ? 1 : 2;
    static constexpr int NB = 2;
    // The query rows lie in TMEM where there is room, else in shared memory (whose rate the scores then also need: a
    // product of 64 columns takes 48 clocks, not 32).
    static constexpr bool QS = D == 128;
    static constexpr int Q_TILE = 128 * D * 2, Q_SLAB = 128 * 128;
    static constexpr int HW = D == 256 ? 4 : 2, DW = 2 * HW;
    static constexpr int ST = PAIR ? 6 : 4;
    static constexpr int SW = 4 * T, WARPS_ALL = SW + DW + 2, CT_ALL = WARPS_ALL * 32;
    static constexpr int ROWS = PAIR ? 256 : 128 * T;                  // of a tile of the work
    static constexpr int KEYS = PAIR ? KB / 2 : KB, COMPS = PAIR ? D / 2 : D;   // a CTA's, of a block
    static constexpr int STAGE = KEYS * D * 2;                         // bytes, of keys or of values
    static constexpr int K_SLAB = KEYS * 128, V_SLAB = KB * 128;       // 64 components of it
    static constexpr int ROUNDS = STAGE / 64 / (32 * HW);              // 16-byte pieces of codes per thread
    // bytes from a thread's piece to its next round's
    static constexpr int K_ROUND = (D == 64 ? 32 : 16) * 128, V_ROUND = (D == 64 || PAIR ? 32 : 16) * 128;
    static constexpr int K = 0, V = ST * STAGE, Q = 2 * ST * STAGE, BARS = Q + (QS ? T * Q_TILE : 0);
    // barriers: keys full, empty, values full, empty (ST each); S full and P ready (T NB each); query rows ready, a second
    // product done, a piece's last one done (T each); end
    // and of the list of pieces, full and empty (LIST each)
    static constexpr int LIST = 4;
    static constexpr int NBARS = 4 * ST + 2 * T * NB + 3 * T + 1 + 2 * LIST;
    // (and behind the TMEM's address whether a wait has run out)
    static constexpr int SCAN = BARS + 8 * NBARS, TMEM = SCAN + 16 * (WARPS_ALL + 1), GONE = TMEM + 8, START = TMEM + 16, PIECES = START + 16;
    static constexpr int OUT = (PIECES + LIST * 64 + 127) / 128 * 128;         // 128 bytes of a row, per thread of the softmax
    static constexpr int BYTES = 1024 + OUT + SW * 32 * 128;
    static constexpr size_t SMEM = BYTES > 120 * 1024 ? BYTES : 120 * 1024;      // one CTA per SM: all of the TMEM
    static constexpr int O_COL = 0, Q_COL = T * D, S_COL = QS ? Q_COL : Q_COL + T * D / 2;
    static_assert(S_COL + T * NB * KB <= 512, "TMEM");
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static constexpr int MOST_SEQS = 2 * ST * STAGE / 4 - 1;            // their list lies where the stages will
};
// The CTAs that share a piece of work count as one.
template <int D>
__device__ __forceinline__ int worker() {
    return int(blockIdx.x) / (Cc<D>::PAIR ? 2 : 1);
}

// Each row's weights are 2^(c s - t) with c = scale * key scale * log2 e and t the
// row's base, one number for all that is summed under it: one fma gives the exponent,
// rounded once, at the size of the difference, so that equal scores get equal weights in
// any block, and weights near the maximum are right whatever the scores' size. The base is
// t0, a float P_SHIFT below a maximum that the row had earlier, and is moved only when an
// exponent passes P_SHIFT + SLACK. From FAR on floats lie too far apart for that: there
// the base is t0 + t1, t0 the float nearest to c times the maximum and t1 what that leaves,
// taken off in a second step (by a loop of its own: as a branch of the common one, never
// taken, that step cost 3 to 7 %).
// The weights go to the second product in FP16, between 2^-32 and 2^15 (that of the
// maximum by which the base was set is a power of two but for the exponent's rounding: the
// largest weight of most rows is not rounded), their sum is taken unrounded.
constexpr float FAR = 0x1p24f;
__device__ __forceinline__ void write_lse(const AttnParams &p, long long row, float t0, float t1, float l) {
    if (p.lse) p.lse[row] = l == 0.f ? NEG_INF : (t0 + (t1 + __log2f(l))) * LN2;
}

// (part_ml: per row of a partial slot t0, t1 and the sum)
struct ChunkParams : AttnParams {
    const int32_t *starts;             // null: M rows of every sequence
    int rows;                          // in all
    sk::Div by_g;
    int whole;                         // every tile is one CTA's (and costs the same)
    int4 *join;                        // of a tile in parts: first CTA, parts (0: whole), and which: head, sequence and tile ...
    int by_tile;                       // ... at its number, or else at its first CTA's
    int *tiles;                        // tiles of a head
};
struct Join {
    static __device__ __forceinline__ int4 of(int first, int parts, int h, int b, int t) {
        return make_int4(first, parts | h << 16, b, t);
    }
};

// Rows of sequence b: [first, first + n), and its positions.
struct Seq {
    int first, n, len;
    __device__ __forceinline__ Seq() {}
    __device__ __forceinline__ Seq(const ChunkParams &p, int b) {
        first = p.starts ? min(max(p.starts[b], 0), p.rows) : b * p.M;
        n = p.starts ? min(max(p.starts[b + 1], first), p.rows) - first : p.M;
        len = min(max(p.lens[b], 0), p.cap);
    }
};
template <int D>
__device__ __forceinline__ int tiles_in(const ChunkParams &p, const Seq &s) {
    return int(((long long)s.n * p.G + Cc<D>::ROWS - 1) / Cc<D>::ROWS);
}

// A tile of a sequence's rows: what it looks at (positions without the records
// between sinks and windows, as in Seen) and what it costs.
template <int D>
struct Tile {
    int idx0, count;                   // first of the list, rows
    int lim0, lim1;                    // first unseen position (numbered without the gap) of its first and last row
    int gap, skip, blocks, cost, per;
    __device__ __forceinline__ Tile() {}
    __device__ __forceinline__ Tile(const ChunkParams &p, const Seq &s, int t) {
        using C = Cc<D>;
        idx0 = t * C::ROWS;
        count = min(C::ROWS, s.n * p.G - idx0);
        const int at0 = s.len - s.n + 1;
        lim0 = at0 + sk::quotient(idx0, p.by_g);
        lim1 = at0 + sk::quotient(idx0 + count - 1, p.by_g);
        gap = skip = 0;
        if (p.window) {
            gap = (min(p.sinks, max(lim1, 0)) + sk::KV4_REC - 1) / sk::KV4_REC;
            skip = max(0, max(0, lim0 - p.window) / sk::KV4_REC - gap);
        }
        lim0 -= skip * sk::KV4_REC;
        lim1 -= skip * sk::KV4_REC;
        blocks = (max(lim1, 0) + KB - 1) / KB;
        // (a block of one tile of 128 rows takes nearly as long as of two: 1730 clocks of 1900, at head size 64 1230 of 1520)
        per = C::T == 1 || count > 128 ? 10 : D == 64 ? 8 : 9;
        cost = p.whole ? 1 : (blocks + SETUP) * per;
    }
    __device__ __forceinline__ int block_at(int x) const {
        return x == cost ? blocks : min(max(x / per - SETUP, 0), blocks);
    }
};

// A piece of work: blocks [k0, k1) of a tile of sequence b and kv head h, one at least; k1 < 0: the
// end. One warp lists a CTA's pieces, the others read them from shared memory.
struct Piece {
    int k0, k1, blocks, h, b;
    int row0, idx0, count;             // the sequence's first row; of its list of rows, the tile's first and how many
    int lim0, lim1, gap, skip;         // as in Tile
    int pad[4];
};
static_assert(sizeof(Piece) == 64, "read in 16-byte words");

// The pieces of a CTA, in order. All (head, sequence, tile) cost a total that
// P CTAs take in equal parts, whatever the lengths; a tile that two of them share
// is joined later.
template <int D>
struct Pieces {
    long long left;                    // of this CTA's share
    int h, b, t, x;                    // where it stands: x into the cost of the tile
    int number;                        // the tile's among those of a head
    Seq seq;                           // of sequence `held`
    int held;
    __device__ __forceinline__ bool next(const ChunkParams &p, Piece &w, int &tile_t, int &tile_number, int &cost) {
        while (left > 0 && h < p.heads) {
            if (b >= p.B) {
                b = 0;
                t = 0;
                number = 0;
                ++h;
                continue;
            }
            if (held != b) {
                seq = Seq(p, b);
                held = b;
            }
            if (t >= tiles_in<D>(p, seq)) {
                ++b;
                t = 0;
                continue;
            }
            const Tile<D> tile(p, seq, t);
            const int x1 = int(min((long long)tile.cost, x + left));
            w.k0 = tile.block_at(x);
            w.k1 = tile.block_at(x1);
            w.blocks = tile.blocks;
            w.h = h;
            w.b = b;
            w.row0 = seq.first;
            w.idx0 = tile.idx0;
            w.count = tile.count;
            w.lim0 = tile.lim0;
            w.lim1 = tile.lim1;
            w.gap = tile.gap;
            w.skip = tile.skip;
            tile_t = t;
            tile_number = number;
            cost = tile.cost;
            const bool last = x1 == tile.cost;
            left -= x1 - x;
            x = last ? 0 : x1;
            t += last;
            number += last;
            if (w.k1 > w.k0 || (last && tile.blocks == 0)) return true;
        }
        return false;
    }
};

// a / b, where both are small by the shorter division.
__device__ __forceinline__ long long divided(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (unsigned int)a / (unsigned int)b;
    return a / b;
}
struct Split {
    long long total;                   // over all heads
    int parts;
};
__device__ __forceinline__ long long bound_of(const Split &s, int c) { return divided(s.total * c, s.parts); }
__device__ __forceinline__ int owner_of(const Split &s, long long u) { return int(divided((u + 1) * s.parts - 1, s.total)); }

// Where this CTA's share begins. With up to FEW sequences one warp comes here, else
// every thread of the CTA; `list` holds p.B + 1 numbers, `scan` one per warp.
constexpr int FEW = 32;
template <int D>
__device__ Split find_share(const ChunkParams &p, Pieces<D> &w, int *list, long long *scan, int *start, int &tiles_of_head) {
    using C = Cc<D>;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, me = worker<D>();
    w.left = 0;
    w.h = w.b = w.t = w.x = w.number = 0;
    w.held = -1;
    // (no part of a tile in parts is empty: MIN_SHARE)
    auto split = [&](long long per_head) {
        Split sh;
        sh.total = per_head * p.heads;
        sh.parts = int(max(1LL, min(p.whole ? sh.total : divided(sh.total, MIN_SHARE), (long long)p.ctas)));
        return sh;
    };
    if (p.B <= FEW) {
        // a lane a sequence, then a lane a tile
        Seq s;
        s.first = s.n = s.len = 0;
        if (lane < p.B) s = Seq(p, lane);
        const int n = tiles_in<D>(p, s), upto = inclusive_scan(n, lane), tiles = __shfl_sync(0xffffffffu, upto, 31);
        tiles_of_head = tiles;
        {
            auto at = [&](int i, int &b, int &t, Seq &of) {        // tile i: all lanes come here
                b = 0;
                int before = 0;
                for (int k = 0; k < p.B; ++k) {
                    const int u = __shfl_sync(0xffffffffu, upto, k);
                    if (u <= i) {
                        b = k + 1;
                        before = u;
                    }
                }
                t = i - before;
                const int from = min(b, 31);
                of.first = __shfl_sync(0xffffffffu, s.first, from);
                of.n = __shfl_sync(0xffffffffu, s.n, from);
                of.len = __shfl_sync(0xffffffffu, s.len, from);
            };
            long long per_head = 0;
            int b, t;
            Seq of;
            for (int i0 = 0; i0 < tiles; i0 += 32) {
                at(min(i0 + lane, tiles - 1), b, t, of);
                long long cost = i0 + lane < tiles ? Tile<D>(p, of, t).cost : 0;      // (32 of them may pass 31 bits)
#pragma unroll
                for (int o = 16; o; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
                per_head += cost;
            }
            const Split sh = split(per_head);
            if (me >= sh.parts || sh.total == 0) return sh;
            const long long u0 = bound_of(sh, me);
            w.left = bound_of(sh, me + 1) - u0;
            w.h = int(divided(u0, per_head));
            long long off = u0 - w.h * per_head;
            for (int i0 = 0; i0 < tiles; i0 += 32) {
                at(min(i0 + lane, tiles - 1), b, t, of);
                const long long cost = i0 + lane < tiles ? Tile<D>(p, of, t).cost : 0, x = inclusive_scan(cost, lane);
                const unsigned int past = __ballot_sync(0xffffffffu, x > off);
                if (past) {
                    const int l = __ffs(past) - 1;
                    w.b = w.held = __shfl_sync(0xffffffffu, b, l);
                    w.t = __shfl_sync(0xffffffffu, t, l);
                    w.x = int(off - __shfl_sync(0xffffffffu, x - cost, l));
                    w.number = i0 + l;
                    w.seq.first = __shfl_sync(0xffffffffu, of.first, l);
                    w.seq.n = __shfl_sync(0xffffffffu, of.n, l);
                    w.seq.len = __shfl_sync(0xffffffffu, of.len, l);
                    break;
                }
                off -= __shfl_sync(0xffffffffu, x, 31);
            }
            return sh;
        }
    }
    auto scanned = [&](long long mine, long long &total) {         // exclusive, over the CTA
        long long v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        __syncthreads();
        if (lane == 31) scan[wid] = v;
        __syncthreads();
        long long w = lane < C::WARPS_ALL ? scan[lane] : 0;
        const long long own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        total = __shfl_sync(0xffffffffu, w, 31);
        return __shfl_sync(0xffffffffu, w - own, wid) + v - mine;
    };
    // tiles before each sequence
    const int each_b = (p.B + C::CT_ALL - 1) / C::CT_ALL, b_lo = min(p.B, tid * each_b), b_hi = min(p.B, b_lo + each_b);
    long long mine = 0, tiles;
    for (int b = b_lo; b < b_hi; ++b) mine += tiles_in<D>(p, Seq(p, b));
    constexpr long long MOST_TILES = 1 << 30;              // (more only where starts descends)
    long long at = scanned(mine, tiles);
    tiles = min(tiles, MOST_TILES);
    for (int b = b_lo; b < b_hi; ++b) {
        list[b] = int(min(at, MOST_TILES));
        at += tiles_in<D>(p, Seq(p, b));
    }
    if (tid == 0) {
        list[p.B] = int(tiles);
        start[0] = p.B;
        start[1] = start[2] = start[3] = 0;
    }
    tiles_of_head = int(tiles);
    __syncthreads();
    // this thread's tiles: [lo, hi)
    const int each = int((tiles + C::CT_ALL - 1) / C::CT_ALL), lo = int(min(tiles, (long long)tid * each)),
              hi = int(min(tiles, (long long)lo + each));
    int b0 = 0;
    if (lo < hi) {                                                 // the last sequence that begins at or before lo
        int l = 0, r = p.B - 1;
        while (l < r) {
            const int m = (l + r + 1) / 2;
            if (list[m] <= lo) l = m;
            else r = m - 1;
        }
        b0 = l;
    }
    auto walk = [&](auto &&visit) {
        int b = b0;
        for (int i = lo; i < hi && b < p.B; ++b) {
            const Seq s(p, b);
            const int n = tiles_in<D>(p, s);
            for (int t = i - list[b]; t < n && i < hi; ++t, ++i)
                if (!visit(b, t, Tile<D>(p, s, t).cost)) return;
        }
    };
    mine = 0;
    walk([&](int, int, int cost) {
        mine += cost;
        return true;
    });
    long long per_head;
    const long long before = scanned(mine, per_head);
    const Split sh = split(per_head);
    if (me < sh.parts && sh.total > 0) {
        const long long u0 = bound_of(sh, me);
        w.left = bound_of(sh, me + 1) - u0;
        w.h = int(divided(u0, per_head));
        long long off = u0 - w.h * per_head;
        if (off >= before && off < before + mine) {
            off -= before;
            walk([&](int b, int t, int cost) {
                if (off < cost) {
                    start[0] = b;
                    start[1] = t;
                    start[2] = int(off);
                    start[3] = list[b] + t;
                    return false;
                }
                off -= cost;
                return true;
            });
        }
    }
    __syncthreads();
    w.b = start[0];
    w.t = start[1];
    w.x = start[2];
    w.number = start[3];
    __syncthreads();                                               // the list's place is free
    return sh;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&d)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(d[0]), "r"(d[1]), "r"(d[2]), "r"(d[3]) : "memory");
}
// Two floats in one register pair, and the operations on both.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 apart(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint16_t ld_u16(const uint8_t *p) { return *reinterpret_cast<const uint16_t *>(p); }

// Eight codes, scaled, to the 16 bytes at `addr` (exact in FP16).
__device__ __forceinline__ void put8(uint32_t addr, uint32_t codes, uint32_t scale) {
    uint32_t d[4];
    sk::e2m1x8_to_f16x2x4(codes, d);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = sk::hmul2(d[e], scale);
    st_shared_v4(addr, d);
}

// What a decoding thread has fetched of a block's keys or values: 16 bytes of codes
// and the scales of their two blocks or positions, ROUNDS times.
template <int D>
struct Raw {
    uint4 c[Cc<D>::ROUNDS];
    uint16_t s[Cc<D>::ROUNDS];
};
// Keys: a warp takes eight positions x four 16-byte pieces (D = 64: sixteen x two)
// at a time, lanes of eight the positions: their stores meet all banks. Decode warp
// w, round r: position and piece.
template <int D>
__device__ __forceinline__ void key_place(int w, int r, int lane, int &row, int &piece) {
    const int u = r * Cc<D>::HW + w;
    if constexpr (D == 256) {
        row = (u >> 1) * 8 + (lane & 7);
        piece = (u & 1) * 4 + (lane >> 3);
    } else if constexpr (D == 128) {
        row = u * 8 + (lane & 7);
        piece = lane >> 3;
    } else {
        row = u * 16 + (lane & 7) + 8 * (lane >> 4);
        piece = (lane >> 3) & 1;
    }
}
// Values: a 16-byte piece is a pair of positions of a block of 16 components:
// half record (eight positions), block (of this CTA's), pair.
template <int D>
__device__ __forceinline__ void value_place(int w, int r, int lane, int &half, int &blk, int &pair) {
    const int u = r * Cc<D>::HW + w;
    pair = lane & 3;
    if constexpr (Cc<D>::COMPS == 128) {
        half = u;
        blk = lane >> 2;
    } else {
        static_assert(Cc<D>::COMPS == 64 || Cc<D>::COMPS == 128, "components of a CTA");
        half = u * 2 + (lane >> 4);
        blk = (lane >> 2) & 3;
    }
}
// The record of a block that decode warp w reads in round r, in the CTA `rank` of a pair.
template <int D>
__device__ __forceinline__ int record_of(bool value, int w, int r, int rank) {
    const int u = r * Cc<D>::HW + w;
    if (value) return Cc<D>::COMPS == 128 ? u >> 1 : u;
    return D == 256 ? (Cc<D>::KEYS / sk::KV4_REC) * rank + (u >> 2) : D == 128 ? u >> 1 : u;
}

// Where in a record a thread's codes and scales lie, the same in every round.
template <int D>
__device__ __forceinline__ void source_offsets(bool value, int w, int lane, int rank, uint32_t &codes, uint32_t &scales) {
    if (value) {
        int half, blk, pair;
        value_place<D>(w, 0, lane, half, blk, pair);
        blk += rank * (Cc<D>::COMPS / 16);
        codes = 9 * D + (half & 1) * 4 * D + blk * 64 + pair * 16;
        scales = 17 * D + blk * 16 + (half & 1) * 8 + pair * 2;
    } else {
        int row, piece;
        key_place<D>(w, 0, lane, row, piece);
        codes = (row & 15) * (D / 2) + piece * 16;
        scales = 8 * D + (row & 15) * (D / 16) + piece * 2;
    }
}
// Where a thread's four 16-byte pieces go in a stage of keys or of values: 64
// components (128 bytes) of a position a row, the rows of 64 components a slab, pieces
// swizzled within eight rows.
template <int D>
__device__ __forceinline__ void key_offsets(int w, int lane, uint32_t (&to)[4]) {
    int row, piece;
    key_place<D>(w, 0, lane, row, piece);
    const uint32_t at = (piece >> 1) * Cc<D>::K_SLAB + row * 128, x = uint32_t(row & 7), c = (piece & 1) * 4;
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) to[e] = at + (((c + e) ^ x) << 4);
}
// (of values: first and second half of the block at the pair's first position, then
// at its second. Lanes of an odd block have the halves exchanged, so that eight
// lanes' stores meet all banks: `odd`.)
template <int D>
__device__ __forceinline__ void value_offsets(int w, int lane, uint32_t (&to)[4], bool &odd) {
    int half, blk, pair;
    value_place<D>(w, 0, lane, half, blk, pair);
    odd = blk & 1;
    const uint32_t at = (blk >> 2) * Cc<D>::V_SLAB + half * 1024, c = (blk & 3) * 2;
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t x = uint32_t(2 * pair) + (e >> 1), z = (e & 1) ^ uint32_t(odd);
        to[e] = at + x * 128 + (((c + z) ^ x) << 4);
    }
}
template <int D>
__device__ __forceinline__ void decode_keys(uint32_t stage, const uint32_t (&to)[4], const Raw<D> &raw) {
    const uint32_t at[4] = {stage + to[0], stage + to[1], stage + to[2], stage + to[3]};
#pragma unroll
    for (int r = 0; r < Cc<D>::ROUNDS; ++r) {
        const uint32_t s = scale_pair(raw.s[r]), lo = sk::bcast_lo(s), hi = sk::bcast_hi(s);
        put8(at[0] + r * Cc<D>::K_ROUND, raw.c[r].x, lo);
        put8(at[1] + r * Cc<D>::K_ROUND, raw.c[r].y, lo);
        put8(at[2] + r * Cc<D>::K_ROUND, raw.c[r].z, hi);
        put8(at[3] + r * Cc<D>::K_ROUND, raw.c[r].w, hi);
    }
}
template <int D>
__device__ __forceinline__ void decode_values(uint32_t stage, const uint32_t (&to)[4], bool odd, const Raw<D> &raw) {
    const uint32_t at[4] = {stage + to[0], stage + to[1], stage + to[2], stage + to[3]};
#pragma unroll
    for (int r = 0; r < Cc<D>::ROUNDS; ++r) {
        const uint32_t s = scale_pair(raw.s[r]), lo = sk::bcast_lo(s), hi = sk::bcast_hi(s);
        const uint4 c = raw.c[r];
        put8(at[0] + r * Cc<D>::V_ROUND, odd ? c.y : c.x, lo);
        put8(at[1] + r * Cc<D>::V_ROUND, odd ? c.x : c.y, lo);
        put8(at[2] + r * Cc<D>::V_ROUND, odd ? c.w : c.z, hi);
        put8(at[3] + r * Cc<D>::V_ROUND, odd ? c.z : c.w, hi);
    }
}

// The results of this CTA's rows of a tile that sees nothing, by one warp.
template <int D>
__device__ __forceinline__ void nothing_seen(const ChunkParams &p, const Piece &w, int lo, int lane) {
    constexpr int LANES = D / 8;                             // of a row, 16 bytes each
    const int hi = min(w.count, lo + 128 * Cc<D>::T);
    for (int r = lo + lane / LANES; r < hi; r += 32 / LANES) {
        const int idx = w.idx0 + r, i = sk::quotient(idx, p.by_g);
        const long long to = (long long)(w.row0 + i) * (p.heads * p.G) + w.h * p.G + idx - i * p.G;
        reinterpret_cast<uint4 *>(p.out + to * D)[lane % LANES] = make_uint4(0u, 0u, 0u, 0u);
        if (lane % LANES == 0) write_lse(p, to, 0.f, 0.f, 0.f);
    }
}

template <int D>
__global__ void __launch_bounds__(Cc<D>::CT_ALL, 1) kv4_chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cc<D>;
    constexpr int T = C::T, NB = C::NB, ST = C::ST, CTAS = C::PAIR ? 2 : 1;
    extern __shared__ unsigned char dyn[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (sk::smem_u32(dyn) + 1023u) & ~1023u;
    unsigned char *const smem = dyn + (base - sk::smem_u32(dyn));
    const uint32_t bars = base + C::BARS;
    const uint32_t k_full = bars, k_empty = k_full + 8 * ST, v_full = k_empty + 8 * ST, v_empty = v_full + 8 * ST,
                   s_full = v_empty + 8 * ST, p_ready = s_full + 8 * T * NB, q_ready = p_ready + 8 * T * NB,
                   o_done = q_ready + 8 * T, o_end = o_done + 8 * T, end = o_end + 8 * T,
                   l_full = end + 8, l_empty = l_full + 8 * C::LIST;

    const int rank = C::PAIR ? int(sk::cluster_rank()) : 0;
    if (warp == 0) t5::alloc<C::PAIR>(base + C::TMEM, 512);
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            sk::mbar_init(k_full + 8 * i, C::HW * CTAS);
            sk::mbar_init(v_full + 8 * i, C::HW * CTAS);
            sk::mbar_init(k_empty + 8 * i, 1);
            sk::mbar_init(v_empty + 8 * i, 1);
        }
        for (int i = 0; i < T * NB; ++i) {
            sk::mbar_init(s_full + 8 * i, 1);
            sk::mbar_init(p_ready + 8 * i, 4 * CTAS);
        }
        for (int i = 0; i < T; ++i) {
            sk::mbar_init(q_ready + 8 * i, 4 * CTAS);
            sk::mbar_init(o_done + 8 * i, 1);
            sk::mbar_init(o_end + 8 * i, 1);
        }
        sk::mbar_init(end, 1);
        for (int i = 0; i < C::LIST; ++i) {
            sk::mbar_init(l_full + 8 * i, 1);
            sk::mbar_init(l_empty + 8 * i, C::SW + C::DW + 1);
        }
        sk::fence_barrier_init();
    }
    // (every place of the list an end: a thread that gave up waiting finds nothing else)
    if (tid < C::LIST * 16) reinterpret_cast<int *>(smem + C::PIECES)[tid] = tid % 16 == 1 ? -1 : 0;
    static_assert(offsetof(Piece, k1) == 4, "the second word of a piece");
    if (tid == 0) *reinterpret_cast<volatile uint32_t *>(smem + C::GONE) = 0u;
    __syncwarp();
    t5::fence_before();
    if constexpr (C::PAIR) sk::cluster_sync();
    else __syncthreads();
    t5::fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::TMEM);
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    Pieces<D> work;
    Split share;
    int tiles;
    const bool lister = warp == C::WARPS_ALL - 1;
    if (p.B > FEW || lister)
        share = find_share<D>(p, work, reinterpret_cast<int *>(smem), reinterpret_cast<long long *>(smem + C::SCAN),
                              reinterpret_cast<int *>(smem + C::START), tiles);
    bool dead = false;
    // Waits for a barrier's phase of this parity, a second at most; after one that
    // ran out the thread waits no more.
    auto give_up = [&] {
        dead = true;
        sk::st_shared_volatile(base + C::GONE, 1u);
        if constexpr (C::PAIR) sk::st_peer_u32(sk::peer(base + C::GONE, rank ^ 1), 1u);
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!dead && !t5::wait_spin(bar, parity)) give_up();
    };
    // The warps that do nothing but follow the list wait for whole pieces: a minute at most, and no longer than until
    // another wait of the CTA (or the pair) has run out. (Read in every wait, that word cost up to 4 %.)
    auto wait_long = [&](uint32_t bar, uint32_t parity) {
        if (!dead && !t5::wait_spin(bar, parity, 60, base + C::GONE)) give_up();
    };
    // This warp's or thread's way through the list: the place of its next piece.
    const Piece *const list = reinterpret_cast<const Piece *>(smem + C::PIECES);
    uint32_t at = 0, lap = 0;
    auto here = [&] { wait(l_full + 8 * at, lap); };
    auto leave = [&](bool one) {       // by one thread, when no other of those it stands for reads the piece any more
        if (one) sk::mbar_arrive(l_empty + 8 * at);
        if (++at == C::LIST) {
            at = 0;
            lap ^= 1u;
        }
    };
    // Arrive at a barrier that the products wait at: the first CTA's.
    auto arrive = [&](uint32_t bar) {
        if constexpr (C::PAIR) t5::arrive_cluster(sk::peer(bar, 0));
        else sk::mbar_arrive(bar);
    };

    if (warp < C::SW) {
        // ------------------------------------------------------- softmax
        const int t = warp >> 2, row = tid & 127;
        const int first = (C::PAIR ? rank : t) * 128;        // of this CTA's or warpgroup's rows in the tile
        const uint32_t mine = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t o_at = mine + C::O_COL + t * D, q_at = mine + C::Q_COL + t * (D / 2),
                       s_at = mine + C::S_COL + t * NB * KB;
        uint32_t blocks_done = 0, ends = 0;                  // blocks of this tile so far, and pieces
        // A piece's query rows of this tile, to TMEM (or shared memory); the products of the piece before it with its own
        // are done.
        auto load_q = [&](const Piece &w) {
            // (a pair's products take both CTAs' rows, also where the second has none)
            if (w.k1 < 0 || (!C::PAIR && first >= w.count)) return;
            const int idx = w.idx0 + first + row, i = sk::quotient(idx, p.by_g);
            const bool there = first + row < w.count;
            const __half *src = p.q + (w.row0 + i) * p.q_stride + (long long)(w.h * p.G + idx - i * p.G) * D;
            constexpr int AT = D < 128 ? D / 8 : 16;         // 16-byte loads in flight
#pragma unroll
            for (int c = 0; c < D / 8; c += AT) {
                uint4 x[AT];
#pragma unroll
                for (int e = 0; e < AT; ++e)
                    x[e] = there ? *reinterpret_cast<const uint4 *>(src + (c + e) * 8) : make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < AT; e += 8) {            // 64 components
                    if constexpr (C::QS) {
                        const uint32_t to = base + C::Q + t * C::Q_TILE + (c + e) / 8 * C::Q_SLAB + row * 128;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t d[4] = {x[e + i].x, x[e + i].y, x[e + i].z, x[e + i].w};
                            st_shared_v4(to + ((i ^ (row & 7)) << 4), d);
                        }
                    } else {
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[4 * i] = x[e + i].x;
                            v[4 * i + 1] = x[e + i].y;
                            v[4 * i + 2] = x[e + i].z;
                            v[4 * i + 3] = x[e + i].w;
                        }
                        t5::st32(q_at + (c + e) * 4, v);
                    }
                }
            }
            if constexpr (C::QS) t5::fence_async_smem();
            else t5::wait_st();
            t5::fence_before();
            __syncwarp();
            if (lane == 0) arrive(q_ready + 8 * t);
        };
        here();
        __syncwarp();
        load_q(list[at]);
        // (a wait that ran out ends every role's way: what is listed after it may be an earlier lap's)
        while (!__any_sync(0xffffffffu, dead) && list[at].k1 >= 0) {
            const Piece &w = list[at];
            const int n = w.k1 - w.k0;
            const bool active = C::PAIR || first < w.count;
            float t0 = 0.f, t1 = 0.f, most = -FLT_MAX;       // the row's base, and what moves it (at first: any score)
            bool far = false;                                // whether a row of the warp has a t1
            uint64_t sum = two(0.f, 0.f);
            if (active) {
                const int i = sk::quotient(w.idx0 + first + row, p.by_g);
                const int lim = first + row < w.count ? w.lim0 + i - sk::quotient(w.idx0, p.by_g) : 0;
                const int low = p.window ? lim - p.window : 0;
                const int lim0 = w.lim0, low1 = p.window ? w.lim1 - p.window : 0;
                int pos = w.k0 * KB;
                for (int j = 0; j < n; ++j) {
                    const uint32_t sb = blocks_done & 1u;
                    const uint32_t s_col = s_at + sb * KB;
                    wait(s_full + 8 * (t * NB + sb), (blocks_done >> 1) & 1u);
                    __syncwarp();
                    ++blocks_done;
                    t5::fence_after();
                    auto weighted = [&] {
                        t5::wait_st();
                        t5::fence_before();
                        __syncwarp();
                        if (lane == 0) arrive(p_ready + 8 * (t * NB + sb));
                        pos += KB;
                    };
                    float s[KB];
                    t5::ld64(s_col, s);
                    if (pos + KB > lim0 || (pos + KB > p.sinks && pos < low1)) {
#pragma unroll
                        for (int e = 0; e < KB; ++e)
                            if (pos + e >= lim || (pos + e >= p.sinks && pos + e < low)) s[e] = NEG_INF;
                    }
                    float m0 = NEG_INF, m1 = NEG_INF, m2 = NEG_INF, m3 = NEG_INF;
#pragma unroll
                    for (int e = 0; e < KB; e += 2) {
                        float &m = e % 8 == 0 ? m0 : e % 8 == 2 ? m1 : e % 8 == 4 ? m2 : m3;
                        m = fmaxf(fmaxf(s[e], s[e + 1]), m);       // (one instruction)
                    }
                    m0 = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
                    const bool moves = fmaf(m0, p.c, -t0) - t1 > most;
                    if (__any_sync(0xffffffffu, moves || far)) {
                        const float h = m0 * p.c, was0 = t0, was1 = t1;
                        if (moves) {
                            t0 = fabsf(h) < FAR ? h - P_SHIFT : h;
                            t1 = fabsf(h) < FAR ? 0.f : __fadd_ru(fmaf(m0, p.c, -h), -P_SHIFT);
                        }
                        const float f = most < 0.f ? 0.f : ex2((was0 - t0) + (was1 - t1));
                        if (moves) most = P_SHIFT + SLACK;
                        far = __any_sync(0xffffffffu, t1 != 0.f);
                        const float2 l = apart(sum);
                        sum = two(l.x * f, l.y * f);
                        if (j > 0) {
                            // The output so far, once the product before this one is done. (A barrier tells a phase from the
                            // next only; the product before that is done, its scores' successors being here.)
                            wait(o_done + 8 * t, (blocks_done - 2) & 1u);
                            __syncwarp();
                            t5::fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                float o[32];
                                t5::ld32(o_at + c, o);
                                uint32_t v[32];
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(o[e] * f);
                                t5::st32(o_at + c, v);
                            }
                        }
                        if (far) {
#pragma unroll 1
                            for (int c = 0; c < KB; c += 8) {          // (weights over scores already read)
                                float x[8];
                                uint32_t y16[4];
                                t5::ld8(s_col + c, x);
#pragma unroll
                                for (int e = 0; e < 8; e += 2) {
                                    float y[2];
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        const int at = pos + c + e + i;
                                        const bool seen = at < lim && (at < p.sinks || at >= low);
                                        y[i] = seen ? ex2(fmaf(x[e + i], p.c, -t0) - t1) : 0.f;
                                    }
                                    sum = add2(sum, two(y[0], y[1]));
                                    y16[e / 2] = pack_f16(y[0], y[1]);
                                }
                                t5::st4(s_col + c / 2, y16);
                            }
                            weighted();
                            continue;
                        }
                    }
                    const uint64_t c2 = two(p.c, p.c), n2 = two(-t0, -t0);
#pragma unroll
                    for (int e = 0; e < KB; e += 2) {
                        const float2 x = apart(fma2(two(s[e], s[e + 1]), c2, n2));
                        s[e] = x.x;
                        s[e + 1] = x.y;
                    }
                    uint32_t y16[KB / 2];
#pragma unroll
                    for (int e = 0; e < KB; e += 2) {
                        const float y0 = ex2(s[e]), y1 = ex2(s[e + 1]);
                        sum = add2(sum, two(y0, y1));
                        y16[e / 2] = pack_f16(y0, y1);
                    }
                    t5::st32(s_col, y16);
                    weighted();
                }
            }
            // The next piece's query rows first: its scores are formed beside this one's end.
            const uint32_t after = at + 1 == C::LIST ? 0 : at + 1;
            wait(l_full + 8 * after, after ? lap : lap ^ 1u);
            __syncwarp();
            if (!__any_sync(0xffffffffu, dead)) load_q(list[after]);      // (else it may be half written)
            // ---- the rows' outputs, or their part of them
            const bool whole = w.k0 == 0 && w.k1 == w.blocks, there = first + row < w.count;
            const size_t slot = size_t(worker<D>()) * 2 + (w.k0 == 0 ? 1 : 0);
            if (active) {
                wait(o_end + 8 * t, ends++ & 1u);
                __syncwarp();
                t5::fence_after();
                const float2 ll = apart(sum);
                const float l = ll.x + ll.y, f = l == 0.f ? 0.f : p.vg / l;
                const int idx = w.idx0 + first + row, i = sk::quotient(idx, p.by_g);
                const int to = (w.row0 + i) * (p.heads * p.G) + w.h * p.G + idx - i * p.G;      // (rows by 31 bits)
                // 128 bytes of every row at a time, turned in shared memory so that eight lanes store them: 64 components
                // of the output, or 32 of a part of it (a lane a row, a store meets 32 lines: 6000 clocks a tile of 256
                // components, this way a third)
                const uint32_t room = base + C::OUT + warp * 4096;
                const int rows = min(32, w.count - first - (warp & 3) * 32);
                auto put = [&](int piece, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
                    const uint32_t v[4] = {a, b, c, d};
                    st_shared_v4(room + lane * 128 + ((piece ^ (lane & 7)) << 4), v);
                };
                const int r0 = lane >> 3, piece = lane & 7;
                if (whole) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            float o[32];
                            t5::ld32(o_at + c + 32 * hf, o);
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                put(4 * hf + e / 8, pack_f16(o[e] * f, o[e + 1] * f), pack_f16(o[e + 2] * f, o[e + 3] * f),
                                    pack_f16(o[e + 4] * f, o[e + 5] * f), pack_f16(o[e + 6] * f, o[e + 7] * f));
                        }
                        __syncwarp();
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const int r = 4 * x + r0;
                            const uint4 v = sk::ld_shared_v4(room + r * 128 + ((piece ^ (r & 7)) << 4));
                            const int its = __shfl_sync(0xffffffffu, to, r);
                            if (r < rows) *reinterpret_cast<uint4 *>(p.out + (long long)its * D + c + piece * 8) = v;
                        }
                        __syncwarp();
                    }
                } else {
                    float *part = p.part_o + (slot * C::ROWS + first + (warp & 3) * 32) * D;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        t5::ld32(o_at + c, o);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            put(e / 4, __float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                                __float_as_uint(o[e + 3]));
                        __syncwarp();
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const int r = 4 * x + r0;
                            const uint4 v = sk::ld_shared_v4(room + r * 128 + ((piece ^ (r & 7)) << 4));
                            if (r < rows) *reinterpret_cast<uint4 *>(part + r * D + c + piece * 4) = v;
                        }
                        __syncwarp();
                    }
                }
                if (there) {
                    if (whole) write_lse(p, to, t0, t1, l);
                    else
                        *reinterpret_cast<float4 *>(p.part_ml + (slot * C::ROWS + first + row) * 4) = make_float4(t0, t1, l, 0.f);
                }
            }
            t5::fence_before();
            __syncwarp();
            leave(lane == 0);
        }
    } else if (warp < C::SW + C::DW) {
        // ------------------------------------------------------- decoding
        // One stream of blocks over all pieces, of keys for the one half of the warps and of values for the other (a
        // warp that does both meets two waits and two fences a block). The records of a block are looked up three blocks
        // ahead of its decoding, their bytes fetched two ahead.
        const bool value = warp >= C::SW + C::HW;
        const int w = warp - C::SW - (value ? C::HW : 0);
        const uint32_t full = value ? v_full : k_full, empty = value ? v_empty : k_empty, ring = base + (value ? C::V : C::K);
        uint32_t to[4];
        bool odd = false;
        if (value) value_offsets<D>(w, lane, to, odd);
        else key_offsets<D>(w, lane, to);
        uint32_t codes_at, scales_at;
        source_offsets<D>(value, w, lane, rank, codes_at, scales_at);
        int block = 0, end_block = 0, last = 0, gap = 0, skip = 0, next_head = 0;
        const int32_t *table = p.table;
        int entry = 0, in_page = 0, head = 0;                // of the block looked up: the page and the record in it that this
                                                             // lane asked for (used only when fetched: the load has time)
        auto look_up = [&] {                                 // the next block's records; false after the last block
            while (block == end_block) {
                here();
                __syncwarp();
                const Piece &w = list[at];
                if (__any_sync(0xffffffffu, dead) || w.k1 < 0) return false;
                block = w.k0;
                end_block = w.k1;
                table = p.table + (long long)w.b * p.width;
                last = max(0, (w.lim1 + sk::KV4_REC - 1) / sk::KV4_REC - 1);
                gap = w.gap;
                skip = w.skip;
                next_head = w.h;
                __syncwarp();
                leave(lane == 0);
            }
            const int v = min(block * (KB / sk::KV4_REC) + (lane & 3), last);
            const int r = v >= gap ? v + skip : v, pg = sk::quotient(r, p.by_recs);
            entry = table[pg];
            in_page = r - pg * p.recs;
            head = next_head;
            ++block;
            return true;
        };
        auto fetch = [&](Raw<D> &raw) {
            const uint8_t *rec[C::ROUNDS];
            const uint32_t found = (uint32_t(min(max(entry, 0), p.pages - 1)) * p.heads + head) * p.recs + in_page;
#pragma unroll
            for (int x = 0; x < C::ROUNDS; ++x)
                rec[x] = p.cache + size_t(__shfl_sync(0xffffffffu, found, record_of<D>(value, w, x, rank))) * sk::kv4_rec_bytes(D);
#pragma unroll
            for (int x = 0; x < C::ROUNDS; ++x) {
                raw.c[x] = *reinterpret_cast<const uint4 *>(rec[x] + codes_at);
                raw.s[x] = ld_u16(rec[x] + scales_at);
            }
        };
        Raw<D> raw[2];
        bool there[2], more = look_up();                     // blocks fetched; whether rec is another's
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            there[x] = more;
            if (more) {
                fetch(raw[x]);
                more = look_up();
            }
        }
        uint32_t st = 0, parity = 1;                         // (the first use of each stage finds it free)
        while (there[0]) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!there[x]) {
                    there[0] = false;
                    break;
                }
                wait(empty + 8 * st, parity);
                if (value) decode_values<D>(ring + st * C::STAGE, to, odd, raw[x]);
                else decode_keys<D>(ring + st * C::STAGE, to, raw[x]);
                t5::fence_async_smem();
                __syncwarp();
                if (lane == 0 && !p.stall) arrive(full + 8 * st);
                if (++st == ST) {
                    st = 0;
                    parity ^= 1u;
                }
                there[x] = more;
                if (more) {
                    fetch(raw[x]);
                    more = look_up();
                }
            }
        }
    } else if (warp == C::SW + C::DW) {
        // ------------------------------------------------------- products
        // One elected lane: what it issues takes its operands from uniform registers (from a lane chosen by number a
        // product of 64 columns takes 45 clocks to issue, of the 32 it runs). Stages, parities and operands are carried
        // along: a lone warp's instructions are ten clocks apart, and a block's turn here is on everyone's path.
        if (rank != 0) {
            while (true) {             // (the first CTA's thread reads the pieces that this one lists)
                wait_long(l_full + 8 * at, lap);
                __syncwarp();
                if (__any_sync(0xffffffffu, dead) || list[at].k1 < 0) break;
                __syncwarp();
                leave(lane == 0);
            }
        } else if (t5::elect()) {
            constexpr uint64_t STEP = C::STAGE / 16;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (!dead && !t5::wait_spin<C::PAIR>(bar, parity)) give_up();
            };
            const uint64_t k_op0 = t5::operand(base + C::K, 16, 1024), v_op0 = t5::operand(base + C::V, C::V_SLAB, 1024),
                           q_op = t5::operand(base + C::Q, 16, 1024);     // (of query rows in shared memory)
            uint64_t k_op = k_op0, v_op = v_op0;
            uint32_t ks = 0, kp = 0, vs = 0, vp = 0;             // stages of keys and values and their parities
            uint32_t sb[2] = {0, 0};                             // blocks scored, of each tile
            uint32_t wb[2] = {0, 0};                             // blocks weighted
            uint32_t pieces[2] = {0, 0};
            // S of tile t from the stage's keys
            auto scores = [&](int t) {
                const uint32_t b = sb[t]++ & 1u, d = tmem + C::S_COL + (t * NB + b) * KB;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t k = k_op + ((s >> 2) * C::K_SLAB + (s & 3) * 32) / 16;
                    if constexpr (C::QS)
                        t5::mma_smem(d, q_op + (t * C::Q_TILE + (s >> 2) * C::Q_SLAB + (s & 3) * 32) / 16, k, t5::shape<C::PAIR>(KB, false),
                                     s > 0);
                    else t5::mma<C::PAIR>(d, tmem + C::Q_COL + t * (D / 2) + 8 * s, k, t5::shape<C::PAIR>(KB, false), s > 0);
                }
                t5::commit<C::PAIR>(s_full + 8 * (t * NB + b));
            };
            auto keys_ready = [&] {
                wait(k_full + 8 * ks, kp);
                t5::fence_after();
            };
            auto keys_used = [&] {
                t5::commit<C::PAIR>(k_empty + 8 * ks);
                k_op += STEP;
                if (++ks == ST) {
                    ks = 0;
                    kp ^= 1u;
                    k_op = k_op0;
                }
            };
            auto values = [&](int t, bool first, bool last) {
                const uint32_t n = wb[t]++, b = n & 1u, a = tmem + C::S_COL + (t * NB + b) * KB;
                wait(p_ready + 8 * (t * NB + b), (n >> 1) & 1u);
                t5::fence_after();
#pragma unroll
                for (int s = 0; s < KB / 16; ++s)
                    t5::mma<C::PAIR>(tmem + C::O_COL + t * D, a + 8 * s, v_op + s * 2048 / 16, t5::shape<C::PAIR>(D, true), !first || s > 0);
                t5::commit<C::PAIR>(o_done + 8 * t);
                if (last) t5::commit<C::PAIR>(o_end + 8 * t);
            };
            while (true) {
                wait(l_full + 8 * at, lap);
                if (dead) break;
                const int k1 = list[at].k1, n = k1 - list[at].k0;
                const bool two = T == 2 && list[at].count > 128;
                if (k1 < 0) break;
                leave(true);
                wait(q_ready, pieces[0]++ & 1u);
                if (two) wait(q_ready + 8, pieces[1]++ & 1u);
                for (int j = 0; j < min(n, 2); ++j) {
                    keys_ready();
                    scores(0);
                    if (T == 2 && two) scores(1);
                    keys_used();
                }
                // A tile's scores two blocks on follow its product directly: a tile need not wait for the other's weights.
                for (int j = 0; j < n; ++j) {
                    const bool last = j + 1 == n, more = j + 2 < n;
                    wait(v_full + 8 * vs, vp);
                    values(0, j == 0, last);
                    if (more) {
                        keys_ready();
                        scores(0);
                    }
                    if (T == 2 && two) {
                        values(1, j == 0, last);
                        if (more) scores(1);
                    }
                    if (more) keys_used();
                    t5::commit<C::PAIR>(v_empty + 8 * vs);
                    v_op += STEP;
                    if (++vs == ST) {
                        vs = 0;
                        vp ^= 1u;
                        v_op = v_op0;
                    }
                }
            }
            // every product is done before the TMEM is given back
            t5::commit<C::PAIR>(end);
            t5::wait_spin(end, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- the list
        if (lane == 0 && blockIdx.x == 0) *p.tiles = tiles;
        Piece w = {};
        int t = 0, number = 0, cost = 0, last_join = 0;
        const int me = worker<D>();
        for (bool more = true; more;) {
            more = work.next(p, w, t, number, cost);
            if (!more) {
                w = Piece{};               // the end: nothing of it may be taken for a piece's
                w.k1 = -1;
            }
            if (more && rank == 0 && !p.whole && w.k0 == 0) {
                // A tile in parts is this CTA's last piece: its share ends within it, and the tile's last unit tells the last
                // part's owner.
                int parts = 0;
                if (w.k1 != w.blocks) parts = owner_of(share, bound_of(share, me + 1) + (cost - work.x) - 1) - me + 1;
                if (lane == 0) {
                    const long long place = (long long)w.h * tiles + number;       // (more only where starts descends)
                    if (p.by_tile && place < p.ctas) p.join[place] = Join::of(me, parts, w.h, w.b, t);
                    if (!p.by_tile && parts) p.join[me] = Join::of(me, parts, w.h, w.b, t);
                }
                last_join |= parts;
            }
            // (after a wait that ran out the tiles in parts are listed all the same: the join reads of every one where it is)
            if (__any_sync(0xffffffffu, dead)) continue;
            // Rows that see nothing are done here: a piece without blocks is not listed. (The decoding warps ask for the
            // next piece while they hold two blocks not decoded, whose pieces keep their places meanwhile: the list has
            // places enough as long as every piece has a block.)
            if (more && w.k1 == w.k0) {
                nothing_seen<D>(p, w, C::PAIR ? rank * 128 : 0, lane);
                continue;
            }
            // its query rows, on their way to L2
            if (more) {
                const int lo = C::PAIR ? rank * 128 : 0, hi = min(w.count, lo + 128 * T);
                for (int r = lo + lane; r < hi; r += 32) {
                    const int i = sk::quotient(w.idx0 + r, p.by_g), g = w.idx0 + r - i * p.G;
                    const __half *src = p.q + (w.row0 + i) * p.q_stride + (long long)(w.h * p.G + g) * D;
#pragma unroll
                    for (int c = 0; c < D; c += 64) sk::prefetch_l2(src + c);
                }
            }
            wait_long(l_empty + 8 * at, lap ^ 1u);
            if (__any_sync(0xffffffffu, dead)) continue;
            if (lane == 0) {
                *reinterpret_cast<Piece *>(smem + C::PIECES + at * 64) = w;
                sk::mbar_arrive(l_full + 8 * at);
            }
            if (++at == C::LIST) {
                at = 0;
                lap ^= 1u;
            }
        }
        if (lane == 0 && rank == 0 && !p.by_tile && !last_join) p.join[me] = Join::of(0, 0, 0, 0, 0);
        __syncwarp();
    }
    if (dead) atomicOr(p.err, 1u);
    if constexpr (C::PAIR) {
        // neither CTA leaves while the other, or a product's end, may arrive at its barriers
        if (warp == 0) t5::wait_spin(end, 0);
        __syncwarp();
        t5::fence_before();
        sk::cluster_sync();
    } else {
        t5::fence_before();
        __syncthreads();
    }
    t5::fence_after();
    if (warp == 0) t5::free<C::PAIR>(tmem, 512);
}

// The tiles that several CTAs had parts of: CTA (c, y) joins eight rows of a tile, a
// warp a row, in the order of the parts.
constexpr int JT = 256;
template <int D>
__global__ void __launch_bounds__(JT) kv4_chunk_join_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cc<D>;
    constexpr int PER = D / 32;
    sk::pdl_wait_primary();
    if (p.by_tile && int(blockIdx.x) >= *p.tiles * p.heads) return;
    const int4 seg = p.join[blockIdx.x];
    const int n = seg.y & 0xFFFF, h = seg.y >> 16;
    if (n == 0) return;
    const Seq s(p, seg.z);
    const Tile<D> tile(p, s, seg.w);
    const int lane = threadIdx.x & 31, r = blockIdx.y * (JT / 32) + (threadIdx.x >> 5);
    if (r >= tile.count) return;
    const int idx = tile.idx0 + r, i = sk::quotient(idx, p.by_g);
    const long long at = (long long)(s.first + i) * (p.heads * p.G) + h * p.G + idx - i * p.G;
    auto slot = [&](int k) { return (size_t(seg.x) + k) * 2 + (k == 0 ? 1 : 0); };
    float top0 = -FLT_MAX, top1 = 0.f, l = 0.f, v[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) v[x] = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {           // 32 parts at a time, under the largest base so far
        float4 ml = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + lane < n) ml = *reinterpret_cast<const float4 *>(p.part_ml + (slot(k0 + lane) * C::ROWS + r) * 4);
        // (a part in which the row saw nothing has no base)
        const float old0 = top0, old1 = top1, base = ml.z == 0.f ? -FLT_MAX : ml.x;
        auto larger = [&](float x0, float x1) {    // (bases of FP64 numbers took 30 us for 57000 rows)
            if ((x0 - top0) + (x1 - top1) > 0.f) {
                top0 = x0;
                top1 = x1;
            }
        };
        larger(base, ml.y);
#pragma unroll
        for (int o = 16; o; o >>= 1) larger(__shfl_xor_sync(0xffffffffu, top0, o), __shfl_xor_sync(0xffffffffu, top1, o));
        const float old = ex2((old0 - top0) + (old1 - top1)), f = ml.z == 0.f ? 0.f : ex2((base - top0) + (ml.y - top1));
        float add = ml.z * f;
#pragma unroll
        for (int o = 16; o; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
        l = l * old + add;
#pragma unroll
        for (int x = 0; x < PER; ++x) v[x] *= old;
        const int kn = min(32, n - k0);
#pragma unroll 4
        for (int k = 0; k < kn; ++k) {
            const float w = __shfl_sync(0xffffffffu, f, k);
            const float2 *src = reinterpret_cast<const float2 *>(p.part_o + (slot(k0 + k) * C::ROWS + r) * D) + lane;
#pragma unroll
            for (int x = 0; x < PER / 2; ++x) {
                const float2 y = src[32 * x];
                v[2 * x] += y.x * w;
                v[2 * x + 1] += y.y * w;
            }
        }
    }
    const float f = l == 0.f ? 0.f : p.vg / l;
    __half2 *const out = reinterpret_cast<__half2 *>(p.out + at * D) + lane;
#pragma unroll
    for (int x = 0; x < PER / 2; ++x) out[32 * x] = __floats2half2_rn(v[2 * x] * f, v[2 * x + 1] * f);
    if (lane == 0) write_lse(p, at, top0, top1, l);
}

template <int D>
sk_status run(ChunkParams &p, unsigned char *scratch, int sms, cudaStream_t s) {
    using C = Cc<D>;
    static_assert(C::MOST_SEQS >= MOST_SEQS, "the list of sequences");
    p.ctas = C::PAIR ? sms / 2 : sms;
    if (p.ctas < 1) return SK_ERR_CUDA;
    // No more tiles than these, and no more blocks in one.
    const long long list = (long long)p.rows * p.G, tiles = ((list + C::ROWS - 1) / C::ROWS + (p.B < p.rows ? p.B : p.rows)) * p.heads;
    const long long seen = p.window ? (long long)p.window + p.sinks + list / p.G + 2 * sk::KV4_REC : p.cap;
    const long long blocks = ((seen < p.cap ? seen : p.cap) + KB - 1) / KB;
    p.whole = tiles <= p.ctas && blocks <= WHOLE_BLOCKS;
    p.by_tile = tiles <= p.ctas;
    p.tiles = reinterpret_cast<int *>(scratch);
    p.join = reinterpret_cast<int4 *>(scratch + 256);
    p.part_ml = reinterpret_cast<float *>(scratch + 256 + (size_t(p.ctas) * sizeof(int4) + 255) / 256 * 256);
    p.part_o = p.part_ml + size_t(p.ctas) * 2 * C::ROWS * 4;
    if (size_t(reinterpret_cast<unsigned char *>(p.part_o + size_t(p.ctas) * 2 * C::ROWS * D) - scratch) > sk::SCRATCH_BYTES)
        return SK_ERR_WORKSPACE;
    if (sk::prepare_kernel<kv4_chunk_kernel<D>>(C::SMEM) != cudaSuccess) return SK_ERR_CUDA;
    const int cluster = C::PAIR ? 2 : 1;
    if (sk::launch_pdl_cluster(kv4_chunk_kernel<D>, cluster, dim3(unsigned(p.ctas * cluster)), dim3(C::CT_ALL), C::SMEM, s, p) !=
        cudaSuccess)
        return SK_ERR_CUDA;
    if (p.whole) return SK_OK;
    const unsigned int rows = unsigned(list < C::ROWS ? list : C::ROWS);
    return sk::launch_pdl(kv4_chunk_join_kernel<D>, dim3(unsigned(p.by_tile ? tiles : p.ctas), (rows + JT / 32 - 1) / (JT / 32)),
                          dim3(JT), 0, s, p) == cudaSuccess
               ? SK_OK
               : SK_ERR_CUDA;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

namespace sk {
namespace attn {

sk_status chunk_rows(const AttnParams &a, int head_dim, unsigned char *scratch, int sms, cudaStream_t s) {
    ChunkParams p = {};
    static_cast<AttnParams &>(p) = a;
    p.cap = a.limit;
    p.rows = a.B * a.M;
    p.by_g = sk::Div(uint32_t(a.G));
    switch (head_dim) {
        case 64: return run<64>(p, scratch, sms, s);
        case 128: return run<128>(p, scratch, sms, s);
        default: return run<256>(p, scratch, sms, s);
    }
}

}  // namespace attn
}  // namespace sk

extern "C" sk_status kv4_chunk_attention(const void *q, long long q_stride, const uint8_t *cache, const int32_t *table,
                                         const int32_t *lens, const int32_t *starts, float k_scale, float v_scale,
                                         float scale, int window, int sinks, void *out, float *lse, int rows, int seqs,
                                         int q_heads, int kv_heads, int head_dim, int pages, int page_size,
                                         int table_width, void *stream) {
    if (seqs < 0 || rows < 0 || q_heads < 1 || kv_heads < 1 || pages < 1 || page_size < 1 || table_width < 1 || window < 0 ||
        sinks < 0)
        return SK_ERR_INVALID_ARG;
    if (q_heads % kv_heads) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_scale_ok(k_scale) || !sk::kv4_scale_ok(v_scale) || !(scale > 0.f && scale < 1e20f)) return SK_ERR_INVALID_ARG;
    const double product = double(scale) * double(k_scale);        // bounds as in kv4_attention
    if (!(product >= 5e-37 && product <= 1e27)) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_shape_ok(pages, kv_heads, head_dim, page_size)) return SK_ERR_UNSUPPORTED_SHAPE;
    // positions and rows of a kv head's list with room for a tile and a block, query rows by 31 bits
    if (seqs > MOST_SEQS || (long long)table_width * page_size > 0x7FFFF000LL || (long long)rows * (q_heads / kv_heads) > 0x3FFFF000LL ||
        (long long)rows * q_heads > 0x7FFFFFFFLL)
        return SK_ERR_UNSUPPORTED_SHAPE;
    if (seqs == 0 || rows == 0) return SK_OK;
    if (!q || !cache || !table || !lens || !starts || !out) return SK_ERR_INVALID_ARG;
    if (q_stride < (long long)q_heads * head_dim) return SK_ERR_INVALID_ARG;
    if (q_stride % 8 || !aligned(q, 16) || !aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(starts, 4) || !aligned(out, 16) || !aligned(lse, 4))
        return SK_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    sk::Scratch sc;
    if (!sk::scratch_for(s, &sc)) return SK_ERR_NOT_INITIALIZED;
    ChunkParams p = {};
    p.q = static_cast<const __half *>(q);
    p.q_stride = q_stride;
    p.cache = cache;
    p.table = table;
    p.lens = lens;
    p.starts = starts;
    p.out = static_cast<__half *>(out);
    p.lse = lse;
    p.err = sc.err;
    p.rows = rows;
    p.B = seqs;
    p.heads = kv_heads;
    p.G = q_heads / kv_heads;
    p.by_g = sk::Div(uint32_t(p.G));
    p.pages = pages;
    p.recs = page_size / sk::KV4_REC;
    p.by_recs = sk::Div(p.recs);
    p.width = table_width;
    p.cap = table_width * page_size;
    p.window = window < p.cap ? window : p.cap;
    p.sinks = sinks < p.cap ? sinks : p.cap;
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
