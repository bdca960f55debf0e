// kv4_evict.cu -- keep the most attended positions of each sequence and kv
// head within a budget, in their order, in other pages.
//
// Per (sequence b, kv head h) with n = lens[b] positions: if n <= budget all
// are kept; otherwise the last `recent` ones and, of the n - recent before
// them, the budget - recent with the largest accumulated weight, ties to the
// lower position.  Kept position number j is copied to slot j of the
// sequence's destination pages.  The source pages are only read, so pages
// shared with another sequence stay valid.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/skinny.h"
#include "cluster.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "launch_util.cuh"

namespace {

constexpr int ET = 256;            // threads per CTA
constexpr int WARPS = ET / 32;
constexpr int KEYS = 8192;         // keys kept in shared memory (the rest are read again)
constexpr int BINS = 512;
constexpr int FEW = 64;            // candidates left at which the selection ends by counting
constexpr int CHUNK = 1024;        // records numbered at a time
constexpr int MAX_CLUSTER = 16;
constexpr int SOLO_MAX = KEYS;     // positions up to which a CTA selects alone

struct EvictParams {
    uint8_t *cache;
    const int32_t *table, *dst, *lens;
    const float *acc;
    float *acc_out;
    int32_t *kept, *new_lens;
    unsigned int *err;
    int stall;                         // issue no copies (sk_inject_wait_timeout)
    int pages, heads, recs, width, dst_width, cap, dst_cap;
    int budget, recent;
    sk::Div by_recs;
};

// Records with something to keep.
struct List {
    uint32_t src[CHUNK], dst[CHUNK][2];    // record in the cache; those of the first kept position and the next
    int rec[CHUNK];                        // number in the sequence
    uint32_t base[CHUNK];                  // slot of the first kept position
    uint16_t mask[CHUNK];                  // positions kept
    uint32_t masks[CHUNK];                 // per record: kept for sure (low half), equal to the threshold (high half)
};

template <int SLOTS>
struct alignas(16) Shared {
    union {
        unsigned int bins[BINS];       // while selecting
        List list;                     // afterwards
    };
    unsigned int hist[2][BINS];
    unsigned long long mine[FEW];      // this CTA's candidates
    unsigned long long few[FEW];       // the cluster's
    unsigned int range[2];             // this CTA's smallest and largest key
    unsigned int counts[3];            // this CTA's: above the digits, equal to the threshold, candidates
    unsigned int first[MAX_CLUSTER + 1];   // of each CTA's candidates among the cluster's
    unsigned int gt[MAX_CLUSTER], eq[MAX_CLUSTER];
    unsigned int scan[ET / 32];
    unsigned int prefix, need, pop, above;
    unsigned long long limit;
    unsigned char nth[WARPS][16];      // the position of a record's n-th kept one
    alignas(8) unsigned long long bar[WARPS][SLOTS];
};

// Source records in flight per warp.
__host__ __device__ constexpr int ring_slots(int d) { return d == 256 ? 2 : 4; }

// Inclusive prefix sum over the CTA in thread order (tmp: ET / 32 words); the
// sum of all goes to *total.  Ends with a barrier before tmp is free again.
__device__ __forceinline__ unsigned int inclusive(unsigned int x, unsigned int *tmp, unsigned int *total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) tmp[wid] = x;
    __syncthreads();
    unsigned int all = 0;
#pragma unroll
    for (int w = 0; w < ET / 32; ++w) {
        if (w < wid) x += tmp[w];
        all += tmp[w];
    }
    *total = all;
    __syncthreads();
    return x;
}

// A position as a candidate: larger weight first, then the lower position.
__device__ __forceinline__ unsigned long long cand_of(unsigned int key, int pos) {
    return (static_cast<unsigned long long>(key) << 32) | static_cast<unsigned int>(~pos);
}

// C CTAs per (sequence, kv head); CTA r copies what is kept of the r-th
// contiguous part of the records.  Up to a length every CTA selects over all
// positions by itself (SOLO), which costs less than talking to the others;
// beyond it the CTAs are a cluster, each selecting over its own part.
//
// The selection is a radix select, nine bits a pass from the highest bit in
// which the weights differ, on histograms (summed over the cluster through
// distributed shared memory).  As soon as the digit that holds the threshold
// has few positions left, every CTA gathers them all and counts each one's
// rank.  The copy streams the records that hold a kept position through shared
// memory, a ring per warp: a position's value codes are eight-byte pieces and
// its value scales single bytes, each in a 32-byte sector of its own, so
// fetching only what is kept moves as many sectors and costs a load for each
// (a kernel of its own for the copies, a warp gathering a record's 16
// positions: 34 us where this takes 30, 19 us where this takes 15).
//
// Bound by latency, and by what the longest sequence's cluster copies: 16
// sequences of up to 16411 positions, 2 heads of 256, 4096 kept, 30 us (59 MB
// read and written at least, 8.8 us); one of 1500 positions, 4 heads of 128, 7 us.
template <int D, bool SOLO>
__global__ void __launch_bounds__(ET) kv4_evict_kernel(const __grid_constant__ EvictParams p, int ctas) {
    constexpr int REC = sk::kv4_rec_bytes(D), NB = D / 16, SLOTS = ring_slots(D);
    extern __shared__ __align__(128) unsigned char smem[];      // keys, later the records' ring
    __shared__ Shared<SLOTS> sh;
    unsigned int *const keys = reinterpret_cast<unsigned int *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (lane == 0)
        for (int s = 0; s < SLOTS; ++s) sk::mbar_init(sk::smem_u32(&sh.bar[warp][s]), 1);
    sk::fence_barrier_init();
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    const unsigned int C = unsigned(ctas), rank = blockIdx.x % C;      // in a cluster, the CTA's rank
    const int bh = blockIdx.x / C, b = bh / p.heads, h = bh - b * p.heads;
    const int n = min(max(p.lens[b], 0), p.cap);
    const int out_n = min(n, p.budget);
    const float *acc = p.acc + size_t(bh) * size_t(p.cap);
    const bool all = n <= p.budget, none_old = !all && p.budget == p.recent, select = !all && !none_old;
    const int old = all ? n : n - p.recent;      // positions the selection decides on
    const int nrec = (n + 15) / 16, part = (nrec + int(C) - 1) / int(C);
    const int rec_lo = min(nrec, int(rank) * part), rec_hi = min(nrec, rec_lo + part);
    const int lo = min(n, rec_lo * 16), hi = min(n, rec_hi * 16);
    // the positions this CTA's selection reads
    const int s_lo = SOLO ? 0 : lo, n_old = SOLO ? old : max(0, min(hi, old) - lo);
    int cached = KEYS;
    auto key_at = [&](int i) { return i < cached ? keys[i] : sk::key_of(acc[s_lo + i]); };  // i counts from s_lo

    unsigned int low = 0, mask = 0, prefix = 0, need = select ? unsigned(p.budget - p.recent) : 0u;
    unsigned int above = 0;                      // this CTA's keys above the digits found so far
    unsigned long long limit = 0ull;             // with `few`: the threshold among candidates
    bool few = false;
    if (tid < 3) sh.counts[tid] = 0u;
    if (select) {
        // ---- keys, and the bits in which they differ
        unsigned int mn = 0xFFFFFFFFu, mx = 0u;
        if (tid == 0) {
            sh.range[0] = 0xFFFFFFFFu;
            sh.range[1] = 0u;
        }
        __syncthreads();
        sh.bins[tid] = 0u;
        sh.bins[tid + ET] = 0u;
        static_assert(BINS == 2 * ET, "two bins per thread");
        for (int i0 = tid; i0 < n_old; i0 += 16 * ET) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = i0 + j * ET < n_old ? acc[s_lo + i0 + j * ET] : 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int i = i0 + j * ET;
                if (i < n_old) {
                    const unsigned int k = sk::key_of(v[j]);
                    if (i < KEYS) keys[i] = k;
                    mn = min(mn, k);
                    mx = max(mx, k);
                }
            }
        }
        mn = __reduce_min_sync(0xffffffffu, mn);
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) {
            atomicMin(&sh.range[0], mn);
            atomicMax(&sh.range[1], mx);
        }
        if constexpr (SOLO) {
            __syncthreads();
            mn = sh.range[0];
            mx = sh.range[1];
        } else {
            sk::cluster_sync();
            const unsigned int of = unsigned(lane) & (C - 1u);
            mn = __reduce_min_sync(0xffffffffu, sk::ld_peer_u32(sk::peer(&sh.range[0], of)));
            mx = __reduce_max_sync(0xffffffffu, sk::ld_peer_u32(sk::peer(&sh.range[1], of)));
        }
        // digits of key - low, from its highest bit down (uniform in the cluster)
        low = mn;
        int top = 32 - __clz(mx - mn);           // bits still undecided
        int pass = 0;
        while (top > 0 && !few) {
            const int bits = min(9, top), shift = top - bits;
            const unsigned int bins = (1u << bits) - 1u;
#pragma unroll 4
            for (int i = tid; i < n_old; i += ET) {
                const unsigned int k = key_at(i) - low;
                if ((k & mask) == prefix) atomicAdd(&sh.bins[(k >> shift) & bins], 1u);
            }
            __syncthreads();
            // thread t takes bins 511 - 2 t and 510 - 2 t, and clears them: an
            // inclusive scan over t is the suffix sum over bins
            uint2 *const two = reinterpret_cast<uint2 *>(&sh.bins[BINS - 2 - 2 * tid]);
            unsigned int t0 = two->y, t1 = two->x;
            *two = make_uint2(0u, 0u);
            unsigned int *const hh = sh.hist[pass & 1];
            if constexpr (!SOLO) {
                hh[BINS - 1 - 2 * tid] = t0;
                hh[BINS - 2 - 2 * tid] = t1;
                sk::cluster_sync();
                unsigned long long w[MAX_CLUSTER];       // all in flight, each CTA beginning with its own
#pragma unroll
                for (unsigned int r = 0; r < MAX_CLUSTER; ++r)
                    w[r] = r < C ? sk::ld_peer_u64(sk::peer(hh + BINS - 2 - 2 * tid, (rank + r) & (C - 1u))) : 0ull;
                t0 = t1 = 0;
#pragma unroll
                for (unsigned int r = 0; r < MAX_CLUSTER; ++r) {
                    t1 += static_cast<unsigned int>(w[r]);
                    t0 += static_cast<unsigned int>(w[r] >> 32);
                }
            }
            unsigned int sum_all;
            const unsigned int x = inclusive(t0 + t1, sh.scan, &sum_all);
            // the digit: >= need keys at or above it, < need above it
            const unsigned int over0 = x - t0 - t1, over1 = x - t1;
            if (over1 >= need && over0 < need) {
                sh.prefix = prefix | (unsigned(BINS - 1 - 2 * tid) << shift);
                sh.need = need - over0;
                sh.pop = t0;
            } else if (x >= need && over1 < need) {
                sh.prefix = prefix | (unsigned(BINS - 2 - 2 * tid) << shift);
                sh.need = need - over1;
                sh.pop = t1;
            }
            if (!SOLO && tid == 0) sh.above = 0u;
            __syncthreads();
            prefix = sh.prefix;
            need = sh.need;
            few = sh.pop <= unsigned(FEW);
            if constexpr (!SOLO) {
                const unsigned int digit = (prefix >> shift) & bins;
                unsigned int mine = (unsigned(2 * tid) > digit ? hh[2 * tid] : 0u) + (unsigned(2 * tid + 1) > digit ? hh[2 * tid + 1] : 0u);
                mine = __reduce_add_sync(0xffffffffu, mine);
                if (lane == 0 && mine) atomicAdd(&sh.above, mine);
                __syncthreads();
                above += sh.above;
            }
            mask |= bins << shift;
            top = shift;
            ++pass;
        }
        if (few) {
            for (int i = tid; i < n_old; i += ET) {
                const unsigned int k = key_at(i);
                if (((k - low) & mask) == prefix) sh.mine[atomicAdd(&sh.counts[2], 1u)] = cand_of(k, s_lo + i);
            }
        } else if (!SOLO) {
            unsigned int eq = 0;
            for (int i = tid; i < n_old; i += ET) eq += key_at(i) - low == prefix;
            eq = __reduce_add_sync(0xffffffffu, eq);
            if (lane == 0 && eq) atomicAdd(&sh.counts[1], eq);
        }
        if (tid == 0) sh.counts[0] = above;
    }

    // ---- what the CTAs before this one keep
    unsigned int gt_before = 0, eq_before = 0;
    if (select && !SOLO) {
        sk::cluster_sync();
        if (tid < 32) {
            const bool in = unsigned(lane) < C;
            const unsigned int c0 = in ? sk::ld_peer_u32(sk::peer(&sh.counts[0], unsigned(lane))) : 0u;
            const unsigned int c1 = in ? sk::ld_peer_u32(sk::peer(&sh.counts[1], unsigned(lane))) : 0u;
            unsigned int x = in ? sk::ld_peer_u32(sk::peer(&sh.counts[2], unsigned(lane))) : 0u;
            if (in) {
                sh.gt[lane] = c0;
                sh.eq[lane] = c1;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (in) sh.first[lane + 1] = x;
            if (lane == 0) sh.first[0] = 0u;
        }
        __syncthreads();
        for (unsigned int r = 0; r < rank; ++r) {
            gt_before += sh.gt[r];
            eq_before += sh.eq[r];
        }
    }
    if (few) {
        // gather every CTA's candidates, and rank them by counting (four threads each)
        const unsigned long long *list = SOLO ? sh.mine : sh.few;
        unsigned int total;
        if constexpr (SOLO) {
            __syncthreads();
            total = sh.counts[2];
        } else {
            total = sh.first[C];
            if (unsigned(tid) < total) {
                unsigned int r = 0;
                while (sh.first[r + 1] <= unsigned(tid)) ++r;
                sh.few[tid] = sk::ld_peer_u64(sk::peer(&sh.mine[unsigned(tid) - sh.first[r]], r));
            }
            __syncthreads();
        }
        static_assert(ET == 4 * FEW, "four threads per candidate");
        const unsigned int c = unsigned(tid) >> 2;
        const unsigned long long v = c < total ? list[c] : 0ull;
        unsigned int larger = 0;
        for (unsigned int j = unsigned(tid) & 3u; j < total; j += 4) larger += list[j] > v;
        larger += __shfl_xor_sync(0xffffffffu, larger, 1);
        larger += __shfl_xor_sync(0xffffffffu, larger, 2);
        if (c < total && larger == need - 1) sh.limit = v;
        __syncthreads();
        limit = sh.limit;
        need = 0;
        if constexpr (!SOLO)    // the candidates of the CTAs before this one that pass
            gt_before += __syncthreads_count(unsigned(tid) < sh.first[rank] && list[tid & (FEW - 1)] >= limit);
    }
    if (select && !SOLO) sk::cluster_sync();     // no CTA leaves while its counts and candidates are read
    // 2: kept, 1: kept if among the first `need` equal to the threshold, 0: not
    auto kind = [&](int i) -> unsigned int {
        if (all || i >= old) return 2u;
        if (none_old) return 0u;
        const unsigned int k = key_at(i - s_lo);
        if (few) return cand_of(k, i) >= limit ? 2u : 0u;
        return k - low > prefix ? 2u : k - low == prefix ? 1u : 0u;
    };
    if (SOLO && select) {
        unsigned int gt = 0, eq = 0;
        for (int i = tid; i < min(lo, old); i += ET) {
            const unsigned int k = kind(i);
            gt += k == 2u;
            eq += k == 1u;
        }
        inclusive(gt, sh.scan, &gt_before);
        inclusive(eq, sh.scan, &eq_before);
    }
    if (all) gt_before = lo;
    else gt_before += max(0, lo - old);          // the recent positions follow the old ones

    // ---- number the kept positions in order and copy them, CHUNK records at a time
    const int32_t *table = p.table + size_t(b) * p.width;
    const int32_t *dtable = p.dst + size_t(b) * p.dst_width;
    int32_t *kept = p.kept + size_t(bh) * size_t(p.budget);
    float *acc_out = p.acc_out ? p.acc_out + size_t(bh) * size_t(p.dst_cap) : nullptr;
    uint32_t done = 0;                           // records this warp has copied: ring position and parity
    const bool issuer = lane == 0 && !p.stall;
    bool dead = false;
    for (int r0 = rec_lo; r0 < rec_hi; r0 += CHUNK) {
        const int nr = min(CHUNK, rec_hi - r0);
        for (int i0 = 0; i0 < nr * 16; i0 += ET) {           // a lane a position: 32 positions are two records
            const int i = r0 * 16 + i0 + tid;
            const unsigned int k = i < hi && i0 + tid < nr * 16 ? kind(i) : 0u;
            const unsigned int two = __ballot_sync(0xffffffffu, k == 2u), one = __ballot_sync(0xffffffffu, k == 1u);
            const int r = (i0 + tid) >> 4;
            if ((lane & 15) == 0 && r < nr) {
                const int s = lane & 16;
                sh.list.masks[r] = ((two >> s) & 0xFFFFu) | (((one >> s) & 0xFFFFu) << 16);
            }
        }
        __syncthreads();
        // base slot of each record, and the list of records with something kept (in order)
        unsigned int listed = 0;
        for (int x0 = 0; x0 < nr; x0 += ET) {
            const unsigned int m = x0 + tid < nr ? sh.list.masks[x0 + tid] : 0u;
            unsigned int two = m & 0xFFFFu, one = m >> 16, tg, te, tl;
            const unsigned int c = (unsigned(__popc(two)) << 16) | unsigned(__popc(one));
            const unsigned int x = inclusive(c, sh.scan, &tg) - c;             // at most 16 ET in each half
            const unsigned int g = gt_before + (x >> 16), e = eq_before + (x & 0xFFFFu);
            unsigned int keep_one = e < need ? need - e : 0u;                  // the first so many of `one`
            while (unsigned(__popc(one)) > keep_one) one &= ~(0x80000000u >> __clz(one));
            const unsigned int keep = two | one;
            te = tg & 0xFFFFu;
            const unsigned int at = inclusive(keep != 0u, sh.scan, &tl);
            if (keep) {
                const unsigned int y = listed + at - 1u, to = g + min(e, need);
                const int rec = r0 + x0 + tid;
                sh.list.rec[y] = rec;
                sh.list.base[y] = to;
                sh.list.mask[y] = uint16_t(keep);
                sh.list.src[y] = sk::kv4_record(table, rec, p.recs, p.by_recs, p.pages, p.heads, h);
                sh.list.dst[y][0] = sk::kv4_record(dtable, int(to >> 4), p.recs, p.by_recs, p.pages, p.heads, h);
                sh.list.dst[y][1] = sk::kv4_record(dtable, int((to + __popc(keep) - 1u) >> 4), p.recs, p.by_recs, p.pages, p.heads, h);
            }
            listed += tl;
            gt_before += tg >> 16;
            eq_before += te;
        }
        const int n_list = int(listed);
        // the ring takes the keys' place (a later chunk reads them again)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        cached = 0;
        unsigned char *const own = smem + warp * SLOTS * REC;
        const uint32_t ring = sk::smem_u32(own);
        auto issue = [&](int y, uint32_t slot) {
            if (issuer && !dead) {
                const uint32_t bar = sk::smem_u32(&sh.bar[warp][slot]);
                sk::mbar_arrive_expect_tx(bar, REC);
                sk::bulk_load(ring + slot * REC, p.cache + size_t(sh.list.src[y]) * REC, REC, bar);
            }
        };
        for (int k = 0; k < SLOTS; ++k)
            if (warp + k * WARPS < n_list) issue(warp + k * WARPS, (done + k) % SLOTS);
        // meanwhile, the kept positions' numbers and weights, eight to a thread in flight
        for (int i0 = tid; i0 < n_list * 16; i0 += 8 * ET) {
            int to[8], from[8];
            float v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int y = (i0 + x * ET) >> 4, j = tid & 15;
                const unsigned int m = y < n_list ? sh.list.mask[y] : 0u;
                to[x] = -1;
                v[x] = 0.f;
                if (m >> j & 1u) {
                    to[x] = int(sh.list.base[y]) + __popc(m & ((1u << j) - 1u));
                    from[x] = sh.list.rec[y] * 16 + j;
                    if (acc_out) v[x] = acc[from[x]];
                }
            }
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (to[x] >= 0) {
                    kept[to[x]] = from[x];
                    if (acc_out) acc_out[to[x]] = v[x];
                }
        }
        for (int y = warp; y < n_list; y += WARPS, ++done) {
            const uint32_t slot = done % SLOTS;
            const unsigned int m = sh.list.mask[y], base = sh.list.base[y];
            const int count = __popc(m);
            if (lane < 16 && (m >> lane & 1u)) sh.nth[warp][__popc(m & ((1u << lane) - 1u))] = uint8_t(lane);
            sk::wait_ring<SLOTS>(sk::smem_u32(&sh.bar[warp][0]), slot, (done / SLOTS) & 1, p.err, dead);
            __syncwarp();
            const unsigned char *src = own + slot * REC;
            // four positions at a time: neighbouring lanes write neighbouring positions of a value block
            for (int q0 = 0; q0 < count; q0 += 4) {
                const int q = q0 + (lane & 3);
                if (q < count) {
                    const int i = sh.nth[warp][q], to = int(base) + q, j = to & 15;
                    uint8_t *dst = p.cache + size_t(sh.list.dst[y][(to >> 4) != int(base >> 4)]) * REC;
#pragma unroll
                    for (int blk = lane >> 2; blk < NB; blk += 8) {
                        *reinterpret_cast<uint2 *>(dst + sk::kv4_code_at<true>(D, j, blk)) =
                            *reinterpret_cast<const uint2 *>(src + sk::kv4_code_at<true>(D, i, blk));
                        *reinterpret_cast<uint2 *>(dst + sk::kv4_code_at<false>(D, j, blk)) =
                            *reinterpret_cast<const uint2 *>(src + sk::kv4_code_at<false>(D, i, blk));
                        dst[sk::kv4_scale_at<true>(D, j, blk)] = src[sk::kv4_scale_at<true>(D, i, blk)];
                        dst[sk::kv4_scale_at<false>(D, j, blk)] = src[sk::kv4_scale_at<false>(D, i, blk)];
                    }
                }
            }
            __syncwarp();
            if (y + SLOTS * WARPS < n_list) issue(y + SLOTS * WARPS, slot);
        }
        __syncthreads();
    }
    for (int j = out_n + int(rank) * ET + tid; j < p.budget; j += int(C) * ET) kept[j] = -1;
    if (acc_out)
        for (int j = out_n + int(rank) * ET + tid; j < p.dst_cap; j += int(C) * ET) acc_out[j] = 0.f;
    if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = out_n;
}

// The keys, and later the records' ring in their place.
template <int D>
constexpr size_t smem_bytes() {
    const size_t ring = size_t(WARPS) * ring_slots(D) * sk::kv4_rec_bytes(D);
    return ring > size_t(KEYS) * 4 ? ring : size_t(KEYS) * 4;
}

template <int D>
sk_status launch(const EvictParams &p, int bh, int ctas, cudaStream_t s) {
    const dim3 grid(unsigned(bh) * unsigned(ctas));
    const size_t smem = smem_bytes<D>();
    cudaError_t e;
    if (p.cap <= SOLO_MAX) {
        e = sk::prepare_kernel<kv4_evict_kernel<D, true>>(smem);
        if (e == cudaSuccess) e = sk::launch_pdl(kv4_evict_kernel<D, true>, grid, dim3(ET), smem, s, p, ctas);
    } else {
        e = sk::prepare_kernel<kv4_evict_kernel<D, false>>(smem, true);
        if (e == cudaSuccess)
            e = sk::launch_pdl_cluster(kv4_evict_kernel<D, false>, ctas, grid, dim3(ET), smem, s, p, ctas);
    }
    return e == cudaSuccess ? SK_OK : SK_ERR_CUDA;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" sk_status kv4_evict(uint8_t *cache, const int32_t *table, const int32_t *lens, const float *acc,
                               const int32_t *dst_table, int32_t *kept, int32_t *new_lens, float *acc_out, int seqs,
                               int budget, int recent, int kv_heads, int head_dim, int pages, int page_size,
                               int table_width, int dst_width, void *stream) {
    if (seqs < 0 || kv_heads < 1 || pages < 1 || page_size < 1 || table_width < 1 || dst_width < 1)
        return SK_ERR_INVALID_ARG;
    if (budget < 1 || recent < 0 || recent > budget) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_shape_ok(pages, kv_heads, head_dim, page_size)) return SK_ERR_UNSUPPORTED_SHAPE;
    if ((long long)table_width * page_size > 0x7FFFFF00LL || (long long)dst_width * page_size > 0x7FFFFF00LL)
        return SK_ERR_UNSUPPORTED_SHAPE;
    if (budget > dst_width * page_size) return SK_ERR_INVALID_ARG;
    if (seqs == 0) return SK_OK;
    if (!cache || !table || !lens || !acc || !dst_table || !kept || !new_lens) return SK_ERR_INVALID_ARG;
    if ((long long)seqs * kv_heads > (1 << 24)) return SK_ERR_UNSUPPORTED_SHAPE;
    if (acc_out == acc || new_lens == lens) return SK_ERR_INVALID_ARG;
    if (!aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(acc, 4) || !aligned(dst_table, 4) ||
        !aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(acc_out, 4))
        return SK_ERR_MISALIGNED;
    EvictParams p = {};
    p.cache = cache;
    p.table = table;
    p.dst = dst_table;
    p.lens = lens;
    p.acc = acc;
    p.acc_out = acc_out;
    p.kept = kept;
    p.new_lens = new_lens;
    p.pages = pages;
    p.heads = kv_heads;
    p.recs = page_size / sk::KV4_REC;
    p.by_recs = sk::Div(p.recs);
    p.width = table_width;
    p.dst_width = dst_width;
    p.cap = table_width * page_size;
    p.dst_cap = dst_width * page_size;
    p.budget = budget;
    p.recent = recent;
    // CTAs per (sequence, head): as many as fill the GPU, at most a cluster
    // of 16, and no more than the longest table can feed with a position a thread.
    const int bh = seqs * kv_heads;
    sk::Scratch sc;                          // its error word, where the stream has a workspace
    if (sk::scratch_for(reinterpret_cast<cudaStream_t>(stream), &sc)) p.err = sc.err;
    int cluster = 1;
    while (cluster < MAX_CLUSTER && bh * cluster <= sk::device_sm_count() && cluster * ET < p.cap) cluster *= 2;
    p.stall = sk::take_inject_stall();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (head_dim) {
        case 64: return launch<64>(p, bh, cluster, s);
        case 128: return launch<128>(p, bh, cluster, s);
        default: return launch<256>(p, bh, cluster, s);
    }
}
