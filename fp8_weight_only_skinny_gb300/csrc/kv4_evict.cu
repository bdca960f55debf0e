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
#include "internal.h"
#include "kv4.cuh"
#include "launch_util.cuh"

namespace {

constexpr int ET = 512;            // threads per CTA
constexpr int CHUNK = ET * 4;      // positions scanned at a time
constexpr int MAX_CLUSTER = 16;

struct EvictParams {
    uint8_t *cache;
    const int32_t *table, *dst, *lens;
    const float *acc;
    float *acc_out;
    int32_t *kept, *new_lens;
    int pages, heads, recs, width, dst_width, cap, dst_cap;
    int budget, recent;
    sk::Div by_recs;
};

// Order of the weights as unsigned keys (larger weight, larger key; -0 = +0).
__device__ __forceinline__ unsigned int key_of(float v) {
    const unsigned int u = __float_as_uint(v + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ unsigned int cluster_rank() {
    unsigned int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned int cluster_size() {
    unsigned int r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned int ld_peer(const unsigned int *p, unsigned int rank) {
    const uint32_t a = sk::smem_u32(p);
    unsigned int v;
    asm volatile("{ .reg .b32 r; mapa.shared::cluster.u32 r, %1, %2; ld.shared::cluster.u32 %0, [r]; }"
                 : "=r"(v) : "r"(a), "r"(rank) : "memory");
    return v;
}

// Exclusive prefix sum over the CTA in thread order of two counts packed as
// (high << 16 | low), each total below 65536; *total gets the sum.
__device__ __forceinline__ unsigned int scan2(unsigned int v, unsigned int *tmp, unsigned int *total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    unsigned int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) tmp[wid] = x;
    __syncthreads();
    unsigned int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < ET / 32; ++w) {
        if (w < wid) before += tmp[w];
        all += tmp[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// Copy m positions (from[x] -> to[x], each the address of a record plus the
// position in it).  A lane always moves the same piece: eight code bytes of a
// block, or its scale byte; a warp moves 32 / PIECES positions (D = 256: half
// of one) at a time, eight in flight.
template <int D>
__device__ __forceinline__ void copy_rows(uint8_t *const *from, uint8_t *const *to, int m) {
    constexpr int NB = D / 16, PIECES = 4 * NB;
    const int piece = threadIdx.x % PIECES, blk = piece % NB, what = piece / NB;
    constexpr int STRIDE = ET / PIECES, FLIGHT = 8;
    auto at = [&](const uint8_t *r) {
        const int i = int(reinterpret_cast<uintptr_t>(r) & 15u);
        const int off = what == 0   ? sk::kv4_code_at<false>(D, i, blk)
                        : what == 1 ? sk::kv4_code_at<true>(D, i, blk)
                        : what == 2 ? sk::kv4_scale_at<false>(D, i, blk)
                                    : sk::kv4_scale_at<true>(D, i, blk);
        return off - i;
    };
    for (int x0 = threadIdx.x / PIECES; x0 < m; x0 += STRIDE * FLIGHT) {
        uint2 v[FLIGHT];
#pragma unroll
        for (int f = 0; f < FLIGHT; ++f) {
            const int x = x0 + f * STRIDE;
            if (x < m) {
                const uint8_t *s = from[x];
                s += at(s);
                if (what < 2) v[f] = *reinterpret_cast<const uint2 *>(s);
                else v[f].x = *s;
            }
        }
#pragma unroll
        for (int f = 0; f < FLIGHT; ++f) {
            const int x = x0 + f * STRIDE;
            if (x < m) {
                uint8_t *d = to[x];
                d += at(d);
                if (what < 2) *reinterpret_cast<uint2 *>(d) = v[f];
                else *d = uint8_t(v[f].x);
            }
        }
    }
}

// One cluster per (sequence, kv head); CTA r takes the r-th contiguous part of
// the positions.  Selection is a radix select over the ordered weights, eight
// bits a pass, on histograms summed over the cluster through distributed
// shared memory; the kept positions of a chunk are then numbered by a scan and
// their codes and scales copied.
template <int D>
__global__ void __launch_bounds__(ET) kv4_evict_kernel(const __grid_constant__ EvictParams p) {
    __shared__ unsigned int hist[2][256];
    __shared__ unsigned int tot[256];
    __shared__ unsigned int counts[2];           // this CTA's keys above / equal to the threshold
    __shared__ unsigned int tmp[ET / 32];
    __shared__ unsigned int s_prefix, s_need;
    __shared__ int src_pos[CHUNK];
    __shared__ uint8_t *from_rec[CHUNK], *to_rec[CHUNK];
    sk::pdl_launch_dependents();
    sk::pdl_wait_primary();
    const int tid = threadIdx.x, lane = tid & 31;
    const unsigned int rank = cluster_rank(), C = cluster_size();
    const int bh = blockIdx.x / C, b = bh / p.heads, h = bh - b * p.heads;
    const int n = min(max(p.lens[b], 0), p.cap);
    const int out_n = min(n, p.budget);
    const float *acc = p.acc + size_t(bh) * size_t(p.cap);
    const bool all = n <= p.budget;
    const int old = all ? n : n - p.recent;      // positions the selection decides on
    const int part = (n + int(C) - 1) / int(C);
    const int lo = min(n, int(rank) * part), hi = min(n, lo + part);
    const int lo_old = min(lo, old), hi_old = min(hi, old);

    // ---- threshold: the (budget - recent)-th largest key of the old positions
    unsigned int prefix = 0, mask = 0, need = all ? 0u : unsigned(p.budget - p.recent);
    if (!all && need > 0) {
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            unsigned int *hh = hist[pass & 1];
            if (tid < 256) hh[tid] = 0u;
            __syncthreads();
            for (int i = lo_old + tid; i < hi_old; i += ET) {
                const unsigned int k = key_of(acc[i]);
                if ((k & mask) == prefix) atomicAdd(&hh[(k >> shift) & 255u], 1u);
            }
            cluster_sync();
            if (tid < 256) {
                unsigned int t = 0;
                for (unsigned int r = 0; r < C; ++r) t += ld_peer(hh + tid, r);
                tot[tid] = t;
            }
            __syncthreads();
            if (tid < 32) {
                // lane l takes bins 255 - 8 l down; suffix sums from the top
                unsigned int mine = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) mine += tot[255 - (8 * lane + j)];
                unsigned int x = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                unsigned int above = x - mine;
                if (above < need && x >= need) {
                    int bin = 255 - 8 * lane;
                    while (above + tot[bin] < need) above += tot[bin--];
                    s_prefix = prefix | (unsigned(bin) << shift);
                    s_need = need - above;
                }
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
            mask |= 255u << shift;
        }
    }
    // kept: keys above `prefix`, and the first `need` equal to it; none of the old when need was 0
    const bool none_old = !all && p.budget == p.recent;
    auto kind = [&](int i) -> unsigned int {     // 2: kept for sure, 1: kept if among the first equal ones
        if (all || i >= old) return 2u;
        if (none_old) return 0u;
        const unsigned int k = key_of(acc[i]);
        return k > prefix ? 2u : k == prefix ? 1u : 0u;
    };
    unsigned int gt = 0, eq = 0;
    for (int i = lo + tid; i < hi; i += ET) {
        const unsigned int k = kind(i);
        gt += k == 2u;
        eq += k == 1u;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        gt += __shfl_xor_sync(0xffffffffu, gt, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (tid < 2) counts[tid] = 0u;
    __syncthreads();
    if (lane == 0) {
        atomicAdd(&counts[0], gt);
        atomicAdd(&counts[1], eq);
    }
    cluster_sync();
    unsigned int gt_before = 0, eq_before = 0;
    for (unsigned int r = 0; r < rank; ++r) {
        gt_before += ld_peer(&counts[0], r);
        eq_before += ld_peer(&counts[1], r);
    }
    cluster_sync();                              // no CTA leaves while its counts are read

    // ---- number the kept positions in order and copy them
    const int32_t *table = p.table + size_t(b) * p.width;
    const int32_t *dtable = p.dst + size_t(b) * p.dst_width;
    int32_t *kept = p.kept + size_t(bh) * size_t(p.budget);
    float *acc_out = p.acc_out ? p.acc_out + size_t(bh) * size_t(p.dst_cap) : nullptr;
    for (int c0 = lo; c0 < hi; c0 += CHUNK) {
        unsigned int k4[4], v = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = c0 + tid * 4 + j;
            k4[j] = i < hi ? kind(i) : 0u;
            v += k4[j] == 2u ? 0x10000u : k4[j] == 1u ? 1u : 0u;
        }
        unsigned int total;
        const unsigned int ex = scan2(v, tmp, &total);
        unsigned int g = gt_before + (ex >> 16), e = eq_before + (ex & 0xFFFFu);
        const unsigned int j0 = gt_before + min(eq_before, need);          // slot of the chunk's first kept position
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (k4[j] == 2u || (k4[j] == 1u && e < need)) src_pos[g + min(e, need) - j0] = c0 + tid * 4 + j;
            g += k4[j] == 2u;
            e += k4[j] == 1u;
        }
        gt_before += total >> 16;
        eq_before += total & 0xFFFFu;
        const int m = int(gt_before + min(eq_before, need) - j0);
        __syncthreads();
        for (int x = tid; x < m; x += ET) {
            const int sp = src_pos[x], dp = int(j0) + x;
            kept[dp] = sp;
            if (acc_out) acc_out[dp] = acc[sp];
            from_rec[x] = p.cache + size_t(sk::kv4_record(table, sp >> 4, p.recs, p.by_recs, p.pages, p.heads, h)) * sk::kv4_rec_bytes(D) + (sp & 15);
            to_rec[x] = p.cache + size_t(sk::kv4_record(dtable, dp >> 4, p.recs, p.by_recs, p.pages, p.heads, h)) * sk::kv4_rec_bytes(D) + (dp & 15);
        }
        __syncthreads();
        // records start at multiples of 16: the low bits hold the position in one
        copy_rows<D>(from_rec, to_rec, m);
        __syncthreads();
    }
    for (int j = out_n + int(rank) * ET + tid; j < p.budget; j += int(C) * ET) kept[j] = -1;
    if (acc_out)
        for (int j = out_n + int(rank) * ET + tid; j < p.dst_cap; j += int(C) * ET) acc_out[j] = 0.f;
    if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = out_n;
}

template <int D>
sk_status launch(const EvictParams &p, int bh, int cluster, cudaStream_t s) {
    if (sk::prepare_kernel<kv4_evict_kernel<D>>(0, true) != cudaSuccess) return SK_ERR_CUDA;
    return sk::launch_pdl_cluster(kv4_evict_kernel<D>, cluster, dim3(unsigned(bh) * unsigned(cluster)), dim3(ET), 0, s,
                                  p) == cudaSuccess
               ? SK_OK
               : SK_ERR_CUDA;
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
    // of 16, and no more than the longest table can feed with a chunk each.
    const int bh = seqs * kv_heads;
    int cluster = 1;
    while (cluster < MAX_CLUSTER && bh * cluster < sk::device_sm_count() && cluster * (CHUNK / 4) < p.cap) cluster *= 2;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (head_dim) {
        case 64: return launch<64>(p, bh, cluster, s);
        case 128: return launch<128>(p, bh, cluster, s);
        default: return launch<256>(p, bh, cluster, s);
    }
}
