// logprobs.cu -- log probability and rank of a given token per row of logits,
// the row's entropy, and its most likely alternatives.
//
// With t_j = z_j / T, m = max t, S = sum exp(t_j - m):
//     logprob = t_tok - m - ln S,   entropy = ln S - sum exp(t_j - m) (t_j - m) / S,
//     rank    = 1 + #{j : z_j > z_tok, or z_j = z_tok and j < tok},
//     top     = the top_n largest z_j, ties to the lower j.
// 2^x and log2 are the hardware's approximations, and the sums FP32: a log
// probability is within 2^-16 where a thread adds up to 128 logits
// (tests/test_logprobs_error_gpu.py); measured against 64 bits 1e-7 relative for
// one to eight rows and 1.9e-7 for 2048 rows of 151936 (exp and log of FP32
// throughout: 0.7e-7 to 2.1e-7).
// One pass over the logits: every thread keeps a running maximum, sum and
// weighted sum (FP32), the count for the rank, and appends what may still be
// among the top_n to a list in shared memory.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/skinny.h"
#include "cluster.cuh"
#include "internal.h"
#include "launch_util.cuh"
#include "ptx.cuh"

namespace {

constexpr int NARROW = 64, WIDE = 256, WIDER = 512;   // threads per CTA (LT below)
constexpr int PER = 16;                  // logits per thread and round
constexpr int MAX_TOP = 64;
constexpr int SOFT = 160;                // the most candidates that a round may start with
constexpr int GROUPS = 64;               // groups of threads whose maxima bound the n-th largest
constexpr int MAX_CLUSTER = 16;
// Logits a row may have: indices run up to two rounds of the widest CTA past a
// row's end, and a row is cut in MAX_CLUSTER parts rounded up, all in 31 bits.
constexpr int MAX_N = 0x7FFF0000;
static_assert(0x7FFFFFFF - MAX_N > 2 * WIDER * PER + MAX_CLUSTER, "indices past a row's end");
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float LOWEST = -3.402823466e38f;

struct LogprobParams {
    const void *logits;
    long long stride;                    // elements between rows
    const int32_t *tokens;
    float *logprob, *entropy, *top_logprobs;
    int32_t *rank, *top_ids;
    float inv_t, inv_t2;                 // 1 / temperature, and times log2 e
    int N, top_n;
};

// max that hands on a NaN instead of dropping it
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float value_of(unsigned int k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// The value as a floor: everything passes one that is no number.
__device__ __forceinline__ float floor_of(unsigned int k) {
    const float v = value_of(k);
    return v == v ? v : -__builtin_huge_valf();
}
__device__ __forceinline__ unsigned long long cand_of(float v, int i) {
    return (static_cast<unsigned long long>(sk::key_of(v)) << 32) | static_cast<unsigned int>(~i);
}

// Running softmax statistics in units of log2: the maximum m of the raw logits
// and, against it, s = sum 2^d and w = sum 2^d d with d = (z - m) log2 e / T.
struct Stats {
    float m, s, w;
};
__device__ __forceinline__ Stats join(const Stats &a, const Stats &b, float c) {
    Stats r;
    r.m = fmaxf(a.m, b.m);
    const float da = max_nan((a.m - r.m) * c, -200.f), db = max_nan((b.m - r.m) * c, -200.f);
    const float fa = sk::ex2(da), fb = sk::ex2(db);
    r.s = a.s * fa + b.s * fb;
    r.w = fa * (a.w + da * a.s) + fb * (b.w + db * b.s);
    return r;
}

// Joined with lane ^ o's, the lower lane's first.
__device__ __forceinline__ Stats join_across(const Stats &a, int o, int lane, float c) {
    Stats x;
    x.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    x.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    x.w = __shfl_xor_sync(0xffffffffu, a.w, o);
    return (lane & o) ? join(x, a, c) : join(a, x, c);
}

// A CTA of few threads has a row to itself: it joins no cluster.
template <int LT>
struct Shared {
    unsigned long long list[SOFT + LT * PER + 2];         // a round can add all of its logits
    unsigned long long best[MAX_TOP];
    unsigned long long maxima[LT];
    alignas(16) unsigned int top[GROUPS];
    unsigned long long all_best[LT == NARROW ? 1 : MAX_CLUSTER * MAX_TOP];
    Stats stats[LT / 32];
    Stats mine, all;
    unsigned int above[LT / 32];
    unsigned int above_mine, above_all;  // logits that rank before the token
    unsigned int place[MAX_TOP];
    int count, kept;
    float zfloor;
    unsigned long long floor;
};

// The `n` largest of sh.list[0 .. count) in descending order into sh.best, by
// counting for each how many are larger (the entries differ: each holds its
// index).  With many candidates, those below the n-th largest of the threads'
// maxima go first: at least n are at or above it.
template <int LT>
__device__ __forceinline__ void pick_best(Shared<LT> &sh, int count, int n) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (count > 2 * LT) {
        unsigned long long mx = 0;
        for (int i = tid; i < count; i += LT) mx = sh.list[i] > mx ? sh.list[i] : mx;
        sh.maxima[tid] = mx;
        if (tid == 0) sh.kept = 0;
        __syncthreads();
        int larger = 0;
        for (int j = 0; j < LT; ++j) larger += sh.maxima[j] > mx;
        if (larger == n - 1) sh.floor = mx;
        __syncthreads();
        const unsigned long long lim = sh.floor;
        // in place, a stretch at a time: kept entries never overtake the reads
        for (int i0 = 0; i0 < count; i0 += LT) {
            const unsigned long long v = i0 + tid < count ? sh.list[i0 + tid] : 0ull;
            __syncthreads();
            if (i0 + tid < count && v >= lim) sh.list[atomicAdd(&sh.kept, 1)] = v;
            __syncthreads();
        }
        count = sh.kept;
    }
    if (tid == 0 && (count & 1)) sh.list[count] = 0ull;     // read in pairs
    __syncthreads();
    for (int i = tid; i < count; i += LT) {
        const unsigned long long v = sh.list[i];
        int larger = 0;
#pragma unroll 4
        for (int j = 0; j < count; j += 2) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sh.list[j]);
            larger += (w.x > v) + (w.y > v);
        }
        if (larger < n) sh.best[larger] = v;
    }
    for (int i = count + tid; i < n; i += LT) sh.best[i] = 0ull;
    __syncthreads();
}

// Sixteen logits of a thread as loaded: NV words of 16 bytes, the v-th holding
// logits i0 + (v LT + tid) VEC and on.
template <typename T, int LT>
struct Raw {
    static constexpr int VEC = 16 / int(sizeof(T)), NV = PER / VEC, ROUND = LT * PER;
    uint4 w[NV];

    // whole: all of the round's logits belong to [lo, hi); the others are read
    // as minus infinity
    __device__ __forceinline__ void load(const T *z, int i0, int lo, int hi) {
        const int tid = threadIdx.x;
        if (i0 >= lo && i0 + ROUND <= hi) {
#pragma unroll
            for (int v = 0; v < NV; ++v) w[v] = __ldcs(reinterpret_cast<const uint4 *>(z + i0 + (v * LT + tid) * VEC));
            return;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int at = i0 + (v * LT + tid) * VEC;
            if (at >= lo && at + VEC <= hi) {
                w[v] = __ldcs(reinterpret_cast<const uint4 *>(z + at));
            } else {
                uint32_t x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (sizeof(T) == 4) {
                        x[q] = at + q >= lo && at + q < hi ? *reinterpret_cast<const uint32_t *>(z + at + q) : 0xFF800000u;
                    } else {
                        uint32_t h[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            h[e] = at + 2 * q + e >= lo && at + 2 * q + e < hi
                                       ? *reinterpret_cast<const uint16_t *>(z + at + 2 * q + e)
                                       : 0xFC00u;
                        x[q] = h[0] | (h[1] << 16);
                    }
                }
                w[v] = make_uint4(x[0], x[1], x[2], x[3]);
            }
        }
    }
    __device__ __forceinline__ void values(float (&z)[PER]) const {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t x[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (sizeof(T) == 4) {
                    z[v * 4 + q] = __uint_as_float(x[q]);
                } else {
                    const float2 f = sk::f16x2_to_f32x2(x[q]);
                    z[v * 8 + 2 * q] = f.x;
                    z[v * 8 + 2 * q + 1] = f.y;
                }
            }
        }
    }
};

__device__ __forceinline__ float one(const float *p) { return *p; }
__device__ __forceinline__ float one(const __half *p) { return __half2float(*p); }

// One cluster per row (a single CTA where the rows alone fill the GPU); CTA r
// takes the r-th contiguous part of the row, a round of 16 logits a thread at
// a time, the next round's loads in flight while one is summed.  Many long
// rows are bound by the reads (2048 of 151936, FP32, top 20: 220 us, 5.7 TB/s);
// few or short ones by the latency of a read, the cut of the candidates and
// the exchange in the cluster (one row of 151936, top 5: 8.4 us).
template <typename T, int LT>
__global__ void __launch_bounds__(LT) logprobs_kernel(const __grid_constant__ LogprobParams p, int first_row, int late) {
    extern __shared__ __align__(16) unsigned char raw_smem[];
    Shared<LT> &sh = *reinterpret_cast<Shared<LT> *>(raw_smem);
    constexpr int VEC = Raw<T, LT>::VEC, ROUND = LT * PER;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const unsigned int rank = LT == NARROW ? 0u : sk::cluster_rank(), C = LT == NARROW ? 1u : sk::cluster_size();
    const int row = first_row + blockIdx.x / C;
    // The first of two launches lets the second start once all of its own CTAs
    // are past their wait, so what the logits depend on is complete; the second
    // (late) waits at its end, so that whatever follows it follows both.
    if (!late) sk::pdl_wait_primary();
    sk::pdl_launch_dependents();
    const T *z0 = static_cast<const T *>(p.logits) + (long long)row * p.stride;
    // this CTA's part, and the 16-byte boundary at or below its first logit
    const int part = (p.N + int(C) - 1) / int(C);
    const int lo = min(p.N, int(rank) * part), hi = min(p.N, lo + part);
    const int first = lo - int((reinterpret_cast<uintptr_t>(z0 + lo) & 15u) / sizeof(T));
    Raw<T, LT> next;
    next.load(z0, first, lo, hi);
    const int tok = p.tokens ? p.tokens[row] : -1;
    const bool given = tok >= 0 && tok < p.N;
    const float ztok = given ? one(z0 + tok) : 0.f, zrank = given ? ztok : __builtin_huge_valf();
    const float ztok_up = value_of(sk::key_of(ztok) + 1u);       // the next larger value
    const bool masked_token = ztok == -__builtin_huge_valf();
    const float c = p.inv_t2;
    const int n = min(p.top_n, p.N);
    // Candidates that trigger a cut after a round: few in a long part, so that
    // the floor keeps up with what has been seen (2048 rows of 151936, top 20:
    // 222 us, 237 us at 192 candidates); short parts end before that pays.
    const int soft = hi - lo > 8 * ROUND ? 2 * n + 24 : SOFT;
    static_assert(2 * MAX_TOP + 24 < SOFT, "the list holds them and a round");
    if (tid == 0) sh.count = 0;
    if (tid < MAX_TOP) sh.place[tid] = 0u;
    static_assert(LT >= MAX_TOP && LT >= GROUPS, "a thread a place, and a group's threads");

    Stats st = {LOWEST, 0.f, 0.f};
    unsigned int above = 0;
    // a candidate is at least zfloor, and its key exceeds `floor`
    float zfloor = n > 0 ? -__builtin_huge_valf() : __builtin_huge_valf();
    unsigned long long floor = 0ull;
    for (int i0 = first; i0 < hi; i0 += ROUND) {
        float z[PER];
        next.values(z);
        if (i0 + ROUND < hi) next.load(z0, i0 + ROUND, lo, hi);
        float mx = z[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) mx = fmaxf(mx, z[j]);
        if (mx > st.m) {
            const float d = max_nan((st.m - mx) * c, -200.f), f = sk::ex2(d);
            st.w = f * (st.w + d * st.s);
            st.s *= f;
            st.m = mx;
        }
        // 2^-200 is zero in FP32, so a logit of minus infinity (or the type's
        // lowest value) adds nothing, and nothing times -200 to the second sum
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const float d = max_nan((z[j] - st.m) * c, -200.f), e = sk::ex2(d);
            st.s += e;
            st.w = fmaf(e, d, st.w);
        }
        if (n > 0 && i0 == first) {
            // The n-th largest of the maxima of 64 groups of threads bounds
            // the n-th largest logit from below (the last byte holds the
            // group, so that they differ: at most a little lower).
            float gm = mx;
#pragma unroll
            for (int o = 1; o < LT / GROUPS; o <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
            if (tid % (LT / GROUPS) == 0)
                sh.top[tid / (LT / GROUPS)] = (sk::key_of(gm) & ~255u) | unsigned(GROUPS - 1 - tid / (LT / GROUPS));
            __syncthreads();
            if (wid == 0) {
                const unsigned int k0 = sh.top[lane], k1 = sh.top[lane + 32];
                int l0 = 0, l1 = 0;
#pragma unroll
                for (int j = 0; j < GROUPS; j += 4) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(&sh.top[j]);
                    l0 += (w.x > k0) + (w.y > k0) + (w.z > k0) + (w.w > k0);
                    l1 += (w.x > k1) + (w.y > k1) + (w.z > k1) + (w.w > k1);
                }
                if (l0 == n - 1) sh.zfloor = floor_of(k0 & ~255u);
                if (l1 == n - 1) sh.zfloor = floor_of(k1 & ~255u);
            }
            __syncthreads();
            zfloor = sh.zfloor;
        }
        // Four logits at a time that hold one to look at: at least the token's
        // (for the rank), or at least the floor (for the list).
        bool full = false;
        const float least = fminf(zfloor, zrank);
        if (!(mx < least)) {
#pragma unroll
            for (int q = 0; q < PER; q += 4) {
                const float most = fmaxf(fmaxf(z[q], z[q + 1]), fmaxf(z[q + 2], z[q + 3]));
                if (most < least) continue;
                const int at = i0 + ((q / VEC) * LT + tid) * VEC + q % VEC;
                if (!(most < zrank)) {
                    // logits before the token rank above it when they are at
                    // least its own, those after it when they exceed it
                    if (masked_token || (at < tok && tok < at + 4)) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            above += at + j >= lo && at + j < hi && (z[q + j] > ztok || (z[q + j] == ztok && at + j < tok));
                    } else {
                        const float t = at < tok ? ztok : ztok_up;
#pragma unroll
                        for (int j = 0; j < 4; ++j) above += z[q + j] >= t;
                    }
                }
                if (n == 0 || most < zfloor) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!(z[q + j] < zfloor)) {
                        const unsigned long long k = cand_of(z[q + j], at + j);
                        if (k > floor && at + j >= lo && at + j < hi) {
                            const int to = atomicAdd(&sh.count, 1);
                            sh.list[to] = k;
                            full |= to >= soft;
                        }
                    }
            }
        }
        if (n > 0) {
            if (__syncthreads_or(full)) {
                pick_best<LT>(sh, sh.count, n);
                for (int i = tid; i < n; i += LT) sh.list[i] = sh.best[i];
                if (tid == 0) sh.count = n;
                floor = sh.best[n - 1];
                zfloor = floor_of(static_cast<unsigned int>(floor >> 32));
                __syncthreads();
            }
        }
    }

    // ---- the CTA's statistics and candidates, in a fixed order
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        st = join_across(st, o, lane, c);
        above += __shfl_xor_sync(0xffffffffu, above, o);
    }
    if (lane == 0) {
        sh.stats[wid] = st;
        sh.above[wid] = above;
    }
    __syncthreads();
    if (n > 0) pick_best<LT>(sh, sh.count, n);
    if (wid == 0) {
        Stats a = lane < LT / 32 ? sh.stats[lane] : Stats{LOWEST, 0.f, 0.f};
        unsigned int r = lane < LT / 32 ? sh.above[lane] : 0u;
#pragma unroll
        for (int o = 1; o < LT / 32; o <<= 1) {
            a = join_across(a, o, lane, c);
            r += __shfl_xor_sync(0xffffffffu, r, o);
        }
        if (lane == 0) {
            sh.mine = a;
            sh.above_mine = r;
            if (C == 1) {
                sh.all = a;
                sh.above_all = r;
            }
        }
    }
    // ---- the cluster's: every CTA joins all the statistics, and places its
    // own candidates among everyone's
    if (C > 1) {
        sk::cluster_sync();
        if (wid == 0) {
            Stats a = {LOWEST, 0.f, 0.f};
            unsigned int r = 0u;
            if (unsigned(lane) < C) {
                const uint32_t q = sk::peer(&sh.mine, unsigned(lane));
                a = Stats{sk::ld_peer_f32(q), sk::ld_peer_f32(q + 4), sk::ld_peer_f32(q + 8)};
                r = __float_as_uint(sk::ld_peer_f32(sk::peer(&sh.above_mine, unsigned(lane))));
            }
#pragma unroll
            for (int o = 1; o < MAX_CLUSTER; o <<= 1) {
                a = join_across(a, o, lane, c);
                r += __shfl_xor_sync(0xffffffffu, r, o);
            }
            if (lane == 0) {
                sh.all = a;
                sh.above_all = r;
            }
        }
        // everyone's entries, then entry e of this CTA against the sorted entries of CTA k, both by thread
        for (int x = tid; x < int(C) * n; x += LT) {
            const int k = x / n;
            sh.all_best[x] = sk::ld_peer_u64(sk::peer(&sh.best[x - k * n], unsigned(k)));
        }
        __syncthreads();
        for (int x = tid; x < int(C) * n; x += LT) {
            const int k = x / n, e = x - k * n;
            if (unsigned(k) == rank) continue;
            const unsigned long long v = sh.best[e];
            const unsigned long long *theirs = sh.all_best + k * n;
            int a = 0, b = n;                    // entries [0, a) are larger, [b, n) are not
            while (a < b) {
                const int h = (a + b) >> 1;
                if (theirs[h] > v) a = h + 1;
                else b = h;
            }
            if (a) atomicAdd(&sh.place[e], unsigned(a));
        }
        sk::cluster_sync();                          // and no CTA leaves while its entries are read
    }
    __syncthreads();
    const Stats a = sh.all;
    // A row of nothing but minus infinity has no distribution: minus infinity
    // for every log probability, no entropy.
    const bool none = a.s == 0.f;
    const float lg = __log2f(a.s);
    auto logprob = [&](float z) { return none ? -__builtin_huge_valf() : fmaf(z - a.m, p.inv_t, -lg * LN2); };
    if (rank == 0 && tid == 0) {
        if (p.logprob) p.logprob[row] = given ? logprob(ztok) : 0.f;
        if (p.rank) p.rank[row] = given ? int32_t(1u + sh.above_all) : 0;
        if (p.entropy) p.entropy[row] = none ? 0.f : (lg - a.w / a.s) * LN2;
    }
    for (int e = tid; e < n; e += LT) {
        const unsigned long long k = sh.best[e];
        const int at = e + int(sh.place[e]);
        if (k != 0ull && at < n) {
            p.top_ids[(long long)row * p.top_n + at] = int32_t(~static_cast<unsigned int>(k));
            p.top_logprobs[(long long)row * p.top_n + at] = logprob(value_of(static_cast<unsigned int>(k >> 32)));
        }
    }
    if (late) sk::pdl_wait_primary();
    if (rank == 0)
        for (int e = n + tid; e < p.top_n; e += LT) {
            p.top_ids[(long long)row * p.top_n + e] = -1;
            p.top_logprobs[(long long)row * p.top_n + e] = -__builtin_huge_valf();
        }
}

template <typename T, int LT>
cudaError_t launch(const LogprobParams &p, int first_row, int rows, int cluster, bool late, cudaStream_t s) {
    const cudaError_t e = sk::prepare_kernel<logprobs_kernel<T, LT>>(sizeof(Shared<LT>), LT != NARROW);
    if (e != cudaSuccess) return e;
    return sk::launch_pdl_cluster(logprobs_kernel<T, LT>, cluster, dim3(unsigned(rows) * unsigned(cluster)), dim3(LT),
                                  sizeof(Shared<LT>), s, p, first_row, int(late));
}

// CTAs that run at a time, four to an SM (64 registers a thread).
constexpr int PER_SM = 4;

template <typename T>
sk_status run(const LogprobParams &p, int rows, cudaStream_t s) {
    const int slots = PER_SM * (sk::device_sm_count() > 0 ? sk::device_sm_count() : 1);
    // Short rows: a CTA of 64 threads for each, where one round holds the row,
    // or where two do and the rows exceed the wide CTAs that run at a time.
    // (2048 rows of 300, FP32, top 20: 11 us, 58 with wide CTAs, whose idle
    // threads leave no floor to the candidates; 1000 of 2000: 10.4 and 12.6;
    // one row of 1000: 5.7 and 5.1; 300 of 2000: 8.8 and 6.0.)
    if (p.N <= (rows > slots ? 2 : 1) * NARROW * PER)
        return launch<T, NARROW>(p, 0, rows, 1, false, s) == cudaSuccess ? SK_OK : SK_ERR_CUDA;
    // CTAs per row: what fits, each with a round or more to read.
    constexpr int ROUND = WIDE * PER;
    auto split = [&](int r) {
        int c = 1;
        while (c < MAX_CLUSTER && r * c * 2 <= slots && c * ROUND < p.N) c *= 2;
        return c;
    };
    // Whole waves of one CTA per row, and what is left over split across the
    // CTAs that fit, so that the last wave is short: 2048 rows of 151936 are
    // 3.4 waves of 608 (measured: 265 us in one launch, 255 us in two).
    const int left = rows > slots ? rows % slots : rows, cluster = split(left);
    cudaError_t e;
    if (rows * cluster <= slots / PER_SM && p.N > 2 * cluster * ROUND) {
        // Few rows of more than two rounds a CTA, an SM to each: twice the
        // threads, and the rounds' reads are in flight together (rows of
        // 151936, FP32, top 20: one 10.6 -> 9.1 us, four 11.4 -> 9.3, eight
        // 12.3 -> 11.6; of 32000, one round each, 7.3 -> 7.7 were they to take
        // it).  With 1024 threads one row takes 10.5.
        e = launch<T, WIDER>(p, 0, rows, cluster, false, s);
    } else if (rows <= slots || cluster == 1) {
        e = launch<T, WIDE>(p, 0, rows, rows <= slots ? cluster : 1, false, s);
    } else {
        e = launch<T, WIDE>(p, 0, rows - left, 1, false, s);
        if (e == cudaSuccess && left) e = launch<T, WIDE>(p, rows - left, left, cluster, sk::pdl_enabled(), s);
    }
    return e == cudaSuccess ? SK_OK : SK_ERR_CUDA;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" sk_status token_logprobs(const void *logits, int f16, long long row_stride, const int32_t *tokens,
                                    float temperature, int top_n, float *logprob, int32_t *rank, float *entropy,
                                    int32_t *top_ids, float *top_logprobs, int rows, int N, void *stream) {
    if (rows < 0 || N < 1 || top_n < 0 || (f16 != 0 && f16 != 1) || row_stride < N) return SK_ERR_INVALID_ARG;
    if (!(temperature >= 1e-6f && temperature <= 1e6f)) return SK_ERR_INVALID_ARG;
    if (top_n > MAX_TOP || rows > (1 << 26) || N > MAX_N) return SK_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return SK_OK;
    if (!logits || (top_n > 0 && (!top_ids || !top_logprobs))) return SK_ERR_INVALID_ARG;
    if (!tokens && (logprob || rank)) return SK_ERR_INVALID_ARG;
    if (!aligned(logits, f16 ? 2 : 4) || !aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(rank, 4) ||
        !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return SK_ERR_MISALIGNED;
    LogprobParams p = {};
    p.logits = logits;
    p.stride = row_stride;
    p.tokens = tokens;
    p.logprob = logprob;
    p.rank = rank;
    p.entropy = entropy;
    p.top_ids = top_ids;
    p.top_logprobs = top_logprobs;
    p.inv_t = 1.f / temperature;
    p.inv_t2 = LOG2E / temperature;
    p.N = N;
    p.top_n = top_n;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return f16 ? run<__half>(p, rows, s) : run<float>(p, rows, s);
}
