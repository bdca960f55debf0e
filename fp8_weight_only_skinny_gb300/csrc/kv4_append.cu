// kv4_append.cu -- keys and values of new tokens, FP16 -> records of the 4-bit
// cache (kv4.cuh), each 16-component block by the rounding steps of the
// weight quantizer (quant.cuh) under a scale the caller fixes.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/skinny.h"
#include "internal.h"
#include "kv4.cuh"
#include "launch_util.cuh"
#include "quant.cuh"

namespace {

constexpr int AT = 256;

struct AppendParams {
    const __half *src[2];      // keys, values
    long long stride[2];       // elements between tokens
    __half *held[2];           // [T][H][D] or null
    float g[2];
    const int32_t *slots;
    uint8_t *cache;
    long long tokens;
    int pages, heads, recs, page;   // recs: records per page
    int hb;                    // blocks per token: heads * D / 16
    int hb_groups;             // ceil(hb / 8)
};

// A warp takes four tokens x eight blocks: lane = block-in-group * 4 + token,
// so that four neighbouring positions of a value block (32 bytes of a record)
// are written by neighbouring lanes, and a token's eight blocks are 256
// contiguous bytes read.  blockIdx.y: 0 keys, 1 values.  Bound by DRAM and the
// rounding's instructions together: 32771 tokens of 4 heads of 128 with the
// held values, 31 us (153 MB, 5.0 TB/s); a single token 1.8 us.  (Two groups of
// four tokens a warp took 31.9, a rounding of a sixth fewer instructions 31.0:
// neither alone is the limit.)
template <int D, bool VALUE>
__device__ __forceinline__ void append_block(const AppendParams &p) {
    constexpr int NB = D / 16;
    const long long w = (long long)blockIdx.x * (AT / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int grp = int(w % p.hb_groups);
    const long long t = (w / p.hb_groups) * 4 + (lane & 3);
    const int hb = grp * 8 + (lane >> 2);
    if (t >= p.tokens || hb >= p.hb) return;
    const int slot = p.slots[t];
    const uint4 *src = reinterpret_cast<const uint4 *>(p.src[VALUE] + t * p.stride[VALUE] + hb * 16);
    const uint4 v0 = src[0], v1 = src[1];
    uint2 codes;
    const float G = p.g[VALUE];
    const uint32_t sc = sk::encode_block(v0, v1, G, codes);
    if (p.held[VALUE]) {
        // code * S is exact in FP16; times G in FP32, rounded once to FP16
        uint32_t h[8], out[8];
        uint32_t (&lo)[4] = *reinterpret_cast<uint32_t (*)[4]>(&h[0]);
        uint32_t (&hi)[4] = *reinterpret_cast<uint32_t (*)[4]>(&h[4]);
        sk::e2m1x8_to_f16x2x4(codes.x, lo);
        sk::e2m1x8_to_f16x2x4(codes.y, hi);
        const float S = sk::e4m3_value(sc);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = sk::f16x2_to_f32x2(h[i]);
            const __half2 r = __floats2half2_rn(__fmul_rn(f.x * S, G), __fmul_rn(f.y * S, G));
            out[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(p.held[VALUE] + (t * p.hb + hb) * 16);
        dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
        dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
    const int page = slot / p.page;
    if (slot < 0 || page >= p.pages) return;
    const int at = slot - page * p.page, head = hb / NB, b = hb - head * NB, i = at & 15;
    uint8_t *rec = p.cache + ((size_t(page) * p.heads + head) * p.recs + (at >> 4)) * sk::kv4_rec_bytes(D);
    *reinterpret_cast<uint2 *>(rec + sk::kv4_code_at<VALUE>(D, i, b)) = codes;
    rec[sk::kv4_scale_at<VALUE>(D, i, b)] = uint8_t(sc);
}

template <int D>
__global__ void __launch_bounds__(AT) kv4_append_kernel(const __grid_constant__ AppendParams p) {
    sk::pdl_wait_primary();
    if (blockIdx.y == 0) append_block<D, false>(p);
    else append_block<D, true>(p);
}

template <int D>
sk_status launch(const AppendParams &p, cudaStream_t s) {
    const long long warps = (p.tokens + 3) / 4 * p.hb_groups;
    const long long grid = (warps + AT / 32 - 1) / (AT / 32);
    if (grid > 0x7FFFFFFFLL) return SK_ERR_UNSUPPORTED_SHAPE;
    return sk::launch_pdl(kv4_append_kernel<D>, dim3(unsigned(grid), 2), dim3(AT), 0, s, p) == cudaSuccess
               ? SK_OK
               : SK_ERR_CUDA;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" sk_status kv4_append(const void *k, long long k_stride, const void *v, long long v_stride,
                                const int32_t *slots, uint8_t *cache, float k_scale, float v_scale, void *k_held,
                                void *v_held, int tokens, int pages, int kv_heads, int head_dim, int page_size,
                                void *stream) {
    if (tokens < 0 || pages < 1 || kv_heads < 1 || page_size < 1) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_scale_ok(k_scale) || !sk::kv4_scale_ok(v_scale)) return SK_ERR_INVALID_ARG;
    if (!sk::kv4_shape_ok(pages, kv_heads, head_dim, page_size)) return SK_ERR_UNSUPPORTED_SHAPE;
    if (tokens == 0) return SK_OK;
    if (!k || !v || !slots || !cache || (!k_held != !v_held)) return SK_ERR_INVALID_ARG;
    const long long row = (long long)kv_heads * head_dim;
    if (k_stride < row || v_stride < row) return SK_ERR_INVALID_ARG;
    if (k_stride % 8 || v_stride % 8 || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) ||
        !aligned(cache, 16) || !aligned(k_held, 16) || !aligned(v_held, 16))
        return SK_ERR_MISALIGNED;
    AppendParams p = {};
    p.src[0] = static_cast<const __half *>(k);
    p.src[1] = static_cast<const __half *>(v);
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.held[0] = static_cast<__half *>(k_held);
    p.held[1] = static_cast<__half *>(v_held);
    p.g[0] = k_scale;
    p.g[1] = v_scale;
    p.slots = slots;
    p.cache = cache;
    p.tokens = tokens;
    p.pages = pages;
    p.heads = kv_heads;
    p.page = page_size;
    p.recs = page_size / sk::KV4_REC;
    p.hb = int(row / 16);
    p.hb_groups = (p.hb + 7) / 8;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (head_dim) {
        case 64: return launch<64>(p, s);
        case 128: return launch<128>(p, s);
        default: return launch<256>(p, s);
    }
}
