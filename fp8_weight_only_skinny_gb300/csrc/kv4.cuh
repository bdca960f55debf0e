// kv4.cuh -- the paged key/value cache held in 4 bits: its record layout and
// the device helpers its kernels share (kv4_append.cu, kv4_attention.cu,
// kv4_evict.cu).
//
// The cache is u8 [pages][kv_heads][page_size / 16][18 D]: one record of 18 D
// bytes holds the keys and values of 16 consecutive positions of one head of
// size D, so that a reader fetches it with a single bulk copy and, a page's
// records of a head being contiguous, streams whole DRAM pages.  In a record:
//
//   [0, 8 D)       key codes    [16 positions][D / 2]
//   [8 D, 9 D)     key scales   [16 positions][D / 16]
//   [9 D, 17 D)    value codes  [2][D / 16][8][8]   (half of the positions,
//                               block of 16 components, position, byte)
//   [17 D, 18 D)   value scales [D / 16][16 positions]
//
// Codes are E2M1, two per byte, the even component in the low nibble; scales
// are E4M3, one per 16 consecutive components of a position.  Keys are the
// k x n operand of q . k^T: a row is read along the components.  Values are
// the operand of p . v, read along the positions: a lane that needs one block
// of two neighbouring positions finds them in one aligned 16-byte word, and
// its pairs of scales in one 16-bit word.
#pragma once
#include <cstddef>
#include <cstdint>

#include "ptx.cuh"

namespace sk {

constexpr int KV4_REC = 16;   // positions per record

// Bytes of a record of a head of size D.
__host__ __device__ constexpr int kv4_rec_bytes(int D) { return 18 * D; }

// Where position i (< 16) of a record keeps block b (16 components): the
// eight code bytes and the scale byte, for keys (VALUE = false) and values.
template <bool VALUE>
__device__ __forceinline__ int kv4_code_at(int D, int i, int b) {
    return VALUE ? 9 * D + (i >> 3) * 4 * D + b * 64 + (i & 7) * 8 : i * (D / 2) + b * 8;
}
template <bool VALUE>
__device__ __forceinline__ int kv4_scale_at(int D, int i, int b) {
    return VALUE ? 17 * D + b * 16 + i : 8 * D + i * (D / 16) + b;
}

// Division by a number fixed at launch, for numerators below 2^31: with
// 2^s < d <= 2^(s + 1) and mul = ceil(2^(32 + s) / d), the product's excess
// mul d - 2^(32 + s) < d <= 2^(s + 1) keeps n mul / 2^(32 + s) below the next
// integer.  mul = 0 stands for d = 1.
struct Div {
    uint32_t mul, shift;
    Div(uint32_t d = 1) : mul(0), shift(0) {
        if (d < 2) return;
        while ((1u << (shift + 1)) < d) ++shift;
        mul = uint32_t(((uint64_t(1) << (32 + shift)) + d - 1) / d);
    }
};
__device__ __forceinline__ int quotient(int n, const Div &d) {
    return d.mul ? int(__umulhi(uint32_t(n), d.mul) >> d.shift) : n;
}

// The record (index into the cache) holding records rec of a sequence whose
// pages are `table`.  A page id outside the pool is brought into it: the read
// stays in the cache's memory, its values are unspecified.
__device__ __forceinline__ uint32_t kv4_record(const int32_t *table, int rec, int recs_per_page, const Div &by,
                                               int pages, int heads, int head) {
    const int pg = quotient(rec, by);
    const int id = min(max(table[pg], 0), pages - 1);
    return (uint32_t(id) * heads + head) * recs_per_page + (rec - pg * recs_per_page);
}

// Untiled bulk copy into this CTA's shared memory (16-byte aligned, bytes a
// multiple of 16), completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

constexpr uint64_t KV4_WAIT_NS = 1000000000ull;

// Wait until `bar`'s phase of this parity is complete, for a second at most.
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > KV4_WAIT_NS) return false;
    return true;
}

// Let the copies land that a ring of SLOTS barriers at `bars` may still have in
// flight: those of the next SLOTS uses from `slot` on, whose parity is `parity`
// (a use that was never issued takes the rest of the second).
template <int SLOTS>
__device__ __forceinline__ void drain_ring(uint32_t bars, uint32_t slot, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    for (int k = 0; k < SLOTS; ++k) {
        while (!mbar_try_wait(bars + slot * 8, parity))
            if (globaltimer_ns() - t0 > KV4_WAIT_NS) return;
        if (++slot == SLOTS) {
            slot = 0;
            parity ^= 1u;
        }
    }
}

// Wait for a ring's copies into `slot`.  When the second runs out the
// workspace's error word is set (where there is one), the copies in flight are
// let land, and the thread is dead: it makes no later wait and issues no copy.
template <int SLOTS>
__device__ __forceinline__ void wait_ring(uint32_t bars, uint32_t slot, uint32_t parity, unsigned int *err, bool &dead) {
    if (dead || wait_limited(bars + slot * 8, parity)) return;
    dead = true;
    if (err) atomicOr(err, 1u);
    drain_ring<SLOTS>(bars, slot, parity);
}

}  // namespace sk
