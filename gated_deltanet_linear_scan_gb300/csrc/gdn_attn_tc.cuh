// gdn_attn_tc.cuh -- what the attention kernels on the tensor cores (prompts, trees of drafts) share:
// operand descriptors, the notes about a key tile, mask words.
#pragma once

#include "gdn_paged.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace tc {

// ---- 128-byte swizzled operands, as tensor-map loads leave them: 1024-byte aligned blocks
// of rows of 128 bytes (64 16-bit elements), 16-byte chunk c of row r at chunk c ^ (r & 7).

// K-major: rows are M or N indices, the 64 elements run along K; a K step of 16 elements
// advances the start address by 32 bytes, 64 elements are the next block.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t start) {
    return static_cast<uint64_t>((start & 0x3FFFFu) >> 4) | static_cast<uint64_t>(1) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 |
           static_cast<uint64_t>(2) << 61;
}

// MN-major: rows are K indices, the 64 elements run along N; `block` bytes lie between one
// block of 64 N elements and the next, `group` between one group of 8 rows and the next.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t start, uint32_t block, uint32_t group) {
    return static_cast<uint64_t>((start & 0x3FFFFu) >> 4) |
           static_cast<uint64_t>((block >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>((group >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1) << 46 |
           static_cast<uint64_t>(2) << 61;
}

// Instruction descriptor of a dense kind::f16 MMA, f32 accumulator, A and B both bf16 or
// both f16, A K-major (or in tensor memory), B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_16bit(bool bf16, int m, int n, bool b_mn_major) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

}  // namespace tc

constexpr int kTcKeys = 128;
constexpr int kTcRows = 128;
constexpr int kChunk = 32;     // keys of a chunk
constexpr int kNotes = 16;     // key tiles: more than K is ever ahead of the softmax
constexpr float kLazy = 8.0f;  // log2 of the growth of a maximum that makes O rescale

// The chunks [x, y) of the key tile at key0 that hold every key a position in [lo_p, hi_p] sees.
__device__ __forceinline__ int2 chunks_seen(const AttnMask &mask, int key0, int lo_p, int hi_p) {
    int a = kTcKeys, b = 0;
    const int lo = mask.first(max(lo_p, 0));
    if (lo < key0 + kTcKeys) {
        a = max(lo - key0, 0);
        b = min(hi_p - key0 + 1, kTcKeys);
    }
    const int sinks = min(mask.sinks, hi_p + 1) - key0;
    if (sinks > 0) {
        a = 0;
        b = max(b, min(sinks, kTcKeys));
    }
    return make_int2(a / kChunk, (b + kChunk - 1) / kChunk);
}

// What the K warp notes about a key tile: bits 0..15 its 8-key blocks that were loaded, then
// eight bits for each row tile.
struct TileNote {
    uint32_t bits;
    __device__ __forceinline__ uint32_t of(int i) const { return bits >> (16 + 8 * i); }
    __device__ __forceinline__ bool active(int i) const { return of(i) & 1u; }
    __device__ __forceinline__ bool first(int i) const { return of(i) & 2u; }  // of the row tile's
    __device__ __forceinline__ bool last(int i) const { return of(i) & 4u; }
    __device__ __forceinline__ int begin(int i) const { return (of(i) >> 3) & 3u; }      // chunks
    __device__ __forceinline__ int end(int i) const { return ((of(i) >> 5) & 3u) + 1; }
    static __device__ __forceinline__ uint32_t make(bool first, bool last, int2 seen) {
        return 1u | (first ? 2u : 0u) | (last ? 4u : 0u) | static_cast<uint32_t>(seen.x) << 3 |
               static_cast<uint32_t>(seen.y - 1) << 5;
    }
};

// Bits lo .. hi - 1 of a 32-bit word (any of them outside the word).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    const uint32_t below = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
    const uint32_t skip = lo >= 32 ? 0xFFFFFFFFu : lo <= 0 ? 0u : (1u << lo) - 1u;
    return below & ~skip;
}

}  // namespace gdn
