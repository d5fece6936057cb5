// gdn_paged.cuh -- the paged key/value cache as the attention and bookkeeping kernels see
// it: element types, the cache's geometry and the lookup of a sequence in it, the mask, the
// walk over the key tiles a batch of queries sees, and tensor-map (TMA) loads of pages.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

// Watchdog flags of the attention kernels' units (a bounded wait that gave up sets a bit).
unsigned read_and_clear_watchdog_attn_decode(cudaStream_t s);
unsigned read_and_clear_watchdog_attn_prefill(cudaStream_t s);

// Bounded-wait self-test kernels on these flags.
gdn_status launch_wait_probe_attn_decode(bool arm, uint64_t limit_ns, float *out, cudaStream_t s);
gdn_status launch_wait_probe_attn_prefill(bool arm, uint64_t limit_ns, float *out, cudaStream_t s);

inline bool supported_dtype(int dtype) {
    return dtype == GDN_F32 || dtype == GDN_F16 || dtype == GDN_BF16;
}

inline int dtype_bytes(int dtype) { return dtype == GDN_F32 ? 4 : 2; }

inline bool supported_head_dim(int d) { return d == 64 || d == 128 || d == 256; }

inline int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Page sizes: powers of two from 8 (one swizzle atom of a shared-memory tile) to 256.
inline bool supported_page_size(int ps) {
    return ps >= 8 && ps <= 256 && (ps & (ps - 1)) == 0;
}

// The cache of one attention layer: K and V planes [n_pages][n_kv_heads][page_size][head_dim]
// (a page's rows of one head are contiguous), and per pool slot a row of page ids and a
// length in positions.
struct PagedCache {
    const int32_t *table;    // [pool][max_pages]
    const int32_t *kv_lens;  // [pool]
    const int32_t *slots;    // [n_seqs] or NULL
    int pool, max_pages, n_pages, n_kv_heads, log2_ps;

    // Slot and length of sequence n; false if either is out of range (the sequence is
    // skipped and counted).
    __device__ __forceinline__ bool lookup(int n, int &slot, int &len) const {
        slot = slots ? slots[n] : n;
        if (slot < 0 || slot >= pool) return false;
        len = kv_lens[slot];
        return len >= 0 && len <= (static_cast<long long>(max_pages) << log2_ps);
    }
    __device__ __forceinline__ int page_of(int slot, int key) const {
        return table[static_cast<size_t>(slot) * max_pages + (key >> log2_ps)];
    }
    __device__ __forceinline__ bool page_ok(int page) const { return page >= 0 && page < n_pages; }
};

// Position p sees key j: causal, inside the window (INT_MAX: no window) or a sink.
struct AttnMask {
    int window, sinks;
    __device__ __forceinline__ bool sees(int p, int j) const {
        return j <= p && (p - j < window || j < sinks);
    }
    // First key inside the window of position p.
    __device__ __forceinline__ int first(int p) const {
        return p - window >= 0 ? p - window + 1 : 0;
    }
};

inline AttnMask make_mask(int window, int n_sinks) {
    return AttnMask{window > 0 ? window : 0x7fffffff, n_sinks};
}

// The tiles of KT keys (tile t: keys t*KT .. t*KT + KT-1) that hold a key visible from some
// position in [p_first, p_last]: those of the sinks before the window, then those of the
// window. Positions before 0 see nothing.
struct TileWalk {
    int n_sink;  // tiles 0 .. n_sink-1 ahead of the window's
    int main0;   // first tile of the window's part
    int count;   // all of them
    __device__ __forceinline__ int tile(int i) const { return i < n_sink ? i : main0 + i - n_sink; }
};

template <int KT>
__device__ __forceinline__ TileWalk walk_tiles(const AttnMask &mask, int p_first, int p_last) {
    TileWalk w{0, 0, 0};
    if (p_last < 0) return w;
    const int lo = mask.first(max(p_first, 0));
    w.main0 = lo / KT;
    w.n_sink = min((min(mask.sinks, lo) + KT - 1) / KT, w.main0);
    w.count = w.n_sink + (p_last / KT + 1 - w.main0);
    return w;
}

// ------------------------------------------------------------------ element types

template <typename T>
struct Elem;

template <>
struct Elem<__nv_bfloat16> {
    static constexpr float kWeightBits = 0.0f;  // log2 of the largest weight held in two parts
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
};

template <>
struct Elem<__half> {
    static constexpr float kWeightBits = 14.0f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
};

// 2^x (the softmax works in base 2: exp(scale s - m) = 2^(scale log2(e) s - m log2(e))).
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2E = 1.4426950408889634f;

// ------------------------------------------------------------------ tensor maps

// Encodes a 3-D tensor map of `rows` rows of `cols` elements, seen as [columns of 128 bytes]
// [rows][128 bytes] and loaded in boxes of box_blocks x box_rows x 128 bytes: the columns of a
// few rows, one behind the other, with the 128-byte swizzle: 16-byte chunk c of row r lands at
// byte r * 128 + ((c ^ (r & 7)) << 4) of a 1024-byte aligned column.
gdn_status encode_blocks_map(CUtensorMap *map, const void *base, int dtype, int cols, uint64_t rows,
                             uint64_t row_bytes, int box_rows, int box_blocks);

// 3-D: [tokens][heads][cols], loaded in boxes of box_tokens x box_heads x 128 bytes (box row
// t * box_heads + h), same swizzle.
gdn_status encode_heads_map(CUtensorMap *map, const void *base, int dtype, int cols, int heads,
                            uint64_t tokens, uint64_t token_bytes, int box_heads, int box_tokens);

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ------------------------------------------------------------------ waits and copies

// Whether phase `parity` of `bar` has completed; does not suspend the thread.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait of a whole warp, in a CTA whose warps wait for one another. True when the phase
// has completed; false when the wait gave up in some lane (which raises *watchdog) or was cut
// short because another of the CTA's had (*dead): the whole warp then leaves its work. So a
// warp only goes on with what has really arrived, and its lanes stay together whichever of
// them gave up. (The votes cost the prompt attention 1 % at head_dim 128 and 3 % at 64.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *dead,
                                          unsigned *watchdog) {
    if (__all_sync(FULL_MASK, mbar_test(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    while (!__all_sync(FULL_MASK, mbar_try_wait(bar, parity))) {
        const bool late = global_timer_ns() - t0 > WAIT_LIMIT_NS;
        if (__any_sync(FULL_MASK, late || *dead)) {
            if (late) atomicOr(watchdog, WD_STAGE_COPY);
            *dead = 1;
            return false;
        }
    }
    return true;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

// For a CTA that leaves after a wait gave up: copies and tensor-core products it may still
// have in flight finish within microseconds, long before this returns, so none of them
// outlives the CTA's shared or tensor memory.
__device__ __forceinline__ void drain_in_flight() {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 500000) __nanosleep(1000);
}

// Waits for every cp_async16 of this thread.
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ------------------------------------------------------------------ host side

// Raises a kernel's shared-memory limit, once per device and kernel (`done` is the kernel's
// own: bit d for device d).
template <typename Kernel>
inline gdn_status allow_smem(Kernel kernel, int bytes, std::atomic<unsigned long long> &done) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return GDN_ERR_LAUNCH;
    const unsigned long long bit = 1ull << (device & 63);
    if (device < 64 && (done.load(std::memory_order_relaxed) & bit)) return GDN_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    done.fetch_or(bit, std::memory_order_relaxed);
    return GDN_OK;
}

// Arguments every call on a paged cache shares.
inline gdn_status check_cache(int n_kv_heads, int head_dim, int page_size, int n_pages,
                              int max_pages, int dtype) {
    if (n_kv_heads < 1 || head_dim < 1 || page_size < 1 || n_pages < 1 || max_pages < 1)
        return GDN_ERR_SHAPE;
    if (!supported_dtype(dtype) || !supported_head_dim(head_dim) || !supported_page_size(page_size))
        return GDN_ERR_UNSUPPORTED;
    // tensor-map row coordinates, and positions, are 32-bit
    if (static_cast<long long>(n_pages) * n_kv_heads * page_size > 0x7fffffffLL ||
        static_cast<long long>(max_pages) * page_size > 0x7fffffffLL)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace gdn
