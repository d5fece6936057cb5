// gdn_attn_again.cuh -- rows of a tree's attention that came out NaN, computed once more key by key.
//
// The tiled products multiply every row's weights with every value of a tile: 0 times an infinity or a NaN, at a
// key that other nodes see and this one does not (a node of another branch), makes the row NaN. And three bf16
// parts of a key or value that is not finite, or above bf16's range, are NaN themselves. What such a row should be
// is told by the keys that it sees, from the pages. A warp takes a row: its NaN columns, if such a value stands in
// them at a key that it does not see and no NaN at a node that it does (else, with whole operands, they are rightly
// NaN), 32 keys at a time until they are NaN all the same. All other rows pay a comparison a column. (Looking for
// such values ahead of the products cost calls with short caches 7 to 20 %. 64 trees of 16 over 64..8192 keys: 0.19 ms,
// 1.4 with a NaN here and there that all nodes see, 5.6 where every value is NaN.)
#pragma once

#include "gdn_paged.cuh"

namespace gdn {

__device__ __forceinline__ float value_at(const float *x) { return *x; }
__device__ __forceinline__ float value_at(const __half *x) { return __half2float(*x); }
__device__ __forceinline__ float value_at(const __nv_bfloat16 *x) { return __bfloat162float(*x); }
__device__ __forceinline__ void put_value(float *to, float x) { *to = x; }
__device__ __forceinline__ void put_value(__half *to, float x) { *to = __float2half_rn(x); }
__device__ __forceinline__ void put_value(__nv_bfloat16 *to, float x) { *to = __float2bfloat16_rn(x); }

// A node's row of a head, the part of its keys that it is summed over (from .. to - 1), and where that went: `out`
// or, unless NULL, `record` (the sums of a split unit's part), whose row has the length l. Where that is NaN the
// record's sums become relative to a maximum of their own; it and the length go to ml, unless that is NULL.
template <typename T>
struct AgainRow {
    const T *q, *k_pages, *v_pages;
    const int32_t *parents;  // of the sequence's nodes
    T *out;
    float *record, *ml;
    int slot, kvh, node, base, len, from, to;
    float scale_log2, l;
};

// Columns c .. c + COLUMNS - 1. By a whole warp, the same row in all lanes. PARTS: the products' operands were three
// bf16 parts.
template <typename T, int D, int COLUMNS, bool PARTS>
__device__ __noinline__ void again(const PagedCache &cache, const AttnMask &mask, const AgainRow<T> &r, int c) {
    constexpr int N = (COLUMNS + 31) / 32, kVec = 16 / static_cast<int>(sizeof(T));
    const int lane = threadIdx.x & 31, from = max(r.from, 0), to = min(r.to, r.len);
    __syncwarp();  // the row has been written
    bool wanted[N];
#pragma unroll
    for (int x = 0; x < N; ++x) {
        const int column = c + lane + 32 * x;
        wanted[x] = false;
        if (lane + 32 * x < COLUMNS) {
            const float y = r.record != nullptr ? __ldcg(r.record + column) : value_at(r.out + column);
            wanted[x] = y != y;
        }
    }
    // the nodes on the path, and those of them that it sees (positions are depths)
    unsigned long long tree = 0;
    int depth = -1;
    for (int a = r.node; a >= 0; a = r.parents[a]) ++depth;
    for (int a = r.node, up = 0; a >= 0; a = r.parents[a], ++up)
        if (up < mask.window || r.base + depth - up < mask.sinks) tree |= 1ull << a;
    auto sees = [&](int key) {
        return key < r.base ? r.base + depth - key < mask.window || key < mask.sinks : ((tree >> ((key - r.base) & 63)) & 1ull) != 0;
    };
    auto page_at = [&](int key) {
        const int page = cache.page_of(r.slot, key);
        return cache.page_ok(page) ? page : -1;
    };
    auto row_of = [&](int page, int key) {
        return (((static_cast<size_t>(page) * cache.n_kv_heads + r.kvh) << cache.log2_ps) + (key & ((1 << cache.log2_ps) - 1))) * D;
    };
    // ---- keys that others see: those the root's window still reaches, and the nodes
    if constexpr (!PARTS) {
        bool found[N] = {}, nan[N] = {};  // among those that it does not see; those that it does
        for (int key = max(from, mask.first(r.base)); key < to; ++key) {
            if (key < r.base && r.len - 1 - key < mask.window) key = max(from, r.base);  // (all see those up to there)
            if (key >= to) break;
            const int page = page_at(key);
            if (page < 0) continue;
            const T *v = r.v_pages + row_of(page, key) + c + lane;
            const bool seen = sees(key);
#pragma unroll
            for (int x = 0; x < N; ++x)
                if (wanted[x]) {
                    const float y = value_at(v + 32 * x);
                    found[x] |= !seen && !(fabsf(y) < INFINITY);
                    nan[x] |= seen && y != y;
                }
        }
        bool any = false;
#pragma unroll
        for (int x = 0; x < N; ++x) any |= wanted[x] = found[x] && !nan[x];
        if (!__any_sync(FULL_MASK, any)) return;
    }
    // ---- the sums: a lane a key for the scores, then a lane a column
    float sums[N] = {}, m = -INFINITY, l = 0.0f;
    for (int key0 = from; key0 < to; key0 += 32) {
        const int key = key0 + lane;
        int page = -1;
        if (key < to && sees(key)) page = page_at(key);
        float score = -INFINITY;
        size_t at = 0;
        if (page >= 0) {
            at = row_of(page, key);
            score = 0.0f;
#pragma unroll 4
            for (int x = 0; x < D; x += kVec) {
                const uint4 q4 = *reinterpret_cast<const uint4 *>(r.q + x), k4 = *reinterpret_cast<const uint4 *>(r.k_pages + at + x);
                T q[kVec], k[kVec];
                memcpy(q, &q4, 16);
                memcpy(k, &k4, 16);
#pragma unroll
                for (int e = 0; e < kVec; ++e) score = fmaf(value_at(q + e), value_at(k + e), score);
            }
            score = __fmul_rn(score, r.scale_log2);  // (rounded, as the maximum is: the largest weight is 1)
        }
        unsigned seen = __ballot_sync(FULL_MASK, page >= 0);
        if (seen == 0) continue;
        float top = fmaxf(m, score);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
        if (top > m) {
            const float f = fast_exp2(m - top);
            l *= f;
#pragma unroll
            for (int x = 0; x < N; ++x) sums[x] *= f;
            m = top;
        }
        const float w = page >= 0 ? fast_exp2(__fsub_rn(score, m == -INFINITY ? 0.0f : m)) : 0.0f;
        float part = w;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) part += __shfl_xor_sync(FULL_MASK, part, o);
        l += part;
#pragma unroll 8
        for (int y = 0; y < 32; ++y) {
            const float wy = __shfl_sync(FULL_MASK, w, y);
            const T *v = r.v_pages + __shfl_sync(FULL_MASK, static_cast<unsigned long long>(at), y) + c + lane;
            if (!((seen >> y) & 1u)) continue;
#pragma unroll
            for (int x = 0; x < N; ++x)
                if (wanted[x]) sums[x] = fmaf(wy, value_at(v + 32 * x), sums[x]);
        }
        bool open = false;  // whether some column can still be other than NaN
#pragma unroll
        for (int x = 0; x < N; ++x) open |= wanted[x] && sums[x] == sums[x];
        if (!__any_sync(FULL_MASK, open) && (!PARTS || r.ml == nullptr)) break;
    }
#pragma unroll
    for (int x = 0; x < N; ++x) {
        const int column = c + lane + 32 * x;
        if (!wanted[x]) continue;
        const float y = sums[x] / l;
        if (r.record == nullptr) {
            put_value(r.out + column, y);
        } else if (PARTS && r.l != r.l) {
            __stcg(r.record + column, sums[x]);
        } else {
            // (a rounding more than the sums had: the largest floats stay finite)
            const float z = y * r.l;
            __stcg(r.record + column, fabsf(y) < INFINITY && !(fabsf(z) < INFINITY) ? copysignf(0x1.fffffep127f, z) : z);
        }
    }
    if (PARTS && r.ml != nullptr && lane == 0) {
        r.ml[0] = m;
        r.ml[1] = l;
    }
    __syncwarp();
}

}  // namespace gdn
