// gdn_tree.cuh -- a sequence's tree of drafted tokens, as the kernels see it.
#pragma once

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr int kMaxNodes = GDN_MAX_TREE_NODES;  // the bits of a path's mask
static_assert(kMaxNodes == 64, "a path is a 64-bit mask, and two nodes go to a lane");

// The paths of a tree, by a whole warp: lane l gets those of nodes l (path[0]) and l + 32
// (path[1]), bit a for a = the node itself and each of its ancestors, 0 where there is no node.
// `path_of` and `up`: shared memory of the warp's own, kMaxNodes entries each; path_of keeps the
// paths of all nodes. Returns, in every lane, whether some parent was not valid: neither below
// its node, nor -1, nor GDN_NO_NODE, or a node that is not there; such a node is not there.
//
// Pointer jumping: after step s a mask holds 2^s nodes of the path, and `up` is the next one.
__device__ __forceinline__ bool tree_paths(const int32_t *__restrict__ parents, int n_nodes,
                                           unsigned long long (&path)[2],
                                           unsigned long long *path_of, int *up) {
    const int lane = threadIdx.x & 31;
    int parent[2], next[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        parent[x] = i < n_nodes ? parents[i] : GDN_NO_NODE;
        const bool ok = parent[x] >= -1 && parent[x] < i;
        path[x] = ok ? 1ull << i : 0ull;
        next[x] = ok ? parent[x] : -1;
        path_of[i] = path[x];
        up[i] = next[x];
    }
    __syncwarp();
#pragma unroll 1
    for (int s = 1; s < n_nodes; s *= 2) {
        unsigned long long more[2] = {0, 0};
        int after[2] = {-1, -1};
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (next[x] >= 0) {
                more[x] = path_of[next[x]];
                after[x] = up[next[x]];
            }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (next[x] >= 0) {
                // (a path that leads to a node that is not there ends with this node's own)
                path[x] = more[x] == 0 || path[x] == 0 ? 0 : path[x] | more[x];
                next[x] = more[x] == 0 ? -1 : after[x];
                path_of[lane + 32 * x] = path[x];
                up[lane + 32 * x] = next[x];
            }
        }
        __syncwarp();
    }
    const bool bad = (parent[0] != GDN_NO_NODE && path[0] == 0) || (parent[1] != GDN_NO_NODE && path[1] == 0);
    return __any_sync(FULL_MASK, bad);
}

// Host-side checks of a tree's arguments.
inline gdn_status check_tree(const int32_t *parents, int n_seqs, int n_nodes) {
    if (!parents) return GDN_ERR_NULL;
    if (n_seqs < 0 || n_nodes < 1) return GDN_ERR_SHAPE;
    if (n_nodes > kMaxNodes || static_cast<long long>(n_seqs) * n_nodes > 0x7fffffffLL)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace gdn
