"""How a watchdog flag is read: against a fake of the two copies on the host, the flag is always
read, and written back to zero only when it is set (gdn_device_error reads six of them)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_linear_scan_gb300", "csrc")

FAKE = r"""
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstring>
#define __device__
#define __forceinline__ inline
using std::min;
typedef struct CUstream_st *cudaStream_t;
enum cudaError_t { cudaSuccess };
enum cudaMemcpyKind { cudaMemcpyHostToDevice, cudaMemcpyDeviceToHost };
inline int reads, writes, waits_behind;
template <typename T>
cudaError_t cudaMemcpyFromSymbolAsync(void *to, const T &from, size_t n, size_t, cudaMemcpyKind, cudaStream_t) {
    std::memcpy(to, &from, n);
    ++reads;
    return cudaSuccess;
}
template <typename T>
cudaError_t cudaMemcpyToSymbolAsync(T &to, const void *from, size_t n, size_t, cudaMemcpyKind, cudaStream_t) {
    std::memcpy(&to, from, n);
    ++writes;
    return cudaSuccess;
}
inline cudaError_t cudaStreamSynchronize(cudaStream_t) { waits_behind = reads + writes; return cudaSuccess; }
inline cudaError_t cudaGetLastError() { return cudaSuccess; }
struct Dim { int x; };
inline Dim threadIdx, blockDim;
inline unsigned __ballot_sync(unsigned, bool) { return 0; }
inline int __clz(unsigned) { return 0; }
inline void __syncthreads() {}
"""

MAIN = r"""
#include <cstdio>
#include "gdn_internal.h"
int main() {
    for (unsigned start : {0u, 2u, 5u}) {
        unsigned flag = start;
        reads = writes = waits_behind = 0;
        const unsigned got = gdn::read_and_clear_flag(flag, nullptr);
        std::printf("%u %u %d %d %d\n", got, flag, reads, writes, waits_behind);
    }
}
"""


def test_a_flag_is_written_only_when_it_is_set(tmp_path):
    (tmp_path / "cuda_runtime.h").write_text(FAKE)
    (tmp_path / "main.cc").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-I", str(tmp_path), "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    str(tmp_path / "main.cc"), "-o", str(tmp_path / "main")], check=True)
    out = subprocess.run([str(tmp_path / "main")], check=True, capture_output=True, text=True).stdout
    # value read, flag left, reads, writes, and all of them waited for
    assert [tuple(map(int, line.split())) for line in out.splitlines()] == [
        (0, 0, 1, 0, 1), (2, 0, 1, 1, 2), (5, 0, 1, 1, 2)]


def test_every_flag_is_read_this_way():
    units = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu")]
    bodies = []
    for name in units:
        text = open(os.path.join(CSRC, name)).read()
        for part in text.split("unsigned read_and_clear_watchdog_")[1:]:
            bodies.append((name, part[part.index("{"):part.index("}")]))
    assert len(bodies) == 6
    for name, body in bodies:
        assert "return read_and_clear_flag(g_watchdog" in body, name
