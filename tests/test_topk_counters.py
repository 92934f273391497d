"""The counters that the threads of the scores' kernel share, on the CPU: the kernel's own function (taken from its
source), a host thread for each warp, with warps that come late out of a barrier.  No warp's count may be lost."""
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "sinkhorn_point_cloud_gb300", "csrc", "topk.cuh")

FRAME = r"""
#include <pthread.h>
#include <stdio.h>
#include <stdlib.h>
#include <unistd.h>
#include <thread>
#include <vector>
#define __device__
#define __forceinline__ inline
struct Dim { int x; };
static thread_local Dim threadIdx;
static thread_local unsigned state;
static int late;  // the warp that is slow
static pthread_barrier_t barrier;
static unsigned __reduce_add_sync(unsigned, unsigned v) { return v; }
static void atomicAdd(volatile unsigned* p, unsigned v) { __atomic_fetch_add(p, v, __ATOMIC_SEQ_CST); }
static void pause_some() {
    state = state * 1664525u + 1013904223u;
    if (threadIdx.x / 32 == late && (state >> 24 & 1)) usleep(300);
}
static void __syncthreads() {
    pause_some();
    pthread_barrier_wait(&barrier);
    pause_some();
}
template <int NT> struct SelectSmem { volatile unsigned count[3]; };
FUNCTION
constexpr int NT = 256, STEPS = 40;
int main(int, char** argv) {
    late = atoi(argv[1]);
    pthread_barrier_init(&barrier, nullptr, NT / 32);
    SelectSmem<NT> sh = {};
    int wrong[NT / 32] = {};
    std::vector<std::thread> warps;
    for (int w = 0; w < NT / 32; ++w)
        warps.emplace_back([&, w] {
            threadIdx.x = w * 32;  // a warp as its first lane, which has the warp's sum
            state = w + 1;
            int step = 0;
            for (int s = 0; s < STEPS; ++s) {
                unsigned all = 0;
                for (int v = 0; v < NT / 32; ++v) all += v + 7 * s + 1;
                if (team_count<NT>(sh, w + 7 * s + 1, step) != all) ++wrong[w];
            }
        });
    for (auto& t : warps) t.join();
    int n = 0;
    for (int v : wrong) n += v;
    printf("%d\n", n);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    text = open(SOURCE).read()
    body = re.search(r"template <int NT>\n__device__ __forceinline__ unsigned team_count\(.*?\n}\n", text, re.S).group(0)
    at = tmp_path_factory.mktemp("counters")
    (at / "count.cpp").write_text(FRAME.replace("FUNCTION", body))
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", str(at / "count.cpp"), "-o", str(at / "count")], check=True)
    return str(at / "count")


@pytest.mark.parametrize("late", [0, 1, 7])
def test_no_count_is_lost(program, late):
    assert subprocess.run([program, str(late)], check=True, capture_output=True, timeout=120).stdout.split() == [b"0"]
