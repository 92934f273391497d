"""What the routed layer's kernel does about copies in flight after a wait that ran out, on the CPU: the kernel's own
function (taken from its source) on barriers that count arrivals and bytes, from any state that the ring's roles can have
stopped in.  Every copy lands, no barrier gets an arrival more than it wants, and no wait runs out."""
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "sinkhorn_point_cloud_gb300", "csrc", "k_routed_tc.cu")

FRAME = r"""
#include <stdint.h>
#include <stdio.h>
#include <algorithm>
#include <random>
#include <vector>
#define __device__
using std::max;
using std::min;
CONSTANTS
constexpr unsigned long long WAIT_NS = 1;
static int wrong = 0;
struct Barrier {
    int pending = 2, flying = 0, phase = 0;
    void look() { if (pending == 0 && flying == 0) { ++phase; pending = 2; } }
    void arrive() { if (pending == 0) ++wrong; else --pending; look(); }
};
static std::vector<Barrier> ring;
static void mbar_arrive(uint32_t s) { ring[s].arrive(); }
static bool mbar_wait_bounded(uint32_t s, uint32_t parity, volatile int*, unsigned long long) {
    ring[s].flying = 0;  // what was on its way comes in the end
    ring[s].look();
    if ((ring[s].phase & 1) == (int)parity) ++wrong;  // this phase would never end
    return true;
}
static bool mbar_try_wait(uint32_t s, uint32_t parity) { return (ring[s].phase & 1) != (int)parity; }
struct Ctx { int S; uint32_t full(int s) const { return s; } };
struct TcArgs { unsigned long long wait_ns; };
FUNCTION
int main() {
    std::mt19937 r(1);
    const auto to = [&](int n) { return n > 0 ? (int)(r() % (n + 1)) : 0; };  // 0 .. n
    for (int trial = 0; trial < 200000; ++trial) {
        const int S = 3 + to(MAX_STAGES - 3), L = min(LOADERS, S), multiplied = to(40);
        const int issued = multiplied + to(S);
        std::vector<int> loaded(LOADERS, 0);
        std::vector<bool> has(issued + 2 * S, false);
        for (int w = 0; w < L; ++w)
            for (int u = w; u < multiplied + S && u < (int)has.size(); u += L) {
                if (u >= multiplied && to(2) == 0) break;  // given up before this unit
                has[u] = true;
                ++loaded[w];
            }
        ring.assign(S, Barrier());
        for (int u = 0; u < (int)has.size(); ++u) {
            Barrier& b = ring[u % S];
            if (u < multiplied) {
                if (!has[u]) return 2;
                ++b.phase;
                continue;
            }
            if (u < issued) {  // the producer's arrival, and bytes that have come or not
                b.flying = to(1);
                b.arrive();
            }
            if (has[u]) b.arrive();
        }
        Ctx c = {S};
        TcArgs t = {1};
        CALL;
        for (int u = max(0, issued - S); u < issued; ++u) wrong += ring[u % S].flying;
        if (wrong) break;
    }
    printf("%d\n", wrong);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    text = open(SOURCE).read()
    constants = "\n".join(re.search(rf"constexpr int (?:[^;]*\b)?{name} = \d+[^;]*;", text).group(0) for name in ("LOADERS", "MAX_STAGES"))
    function = re.search(r"__device__ void settle\((.*?)\) {\n.*?\n}\n", text, re.S)
    arguments = {"const Ctx& c": "c", "const TcArgs& t": "t", "int issued": "issued", "const int* loaded": "loaded.data()"}
    call = "settle(%s)" % ", ".join(arguments[a.strip()] for a in function.group(1).split(","))
    at = tmp_path_factory.mktemp("settling")
    body = FRAME.replace("CONSTANTS", constants).replace("FUNCTION", function.group(0)).replace("CALL", call)
    (at / "settle.cpp").write_text(body)
    subprocess.run(["g++", "-std=c++17", "-O1", str(at / "settle.cpp"), "-o", str(at / "settle")], check=True)
    return str(at / "settle")


def test_copies_in_flight_land(program):
    assert subprocess.run([program], check=True, capture_output=True, timeout=120).stdout.split() == [b"0"]
