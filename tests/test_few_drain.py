"""The activation-copy warp of few_experts_kernel waits, before its block ends,
for every copy that it started, whichever of its waits runs out.

The warp's code is taken from few.cu as it stands and compiled for the host,
with barriers that know which copies are in flight and a wait that runs out at
a chosen turn."""
import os
import re
import shutil
import subprocess

import pytest

from mixture_experts_layer_11_gb300 import build as mbuild

HARNESS = r"""
#include <cstdint>
#include <cstdio>
#include <cstring>
#define __device__
#define __forceinline__ inline
enum : int { kFirst = 0, kSecond = 1, kSum = 2, kEnd = 3 };
constexpr int kMaxAStages = 12, kMaxBStages = 8, kBlockBytes = 128, BOX = %(box)d, RPS = %(rps)d;
constexpr uint64_t kDrainNs = 1000000000ull;
struct K { static constexpr int kBlock = 64; };
struct FewCtrl { uint64_t a_empty[kMaxAStages], b_full[2][kMaxBStages]; int abort_flag; } c;
struct Counters { int done; } counters;
struct FewArgs { int tokens, a_stages, b_ring, tiles1; uint64_t limit_ns; int32_t* status; Counters* cnt; } g;
struct Seg { int a, m, kb0, kb1, c0, c1; } s;
struct Plan { int nact = 1, most_rows = 5, act[1] = {0}, off[2] = {0, 5}; } plan;
struct CUtensorMap {} mapX, mapH;
uint8_t ring_memory[1 << 16], *b_ring = ring_memory;

int turns, fails_at, polls;          // waits for an emptied stage so far; the one that runs out
bool poll_fails;                     // the wait for the first product's rows runs out
struct Bar { int phase; bool in_flight; } full[2][kMaxBStages];
int empty_phase[kMaxAStages], lost;

uint32_t smem_u32(const void* p) { return (uint32_t)((const uint8_t*)p - (const uint8_t*)&c); }
Bar& bar_of(uint32_t at) {
    const int i = (int)((at - smem_u32(c.b_full)) / 8);
    return full[i / kMaxBStages][i %% kMaxBStages];
}
int oldest[kMaxBStages * 64], first_open, last_open, products[kMaxBStages * 64];
void few_abort(FewCtrl& x, int32_t*) { x.abort_flag = 1; }
bool mbar_wait_bounded(uint32_t at, uint32_t parity, uint64_t, volatile int*) {
    if (at < smem_u32(c.b_full)) {   // a stage is emptied: the oldest copy has landed and been used
        if (turns++ == fails_at) return false;
        Bar& b = full[products[first_open]][oldest[first_open]];
        ++first_open;
        if (b.in_flight) { b.in_flight = false; ++b.phase; }
        return true;
    }
    Bar& b = bar_of(at);
    if ((uint32_t)(b.phase & 1) != parity) return true;     // that phase is over: returns at once
    if (b.in_flight) { b.in_flight = false; ++b.phase; return true; }
    return false;
}
void mbar_arrive_expect_tx(uint32_t at, uint32_t) {
    Bar& b = bar_of(at);
    if (b.in_flight) ++lost;
    b.in_flight = true;
    const int i = (int)((at - smem_u32(c.b_full)) / 8);
    products[last_open] = i / kMaxBStages;
    oldest[last_open++] = i %% kMaxBStages;
}
void tma_load_2d(uint32_t, const CUtensorMap*, uint32_t, int, int) {}
int load_acquire(const int*) { return poll_fails ? 0 : 1 << 20; }
void fence_proxy_async_all() {}
uint64_t globaltimer_ns() { static uint64_t t; return t += 1000; }

%(ring)s

struct Walk {
    int phase, left;
    bool next(const Plan&, Seg& x) {
        if (left == 0) return false;
        --left;
        x = {0, 0, 0, 3, 0, 0};
        return true;
    }
} walk;

int in_flight_after(int fail, bool poll, int stages) {
    memset(&c, 0, sizeof c);
    memset(full, 0, sizeof full);
    turns = 0; fails_at = fail; poll_fails = poll; first_open = last_open = lost = 0;
    static int32_t status;
    g = {5, stages, 8 * %(box)d * kBlockBytes, 1, 100000, &status, &counters};
    int taken = 0;
    auto take = [&]() {
        walk = {taken == 0 ? kFirst : taken == 1 ? kSecond : taken == 2 ? kSum : kEnd, 4};
        return ++taken < 4 && !c.abort_flag;
    };
    {
%(loader)s
    }
    int n = lost;
    for (auto& p : full) for (auto& b : p) n += b.in_flight;
    return n;
}

int main() {
    int bad = 0;
    for (int stages = 2; stages <= 12; ++stages) {
        for (int fail = 0; fail <= 30; ++fail)
            if (const int n = in_flight_after(fail, false, stages)) {
                printf("%%d stages, wait %%d runs out: %%d copies in flight\n", stages, fail, n);
                ++bad;
            }
        if (in_flight_after(-1, true, stages) || in_flight_after(-1, false, stages)) ++bad;
    }
    return bad != 0;
}
"""


@pytest.mark.parametrize("box,rps", [(16, 2), (8, 1)])
def test_every_copy_lands_before_the_block_ends(tmp_path, box, rps):
    with open(os.path.join(mbuild.CSRC, "few.cu")) as fh:
        source = fh.read()
    ring = re.search(r"^struct Ring \{.*?^\};", source, re.M | re.S).group(0)
    loader = re.search(r"^            Ring r;\n(?:(?!^            Ring r;\n).)*?tma_load_2d.*?(?=^        \}\n        __syncwarp\(\);)",
                       source, re.M | re.S).group(0)
    assert "kDrainNs" in loader
    src = tmp_path / "drain.cc"
    src.write_text(HARNESS % dict(box=box, rps=rps, ring=ring, loader=loader))
    exe = str(tmp_path / "drain")
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-w", str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[:3000]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout[:2000]
