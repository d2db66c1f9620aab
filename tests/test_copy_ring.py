"""The ring of copies of k_attn_rows (csrc/ring.cuh) on the CPU, against copies that
are late or never come: none is begun into a stage that one is still writing to,
and none is in flight when the kernel ends."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "speculative_decoding_verification_51_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "ring.cuh"

#define REQUIRE(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

// a stage's barrier and the copy that completes its phase at `lands`
struct Stage { long lands = -1; bool armed = false; unsigned phase = 0; };

template <unsigned N>
void run(unsigned seed, int chunks, int late_one_in, long limit) {
    std::mt19937 rng(seed);
    std::vector<Stage> st(N);
    long now = 0;
    auto settle = [&](Stage& s) {
        if (s.armed && s.lands <= now) { s.armed = false; s.phase ^= 1; }
    };
    // what mbar_wait_bounded does: waits until the phase of that parity is over, at most `limit`
    auto wait = [&](unsigned i, unsigned parity, long lim) {
        Stage& s = st[i];
        settle(s);
        if (s.phase != parity) return true;
        REQUIRE(s.armed);                       // a wait for a copy that was begun
        if (s.lands - now > lim) { now += lim; return false; }
        now = s.lands;
        settle(s);
        return true;
    };
    sv::CopyRing<N> ring;
    int left = chunks, waits = 0, lost = 0;
    auto issue = [&]() {
        if (!left || !ring.alive()) return;
        const unsigned i = ring.begin();
        settle(st[i]);
        REQUIRE(!st[i].armed);                  // nothing in flight into this stage
        --left;
        st[i].armed = true;
        const bool late = late_one_in && rng() % late_one_in == 0;
        st[i].lands = now + 1 + rng() % 20 + (late ? limit + long(rng() % (3 * limit)) : 0);
    };
    for (unsigned i = 0; i < N; ++i) issue();
    for (int c = 0; c < chunks; ++c) {
        const unsigned i = ring.stage();
        if (ring.alive()) {
            ++waits;
            if (!wait(i, ring.parity(), limit)) { ring.lose(); ++lost; }
        }
        ring.next();
        now += 1 + rng() % 5;
        issue();
    }
    REQUIRE(lost <= 1);
    ring.drain([&](unsigned i, unsigned parity) { wait(i, parity, 100 * limit); });
    for (auto& s : st) { settle(s); REQUIRE(!s.armed); }
    if (!lost) REQUIRE(waits == chunks && left == 0);
}

int main() {
    for (unsigned seed = 0; seed < 3000; ++seed)
        for (int late : {0, 3, 20, 200})
            for (int chunks : {0, 1, 2, 5, 6, 7, 40, 133}) {
                run<2>(seed, chunks, late, 1000);
                run<3>(seed, chunks, late, 1000);
                run<6>(seed, chunks, late, 1000);
            }
    std::puts("ok");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_no_copy_outlives_a_wait_that_ran_out(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("mistake", [("if (!left || !ring.alive()) return;", "if (!left) return;"),
                                     ("ring.drain([&]", "if (0) ring.drain([&]")])
def test_the_model_sees_both_mistakes(tmp_path, mistake):
    """Copies that go on after a lost wait, and an end without waiting for them."""
    assert PROGRAM.count(mistake[0]) == 1
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM.replace(*mistake))
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, timeout=120).returncode == 1
