"""Waits that last as long as an item's work (csrc/ring.cuh) on the CPU: they go on while the kernel's count of copied stages
changes, however long that takes in all, and end one limit after it has stopped."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "speculative_decoding_verification_51_gb300", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include "ring.cuh"

#define REQUIRE(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

// An item of `steps` steps of up to `step` time units, stuck from `stops` on (-1: never), and a warp that waits for its end by
// attempts of at most `most`: the time at which its wait ended, whether it came, and when the item last moved.
struct End { bool came; long at; long last; };
End item(std::mt19937& rng, long steps, long step, long stops, long limit, long most, long gives_up = -1) {
    long now = 1, next = 0, done = 0, last = 1;
    auto advance = [&](long to) {
        while (done < steps && done != stops) {
            if (!next) next = last + 1 + long(rng() % step);
            if (next > to) break;
            last = next;
            next = 0;
            ++done;
        }
        now = to;
    };
    auto attempt = [&]() {
        const long until = now + 1 + long(rng() % most);
        while (now < until) {
            advance(now + 1);
            if (done == steps) return true;
        }
        return false;
    };
    const bool came = sv::wait_while_moving(attempt, [&]() { return gives_up >= 0 && now >= gives_up; },
                                            [&]() { return (unsigned)done; }, [&]() { return (uint64_t)now; }, limit);
    return {came, now, last};
}

int main() {
    std::mt19937 rng(1);
    const long limit = 2000, most = 100;
    for (int i = 0; i < 3000; ++i) {
        const long steps = 1 + rng() % 300, step = 1 + rng() % 900;  // up to 100 limits in all
        const End e = item(rng, steps, step, -1, limit, most);
        REQUIRE(e.came);
        const End f = item(rng, steps, step, rng() % steps, limit, most);
        REQUIRE(!f.came);
        REQUIRE(f.at - f.last >= limit && f.at - f.last <= limit + 3 * most);
        const long at = 1 + long(rng() % (steps * 10));
        const End g = item(rng, steps, 1000000, 0, limit, most, std::min(at, limit));
        REQUIRE(!g.came && g.at <= std::min(at, limit) + most);
    }
    std::puts("ok");
}
"""


def build(tmp_path, program):
    src, exe = tmp_path / "wait.cpp", tmp_path / "wait"
    src.write_text(program)
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_long_items_do_not_run_out(tmp_path):
    r = build(tmp_path, PROGRAM)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_model_sees_one_limit_for_all(tmp_path):
    """A wait of one limit, however much moves meanwhile."""
    counts = "[&]() { return (unsigned)done; }"
    assert PROGRAM.count(counts) == 1
    assert build(tmp_path, PROGRAM.replace(counts, "[&]() { return 0u; }")).returncode == 1


def test_the_prompt_kernel_waits_by_progress():
    """For what may be an item's length ahead: the first tile that is not seen whole, and a row tile's next scores."""
    with open(os.path.join(CSRC, "prompt_attn.cuh")) as f:
        text = f.read()
    wait = text[text.index("auto wait_long = "):]
    assert "wait_while_moving(" in wait[:wait.index("\n    };")]
    assert "wait_long(&near," in text and "wait(&near," not in text
    softmax = text[text.index("else wait_long(&sf["):]
    assert softmax.index("for (int j = ja; j < jb;") < softmax.index("wait(&sf[")
