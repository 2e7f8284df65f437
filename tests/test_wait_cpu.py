"""The kernels' bounded wait against a clock of the test's own: it lasts as long as its limit says, however long the
hardware suspends a test that fails."""
import os
import subprocess

import pytest

from helpers import ROOT

PROGRAM = r"""
#include <stdio.h>
#define __host__
#define __device__
#define __forceinline__ inline
#include "fa3_wait.cuh"
using fa3::Waited;
// One wait: a test that fails takes `step` ns, `done` and `stopped` hold from those times on (0: never); prints how it ended and
// when, in ns, and how often the clock was read.
int main(int argc, char** argv) {
  unsigned long long step, done, stopped, limit, now, start;
  while (scanf("%llu %llu %llu %llu %llu", &step, &done, &stopped, &limit, &start) == 5) {
    unsigned long long reads = 0;
    now = 0;
    const Waited w = fa3::bounded_wait([&] { now += step; return done && now >= done; }, [&] { return stopped && now >= stopped; },
                                       [&] { ++reads; return (uint32_t)((start + now) >> 20); }, (uint32_t)limit);
    printf("%d %llu %llu\n", w == Waited::kDone ? 0 : w == Waited::kStopped ? 1 : 2, now, reads);
  }
}
"""
TICK = 1 << 20
DONE, STOPPED, LATE = 0, 1, 2


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    src, exe = d / "wait.cpp", d / "wait"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wno-unknown-pragmas", "-I", os.path.join(ROOT, "int8_head_kv_gb300", "csrc"), str(src), "-o",
                    str(exe)], check=True)

    def run(*cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


@pytest.mark.parametrize("step", [10, 100, 3940, 50000])
@pytest.mark.parametrize("limit", [19, 954, 3816])
@pytest.mark.parametrize("start", [0, ((1 << 32) - 10) * TICK])           # the clock's 32 bits may wrap
def test_nothing_ends_a_wait_before_its_limit(waits, step, limit, start):
    how, when, _ = waits((step, 0, 0, limit, start))[0]
    first = 256 * step                                                    # the first look at the clock
    assert how == LATE
    assert first + limit * TICK <= when <= first + (limit + 2) * TICK + first


def test_what_is_waited_for_ends_it_without_the_clock(waits):
    assert waits((3940, 3940, 0, 954, 0), (3940, 255 * 3940, 0, 954, 0)) == [(DONE, 3940, 0), (DONE, 255 * 3940, 0)]
    how, when, reads = waits((3940, 400 * TICK, 0, 954, 0))[0]
    assert how == DONE and 400 * TICK <= when < 400 * TICK + 3940 and reads <= 400 * TICK // (256 * 3940) + 1


def test_a_stop_elsewhere_ends_it_at_the_next_look(waits):
    how, when, _ = waits((3940, 0, 100 * TICK, 954, 0))[0]
    assert how == STOPPED and 100 * TICK <= when <= 100 * TICK + 256 * 3940
