"""A bounded wait whose clock need not be right every time: the kernels' own loop, in a host program."""
import os
import shutil
import subprocess

import pytest

from moe_expert_layer_05_gb300 import build

SRC = r"""
#include <cstdio>
#include <cstdlib>
#include "wait_clock.h"
// limit, number of tests after which it is done, of readings after which it is stopped (0: never), then the clock's
// readings, the last two steps of which go on for ever -> how it ended, tests, readings
int main(int n, char** v) {
  const unsigned long long limit = strtoull(v[1], nullptr, 10), done_at = strtoull(v[2], nullptr, 10),
                           stop_at = strtoull(v[3], nullptr, 10);
  unsigned long long tests = 0, reads = 0, last = 0, before = 0;
  const auto now = [&] {
    const unsigned long long at = 4 + reads++;
    const unsigned long long r = at < static_cast<unsigned long long>(n) ? strtoull(v[at], nullptr, 10) : last + (last - before);
    before = last;
    return last = r;
  };
  const moe::Waited w = moe::bounded_wait<64>([&] { return ++tests == done_at; }, [&] { return reads == stop_at; }, now, limit);
  printf("%d %llu %llu\n", static_cast<int>(w), tests, reads);
  return 0;
}
"""
DONE, STOPPED, OVER = range(3)
LIMIT = 2_000_000_000
CARRY = 1 << 32
T0 = 7 * CARRY + 12345
MS = 1_000_000


@pytest.fixture(scope="module")
def wait(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("clock")
    src, exe = str(d / "clock.cpp"), str(d / "clock")
    with open(src, "w") as fh:
        fh.write(SRC)
    csrc = os.path.join(os.path.dirname(os.path.abspath(build.__file__)), "csrc")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", csrc, src, "-o", exe], check=True)

    def run(readings, limit=LIMIT, done=0, stop=0):
        words = [limit, done, stop, *(r % (1 << 64) for r in readings)]
        return tuple(int(x) for x in subprocess.run([exe, *map(str, words)], check=True, capture_output=True,
                                                    text=True).stdout.split())

    return run


def test_a_wait_ends_after_its_limit(wait):
    how, tests, reads = wait([T0, T0 + MS])
    assert how == OVER and tests == 64 * (reads - 8) and 2000 < reads < 2020           # (a lap's first reading has no tests)
    how, _, reads = wait([T0, T0 + 10_000 * MS])                                       # readings further apart than it
    assert how == OVER and reads == 16
    assert wait([T0, T0 + MS], limit=(1 << 64) - 1, done=64 * 100_000)[0] == DONE      # one that nothing reaches


def test_a_wait_ends_when_it_is_done_or_stopped(wait):
    assert wait([T0, T0 + MS], done=1) == (DONE, 1, 1)
    assert wait([T0, T0 + MS], done=700) == (DONE, 700, 11)
    assert wait([T0, T0 + MS], stop=5) == (STOPPED, 320, 5)
    assert wait([T0, T0 + 10_000 * MS], stop=1) == (STOPPED, 64, 1)


@pytest.mark.parametrize("wrong", [-1, -MS, -CARRY, CARRY, -T0, (1 << 64) - 1 - T0, 1 << 62, -(1 << 34)])
@pytest.mark.parametrize("at", [0, 1, 25, 700])
def test_one_wrong_reading_ends_no_wait_and_keeps_none(wait, wrong, at):
    good = [T0 + 1000 * i + (wrong if i == at else 0) for i in range(at + 3)]
    assert wait(good, done=64 * 2000)[0] == DONE                                      # two milliseconds of waiting
    good = [T0 + MS * i + (wrong if i == at else 0) for i in range(at + 3)]
    how, _, reads = wait(good)
    assert how == OVER and 2000 - 251 <= reads <= 2020 + 502


def test_a_clock_of_two_units(wait):
    """Readings in turns of two units a second apart: a step ahead counts an eighth of the limit, one back nothing."""
    turns = [T0 + 1000 * i + (1_000_000_000 if i % 2 else 0) for i in range(100)]
    assert wait(turns, done=64 * 6)[0] == DONE
    how, _, reads = wait(turns)
    assert how == OVER and reads <= 40
