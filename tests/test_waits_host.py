"""The waits of the experts' products (csrc/wait.h) on the host, with a clock and a barrier
of the test's own."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sequence_head_relayout_gb300", "csrc")

SOURCE = r"""
#include "wait.h"

#include <cstdio>

// A kernel's time: every look at the barrier takes 4 us, and the context is away for
// `away` in every `every`th look, before the clock is read.
struct World {
    uint64_t t = 1000, away, every;
    int64_t looks = 0, ready, broken;      // looks from which on the barrier is there, a role failed

    bool done() {
        t += 4000;
        ++looks;
        const bool there = looks >= ready;
        if (every && looks % every == 0) t += away;
        return there;
    }
};

void run(uint64_t away, uint64_t every, int64_t ready, int64_t broken) {
    World w;
    w.away = away, w.every = every, w.ready = ready, w.broken = broken;
    const bool ok = vfp::wait_until([&] { return w.done(); }, [&] { return w.looks >= w.broken; },
                                    [&] { return w.t; });
    std::printf("%d %lld\n", int(ok), static_cast<long long>(w.looks));
}

int main() {
    const uint64_t s = 1000000000ull;
    const int64_t never = int64_t(1) << 60;
    run(0, 0, 1, never);           // there at once
    run(0, 0, 400000, never);      // in 1.6 s
    run(0, 0, never, never);       // never
    run(3 * s, 5, 6, never);       // the context away for 3 s behind a look that found nothing
    run(3 * s, 1, 10000, never);   // away behind every look, which comes to 1 s of turns
    run(3 * s, 1, never, never);   // the same, and the barrier is stuck
    run(0, 0, never, 7);           // another role gave up
    run(0, 0, 500002, never);      // there just when the time is over
}
"""


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    where = tmp_path_factory.mktemp("waits")
    src, exe = str(where / "waits.cc"), str(where / "waits")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", exe, src], check=True)
    out = subprocess.run([exe], capture_output=True, check=True, text=True, timeout=60).stdout
    return [tuple(int(n) for n in line.split()) for line in out.splitlines()]


def test_a_barrier_that_comes(results):
    assert results[0] == (1, 1) and results[1] == (1, 400000)


def test_a_wait_ends(results):
    """Two seconds in looks of 4 us, and one look more; stuck in a context that is away
    behind each look, in turns that count 100 us."""
    assert results[2] == (0, 500002) and results[5] == (0, 20002)


def test_time_away_is_not_waited(results):
    """A barrier that comes is never given up because the context was switched out."""
    assert results[3] == (1, 6) and results[4] == (1, 10000)


def test_others_that_gave_up(results):
    assert results[6] == (0, 7)


def test_the_last_look_counts(results):
    assert results[7] == (1, 500002)
