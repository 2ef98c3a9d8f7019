"""The compile-time check of the waits in a ring of LDS stages (csrc/loadorder.hpp)
against a simulation of loads that land in order, for every ring and number of
loads that the kernels use (CPU only; built with the host compiler)."""
import os
import shutil
import subprocess

import pytest

import bf16_activation_quantized_amd as w4

CSRC = os.path.join(os.path.dirname(w4.LIB_PATH), "csrc")
RINGS = [(NS, parts) for NS in range(3, 9) for parts in range(1, 8)]


def landed_in_time(NS, parts, worded, start, step):
    """Requests one by one; before each use at most `start` or `step` of them may be in flight. A stage's scale word
    comes ahead of its parts, where it helps least."""
    order = []

    def request(s):
        order.extend((["word"] if s >= worded or s >= NS - 1 else []) + [s] * parts)

    def late(n, needed):
        return any(s != "word" and s <= needed for s in order[max(0, len(order) - n):])

    for s in range(NS - 1):
        request(s)
    if late(start, 1):
        return False
    for j in range(4 * NS):
        request(j + NS - 1)
        if late(step, j + 2):
            return False
    return True


def kernel(NS, parts):
    """The order and the waits of the input gradient of the 4-bit products."""
    ahead = 4 if NS > 5 else 2
    return NS - 1 - ahead, (NS - 3) * parts + min(ahead, NS - 3), (NS - 3) * (parts + 1)


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("order")
    (d / "a.cpp").write_text('#include "loadorder.hpp"\n#include <cstdio>\nint main() { int a, b, c, d, e; while '
                             '(scanf("%d %d %d %d %d", &a, &b, &c, &d, &e) == 5) printf("%d\\n", '
                             'w4a16::ring_waits_hold(a, b, c, d, e)); }\n')
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, "-o", d / "a", d / "a.cpp"], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([d / "a"], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [v == "1" for v in out]
    return run


def test_the_kernels_waits_hold(check):
    cases = [(NS, parts, *kernel(NS, parts)) for NS, parts in RINGS]
    assert all(check(cases)) and all(landed_in_time(*c) for c in cases)


def test_the_check_is_the_simulation(check):
    cases = [(NS, parts, worded, start, step) for NS, parts in RINGS if parts < 5 for worded in range(NS)
             for start in range(0, NS * parts + 2, 2) for step in range(0, NS * (parts + 1))]
    assert check(cases) == [landed_in_time(*c) for c in cases]


def test_a_word_less_ahead_of_the_loop_is_refused(check):
    """Stages ahead of the loop with no word of their own, but counted as if they had one: from 5 stages on stage j + 2
    may be missing at the end of step j."""
    cases = [(NS, parts, NS - 1, (NS - 3) * parts, (NS - 3) * (parts + 1)) for NS, parts in RINGS]
    assert check(cases) == [NS < 5 for NS, _ in RINGS] == [landed_in_time(*c) for c in cases]
