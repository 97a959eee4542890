"""The merge of tree attention's partials follows no record that leads out of the workspace (CPU)."""
import ctypes
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_164_gb300", "csrc")
SOURCE = """#include "pkv_tree_parts.cuh"
extern "C" int partials(int ctas) { return pkv::tree_partials(ctas); }
extern "C" int partial(int cta, int begins) { return pkv::tree_partial(cta, begins != 0); }
extern "C" int valid(int a, int b, int ctas) { return pkv::tree_parts_valid(a, b, ctas); }
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    folder = tmp_path_factory.mktemp("parts")
    (folder / "parts.cpp").write_text(SOURCE)
    out = folder / "parts.so"
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(out),
                    str(folder / "parts.cpp")], check=True)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("ctas", [1, 2, 3, 9])
def test_every_record_of_a_launch_is_followed_within_its_partials(parts, ctas):
    assert parts.partials(ctas) == 2 * ctas
    for first in range(ctas):
        for last in range(first, ctas):
            assert parts.valid(first, last, ctas)
            at = [parts.partial(c, c == first) for c in range(first, last + 1)]
            assert len(set(at)) == len(at) and min(at) >= 0 and max(at) < parts.partials(ctas)
    # two units that share a CTA keep their partials apart
    assert len({parts.partial(c, b) for c in range(ctas) for b in (0, 1)}) == 2 * ctas


def test_what_an_unwritten_record_holds_is_not_followed(parts):
    """A CTA that gave up a wait leaves its later units' records as the workspace came."""
    ctas, big = 152, 2 ** 31 - 1
    words = [0, 1, 151, 152, 153, -1, -2, -2 ** 31, big, 0x7F7F7F7F, -0x5A5A5A5B, 2 ** 30]
    for first, last in itertools.product(words, words):
        if parts.valid(first, last, ctas):
            assert 0 <= first <= last < ctas
            assert 0 <= parts.partial(first, 1) and parts.partial(last, 1) < parts.partials(ctas)
        else:
            assert not 0 <= first <= last < ctas
