"""Infinities and NaN in the nodes' K and V, and long trees, on the NaN-sentinel build (GPU):
what takes them out writes the ring of tiles that this build fills with NaN."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_164_gb300 import build as pkv_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITE = ["tests/test_gpu_tree.py::"
         "test_attention_rows_see_nothing_of_what_they_do_not_attend_to",
         "tests/test_gpu_tree.py::test_attention_of_about_a_warp_of_sequences",
         "tests/test_gpu_tree_ranges.py::test_attention_of_the_longest_trees",
         "tests/test_gpu_debug_build.py::test_child_loaded_the_debug_build"]


@pytest.mark.gpu
def test_values_that_are_not_finite_on_the_nan_sentinel_build():
    lib = pkv_build.build(debug=True)
    env = dict(os.environ, PKV_LIBRARY=lib, PKV_EXPECT_DEBUG_BUILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu",
                        "-p", "no:cacheprovider", *SUITE],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
