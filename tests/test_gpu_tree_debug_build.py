"""The tree-attention parity cases on the NaN-sentinel build (GPU).

The -DPKV_DEBUG build fills every ring slot with NaN bytes at the start and
whenever its tile is released, so a tensor-core product that reads a slot before
its copy lands, or after its release, writes NaN.  The cases run in a child
process that loads that build in place of the normal one.
"""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_164_gb300 import build as pkv_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITE = ["tests/test_gpu_tree.py::test_attention_matches_the_definition",
         "tests/test_gpu_tree.py::test_attention_skips_and_flags_bad_blocks",
         "tests/test_gpu_tree.py::test_attention_is_the_same_every_time",
         "tests/test_gpu_debug_build.py::test_child_loaded_the_debug_build"]


@pytest.mark.gpu
def test_tree_attention_on_the_nan_sentinel_build():
    lib = pkv_build.build(debug=True)
    env = dict(os.environ, PKV_LIBRARY=lib, PKV_EXPECT_DEBUG_BUILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu",
                        "-p", "no:cacheprovider", *SUITE],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
