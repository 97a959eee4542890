"""The chunk-attention parity cases on the NaN-sentinel build (GPU).

The -DPKV_DEBUG build fills the ring with NaN bytes at the start and a slot whenever its
tile is released, so a product that reads a slot before its copy lands, or after its
release, writes NaN.  The cases run in a child process that loads that build in place of
the normal one.
"""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_164_gb300 import build as pkv_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = "tests/test_gpu_chunk_attention.py::test_"
SUITE = [CASES + "short_sequences", CASES + "pages_and_layouts",
         CASES + "chunks_of_several_row_blocks", CASES + "sliding_windows",
         CASES + "pages_that_are_not_there", CASES + "everything_at_once",
         CASES + "in_place_and_the_same_bits_each_time",
         "tests/test_gpu_debug_build.py::test_child_loaded_the_debug_build"]


@pytest.mark.gpu
def test_chunk_attention_on_the_nan_sentinel_build():
    lib = pkv_build.build(debug=True)
    env = dict(os.environ, PKV_LIBRARY=lib, PKV_EXPECT_DEBUG_BUILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu",
                        "-p", "no:cacheprovider", *SUITE],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
