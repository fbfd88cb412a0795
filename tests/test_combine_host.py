"""The combine follows every attention call: what one cache's pieces need in it must not cost the others."""

import os
import re
import subprocess

import paged_kv_cache_111_gb300 as pkv
from paged_kv_cache_111_gb300 import _build


def test_the_combine_has_no_stack_frame(tmp_path):
    """A kernel with local memory takes 0.2 us longer to launch, and a small decode step has 8 in all."""
    res = subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-Xptxas", "-v", "-c",
                          os.path.join(_build.CSRC, "paged_attn.cu"), "-o", str(tmp_path / "x.o")],
                         capture_output=True, text=True, check=True)
    frames = dict(re.findall(r"Function properties for (\S*combine_kernel\S*)\n\s*(\d+) bytes stack frame", res.stderr))
    assert len(frames) == 2, res.stderr
    assert set(frames.values()) == {"0"}, frames


def test_more_rows_than_the_combine_counts_are_refused():
    _build.build()
    combine = pkv.load().pkv_paged_attn_combine
    assert combine(0x10000, 0x20000, 1 << 20, (1 << 31) - 1, 1 << 10, 64, None) == 2       # PKV_ERR_SHAPE
