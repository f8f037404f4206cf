"""Kernels that may start while the one before them in the stream still runs.
What they read is written during their own life, so none of it may come by the
non-coherent path, which wants memory that nobody writes while a kernel runs."""
import os
import re

import shape_adaptive_tile_gb300 as sat

CSRC = os.path.join(os.path.dirname(os.path.abspath(sat.__file__)), "csrc")


def test_no_non_coherent_loads():
    early = []
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
        if name.endswith((".cu", ".cuh")) and re.search(r"wait_for_earlier|griddepcontrol\.wait", text):
            early.append(name)
            assert not re.search(r"__ldg\b|\.nc\b|__restrict__", text), name
    assert {"ffn.cu", "ffn_tile.cuh", "mxfp4.cu"} <= set(early)
