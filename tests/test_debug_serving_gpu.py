"""The bounds-checked build (compiled with -DFA_DEBUG) under the GPU tests of rotary
positions and of the 4-bit cache: no check may fire, and the results hold.  It runs in
a child process (FA_LIBRARY selects it), apart from this process's release library."""
import os
import re
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "exact_attention_117_b200", "csrc")


@pytest.mark.parametrize("name", ["rotary.cuh", "kv4.cuh", "kv4_attend.cuh", "kv4_chunk.cuh"])
def test_every_serving_kernel_has_checks(name):
    """Each kernel of a file, or a function that it calls, checks before it accesses."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert re.search(r"dbg_(check|access)\(", text), name


@pytest.mark.gpu
def test_debug_build_of_the_serving_calls():
    from exact_attention_117_b200 import build
    build.build()
    env = dict(os.environ, FA_LIBRARY=build.build(debug=True))
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_serving_check.py")], env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert re.search(r"debug build: [1-9]\d* cases clean", r.stdout)
