"""The bounded waits of tv_chunk_attn's tcgen05 kernel, run out on purpose, as
in test_gpu_timeout.py: the development build withholds the TMA loads of one
tile and shortens the wait limit, so the waits on that tile run out; the call
reports TV_DEV_TIMEOUT and the next one on the stream is right."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_timeout_exit_reports_and_leaves_the_context_usable():
    from speculative_decoding_tree_attn_gb300 import build as B
    from speculative_decoding_tree_attn_gb300 import capi

    lib = B.build(dev=True)
    env = dict(os.environ, TREEVERIFY_LIB=lib)
    r = subprocess.run([sys.executable, os.path.join(HERE, "chunk_timeout_child.py")], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    lines = [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]
    assert len(lines) == 4, r.stdout
    for x in lines:
        assert x["status"] & capi.TV_DEV_TIMEOUT and x["after"] == 0, x
