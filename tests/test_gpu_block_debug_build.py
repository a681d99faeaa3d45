"""The -DMUON_DEBUG build's checks in the mixture-of-experts block's kernels: the
products' tile, row and K-block ranges, the row copies' and the weight
gradients' ranges, the ring's copies (alignment, stage), rows covered by their
threads, and the routing's indices.  One case per kernel
(tests/debug_block_cases.py) under each library: no call reports a status, and
the results agree bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest

from newton_schulz_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def _run(tmp_path, name, lib):
    out = str(tmp_path / f"{name}.npz")
    env = dict(os.environ, MUON_LIB_PATH=lib)
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_block_cases.py"), out], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    return np.load(out)


def test_debug_build_checks_pass_and_match_release(tmp_path, cuda_ok):
    debug_lib = build.build(debug=True)
    rel = _run(tmp_path, "release", build.LIB)
    dbg = _run(tmp_path, "debug", debug_lib)
    assert int(rel["debug_build"]) == 0 and int(dbg["debug_build"]) == 1
    assert list(rel["names"]) == list(dbg["names"])
    for n, code_r, code_d in zip(dbg["names"], rel["codes"], dbg["codes"]):
        assert code_d == 0 and code_r == 0, (n, int(code_r), int(code_d))
    keys = sorted(k for k in rel.files if k not in ("names", "codes", "debug_build"))
    assert keys == sorted(k for k in dbg.files if k not in ("names", "codes", "debug_build"))
    for k in keys:
        assert np.array_equal(rel[k], dbg[k], equal_nan=True), k
