"""Experts that leave rows out, many experts and dimensions of size one in the
bounds-checked build: the device status stays clean and every output equals the
product build's, bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_bounds_checked_build_clean_and_identical(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, ops
    checked = build.build_bounds_checked()
    build.build()
    assert ops.load_library().ql_bounds_checked() == 0
    env = dict(os.environ, QL_LIBRARY=checked, PYTHONPATH=ROOT + os.pathsep + os.path.join(ROOT, "tests"))
    npz = str(tmp_path / "checked.npz")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "fp4_bounds_experts_cases.py"), npz], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "flag 1" in r.stdout, "the child did not load the bounds-checked build"
    got = np.load(npz)
    import fp4_bounds_experts_cases
    ref = fp4_bounds_experts_cases.run(ops)
    assert len(ref) > 50
    for name, (arrs, st) in ref.items():
        assert st == 0, f"{name}: product build status {st}"
        assert int(got[f"{name}__status"][0]) == 0, f"{name}: bounds-checked build reported {got[f'{name}__status'][0]}"
        for i, arr in enumerate(arrs):
            same = got[f"{name}__{i}"]
            assert np.array_equal(same, arr, equal_nan=arr.dtype.kind == "f"), f"{name}[{i}] differs"
