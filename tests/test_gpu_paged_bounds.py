"""The bounds-checked build on small ragged runs of the paged cache: no device check fires, and both
builds give the same tables, values, outputs and log-sum-exps bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def _run(tmp_path, bounds):
    from compressed_attention_turboquantprod_b200 import build
    build.build(bounds=bounds)
    out = tmp_path / ("bounds.npz" if bounds else "plain.npz")
    env = dict(os.environ)
    env.pop("TQ_LIBRARY", None)
    if bounds:
        env["TQ_LIBRARY"] = "bounds"
    r = subprocess.run([sys.executable, os.path.join(HERE, "paged_bounds_cases.py"), str(out)], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    return np.load(out)


def test_paged_paths_stay_in_bounds_and_results_are_identical(tmp_path):
    plain, checked = _run(tmp_path, False), _run(tmp_path, True)
    assert int(checked["bounds_enabled"][0]) == 1 and int(plain["bounds_enabled"][0]) == 0
    assert set(plain.files) == set(checked.files)
    for k in plain.files:
        if k != "bounds_enabled":
            assert np.array_equal(plain[k].view(np.uint8), checked[k].view(np.uint8)), f"{k} differs between the builds"
