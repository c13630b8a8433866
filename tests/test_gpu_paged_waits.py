"""The decode's bounded waits, made to run out in the bounds-checked build by leaving its copies out."""
import os
import subprocess
import sys

import pytest

from gpu_common import nat

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_waits_that_run_out_are_reported():
    from compressed_attention_turboquantprod_b200 import build
    build.build(bounds=True)
    r = subprocess.run([sys.executable, os.path.join(HERE, "paged_wait_case.py")], env={**os.environ, "TQ_LIBRARY": "bounds"},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "reported" in r.stdout


def test_the_normal_build_has_no_such_switch():
    n = nat()
    with pytest.raises(n.TQError) as e:
        n.tq_debug_paged_lose_copies(True)
    assert e.value.status == n.TQ_ERR_UNSUPPORTED
