"""The 4-bit GEMV, the balance loss and sampling on the bounds-check build: the
small cases are right, and no checked index, of global memory or of the rings,
lists and sums in shared memory, leaves its buffer."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_small_cases_on_the_bounds_check_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = os.path.join(os.path.dirname(HERE), "lfsr_seeded_moe_b200", "_build", "boundscheck", "libnslm.so")
    assert os.path.exists(lib), "build it with python -m lfsr_seeded_moe_b200.build --bounds-check"
    env = dict(os.environ, NSLM_LIB_VARIANT="boundscheck")
    env.pop("NSLM_STREAM_SOURCE", None)
    r = subprocess.run([sys.executable, os.path.join(HERE, "bounds_logits_cases.py")], env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    status = {k: v for k, v in res.items() if k.startswith("status_")}
    assert set(status.values()) == {0} and len(status) == 4, status
    wrong = [k for k, v in res.items() if not k.startswith("status_") and v is not True]
    assert not wrong, wrong
    assert sum(k.startswith("sample_") for k in res) == 80
