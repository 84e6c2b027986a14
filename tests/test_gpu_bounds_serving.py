"""The serving operators' GPU tests under the bounds-checked build
(libexl3_bounds.so), and its reporting self-test for their translation units.
A child process loads that build; every test must leave the device error word
clear, and no check may print."""
import re

import pytest

import trellis_quantized_linear_gb300 as tql
from test_gpu_bounds import _child

pytestmark = pytest.mark.gpu

SELFTEST = """
import torch
import trellis_quantized_linear_gb300 as tql
assert tql.BOUNDS_CHECKED
tql.build()
torch.cuda.set_device(0)
tql.exl3_init(0)
rep, tot = tql.exl3_selftest_bounds_serving()
assert rep == tot and tot >= 3, (rep, tot)
assert tql.exl3_get_device_status() == 0
print("bounds selftest ok")
"""


def test_bounds_checked_selftest_every_serving_unit_reports():
    r = _child(["-c", SELFTEST], timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "bounds selftest ok" in r.stdout


@pytest.mark.parametrize("suite,least", [("test_gpu_serving.py", 140), ("test_gpu_serving_limits.py", 30)])
def test_serving_suite_under_bounds_checks(suite, least):
    r = _child(["-m", "pytest", f"tests/{suite}", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], timeout=1800)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-4000:]
    assert "exl3 bounds check failed" not in r.stdout + r.stderr
    summary = r.stdout.strip().splitlines()[-1]
    m = re.search(r"(\d+) passed", summary)
    assert m and int(m.group(1)) >= least and "skipped" not in summary and "failed" not in summary, summary
