"""The later GPU tests of the step operators under the bounds-checked build, as
test_gpu_bounds_step.py runs the first ones."""
import re

import pytest

from test_gpu_bounds import _child

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("suite,least", [("test_gpu_step_more.py", 110), ("test_gpu_step_scores.py", 70)])
def test_later_step_suite_under_bounds_checks(suite, least):
    r = _child(["-m", "pytest", f"tests/{suite}", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], timeout=1800)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-4000:]
    assert "exl3 bounds check failed" not in r.stdout + r.stderr
    summary = r.stdout.strip().splitlines()[-1]
    m = re.search(r"(\d+) passed", summary)
    assert m and int(m.group(1)) >= least and "skipped" not in summary and "failed" not in summary, summary
