"""The further GPU tests of the serving operators under the bounds-checked build, as
test_gpu_bounds_serving.py runs the first ones."""
import re

import pytest

from test_gpu_bounds import _child

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("suite,least", [("test_gpu_serving_values.py", 80), ("test_gpu_serving_many_rows.py", 20),
                                         ("test_gpu_serving_logits.py", 10)])
def test_serving_suite_under_bounds_checks(suite, least):
    r = _child(["-m", "pytest", f"tests/{suite}", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], timeout=1800)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-4000:]
    assert "exl3 bounds check failed" not in r.stdout + r.stderr
    summary = r.stdout.strip().splitlines()[-1]
    m = re.search(r"(\d+) passed", summary)
    assert m and int(m.group(1)) >= least and "skipped" not in summary and "failed" not in summary, summary
