"""How many CTAs of a prompt attention call share an item: by the counts of the call's own device."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trellis_quantized_linear_gb300", "csrc")


@pytest.fixture(scope="module")
def ranks(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("ranks")
    (d / "r.cpp").write_text('#include "exl3_prompt_ranks.h"\nextern "C" int ranks(int n, long long rows, int causal, long long items, int sms, '
                             "const int *clusters) { return exl3::prompt_ranks(n, rows, causal, items, sms, clusters); }\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "r.so"), str(d / "r.cpp")], check=True)
    f = ctypes.CDLL(str(d / "r.so")).ranks
    f.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]
    return lambda n, rows, items, two, four, causal=1, sms=152: f(n, rows, causal, items, sms, (ctypes.c_int * 2)(two, four))


def test_few_items_are_shared(ranks):
    assert ranks(1, 8192, 33, 76, 36) == 4 and ranks(1, 4096, 83, 76, 36) == 2
    assert ranks(1, 8192, 1376, 76, 36) == 1 and ranks(1, 512, 12, 76, 36) == 1
    assert ranks(129, 129 * 8192, 33, 76, 36) == 1


@pytest.mark.parametrize("causal", [0, 1])
def test_no_more_ctas_share_an_item_than_the_device_runs_clusters_of(ranks, causal):
    for n, rows, items in ((1, 8192, 33), (1, 4096, 83), (3, 100, 6), (1, 1, 2), (128, 128 * 64, 300)):
        assert ranks(n, rows, items, 0, 0, causal) == 1
        assert ranks(n, rows, items, 76, 0, causal) in (1, 2) and ranks(n, rows, items, 0, 36, causal) in (1, 4)


def test_two_devices_each_have_their_own_answer(ranks):
    assert [ranks(1, 8192, 33, *counts) for counts in ((76, 36), (76, 0), (0, 0), (76, 36))] == [4, 2, 1, 4]
