"""What the serving operators' entry points refuse before anything is launched; needs no
GPU (a call with nothing to refuse gets as far as the device, which is not initialized)."""
import ctypes

import pytest

import trellis_quantized_linear_gb300 as tql

GOOD = 1 << 20  # a 16-byte aligned fake address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that no GPU may read: only where no device can be initialized")
    tql.build()
    return tql.load()


def test_one_logits_buffer_has_one_row_distance(lib):
    rules = ctypes.byref(tql._LogitsRules())

    def call(M, logits, ldl, out, ldo):
        return lib.exl3_logits_adjust(logits, ldl, M, 250, rules, out, ldo, GOOD, None)

    assert call(2, GOOD, 256, GOOD, 260) == 1
    assert call(1, GOOD, 256, GOOD, 260) == 5 and call(2, GOOD, 256, GOOD, 256) == 5 and call(2, GOOD, 256, 2 * GOOD, 260) == 5
