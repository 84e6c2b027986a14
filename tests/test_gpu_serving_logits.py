"""The adjustment of logits where rules meet: masks with penalties that are not finite,
long lists of biases. Outputs are equal to the same fp32 operations done one by one.
"""
import numpy as np
import pytest

import serving_ref as ref
import trellis_quantized_linear_gb300 as tql
from gpu_util import torch_mod
from test_gpu_serving import dev, gpu  # noqa: F401 (gpu: fixture)

pytestmark = pytest.mark.gpu


def test_forbidden_tokens_stay_out_whatever_their_penalties():
    """The mask comes last: -inf, also where a penalty alone would make a NaN or an infinity of the token."""
    torch = torch_mod()
    n, M = 5000, 6
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((M, n)).astype(np.float32)
    hist = rng.integers(0, n, (M, 600)).astype(np.int32)
    rep = np.array([1.2, np.nan, 1.2, 1.2, 0.0, 1.2], dtype=np.float32)
    pres = np.array([-np.inf, 0, np.nan, 0, 0, np.inf], dtype=np.float32)
    freq = np.array([0, 0, 0, -3e38, 0, 0], dtype=np.float32)
    hist[3, :5] = 77
    bias = [(int(t), 1.5) for t in rng.integers(0, n, 30)]
    allow = np.zeros((M, -(-n // 32) * 32), dtype=bool)
    allow[:, :n] = rng.random((M, n)) < 0.5
    allow[3, 77] = False
    x = dev(logits)
    am = torch.empty((M,), dtype=torch.int32, device="cuda")
    tql.exl3_logits_adjust(x, n, x, am, history=dev(hist.ravel()), history_start=dev(np.arange(M + 1, dtype=np.int32) * 600),
                           repetition=dev(rep), presence=dev(pres), frequency=dev(freq),
                           bias_id=dev(np.array([t for t, _ in bias] * M, dtype=np.int32)),
                           bias_value=dev(np.array([v for _, v in bias] * M, dtype=np.float32)),
                           bias_start=dev(np.arange(M + 1, dtype=np.int32) * 30),
                           allowed=dev(np.packbits(allow, axis=1, bitorder="little").view(np.uint32).view(np.int32)))
    got = x.cpu().numpy()
    assert np.all(np.isneginf(got[~allow[:, :n]]))
    for m in range(M):
        with np.errstate(all="ignore"):
            want, pick = ref.adjust(logits[m], hist[m], 0, rep[m], pres[m], freq[m], bias, allow[m, :n], np.float32)
        assert np.array_equal(got[m], want, equal_nan=True) and int(am[m]) == pick
