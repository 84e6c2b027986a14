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


@pytest.mark.parametrize("M,n,entries", [(1, 200003, 120000), (3, 5000, 20000), (11, 70001, 3000), (40, 130000, 5000), (2, 300, 4000),
                                         (1, 500000, 300000)])
@pytest.mark.parametrize("masked", [False, True])
def test_many_biases_of_the_same_tokens(M, n, entries, masked):
    """Entries of a token add up in their order, also where a row has very many, or all of one token."""
    torch = torch_mod()
    rng = np.random.default_rng([M, n])
    ld = -(-n // 4) * 4
    logits = rng.standard_normal((M, ld)).astype(np.float32)
    ids = rng.integers(-2, n + 2, (M, entries)).astype(np.int32)
    ids[0, ::7] = n - 1
    ids[M - 1, 5:2005] = n // 2
    if M > 1:
        ids[1] = np.arange(entries) % n  # each in its place
    value = (rng.standard_normal((M, entries)) * 2.0 ** rng.integers(-8, 8, (M, entries))).astype(np.float32)
    hist = rng.integers(0, n, (M, 500)).astype(np.int32)
    if M == 2:
        hist = np.concatenate([hist] * 40, axis=1)  # words of 32 bits
    rep, pres, freq = (rng.uniform(a, b, M).astype(np.float32) for a, b in ((0.8, 1.6), (-0.5, 1.0), (-0.1, 0.5)))
    kw = {}
    allow = None
    if masked:
        allow = np.zeros((M, -(-n // 32) * 32), dtype=bool)
        allow[:, :n] = rng.random((M, n)) < 0.7
        kw = dict(allowed=dev(np.packbits(allow, axis=1, bitorder="little").view(np.uint32).view(np.int32)))
    x = dev(logits)
    am = torch.empty((M,), dtype=torch.int32, device="cuda")
    tql.exl3_logits_adjust(x, n, x, am, history=dev(hist.ravel()), history_start=dev(np.arange(M + 1, dtype=np.int32) * hist.shape[1]),
                           repetition=dev(rep), presence=dev(pres), frequency=dev(freq), bias_id=dev(ids.ravel()),
                           bias_value=dev(value.ravel()), bias_start=dev(np.arange(M + 1, dtype=np.int32) * entries), **kw)
    got = x.cpu().numpy()
    for m in range(M):
        want, pick = ref.adjust(logits[m, :n], hist[m], 0, rep[m], pres[m], freq[m], list(zip(ids[m].tolist(), value[m])),
                                allow[m, :n] if masked else None, np.float32)
        assert np.array_equal(got[m, :n], want) and int(am[m]) == pick
