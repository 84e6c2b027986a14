"""The serving loop of examples/serve_step.py: a captured step gives the tokens of an
eager one, through an eviction, and the layer's attention agrees with plain attention
over the same projections."""
import importlib.util
import os

import numpy as np
import pytest

import trellis_quantized_linear_gb300 as tql

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("serve_step", os.path.join(ROOT, "examples", "serve_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_captured_steps_say_what_eager_steps_say(example):
    eager, graph = example.main(graph=False), example.main(graph=True)
    assert eager == graph
    said, lengths, status = graph
    assert status == 0 and lengths == [150 + 12] * 3
    assert all(0 <= t < example.VOCAB for step in said for t in step)


def test_layer_attention_agrees_with_plain_attention(example):
    """Prompt rows through the 8-bit cache against fp64 attention over the unquantized
    keys and values of the same projection: E4M3 keeps 3 bits, 2^-4 relative at most,
    so scores of rms 1 move by a few hundredths and outputs by a few percent."""
    import torch
    layer = example.Layer(n_seqs=2, max_tokens=320, max_rows=400)
    tokens = torch.randint(0, example.VOCAB, (2, 150), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    layer.kv_len += 150
    b = layer.batch(150)
    layer.mix(b, layer.embed[tokens.reshape(-1).long()])
    torch.cuda.synchronize()
    H, K, D = example.HEADS, example.KV_HEADS, example.DIM
    qkv = b.work["qkv"].double().cpu().numpy().reshape(2, 150, H + 2 * K, D)
    got = b.work["mixed"].double().cpu().numpy().reshape(2, 150, H, D)
    for s in range(2):
        for h in range(H):
            q, k, v = qkv[s, :, h], qkv[s, :, H + h // (H // K)], qkv[s, :, H + K + h // (H // K)]
            x = 50.0 * np.tanh(q @ k.T * D ** -0.5 / 50.0)
            x[np.triu_indices(150, 1)] = -np.inf
            p = np.exp(x - x.max(1, keepdims=True))
            want = (p / p.sum(1, keepdims=True)) @ v
            err = np.linalg.norm(got[s, :, h] - want) / np.linalg.norm(want)
            assert err < 0.2, (s, h, err)
    assert tql.exl3_get_device_status() == 0
