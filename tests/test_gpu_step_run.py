"""The step operators together with the projections, the cache and its attention, as
examples/serve_requests.py runs them: each stage of a prompt step against its formula in 64
bits on what the stage before left, captured steps against eager ones, pages that come and
go, and a token through the cache against the same token in a prompt."""
import importlib.util
import os

import numpy as np
import pytest

import step_ref
import trellis_quantized_linear_gb300 as tql

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("serve_requests", os.path.join(ROOT, "examples", "serve_requests.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    torch.cuda.set_device(0)
    return m


def prompts(example, lens, seed=0):
    g = np.random.default_rng(seed)
    return {slot: g.integers(0, example.VOCAB, n).tolist() for slot, n in lens.items()}


def test_stages_of_a_prompt_step(example, monkeypatch):
    """Every call's inputs and outputs are recorded, and its outputs compared with what
    its formula makes of its inputs. fp16 results: half a step and 2^-9 of the largest
    value that they are made of (sums of up to 200 probabilities with 11 bits)."""
    import torch
    seen = []

    def record(name, outputs):
        real = getattr(tql, name)

        def call(*a, **k):
            before = [x.clone() if isinstance(x, torch.Tensor) else x for x in a], {n: x.clone() if isinstance(x, torch.Tensor) else x for n, x in k.items()}
            real(*a, **k)
            seen.append((name, *before, [x.clone() for x in outputs(a, k) if x is not None]))
        monkeypatch.setattr(tql, name, call)

    record("exl3_rms_norm", lambda a, k: (a[1], k.get("residual_out")))
    record("exl3_qk_rotary", lambda a, k: (a[1],))
    record("exl3_prompt_attention", lambda a, k: (a[8],))
    e = example.Engine(4, 24, 512)
    lens = {0: 130, 2: 1, 3: 70}
    w = e.prompts(prompts(example, lens))
    torch.cuda.synchronize()
    assert e.kv_len.tolist() == [130, 0, 1, 70] and e.q_start.tolist() == [0, 130, 130, 131, 201] and e.served.item() == 4
    assert w["position"].tolist() == list(range(130)) + [0] + list(range(70))
    assert [n for n, *_ in seen].count("exl3_prompt_attention") == example.LAYERS

    def n(t):
        return t.double().cpu().numpy()

    for name, a, k, out in seen:
        if name == "exl3_rms_norm":
            r = k.get("residual")
            h, y = step_ref.rms_norm(n(a[0]), None if r is None else n(r), n(k["weight"]), 0.0, 1e-6)
            assert np.all(np.abs(n(out[0]) - y) <= np.abs(y) * (2.0 ** -11 + 2.0 ** -18) + 2.0 ** -25)
            if r is not None:
                assert np.all(np.abs(n(out[1]) - h) <= np.abs(h) * 2.0 ** -10 + 2.0 ** -25)
        elif name == "exl3_qk_rotary":
            want = step_ref.rotary(n(a[0])[:, :example.K], example.HEADS, example.KV_HEADS, example.DIM, a[5].tolist(), n(a[6]), False,
                                   n(k["q_weight"]), n(k["k_weight"]), 1e-6, 0.0)
            assert np.all(np.abs(n(out[0])[:, :example.K] - want) <= np.abs(want) * 2.0 ** -11 + np.abs(want).max() * 2.0 ** -20)
            assert np.array_equal(n(out[0])[:, example.K:], n(a[0])[:, example.K:])
        else:
            want, _ = step_ref.prompt_attention(n(a[0]), n(a[1]), n(a[2]), a[6].tolist(), example.HEADS, example.KV_HEADS, example.DIM, a[7], 0.0, True)
            assert np.all(np.abs(n(out[0]) - want) <= np.abs(want) * 2.0 ** -11 + np.abs(n(a[2])).max() * 2.0 ** -9)
    assert tql.exl3_get_device_status() == 0


def test_captured_steps_say_what_eager_steps_say(example):
    eager, graph = example.main(graph=False), example.main(graph=True)
    assert eager == graph
    said, free, status = graph
    assert status == 0 and free == 24
    assert [len(s) for s in said] == [5 + 11 * i % 17 for i in range(7)]
    assert all(0 <= t < example.VOCAB for s in said for t in s)


def test_pages_come_and_go(example):
    e = example.Engine(4, 12, 1024)
    p = prompts(example, {0: 200, 1: 64, 2: 65, 3: 1})
    e.prompts(p)
    used = e.table.cpu().numpy()
    assert e.free_count.item() == 12 - (4 + 1 + 2 + 1)
    held = [used[s, :b].tolist() for s, b in ((0, 4), (1, 1), (2, 2), (3, 1))]
    pages = sum(held, [])
    assert len(set(pages)) == 8 and set(pages) | set(e.free[:4].tolist()) == set(range(12))
    e.step([1, 2, 3])  # the 65th token of slot 1 needs a page
    assert e.free_count.item() == 3 and e.kv_len.tolist() == [200, 65, 66, 2]
    e.ended([0, 2])
    assert e.free_count.item() == 9 and e.kv_len.tolist() == [0, 65, 0, 2]
    e.prompts(prompts(example, {0: 512, 2: 60}))
    assert e.served.item() == 4 and e.free_count.item() == 0
    e.step([0, 1, 2, 3])  # slot 0's table is full: from it on, nobody is served
    assert e.served.item() == 0 and e.kv_len.tolist() == [512, 65, 60, 2] and e.free_count.item() == 0
    t = e.table.cpu().numpy()
    now = t[0, :8].tolist() + t[1, :2].tolist() + t[2, :1].tolist() + t[3, :1].tolist()
    assert sorted(now) == list(range(12))
    assert tql.exl3_get_device_status() == 0


def test_a_token_through_the_cache_and_in_a_prompt(example):
    """The last of n tokens as a step behind n - 1 cached ones and at the end of a prompt:
    E4M3 keeps 3 bits, so scores of rms 1 move by a few hundredths and outputs by a few percent."""
    import torch
    ids = prompts(example, {1: 150})[1]
    a, b = example.Engine(3, 12, 512), example.Engine(3, 12, 512)
    w = a.prompts({1: ids})
    whole = w["normed"][149].double()
    b.prompts({1: ids[:-1]})
    b.last[1] = ids[-1]
    b.step([1], graph=False)
    torch.cuda.synchronize()
    through = b.step_work["normed"][0].double()
    assert float((through - whole).norm() / whole.norm()) < 0.2
    assert tql.exl3_get_device_status() == 0
