"""The step operators past what test_gpu_step.py and test_gpu_step_attention.py reach."""
import numpy as np
import pytest

import step_ref
import trellis_quantized_linear_gb300 as tql
from test_gpu_step import Plan, random_requests
from test_gpu_step_attention import check, gpu, inputs, split, starts  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads,dim,lens,causal", [(1, 1, 128, [4000], True), (5, 1, 128, [2600, 1200], False), (3, 3, 64, [1500, 1, 2100], True),
                                                            (2, 2, 64, [2400], False)])
def test_shared_items_say_the_same_each_time(heads, kv_heads, dim, lens, causal):
    """Items of 2 and of 4 CTAs, several for each cluster, so that what the CTAs send each other takes the
    place of what was sent before: 60 calls, right once and the same bits always."""
    import torch
    rows, qs = sum(lens), starts(lens)
    x = inputs(rows, heads, kv_heads, dim, 50)
    q, k, v = split(torch.from_numpy(x).cuda(), heads, kv_heads, dim)
    outs = torch.full((60, rows, heads * dim), 7.0, dtype=torch.float16, device="cuda")
    lses = torch.full((60, rows, heads), 7.0, device="cuda")
    start = torch.from_numpy(qs).cuda()
    for out, lse in zip(outs, lses):
        tql.exl3_prompt_attention(q, k, v, heads, kv_heads, dim, start, dim ** -0.5, out, causal=causal, lse=lse)
    torch.cuda.synchronize()
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, 0.0, causal, outs[0].cpu().numpy(), lses[0].cpu().numpy())
    assert torch.all(outs.view(torch.int16) == outs[:1].view(torch.int16)) and torch.all(lses == lses[:1])


# --------------------------------------------------------------------------- plan


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,most,cached", [(32768, 1, 130), (32769, 2, 70), (40000, 3, 200), (65535, 1, 65)])
def test_plan_of_more_sequences_than_a_pass_takes(n, most, cached, in_place):
    """From 32769 on each of the eight CTAs goes through its part several times."""
    p = Plan(*random_requests(n, most, cached, n))
    p.call(in_place)
    p.check()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("where", [0, 4095, 4096, 4999, 5000, 9100, 39999])
@pytest.mark.parametrize("why", ["pages", "rows", "max_rows", "width"])
def test_plan_of_many_stops_at_the_first_that_does_not_fit(where, why, in_place):
    """Before, at and after the ends of passes (4096) and of the CTAs' parts (5000)."""
    t, c = random_requests(40000, 2, 100, 6, ended=0.02)
    t[where], c[where] = 70, 64
    kw = {}
    if why == "rows":
        kw = dict(rows=int(np.maximum(t[:where], 0).sum()) + 69)
    elif why == "max_rows":
        kw = dict(max_rows=69)
    elif why == "width":
        c[where] = 64 * 6 - 69
        kw = dict(max_pages=6)
    p = Plan(t, c, **kw)
    if why == "pages":  # one of the two that it needs
        p.tokens[:] = np.where(p.tokens < 0, 0, p.tokens)
        p.count = 1 + sum(step_ref.blocks(int(x + y)) - step_ref.blocks(int(x)) for x, y in zip(c[:where], t[:where]) if y > 0)
    p.call(in_place)
    p.check()
    assert p.d_served.item() == where
