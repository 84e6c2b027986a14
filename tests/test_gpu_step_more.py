"""The step operators past what test_gpu_step.py and test_gpu_step_attention.py reach."""
import numpy as np
import pytest

import trellis_quantized_linear_gb300 as tql
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
