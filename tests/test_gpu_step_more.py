"""The step operators past what test_gpu_step.py and test_gpu_step_attention.py reach."""
import numpy as np
import pytest

import step_ref
import trellis_quantized_linear_gb300 as tql
from test_gpu_step import Plan, check_norm, norm_inputs, random_requests, run_norm
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


# --------------------------------------------------------------------------- norm


def check_codes(y, codes, group, scale=None):
    """Each code is the nearest one, ties to even, of y / scale: of all that a quotient may be that is 2^-20
    off (fp32: the sum, its product with the weight, the factor 448 / most and the product with it,
    each half a step off, for the value and for the group's largest; the least scale brings the
    root's reciprocal with 2 steps)."""
    scale = step_ref.scales(y, group) if scale is None else scale
    near, far = (step_ref.codes(y * (1 + d), scale, group) for d in (-2.0 ** -20, 2.0 ** -20))
    nan = np.isnan(y)
    assert np.array_equal(codes & 127 == 127, nan)
    assert np.all((codes == near) | (codes == far) | nan)
    assert (near != far).mean() < 2e-3  # hardly ever two choices


@pytest.mark.parametrize("x_type,r_type", [(np.float16, None), (np.float32, np.float32), (np.float16, np.float32)])
@pytest.mark.parametrize("rows,cols,group", [(1, 5120, 128), (40, 256, 256), (40, 640, 64), (333, 1024, 32), (777, 5120, 128), (160, 17408, 17408),
                                             (310, 10240, 64), (40, 32768, 128)])
def test_norm_codes_are_the_nearest(rows, cols, group, x_type, r_type):
    x, r, w = norm_inputs(rows, cols, x_type, r_type, rows + cols)
    if rows > 4:
        x[3] = 0  # of the least scale, with a residual of the least, or without
        x[4] *= np.float16(1e-3)
        if r is not None:
            r[3] = 1e-9
            r[4] *= 1e-6
    got = run_norm(x, r, w, cols, offset=1.0, group=group)
    _, y = step_ref.rms_norm(x, r, w, 1.0, 1e-6)
    check_codes(y, got[2], group)


@pytest.mark.parametrize("rows", [1, 5, 700])
@pytest.mark.parametrize("cols,group", [(256, 64), (256, 256), (1024, 1024), (5120, 128), (8192, 8192)])
def test_norm_codes_of_ties_are_even(rows, cols, group):
    """The row's factor cancels in y / scale: with 448 as the largest value of each group, codes are those of h itself,
    and h in the middle between two of them takes the even one, of either sign."""
    values = step_ref.nearest_code.__globals__["VALUES"][:127]
    middle = (values[1:] + values[:-1]) / 2  # exact in fp16
    x = np.random.default_rng(cols + rows).choice(np.concatenate([middle, -middle, values]), (rows, cols)).astype(np.float16)
    x[:, ::group] = 448.0
    x[1::2, ::group] = -448.0
    got = run_norm(x, None, None, cols, group=group)
    want = step_ref.nearest_code(x.astype(np.float64))
    assert np.array_equal(got[2], want)
    up = np.isin(np.abs(x.astype(np.float64)), middle)
    assert up.any() and np.all(got[2][up] % 2 == 0)


@pytest.mark.parametrize("x_type", [np.float16, np.float32])
def test_norm_codes_of_the_least_scale(x_type):
    """Groups of values below 448 * 2^-40, whose codes are of y * 2^40; of zeros; and of values beside a NaN or an infinity."""
    cols, group = 512, 64
    g = np.random.default_rng(9)
    h = g.standard_normal((6, cols))
    w = np.ones(cols)
    x = h.astype(x_type)
    x[:, :64] = 0
    if x_type is np.float32:
        x[:, 64:128] *= np.float32(1e-12)
        x[:, 128:192] *= np.float32(1e-11)
    x[1, 200], x[2, 300], x[3, 400] = np.nan, np.inf, -np.inf
    got = run_norm(x, None, w.astype(np.float16), cols, group=group)
    _, y = step_ref.rms_norm(x, None, w, 0.0, 1e-6)
    want = step_ref.scales(y, group)
    assert np.all(np.abs(got[3] - want) <= want * 2.0 ** -18)
    rows = [0, 4, 5]
    check_codes(y[rows], got[2][rows], group)
    assert np.all(got[2][1] & 127 == 127)
    for r, at in ((2, 300), (3, 400)):
        assert got[2][r, at] & 127 == 127 and not (np.delete(got[2][r], at) & 127).any()


@pytest.mark.parametrize("rows,cols,x_type,r_type,group", [(608, 512, np.float16, np.float16, 64), (609, 264, np.float16, np.float32, 264), (609, 520, np.float32, None, 0),
                                                           (609, 1024, np.float32, np.float16, 1024), (640, 1024, np.float16, np.float16, 128),
                                                           (700, 512, np.float16, None, 512), (1300, 768, np.float32, np.float32, 32)])
def test_norm_rows_by_warps(rows, cols, x_type, r_type, group):
    """On both sides of four rows an SM, from which on a row of 264 to 1024 columns is a warp's."""
    x, r, w = norm_inputs(rows, cols, x_type, r_type, rows + cols, gap=8)
    got = run_norm(x, r, w, cols, offset=1.0, group=group)
    check_norm(x, r, w, cols, got, offset=1.0, group=group)
