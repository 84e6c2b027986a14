"""exl3_prompt_attention where scores are far from those of a normed model: so large that a
step of fp32 is larger than the softmax's range.

Queries and keys of small whole numbers, times powers of two: products are exact in fp32, and
those of different keys so far apart that a row's weights are 1 / n on the n keys of its largest
score and 0 elsewhere. Tolerance: a probability's rounding to fp16 (2^-11), the sums' steps as in
test_gpu_step_attention.py, the result's own rounding; lse by a few roundings of fp32."""
import numpy as np
import pytest

import step_ref
import trellis_quantized_linear_gb300 as tql
from test_gpu_step_attention import check, gpu, inputs, run, split, starts  # noqa: F401

pytestmark = pytest.mark.gpu


def whole_numbers(rows, heads, kv_heads, dim, seed, q_size=1.0, k_size=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, (heads + 2 * kv_heads) * dim))
    qk = (heads + kv_heads) * dim
    x[:, :qk] = g.integers(-2, 3, (rows, qk))
    x[:, :heads * dim] *= q_size
    x[:, heads * dim:qk] *= k_size
    assert np.abs(x).max() < 65504
    return x.astype(np.float16)


def check_choice(x, qs, heads, kv_heads, dim, scale, causal, out, lse):
    q, k, v = split(x, heads, kv_heads, dim)
    want, want_lse = step_ref.prompt_attention(q, k, v, qs, heads, kv_heads, dim, scale, 0.0, causal)
    size, _ = step_ref.prompt_attention(q, k, np.abs(v), qs, heads, kv_heads, dim, scale, 0.0, causal)
    n = max(b - a for a, b in zip(qs[:-1], qs[1:]))
    tol = size * (2.0 ** -11 + (n / 16 + 1) * 2.0 ** -22) + np.abs(want) * 2.0 ** -11 + 2.0 ** -25
    assert np.all(np.abs(out.astype(np.float64) - want) <= tol)
    assert np.all(np.abs(lse.astype(np.float64) - want_lse) <= np.abs(want_lse) * 2.0 ** -21 + 2.0 ** -19)
    assert tql.exl3_get_device_status() == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,kv_heads,dim,lens", [(6, 2, 64, [300, 1, 150]), (5, 1, 128, [130, 260]), (1, 1, 128, [1500]), (4, 4, 64, [1600])])
@pytest.mark.parametrize("size,scale", [(4096.0, None), (8192.0, 1.0), (1.0, 2.0 ** 12), (1.0, 2.0 ** 21), (1.0, -2.0 ** 27), (1.0, 1e10), (1.0, -1e30)])
def test_scores_larger_than_the_range_of_the_softmax(heads, kv_heads, dim, lens, size, scale, causal):
    """Queries and keys near fp16's largest at the usual scale, and scales of any size."""
    scale = dim ** -0.5 if scale is None else scale
    x, qs = whole_numbers(sum(lens), heads, kv_heads, dim, 41, size, size), starts(lens)
    out, lse = run(x, qs, heads, kv_heads, dim, scale, causal=causal)
    check_choice(x, qs, heads, kv_heads, dim, scale, causal, out, lse)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (40, 8, 128), (1, 1, 128)])
@pytest.mark.parametrize("back", [False, True])
def test_scores_that_grow_along_the_sequence(heads, kv_heads, dim, back):
    """From hundreds to 2^30 within a row, and the other way round: references of both kinds, one after the other."""
    rows = 1400
    x, qs = whole_numbers(rows, heads, kv_heads, dim, 42, 16.0), starts([rows])
    keys = slice(heads * dim, (heads + kv_heads) * dim)
    grow = 2.0 ** (np.arange(rows) // 128)
    x[:, keys] *= (grow[::-1] if back else grow)[:, None].astype(np.float16)
    out, lse = run(x, qs, heads, kv_heads, dim, 128.0)
    check_choice(x, qs, heads, kv_heads, dim, 128.0, True, out, lse)


@pytest.mark.parametrize("heads,kv_heads,dim,rows", [(6, 2, 64, 700), (1, 1, 128, 1500)])
def test_rows_of_large_scores_beside_usual_ones(heads, kv_heads, dim, rows):
    x, qs = inputs(rows, heads, kv_heads, dim, 43), starts([rows])
    x[::3, :heads * dim] = np.sign(x[::3, :heads * dim]) * np.float16(30000)
    x[:, heads * dim:(heads + kv_heads) * dim] *= np.float16(2)
    for causal in (True, False):
        out, lse = run(x, qs, heads, kv_heads, dim, 2.0, causal=causal)
        few = np.arange(rows) % 3 > 0
        assert np.all(np.isfinite(out)) and np.all(np.isfinite(lse))
        usual = np.where(few[:, None], x, 0).astype(np.float16)
        usual[:, heads * dim:] = x[:, heads * dim:]
        want, want_lse = run(usual, qs, heads, kv_heads, dim, 2.0, causal=causal)
        check(usual, qs, heads, kv_heads, dim, 2.0, 0.0, causal, np.where(few[:, None], out, want), np.where(few[:, None], lse, want_lse))


@pytest.mark.parametrize("heads,kv_heads,dim,rows", [(6, 2, 64, 300), (1, 1, 128, 1500)])
@pytest.mark.parametrize("scale,cap", [(1e30, 1e-30), (-1e30, 1e-28), (3.4e38, 0.0), (-3.4e38, 0.0), (3.4e38, 30.0), (3.4e38, 1e38)])
def test_scores_of_zero_stay_zero_beside_any_scale(heads, kv_heads, dim, rows, scale, cap):
    """Also where scale / cap or the scale in log2 units leaves fp32."""
    x, qs = inputs(rows, heads, kv_heads, dim, 44), starts([rows])
    x[:, :heads * dim] = 0
    x[:, 1:heads * dim:2] = -0.0
    for causal in (True, False):
        out, lse = run(x, qs, heads, kv_heads, dim, scale, cap, causal)
        check(x, qs, heads, kv_heads, dim, scale, cap, causal, out, lse)
