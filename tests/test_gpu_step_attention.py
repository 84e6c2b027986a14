"""exl3_prompt_attention on the GPU against its formula in 64 bits.

Tolerance: the products' sums are cut at each of their steps (2^-22 of what they hold:
D / 16 steps for a score, tokens / 16 for an output), a probability is off by the error
of its score, by exp2's and a rounding to fp16 (2^-11; the smallest by half of fp16's
least step, 2^-25, where the largest is 2^8 at least: 2^-33 of it), the result by its
own rounding."""
import numpy as np
import pytest

import step_ref
import trellis_quantized_linear_gb300 as tql

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tql.build()
    torch.cuda.set_device(0)
    tql.exl3_init(0)
    yield


def starts(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def inputs(rows, heads, kv_heads, dim, seed, q_gain=2.0, pad=0):
    """Columns of one fused projection, `pad` more between its rows."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, (heads + 2 * kv_heads) * dim + pad))
    x[:, :heads * dim] *= q_gain
    return x.astype(np.float16)


def split(x, heads, kv_heads, dim):
    a, b, c = heads * dim, (heads + kv_heads) * dim, (heads + 2 * kv_heads) * dim
    return x[:, :a], x[:, a:b], x[:, b:c]


def run(x, q_start, heads, kv_heads, dim, scale, cap=0.0, causal=True, stream=None, lse=True, fill=7.0):
    import torch
    xd = torch.from_numpy(x).cuda()
    q, k, v = split(xd, heads, kv_heads, dim)
    out = torch.full((x.shape[0], heads * dim), fill, dtype=torch.float16, device="cuda")
    le = torch.full((x.shape[0], heads), fill, device="cuda") if lse else None
    qs = torch.from_numpy(np.asarray(q_start, dtype=np.int32)).cuda()
    torch.cuda.synchronize()
    tql.exl3_prompt_attention(q, k, v, heads, kv_heads, dim, qs, scale, out, softcap=cap, causal=causal, lse=le, stream=stream)
    torch.cuda.synchronize()
    return out.cpu().numpy(), None if le is None else le.cpu().numpy()


def check(x, q_start, heads, kv_heads, dim, scale, cap, causal, out, lse):
    q, k, v = split(x, heads, kv_heads, dim)
    want, want_lse = step_ref.prompt_attention(q, k, v, q_start, heads, kv_heads, dim, scale, cap, causal)
    # Sum of p |v|, and the largest sum of |q k| that a row's scores are made of
    weight, _ = step_ref.prompt_attention(q, k, np.abs(np.where(np.isfinite(v), v, 0)), q_start, heads, kv_heads, dim, scale, cap, causal)
    g = heads // kv_heads
    for a, z in zip(q_start[:-1], q_start[1:]):
        n = int(z - a)
        if n <= 0:
            continue
        qa, ka = (np.abs(np.nan_to_num(t[a:z].astype(np.float64), posinf=0, neginf=0)).reshape(n, -1, dim) for t in (q, k))
        parts = np.stack([qa[:, h] @ ka[:, h // g].T for h in range(heads)], 1).max(2) * abs(scale)
        off = parts * (dim / 16) * 2.0 ** -22 + 2.0 ** -19 + (2.0 ** -19 * np.minimum(parts, cap) if cap else parts * 2.0 ** -22)
        vmax = np.abs(np.where(np.isfinite(v[a:z]), v[a:z], 0).astype(np.float64)).max(initial=0.0)
        rel = 2.0 ** -11 + (n / 16 + 1) * 2.0 ** -22 + 2 * off
        tol = weight[a:z] * np.repeat(rel, dim, 1) + np.abs(want[a:z]) * 2.0 ** -11 + 2.0 ** -25 + n * 2.0 ** -33 * vmax
        got, w = out[a:z].astype(np.float64), want[a:z]
        fine = np.isfinite(w)
        assert np.array_equal(np.isnan(got), np.isnan(w)) and np.array_equal(got[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)])
        with np.errstate(invalid="ignore"):
            err = np.where(fine, np.abs(got - np.where(fine, w, 0)) - tol, -1)
        assert err.max() <= 0, (a, z, np.unravel_index(err.argmax(), err.shape), err.max())
        if lse is not None:
            gl, wl = lse[a:z].astype(np.float64), want_lse[a:z]
            assert np.array_equal(np.isnan(gl), np.isnan(wl))
            d = np.where(np.isfinite(wl), np.abs(gl - np.where(np.isfinite(wl), wl, 0)) - off - 2.0 ** -21 * np.abs(wl), -1)
            assert d.max() <= 0, (a, z, d.max())
    outside = np.ones(len(out), dtype=bool)
    for a, z in zip(q_start[:-1], q_start[1:]):
        outside[a:max(a, z)] = False
    assert np.all(out[outside] == 7.0) and (lse is None or np.all(lse[outside] == 7.0))
    assert tql.exl3_get_device_status() == 0


SHAPES = [(5, 1, 128), (8, 8, 64), (10, 2, 128), (8, 1, 64), (6, 2, 64), (7, 1, 128), (128, 1, 64), (100, 1, 128)]


@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [127], [128], [129], [61, 0, 1, 64, 300], [255, 256, 257]])
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
def test_lengths_and_heads(lens, heads, kv_heads, dim):
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 1), starts(lens)
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, 0.0, True, out, lse)


@pytest.mark.parametrize("lens", [[1, 5], [130, 128, 2], [700, 33]])
@pytest.mark.parametrize("heads,kv_heads,dim", [(10, 2, 128), (8, 8, 64), (3, 1, 128)])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("causal", [True, False])
def test_caps_and_whole_sequences(lens, heads, kv_heads, dim, cap, causal):
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 2, q_gain=4.0), starts(lens)
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, cap, causal)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, cap, causal, out, lse)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-6, 2.0])
def test_scales(scale):
    x, qs = inputs(390, 4, 2, 64, 3), starts([200, 190])
    out, lse = run(x, qs, 4, 2, 64, scale)
    check(x, qs, 4, 2, 64, scale, 0.0, True, out, lse)


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_of_no_sequence_are_left_and_not_read(dim):
    lens, heads, kv_heads = [100, 29, 200], 6, 2
    rows = sum(lens) + 40
    x, qs = inputs(rows, heads, kv_heads, dim, 4, pad=8), starts(lens, first=17)
    x[:17], x[qs[-1]:] = np.nan, np.inf
    for causal in (True, False):
        out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, causal=causal)
        check(x, qs, heads, kv_heads, dim, dim ** -0.5, 0.0, causal, out, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("at", [[0], [60], [127, 128], [199], [230, 299]])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(causal, what, at):
    lens, heads, kv_heads, dim = [200, 150], 10, 2, 64
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 5), starts(lens)
    for i, r in enumerate(at):
        x[r, (heads + kv_heads) * dim + 3 + 65 * (i % 2)] = what
    x[at[0], -1] = -what
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, causal=causal)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, 0.0, causal, out, lse)


@pytest.mark.parametrize("causal", [True, False])
def test_keys_and_queries_that_are_not_finite(causal):
    lens, heads, kv_heads, dim = [150, 140], 4, 2, 128
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 6), starts(lens)
    x[100, heads * dim + 5] = np.nan   # a key of the first sequence, first key head
    x[200, 3] = np.nan                 # one query row
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, causal=causal)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, 0.0, causal, out, lse)


@pytest.mark.parametrize("cap", [0.0, 3.0])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,at", [([200, 140], [5, 250]), ([400], [130]), ([1, 300], [1, 300])])
def test_infinite_scores(cap, causal, lens, at):
    """An infinite key: a score of infinity for half of the rows that see it (NaN), of minus
    infinity for the others (no part in the sum); capped, plus and minus the cap."""
    heads, kv_heads, dim = 6, 2, 64
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 21), starts(lens)
    g = np.random.default_rng(3)
    d = np.arange(heads) * dim + 9
    x[:, d] = np.where(g.random((len(x), heads)) < 0.5, 1, -1) * (np.abs(x[:, d]) + 0.25)
    for r in at:
        x[r, d] = np.abs(x[r, d])  # else a row that sees nothing else has no score
        x[r, heads * dim + 9::dim][:kv_heads] = np.inf
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, cap, causal)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, cap, causal, out, lse)


def test_a_row_of_minus_infinity_alone():
    x = inputs(131, 2, 1, 64, 22)
    x[:, 5] = -1.0              # first head
    x[:, 2 * 64 + 5] = np.inf   # every key
    out, lse = run(x, [0, 1, 131], 2, 1, 64, 0.125)
    assert not out[:, :64].any() and np.all(lse[:, 0] == -np.inf)


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 0.5, 8.0, 30.0, 1e38])
@pytest.mark.parametrize("q_gain", [0.1, 3.0, 60.0])
def test_caps_far_below_and_far_above_the_scores(cap, q_gain):
    x, qs = inputs(700, 6, 2, 128, 23, q_gain=q_gain), starts([500, 200])
    x[::7, :6 * 128] /= 16  # rows of small scores beside those of large ones
    out, lse = run(x, qs, 6, 2, 128, 128 ** -0.5, cap)
    check(x, qs, 6, 2, 128, 128 ** -0.5, cap, True, out, lse)


@pytest.mark.parametrize("heads,kv_heads,dim,lens", [(4, 2, 128, [1500, 3, 700]), (12, 2, 64, [1100, 1024])])
def test_long_whole_sequences(heads, kv_heads, dim, lens):
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 24), starts(lens)
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, 20.0, causal=False)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, 20.0, False, out, lse)


# Few heads and long sequences: CTAs share an item's keys and join what they have of its rows.
FEW = [(1, 1, 128), (1, 1, 64), (3, 3, 64), (5, 1, 128), (8, 2, 64), (8, 8, 128)]


@pytest.mark.parametrize("lens", [[1024], [1153], [1600, 900], [2100, 1, 1000]])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("heads,kv_heads,dim", FEW)
def test_few_heads(heads, kv_heads, dim, cap, causal, lens):
    x, qs = inputs(sum(lens) + 5, heads, kv_heads, dim, 30, q_gain=3.0), starts(lens, first=2)
    x[:2], x[qs[-1]:] = np.nan, np.inf
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, cap, causal)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, cap, causal, out, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 128), (4, 2, 64), (8, 8, 128)])
def test_few_heads_values_that_are_not_finite(heads, kv_heads, dim, causal):
    lens = [1500, 1300]
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 31), starts(lens)
    for i, r in enumerate([0, 700, 1279, 1280, 1499, 1500, 2600]):
        x[r, (heads + kv_heads) * dim + 5 * i] = [np.inf, -np.inf, np.nan][i % 3]
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5, causal=causal)
    q, k, v = split(x, heads, kv_heads, dim)
    want, _ = step_ref.prompt_attention(q, k, v, qs, heads, kv_heads, dim, dim ** -0.5, 0.0, causal)
    fine = np.isfinite(want)
    # a row that sees one gets it or NaN there, and all else is as if it were not there
    assert np.array_equal(np.isfinite(out), fine)
    clean, clean_lse = run(np.where(np.isfinite(x), x, 0).astype(np.float16), qs, heads, kv_heads, dim, dim ** -0.5, causal=causal)
    assert np.array_equal(out[fine], clean[fine]) and np.array_equal(lse, clean_lse)
    assert tql.exl3_get_device_status() == 0


def test_few_heads_growing_scores_and_rows_without_any():
    """References that differ by far between the CTAs of an item; keys whose scores are minus
    infinity for a CTA's whole range, and for all."""
    heads, kv_heads, dim = 2, 1, 64
    x, qs = inputs(1400, heads, kv_heads, dim, 32), starts([1400])
    x[:, :heads * dim] = np.abs(x[:, :heads * dim])
    k = slice(heads * dim, (heads + 1) * dim)
    grow = (np.arange(1400)[:, None] / 50.0 + 0.1 * np.abs(x[:, k])).astype(np.float16)
    for keys in (grow, grow[::-1]):
        x[:, k] = keys
        for scale in (0.125, -0.125):
            out, lse = run(x, qs, heads, kv_heads, dim, scale)
            check(x, qs, heads, kv_heads, dim, scale, 0.0, True, out, lse)
    x[:, 3], x[:, dim + 3] = -1.0, -1.0
    x[600:, heads * dim + 3] = np.inf  # minus infinity
    out, lse = run(x, qs, heads, kv_heads, dim, 0.125, causal=False)
    check(x, qs, heads, kv_heads, dim, 0.125, 0.0, False, out, lse)
    x[:, heads * dim + 3] = np.inf
    out, lse = run(x, qs, heads, kv_heads, dim, 0.125)
    assert not out.any() and np.all(lse == -np.inf)


@pytest.mark.parametrize("heads,kv_heads,dim,lens", [(1, 1, 128, [2500]), (8, 8, 64, [1500]), (6, 3, 128, [1024, 1400])])
def test_few_heads_twice_at_once_and_captured(heads, kv_heads, dim, lens):
    import torch
    rows, qs = sum(lens), torch.from_numpy(starts(lens)).cuda()
    xs = [torch.from_numpy(inputs(rows, heads, kv_heads, dim, 33 + i)).cuda() for i in range(2)]
    outs = [[(torch.zeros((rows, heads * dim), dtype=torch.float16, device="cuda"), torch.zeros((rows, heads), device="cuda")) for _ in range(7)] for _ in range(2)]

    def go(i, o, stream=None):
        tql.exl3_prompt_attention(*split(xs[i], heads, kv_heads, dim), heads, kv_heads, dim, qs, dim ** -0.5, outs[i][o][0], lse=outs[i][o][1], stream=stream)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o in range(5):
        for i in range(2):
            go(i, o, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        go(i, 5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(2):
            go(i, 6)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in outs[i][1:]:
            assert torch.equal(out, outs[i][0][0]) and torch.equal(lse, outs[i][0][1])
    assert tql.exl3_get_device_status() == 0


@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 1, 64), (1, 1, 128), (8, 8, 64)])
def test_few_heads_captured_call_serves_other_lengths(heads, kv_heads, dim):
    """The rows that a call has room for say how many CTAs share an item; the lengths may be any."""
    import torch
    rows = 4000
    x = inputs(rows, heads, kv_heads, dim, 35)
    xd = torch.from_numpy(x).cuda()
    out, lse = torch.empty((rows, heads * dim), dtype=torch.float16, device="cuda"), torch.empty((rows, heads), device="cuda")
    qs = torch.zeros(4, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tql.exl3_prompt_attention(*split(xd, heads, kv_heads, dim), heads, kv_heads, dim, qs, dim ** -0.5, out, lse=lse)
    for lens in ([1500, 0, 1200], [1, 2, 3], [0, 0, 0], [129, 700, 64], [0, 1281, 0], [385, 513, 641]):
        s = starts(lens)
        qs.copy_(torch.from_numpy(s))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(x, s, heads, kv_heads, dim, dim ** -0.5, 0.0, True, out.cpu().numpy(), lse.cpu().numpy())
    qs.copy_(torch.tensor([100, 1200, 1100, 5000], dtype=torch.int32))  # a good range and two that are none
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert tql.exl3_get_device_status() == 10
    check(x[100:1200], [0, 1100], heads, kv_heads, dim, dim ** -0.5, 0.0, True, out.cpu().numpy()[100:1200], lse.cpu().numpy()[100:1200])
    assert torch.all(out[:100] == 7.0) and torch.all(out[1200:] == 7.0)


def test_heavy_and_growing_scores():
    """Maxima that grow along a row, so that its output is rescaled again and again."""
    lens, heads, kv_heads, dim = [1000], 2, 1, 64
    x, qs = inputs(1000, heads, kv_heads, dim, 7), starts(lens)
    x[:, :heads * dim] = np.abs(x[:, :heads * dim])
    x[:, heads * dim:(heads + 1) * dim] = (np.arange(1000)[:, None] / 100.0 + 0.1 * np.abs(x[:, heads * dim:(heads + 1) * dim])).astype(np.float16)
    for scale in (0.125, -0.125, 0.01):
        out, lse = run(x, qs, heads, kv_heads, dim, scale)
        check(x, qs, heads, kv_heads, dim, scale, 0.0, True, out, lse)


def test_more_sequences_than_one_launch_takes():
    lens = [1 + i % 3 for i in range(2100)]
    x, qs = inputs(sum(lens), 2, 1, 64, 8), starts(lens)
    for causal in (True, False):
        out, lse = run(x, qs, 2, 1, 64, 0.125, causal=causal)
        check(x, qs, 2, 1, 64, 0.125, 0.0, causal, out, lse)


@pytest.mark.parametrize("heads,kv_heads,dim,lens", [(2, 1, 128, [5000]), (16, 2, 64, [2500, 1, 1300]), (1, 1, 64, [4097, 4096])])
def test_long(heads, kv_heads, dim, lens):
    x, qs = inputs(sum(lens), heads, kv_heads, dim, 9), starts(lens)
    out, lse = run(x, qs, heads, kv_heads, dim, dim ** -0.5)
    check(x, qs, heads, kv_heads, dim, dim ** -0.5, 0.0, True, out, lse)


def test_without_lse_and_on_another_stream():
    import torch
    x, qs = inputs(300, 4, 4, 128, 10), starts([300])
    a, _ = run(x, qs, 4, 4, 128, 0.1, lse=False)
    b, _ = run(x, qs, 4, 4, 128, 0.1, stream=torch.cuda.Stream())
    assert np.array_equal(a, b)


@pytest.mark.parametrize("q_start,good", [([20, 10, 300], [(10, 300)]), ([0, 100, 301], [(0, 100)]), ([-5, 100, 200], [(100, 200)])])
def test_ranges_outside_the_rows_are_reported_and_left_out(q_start, good):
    heads, kv_heads, dim = 4, 2, 64
    x = inputs(300, heads, kv_heads, dim, 11)
    out, lse = run(x, q_start, heads, kv_heads, dim, 0.125)
    assert tql.exl3_get_device_status() == 10
    for a, z in good:
        check(x[a:z], [0, z - a], heads, kv_heads, dim, 0.125, 0.0, True, out[a:z], lse[a:z])
    if len(q_start) == 3:
        a, z = good[0]
        assert np.all(out[:a] == 7.0) and np.all(out[z:] == 7.0)


def test_past_32_bit_offsets():
    """Queries, keys, values and outputs in the last columns of a matrix of more than 2^31 elements."""
    import torch
    heads, kv_heads, dim, rows, ld = 4, 2, 64, 2100, 1 << 20
    x = torch.from_numpy(inputs(rows, heads, kv_heads, dim, 14)).cuda()
    qs = torch.tensor([0, 1200, rows], dtype=torch.int32, device="cuda")
    want = torch.empty((rows, heads * dim), dtype=torch.float16, device="cuda")
    tql.exl3_prompt_attention(*split(x, heads, kv_heads, dim), heads, kv_heads, dim, qs, 0.125, want)
    big = torch.zeros((rows, ld), dtype=torch.float16, device="cuda")
    big[:, -x.shape[1]:] = x
    out = big[:, -x.shape[1] - heads * dim:-x.shape[1]]
    tql.exl3_prompt_attention(*split(big[:, -x.shape[1]:], heads, kv_heads, dim), heads, kv_heads, dim, qs, 0.125, out)
    assert torch.equal(out, want) and torch.equal(big[:, -x.shape[1]:], x) and not big[:, :-x.shape[1] - heads * dim].any()


def test_captured_call_serves_other_lengths():
    import torch
    heads, kv_heads, dim, rows = 10, 2, 128, 700
    x = inputs(rows, heads, kv_heads, dim, 12)
    xd = torch.from_numpy(x).cuda()
    q, k, v = split(xd, heads, kv_heads, dim)
    out, lse = torch.empty((rows, heads * dim), dtype=torch.float16, device="cuda"), torch.empty((rows, heads), device="cuda")
    qs = torch.tensor([0, 0, 0, 0], dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tql.exl3_prompt_attention(q, k, v, heads, kv_heads, dim, qs, 0.09, out, lse=lse)
    for lens in ([700, 0, 0], [1, 600, 99], [0, 0, 5], [128, 128, 128]):
        s = starts(lens)
        qs.copy_(torch.from_numpy(s))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(x, s, heads, kv_heads, dim, 0.09, 0.0, True, out.cpu().numpy(), lse.cpu().numpy())


def test_two_calls_at_once_and_the_same_twice():
    import torch
    xs = [inputs(600, 8, 2, 64, 13 + i) for i in range(2)]
    qs = starts([400, 200])
    want = [run(x, qs, 8, 2, 64, 0.125) for x in xs]
    dev = [torch.from_numpy(x).cuda() for x in xs]
    qd = torch.from_numpy(qs).cuda()
    outs = [[torch.empty((600, 512), dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(10)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o in outs:
        for i in range(2):
            tql.exl3_prompt_attention(*split(dev[i], 8, 2, 64), 8, 2, 64, qd, 0.125, o[i], stream=streams[i])
    torch.cuda.synchronize()
    for o in outs:
        for i in range(2):
            assert np.array_equal(o[i].cpu().numpy(), want[i][0])
