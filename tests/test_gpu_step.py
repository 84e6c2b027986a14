"""exl3_kv8_plan, exl3_rms_norm and exl3_qk_rotary on the GPU against their definitions
in 64 bits (whole numbers equal). Tolerances: half a step of the result's type, and what
fp32 sums of up to 32768 squares and a few products may be off (2^-18 of a value)."""
import numpy as np
import pytest

import step_ref
import trellis_quantized_linear_gb300 as tql

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tql.build()
    torch.cuda.set_device(0)
    tql.exl3_init(0)
    yield


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# --------------------------------------------------------------------------- plan


class Plan:
    """Sequences whose first blocks hold distinct pages, and a stack of the others."""

    def __init__(self, tokens, cached, max_pages=None, rows=None, max_rows=None, spare=5, capacity=None, seed=0):
        self.tokens, self.cached = np.array(tokens, dtype=np.int32), np.array(cached, dtype=np.int32)
        n = len(tokens)
        have = [step_ref.blocks(int(np.clip(c, 0, 1 << 20))) for c in cached]
        self.max_pages = max([step_ref.blocks(int(c + max(t, 0))) for t, c in zip(tokens, cached)] + [0]) if max_pages is None else max_pages
        total = int(sum(max(t, 0) for t in tokens))
        self.rows = total + 3 if rows is None else rows
        self.max_rows = max([max(t, 0) for t in tokens] + [0]) if max_rows is None else max_rows
        need = sum(step_ref.blocks(c + t) - step_ref.blocks(c) for t, c in zip(tokens, cached) if t > 0)
        self.n_pages = max(1, sum(have) + need + spare)
        pages = np.random.default_rng(seed).permutation(self.n_pages).astype(np.int32)
        self.table = np.full((n, self.max_pages), -7, dtype=np.int32)
        at = 0
        for s, h in enumerate(have):
            h = min(h, self.max_pages)
            self.table[s, :h] = pages[at:at + h]
            at += h
        self.count = self.n_pages - at
        self.stack = np.full(self.n_pages if capacity is None else capacity, -9, dtype=np.int32)
        self.count = min(self.count, len(self.stack))
        self.stack[:self.count] = pages[at:at + self.count]

    def call(self, in_place=False, stream=None):
        import torch
        n = len(self.tokens)
        d = dict(dtype=torch.int32, device="cuda")
        self.d_table, self.d_stack, self.d_count = dev(self.table), dev(self.stack), dev(np.array([self.count], dtype=np.int32))
        self.d_cached, self.d_tokens = dev(self.cached), dev(self.tokens)
        self.d_kv_len = self.d_cached if in_place else torch.full((n,), -3, **d)
        self.d_left = self.d_count if in_place else torch.full((1,), -3, **d)
        self.d_start, self.d_pos, self.d_slot, self.d_served = (torch.full((k,), -3, **d) for k in (n + 1, self.rows, self.rows, 1))
        self.batch = tql.Exl3Kv8Batch(self.d_table, self.d_kv_len, self.d_start, self.rows, self.max_rows)
        torch.cuda.synchronize()
        self.again(stream)
        torch.cuda.synchronize()

    def again(self, stream=None):
        tql.exl3_kv8_plan(self.batch, self.d_tokens, self.d_cached, self.d_stack, self.d_count, self.d_left, self.n_pages, self.d_pos,
                          self.d_slot, self.d_served, stream=stream)

    def check(self):
        table, stack = self.table.copy(), self.stack.copy()
        kv_len, start, pos, slot, served, left, bad = step_ref.plan(self.tokens, self.cached, table, stack, self.count, self.n_pages, self.rows, self.max_rows)
        for name, got, want in (("kv_len", self.d_kv_len, kv_len), ("q_start", self.d_start, start), ("position", self.d_pos, pos),
                                ("slot", self.d_slot, slot), ("served", self.d_served, [served]), ("left", self.d_left, [left]),
                                ("table", self.d_table, table), ("stack", self.d_stack, stack)):
            assert np.array_equal(got.cpu().numpy(), np.asarray(want, dtype=np.int32).reshape(got.shape)), name
        assert tql.exl3_get_device_status() == (10 if bad else 0)


def random_requests(n, most, cached, seed, ended=0.1, none=0.1):
    g = np.random.default_rng(seed)
    t = g.integers(1, most + 1, n)
    u = g.random(n)
    t = np.where(u < ended, -1, np.where(u < ended + none, 0, t))
    return t, np.where(g.random(n) < 0.2, 0, g.integers(0, cached + 1, n))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,most,cached", [(1, 1, 0), (1, 5, 63), (1, 5000, 64), (3, 200, 128), (33, 1, 500), (70, 130, 4000), (1024, 3, 200),
                                           (1025, 20, 70), (5000, 2, 300), (11264, 2, 100), (11265, 1, 65), (20000, 1, 3)])
def test_plan(n, most, cached, in_place):
    p = Plan(*random_requests(n, most, cached, n))
    p.call(in_place)
    p.check()


def test_plan_of_nothing():
    for tokens, cached in (([], []), ([0, 0], [5, 0]), ([-1, -1], [70, 0]), ([0], [0])):
        p = Plan(tokens, cached)
        p.call()
        p.check()
    p = Plan([], [], rows=0)
    p.call()
    p.check()


def test_plan_twice_gives_the_same():
    p = Plan(*random_requests(300, 40, 900, 1))
    p.call()
    p.again()
    p.check()


@pytest.mark.parametrize("where", [0, 1, 511, 1023, 1024, 1500, 2999])
@pytest.mark.parametrize("why", ["pages", "rows", "max_rows", "width"])
def test_plan_stops_at_the_first_that_does_not_fit(where, why):
    t, c = random_requests(3000, 3, 300, 5, ended=0.05)
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
    if why == "pages":  # as many as those before it need beside what comes back, and one of its own two
        back = sum(step_ref.blocks(int(x)) for x, y in zip(c, t) if y < 0)
        need = sum(step_ref.blocks(int(x + y)) - step_ref.blocks(int(x)) for x, y in zip(c[:where], t[:where]) if y > 0)
        if need + 1 - back < 0:
            p.tokens[:] = np.where(p.tokens < 0, 0, p.tokens)
            back = 0
        p.count = need + 1 - back
    p.call()
    p.check()
    assert p.d_served.item() == where


def test_plan_reports_what_is_out_of_range():
    for change in ("cached", "cached_long", "cached_ended", "page", "stack_page", "count", "count_negative", "capacity"):
        p = Plan([5, 60, 1, -1, 3], [10, 64, 100, 130, 0])
        if change == "cached":
            p.cached[2] = -4
        elif change == "cached_long":
            p.cached[1] = 64 * p.max_pages + 1
        elif change == "cached_ended":
            p.cached[3] = -1
        elif change == "page":
            p.table[0, 0] = p.n_pages
        elif change == "stack_page":
            p.stack[p.count - 1] = -1
            p.tokens[3] = 0
        elif change == "count":
            p.count = len(p.stack) + 1
        elif change == "count_negative":
            p.count = -1
        else:
            p.stack = p.stack[:p.count + 2].copy()
        p.call()
        p.check()
        assert p.d_served.item() in (5, 2, 1, 3)


def test_plan_captured_steps():
    """Steps of a graph: kv_len and the stack's count stay where they are and go on."""
    import torch
    p = Plan([1] * 40, [0] * 40, max_pages=4, spare=200)
    n = 40
    kv_len, count = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.tensor([p.count], dtype=torch.int32, device="cuda")
    table, stack, tokens = dev(p.table), dev(p.stack), dev(p.tokens)
    rows = 100
    start, pos, slot, served = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (n + 1, rows, rows, 1))
    batch = tql.Exl3Kv8Batch(table, kv_len, start, rows, 70)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tql.exl3_kv8_plan(batch, tokens, kv_len, stack, count, count, p.n_pages, pos, slot, served)
    r = np.random.default_rng(3)
    c, t_h, s_h, k_h = p.count, p.table.copy(), p.stack.copy(), np.zeros(n, dtype=np.int32)
    for _ in range(30):
        t = r.integers(-1, 4, n).astype(np.int32)
        t[r.integers(0, n)] = 40
        tokens.copy_(dev(t))
        g.replay()
        k, q, po, sl, sv, c, bad = step_ref.plan(t, k_h, t_h, s_h, c, p.n_pages, rows, 70)
        k_h = np.array(k, dtype=np.int32)
        torch.cuda.synchronize()
        for got, want in ((kv_len, k), (start, q), (pos, po), (slot, sl), (served, [sv]), (count, [c]), (table, t_h), (stack, s_h)):
            assert np.array_equal(got.cpu().numpy(), np.asarray(want).reshape(got.shape))
        assert not bad
    assert tql.exl3_get_device_status() == 0


# --------------------------------------------------------------------------- norm


def norm_inputs(rows, cols, x_type, r_type, seed, weight=True, gap=0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols + gap)).astype(x_type)
    r = None if r_type is None else (3 * g.standard_normal((rows, cols + 2 * gap)) * (1 + 40 * (g.random(cols + 2 * gap) < 0.01))).astype(r_type)
    return x, r, (1 + 0.3 * g.standard_normal(cols)).astype(np.float16) if weight else None


def run_norm(x, r, w, cols, offset=0.0, eps=1e-6, group=0, y=True, sum_out=True, stream=None):
    import torch
    rows = x.shape[0]
    xd, rd, wd = dev(x)[:, :cols], None if r is None else dev(r)[:, :cols], None if w is None else dev(w)
    so = torch.zeros((rows, cols + 8), dtype=rd.dtype, device="cuda")[:, :cols] if r is not None and sum_out else None
    yo = torch.zeros((rows, cols + 16), dtype=torch.float16, device="cuda")[:, :cols] if y else None
    co = torch.zeros((rows, cols + 8), dtype=torch.uint8, device="cuda")[:, :cols] if group else None
    sc = torch.zeros((rows, cols // group), device="cuda") if group else None
    torch.cuda.synchronize()
    tql.exl3_rms_norm(xd, yo, weight=wd, residual=rd, residual_out=so, eps=eps, weight_offset=offset, codes=co, scales=sc, stream=stream)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (so, yo, co, sc)]


def check_norm(x, r, w, cols, got, offset=0.0, eps=1e-6, group=0):
    so, yo, co, sc = got
    h, y = step_ref.rms_norm(x[:, :cols], None if r is None else r[:, :cols], w, offset, eps)
    with np.errstate(invalid="ignore"):
        if so is not None:
            step = 2.0 ** -11 if so.dtype == np.float16 else 2.0 ** -24
            assert np.all(np.abs(so - h) <= np.abs(h) * (step + 2.0 ** -24) + (2.0 ** -25 if so.dtype == np.float16 else 0))
        if yo is not None:
            fine = np.isfinite(y)
            assert np.array_equal(np.isnan(yo), np.isnan(y))
            assert np.all((np.abs(yo - y) <= np.abs(y) * (2.0 ** -11 + FP32) + 2.0 ** -25)[fine])
        if co is not None:
            want = step_ref.scales(y, group)
            assert np.all(np.abs(sc - want) <= want * FP32)
            value = step_ref.nearest_code.__globals__["VALUES"][co] * np.repeat(sc.astype(np.float64), group, 1)
            s = np.repeat(want, group, 1)
            limited = np.clip(y, -448 * s, 448 * s)
            assert np.array_equal(np.isnan(value), np.isnan(y))
            fine = ~np.isnan(y)
            assert np.all((np.abs(value - limited) <= np.abs(limited) * (2.0 ** -4 + 2 * FP32) + s * 2.0 ** -10)[fine])
    assert tql.exl3_get_device_status() == 0


@pytest.mark.parametrize("cols", [8, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 5120, 8192, 8200, 17408, 32768])
@pytest.mark.parametrize("rows", [1, 3, 160])
@pytest.mark.parametrize("x_type,r_type", [(np.float16, np.float16), (np.float32, None), (np.float16, np.float32)])
def test_norm_sizes(cols, rows, x_type, r_type):
    x, r, w = norm_inputs(rows, cols, x_type, r_type, cols, gap=8)
    check_norm(x, r, w, cols, run_norm(x, r, w, cols))


@pytest.mark.parametrize("x_type,r_type", [(a, b) for a in (np.float16, np.float32) for b in (None, np.float16, np.float32)])
@pytest.mark.parametrize("cols,group", [(128, 128), (128, 32), (256, 256), (640, 64), (1152, 128), (5120, 128), (5120, 5120), (264, 264), (8, 8),
                                        (17408, 17408), (17408, 32), (32768, 64)])
def test_norm_codes(x_type, r_type, cols, group):
    rows = 40
    x, r, w = norm_inputs(rows, cols, x_type, r_type, cols + group)
    x[3] = 0
    if r is not None:
        r[3] = 0
    x[4] *= np.float16(1e-3)
    for y in (True, False):
        check_norm(x, r, w, cols, run_norm(x, r, w, cols, offset=1.0, group=group, y=y, sum_out=y), offset=1.0, group=group)


@pytest.mark.parametrize("rows", [1, 5000])
def test_norm_without_weight_and_with_large_eps(rows):
    x, r, _ = norm_inputs(rows, 256, np.float16, np.float16, 3)
    check_norm(x, r, None, 256, run_norm(x, r, None, 256, offset=5.0, eps=2.0), eps=2.0)


def test_norm_values_that_are_not_finite_stay_in_their_row():
    x, r, w = norm_inputs(40, 640, np.float16, np.float16, 4)
    x[5, 7], x[9, 639], r[20, 100] = np.nan, np.inf, -np.inf
    got = run_norm(x, r, w, 640, group=64)
    for i in range(40):
        if i not in (5, 9, 20):
            check_norm(x[i:i + 1], r[i:i + 1], w, 640, [t[i:i + 1] for t in got], group=64)
    assert np.all(np.isnan(got[1][5])) and np.isnan(got[1][9, 639]) and np.all(got[1][9, :639] == 0)


@pytest.mark.parametrize("rows,cols,x_type,r_type,group",
                         [(305, 1032, np.float16, None, 0), (305, 1152, np.float32, None, 128), (641, 1032, np.float16, np.float16, 1032),
                          (1300, 5120, np.float16, np.float16, 0), (777, 5120, np.float32, np.float32, 128), (700, 5120, np.float32, np.float16, 5120),
                          (330, 8200, np.float16, np.float16, 8200), (310, 10240, np.float16, np.float32, 64), (457, 13824, np.float32, None, 13824),
                          (400, 17408, np.float16, np.float16, 32), (306, 20480, np.float16, None, 20480), (306, 20488, np.float16, None, 0),
                          (307, 27648, np.float16, None, 128), (305, 32768, np.float32, np.float32, 64),
                          (305, 264, np.float16, np.float16, 264), (1000, 512, np.float32, None, 64), (321, 520, np.float16, np.float32, 0),
                          (3001, 640, np.float16, np.float16, 64), (400, 1024, np.float32, np.float16, 1024), (456, 5120, np.float16, None, 64),
                          (153, 8200, np.float16, np.float16, 0), (500, 2048, np.float16, np.float16, 32), (500, 2056, np.float16, np.float32, 0),
                          (1217, 2560, np.float16, np.float16, 128), (460, 17408, np.float16, np.float32, 0), (153, 17408, np.float32, np.float32, 0)])
def test_norm_many_rows(rows, cols, x_type, r_type, group):
    """A row by a warp, by a CTA, and many rows of a CTA one behind the other through shared memory."""
    x, r, w = norm_inputs(rows, cols, x_type, r_type, rows + cols, gap=8)
    check_norm(x, r, w, cols, run_norm(x, r, w, cols, offset=1.0, group=group), offset=1.0, group=group)


@pytest.mark.parametrize("cols", [1032, 5120, 17408])
def test_norm_many_rows_in_place_not_finite_and_repeated(cols):
    x, r, w = norm_inputs(1500, cols, np.float16, np.float16, cols)
    x[5, 7], x[309, cols - 1], r[1499, 100] = np.nan, np.inf, -np.inf
    want = run_norm(x, r, w, cols, group=cols)
    clean = np.delete(np.arange(1500), [5, 309, 1499])
    check_norm(x[clean], r[clean], w, cols, [t[clean] for t in want], group=cols)
    assert np.all(np.isnan(want[1][5])) and np.all(want[1][309, :-1] == 0) and np.isnan(want[1][1499, 100])
    for _ in range(3):
        xd, rd = dev(x), dev(r)
        tql.exl3_rms_norm(xd, xd, weight=dev(w), residual=rd, residual_out=rd)
        assert np.array_equal(xd.cpu().numpy().view(np.int16), want[1].view(np.int16))
        assert np.array_equal(rd.cpu().numpy().view(np.int16), want[0].view(np.int16))


def test_norm_in_place():
    import torch
    x, r, w = norm_inputs(200, 5120, np.float16, np.float16, 5)
    want = run_norm(x, r, w, 5120)
    xd, rd = dev(x), dev(r)
    tql.exl3_rms_norm(xd, xd, weight=dev(w), residual=rd, residual_out=rd)
    assert np.array_equal(xd.cpu().numpy(), want[1]) and np.array_equal(rd.cpu().numpy(), want[0])
    xd = dev(x.astype(np.float32))
    rd = dev(r.astype(np.float32))
    tql.exl3_rms_norm(xd, residual=rd, residual_out=xd)
    assert np.array_equal(xd.cpu().numpy(), x.astype(np.float32) + r.astype(np.float32))
    assert torch.equal(rd, dev(r.astype(np.float32)))


def test_norm_of_no_rows():
    import torch
    e = torch.empty((0, 128), dtype=torch.float16, device="cuda")
    tql.exl3_rms_norm(e, e)


def test_norm_past_32_bit_offsets():
    """The last rows of a matrix of more than 2^31 elements, by its row stride."""
    import torch
    ld, rows = 1 << 20, 2100
    big = torch.zeros((rows, ld), dtype=torch.float16, device="cuda")
    x = torch.randn((rows, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).half()
    big[:, -64:] = x
    y = torch.zeros((rows, ld), dtype=torch.float16, device="cuda")
    tql.exl3_rms_norm(big[:, -64:], y[:, 8:72])
    want = torch.empty_like(x)
    tql.exl3_rms_norm(x, want)
    assert torch.equal(y[:, 8:72], want) and not y[:, 72:].any() and not y[:, :8].any()


# --------------------------------------------------------------------------- rotary


def table(positions, rot, base=1e4):
    a = np.arange(positions)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def run_rotary(x, qh, kh, dim, pos, tab, interleaved, qw, kw, eps=1e-6, offset=0.0, in_place=False):
    import torch
    xd = dev(x)
    out = xd if in_place else dev(np.full((x.shape[0], (qh + kh) * dim + 8), 7, dtype=np.float16))
    torch.cuda.synchronize()
    tql.exl3_qk_rotary(xd, out, qh, kh, dim, dev(np.asarray(pos, dtype=np.int32)), dev(tab), interleaved=interleaved,
                       q_weight=None if qw is None else dev(qw), k_weight=None if kw is None else dev(kw), eps=eps, weight_offset=offset)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def check_rotary(x, out, qh, kh, dim, pos, tab, interleaved, qw, kw, eps=1e-6, offset=0.0, in_place=False):
    width = (qh + kh) * dim
    want = step_ref.rotary(x[:, :width], qh, kh, dim, pos, tab, interleaved, qw, kw, eps, offset)
    # a pair's partners bound each other's error: both are at most the pair's length
    size = np.abs(want).reshape(len(x), qh + kh, dim).max(2, keepdims=True).repeat(dim, 2).reshape(len(x), width)
    moved = np.array([0 <= p < len(tab) for p in pos])
    tol = np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * 2.0 ** -20
    assert np.all((np.abs(out[:, :width] - want) <= tol)[moved])
    rest = x if in_place else np.full_like(out, 7)
    assert np.array_equal(out[~moved], rest[~moved]) and np.array_equal(out[:, width:], rest[:, width:])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("qh,kh", [(1, 0), (0, 1), (5, 1), (40, 8), (17, 17)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary(dim, qh, kh, interleaved, norm):
    g = np.random.default_rng(dim + qh)
    for rot in (16, 48, dim):
        x = g.standard_normal((37, (qh + kh) * dim + 24)).astype(np.float16)
        pos = g.integers(-1, 5000, 37)
        tab = table(5000, rot)
        qw, kw = ((1 + 0.3 * g.standard_normal(dim)).astype(np.float16) if norm and n else None for n in (qh, kh))
        for in_place in (False, True):
            out = run_rotary(x, qh, kh, dim, pos, tab, interleaved, qw, kw, offset=0.5 if norm else 0.0, in_place=in_place)
            check_rotary(x, out, qh, kh, dim, pos, tab, interleaved, qw, kw, offset=0.5 if norm else 0.0, in_place=in_place)
        assert tql.exl3_get_device_status() == 0


@pytest.mark.parametrize("rows", [1, 607, 608, 3000])
def test_rotary_rows_and_far_positions(rows):
    g = np.random.default_rng(rows)
    x = g.standard_normal((rows, 3 * 64)).astype(np.float16)
    pos = g.integers(130000, 131072, rows)
    tab = table(131072, 64, 1e6)
    out = run_rotary(x, 2, 1, 64, pos, tab, False, None, None)
    check_rotary(x, out, 2, 1, 64, pos, tab, False, None, None)


@pytest.mark.parametrize("dim,qh,kh", [(128, 1, 0), (128, 2, 1), (128, 8, 1), (128, 15, 1), (128, 16, 1), (64, 5, 5), (64, 31, 1), (64, 32, 1)])
@pytest.mark.parametrize("rows", [1, 2, 31, 1217, 3001])
def test_rotary_few_heads(dim, qh, kh, rows):
    """Several rows of a CTA at once, with rows among them that are left as they are."""
    g = np.random.default_rng(rows + qh)
    x = g.standard_normal((rows, (qh + kh) * dim + 8)).astype(np.float16)
    pos = g.integers(-300, 1000, rows)
    qw, kw = ((1 + 0.3 * g.standard_normal(dim)).astype(np.float16) if n else None for n in (qh, kh))
    for in_place in (False, True):
        out = run_rotary(x, qh, kh, dim, pos, table(1000, dim // 2), False, qw, kw, in_place=in_place)
        check_rotary(x, out, qh, kh, dim, pos, table(1000, dim // 2), False, qw, kw, in_place=in_place)
    assert tql.exl3_get_device_status() == 0


@pytest.mark.parametrize("qh,kh", [(2, 1), (40, 8)])
def test_rotary_positions_past_the_table_among_others(qh, kh):
    g = np.random.default_rng(qh)
    x = g.standard_normal((100, (qh + kh) * 64 + 8)).astype(np.float16)
    pos = g.integers(0, 130, 100)
    out = run_rotary(x, qh, kh, 64, pos, table(100, 64), True, None, None)
    check_rotary(x, out, qh, kh, 64, pos, table(100, 64), True, None, None)
    assert tql.exl3_get_device_status() == 10


def test_rotary_positions_past_the_table():
    x = np.random.default_rng(1).standard_normal((9, 128)).astype(np.float16)
    pos = [0, 99, 100, -1, 2**31 - 1, -2**31, 5, 98, 101]
    out = run_rotary(x, 1, 1, 64, pos, table(100, 32), False, None, None)
    check_rotary(x, out, 1, 1, 64, pos, table(100, 32), False, None, None)
    assert tql.exl3_get_device_status() == 10


def test_rotary_values_that_are_not_finite_stay_in_their_head():
    x = np.random.default_rng(2).standard_normal((4, 256)).astype(np.float16)
    x[1, 3], x[2, 100] = np.inf, np.nan
    tab = table(10, 32)
    clean = run_rotary(np.where(np.isfinite(x), x, 0).astype(np.float16), 3, 1, 64, [1, 2, 3, 4], tab, False, None, None)
    out = run_rotary(x, 3, 1, 64, [1, 2, 3, 4], tab, False, None, None)
    differs = ~((out == clean) | (np.isnan(out) & np.isnan(clean)))
    assert sorted(zip(*np.nonzero(differs))) == [(1, 3), (1, 19), (2, 100)]


@pytest.mark.parametrize("qh,kh", [(2, 1), (24, 8)])
def test_rotary_past_32_bit_offsets(qh, kh):
    import torch
    rows, ld, cols = 2100, 1 << 20, (qh + kh) * 128
    g = np.random.default_rng(qh)
    x, pos = dev(g.standard_normal((rows, cols)).astype(np.float16)), dev(g.integers(0, 500, rows).astype(np.int32))
    tab, want = dev(table(500, 128)), torch.empty((rows, cols), dtype=torch.float16, device="cuda")
    tql.exl3_qk_rotary(x, want, qh, kh, 128, pos, tab)
    big = torch.zeros((rows, ld), dtype=torch.float16, device="cuda")
    big[:, -cols:] = x
    tql.exl3_qk_rotary(big[:, -cols:], big[:, -cols:], qh, kh, 128, pos, tab)
    assert torch.equal(big[:, -cols:], want) and not big[:, :-cols].any()


def test_norm_ring_past_32_bit_offsets():
    import torch
    rows, ld, cols = 2100, 1 << 20, 4096
    x = torch.randn((rows, cols), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).half()
    want, codes, scales = torch.empty_like(x), torch.empty((rows, cols), dtype=torch.uint8, device="cuda"), torch.empty((rows, 32), device="cuda")
    tql.exl3_rms_norm(x, want, residual=x, codes=codes, scales=scales)
    big = torch.zeros((rows, ld), dtype=torch.float16, device="cuda")
    big[:, -cols:] = x
    far, far_scales = big[:, -cols:], torch.empty_like(scales)
    far_codes = torch.zeros((rows, 2 * ld), dtype=torch.uint8, device="cuda")[:, -cols:]
    tql.exl3_rms_norm(far, far, residual=far, codes=far_codes, scales=far_scales)
    assert torch.equal(far, want) and torch.equal(far_codes, codes) and torch.equal(far_scales, scales) and not big[:, :-cols].any()


# --------------------------------------------------------------------------- together


def test_two_of_each_at_once_and_captured():
    """Calls on two streams at once, and a captured graph's, give what single calls give."""
    import torch
    rows, qh, kh, dim = 900, 10, 2, 128
    cols = (qh + 2 * kh) * dim
    tab, pos = dev(table(4000, dim)), dev(np.random.default_rng(1).integers(0, 4000, rows).astype(np.int32))
    w = dev((1 + 0.3 * np.random.default_rng(2).standard_normal(dim)).astype(np.float16))

    class Work:
        def __init__(self, seed):
            x, r, nw = norm_inputs(rows, cols, np.float16, np.float32, seed)
            self.x, self.r, self.w = dev(x), dev(r), dev(nw)
            self.y = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
            self.so = torch.zeros((rows, cols), device="cuda")
            self.codes = torch.zeros((rows, cols), dtype=torch.uint8, device="cuda")
            self.scales = torch.zeros((rows, cols // 128), device="cuda")
            self.out = torch.zeros((rows, (qh + kh) * dim), dtype=torch.float16, device="cuda")

        def go(self, stream=None):
            tql.exl3_rms_norm(self.x, self.y, weight=self.w, residual=self.r, residual_out=self.so, codes=self.codes, scales=self.scales,
                              stream=stream)
            tql.exl3_qk_rotary(self.y, self.out, qh, kh, dim, pos, tab, q_weight=w, k_weight=w, stream=stream)

        def results(self):
            got = [t.cpu().numpy() for t in (self.y, self.so, self.codes, self.scales, self.out)]
            for t in (self.y, self.so, self.codes, self.scales, self.out):
                t.zero_()
            torch.cuda.synchronize()
            return got

    works = [Work(7), Work(8)]
    want = []
    for k in works:
        k.go()
        torch.cuda.synchronize()
        want.append(k.results())
        check_norm(k.x.cpu().numpy(), k.r.cpu().numpy(), k.w.cpu().numpy(), cols, [want[-1][1], *(want[-1][i] for i in (0, 2, 3))], group=128)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for k, st in zip(works, streams):
            k.go(st)
    torch.cuda.synchronize()
    for k, a in zip(works, want):
        assert all(np.array_equal(g, b) for g, b in zip(k.results(), a))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for k in works:
            k.go()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for k, a in zip(works, want):
            assert all(np.array_equal(g, b) for g, b in zip(k.results(), a))


def test_two_plans_at_once():
    import torch
    plans = [Plan(*random_requests(n, 30, 700, n)) for n in (1500, 90)]
    for p in plans:
        p.call()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for p, st in zip(plans, streams):
            p.again(st)
    torch.cuda.synchronize()
    for p in plans:
        p.check()
