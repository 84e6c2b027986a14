"""What the serving operators' entry points refuse before anything is launched; needs no
GPU (a call with nothing to refuse gets as far as the device, which is not initialized)."""
import ctypes

import pytest

import trellis_quantized_linear_gb300 as tql

GOOD = 1 << 20  # a 16-byte aligned fake address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that no GPU may read: only where no device can be initialized")
    tql.build()
    return tql.load()


def test_one_logits_buffer_has_one_row_distance(lib):
    rules = ctypes.byref(tql._LogitsRules())

    def call(M, logits, ldl, out, ldo):
        return lib.exl3_logits_adjust(logits, ldl, M, 250, rules, out, ldo, GOOD, None)

    assert call(2, GOOD, 256, GOOD, 260) == 1
    assert call(1, GOOD, 256, GOOD, 260) == 5 and call(2, GOOD, 256, GOOD, 256) == 5 and call(2, GOOD, 256, 2 * GOOD, 260) == 5


def goes(f):
    """The call gets past every check of its arguments."""
    with pytest.raises(tql.Exl3Error) as e:
        f()
    assert e.value.status == 5


def objects():
    import torch
    codes, s, w = torch.zeros((3, 2, 64, 64), dtype=torch.uint8), torch.ones((3, 2)), torch.zeros((3, 2, 64))
    cache = tql.Exl3Kv8Cache(codes, codes, s, s, w)
    start = torch.tensor([0, 2, 5], dtype=torch.int32)
    batch = tql.Exl3Kv8Batch(torch.zeros((2, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32), start, 5, 3)
    return torch, cache, batch


def test_append_looks_at_its_tensors(lib):
    torch, cache, batch = objects()
    x = torch.zeros((5, 2 * 128), dtype=torch.float16)

    def call(k, v):
        tql.exl3_kv8_append(cache, batch, k, v, stream=0)

    for good in (x[:, :128], x[:, 128:], torch.zeros((7, 128)).half(), x[:, :128].reshape(5, 2, 64), x):
        goes(lambda: call(good, x[:, :128]))
        goes(lambda: call(x[:, :128], good))
    for bad in (x.float()[:, :128], x.bfloat16()[:, :128], x[:4, :128], x[:, :120], torch.zeros((128, 5)).half().t(), x[:, ::2], x.view(-1),
                x[:, :128].reshape(5, 2, 64).transpose(1, 2), torch.zeros((5, 3, 64)).half()[:, ::2]):
        for args in ((bad, x[:, :128]), (x[:, :128], bad)):
            with pytest.raises(ValueError):
                call(*args)


def test_one_row_needs_no_row_stride(lib):
    torch, cache, _ = objects()
    one = tql.Exl3Kv8Batch(torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32), 1, 1)
    x = torch.zeros((128, 1), dtype=torch.float16).t()  # strides (1, 1)
    goes(lambda: tql.exl3_kv8_append(cache, one, x, x.contiguous(), stream=0))
    logits = torch.zeros((1, 1001))  # a row stride that is no multiple of 4
    goes(lambda: tql.exl3_logits_adjust(logits, 1001, logits, torch.zeros(1, dtype=torch.int32), stream=0))


def test_attention_and_weigh_look_at_their_tensors(lib):
    torch, cache, batch = objects()
    q, out, lse = torch.zeros((5, 300)).half()[:, :256], torch.zeros((5, 256)).half(), torch.zeros((5, 4))
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    q = torch.zeros((5, 304)).half()[:, :256]

    def attend(**kw):
        a = dict(q=q, out=out, lse=lse) | kw
        tql.exl3_kv8_attention(cache, batch, a["q"], 4, 0.1, a["out"], ws, lse=a["lse"], workspace_bytes=1 << 40, stream=0)

    def weigh(**kw):
        a = dict(q=q, lse=lse) | kw
        tql.exl3_kv8_weigh(cache, batch, a["q"], 4, 0.1, a["lse"], stream=0)

    goes(attend)
    goes(weigh)
    goes(lambda: attend(lse=None))
    goes(lambda: attend(lse=lse.view(-1)))
    for bad in (q.float(), q[:4], q[:, :248], torch.zeros((256, 5)).half().t()):
        for call in (lambda: attend(q=bad), lambda: attend(out=bad), lambda: weigh(q=bad)):
            with pytest.raises(ValueError):
                call()
    for bad in (lse.double(), lse.half(), lse[:4], torch.zeros((4, 5)).t(), lse[:, :3]):
        for call in (lambda: attend(lse=bad), lambda: weigh(lse=bad)):
            with pytest.raises(ValueError):
                call()


def test_evict_looks_at_its_tensors(lib):
    torch, cache, batch = objects()
    a = dict(dst=torch.zeros((2, 2), dtype=torch.int32), kept=torch.zeros((2, 2, 100), dtype=torch.int32), new_len=torch.zeros(2, dtype=torch.int32))

    def call(**kw):
        b = a | kw
        tql.exl3_kv8_evict(cache, batch, b["dst"], 100, 10, b["kept"], b["new_len"], stream=0)

    goes(call)
    for name, t in a.items():
        for bad in (t.long(), t.float(), t.view(-1)[:-1], torch.zeros(2 * t.numel(), dtype=torch.int32)[::2]):
            with pytest.raises(ValueError):
                call(**{name: bad})


def test_logits_look_at_their_tensors(lib):
    torch, _, _ = objects()
    M, n = 3, 250
    i32 = dict(dtype=torch.int32)
    x = torch.zeros((M, 256))
    a = dict(logits=x, out=x, argmax=torch.zeros(M, **i32), history=torch.zeros(9, **i32), history_start=torch.zeros(M + 1, **i32),
             generated_from=torch.zeros(M, **i32), repetition=torch.ones(M), presence=torch.ones(M), frequency=torch.ones(M),
             bias_id=torch.zeros(7, **i32), bias_value=torch.zeros(7), bias_start=torch.zeros(M + 1, **i32), allowed=torch.zeros((M, 8), **i32))

    def call(**kw):
        b = a | kw
        tql.exl3_logits_adjust(b.pop("logits"), n, b.pop("out"), b.pop("argmax"), stream=0, **b)

    goes(call)
    goes(lambda: call(allowed=a["allowed"].view(torch.uint32), out=torch.zeros((M, 252))))
    goes(lambda: call(bias_id=None, bias_value=None, bias_start=None, allowed=None))
    for name, t in a.items():
        bad = [t.double() if t.is_floating_point() else t.long(), t.int() if t.is_floating_point() else t.float()]
        if name in ("logits", "out"):
            bad += [t[:, :249], torch.zeros((256, M)).t()] + ([t[:2]] if name == "out" else [])
        else:
            bad += [torch.zeros(2 * t.numel(), dtype=t.dtype)[::2]]
            if name not in ("history", "bias_id"):
                bad += [t.reshape(-1)[:-1]]
        for b in bad:
            with pytest.raises(ValueError, match=name):
                call(**{name: b})


def test_empty_lists_are_lists(lib):
    """No token said yet, no bias on any row: not a rule with parts missing."""
    torch, _, _ = objects()
    x, am = torch.zeros((2, 256)), torch.zeros(2, dtype=torch.int32)
    none, starts = torch.zeros(0, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    goes(lambda: tql.exl3_logits_adjust(x, 250, x, am, history=none, history_start=starts, generated_from=am, presence=torch.ones(2), stream=0))
    goes(lambda: tql.exl3_logits_adjust(x, 250, x, am, bias_id=none, bias_value=torch.zeros(0), bias_start=starts, stream=0))
    for kw in (dict(history_start=starts), dict(bias_start=starts), dict(generated_from=am), dict(bias_id=none.new_zeros(1), bias_value=torch.zeros(1))):
        with pytest.raises(tql.Exl3Error) as e:
            tql.exl3_logits_adjust(x, 250, x, am, stream=0, **kw)
        assert e.value.status == 1


def test_calls_without_rows_do_nothing(lib):
    """Also with the tensors of an empty batch, which have no addresses."""
    torch, cache, _ = objects()
    i32 = dict(dtype=torch.int32)
    none = tql.Exl3Kv8Batch(torch.zeros((0, 4), **i32), torch.zeros(0, **i32), torch.zeros(1, **i32), 0, 0)
    idle = tql.Exl3Kv8Batch(torch.zeros((2, 4), **i32), torch.ones(2, **i32), torch.zeros(3, **i32), 0, 0)
    x, q, lse = torch.zeros((0, 128)).half(), torch.zeros((0, 256)).half(), torch.zeros((0, 4))
    for batch in (none, idle):
        tql.exl3_kv8_append(cache, batch, x, x, stream=0)
        tql.exl3_kv8_attention(cache, batch, q, 4, 0.1, torch.empty_like(q), torch.zeros(16, dtype=torch.uint8), lse=lse, stream=0)
        tql.exl3_kv8_weigh(cache, batch, q, 4, 0.1, lse, stream=0)
        with pytest.raises(tql.Exl3Error):  # shapes are looked at all the same
            tql.exl3_kv8_weigh(cache, batch, torch.zeros((0, 192)).half(), 3, 0.1, lse, stream=0)
    tql.exl3_kv8_evict(cache, none, torch.zeros((0, 1), **i32), 64, 0, torch.zeros((0, 2, 64), **i32), torch.zeros(0, **i32), stream=0)
    tql.exl3_logits_adjust(torch.zeros((0, 256)), 250, torch.zeros((0, 256)), torch.zeros(0, **i32), stream=0)
