"""What the step operators refuse before anything is launched, in the order shapes,
pointers, device; needs no GPU (a call with nothing to refuse gets as far as the device,
which is not initialized)."""
import ctypes
import math

import pytest

import trellis_quantized_linear_gb300 as tql

GOOD = 1 << 20  # a 16-byte aligned fake address; never dereferenced
INVALID, ALIGNMENT, NOT_INITIALIZED = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that no GPU may read: only where no device can be initialized")
    tql.build()
    return tql.load()


def at(i):
    return GOOD + i * (1 << 28)


def plan(lib, none=False, n_pages=100, capacity=50, rows=6, max_rows=3, n_seqs=4, max_pages=10, **kw):
    b = tql.Exl3Kv8Batch.__new__(tql.Exl3Kv8Batch)
    ctypes.Structure.__init__(b, kw.get("table", at(0)), kw.get("kv_len", at(1)), kw.get("q_start", at(2)), n_seqs, max_pages, rows, max_rows)
    return lib.exl3_kv8_plan(None if none else ctypes.byref(b), kw.get("tokens", at(3)), kw.get("cached", at(4)), kw.get("free", at(5)), capacity,
                             kw.get("count", at(6)), kw.get("left", at(7)), n_pages, kw.get("position", at(8)), kw.get("slot", at(9)),
                             kw.get("served", at(10)), None)


def test_plan(lib):
    assert plan(lib) == NOT_INITIALIZED
    assert plan(lib, none=True) == INVALID
    for kw in (dict(n_pages=0), dict(n_pages=1 << 25), dict(capacity=-1), dict(capacity=1 << 30), dict(rows=-1), dict(rows=1 << 30),
               dict(max_rows=-1), dict(n_seqs=-1), dict(n_seqs=65536), dict(max_pages=-1), dict(max_pages=1 << 26)):
        assert plan(lib, **kw) == INVALID, kw
    for name in ("table", "kv_len", "q_start", "tokens", "cached", "free", "count", "left", "position", "slot", "served"):
        assert plan(lib, **{name: None}) == ALIGNMENT, name
        assert plan(lib, **{name: GOOD + 2}) == ALIGNMENT, name
    # what an empty array is may be null
    assert plan(lib, n_seqs=0, table=None, kv_len=None, tokens=None, cached=None) == NOT_INITIALIZED
    assert plan(lib, rows=0, position=None, slot=None) == NOT_INITIALIZED
    assert plan(lib, capacity=0, free=None) == NOT_INITIALIZED and plan(lib, max_pages=0, table=None) == NOT_INITIALIZED
    # in place
    assert plan(lib, cached=at(1), left=at(6)) == NOT_INITIALIZED


def norm(lib, none=False, **kw):
    n = tql._Norm(x=at(0), residual=at(1), residual_out=at(2), weight=at(3), y=at(4), codes=at(5), scales=at(6), rows=10, cols=256,
                  ldx=256, ldr=256, ldro=256, ldy=256, ldc=256, x_dtype=0, residual_dtype=0, group=128, eps=1e-6, weight_offset=0.0)
    for k, v in kw.items():
        setattr(n, k, v)
    return lib.exl3_rms_norm(None if none else ctypes.byref(n), None)


def test_norm(lib):
    assert norm(lib) == NOT_INITIALIZED
    assert norm(lib, none=True) == INVALID
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=4), dict(cols=260), dict(cols=32776, ldx=40000, ldr=40000, ldro=40000, ldy=40000, ldc=40000),
               dict(x_dtype=2), dict(x_dtype=-1), dict(residual_dtype=2), dict(ldx=248), dict(ldx=260), dict(ldx=1 << 31), dict(ldr=248), dict(ldro=252),
               dict(ldy=8), dict(ldc=255), dict(eps=-1e-9), dict(eps=math.inf), dict(eps=math.nan), dict(weight_offset=math.nan),
               dict(group=0), dict(group=16), dict(group=96), dict(group=512), dict(cols=264, ldx=264, ldr=264, ldro=264, ldy=264, ldc=264),
               dict(scales=None), dict(codes=None), dict(residual=None), dict(residual_out=None, y=None, codes=None, scales=None)):
        assert norm(lib, **kw) == INVALID, kw
    for kw in (dict(x=None), dict(x=at(0) + 8), dict(residual=at(1) + 4), dict(residual_out=at(2) + 8), dict(weight=at(3) + 2), dict(y=at(4) + 8),
               dict(codes=at(5) + 8), dict(scales=at(6) + 2)):
        assert norm(lib, **kw) == ALIGNMENT, kw
    # one buffer: with one type and one row distance
    assert norm(lib, y=at(0)) == NOT_INITIALIZED and norm(lib, residual_out=at(1)) == NOT_INITIALIZED and norm(lib, residual_out=at(0)) == NOT_INITIALIZED
    for kw in (dict(y=at(0), ldy=512), dict(y=at(0), x_dtype=1), dict(residual_out=at(1), ldro=512), dict(residual_out=at(0), residual_dtype=1),
               dict(y=at(2)), dict(codes=at(0)), dict(codes=at(4)), dict(y=at(1), residual_dtype=1)):
        assert norm(lib, **kw) == INVALID, kw
    assert norm(lib, rows=0, x=None, residual=None, residual_out=None, weight=None, y=None, codes=None, scales=None) == 0
    for kw in (dict(weight=None), dict(residual=None, residual_out=None), dict(codes=None, scales=None), dict(y=None), dict(group=256), dict(group=32)):
        assert norm(lib, **kw) == NOT_INITIALIZED, kw


def rotary(lib, x=GOOD, ldx=1024, out=at(1), ldo=1024, rows=5, qh=4, kh=2, dim=128, pos=at(2), table=at(3), n=100, rot=128, qw=at(4), kw=at(5),
           eps=1e-6, offset=0.0):
    return lib.exl3_qk_rotary(x, ldx, out, ldo, rows, qh, kh, dim, pos, table, n, rot, 0, qw, kw, eps, offset, None)


def test_rotary(lib):
    assert rotary(lib) == NOT_INITIALIZED
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(qh=-1), dict(kh=-1), dict(qh=0, kh=0), dict(qh=65535, kh=1, ldx=1 << 24, ldo=1 << 24),
               dict(dim=96), dict(dim=256), dict(n=0), dict(n=1 << 31), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(eps=-1.0),
               dict(eps=math.nan), dict(offset=math.inf), dict(ldx=760), dict(ldx=770), dict(ldo=760), dict(out=GOOD, ldo=2048),
               dict(qw=None), dict(kw=None)):
        assert rotary(lib, **kw) == INVALID, kw
    for kw in (dict(x=None), dict(x=GOOD + 8), dict(out=None), dict(out=at(1) + 8), dict(pos=None), dict(pos=at(2) + 1), dict(table=None),
               dict(table=at(3) + 8), dict(qw=at(4) + 8), dict(kw=at(5) + 8)):
        assert rotary(lib, **kw) == ALIGNMENT, kw
    assert rotary(lib, rows=0, x=None, out=None, pos=None) == 0
    for kw in (dict(out=GOOD), dict(qw=None, kw=None), dict(qh=0, qw=None), dict(kh=0, kw=None), dict(rot=16), dict(dim=64, rot=64)):
        assert rotary(lib, **kw) == NOT_INITIALIZED, kw


def attend(lib, q=at(0), ldq=2048, k=at(1), ldk=1024, v=at(2), ldv=1024, heads=8, kv=2, dim=128, qs=at(3), n=3, rows=100, scale=0.1, cap=0.0,
           out=at(4), ldo=1024, lse=at(5)):
    return lib.exl3_prompt_attention(q, ldq, k, ldk, v, ldv, heads, kv, dim, qs, n, rows, scale, cap, 1, out, ldo, lse, None)


def test_prompt_attention(lib):
    assert attend(lib) == NOT_INITIALIZED
    for kw in (dict(dim=96), dict(dim=0), dict(heads=0), dict(heads=9), dict(kv=0), dict(kv=-2), dict(heads=258, kv=2, ldq=1 << 17, ldo=1 << 17),
               dict(heads=65536, kv=65536), dict(n=-1), dict(n=65536), dict(rows=-1), dict(rows=1 << 31), dict(rows=1 << 28), dict(rows=1 << 62),
               dict(scale=math.inf), dict(scale=math.nan), dict(cap=-1.0), dict(cap=1e-31), dict(cap=math.inf), dict(ldq=1016), dict(ldq=1026),
               dict(ldk=248), dict(ldv=257), dict(ldo=8), dict(out=at(0)), dict(out=at(1)), dict(out=at(2))):
        assert attend(lib, **kw) == INVALID, kw
    for kw in (dict(q=None), dict(q=at(0) + 8), dict(k=None), dict(k=at(1) + 8), dict(v=at(2) + 2), dict(out=None), dict(out=at(4) + 8),
               dict(qs=None), dict(qs=at(3) + 2), dict(lse=at(5) + 1)):
        assert attend(lib, **kw) == ALIGNMENT, kw
    assert attend(lib, rows=0, q=None, k=None, v=None, out=None) == 0 and attend(lib, n=0, qs=None) == 0
    for kw in (dict(lse=None), dict(scale=-0.1), dict(scale=0.0), dict(cap=30.0), dict(heads=256, kv=2, ldq=32768, ldo=32768), dict(dim=64)):
        assert attend(lib, **kw) == NOT_INITIALIZED, kw


# --------------------------------------------------------------------------- the Python entry points


def goes(f):
    with pytest.raises(tql.Exl3Error) as e:
        f()
    assert e.value.status == NOT_INITIALIZED


def refused(f):
    with pytest.raises(ValueError):
        f()


def test_plan_looks_at_its_tensors(lib):
    import torch
    def i(*shape):
        return torch.zeros(shape, dtype=torch.int32)
    batch = tql.Exl3Kv8Batch(i(2, 3), i(2), i(3), 9, 5)
    good = dict(tokens=i(2), cached=i(2), free_pages=i(7), free_count=i(1), free_left=i(1), n_pages=10, position=i(9), slot=i(9), served=i(1))
    goes(lambda: tql.exl3_kv8_plan(batch, **good, stream=0))
    for name, bad in (("tokens", i(1)), ("tokens", i(2).long()), ("cached", i(4)[::2]), ("cached", i(2).float()), ("free_count", i(0)),
                      ("free_left", i(1).long()), ("position", i(8)), ("slot", i(18)[::2]), ("served", i(0)), ("free_pages", i(7).short())):
        refused(lambda: tql.exl3_kv8_plan(batch, **{**good, name: bad}, stream=0))
    refused(lambda: tql.exl3_kv8_plan(tql.Exl3Kv8Batch(i(2, 3), i(2)), **good, stream=0))


def test_norm_looks_at_its_tensors(lib):
    import torch
    def h(*shape):
        return torch.zeros(shape, dtype=torch.float16)
    x, w = h(5, 256), h(256)
    codes, scales = torch.zeros((5, 256), dtype=torch.uint8), torch.zeros((5, 2))
    goes(lambda: tql.exl3_rms_norm(x, h(5, 256), weight=w, residual=x.float(), residual_out=x.float(), codes=codes, scales=scales, stream=0))
    goes(lambda: tql.exl3_rms_norm(h(5, 304)[:, 48:], h(7, 264), codes=codes.view(torch.float8_e4m3fn), scales=scales, stream=0))
    for kw in (dict(y=x.float()), dict(y=h(4, 256)), dict(y=h(5, 128)), dict(y=h(5, 512)[:, ::2]), dict(weight=h(128)), dict(weight=w.float()),
               dict(weight=h(512)[::2]), dict(residual=h(4, 256)), dict(residual=x.double()), dict(residual=x, residual_out=x.float()),
               dict(residual=x, residual_out=h(5, 8)), dict(residual_out=x), dict(codes=codes), dict(scales=scales), dict(codes=codes, scales=torch.zeros((5, 3))),
               dict(codes=codes.short(), scales=scales), dict(codes=codes[:4], scales=scales), dict(codes=codes, scales=torch.zeros(10)),
               dict(codes=codes, scales=torch.zeros((4, 2)))):
        refused(lambda: tql.exl3_rms_norm(x, **{"y": h(5, 256), **kw}, stream=0))
    refused(lambda: tql.exl3_rms_norm(x.bfloat16(), h(5, 256), stream=0))
    refused(lambda: tql.exl3_rms_norm(h(256, 5).t(), h(5, 256), stream=0))


def test_rotary_looks_at_its_tensors(lib):
    import torch
    x, pos, table, w = torch.zeros((5, 768)).half(), torch.zeros(5, dtype=torch.int32), torch.zeros((10, 64)), torch.zeros(128).half()
    def call(x=x, out=x, pos=pos, table=table, qw=None, kw=None):
        tql.exl3_qk_rotary(x, out, 4, 2, 128, pos, table, q_weight=qw, k_weight=kw, stream=0)
    goes(call)
    goes(lambda: call(qw=w, kw=w, out=torch.zeros((6, 1024)).half()))
    for kw in (dict(x=x.float()), dict(x=x[:, :760]), dict(out=x[:4]), dict(out=torch.zeros((768, 5)).half().t()), dict(pos=pos[:4]), dict(pos=pos.long()),
               dict(table=table.half()), dict(table=table[0]), dict(table=torch.zeros((64, 10)).t()), dict(qw=w[:64], kw=w), dict(qw=w, kw=w.float())):
        refused(lambda: call(**kw))


def test_prompt_attention_looks_at_its_tensors(lib):
    import torch
    x = torch.zeros((9, 8 * 64)).half()
    q, k, v, qs = x[:, :256], x[:, 256:384], x[:, 384:], torch.zeros(3, dtype=torch.int32)
    def call(q=q, k=k, v=v, qs=qs, out=torch.zeros((9, 256)).half(), lse=torch.zeros((9, 4))):
        tql.exl3_prompt_attention(q, k, v, 4, 2, 64, qs, 0.1, out, lse=lse, stream=0)
    goes(call)
    goes(lambda: call(lse=None))
    for kw in (dict(q=q.float()), dict(q=x[:, :128]), dict(k=k[:8]), dict(v=v.bfloat16()), dict(v=x[:, 1:129:2]), dict(qs=qs.long()), dict(qs=qs[:0]),
               dict(qs=torch.zeros(6, dtype=torch.int32)[::2]), dict(out=torch.zeros((8, 256)).half()), dict(out=torch.zeros((9, 256))),
               dict(lse=torch.zeros((8, 4))), dict(lse=torch.zeros((9, 4)).half()), dict(lse=torch.zeros((9, 8))[:, ::2])):
        refused(lambda: call(**kw))


def test_tensors_of_another_device_are_refused(lib, monkeypatch):
    import torch
    monkeypatch.setattr(tql, "_ready", True)
    monkeypatch.setattr(tql, "_raw_device", lambda: 0)
    x, i, table = torch.zeros((3, 768)).half(), torch.zeros(9, dtype=torch.int32), torch.zeros((10, 64))
    batch = tql.Exl3Kv8Batch(i[:2].view(2, 1), i[:2], i[:3], 3, 3)
    for f in (lambda: tql.exl3_kv8_plan(batch, i, i, i, i, i, 10, i, i, i, stream=0), lambda: tql.exl3_rms_norm(x, x, stream=0),
              lambda: tql.exl3_qk_rotary(x, x, 4, 2, 128, i, table, stream=0),
              lambda: tql.exl3_prompt_attention(x[:, :256], x[:, 256:512], x[:, 512:], 4, 4, 64, i[:2], 0.1, torch.zeros((3, 256)).half(), stream=0)):
        with pytest.raises(ValueError, match="current device"):
            f()
    monkeypatch.setattr(tql, "_raw_device", lambda: -1)  # where the tensors are
    goes(lambda: tql.exl3_rms_norm(x, x, stream=0))
