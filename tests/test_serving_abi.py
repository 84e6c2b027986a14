"""Host-side checks of the serving operators that need no GPU: every refusal,
in the order shapes, pointers, device."""
import ctypes

import pytest

import trellis_quantized_linear_gb300 as tql

GOOD = 1 << 20  # a 16-byte aligned fake address; never dereferenced
INVALID, ALIGNMENT, NOT_INITIALIZED = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    tql.build()
    return tql.load()


def cache(**kw):
    c = tql.Exl3Kv8Cache.__new__(tql.Exl3Kv8Cache)
    ctypes.Structure.__init__(c, GOOD, GOOD, GOOD, GOOD, GOOD, 100, 8, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = tql.Exl3Kv8Batch.__new__(tql.Exl3Kv8Batch)
    ctypes.Structure.__init__(b, GOOD, GOOD, GOOD, 4, 10, 6, 3)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def ref(s):
    return None if s is None else ctypes.byref(s)


def append(lib, c=None, b=None, k=GOOD, ldk=1024, v=GOOD, ldv=1024, none=False):
    return lib.exl3_kv8_append(None if none else ref(c or cache()), ref(b or batch()), k, ldk, v, ldv, None)


def attend(lib, c=None, b=None, q=GOOD, ldq=4096, heads=32, scale=0.1, cap=0.0, out=GOOD, ldo=4096, lse=GOOD, ws=GOOD):
    return lib.exl3_kv8_attention(ref(c or cache()), ref(b or batch()), q, ldq, heads, scale, cap, 1, out, ldo, lse, ws,
                                  1 << 40, None)


def weigh(lib, c=None, b=None, q=GOOD, ldq=4096, heads=32, scale=0.1, cap=0.0, lse=GOOD):
    return lib.exl3_kv8_weigh(ref(c or cache()), ref(b or batch()), q, ldq, heads, scale, cap, 1, lse, None)


def evict(lib, c=None, b=None, dst=GOOD, budget=100, recent=10, kept=GOOD, new_len=GOOD):
    return lib.exl3_kv8_evict(ref(c or cache()), ref(b or batch()), dst, budget, recent, kept, new_len, None)


BAD_CACHES = [dict(head_dim=96), dict(head_dim=0), dict(n_kv_heads=0), dict(n_kv_heads=-8), dict(n_kv_heads=1025),
              dict(n_pages=-1), dict(n_pages=1 << 31), dict(n_pages=1 << 23)]
BAD_BATCHES = [dict(n_seqs=-1), dict(n_seqs=65536), dict(max_pages=-1), dict(max_pages=1 << 30)]
BAD_ROWS = [dict(rows=-1), dict(max_rows=-1), dict(max_rows=7)]
BAD_POINTERS = [dict(k=None), dict(v=GOOD + 8), dict(k_scale=None), dict(v_scale=GOOD + 2), dict(weight=GOOD + 4)]


@pytest.mark.parametrize("call", [append, attend, weigh, evict])
def test_caches_and_batches_out_of_range(lib, call):
    for kw in BAD_CACHES:
        assert call(lib, c=cache(**kw)) == INVALID, kw
    for kw in BAD_BATCHES + (BAD_ROWS if call is not evict else []):
        assert call(lib, b=batch(**kw)) == INVALID, kw
    for kw in BAD_POINTERS:
        assert call(lib, c=cache(**kw)) == ALIGNMENT, kw
    for kw in [dict(page_table=None), dict(kv_len=GOOD + 1)] + ([dict(q_start=None)] if call is not evict else []):
        assert call(lib, b=batch(**kw)) == ALIGNMENT, kw


def test_valid_calls_get_as_far_as_the_device(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where no device can be initialized")
    for call in (append, attend, weigh, evict):
        assert call(lib) == NOT_INITIALIZED
    r = tql._LogitsRules()
    assert lib.exl3_logits_adjust(GOOD, 256, 2, 250, ref(r), GOOD, 256, GOOD, None) == NOT_INITIALIZED


def test_append_refusals(lib):
    assert append(lib, none=True) == INVALID
    assert append(lib, ldk=1016) == INVALID and append(lib, ldv=1028) == INVALID
    assert append(lib, k=GOOD + 2) == ALIGNMENT and append(lib, v=None) == ALIGNMENT


def test_attention_refusals(lib):
    for call in (attend, weigh):
        for kw in (dict(heads=0), dict(heads=-8), dict(heads=12), dict(ldq=4088), dict(ldq=4100), dict(scale=float("nan")),
                   dict(scale=float("inf")), dict(cap=-1.0), dict(cap=1e-35), dict(cap=float("nan")), dict(cap=float("inf"))):
            assert call(lib, **kw) == INVALID, kw
    for kw in (dict(q=None), dict(q=GOOD + 8), dict(lse=GOOD + 2)):
        assert attend(lib, **kw) == ALIGNMENT and weigh(lib, **kw) == ALIGNMENT, kw
    assert attend(lib, ws=GOOD + 8) == ALIGNMENT and attend(lib, out=GOOD + 2) == ALIGNMENT
    assert weigh(lib, lse=None) == ALIGNMENT and weigh(lib, c=cache(weight=None)) == ALIGNMENT
    assert attend(lib, ldo=4088) == INVALID
    assert attend(lib, b=batch(rows=1 << 30, max_rows=1)) == INVALID  # rows x heads past 31 bits
    c, b = cache(), batch()
    assert lib.exl3_kv8_attention_workspace_bytes(ref(c), ref(b), 12) == 0
    assert lib.exl3_kv8_attention_workspace_bytes(None, ref(b), 8) == 0


def test_evict_refusals(lib):
    for kw in (dict(budget=0), dict(budget=-5), dict(recent=-1), dict(budget=10, recent=11), dict(budget=(1 << 30) + 1)):
        assert evict(lib, **kw) == INVALID, kw
    for kw in (dict(dst=None), dict(kept=GOOD + 1), dict(new_len=None), dict(c=cache(weight=None))):
        assert evict(lib, **kw) == ALIGNMENT, kw


def test_logits_refusals(lib):
    def call(M=2, n=250, ldl=256, ldo=256, logits=GOOD, out=GOOD, argmax=GOOD, **kw):
        r = tql._LogitsRules()
        for k, v in kw.items():
            setattr(r, k, v)
        return lib.exl3_logits_adjust(logits, ldl, M, n, ref(r), out, ldo, argmax, None)

    for kw in (dict(M=-1), dict(M=65536), dict(n=0), dict(n=(1 << 19) + 1, ldl=1 << 20, ldo=1 << 20), dict(ldl=248), dict(ldl=254),
               dict(ldo=248), dict(ldo=255), dict(history=GOOD), dict(history_start=GOOD), dict(generated_from=GOOD),
               dict(bias_id=GOOD), dict(bias_id=GOOD, bias_value=GOOD), dict(history_size=-1), dict(bias_size=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(logits=None), dict(out=GOOD + 4), dict(argmax=GOOD + 2), dict(repetition=GOOD + 2), dict(allowed=GOOD + 1),
               dict(history=GOOD + 1, history_start=GOOD)):
        assert call(**kw) == ALIGNMENT, kw
    assert lib.exl3_logits_adjust(GOOD, 256, 2, 250, None, GOOD, 256, GOOD, None) == INVALID


def test_cache_and_batch_objects_check_their_tensors():
    import torch
    k = torch.zeros((3, 2, 64, 128), dtype=torch.uint8)
    s, w = torch.ones((3, 2)), torch.zeros((3, 2, 64))
    c = tql.Exl3Kv8Cache(k, k, s, s, w)
    assert (c.n_pages, c.n_kv_heads, c.head_dim) == (3, 2, 128) and c.weight == w.data_ptr()
    assert tql.Exl3Kv8Cache(k, k, s, s).weight is None
    for bad in ((k[:, :, :32], k, s, s, w), (k, k[:2], s, s, w), (k.to(torch.int16), k, s, s, w), (k, k, s[:2], s, w),
                (k, k, s.double(), s, w), (k, k, s, s, w[:, :, :3]), (k.transpose(0, 1), k.transpose(0, 1), s.t(), s.t(), None)):
        with pytest.raises(ValueError):
            tql.Exl3Kv8Cache(*bad)
    t, n, q = torch.zeros((4, 5), dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    b = tql.Exl3Kv8Batch(t, n, q, 6, 2)
    assert (b.n_seqs, b.max_pages, b.rows, b.max_rows) == (4, 5, 6, 2)
    for bad in ((t, n[:3], q), (t, n, q[:4]), (t.long(), n, q), (t.t(), torch.zeros(5, dtype=torch.int32), None), (t, n.float(), q)):
        with pytest.raises(ValueError):
            tql.Exl3Kv8Batch(*bad, 6, 2)


def test_new_status_has_text(lib):
    assert "range" in tql.exl3_status_string(10) and tql.STATUS_NAMES[10] == "EXL3_ERR_DEVICE_INDEX"
