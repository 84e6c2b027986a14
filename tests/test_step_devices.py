"""The step operators refuse a call of which any one tensor is not on the current device; needs
no GPU (tensors without storage stand for those of another device)."""
import pytest

import trellis_quantized_linear_gb300 as tql

NOT_INITIALIZED = 5
CPU = -1  # what get_device says of a CPU tensor


@pytest.fixture(autouse=True)
def cpu_is_the_current_device(monkeypatch):
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that no GPU may read: only where no device can be initialized")
    tql.build()
    monkeypatch.setattr(tql, "_ready", True)
    monkeypatch.setattr(tql, "_raw_device", lambda: CPU)


class Elsewhere:
    """A tensor that says it is on another device."""

    def __init__(self, t):
        self._t = t

    def get_device(self):
        return 1

    def __getattr__(self, name):
        return getattr(self._t, name)

    def __getitem__(self, i):
        return self._t[i]


def one_at_a_time(call, good):
    """Goes as far as the device with all tensors of `good` here, and is refused with any one elsewhere."""
    with pytest.raises(tql.Exl3Error) as e:
        call(**good)
    assert e.value.status == NOT_INITIALIZED
    for name, t in good.items():
        with pytest.raises(ValueError, match="current device"):
            call(**{**good, name: Elsewhere(t)})


def i32(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.int32)


def f16(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.float16)


def test_plan():
    def call(page_table, kv_len, q_start, **kw):
        tql.exl3_kv8_plan(tql.Exl3Kv8Batch(page_table, kv_len, q_start, 9, 5), n_pages=10, stream=0, **kw)
    one_at_a_time(call, dict(page_table=i32(2, 3), kv_len=i32(2), q_start=i32(3), tokens=i32(2), cached=i32(2), free_pages=i32(7), free_count=i32(1),
                             free_left=i32(1), position=i32(9), slot=i32(9), served=i32(1)))


def test_norm():
    import torch
    def call(**kw):
        tql.exl3_rms_norm(stream=0, **kw)
    one_at_a_time(call, dict(x=f16(5, 256), y=f16(5, 256), weight=f16(256), residual=f16(5, 256), residual_out=f16(5, 256),
                             codes=torch.zeros((5, 256), dtype=torch.uint8), scales=torch.zeros((5, 2))))


def test_rotary():
    import torch
    def call(**kw):
        tql.exl3_qk_rotary(q_heads=4, k_heads=2, head_dim=128, stream=0, **kw)
    one_at_a_time(call, dict(x=f16(5, 768), out=f16(5, 768), position=i32(5), cos_sin=torch.zeros((10, 64)), q_weight=f16(128), k_weight=f16(128)))


def test_prompt_attention():
    import torch
    def call(**kw):
        tql.exl3_prompt_attention(n_heads=4, n_kv_heads=2, head_dim=64, scale=0.1, stream=0, **kw)
    one_at_a_time(call, dict(q=f16(9, 256), k=f16(9, 128), v=f16(9, 128), q_start=i32(3), out=f16(9, 256), lse=torch.zeros((9, 4))))


def test_what_is_left_out_and_addresses_are_not_looked_at():
    import torch
    for kw in (dict(weight=None), dict(weight=1 << 20)):
        with pytest.raises(tql.Exl3Error) as e:
            tql.exl3_rms_norm(f16(5, 256), f16(5, 256), stream=0, **kw)
        assert e.value.status == NOT_INITIALIZED
    with pytest.raises(tql.Exl3Error) as e:
        tql.exl3_prompt_attention(f16(9, 256), f16(9, 128), f16(9, 128), 4, 2, 64, torch.zeros(3, dtype=torch.int32), 0.1, f16(9, 256), stream=0)
    assert e.value.status == NOT_INITIALIZED
