"""Argument checks of the rotary and paged-cache entries: no call here reaches
the GPU (they return before any CUDA call)."""
import ctypes

import pytest
import torch

import hybrid_softmax_gated_b200 as arl2

FAKE = 0x1000  # never dereferenced: validation fails first


def rotary_config(head_dim=128, dims=(44, 42, 42), base=1e4, pairs=0, freqs=0, axes=None):
    return arl2.Arl2RotaryConfig(head_dim, len(dims) if axes is None else axes, (ctypes.c_int * 4)(*dims), base, pairs,
                                 freqs)


def test_rotary_config_is_validated():
    lib, h = arl2._lib, ctypes.c_void_p()
    assert lib.arl2_rotary_create(None, ctypes.byref(h)) == -1
    assert lib.arl2_rotary_create(ctypes.byref(rotary_config()), None) == -1
    for bad in (dict(pairs=2), dict(freqs=-1), dict(base=0.5), dict(base=float("nan")), dict(base=float("inf"))):
        assert lib.arl2_rotary_create(ctypes.byref(rotary_config(**bad)), ctypes.byref(h)) == -1, bad
    for bad in (dict(head_dim=1), dict(head_dim=258), dict(axes=0), dict(axes=5), dict(dims=(3, 2)), dict(dims=(0, 0)),
                dict(dims=(-2, 8)), dict(dims=(64, 66)), dict(dims=(2 ** 30, 2 ** 30, 2 ** 30, 2 ** 30))):
        assert lib.arl2_rotary_create(ctypes.byref(rotary_config(**bad)), ctypes.byref(h)) == -2, bad
    assert h.value is None
    lib.arl2_rotary_destroy(None)


def test_rotary_apply_is_validated_before_cuda():
    lib = arl2._lib
    plan = arl2.RotaryAxes(128, [44, 42, 42])
    good = dict(h=plan.handle, dtype=0, tokens=2, pos=FAKE, qh=2, q=FAKE, qs=0, qo=FAKE, qos=0, kh=1, k=FAKE, ks=0,
                ko=FAKE, kos=0, inverse=0, stream=None)

    def call(**kw):
        return lib.arl2_rotary_apply(*{**good, **kw}.values())

    for bad in (dict(h=None), dict(dtype=7), dict(pos=None), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(tokens=-1), dict(qh=-1), dict(kh=-2), dict(qh=2000), dict(qs=255), dict(kos=127)):
        assert call(**bad) == -2, bad
    for bad in (dict(q=FAKE + 1), dict(ko=FAKE + 1), dict(pos=FAKE + 2)):
        assert call(**bad) == -3, bad
    assert call(tokens=0) == 0 and call(qh=0, kh=0) == 0


def paged_config(q_heads=4, kv_heads=2, head_dim=128, pages=8, page_tokens=16, dtype=0, fmt=0, scale=0.0, impl=0,
                 max_ctas=0):
    return arl2.Arl2PagedConfig(q_heads, kv_heads, head_dim, pages, page_tokens, dtype, fmt, scale, impl, max_ctas)


def test_paged_config_is_validated():
    lib, h = arl2._lib, ctypes.c_void_p()
    assert lib.arl2_paged_create(None, None, ctypes.byref(h)) == -1
    assert lib.arl2_paged_create(ctypes.byref(paged_config()), None, None) == -1
    for bad in (dict(dtype=2), dict(fmt=2), dict(impl=3), dict(scale=-1.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(max_ctas=-1)):
        assert lib.arl2_paged_create(ctypes.byref(paged_config(**bad)), None, ctypes.byref(h)) == -1, bad
    for bad in (dict(q_heads=0), dict(kv_heads=0), dict(q_heads=5), dict(q_heads=1026, kv_heads=1026),
                dict(q_heads=130, kv_heads=2), dict(head_dim=0), dict(head_dim=129), dict(pages=0), dict(page_tokens=8),
                dict(page_tokens=48), dict(page_tokens=512), dict(page_tokens=0)):
        assert lib.arl2_paged_create(ctypes.byref(paged_config(**bad)), None, ctypes.byref(h)) == -2, bad
    assert lib.arl2_paged_create(ctypes.byref(paged_config(head_dim=64)), None, ctypes.byref(h)) == -7
    assert h.value is None


def test_null_handles_are_rejected():
    lib = arl2._lib
    pool, batch = arl2.Arl2PagedPool(FAKE, FAKE, None, None), arl2.Arl2PagedBatch(1, 1, 1, 1, FAKE, FAKE, FAKE)
    p, b = ctypes.byref(pool), ctypes.byref(batch)
    assert lib.arl2_paged_write(None, p, b, FAKE, 0, FAKE, 0, None) == -1
    assert lib.arl2_paged_read(None, p, 1, 1, 1, FAKE, None, FAKE, FAKE, FAKE, None) == -1
    assert lib.arl2_paged_attend(None, p, b, 1, 0, 0, FAKE, 0, FAKE, None) == -1
    assert lib.arl2_paged_forward(None, p, b, None, None, 1, 0, 0, FAKE, 0, FAKE, 0, FAKE, 0, None, FAKE, None) == -1
    assert lib.arl2_paged_device_status(None, None) == -1
    assert lib.arl2_paged_device_bytes(None) == 0 and lib.arl2_paged_kernel_launches(None) == 0
    lib.arl2_paged_destroy(None)


def test_python_checks():
    with pytest.raises(KeyError):
        arl2.RotaryAxes(128, [128], pairs="none")
    with pytest.raises(arl2.Arl2Error):
        arl2.RotaryAxes(128, [64, 64, 2])
    with pytest.raises(arl2.Arl2Error):
        arl2.RotaryAxes(128, [2, 2, 2, 2, 2])
    plan = arl2.RotaryAxes(8, [8])
    with pytest.raises(ValueError):
        plan.apply(torch.zeros(1, 1, 8), None, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        arl2.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                        torch.zeros(1, 1, dtype=torch.int32))
    plan.close()
    with pytest.raises(RuntimeError):
        plan.handle
