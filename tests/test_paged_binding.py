"""The paged cache's binding: argument checks that need no GPU."""
import pytest
import torch

import hybrid_softmax_gated_b200 as arl2


def test_the_device_must_be_a_gpu():
    with pytest.raises(ValueError, match="device"):
        arl2.PagedCache(2, 2, 128, 4, 16, device="cpu")


class Fake:
    """What the checks ask of a tensor."""

    def __init__(self, shape, dtype, index=0, contiguous=True):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, torch.device("cuda", index), True
        self.is_contiguous = lambda: contiguous


SHAPE = (2, 4, 2, 16, 128)


def pool(e4m3, **change):
    store = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kinds = [(SHAPE, store), (SHAPE, store), (SHAPE[:4], torch.float32), (SHAPE[:4], torch.float32)]
    names = ["k", "v", "ks", "vs"]
    return tuple(None if n not in ("k", "v") and not e4m3 and n not in change else Fake(*kind, **change.get(n, {}))
                 for n, kind in zip(names, kinds))


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_pool_is_on_one_device(e4m3):
    store = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    good = pool(e4m3)
    assert arl2._check_pool(good, SHAPE, store, e4m3) == good
    moved = {n: dict(index=1) for n in ("k", "v", "ks", "vs")}
    if e4m3:
        arl2._check_pool(pool(True, **moved), SHAPE, store, True)  # all on another one
    for n in ("k", "v", "ks", "vs") if e4m3 else ("k", "v"):
        with pytest.raises(ValueError, match="device"):
            arl2._check_pool(pool(e4m3, **{n: dict(index=1)}), SHAPE, store, e4m3)
        with pytest.raises(ValueError, match="contiguous"):
            arl2._check_pool(pool(e4m3, **{n: dict(contiguous=False)}), SHAPE, store, e4m3)
    if e4m3:
        with pytest.raises(ValueError, match="k_scales"):
            arl2._check_pool(good[:2] + (None, good[3]), SHAPE, store, True)
    else:
        with pytest.raises(ValueError, match="none"):
            arl2._check_pool(pool(False, vs={}), SHAPE, store, False)


def test_rotary_takes_at_most_2_30_tokens():
    plan, fake = arl2.RotaryAxes(2, [2]), 0x1000  # never dereferenced

    def call(tokens):
        return arl2._lib.arl2_rotary_apply(plan.handle, 0, tokens, fake + 2, 1, fake, 0, fake, 0, 0, None, 0, None, 0, 0, None)

    assert call(2 ** 30) == -3  # (the misaligned positions come next)
    for tokens in (2 ** 30 + 1, 2 ** 31 - 32, 2 ** 31 - 1):
        assert call(tokens) == -2


def test_sizes_of_the_mask_keep_their_meaning():
    top = 2 ** 31 - 1
    assert arl2._mask(1, 0, 0) == (1, 0, 0) and arl2._mask(1560, 21, 3) == (1560, 21, 3)
    for big in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1):
        assert arl2._mask(1, big, 0) == (1, top, 0)
        assert arl2._mask(big, 7, big) == (top, 7, top)
    for low in (-1, -2 ** 32 + 5, -2 ** 63):
        assert arl2._mask(1, low, 0) == (1, -1, 0)
