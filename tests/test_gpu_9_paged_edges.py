"""The paged cache, its attention and the rotary positions at calls that their
documentation allows and that are easily got wrong: tables out of order, other
streams and devices, values that are not finite, the smallest and largest
numbers."""
import numpy as np
import pytest
import torch

import paged_reference as ref
from hybrid_softmax_gated_b200 import PagedBatch, PagedCache

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


# ---- tables ------------------------------------------------------------------

def shuffled(seqs, tokens, seed):
    """Offsets in a random order, ends in place."""
    inner = torch.randint(0, tokens, (seqs - 1,), generator=torch.Generator().manual_seed(seed)).tolist()
    return [0] + inner + [tokens]


@pytest.mark.parametrize("dtype,store,d", [(BF16, "native", 128), (BF16, "e4m3", 128), (FP32, "e4m3", 64), (FP32, "native", 40)])
@pytest.mark.parametrize("offsets,tokens", [
    ([0, 100, 1, 2], 64), ([0, 2, 100, 3, 5], 100), ([0, 60, 70, 40], 70), ([0, 60, 70, 40], 100), ([5, 3, 9, 64], 64),
    (shuffled(40, 90, 1), 90), (shuffled(300, 200, 2), 200),
])
def test_offsets_out_of_order(dtype, store, d, offsets, tokens):
    """Every row is written to, and read from, its own position of a sequence
    that holds it, or not at all; the error word is set."""
    seqs, page, columns, hk, length = len(offsets) - 1, 16, 14, 2, 210
    g = torch.Generator().manual_seed(5)
    pages = seqs * columns + 64
    cache = PagedCache(2, hk, d, pages, page, dtype=dtype, cache_format=store, impl="auto" if d == 128 else "simt")
    # (a slice: what lies behind the table are pages, too)
    table = torch.randperm(pages, generator=g).to(torch.int32)[:(seqs + 4) * columns].view(-1, columns).cuda()[:seqs]
    batch = PagedBatch(torch.tensor(offsets, dtype=torch.int32).cuda(),
                       torch.full((seqs,), length, dtype=torch.int32).cuda(), table)
    k, v = (torch.randn(tokens, hk, d, generator=g).to(dtype).cuda() for _ in range(2))
    pools = [raw(t) for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales) if t is not None]
    before = [t.clone() for t in pools]
    cache.write(k, v, batch)
    assert cache.device_status() == -1
    free = torch.zeros(pages, page, dtype=torch.bool)  # slots that some row may go to
    for s, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if a <= b <= tokens:
            at = torch.arange(length - (b - a), length)
            at = at[at >= 0]
            free[table.cpu()[s, at // page].long(), at % page] = True
    for now, old in zip(pools, before):
        changed = (now != old)[0].movedim(1, 2)  # [pages, page, heads, ...]
        assert not (changed.flatten(2).any(2).cpu() & ~free).any()
    # reading: a row gets its position's values or is left as it was
    cache.write(*[torch.randn(length, hk, d, generator=g).to(dtype).cuda() for _ in range(2)],
                PagedBatch(*[torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, length], [length])], table[:1]))
    assert cache.device_status() == 0
    whole = [t.clone() for t in cache.read(table, torch.arange(0, (seqs + 1) * length, length, dtype=torch.int32).cuda(),
                                           seqs * length)]
    assert cache.device_status() == 0
    outs = [torch.full((tokens, hk, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    cache.read(table, batch.tensors[0], tokens, k_out=outs[0], v_out=outs[1])
    assert cache.device_status() == -1
    for got, of in zip(outs, whole):
        fine = (got == 7.0).flatten(1).all(1)
        for s, (a, b) in enumerate(zip(offsets, offsets[1:])):
            if a < b <= tokens:
                fine[a:b] |= (got[a:b] == of[s * length:s * length + b - a]).flatten(1).all(1)
        assert fine.all()
