"""The paged cache, its attention and the rotary positions at calls that their
documentation allows and that are easily got wrong: tables out of order, other
streams and devices, values that are not finite, the smallest and largest
numbers."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_softmax_gated_b200 as arl2
import paged_reference as ref
from hybrid_softmax_gated_b200 import PagedBatch, PagedCache, RotaryAxes

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


# ---- streams -----------------------------------------------------------------

def busy(stream, cycles=60_000_000):
    """Tens of milliseconds of nothing on a stream: what follows there is late."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(cycles)


def fill_free_memory(sizes):
    """Takes what the current stream's allocator has free at these sizes, and
    writes it."""
    held = [torch.full((n,), float("nan"), dtype=BF16, device="cuda") for n in sizes for _ in range(8)]
    torch.cuda.current_stream().synchronize()
    return held


def step_case(store="native", new=40):
    case = ref.Case([(new, 300), (3, 90)], 4, 2, store=store, seed=11, page=32)
    cache = PagedCache(4, 2, 128, case.pages, 32, cache_format=store)
    batch = PagedBatch(case.q_offsets.cuda(), case.kv_lens.cuda(), case.table.cuda(), max_new=new)
    positions = torch.arange(case.tokens, dtype=torch.int32)[:, None].cuda()
    return cache, batch, case.q.cuda(), case.k.cuda(), case.v.cuda(), positions


@pytest.mark.parametrize("handle", ["stream", "raw"])
def test_scratch_and_outputs_live_on_the_calls_stream(handle):
    """What a call allocates for another stream is not given away while that
    stream still has to use it."""
    cache, batch, q, k, v, positions = step_case()
    plan = RotaryAxes(128, [128])
    want = cache.forward(q, k, v, batch, rotary=plan, positions=positions)
    turned = plan.apply(q, k, positions)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = s if handle == "stream" else s.cuda_stream
    sizes = [q.shape[0] * (4 + 2) * 128, q.numel(), k.numel()]
    busy(s)
    out = cache.forward(q, k, v, batch, rotary=plan, positions=positions, out=torch.empty_like(q), stream=on)
    held = fill_free_memory(sizes)  # (the scratch was free for the current stream?)
    s.synchronize()
    assert torch.equal(out, want)
    busy(s)
    plan.apply(q, k, positions, stream=on)  # outputs dropped at once
    cache.attend(q, batch, stream=on)
    late = fill_free_memory(sizes)
    s.synchronize()
    assert all(torch.isnan(t).all() for t in held + late)


@pytest.mark.parametrize("handle", ["stream", "raw"])
def test_outputs_on_a_side_stream_are_not_memory_in_use(handle):
    """A block that the current stream has freed but is not done with is no
    output for another stream."""
    cache, batch, q, k, v, positions = step_case()
    plan = RotaryAxes(128, [128])
    want = [cache.attend(q, batch), *plan.apply(q, k, positions), *cache.read(batch.tensors[2][:1], batch.tensors[0][:2], 40)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = s if handle == "stream" else s.cuda_stream
    old = fill_free_memory([q.numel(), k.numel(), 40 * 2 * 128])
    busy(torch.cuda.current_stream())
    for t in old:
        t.fill_(3.0)
    del old, t
    got = [cache.attend(q, batch, stream=on), *plan.apply(q, k, positions, stream=on),
           *cache.read(batch.tensors[2][:1], batch.tensors[0][:2], 40, stream=on)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("handle", ["stream", "raw"])
def test_a_new_cache_is_cleared_on_its_stream(handle, store):
    """Pages written right after the cache was made on a busy day of the
    current stream keep what was written."""
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(64, 2, 128, generator=g).to(BF16).cuda() for _ in range(2))
    table, offsets = torch.arange(4, dtype=torch.int32)[None].cuda(), torch.tensor([0, 64], dtype=torch.int32).cuda()
    batch = PagedBatch(offsets, offsets[1:], table)
    PagedCache(2, 2, 128, 4, 16, cache_format=store).close()  # (memory that the current stream has at hand)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy(torch.cuda.current_stream())
    on = s if handle == "stream" else s.cuda_stream
    cache = PagedCache(2, 2, 128, 4, 16, cache_format=store, stream=on)
    cache.write(k, v, batch, stream=on)
    s.synchronize()
    torch.cuda.synchronize()
    got = cache.read(table, offsets, 64)
    if store == "native":
        assert torch.equal(got[0], k) and torch.equal(got[1], v)
    for x, y in zip(got, (k, v)):  # (a code is off by half a step of 2^-4 at most, and the value is rounded once)
        tol = (2.0 ** -4 + 2.0 ** -8) * y.float().abs() + 2.0 ** -10 * y.float().abs().amax(-1, keepdim=True) / 448
        assert ((x.float() - y.float()).abs() <= tol * 1.01).all()


def test_a_device_without_an_index_is_the_current_one():
    cache = PagedCache(2, 2, 128, 4, 16, device="cuda")
    assert cache.device == torch.device("cuda", torch.cuda.current_device()) == cache.k_pages.device
    k = torch.randn(5, 2, 128, device="cuda").to(BF16)
    table, offsets = torch.arange(4, dtype=torch.int32)[None].cuda(), torch.tensor([0, 5], dtype=torch.int32).cuda()
    batch = PagedBatch(offsets, offsets[1:], table)
    cache.write(k, k, batch)
    cache.attend(k, batch)
    assert torch.equal(cache.read(table, offsets, 5)[0], k) and cache.device_status() == 0


# ---- values that are not finite -------------------------------------------------

def loaded(case, impl="auto", max_ctas=0):
    cache = PagedCache(case.hq, case.hk, case.d, case.pages, case.page, dtype=case.dtype, cache_format=case.store,
                       impl=impl, max_ctas=max_ctas)
    raw(cache.k_pages)[0].copy_(raw(case.kp))
    raw(cache.v_pages)[0].copy_(raw(case.vp))
    if case.store == "e4m3":
        cache.k_scales[0].copy_(case.ks)
        cache.v_scales[0].copy_(case.vs)
    batch = PagedBatch(case.q_offsets.cuda(), case.kv_lens.cuda(), case.table.cuda(), max_new=max(n for n, _ in case.lens))
    return cache, batch


def spoil(cache, case, s, j, head, feature, x):
    """Key j's value of sequence s: not finite (codes: the whole row)."""
    at = int(case.table[s, j // case.page]), j % case.page
    if case.store == "e4m3":
        cache.v_scales[0, at[0], head, at[1]] = float("nan")
    else:
        cache.v_pages[0, at[0], head, at[1], feature] = x


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("hq,hk", [(2, 2), (6, 2), (2, 1)])
@pytest.mark.parametrize("new,total,block,window,sinks", [
    (3, 700, 1, 0, 0), (8, 3000, 1, 500, 20), (5, 900, 3, 40, 7), (300, 1500, 1, 0, 0), (300, 1500, 1, 400, 300),
    (280, 1400, 100, 3, 1), (150, 2000, 1000, 1, 0), (600, 600, 1, 0, 0),
])
@pytest.mark.parametrize("max_ctas", [0, 5])
def test_a_value_reaches_the_queries_that_see_it_and_no_other(store, hq, hk, new, total, block, window, sinks, max_ctas):
    """A value that is not finite: the queries that do not see it, other
    heads and other sequences are bit for bit as before; those that see it have
    it, in its feature."""
    case = ref.Case([(new, total), (min(new, 90), 200)], hq, hk, store=store, seed=new + hq, page=64)
    cache, batch = loaded(case, max_ctas=max_ctas)
    q, g = case.q.cuda(), hq // hk
    kw = dict(block=block, window=window, sinks=sinks)
    clean = cache.attend(q, batch, **kw)
    sight = np.stack([ref.bounds(total - new + i, total, block, window, sinks) for i in range(new)])
    some = [j for j in range(total) if sight[:, j].any() and not sight[:, j].all()]
    near = some[len(some) // 3] if some else total - 1
    spots = [(near, 5, float("inf")), (near, 70, float("nan")), (total - 1, 5, float("inf")),
             (max(0, total - 2), 64, float("-inf")), (total - new // 2 - 1, 64, float("inf")), (0, 127, float("nan"))]
    gone = [(int(case.table[0, j // 64]), j % 64) for j in range(total) if not sight[:, j].any()]
    for p, sl in gone:  # keys that nobody sees
        (cache.v_scales if store == "e4m3" else cache.v_pages)[0, p, :, sl] = float("nan")
        if store == "e4m3":
            raw(cache.v_pages)[0, p, :, sl] = 0x7f
    assert torch.equal(cache.attend(q, batch, **kw), clean)
    for j, f, x in spots:
        spoil(cache, case, 0, j, 0, f, x)
    got = cache.attend(q, batch, **kw)
    assert cache.device_status() == 0
    want = clean.clone()
    held = {(j, f): x for j, f, x in spots}  # (the same element twice: the last one)
    for i in range(new):
        for (j, f), x in held.items():
            if sight[i, j]:
                want[i, :g, slice(None) if store == "e4m3" else f] += x
    assert torch.equal(got.isnan(), want.isnan())
    where = ~want.isnan()
    # (an element that is not finite leaves its row's other features alone)
    assert torch.equal(got[where], want[where])


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("new", [8, 1000])
def test_a_value_that_is_not_finite_costs_no_second_computation(store, new):
    """One such value, seen by all, by some or by few queries of a chunk on a
    long history: right, and not slower by more than the keys at the mask's edge."""
    total = 30000
    case = ref.Case([(new, total), (5, 400)], 2, 2, store=store, seed=3, page=256)
    cache, batch = loaded(case)
    q = case.q.cuda()

    def timed():
        torch.cuda.synchronize()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        cache.attend(q, batch)
        b.record()
        b.synchronize()
        return a.elapsed_time(b)

    clean = cache.attend(q, batch)
    usual = min(timed() for _ in range(5))
    for hurt in (100, total - new // 2, total - 2):
        raw(cache.v_pages)[0].copy_(raw(case.vp))
        if store == "e4m3":
            cache.v_scales[0].copy_(case.vs)
        spoil(cache, case, 0, hurt, 0, 5, float("nan"))
        got = cache.attend(q, batch)
        first = max(0, hurt - (total - new))  # of the queries that see it
        assert torch.isnan(got[first:new, 0, 5]).all()
        assert torch.equal(got[:first], clean[:first]) and torch.equal(got[new:], clean[new:])
        assert torch.equal(got[:, 1], clean[:, 1])
        assert min(timed() for _ in range(3)) < 5 * usual + 0.3  # milliseconds
        assert cache.device_status() == 0


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("lens", [[(40, 25), (3, 60)], [(300, 200), (5, 90)], [(6, 3), (2, 1)], [(200, 130), (150, 700)],
                                  [(8, 0), (1, 5)]])
@pytest.mark.parametrize("max_ctas", [0, 1])
def test_padding_on_the_left_may_hold_anything(store, lens, max_ctas):
    """Rows at negative positions: zeros, whatever their queries and the
    others' values are."""
    case = ref.Case(lens, 4, 2, store=store, seed=7, page=16)
    cache, batch = loaded(case, max_ctas=max_ctas)
    clean = cache.attend(case.q.cuda(), batch)
    q = case.q.cuda()
    pad = torch.zeros(case.tokens, dtype=torch.bool)
    for s, (n, t) in enumerate(lens):
        pad[int(case.q_offsets[s]):int(case.q_offsets[s]) + max(0, n - t)] = True
    for i, at in enumerate(pad.nonzero().flatten().tolist()):
        q[at] = [float("nan"), float("inf"), float("-inf"), 3e38][i % 4]
    got = cache.attend(q, batch)
    assert cache.device_status() == 0
    assert torch.equal(got, clean) and (got[pad.cuda()] == 0).all()
    s, t = next((s, t) for s, (_, t) in enumerate(lens) if t)
    spoil(cache, case, s, t // 2, 0, 9, float("nan"))
    got = cache.attend(q, batch)
    assert (got[pad.cuda()] == 0).all()
    assert torch.equal(got[:, 2:], clean[:, 2:])


@pytest.mark.parametrize("dtype,store,impl", [(BF16, "native", "auto"), (BF16, "e4m3", "auto"), (FP32, "native", "auto"),
                                              (FP32, "e4m3", "auto"), (BF16, "e4m3", "simt"), (BF16, "native", "simt")])
@pytest.mark.parametrize("new", [1, 6, 100])
def test_a_value_counts_however_small_its_weight(dtype, store, impl, new):
    """A value that is not finite and has a weight that rounds to 0 reaches the
    queries that see it all the same: 0 x infinity is no number."""
    total = 300
    case = ref.Case([(new, total)], 2, 2, dtype=dtype, store=store, seed=13, page=32)
    case.q = torch.ones_like(case.q)
    case.kp, case.ks = case.kp.float() * 0 + 1, None  # scores of 0 ...
    for j in (total - 2, total - new, 40):
        case.kp[int(case.table[0, j // 32]), :, j % 32] = -100.0  # ... and of -1143
    if store == "e4m3":
        case.kp, case.ks = ref.quantise(case.kp)
    else:
        case.kp = case.kp.to(dtype)
    cache, batch = loaded(case, impl)
    q = case.q.cuda()
    clean = cache.attend(q, batch)
    assert torch.isfinite(clean).all()
    for j in (total - 2, total - new, 40):
        raw(cache.v_pages)[0].copy_(raw(case.vp))
        if store == "e4m3":
            cache.v_scales[0].copy_(case.vs)
        spoil(cache, case, 0, j, 0, 77, float("inf"))
        got = cache.attend(q, batch)
        first = max(0, j - (total - new))
        assert not torch.isfinite(got[first:, 0, 77]).any(), j
        assert torch.equal(got[:first], clean[:first]) and torch.equal(got[:, 1], clean[:, 1])
        if store == "native":  # the key is infinite as well: a weight of 0 exactly
            cache.k_pages[0, int(case.table[0, j // 32]), 0, j % 32, 3] = float("-inf")
            assert not torch.isfinite(cache.attend(q, batch)[first:, 0, 77]).any(), j
            raw(cache.k_pages)[0].copy_(raw(case.kp))


@pytest.mark.parametrize("gain", [1.0, 1e-27, 1e-30, 1e-34, 1e30])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 40)], [(4, 700), (2, 90)]])
@pytest.mark.parametrize("max_ctas", [0, 3])
@pytest.mark.parametrize("mixed", [False, True])
def test_weights_of_few_rows_over_codes(gain, lens, max_ctas, mixed):
    """Few query rows over codes: weights to 12 bits, however small or large all
    of a row's values are; mixed: every seventh value row is of zeros, every
    fifth a thousand times smaller.

    Off by: the output's rounding; a weight's three terms (2^-12 of the weight, and
    2^-25 of the row's largest weight times value scale, counted against a value of
    448 scales: 2^-16 of the largest contribution); q in two terms, 2^-17 of its
    row's largest element in each of d products, which moves a score by delta and the
    weights by 2 delta; fp32 sums as in the other tests."""
    case = ref.Case(lens, 4, 1, store="e4m3", seed=31, page=32)
    g = torch.Generator().manual_seed(37)
    x = gain * torch.randn(case.vp.shape, generator=g)
    if mixed:
        x[:, :, ::7] = 0.0
        x[:, :, ::5] *= 1e-3
    case.vp, case.vs = ref.quantise(x)
    cache, batch = loaded(case, max_ctas=max_ctas)
    out = cache.attend(case.q.cuda(), batch)
    assert cache.device_status() == 0
    got = out.double().cpu().numpy()
    want, absolute, slack = case.expect()
    v = np.abs(case.values("v").numpy()).max()
    n, q, k = max(t for _, t in lens), case.q.double().abs(), case.values("k").abs().max().item()
    delta = (2.0 ** -17 * q.amax(-1, keepdim=True) * k * 128 * 128 ** -0.5).numpy()
    tol = 2.0 ** -8 * np.abs(want) + absolute * (2 * slack + 2 * delta + (16 + n / 16) * 2.0 ** -24 + 2.0 ** -12) \
        + 2.0 ** -16 * v
    bad = ~(np.abs(got - want) <= 1.01 * tol)
    assert not bad.any(), (np.abs(got - want)[bad][:4], tol[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype,impl", [(BF16, "auto"), (FP32, "auto"), (BF16, "simt")])
@pytest.mark.parametrize("new,max_ctas", [(1, 0), (1, 2), (40, 0), (40, 3), (5, 1)])
def test_weights_of_nothing_but_minus_infinity(dtype, impl, new, max_ctas):
    """Queries all of whose scores are -infinity: every weight is 0, so a finite
    value gives 0 and one that is not finite no number."""
    case = ref.Case([(new, 600), (3, 700)], 2, 2, dtype=dtype, seed=47, page=32)
    case.q = torch.ones_like(case.q)
    cache, batch = loaded(case, impl, max_ctas)
    q = case.q.cuda()
    other = cache.attend(q, batch)[new:]
    for j in range(600):
        cache.k_pages[0, int(case.table[0, j // 32]), :, j % 32, 8] = float("-inf")
    assert (cache.attend(q, batch)[:new] == 0).all()
    spoil(cache, case, 0, 11, 0, 77, float("inf"))
    spoil(cache, case, 0, 599, 1, 12, float("-inf"))
    got = cache.attend(q, batch)
    assert torch.equal(got[new:], other) and cache.device_status() == 0
    assert not torch.isfinite(got[:new, 0, 77]).any() and not torch.isfinite(got[new - 1, 1, 12])
    got[:new, 0, 77], got[new - 1, 1, 12] = 0, 0
    assert (got[:new] == 0).all()


# ---- sizes -----------------------------------------------------------------------

def test_more_tokens_than_an_int_can_count_on_are_refused():
    """Nothing is launched: the addresses are never used."""
    cache, batch, q, k, v, positions = step_case()
    lib, fake, before = arl2._lib, 0x1000, cache.kernel_launches()
    p = ctypes.byref(cache._pools[0])
    for tokens in (2 ** 30 + 1, 2 ** 31 - 100, 2 ** 31 - 1):
        b = ctypes.byref(arl2.Arl2PagedBatch(2, tokens, 10, 1, fake, fake, fake))
        assert lib.arl2_paged_write(cache.handle, p, b, fake, 0, fake, 0, None) == -2
        assert lib.arl2_paged_read(cache.handle, p, 2, tokens, 10, fake, None, fake, fake, fake, None) == -2
        assert lib.arl2_paged_attend(cache.handle, p, b, 1, 0, 0, fake, 0, fake * 2, None) == -2
        assert lib.arl2_paged_forward(cache.handle, p, b, None, None, 1, 0, 0, fake, 0, fake, 0, fake, 0, None,
                                      fake * 2, None) == -2
    assert cache.kernel_launches() == before


def test_a_window_longer_than_an_int_is_no_window():
    cache, batch, q, k, v, positions = step_case()
    want = cache.attend(q, batch)
    for big in (2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1):
        assert torch.equal(cache.attend(q, batch, window=big, sinks=big), want)
        assert torch.equal(cache.forward(q, k, v, batch, window=big), cache.forward(q, k, v, batch))
        want = cache.attend(q, batch)
    for kw in (dict(block=-2 ** 32 + 1), dict(window=-2 ** 32 + 5), dict(sinks=-2 ** 63)):
        with pytest.raises(arl2.Arl2Error):
            cache.attend(q, batch, **kw)


@pytest.mark.parametrize("dtype,store,impl", [(BF16, "native", "auto"), (BF16, "e4m3", "auto"), (FP32, "native", "auto"),
                                              (BF16, "e4m3", "simt")])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("keys,queries,values", [
    (1.0, 5e6, 1.0), (1e29, 5e-23, 1e29), (1e-29, 1e29, 1e-29), (1e-29, 1e-29, 1e29), (1e29, 1e-29, 1e-29),
])
def test_magnitudes_over_the_documented_range(dtype, store, impl, new, keys, queries, values):
    """Keys, queries and values from 2^-100 to 2^100, scores up to 2^29: where one
    key's score stands out by more than the scores' rounding, its value; scores
    near 0: within the usual bounds, relative to the values."""
    case = ref.Case([(new, 300), (new, 90)], 4, 2, dtype=dtype, store=store, seed=41, page=32)
    g = torch.Generator().manual_seed(43)
    case.q = (queries * torch.randn(case.q.shape, generator=g)).to(dtype)
    for name, gain in (("k", keys), ("v", values)):
        x = gain * torch.randn(case.kp.shape, generator=g)
        pages, scales = ref.quantise(x) if store == "e4m3" else (x.to(dtype), None)
        setattr(case, name + "p", pages), setattr(case, name + "s", scales)
    cache, batch = loaded(case, impl)
    got = cache.attend(case.q.cuda(), batch).double().cpu().numpy()
    assert cache.device_status() == 0 and np.isfinite(got).all()
    want, absolute, slack = case.expect()
    sharp = 0
    for s, (n, t) in enumerate(case.lens):
        at, k, v = int(case.q_offsets[s]), case.sequence("k", s), case.sequence("v", s)
        for i in range(n):
            for h in range(4):
                score = k[:t - n + i + 1, h // 2] @ case.q[at + i, h].double().numpy() * 128 ** -0.5
                # (q of codes is off by 2^-17 of its row's largest in each of 128 products, fp32 sums by `slack`)
                off = slack[at + i, h, 0] + 2.0 ** -17 * 128 ** 0.5 * case.q[at + i, h].double().abs().max().item() * np.abs(k).max()
                order = np.argsort(score)
                if off < 0.0099:  # (weights move by a factor of e^(2 off) <= 1 + 2.02 off)
                    bound = case.tolerance(want, absolute, slack, impl) - 1.01e-30 + 2.02 * 2 * off * absolute
                    assert (np.abs(got - want) <= bound)[at + i, h].all()
                elif score[order[-1]] - score[order[-2]] > 2 * off + 40:
                    sharp += 1
                    assert (np.abs(got[at + i, h] - v[order[-1], h // 2]) <= 2.0 ** -7 * np.abs(v[order[-1], h // 2])).all()
    assert sharp or off < 0.0099
