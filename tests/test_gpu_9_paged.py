"""The paged cache, its attention and the rotary positions on the GPU, against
the definitions in 64 bits (tests/paged_reference.py)."""
import numpy as np
import pytest
import torch

import paged_reference as ref
from hybrid_softmax_gated_b200 import Arl2Error, PagedBatch, PagedCache, RotaryAxes, TeacherLayer

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def make(case, impl="auto", max_ctas=0, layers=1):
    c = PagedCache(case.hq, case.hk, case.d, case.pages, case.page, dtype=case.dtype, layers=layers,
                   cache_format=case.store, impl=impl, max_ctas=max_ctas)
    for i in range(layers):
        c.k_pages[i].view(torch.uint8).copy_(case.kp.view(torch.uint8))
        c.v_pages[i].view(torch.uint8).copy_(case.vp.view(torch.uint8))
        if case.store == "e4m3":
            c.k_scales[i].copy_(case.ks)
            c.v_scales[i].copy_(case.vs)
    return c


def batch_of(case, max_new=None):
    return PagedBatch(case.q_offsets.cuda(), case.kv_lens.cuda(), case.table.cuda(),
                      max_new=max([n for n, _ in case.lens] + [0]) if max_new is None else max_new)


def check_attend(case, impl="auto", block=1, window=0, sinks=0, max_ctas=0, max_new=None):
    cache = make(case, impl, max_ctas)
    out = torch.full((case.tokens, case.hq, case.d), 7.0, dtype=case.dtype, device="cuda")
    cache.attend(case.q.cuda(), batch_of(case, max_new), block=block, window=window, sinks=sinks, out=out)
    assert cache.device_status() == 0
    got = out.double().cpu().numpy()
    want, absolute, slack = case.expect(block, window, sinks)
    n = int(case.q_offsets[-1])
    assert (got[n:] == 7.0).all()  # rows of no sequence
    err = np.abs(got[:n] - want[:n])
    tol = case.tolerance(want, absolute, slack, impl)[:n]
    bad = ~(err <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], err[bad][:4], tol[bad][:4], got[:n][bad][:4], want[:n][bad][:4])
    cache.close()
    return got


# dtype, store, impl, head width
FORMS = [(BF16, "native", "auto", 128), (BF16, "e4m3", "auto", 128), (FP32, "native", "auto", 128),
         (FP32, "e4m3", "auto", 40), (BF16, "native", "simt", 64), (BF16, "e4m3", "simt", 7)]


@pytest.mark.parametrize("dtype,store,impl,d", FORMS)
@pytest.mark.parametrize("lens", [
    [(1, 1)], [(1, 2), (1, 15), (1, 16), (1, 17)], [(1, 63), (1, 64), (1, 65)], [(1, 127), (1, 128), (1, 129), (1, 300)],
    [(2, 2), (3, 40), (0, 9), (1, 130)], [(17, 17)], [(130, 130)], [(129, 300), (1, 5), (64, 64)],
    [(0, 0), (5, 5), (0, 7)],
])
def test_attend_lengths(dtype, store, impl, d, lens):
    check_attend(ref.Case(lens, 4, 2, d=d, dtype=dtype, store=store, seed=3, extra_rows=2), impl)


@pytest.mark.parametrize("dtype,store,impl,d", FORMS)
@pytest.mark.parametrize("block,window,sinks", [
    (1, 1, 0), (1, 3, 2), (1, 64, 0), (1, 65, 1), (1, 100, 130), (1, 128, 128), (1, 1000, 4), (40, 0, 0), (40, 1, 0),
    (40, 2, 1), (40, 3, 9), (7, 5, 3), (1 << 30, 3, 0),
])
def test_attend_masks(dtype, store, impl, d, block, window, sinks):
    lens = [(90, 410), (1, 333), (41, 41), (1, 1), (37, 200)]
    check_attend(ref.Case(lens, 2, 2, d=d, dtype=dtype, store=store, seed=5, page=32), impl, block, window, sinks)


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (6, 3), (5, 1), (16, 2), (12, 1), (24, 1), (64, 1), (40, 1), (12, 12)])
def test_attend_head_groups(store, hq, hk):
    for lens in ([(1, 150), (1, 40)], [(3, 150), (70, 90)]):
        check_attend(ref.Case(lens, hq, hk, store=store, seed=7), "auto", window=64, sinks=3)


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attend_page_sizes(store, page):
    check_attend(ref.Case([(1, 700), (150, 600), (5, 257)], 2, 2, page=page, store=store, seed=11), window=200, sinks=20)


@pytest.mark.parametrize("dtype,store,impl,d", FORMS)
def test_attend_left_padded_chunk(dtype, store, impl, d):
    """Rows before position 0 (more new rows than the sequence is long) give
    zeros and do not disturb the others."""
    got = check_attend(ref.Case([(9, 4), (3, 0), (200, 100), (1, 1)], 4, 2, d=d, dtype=dtype, store=store, seed=2), impl)
    assert (got[:5] == 0).all() and (got[9:12] == 0).all()


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("max_ctas", [0, 1, 2, 7, 40])
@pytest.mark.parametrize("lens", [[(1, 3000), (1, 900), (1, 10)], [(140, 1500), (30, 2100)]])
def test_attend_split_over_ctas(store, max_ctas, lens):
    """Tiles cut between CTAs are merged: few CTAs, many, and a long context."""
    case = ref.Case(lens, 2, 1, page=64, store=store, seed=13)
    for dtype_impl in ("auto", "simt"):
        a = check_attend(case, dtype_impl, max_ctas=max_ctas)
        b = check_attend(case, dtype_impl, max_ctas=max_ctas)
        assert (a == b).all()  # the merge order does not depend on who arrives last


def test_attend_max_new_is_only_a_hint():
    case = ref.Case([(1, 200), (40, 300), (1, 7)], 4, 4, seed=17)
    for max_new in (0, 1, 40, 10 ** 6):
        check_attend(case, max_new=max_new)


@pytest.mark.parametrize("dtype,store,impl,d", FORMS)
@pytest.mark.parametrize("block,window,sinks,new", [(1, 0, 0, 1), (1, 20, 3, 1), (1, 20, 3, 150), (40, 2, 1, 80)])
def test_unseen_keys_have_no_effect(dtype, store, impl, d, block, window, sinks, new):
    """Infinities and NaN in slots past the end, in pages of nobody and in
    keys that a query does not see leave its output bit for bit."""
    lens = [(new, 333), (1, 50)]
    case = ref.Case(lens, 2, 2, d=d, dtype=dtype, store=store, seed=19, page=32)
    clean = check_attend(case, impl, block, window, sinks)
    cache = make(case, impl)
    used = torch.zeros(case.pages, case.page, dtype=torch.bool)
    live = {}
    for s, (n, t) in enumerate(lens):
        for j in range(t):
            used[int(case.table[s, j // case.page]), j % case.page] = True
            live[(s, j)] = (int(case.table[s, j // case.page]), j % case.page)
    bad = [float("nan"), float("inf"), float("-inf")]
    spots = [(int(p), int(sl)) for p, sl in (~used).nonzero()]
    hurt = 200  # a live key of sequence 0: rows that see it may change, the others not
    spots.append(live[(0, hurt)])
    for i, (p, sl) in enumerate(spots):
        for x, sc in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
            if store == "e4m3":
                x[0, p, :, sl].view(torch.uint8).fill_(0x7f)  # the NaN code
                sc[0, p, :, sl] = bad[i % 3] if i < len(spots) - 1 else bad[0]
            else:
                x[0, p, :, sl] = bad[i % 3] if i < len(spots) - 1 else bad[0]
    out = cache.attend(case.q.cuda(), batch_of(case), block=block, window=window, sinks=sinks)
    assert cache.device_status() == 0
    got = out.double().cpu().numpy()
    for i in range(new):
        if not ref.bounds(333 - new + i, 333, block, window, sinks)[hurt]:
            want = clean[i]
            err = np.abs(got[i] - want)
            # (a row next to hurt ones may take another path: the same value up to its tolerance)
            tol = case.tolerance(*case_row(case, block, window, sinks), impl)[i]
            assert (err <= 2 * tol).all(), (i, err.max())
        else:
            assert np.isnan(got[i]).any(), i
    assert (got[new:] == clean[new:]).all()


_rows = {}


def case_row(case, block, window, sinks):
    key = (id(case), block, window, sinks)
    if key not in _rows:
        _rows.clear()
        _rows[key] = case, case.expect(block, window, sinks)  # (the case kept alive: its id is not used again)
    return _rows[key][1]


def test_attend_large_scores_stay_finite():
    """Scores of several hundred: the running maximum keeps the weights finite."""
    check_attend(ref.Case([(1, 500), (90, 400)], 2, 2, seed=23, spread=60.0))
    check_attend(ref.Case([(1, 500), (90, 400)], 2, 2, store="e4m3", seed=23, spread=60.0))


@pytest.mark.parametrize("impl", ["auto", "simt"])
def test_strided_tokens(impl):
    """q, k, v as slices of one joint projection."""
    case = ref.Case([(5, 90), (1, 33), (60, 60)], 4, 2, seed=29)
    joint = torch.empty(case.tokens, (4 + 2 + 2) * 128, dtype=BF16, device="cuda")
    q, k, v = (t.view(case.tokens, h, 128) for t, h in zip(joint.split([512, 256, 256], 1), (4, 2, 2)))
    q.copy_(case.q), k.copy_(case.k), v.copy_(case.v)
    batch = batch_of(case)
    a, b = make(case, impl), make(case, impl)
    a.write(k, v, batch)
    b.write(case.k.cuda(), case.v.cuda(), batch)
    assert torch.equal(a.k_pages, b.k_pages) and torch.equal(a.v_pages, b.v_pages)
    assert torch.equal(a.attend(q, batch), b.attend(case.q.cuda(), batch))


@pytest.mark.parametrize("dtype,store,d", [(BF16, "native", 128), (BF16, "e4m3", 128), (FP32, "native", 128),
                                           (FP32, "e4m3", 128), (BF16, "e4m3", 64), (FP32, "e4m3", 64),
                                           (FP32, "e4m3", 33), (FP32, "native", 5), (BF16, "e4m3", 100)])
@pytest.mark.parametrize("lens", [[(1, 1)], [(3, 40), (0, 5), (1, 17), (9, 4), (2, 0)], [(900, 1000), (7, 700)]])
def test_write_and_read_back(dtype, store, d, lens):
    case = ref.Case(lens, 3, 3, d=d, dtype=dtype, store=store, seed=31, extra_rows=3)
    case.k[0, 0] = 0.0                       # a row of zeros
    if dtype == FP32:
        case.k[0, 1] *= 1e-38                # its scale is the smallest one
    case.v[0, 1] *= 1e30
    if lens[0][0] > 2:
        case.k[1, 2, d // 2] = float("inf")
        case.v[2, 0, 0] = float("nan")
    cache = make(case, "auto" if d == 128 else "simt")
    batch = batch_of(case)
    before = [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8))]
    cache.write(case.k.cuda(), case.v.cuda(), batch)
    assert cache.device_status() == 0
    touched = torch.zeros(case.pages, case.page, dtype=torch.bool)
    for name, src, pages, scales in (("k", case.k, cache.k_pages, cache.k_scales),
                                     ("v", case.v, cache.v_pages, cache.v_scales)):
        codes, want_s = ref.quantise(src) if store == "e4m3" else (src, None)
        pages = pages[0].cpu()
        for s, (n, t) in enumerate(lens):
            for i in range(n):
                j = t - n + i
                if j < 0:
                    continue
                p, sl, row = int(case.table[s, j // case.page]), j % case.page, int(case.q_offsets[s]) + i
                touched[p, sl] = True
                assert torch.equal(pages[p, :, sl].view(torch.uint8), codes[row].view(torch.uint8)), (name, s, i)
                if store == "e4m3":
                    got_s = scales[0, p, :, sl].cpu()
                    assert torch.equal(got_s.view(torch.int32)[~want_s[row].isnan()],
                                       want_s[row].view(torch.int32)[~want_s[row].isnan()])
                    assert torch.equal(got_s.isnan(), want_s[row].isnan())
    for old, new in zip(before, (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8))):
        keep = ~touched.cuda()
        assert torch.equal(old[0].transpose(1, 2)[keep], new[0].transpose(1, 2)[keep])  # nothing else
    # back again
    total = [t for _, t in lens]
    offs = torch.tensor(np.cumsum([0] + total), dtype=torch.int32).cuda()
    kr, vr = (torch.full((sum(total) + 2, 3, d), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    cache.read(case.table.cuda(), offs, sum(total) + 2, k_out=kr, v_out=vr)
    assert cache.device_status() == 0
    for got, pages, scales in ((kr, cache.k_pages, cache.k_scales), (vr, cache.v_pages, cache.v_scales)):
        assert (got[sum(total):] == 9.0).all()
        x = pages[0].float().cpu()
        if scales is not None:
            x = x * scales[0].cpu()[..., None]
        at = 0
        for s, t in enumerate(total):
            for j in range(t):
                want = x[int(case.table[s, j // case.page]), :, j % case.page].to(dtype)
                assert torch.equal(torch.nan_to_num(got[at].cpu(), nan=-1.0), torch.nan_to_num(want, nan=-1.0))
                at += 1
    # a part of each
    starts = torch.tensor([max(0, t // 2 - 1) for t in total], dtype=torch.int32)
    count = [min(2, t - int(st)) if t else 0 for t, st in zip(total, starts)]
    offs2 = torch.tensor(np.cumsum([0] + count), dtype=torch.int32).cuda()
    k2, _ = cache.read(case.table.cuda(), offs2, sum(count), starts=starts.cuda())
    at = 0
    for s, n in enumerate(count):
        a = int(offs[s]) + int(starts[s])
        assert torch.equal(torch.nan_to_num(k2[at:at + n].float()), torch.nan_to_num(kr[a:a + n].float()))
        at += n


ROT = [("128", "adjacent", "per_axis", 128), ("44,42,42", "adjacent", "per_axis", 128), ("32,48,48", "halves", "shared", 128),
       ("16,24,24", "halves", "per_axis", 64), ("8,0,6", "adjacent", "shared", 33), ("2", "halves", "per_axis", 2),
       ("10,10,10,10", "halves", "shared", 47), ("64", "halves", "per_axis", 128), ("100,100", "adjacent", "shared", 256)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("axes,pairs,freqs,d", ROT)
@pytest.mark.parametrize("tokens", [1, 3, 601])
def test_rotary(dtype, axes, pairs, freqs, d, tokens):
    dims = [int(a) for a in axes.split(",")]
    g = torch.Generator().manual_seed(37)
    q, k = (torch.randn(tokens, h, d, generator=g).to(dtype) for h in (3, 2))
    pos = torch.randint(-50, 2000, (tokens, len(dims)), generator=g).to(torch.int32)
    pos[0] = 1 << 30  # far
    plan = RotaryAxes(d, dims, base=1e4, pairs=pairs, freqs=freqs)
    for inverse in (False, True):
        qo, ko = plan.apply(q.cuda(), k.cuda(), pos.cuda(), inverse=inverse)
        for got, x in ((qo, q), (ko, k)):
            want = ref.rotary(x, pos, dims, 1e4, pairs, freqs, inverse)
            # the output's rounding, and in fp32 the sine's, the angle's (2 pi
            # 2^-25 each way) and the products': 8 roundings of |x| + |y| in
            # all; the reference's own angle of position 2^30 is good to 2^-23
            size = np.abs(x.double().numpy()).max()
            tol = ref.HALF_STEP[dtype] * np.abs(want) + 2 * size * (8 * 2.0 ** -24 + 2.0 ** -22)
            assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
            assert torch.equal(got.cpu()[..., sum(dims):], x[..., sum(dims):])
    # in place, q alone, and strided tokens
    qc = q.cuda()
    plan.apply(qc, None, pos.cuda(), q_out=qc)
    assert torch.equal(qc, plan.apply(q.cuda(), k.cuda(), pos.cuda())[0])
    wide = torch.zeros(tokens, 3 * d + 5, dtype=dtype, device="cuda")
    view = wide[:, 1:1 + 3 * d].view(tokens, 3, d)
    view.copy_(q)
    plan.apply(view, None, pos.cuda(), q_out=view)
    assert torch.equal(view, qc) and (wide[:, 0] == 0).all() and (wide[:, 1 + 3 * d:] == 0).all()


def test_rotary_gradient_is_the_inverse():
    """d/dx of <apply(x), w> is apply(w, inverse): the formula's and differences
    in fp32."""
    g = torch.Generator().manual_seed(41)
    plan = RotaryAxes(128, [44, 42, 42])
    x, w = (torch.randn(7, 2, 128, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 500, (7, 3), generator=g).to(torch.int32).cuda()
    grad = plan.apply(w, None, pos, inverse=True)[0]
    want = ref.rotary(w.cpu(), pos, [44, 42, 42], 1e4, "adjacent", "per_axis", True)
    assert np.abs(grad.double().cpu().numpy() - want).max() <= 2 * float(w.abs().max()) * 10 * 2.0 ** -24 + 2e-7
    f = lambda t: float((plan.apply(t, None, pos)[0].double() * w.double()).sum())  # noqa: E731
    for i in range(5):
        e = torch.zeros_like(x)
        e.view(-1)[i * 311] = 0.5  # the map is linear: any step
        diff = f(x + e) - f(x - e)
        # 2 x 256 products, each off by a few fp32 roundings of values below 5
        assert abs(diff - float(grad.view(-1)[i * 311])) < 1792 * 2 * 25 * 2.0 ** -24


@pytest.mark.parametrize("impl,d", [("auto", 128), ("simt", 32)])
@pytest.mark.parametrize("store", ["native", "e4m3"])
def test_forward_is_the_three_calls(impl, d, store):
    case = ref.Case([(40, 140), (1, 60), (3, 3), (0, 4)], 4, 2, d=d, store=store, seed=43)
    plan = RotaryAxes(d, [d // 2, d // 4, d // 4])
    pos = torch.randint(0, 90, (case.tokens, 3)).to(torch.int32).cuda()
    batch = batch_of(case)
    q, k, v = case.q.cuda(), case.k.cuda(), case.v.cuda()
    kw = dict(block=20, window=3, sinks=1, layer=1)
    a, b = make(case, impl, layers=2), make(case, impl, layers=2)
    got = a.forward(q, k, v, batch, rotary=plan, positions=pos, **kw)
    qt, kt = plan.apply(q, k, pos)
    b.write(kt, v, batch, layer=1)
    want = b.attend(qt, batch, **kw)
    assert torch.equal(got, want)
    for x, y in ((a.k_pages, b.k_pages), (a.v_pages, b.v_pages)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    case2 = ref.Case([(40, 140), (1, 60), (3, 3), (0, 4)], 4, 2, d=d, store=store, seed=43)
    c = make(case2, impl)
    c.write(k, v, batch)
    assert torch.equal(make(case2, impl).forward(q, k, v, batch), c.attend(q, batch))


def test_rollout_matches_the_teacher_layer():
    """Frames generated one after the other through the paged cache (block =
    tokens per frame, no window) give what the teacher layer's dense cache
    gives: both are within their rounding of the same attention."""
    L, H, frames = 200, 2, 4
    teacher = TeacherLayer(1, H, 128, L, frames)
    pages = 4 * frames
    cache = PagedCache(H, H, 128, pages, 64)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].cuda()
    g = torch.Generator().manual_seed(47)
    for f in range(frames):
        q, k, v = (torch.randn(L, H, 128, generator=g).to(BF16).cuda() for _ in range(3))
        batch = PagedBatch(torch.tensor([0, L], dtype=torch.int32).cuda(),
                           torch.tensor([(f + 1) * L], dtype=torch.int32).cuda(), table, max_new=L)
        a = cache.forward(q, k, v, batch, block=L).float()
        b = teacher.forward(q[None], k[None], v[None], clean_pass=True)[0].float()
        # two roundings (weights, output) on each side of values whose
        # absolute sums stay below the largest |v| = max
        assert (a - b).abs().max() <= 4 * 2.0 ** -8 * float(v.float().abs().max()) * 1.2
    n = frames * L
    kr, _ = cache.read(table, torch.tensor([0, n], dtype=torch.int32).cuda(), n)
    assert torch.equal(kr[None], teacher.cache_get()[0])
    assert cache.device_status() == 0


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("new", [1, 70])
def test_graph_replays_see_new_lengths(store, new):
    """A captured step reads lengths and tables when it is replayed."""
    case = ref.Case([(new, 400), (new, 300)], 4, 2, store=store, seed=53, page=32)
    cache = make(case)
    batch = batch_of(case, max_new=new)
    q, k, v = case.q.cuda(), case.k.cuda(), case.v.cuda()
    plan = RotaryAxes(128, [128])
    pos = torch.zeros(case.tokens, 1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        cache.forward(q, k, v, batch, rotary=plan, positions=pos, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.forward(q, k, v, batch, rotary=plan, positions=pos, out=out)
    for total in ((400, 300), (new, 71), (250, 399)):
        batch.tensors[1].copy_(torch.tensor(total, dtype=torch.int32))
        q.copy_(torch.randn_like(q))
        pos.fill_(total[0])
        graph.replay()
        got = out.clone()
        fresh = make(case)
        for x, y in ((fresh.k_pages, cache.k_pages), (fresh.v_pages, cache.v_pages)):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        if store == "e4m3":
            fresh.k_scales.copy_(cache.k_scales), fresh.v_scales.copy_(cache.v_scales)
        assert torch.equal(got, fresh.forward(q, k, v, batch, rotary=plan, positions=pos))
        # (399 keys are more than the second sequence's table has pages for)
        assert cache.device_status() == (-1 if total[1] > 300 else 0)


def test_side_stream():
    case = ref.Case([(1, 400), (60, 300)], 4, 2, seed=59)
    cache, batch = make(case), batch_of(case)
    q = case.q.cuda()
    want = cache.attend(q, batch)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = cache.attend(q, batch, stream=s)
        s.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,store,impl", [(BF16, "native", "auto"), (BF16, "e4m3", "auto"), (FP32, "native", "auto")])
@pytest.mark.parametrize("new", [1, 40])
def test_wrong_tables_are_reported(dtype, store, impl, new):
    """Lengths past the table, offsets out of order and page numbers outside
    the pool are caught before they become an address; the other sequences
    and the handle stay usable."""
    lens = [(new, 100), (new, 90), (new, 80)]
    case = ref.Case(lens, 2, 2, dtype=dtype, store=store, seed=61)
    good = check_attend(case, impl)
    cache = make(case, impl)
    q, k, v = case.q.cuda(), case.k.cuda(), case.v.cuda()
    width = case.table.shape[1]

    def run(offs=None, kv=None, table=None):
        b = PagedBatch((case.q_offsets if offs is None else offs).cuda(), (case.kv_lens if kv is None else kv).cuda(),
                       (case.table if table is None else table).cuda(), max_new=new)
        out = cache.attend(q, b)
        assert cache.device_status() == -1
        cache.write(k, v, b)
        assert cache.device_status() == -1
        cache.k_pages[0].view(torch.uint8).copy_(case.kp.view(torch.uint8))
        cache.v_pages[0].view(torch.uint8).copy_(case.vp.view(torch.uint8))
        if store == "e4m3":
            cache.k_scales[0].copy_(case.ks), cache.v_scales[0].copy_(case.vs)
        return out.double().cpu().numpy()

    for kv in ([100, 16 * width + 1, 80], [100, -1, 80], [100, 2 ** 31 - 1, 80]):
        got = run(kv=torch.tensor(kv, dtype=torch.int32))
        assert (got[:new] == good[:new]).all() and (got[2 * new:] == good[2 * new:]).all()
    for page in (-1, case.pages, 2 ** 31 - 1, -2 ** 31):
        t = case.table.clone()
        t[1, 89 // 16] = page  # (the page of the sequence's last key: written too)
        got = run(table=t)
        assert (got[:new] == good[:new]).all() and (got[2 * new:] == good[2 * new:]).all()
    run(offs=torch.tensor([0, 2 * new, new, 3 * new], dtype=torch.int32))
    run(offs=torch.tensor([0, new, 2 * new, 3 * new + 1], dtype=torch.int32))
    run(offs=torch.tensor([0, -5, 2 * new, 3 * new], dtype=torch.int32))
    assert (cache.attend(q, batch_of(case)).double().cpu().numpy() == good).all() and cache.device_status() == 0


def test_refusals():
    case = ref.Case([(2, 20)], 4, 2, seed=67)
    cache, batch = make(case), batch_of(case)
    q, k, v = case.q.cuda(), case.k.cuda(), case.v.cuda()
    for bad in (q.float(), q[:, :3], q[..., :64], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError):
            cache.attend(bad, batch)
    with pytest.raises(ValueError):
        cache.write(k, v[:1], batch)
    with pytest.raises(ValueError):
        cache.attend(q, batch, out=torch.empty(2, 4, 256, dtype=BF16, device="cuda")[..., ::2])
    with pytest.raises(ValueError):
        cache.attend(q, batch, layer=1)
    for kw in (dict(block=0), dict(window=-1), dict(sinks=-1)):
        with pytest.raises(Arl2Error):
            cache.attend(q, batch, **kw)
    with pytest.raises(Arl2Error):
        cache.attend(q, batch, out=q)
    buf = torch.empty(2 * 512 + 1, dtype=BF16, device="cuda")[1:].view(2, 4, 128)  # not on 16 bytes
    with pytest.raises(Arl2Error):
        cache.attend(buf, batch)
    with pytest.raises(ValueError):
        PagedBatch(torch.zeros(3, dtype=torch.int64).cuda(), case.kv_lens.cuda(), case.table.cuda())
    with pytest.raises(ValueError):
        PagedCache(4, 2, 128, 8, 16, pool=(q, q, None, None))
    # nothing to do: no sequences, no rows
    empty = PagedBatch(torch.zeros(1, dtype=torch.int32).cuda(), torch.zeros(0, dtype=torch.int32).cuda(),
                       torch.zeros(0, 4, dtype=torch.int32).cuda())
    before = cache.kernel_launches()
    cache.attend(q, empty)
    cache.attend(q[:0], batch)
    cache.write(k[:0], v[:0], batch)
    assert cache.kernel_launches() == before and cache.device_status() == 0


def test_many_sequences():
    lens = [(1, 1 + (i * 37) % 90) for i in range(1024)]
    check_attend(ref.Case(lens, 2, 1, seed=71, page=16))


@pytest.mark.parametrize("dtype,store,impl,d", FORMS)
@pytest.mark.parametrize("new", [1, 30])
def test_pages_behind_the_window_may_be_gone(dtype, store, impl, d, new):
    """Pages that no query of the chunk sees are not looked up."""
    case = ref.Case([(new, 700), (new, 90)], 2, 2, d=d, dtype=dtype, store=store, seed=83, page=16)
    want = check_attend(case, impl, window=100, sinks=20)
    keep = case.table.clone()
    first = 700 - new + 1 - 100  # first key of the first query's window
    keep[0, 2:first // 16] = -1  # (the sinks are in pages 0 and 1)
    cache = make(case, impl)
    b = PagedBatch(case.q_offsets.cuda(), case.kv_lens.cuda(), keep.cuda(), max_new=new)
    got = cache.attend(case.q.cuda(), b, window=100, sinks=20)
    assert cache.device_status() == 0 and (got.double().cpu().numpy() == want).all()


def test_batches_without_a_largest_chunk():
    """max_new unknown: single tokens take the few-row kernel all the same."""
    case = ref.Case([(1, 1 + 37 * i) for i in range(30)], 8, 2, seed=89)
    assert (check_attend(case, max_new=0) == check_attend(case, max_new=1)).all()


def test_two_handles_at_once_on_two_streams():
    """Each handle has its own workspace: cut tiles of both in flight together."""
    cases = [ref.Case([(1, 3000), (1, 2500)], 4, 1, seed=97, page=64), ref.Case([(200, 2500)], 4, 4, seed=101, page=64)]
    caches, batches = [make(c) for c in cases], [batch_of(c) for c in cases]
    qs = [c.q.cuda() for c in cases]
    want = [c.attend(q, b) for c, q, b in zip(caches, qs, batches)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(caches[i].attend(qs[i], batches[i], stream=s))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("maker", ["zeros", "tiny", "huge", "mixed"])
def test_extreme_rows(store, maker):
    """Value rows of zeros, of 1e-30 and of 1e30 beside ordinary ones, and
    queries of the same kinds."""
    case = ref.Case([(1, 300), (40, 200), (3, 60)], 4, 2, store=store, seed=103, page=32)
    gain = {"zeros": 0.0, "tiny": 1e-30, "huge": 1e25, "mixed": None}[maker]
    g = torch.Generator().manual_seed(107)
    x = torch.randn(case.vp.shape, generator=g)
    each = torch.rand(x.shape[:3], generator=g)
    rows = torch.where(each < 0.3, torch.tensor(0.0 if gain is None else gain),
                       torch.where(each < 0.5, torch.tensor(1e-12 if gain is None else 1.0), torch.tensor(1.0)))
    x = x * rows[..., None]
    case.vp, case.vs = ref.quantise(x) if store == "e4m3" else (x.to(BF16), None)
    case.q[0] *= 0.0
    case.q[1] *= 1e-20
    case.q[2, :, ::2] *= 1e-4  # elements far below their row's largest
    check_attend(case)
    check_attend(case, window=64, sinks=5)


@pytest.mark.parametrize("store", ["native", "e4m3"])
@pytest.mark.parametrize("max_ctas", [1, 3])
@pytest.mark.parametrize("new", [1, 20])
def test_many_short_sequences_on_few_ctas(store, max_ctas, new):
    """One ragged block after the other through the same rings, the slots
    behind each sequence's end holding NaN."""
    lens = [(min(new, t), t) for t in (1 + (i * 29) % 140 for i in range(60))]
    case = ref.Case(lens, 2, 2, store=store, seed=79, page=16)
    want = check_attend(case, max_ctas=max_ctas)
    used = torch.zeros(case.pages, case.page, dtype=torch.bool)
    for s, (_, t) in enumerate(lens):
        for j in range(t):
            used[int(case.table[s, j // case.page]), j % case.page] = True
    cache = make(case, max_ctas=max_ctas)
    for p, sl in (~used).nonzero():
        for x, sc in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
            if store == "e4m3":
                x[0, p, :, sl].view(torch.uint8).fill_(0x7f)
                sc[0, p, :, sl] = float("nan")
            else:
                x[0, p, :, sl] = float("nan")
    assert (cache.attend(case.q.cuda(), batch_of(case)).double().cpu().numpy() == want).all()
    assert cache.device_status() == 0


def test_pool_past_four_gigabytes():
    """Rows whose offsets need more than 32 bits."""
    pages, page = 80000, 128  # 2 heads x 128 tokens x 128 features: 2.6e9 elements, 5.2 GB of keys
    cache = PagedCache(2, 2, 128, pages, page, cache_format="native")
    high = torch.tensor([[pages - 1, pages - 2, pages - 3]], dtype=torch.int32).cuda()
    low = torch.tensor([[0, 1, 2]], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(73)
    k, v, q = (torch.randn(300, 2, 128, generator=g).to(BF16).cuda() for _ in range(3))
    offs, lens = torch.tensor([0, 300], dtype=torch.int32).cuda(), torch.tensor([300], dtype=torch.int32).cuda()
    outs = [cache.forward(q, k, v, PagedBatch(offs, lens, t, max_new=300)) for t in (high, low)]
    assert torch.equal(*outs)
    assert torch.equal(cache.read(high, offs, 300)[1], v)
    assert cache.device_status() == 0
