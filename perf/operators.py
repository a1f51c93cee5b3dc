"""Operators around a paged KV cache: what they compute in plain torch, and
the framework's calls for the same.

Three operators, used one after the other by a softmax layer whose keys and
values live in pages (a video stream's frames, or the tokens of a text
model):

  rotary   rotary positions with up to three axes (time, height, width) on q
           and k; `inverse` turns the other way, which is the gradient
  write    new keys and values into their pages, as they are or quantised to
           e4m3 codes with one scale per token and head; read: back again
  attend   a chunk of new tokens per sequence (one token included) against
           everything its sequence has in the pages, causal by token or by
           frame, with an optional window and first blocks that stay visible

`own` picks the side: False computes the plain form, True calls the
framework.
"""
import math
import random

import torch

own = False

BF16, FP32, E4M3 = "bf16", "fp32", "e4m3"
DTYPES = {BF16: torch.bfloat16, FP32: torch.float32}
CODE_MAX = 448.0        # largest e4m3 value
SCALE_MIN = 2.0 ** -126  # smallest scale: a normal number, also for rows of zeros


# ---- cases -----------------------------------------------------------------

def rotary_case(tokens, q_heads, kv_heads, axes, *, dtype=BF16, pairs="adjacent", freqs="per_axis", base=10000.0,
                inverse=False, far=0, **kw):
    return dict(kind="rotary", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, d=128, axes=axes, dtype=dtype,
                pairs=pairs, freqs=freqs, base=base, inverse=inverse, far=far, **kw)


def cache_case(kind, seqs, new, context, kv_heads, *, page=64, dtype=BF16, store=E4M3, lens=1, **kw):
    return dict(kind=kind, seqs=seqs, new=new, context=context, kv_heads=kv_heads, d=128, page=page, dtype=dtype,
                store=store, lens=lens, **kw)


def attend_case(seqs, new, context, q_heads, kv_heads, *, page=64, dtype=BF16, store=BF16, block=1, window=0, sinks=0,
                ragged=True, lens=1, d=128, **kw):
    return dict(kind="attend", seqs=seqs, new=new, context=context, q_heads=q_heads, kv_heads=kv_heads, d=d, page=page,
                dtype=dtype, store=store, block=block, window=window, sinks=sinks, ragged=ragged, lens=lens, **kw)


def listed():
    return [
        # one generated token of a text stream: latency
        rotary_case(1, 12, 12, "128", far=40000, name="rotary_token"),
        # a 720p frame of four video streams, time, height and width
        rotary_case(14400, 12, 12, "44,42,42", name="rotary_frames_720p"),
        # the gradient of a 480p frame's rotation in fp32, shared key heads,
        # halves paired and frequencies shared by the axes
        rotary_case(1560, 32, 8, "32,48,48", dtype=FP32, pairs="halves", freqs="shared", base=1e6, inverse=True,
                    name="rotary_grad_480p"),
        # one new token for each of 24 streams, quantised into its page
        cache_case("write", 24, 1, 900, 12, name="write_tokens_e4m3"),
        # a clean 480p frame of four streams, quantised as it is written
        cache_case("write", 4, 1560, 1560, 12, name="write_frames_e4m3"),
        # a stream's quantised history read back (a checkpoint, another layer)
        cache_case("read", 3, 1, 9360, 12, name="read_history_e4m3"),
        # the smallest serving step: four short streams, one token each
        attend_case(4, 1, 300, 12, 12, store=E4M3, name="attend_few_tokens_e4m3"),
        # a serving step of 48 text streams with shared key heads, ragged contexts
        attend_case(48, 1, 12000, 32, 8, page=32, name="attend_tokens_gqa"),
        # the same with a quantised cache, a rolling window and sinks
        attend_case(64, 1, 24000, 32, 8, store=E4M3, window=8192, sinks=64, name="attend_tokens_window_e4m3"),
        # one denoising pass of a 480p frame over a rolling window of 21
        # frames, the first three kept visible
        attend_case(1, 1560, 62400, 12, 12, page=128, block=1560, window=21, sinks=3, ragged=False,
                    name="attend_frame_window"),
        # the same over a quantised history, two streams of unlike length
        attend_case(2, 1560, 18720, 12, 12, page=64, store=E4M3, block=1560, name="attend_frames_e4m3"),
        # chunks of prompts, causal by token, shared key heads, odd lengths
        attend_case(5, 1500, 5000, 32, 8, page=16, name="attend_prompts_gqa"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "write", "read", "attend", "attend", "attend"])
    heads = rng.choice([(12, 12), (32, 8), (16, 2), (8, 1), (24, 8), (6, 6)])
    lens = rng.randrange(1 << 30)
    if kind == "rotary":
        return rotary_case(log_int(rng, 1, 12000), *heads, rng.choice(["44,42,42", "32,48,48", "128", "64,64", "16,24,24"]),
                           dtype=rng.choice([BF16, BF16, FP32]), pairs=rng.choice(["adjacent", "halves"]),
                           freqs=rng.choice(["per_axis", "shared"]), base=rng.choice([1e4, 1e6]),
                           inverse=rng.random() < 0.5, far=rng.choice([0, 0, 100000]))
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice([BF16, BF16, BF16, FP32])
    store = rng.choice([dtype, E4M3])
    if kind in ("write", "read"):
        seqs = log_int(rng, 1, 24)
        new = log_int(rng, 1, max(1, 6000 // seqs))
        return cache_case(kind, seqs, new, new + log_int(rng, 1, max(1, 20000 // seqs)), heads[1], page=page, dtype=dtype,
                          store=store, lens=lens)
    if dtype == FP32:  # (the fp32 form is there for parity: modest sizes)
        seqs, new = log_int(rng, 1, 8), log_int(rng, 1, 64)
        return attend_case(seqs, new, new + log_int(rng, 1, 1500), *heads, page=page, dtype=FP32, store=store,
                           block=rng.choice([1, 1, 40]), window=rng.choice([0, 9]), sinks=rng.choice([0, 2]), lens=lens)
    form = rng.choice(["token", "chunk", "frame"])
    if form == "frame":
        block = rng.choice([390, 880, 1560])
        hist = rng.randrange(0, 16)
        return attend_case(1 + rng.randrange(2), block, block * (1 + hist), *rng.choice([(12, 12), (6, 6), (8, 2)]), page=page,
                           store=store, block=block, window=rng.choice([0, 5]), sinks=rng.choice([0, 1]), ragged=False,
                           lens=lens)
    seqs = log_int(rng, 1, 48) if form == "token" else log_int(rng, 1, 6)
    new = rng.choice([1, 1, 1, 2, 5]) if form == "token" else log_int(rng, 10, 1500)
    context = new + log_int(rng, 1, 12000 if form == "token" else 4000)
    window = rng.choice([0, 0, 257, 2048])
    return attend_case(seqs, new, context, *heads, page=page, store=store, window=window,
                       sinks=rng.choice([0, 4, 130]) if window else 0, lens=lens)


def lengths(case):
    """(new, total) tokens of each sequence: whole for frames, else spread up
    to the case's sizes, the first sequence at its full size."""
    r = random.Random(case["lens"])
    new, total = [], []
    for s in range(case["seqs"]):
        n, t = case["new"], case["context"]
        if s and case.get("ragged", True):
            n = r.randint(max(1, n // 3), n)
            t = max(n, r.randint(max(1, t // 5), t))
        elif s:  # frames: another number of whole ones
            t = n * r.randint(max(1, t // n // 2), t // n)
        new.append(n)
        total.append(t)
    return new, total


def axes_of(case):
    return [int(a) for a in case["axes"].split(",")]


# ---- inputs ----------------------------------------------------------------

def quantise(x):
    """x [..., d] fp32 -> e4m3 codes and one fp32 scale per row; a row that is
    not finite has the scale NaN and codes 0."""
    amax = x.abs().amax(-1)
    scale = (amax / CODE_MAX).clamp(min=SCALE_MIN)
    fine = torch.isfinite(amax)
    codes = torch.where(fine[..., None], (x * (1.0 / scale)[..., None]).clamp(-CODE_MAX, CODE_MAX), torch.zeros_like(x))
    return codes.to(torch.float8_e4m3fn), torch.where(fine, scale, torch.full_like(scale, float("nan")))


def pool_for(case, total, gen):
    """Pages of the sequences in a random order, with values in them as they
    come out of a layer (N(0, 1), some key channels larger)."""
    page, hk, d = case["page"], case["kv_heads"], case["d"]
    counts = [(t + page - 1) // page for t in total]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    width = max(counts)
    table = torch.zeros(len(total), width, dtype=torch.int32, device="cuda")
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = order[at:at + c]
        at += c
    pool = {}
    channel = torch.exp(0.5 * torch.randn(hk, 1, d, generator=gen, device="cuda"))
    for name, gain in (("k", channel), ("v", 1.0)):
        x = torch.randn(pages, hk, page, d, generator=gen, device="cuda") * gain
        if case["store"] == E4M3:
            pool[name], pool[name + "_scale"] = quantise(x)
        else:
            pool[name], pool[name + "_scale"] = x.to(DTYPES[case["store"]]), None
    return pool, table


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = {"case": case}

    def tokens(n, heads):
        return torch.randn(n, heads, case["d"], generator=gen, device="cuda").to(DTYPES[case["dtype"]])

    if case["kind"] == "rotary":
        n, axes = case["tokens"], axes_of(case)
        state["q"], state["k"] = tokens(n, case["q_heads"]), tokens(n, case["kv_heads"])
        i = torch.arange(n, device="cuda")
        first = case["far"] + int(seed) % 97
        grid = [first + i // 1560, i % 1560 // 52, i % 52] if len(axes) > 1 else [first + i]
        state["positions"] = torch.stack(grid[:len(axes)], 1).to(torch.int32).contiguous()
        if own:
            from hybrid_softmax_gated_b200 import RotaryAxes
            state["rotary"] = RotaryAxes(case["d"], axes, base=case["base"], pairs=case["pairs"], freqs=case["freqs"])
        return state
    new, total = lengths(case)
    pool, table = pool_for(case, total, gen)
    state.update(pool=pool, table=table, new=new, total=total, q_offsets=ints(offsets(new)), kv_lens=ints(total),
                 kv_offsets=ints(offsets(total)), max_new=max(new), max_total=max(total))
    if case["kind"] == "write":
        state["k"], state["v"] = tokens(sum(new), case["kv_heads"]), tokens(sum(new), case["kv_heads"])
    if case["kind"] == "attend":
        state["q"] = tokens(sum(new), case["q_heads"])
    if own:
        from hybrid_softmax_gated_b200 import PagedBatch, PagedCache
        state["cache"] = PagedCache(case.get("q_heads", case["kv_heads"]), case["kv_heads"], case["d"], pool["k"].shape[0],
                                    case["page"], dtype=DTYPES[case["dtype"]],
                                    cache_format="e4m3" if case["store"] == E4M3 else "native",
                                    pool=(pool["k"][None], pool["v"][None],
                                          None if pool["k_scale"] is None else pool["k_scale"][None],
                                          None if pool["v_scale"] is None else pool["v_scale"][None]))
        state["batch"] = PagedBatch(state["q_offsets"], state["kv_lens"], table, max_new=state["max_new"])
    return state


# ---- plain forms -----------------------------------------------------------

def plain_rotary(state):
    case = state["case"]
    axes, rot = axes_of(case), sum(axes_of(case))
    per = [torch.arange(a // 2, device="cuda", dtype=torch.float64) / (a // 2) for a in axes]
    if case["freqs"] == "shared":
        part = torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2)
    else:
        part = torch.cat(per)
    freq = torch.exp(-math.log(case["base"]) * part)
    axis = torch.repeat_interleave(torch.arange(len(axes), device="cuda"),
                                   torch.tensor([a // 2 for a in axes], device="cuda"), output_size=rot // 2)
    angle = state["positions"].double()[:, axis] * freq  # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    if case["inverse"]:
        sin = -sin

    def turn(x):
        y = x.float()
        if case["pairs"] == "adjacent":
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([z, y[..., rot:]], -1).to(x.dtype)

    return turn(state["q"]), turn(state["k"])


def spots(state, of, at):
    """Page and slot of the positions `at` of the sequences `of`."""
    page = state["case"]["page"]
    return state["table"][of, at // page].long(), at % page


def owners(first, n):
    """Sequence of each of n rows, from the rows' offsets."""
    return torch.searchsorted(first[1:].long(), torch.arange(n, device="cuda"), right=True)


def plain_write(state):
    pool, n = state["pool"], state["k"].shape[0]
    of = owners(state["q_offsets"], n)
    at = torch.arange(n, device="cuda") - state["q_offsets"][of] + (state["kv_lens"] - state["q_offsets"].diff())[of]
    where = spots(state, of, at)
    for name in ("k", "v"):
        if pool[name + "_scale"] is not None:
            codes, scale = quantise(state[name].float())
            pool[name].view(torch.uint8)[where[0], :, where[1]] = codes.view(torch.uint8)
            pool[name + "_scale"][where[0], :, where[1]] = scale
        else:
            pool[name][where[0], :, where[1]] = state[name].to(pool[name].dtype)
    return pool


def fetch(state, name, where):
    pool = state["pool"]
    if pool[name + "_scale"] is None:
        return pool[name][where[0], :, where[1]].float()
    return pool[name].view(torch.uint8)[where[0], :, where[1]].view(torch.float8_e4m3fn).float() \
        * pool[name + "_scale"][where[0], :, where[1]][..., None]


def plain_read(state):
    n = sum(state["total"])
    of = owners(state["kv_offsets"], n)
    where = spots(state, of, torch.arange(n, device="cuda") - state["kv_offsets"][of])
    to = DTYPES[state["case"]["dtype"]]
    return fetch(state, "k", where).to(to), fetch(state, "v", where).to(to)


def visible(case, at, total, j):
    """Whether the query at position `at` of `total` sees the key j."""
    c = torch.div(at, case["block"], rounding_mode="floor")
    see = (j < total) & (j < (c + 1) * case["block"]) & (at >= 0)
    if case["window"]:
        see &= (j >= (c + 1 - case["window"]) * case["block"]) | (j < case["sinks"] * case["block"])
    return see


def plain_attend(state):
    case, q = state["case"], state["q"]
    seqs, nq, nk = case["seqs"], state["max_new"], state["max_total"]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["d"]
    n = q.shape[0]
    of = owners(state["q_offsets"], n)
    row = torch.arange(n, device="cuda") - state["q_offsets"][of]
    padded = torch.zeros(seqs, nq, hq, d, device="cuda")
    padded[of, row] = q.float()
    j = torch.arange(nk, device="cuda")
    at = torch.arange(nq, device="cuda")[None, :] + (state["kv_lens"] - state["q_offsets"].diff())[:, None]
    see = visible(case, at[:, :, None], state["kv_lens"][:, None, None], j)[:, None, None]  # [S, 1, 1, nq, nk]
    every = torch.arange(seqs, device="cuda")[:, None].expand(seqs, nk), j[None, :].expand(seqs, nk)
    where = spots(state, *every)  # (the table's padding points at some page: never visible)
    inside = (j[None, :] < state["kv_lens"][:, None])[..., None, None]
    k = torch.where(inside, fetch(state, "k", where), 0.0).permute(0, 2, 3, 1)  # [S, hk, d, nk]
    s = padded.view(seqs, nq, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(seqs, hk, -1, d) @ k
    s = (s.view(seqs, hk, hq // hk, nq, nk) / math.sqrt(d)).masked_fill_(~see, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > float("-inf"), top, 0.0))
    del s
    total = p.sum(-1, keepdim=True)
    v = torch.where(inside, fetch(state, "v", where), 0.0).permute(0, 2, 1, 3)
    o = (p.view(seqs, hk, -1, nk) @ v).view(seqs, hk, hq // hk, nq, d) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, nq, hq, d)[of, row].to(q.dtype)


# ---- one pass --------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        if case["kind"] == "rotary":
            return state["rotary"].apply(state["q"], state["k"], state["positions"], inverse=case["inverse"])
        if case["kind"] == "write":
            state["cache"].write(state["k"], state["v"], state["batch"])
            return state["pool"]
        if case["kind"] == "read":
            return state["cache"].read(state["table"], state["kv_offsets"], sum(state["total"]))
        return state["cache"].attend(state["q"], state["batch"], block=case["block"], window=case["window"],
                                     sinks=case["sinks"])
    return {"rotary": plain_rotary, "write": plain_write, "read": plain_read, "attend": plain_attend}[case["kind"]](state)


# ---- what a pass cannot do without ------------------------------------------

def seen_by(case, at, total):
    """(first, last + 1) runs of keys that the query at `at` sees."""
    if at < 0:
        return []
    end = min(total, (at // case["block"] + 1) * case["block"])
    if not case["window"]:
        return [(0, end)]
    low = max(0, (at // case["block"] + 1 - case["window"]) * case["block"])
    sink = min(case["sinks"] * case["block"], end)
    return [(0, end)] if sink >= low else [(0, sink), (low, end)]


def work(case):
    size = {BF16: 2, FP32: 4}[case["dtype"]]
    d = case["d"]
    if case["kind"] == "rotary":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        rot = sum(axes_of(case))
        return {"bytes": 2 * n * d * size + 4 * case["tokens"] * len(axes_of(case)), "flops": 3 * n * rot}
    new, total = lengths(case)
    stored = d + 4 if case["store"] == E4M3 else d * size
    if case["kind"] == "write":
        n = 2 * sum(new) * case["kv_heads"]
        return {"bytes": n * (d * size + stored), "flops": 2 * n * d}
    if case["kind"] == "read":
        n = 2 * sum(total) * case["kv_heads"]
        return {"bytes": n * (d * size + stored), "flops": n * d}
    pairs = keys = 0
    for n, t in zip(new, total):
        runs = [seen_by(case, t - n + i, t) for i in range(n)]
        pairs += sum(b - a for r in runs for a, b in r)
        if any(runs):  # keys that some query of the chunk sees
            low = min(r[-1][0] for r in runs if r)
            high = max(r[-1][1] for r in runs if r)
            keys += high - low + min(low, max(r[0][1] for r in runs if r) if any(len(r) > 1 for r in runs) else 0)
    return {"bytes": 2 * sum(new) * case["q_heads"] * d * size + 2 * keys * case["kv_heads"] * stored,
            "flops": 4 * d * case["q_heads"] * pairs}


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    """What run() returns, in 64 bits: one sequence and one key head at a
    time, straight from the definitions."""
    state = prepare(case, seed)
    d = case["d"]
    if case["kind"] == "rotary":
        axes = axes_of(case)
        rot = sum(axes)
        freq, axis = [], []
        for a, width in enumerate(axes):
            for i in range(width // 2):
                freq.append(case["base"] ** (-(len(axis) / (rot // 2) if case["freqs"] == "shared" else i / (width // 2))))
                axis.append(a)
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                           (-1.0 if case["inverse"] else 1.0) * state["positions"].double()[:, axis]
                           * torch.tensor(freq, dtype=torch.float64, device="cuda"))[:, None, :]
        outs = []
        for x in (state["q"].double(), state["k"].double()):
            pair = (x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["pairs"] == "adjacent"
                    else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            z = z if case["pairs"] == "adjacent" else z.transpose(-1, -2)
            outs.append(torch.cat([z.flatten(-2), x[..., rot:]], -1))
        return tuple(outs)
    pool, page = state["pool"], case["page"]
    if case["kind"] == "write":
        coded = case["store"] == E4M3  # (codes are a rounding, not a number computed: their scales are)
        want = {n: (None if x is None or coded != n.endswith("scale") else x.double()) for n, x in pool.items()}
        for s, (n, t) in enumerate(zip(state["new"], state["total"])):
            at = torch.arange(t - n, t, device="cuda")
            rows = slice(int(state["q_offsets"][s]), int(state["q_offsets"][s]) + n)
            for name in ("k", "v"):
                x = state[name][rows].double()
                if coded:
                    name, x = name + "_scale", x.abs().amax(-1) / CODE_MAX
                want[name][state["table"][s, at // page].long(), :, at % page] = x
        return want

    def rows(name, s, keys, h):
        p, slot = state["table"][s, keys // page].long(), keys % page
        x = pool[name][:, h].view(torch.uint8) if case["store"] == E4M3 else pool[name][:, h]
        x = x[p, slot]
        if case["store"] == E4M3:
            return x.view(torch.float8_e4m3fn).double() * pool[name + "_scale"][p, h, slot].double()[:, None]
        return x.double()

    if case["kind"] == "read":
        got = []
        for name in ("k", "v"):
            got.append(torch.cat([torch.stack([rows(name, s, torch.arange(t, device="cuda"), h)
                                               for h in range(case["kv_heads"])], 1) for s, t in enumerate(state["total"])]))
        return tuple(got)
    if work(case)["flops"] > 4e11:
        return None
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    for s, (n, t) in enumerate(zip(state["new"], state["total"])):
        first = int(state["q_offsets"][s])
        at = torch.arange(t - n, t, device="cuda")
        last = at // case["block"] * case["block"] + case["block"]
        keys = torch.arange(t, device="cuda")
        hidden = keys[None, :] >= last[:, None]
        if case["window"]:
            hidden |= (keys[None, :] < last[:, None] - case["window"] * case["block"]) \
                & (keys[None, :] >= case["sinks"] * case["block"])
        for h in range(case["kv_heads"]):
            k, v = rows("k", s, keys, h), rows("v", s, keys, h)
            for g in range(h * group, (h + 1) * group):
                w = torch.softmax((state["q"][first:first + n, g].double() @ k.T * d ** -0.5)
                                  .masked_fill(hidden, -math.inf), -1)
                out[first:first + n, g] = w @ v
    return out
