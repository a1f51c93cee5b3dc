"""The paged-cache operators in 64 bits, straight from their definitions, and
seeded cases for them.  Test infrastructure: shares no code with the library.

Tolerances count roundings: one rounding to bf16 is off by at most 2^-8 of
the value (half a step), one to fp32 by 2^-24.
"""
import math

import numpy as np
import torch

E4M3_MAX = 448.0
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rotary(x, positions, axis_dims, base, pairs, freqs, inverse=False):
    """x [n, h, d], positions [n, axes] -> float64 [n, h, d]."""
    x = x.double().cpu().numpy()
    pos = positions.double().cpu().numpy()
    rot = sum(axis_dims)
    out = x.copy()
    p = 0
    for a, width in enumerate(axis_dims):
        for i in range(width // 2):
            f = base ** (-(2.0 * p / rot if freqs == "shared" else 2.0 * i / width))
            ang = pos[:, a] * f * (-1.0 if inverse else 1.0)
            c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
            j, k = (2 * p, 2 * p + 1) if pairs == "adjacent" else (p, p + rot // 2)
            out[..., j] = x[..., j] * c - x[..., k] * s
            out[..., k] = x[..., j] * s + x[..., k] * c
            p += 1
    return out


def quantise(x):
    """fp32 rows [..., d] -> (codes float8_e4m3fn, scale fp32), the
    definition's fp32 steps."""
    x = x.float().cpu()
    amax = x.abs().amax(-1)
    scale = torch.clamp(amax / E4M3_MAX, min=2.0 ** -126)
    ok = torch.isfinite(amax)
    y = (x * (1.0 / scale)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes = torch.where(ok[..., None], y, torch.zeros_like(y)).to(torch.float8_e4m3fn)
    return codes, torch.where(ok, scale, torch.full_like(scale, math.nan))


def bounds(at, total, block, window, sinks):
    """Boolean [total]: the keys that the query at position `at` sees."""
    j = np.arange(total)
    if at < 0:
        return np.zeros(total, bool)
    c = at // block
    see = j < min(total, (c + 1) * block)
    if window:
        see &= (j >= (c + 1 - window) * block) | (j < sinks * block)
    return see


def attend(q, k, v, new, total, block, window, sinks, scale):
    """One sequence: q [new, hq, d], k, v [total, hk, d] (float64) ->
    (out, absolute, slack): absolute = sum p |v|, and slack bounds the
    relative error that fp32 sums of d products bring into the weights."""
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    g = hq // hk
    out = np.zeros((new, hq, d))
    absolute = np.zeros((new, hq, d))
    slack = np.zeros((new, hq, 1))
    for i in range(new):
        see = bounds(total - new + i, total, block, window, sinks)
        if not see.any():
            continue
        for h in range(hq):
            ks, vs = k[see, h // g], v[see, h // g]
            s = ks @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vs
            absolute[i, h] = p @ np.abs(vs)
            slack[i, h] = (np.abs(ks) @ np.abs(q[i, h])).max() * scale * (d + 8) * 2.0 ** -24
    return out, absolute, slack


class Case:
    """Pages, tables and chunks of a batch, on the CPU; .cuda() pieces are made
    by the tests."""

    def __init__(self, lens, hq, hk, d=128, page=16, dtype=torch.bfloat16, store="native", seed=0, extra_rows=0,
                 spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hk, self.d, self.page = lens, hq, hk, d, page
        self.dtype, self.store = dtype, store
        counts = [max(0, -(-t // page)) for _, t in lens]
        self.pages = sum(counts) + 2
        width = max(counts + [1]) + 1
        order = torch.randperm(self.pages, generator=g)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)  # (unused entries: never read)
        at = 0
        for s, c in enumerate(counts):
            self.table[s, :c] = order[at:at + c].to(torch.int32)
            at += c
        offs = [0]
        for n, _ in lens:
            offs.append(offs[-1] + n)
        self.tokens = offs[-1] + extra_rows
        self.q_offsets = torch.tensor(offs, dtype=torch.int32)
        self.kv_lens = torch.tensor([t for _, t in lens], dtype=torch.int32)
        self.q = (spread * torch.randn(self.tokens, hq, d, generator=g)).to(dtype)
        self.k = torch.randn(self.tokens, hk, d, generator=g).to(dtype)
        self.v = torch.randn(self.tokens, hk, d, generator=g).to(dtype)
        shape = (self.pages, hk, page, d)
        pools = []
        for _ in range(2):
            x = torch.randn(shape, generator=g)
            pools.append(quantise(x) if store == "e4m3" else (x.to(dtype), None))
        (self.kp, self.ks), (self.vp, self.vs) = pools

    def values(self, name):
        """The pool's values in float64 [pages, hk, page, d]."""
        x, s = (self.kp, self.ks) if name == "k" else (self.vp, self.vs)
        x = x.float().double()
        return x if s is None else x * s.double()[..., None]

    def sequence(self, name, s):
        """[total, hk, d] float64 of sequence s."""
        t = self.lens[s][1]
        x = self.values(name)
        rows = [x[int(self.table[s, j // self.page]), :, j % self.page] for j in range(t)]
        return (torch.stack(rows) if rows else torch.zeros(0, self.hk, self.d, dtype=torch.float64)).numpy()

    def expect(self, block=1, window=0, sinks=0, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        out = np.zeros((self.tokens, self.hq, self.d))
        absolute, slack = np.zeros_like(out), np.zeros((self.tokens, self.hq, 1))
        for s, (n, t) in enumerate(self.lens):
            if n == 0:
                continue
            a = int(self.q_offsets[s])
            q = self.q[a:a + n].double().numpy()
            out[a:a + n], absolute[a:a + n], slack[a:a + n] = attend(
                q, self.sequence("k", s), self.sequence("v", s), n, t, block, window, sinks, scale)
        return out, absolute, slack

    def tolerance(self, out, absolute, slack, impl):
        """Bound of |kernel - out|: the output's rounding; the weights'
        rounding to bf16 (tensor-core kernels: once per weight, and the sum of
        the weights is of unrounded ones); the scores' fp32 sums, which move a
        weight and the sum of all by `slack` each, and 16 fp32 roundings for
        the exponential, the scales, the rescaling and the sums' own steps
        (sums of n terms: pairwise and per block, well below n / 16 more)."""
        n = max([t for _, t in self.lens] + [1])
        steps = 16 + n / 16
        tol = HALF_STEP[self.dtype] * np.abs(out) + absolute * (2 * slack + steps * 2.0 ** -24)
        if self.dtype == torch.bfloat16 and impl == "auto":
            tol = tol + 2.0 ** -8 * absolute
        return tol * 1.01 + 1e-30
