"""A plain 64-bit reading of the paged key/value cache and of attention over it
(no code shared with the package), with the error bounds that follow from the
formats.  Half a step of a type is eps / 2 relative to the value: bf16 2^-8,
e4m3 2^-4 (or half of its smallest step, 2^-10, where codes are subnormal).
"""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_BF16 = 2.0 ** -8
E4M3_MAX, AMAX_LO, AMAX_HI = 448.0, 2.0 ** -100, float(torch.finfo(torch.float32).max)


class Cache:
    """A pool of pages on the CPU (use .cuda() for the kernels' copies)."""

    def __init__(self, lens, Hkv, d, page, kind, layout="hnd", seed=0, slack=3, width=None, fill=0.0):
        g = torch.Generator("cpu").manual_seed(seed)
        self.lens, self.Hkv, self.d, self.page, self.kind = list(lens), Hkv, d, page, kind
        per = [-(-n // page) for n in self.lens]
        used = sum(per)
        self.P = P = used + slack
        M = width if width is not None else max(1, *per)
        order = torch.randperm(P, generator=g)[:used].int()
        self.table = torch.full((len(self.lens), M), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.seqlens = torch.tensor(self.lens, dtype=torch.int32)
        shape = (P, page, Hkv, d) if layout == "nhd" else (P, Hkv, page, d)
        dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        self.t = {}
        for n in ("k", "v"):
            x = torch.full(shape, fill, dtype=torch.float32).to(dt)
            self.t[n + "_pages"] = x.transpose(1, 2) if layout == "nhd" else x
            if kind != "bf16":
                s = torch.full(shape[:3], fill)
                self.t[n + "_scale"] = s.transpose(1, 2) if layout == "nhd" else s

    def places(self, b, pos):
        return self.table[b].long()[pos // self.page], pos % self.page

    def put(self, name, b, pos, x):
        """Stores rows x [n, Hkv, d] (bf16) at positions pos, quantised by the definition."""
        pid, slot = self.places(b, pos)
        if self.kind == "bf16":
            self.t[name + "_pages"][pid, :, slot] = x
            return
        code, scale = quantise(x)
        for i in range(len(pos)):
            self.t[name + "_pages"][pid[i], :, slot[i]] = code[i]
            self.t[name + "_scale"][pid[i], :, slot[i]] = scale[i]

    def fill_random(self, seed, spread=1.0):
        g = torch.Generator("cpu").manual_seed(seed)
        for b, n in enumerate(self.lens):
            for name in ("k", "v"):
                x = (torch.randn((n, self.Hkv, self.d), generator=g) * spread).to(torch.bfloat16)
                if n:
                    self.put(name, b, torch.arange(n), x)
        return self

    def rows(self, name, b, pos):
        """fp64 values [len(pos), Hkv, d]."""
        pid, slot = self.places(b, pos)
        pages = self.t[name + "_pages"]
        x = torch.stack([pages[p, :, s].float() for p, s in zip(pid.tolist(), slot.tolist())]) if len(pos) else \
            torch.zeros((0, self.Hkv, self.d))
        x = x.double()
        if self.kind != "bf16" and len(pos):
            x = x * self.t[name + "_scale"][pid, :, slot].double()[..., None]
        return x.numpy()

    def cuda(self):
        """The package's arguments, layouts kept: (k_pages, v_pages, page_table), and the scales' keywords."""
        def move(x):
            out = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
            out.copy_(x)
            return out
        kw = {n: move(self.t[n]) for n in ("k_scale", "v_scale") if n in self.t}
        return (move(self.t["k_pages"]), move(self.t["v_pages"]), self.table.cuda()), kw


def quantise(x):
    """Codes and scales of rows x [..., d]: the definition's fp32 arithmetic."""
    x = x.float()
    a = x.abs().amax(-1).clamp(AMAX_LO, AMAX_HI)
    y = x * (torch.full_like(a, E4M3_MAX) / a)[..., None]  # a true division: number / tensor is not one in torch
    y = torch.where(y.abs() > E4M3_MAX, torch.sign(y) * E4M3_MAX, y)  # infinities and the last half step saturate
    return y.to(torch.float8_e4m3fn), a / E4M3_MAX


def attend(cache, q, causal, window, scale=None):
    """O, LSE and their bounds in fp64 for q [B, H, Nq, d] (a bf16 tensor).

    Bounds.  The weights p enter the second product as bf16 numbers (times the
    value scale when the cache is quantised), so the numerator is off by at most
    HALF_BF16 * A, A = sum_j p_j |v_j|, and where the denominator sums the
    rounded weights it is off by HALF_BF16 as well; the output's own rounding is
    HALF_BF16 * |O|.  Scores: d products of bf16 numbers summed in fp32, each
    partial sum off by at most 2^-23 of the sum of magnitudes, then a factor and
    a base-2 exponential (2 units in the last place of 2^-23 each on an argument
    of size |s|): delta below bounds the error of s, which scales a weight by
    e^delta.  Sums of n fp32 terms add n * 2^-23.
    """
    B, H, Nq, d = q.shape
    g = H // cache.Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    qd = q.double().numpy()
    o = np.zeros((B, H, Nq, d))
    lse = np.full((B, H, Nq), -np.inf)
    tol_o, tol_l = np.zeros_like(o), np.zeros_like(lse)
    cap = cache.table.shape[1] * cache.page
    for b in range(B):
        L = max(0, min(int(cache.seqlens[b]), cap))
        pos = torch.arange(L)
        if L:
            ids = cache.table[b].long()[pos // cache.page]
            pos = pos[(ids >= 0) & (ids < cache.P)]
        K, V = cache.rows("k", b, pos), cache.rows("v", b, pos)
        j = pos.numpy()
        for i in range(Nq):
            p = L - Nq + i
            keep = np.zeros(len(j), bool) if p < 0 else np.ones(len(j), bool)
            if causal:
                keep &= j <= p
            if window >= 0:
                keep &= np.abs(j - p) <= window
            if not keep.any():
                continue
            for h in range(H):
                k, v = K[keep, h // g], V[keep, h // g]
                s = scale * (k @ qd[b, h, i])
                m = s.max()
                w = np.exp(s - m)
                l = w.sum()
                w /= l
                o[b, h, i] = w @ v
                lse[b, h, i] = m + np.log(l)
                n = len(s)
                mag = scale * (np.abs(k) @ np.abs(qd[b, h, i])).max()
                delta = (d + 8) * 2.0 ** -23 * mag + 2.0 ** -21 * (1 + np.abs(s).max())
                A = w @ np.abs(v)
                tol_o[b, h, i] = HALF_BF16 * (A + 2 * np.abs(o[b, h, i])) * 1.02 + (2 * delta + 2 * n * 2.0 ** -23) * A + 1e-30
                tol_l[b, h, i] = delta + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse[b, h, i])
    return o, lse, tol_o, tol_l


def check(name, got, want, tol):
    """Every finite value within its bound, every infinity equal."""
    got = got.detach().float().cpu().double().numpy() if torch.is_tensor(got) else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all(), f"{name}: rows without a key differ"
    assert np.isfinite(got[~inf]).all(), f"{name}: non-finite values at {np.argwhere(~np.isfinite(got) & ~inf)[:5].tolist()}"
    err = np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, want))
    bad = err > np.where(inf, 0.0, tol)
    at = np.unravel_index(np.argmax(np.where(inf, -1.0, err - tol)), err.shape) if err.size else None
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} over the bound; worst at {tuple(int(x) for x in at)}: " \
                          f"got {got[at]:.6g}, want {want[at]:.6g}, bound {tol[at]:.3g}"
