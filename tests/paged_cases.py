"""Shared by the paged-cache tests: building a ragged batch over a paged cache, the plain
attention of it in 64 bits, and error bounds.

Error bounds (u = eps / 2 of the 16-bit type, the relative rounding of one value):

* A rotated value y = m (x0 c -+ x1 s) is computed in fp32 from sines within 4e-7 (the
  angle reduced by whole turns in 64 bits, then rounded to 24 bits of a half turn,
  pi * 2^-25, and two units of the fp32 sine) and rounded once:
  |error| <= u |y| + (|x0| + |x1|) m * 1e-6, and half the smallest fp16 step (2^-25).
* O = sum w v / sum w with weights rounded to 16 bits, each off by a factor within 1 +- u,
  numerator and denominator alike: |error| <= 2 u / (1 - u) * W with W = sum w |v| / sum w,
  and u |O| for the rounding of O. A score is a sum of d products in fp32 with at most one
  step (2^-23: the accumulator may truncate) lost at each, so it is off by at most
  e = A d 2^-23 with A = scale * max_j sum_t |q_t k_jt|, which moves w by a factor within
  1 +- 2 e, O by 4 e W and L by e; sums of up to 2^17 weights in fp32 lanes and their
  logarithm add 2e-6 (1 + |L|).
  Below 2^-14 an fp16 weight is off by up to 2^-25 instead. The key that set a row's last
  reference has weight 1, so sum w >= 1 in every part, and this moves O by at most
  2^-25 (|v| + |O|) per visible key, numerator and denominator.
"""

from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


@dataclass
class Batch:
    lengths: list          # [(new tokens, keys)]
    q: object
    k_pages: object
    v_pages: object
    page_table: object
    cu_q: object
    seq_k: object
    keys: list             # per sequence, [keys, Hkv, d] as they were written
    values: list
    layout: str
    max_q: int

    @property
    def cache(self):
        return self.k_pages, self.v_pages, self.page_table, self.cu_q, self.seq_k


def make_batch(lengths, hq, hkv, d, page, dtype, layout="bnhd", seed=0, behind=0, spare=2,
               fill=float("nan"), gain=1.0, one_pool=False, device="cuda"):
    """A batch whose sequences have `lengths` (new tokens, keys), its keys written into
    shuffled pages; every row of the pool that holds no key is `fill`, and table entries
    behind a sequence's pages point nowhere. `behind` packed rows belong to nobody."""
    import torch
    gen = torch.Generator("cpu").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=gen).to(dtype)
    need = [-(-k // page) for _, k in lengths]
    total, width = sum(need) + spare, max(need + [1]) + 1
    order = torch.randperm(total, generator=gen)
    shape = (total, page, hkv, d) if layout == "bnhd" else (total, hkv, page, d)
    if one_pool:  # K and V as views of one pool
        pool = torch.full((total, 2) + shape[1:], fill, dtype=dtype)
        kp, vp = pool[:, 0], pool[:, 1]
    else:
        kp, vp = (torch.full(shape, fill, dtype=dtype) for _ in range(2))
    table = torch.full((len(lengths), width), -1, dtype=torch.int32)
    table[:, -1] = 2**30
    keys, values, used = [], [], 0
    for b, (_, k) in enumerate(lengths):
        pages = order[used:used + need[b]]
        used += need[b]
        table[b, :need[b]] = pages.int()
        kk, vv = rand(k, hkv, d), rand(k, hkv, d)
        for pool_, rows in ((kp, kk), (vp, vv)):
            view = pool_ if layout == "bnhd" else pool_.transpose(1, 2)
            j = torch.arange(k)
            view[pages[j // page], j % page] = rows
        keys.append(kk)
        values.append(vv)
    n = [n for n, _ in lengths]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
    q = (torch.randn((sum(n) + behind, hq, d), generator=gen) * gain).to(dtype)
    if one_pool:
        pool = pool.to(device)
        kp, vp = pool[:, 0], pool[:, 1]
    return Batch(lengths, q.to(device), kp.to(device), vp.to(device), table.to(device),
                 cu.to(device), torch.tensor([k for _, k in lengths], dtype=torch.int32).to(device),
                 keys, values, layout, max(n + [0]))


def reference(batch, scale, window):
    """Per sequence (O, L, O's bound, L's bound) in 64 bits, [n, Hq, d] and [Hq, n]."""
    import torch
    u = half_step(batch.q.dtype)
    out, at = [], 0
    for b, (n, k) in enumerate(batch.lengths):
        q = batch.q[at:at + n].double()
        at += n
        hq, d = q.shape[1:]
        g = hq // batch.keys[b].shape[1]
        kk = batch.keys[b].to(q.device).double().repeat_interleave(g, 1)
        vv = batch.values[b].to(q.device).double().repeat_interleave(g, 1)
        s = scale * torch.einsum("ihd,jhd->hij", q, kk)
        i = torch.arange(n, device=q.device)[:, None] + k - n
        j = torch.arange(k, device=q.device)
        hidden = torch.zeros((n, k), dtype=torch.bool, device=q.device)
        if window[0] >= 0:
            hidden |= j < i - window[0]
        if window[1] >= 0:
            hidden |= j > i + window[1]
        s = s.masked_fill(hidden, -math.inf)
        L = torch.logsumexp(s, -1) if k else s.new_full(s.shape[:2], -math.inf)
        w = torch.exp(s - L.nan_to_num(neginf=0.0)[..., None])
        o = torch.einsum("hij,jhd->ihd", w, vv)
        W = torch.einsum("hij,jhd->ihd", w, vv.abs())
        a = scale * torch.einsum("ihd,jhd->hij", q.abs(), kk.abs()).amax(-1) if k \
            else torch.zeros_like(L)
        e = a * d * 2.0 ** -23
        bound = (2 * u / (1 - u) + 4 * e.T[..., None]) * W + u * o.abs() + 2.0 ** -25
        if batch.q.dtype == torch.float16:
            seen = (~hidden).double()
            bound = bound + 2.0 ** -25 * (torch.einsum("ij,jhd->ihd", seen, vv.abs())
                                          + seen.sum(-1)[:, None, None] * o.abs())
        out.append((o, L, bound, e + 2e-6 * (1 + L.abs().nan_to_num(posinf=0.0))))
    return out


def check(batch, o, lse, scale, window):
    """O and L against reference(), every value within its bound."""
    import torch
    at = 0
    for b, ((n, _), (ro, rl, bo, bl)) in enumerate(zip(batch.lengths,
                                                       reference(batch, scale, window))):
        go, gl = o[at:at + n].double(), lse[:, at:at + n].double()
        at += n
        if n == 0:
            continue
        empty = torch.isneginf(rl)
        assert torch.equal(torch.isneginf(gl), empty), f"sequence {b}: rows without keys differ"
        assert torch.isfinite(go).all(), f"sequence {b}: O is not finite"
        worst = ((go - ro).abs() / bo).max().item()
        assert worst <= 1, f"sequence {b}: O is off by {worst:.2f} times its bound"
        if (~empty).any():
            worst = ((gl - rl).abs() / bl)[~empty].max().item()
            assert worst <= 1, f"sequence {b}: L is off by {worst:.2f} times its bound"
        assert (go[empty.T] == 0).all(), f"sequence {b}: rows without keys are not 0"
