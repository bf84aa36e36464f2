"""CPU oracle (torch fp64) of the target-side operators: append to pages,
attention of new rows over paged or packed K/V, and token log probabilities,
written from their definitions, with the error bounds the GPU tests use.

Rounding unit of a type: half a step relative to the value (bf16 2^-8 as
eps / 2, fp32 2^-24).  What an fp32 kernel may differ by, for one row:
  score    s = scale q . k:      |ds| <= (d + 4) 2^-24 scale sum |q_c k_c|
  weight   p = e^(s - m) / l:    relative 2 |ds| + 2^-20 (exp2, its argument's
           rounding for |s - m| <= 100 comes in as |s - m| 2^-22) + L 2^-23
  output   o = sum p v:          |do| <= sum p |v| (weight error + L 2^-23)
A bf16 call rounds p once (u = 2^-8 relative) and o once.
"""
from __future__ import annotations

import math

import torch


def attention_row_block(q, k, v, pos, length, causal, window, scale, bf16):
    """q [n, d], k, v [length, d] (fp64), pos [n]: outputs, lse and bounds of both."""
    n, d = q.shape
    s = (q @ k.t()) * scale
    j = torch.arange(length)
    see = torch.ones((n, length), dtype=torch.bool)
    if causal:
        see &= j[None, :] <= pos[:, None]
    if window:
        see &= pos[:, None] - j[None, :] < window
    s = torch.where(see, s, -math.inf)
    empty = ~see.any(1)
    m = torch.where(empty, 0.0, s.amax(1) if length else torch.zeros(n, dtype=torch.float64))
    e = torch.where(see, torch.exp(s - m[:, None]), 0.0)
    l = e.sum(1)
    p = e / torch.where(empty, 1.0, l)[:, None]
    vz = v
    o = torch.zeros((n, v.shape[1]), dtype=torch.float64)
    av = torch.zeros_like(o)
    for i in range(n):   # hidden keys never enter, whatever their bits
        if not empty[i]:
            o[i] = p[i, see[i]] @ vz[see[i]]
            av[i] = p[i, see[i]] @ vz[see[i]].abs()
    lse = torch.where(empty, -math.inf, m + torch.log(l))
    ds = torch.where(see, (q.abs() @ k.abs().t()) * scale, 0.0)
    spread = torch.where(see, (m[:, None] - s), 0.0).clamp(max=100.0)
    ds_max = ((d + 4) * 2.0 ** -24 * ds).amax(1) if length else torch.zeros(n, dtype=torch.float64)
    w = 2 * ds_max + 2.0 ** -20 + spread.amax(1) * 2.0 ** -22 + length * 2.0 ** -23 if length else ds_max
    u = 2.0 ** -8 if bf16 else 2.0 ** -24
    tol = av * ((w + length * 2.0 ** -23)[:, None] + (2.0 ** -8 if bf16 else 0.0)) + o.abs() * u + 1e-30
    tol_lse = w + 2.0 ** -22 * torch.where(empty, 0.0, lse).abs()
    return o, lse, tol, tol_lse


def attention(q, seq_k, seq_v, starts, lens, causal, window, scale, bf16):
    """q [rows, hq, d]; seq_k[b], seq_v[b] [len_b, hkv, d].  Rows of no sequence stay NaN."""
    rows, hq, d = q.shape
    o = torch.full((rows, hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((rows, hq), math.nan, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    for b, L in enumerate(lens):
        s, e = starts[b], starts[b + 1]
        g = hq // seq_k[b].shape[1]
        pos = torch.arange(L - (e - s), L)
        for h in range(hq):
            r = attention_row_block(q[s:e, h].double(), seq_k[b][:, h // g].double(), seq_v[b][:, h // g].double(),
                                    pos, L, causal, window, scale, bf16)
            o[s:e, h], lse[s:e, h], tol[s:e, h], tol_lse[s:e, h] = r
    return o, lse, tol, tol_lse


def append(k_pages, k, starts, lens, table):
    """k_pages [n_pages, page, hkv, d] with the rows of k in their slots (a copy)."""
    out = k_pages.clone()
    page = out.shape[1]
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            pos = L - n + i
            out[int(table[b, pos // page]), pos % page] = k[starts[b] + i]
    return out


def gather(k_pages, lens, table):
    page = k_pages.shape[1]
    out = []
    for b, L in enumerate(lens):
        p = torch.arange(L)
        out.append(k_pages[table[b].long()[p // page], p % page])
    return out


def logprobs(logits, tokens, top, temperature):
    """logits [rows, V]: logprob, entropy, top ids, top logprobs and the bounds of the first two and the last.

    fp32 errors: z = l / T off by 2^-23 |z|, d = z - m by 2^-22 (|z| + |m|), e^d relative by that and 2^-20,
    sums of V terms by at most (V / 256 + 64) 2^-24 (a thread's own terms one after another, then trees)."""
    x = logits.double()
    z = x / temperature
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    lse = m + torch.log(s)
    logp = z - lse
    p = e / s
    ent = torch.where(p > 0, -p * logp, 0.0).sum(1)
    rows = torch.arange(x.shape[0])
    t = tokens.long()
    lp = torch.where(t < 0, 0.0, logp[rows, t.clamp(min=0)])
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    tlp = torch.gather(logp, 1, ids)
    sums = (x.shape[1] / 256 + 64) * 2.0 ** -24
    fin = torch.where(torch.isfinite(d), d, 0.0)
    zf = torch.where(torch.isfinite(z), z, 0.0).abs()
    de = 2.0 ** -22 * (zf + m.abs()) + 2.0 ** -20
    base = (p * de).sum(1) + sums

    def tol_of(zz):
        return base + 2.0 ** -22 * (torch.where(torch.isfinite(zz), zz, 0.0).abs() + m[:, 0].abs() +
                                    torch.log(s[:, 0]).abs() + 1)
    tol_lp = tol_of(z[rows, t.clamp(min=0)])
    tol_ent = (p * de * (fin.abs() + 1)).sum(1) + (1 + (p * fin.abs()).sum(1)) * (2 * sums + 2.0 ** -21) + base
    tol_top = torch.stack([tol_of(torch.gather(z, 1, ids)[:, i]) for i in range(top)], 1) if top else tlp
    return lp, ent, ids, tlp, tol_lp, tol_ent, tol_top
