"""CPU oracle of the compressed cache's operators, written from their definitions:
rotary positions (fp64), append into 8-bit pages, attention over them (fp64), and
the bookkeeping of pages (Python integers), with the bounds the GPU tests use.
"""
from __future__ import annotations

import math

import torch

from . import target_ops_oracle as T

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_freqs(rot, theta, scaling=None):
    """Radians a position of each pair, and the factor on cos and sin."""
    p = dict(scaling or {})
    kind, amplitude = p.get("kind"), 1.0
    if kind == "ntk":
        theta = theta * p["factor"] ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if kind == "linear":
            f /= p["factor"]
        elif kind == "bands":
            u = p["original_len"] * f / (2 * math.pi)
            s = min(1.0, max(0.0, (u - p["low"]) / (p["high"] - p["low"])))
            f *= (1 - s) / p["factor"] + s
        elif kind == "yarn":
            at = lambda u: rot * math.log(p["original_len"] / (2 * math.pi * u)) / (2 * math.log(theta))
            lo, hi = max(math.floor(at(p["high"])), 0), min(math.ceil(at(p["low"])), rot - 1)
            s = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / p["factor"] * s + f * (1 - s)
            amplitude = 0.1 * math.log(p["factor"]) + 1
        out.append(f)
    return torch.tensor(out, dtype=torch.float64), amplitude


def rope(x, pos, freqs, amplitude, layout, offset, transpose):
    """x [rows, heads, d], pos [rows]: the turned rows (fp64) and what a fp32 kernel may be off by, before the
    rounding to x's type.

    The angle in fp32 half turns is off by pi 2^-24 (its conversion), its cos and sin by 2^-22 more (two units in
    the last place of values up to 1), the frequency by 2^-50 relative (a power and a few products in fp64);
    amplitude and the three operations of an output by 4 2^-24 of the two products."""
    h = len(freqs)
    angle = pos.double()[:, None] * freqs[None, :]
    c, s = (torch.cos(angle) * amplitude)[:, None], (torch.sin(angle) * amplitude * (-1 if transpose else 1))[:, None]
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    first = slice(offset, offset + h) if layout == "half" else slice(offset, offset + 2 * h, 2)
    second = slice(offset + h, offset + 2 * h) if layout == "half" else slice(offset + 1, offset + 2 * h, 2)
    a, b = x[..., first].double(), x[..., second].double()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    unit = math.pi * 2.0 ** -24 + 2.0 ** -22 + angle[:, None] * 2.0 ** -50 + 4 * 2.0 ** -24
    tol[..., first] = tol[..., second] = (a.abs() + b.abs()) * amplitude * unit
    return y, tol


# ---------------------------------------------------------------------------
# append into 8-bit pages
# ---------------------------------------------------------------------------
def needed_scale(most: float) -> float:
    """The smallest power of two s in 2^-60 .. 2^60 with most <= 448 s (2^60 where none has)."""
    e = -60
    while e < 60 and most > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def encode(x):
    """Codes (uint8) of fp32 values: to nearest even, saturating; not finite: 0x7f."""
    c = x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
    return torch.where(torch.isfinite(x), c, torch.tensor(0x7F, dtype=torch.uint8))


def decode(codes, scale):
    """Values (fp64) of codes [n_pages, page, heads, d] with scales [n_pages, heads]."""
    return codes.view(E4M3).double() * scale.double()[:, None, :, None]


def append8(codes, scale, x, starts, lens, table):
    """codes uint8 [n_pages, page, heads, d], scale fp32 [n_pages, heads]: both with the rows of x."""
    codes, scale = codes.clone(), scale.clone()
    page = codes.shape[1]
    for b, L in enumerate(lens):
        p = L - (starts[b + 1] - starts[b])
        row = starts[b]
        while p < L:
            pg, s0 = int(table[b, p // page]), p % page
            m = min(page - s0, L - p)
            new = x[row:row + m].float()
            for h in range(codes.shape[2]):
                v = new[:, h]
                fin = v[torch.isfinite(v)].abs()
                s = torch.tensor(needed_scale(float(fin.max()) if len(fin) else 0.0))
                if s0:
                    old = scale[pg, h]
                    if not s > old:
                        s = old
                    if float(s) != float(old):
                        again = codes[pg, :s0, h].view(E4M3).float() * (old / s)
                        codes[pg, :s0, h] = encode(again)
                codes[pg, s0:s0 + m, h] = encode(torch.where(torch.isfinite(v), v / s, v))
                scale[pg, h] = s
            p, row = p + m, row + m
    return codes, scale


def gather8(codes, scale, lens, table):
    return T.gather(decode(codes, scale), lens, table)


def largest_share(q, k, v, L, causal, window, scale):
    """[n, hq]: the largest probability times value (its size) of the keys that a row sees."""
    n, hq, _ = q.shape
    out = torch.zeros((n, hq), dtype=torch.float64)
    if not n:
        return out
    g = hq // k.shape[1]
    rel = torch.arange(L - n, L)[:, None] - torch.arange(L)[None, :]
    see = (rel >= 0 if causal else torch.ones_like(rel, dtype=torch.bool)) & (rel < window if window else True)
    for h in range(hq):
        s = torch.where(see, (q[:, h].double() @ k[:, h // g].double().t()) * scale, -math.inf)
        out[:, h] = torch.nan_to_num(torch.softmax(s, 1) * v[:, h // g].amax(-1), nan=0.0).amax(1)
    return out


def attention8(q, seq_k, seq_v, starts, lens, causal, window, scale, bf16, tensor_cores, q_pieces=False):
    """As T.attention over the decoded values, with the bounds of these kernels.

    fp32 arithmetic is T's, with the two scales' products (2 2^-24 of a score and of a value, within its d + 4 and
    its sums' slack).  The output is rounded once.  On the tensor cores a probability times its key's scale of V is
    rounded to fp16: 2^-11 relative, and half a step of 2^-24 below the smallest normal number.  The row's unit is such
    that the largest such product of the keys that the row sees is 2^7 or more, so that half step is at most 2^-32 of
    it, for each key, times a code of up to 448.  (A key's largest code is at least 1 here: its largest value stands for
    its scale.)  q_pieces: q is the sum of two e4m3
    pieces, scaled so that its largest element is 2^7 or more; the second piece is off by at most half its step
    of 2^-9, that is 2^-17 of the largest, where an element is below 2^-9 of that (larger ones are exact): twice
    that error of a score for a weight, once for the log-sum-exp."""
    o, lse, tol, tol_lse = T.attention(q, seq_k, seq_v, starts, lens, causal, window, scale, False)
    for b, L in enumerate(lens):
        s, e = starts[b], starts[b + 1]
        if tensor_cores:
            fin = lambda x: torch.where(torch.isfinite(x), x, 0.0).abs()
            av = T.attention(q[s:e], [seq_k[b]], [fin(seq_v[b])], [0, e - s], [L], causal, window, scale, False)[0]
            most = largest_share(q[s:e], seq_k[b], fin(seq_v[b]), L, causal, window, scale)
            tol[s:e] += av * 2.0 ** -10 + L * 2.0 ** -32 * 448 * most[..., None]
            if q_pieces and L:
                x = fin(q[s:e].double())
                top = x.amax(-1, keepdim=True)
                off = torch.where(x < top * 2.0 ** -9, top * 2.0 ** -17, 0.0)                  # [n, hq, d]
                g = q.shape[1] // seq_k[b].shape[1]
                ds = torch.stack([(off[:, h] @ fin(seq_k[b][:, h // g]).t()).amax(-1) for h in range(q.shape[1])], 1) * scale
                tol[s:e] += av * 2 * ds[..., None]
                tol_lse[s:e] += ds
    if bf16:
        tol = tol + o.abs() * 2.0 ** -8
    return o, lse, tol, tol_lse


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def n_pages_of(length, page):
    return -(-length // page)


def reorder(refs, table, lens, parents, page, width):
    refs, rows, out = list(refs), [], []
    for t, n in zip(table, lens):
        for p in t[:n_pages_of(n, page)]:
            refs[p] -= 1
    for parent in parents:
        n = lens[parent] if parent >= 0 else 0
        held = list(table[parent][:n_pages_of(n, page)]) if parent >= 0 else []
        for p in held:
            refs[p] += 1
        rows.append(held + [-1] * (width - len(held)))
        out.append(n)
    return refs, rows, out


def resize(refs, table, lens, new_lens, page):
    """refs, table, lens afterwards, the copies (src, dst) and which rows were refused."""
    refs, table, lens = list(refs), [list(t) for t in table], list(lens)
    for i, (n, m) in enumerate(zip(lens, new_lens)):
        for j in range(n_pages_of(m, page), n_pages_of(n, page)):
            refs[table[i][j]] -= 1
            table[i][j] = -1
    writers, begun, asks = {}, {}, []
    for i, (n, m) in enumerate(zip(lens, new_lens)):
        if m > n and n % page:
            begun[i] = table[i][n_pages_of(n, page) - 1]
            writers.setdefault(begun[i], []).append(i)
    free = [p for p, c in enumerate(refs) if c <= 0]
    taken, copies, refused, before = 0, [], set(), list(refs)
    for i, (n, m) in enumerate(zip(lens, new_lens)):
        p = begun.get(i)
        copy = p is not None and before[p] > 1 and not (before[p] == len(writers[p]) and writers[p][0] == i)
        ask = max(n_pages_of(m, page) - n_pages_of(n, page), 0) + copy
        asks.append((taken, copy))
        taken += ask
        if ask and taken > len(free):          # nor does any row behind it that asks for pages
            refused.add(i)
    # the row that would keep a page writes to it only if all others that hold it have their copies
    refused |= {i for i, p in begun.items() if not asks[i][1] and before[p] > 1 and any(w in refused for w in writers[p])}
    for i, (n, m) in enumerate(zip(lens, new_lens)):
        if i in refused:
            continue
        at, copy = asks[i]
        if copy:
            copies.append((begun[i], free[at]))
            refs[begun[i]] -= 1
            refs[free[at]] = 1
            table[i][n_pages_of(n, page) - 1] = free[at]
            at += 1
        for j in range(n_pages_of(n, page), n_pages_of(m, page)):
            table[i][j] = free[at]
            refs[free[at]] = 1
            at += 1
        lens[i] = m
    return refs, table, lens, copies, sorted(refused)


def compact(refs, table, lens, page):
    used = sum(c > 0 for c in refs)
    src = [p for p, c in enumerate(refs) if c > 0 and p >= used]
    dst = [p for p, c in enumerate(refs) if c <= 0 and p < used]
    to = dict(zip(src, dst))
    new = [max(c, 0) for c in refs]
    for a, b in to.items():
        new[b], new[a] = refs[a], 0
    rows = [[to.get(p, p) if j < n_pages_of(n, page) else -1 for j, p in enumerate(t)] for t, n in zip(table, lens)]
    return new, rows, used, list(zip(src, dst))
