"""The target-side operators' workloads: their cases, plain forms and work.

Four operators of a target model that serves speculative rounds: the new K/V
rows into a paged cache (append), the attention of a chunk of new tokens over
that cache (paged), the attention of packed prompts (prompt) and the log
probabilities of given tokens with entropy and alternatives (logprobs).

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the library's calls.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    qwen = dict(dtype="bf16", hq=32, hkv=8, d=128)      # the 8B-shaped draft's heads
    laguna = dict(dtype="bf16", hq=24, hkv=8, d=128)    # the windowed draft's heads
    tiny = dict(dtype="f32", hq=4, hkv=4, d=64)         # the small fp32 target's heads
    return [
        # one decode step of a 64-sequence server writes its 64 new rows
        _append("append_decode_64", **qwen, page=16, batch=64, rows_lo=1, rows_hi=1, ctx_lo=1024, ctx_hi=16384),
        # chunks of prompts being read in: thousands of rows, odd lengths
        _append("append_chunks", **qwen, page=64, batch=7, rows_lo=301, rows_hi=2048, ctx_lo=1, ctx_hi=4096),
        # the block of one user's verify step at the headline context
        _paged("verify_one_user", **qwen, page=16, batch=1, rows_lo=16, rows_hi=16, ctx_lo=4096, ctx_hi=4096),
        # a decode step of the serving mix: single tokens, contexts 1k to 16k
        _paged("decode_mix_64", **qwen, page=16, batch=64, rows_lo=1, rows_hi=1, ctx_lo=1024, ctx_hi=16384),
        # verify steps of eight users of a sliding-window model, blocks of up to 8
        _paged("verify_window", **laguna, page=32, batch=8, rows_lo=2, rows_hi=8, ctx_lo=257, ctx_hi=32768,
               window=512),
        # chunked prefill over long caches
        _paged("chunked_prefill", **qwen, page=64, batch=6, rows_lo=129, rows_hi=512, ctx_lo=1000, ctx_hi=16000),
        # the small fp32 target verifying blocks of 8
        _paged("verify_fp32", **tiny, page=16, batch=3, rows_lo=8, rows_hi=8, ctx_lo=300, ctx_hi=1500),
        # a single short prompt: the latency of the smallest call
        _prompt("prompt_short", **qwen, batch=1, rows_lo=37, rows_hi=37),
        # a packed batch of prompts, from one-token to long ones
        _prompt("prompt_packed", **qwen, batch=10, rows_lo=1, rows_hi=8192),
        # prompts of the small fp32 target
        _prompt("prompt_fp32", **tiny, batch=4, rows_lo=99, rows_hi=1200),
        # what the API answers for one verified block: 16 rows, 20 alternatives, a grammar's bans
        _logprobs("logprobs_block", "f32", rows=16, vocab=151936, top=20, temperature=0.7, banned=0.2),
        # scoring a prompt: every token's log probability with 5 alternatives
        _logprobs("logprobs_prompt", "bf16", rows=2047, vocab=151936, top=5, temperature=1.0, banned=0.0),
    ]


def _append(name, dtype, hq, hkv, d, page, batch, rows_lo, rows_hi, ctx_lo, ctx_hi, sizes=11):
    return dict(name=name, kind="append", dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, batch=batch, rows_lo=rows_lo,
                rows_hi=rows_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, sizes=sizes)


def _paged(name, dtype, hq, hkv, d, page, batch, rows_lo, rows_hi, ctx_lo, ctx_hi, causal=True, window=0, sizes=12):
    return dict(name=name, kind="paged", dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, batch=batch, rows_lo=rows_lo,
                rows_hi=rows_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, causal=causal, window=window, sizes=sizes)


def _prompt(name, dtype, hq, hkv, d, batch, rows_lo, rows_hi, causal=True, window=0, sizes=13):
    return dict(name=name, kind="prompt", dtype=dtype, hq=hq, hkv=hkv, d=d, batch=batch, rows_lo=rows_lo,
                rows_hi=rows_hi, causal=causal, window=window, sizes=sizes)


def _logprobs(name, dtype, rows, vocab, top, temperature, banned):
    return dict(name=name, kind="logprobs", dtype=dtype, rows=rows, vocab=vocab, top=top, temperature=temperature,
                banned=banned)


def _log_int(rng, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the same ranges: any operator, head layout, page size and length."""
    kind = rng.choice(["append", "paged", "paged", "prompt", "prompt", "logprobs"])
    if kind == "logprobs":
        vocab = _log_int(rng, 500, 160000)
        rows = _log_int(rng, 1, max(2, min(4000, 300_000_000 // vocab)))
        c = _logprobs("", rng.choice(["f32", "bf16"]), rows, vocab, rng.choice([0, 1, 3, 5, 8, 13, 20, 32]),
                      rng.choice([1.0, 0.6, 1.3]), rng.choice([0.0, 0.0, 0.3]))
        del c["name"]
        return c
    f32 = rng.random() < 0.25
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    heads = dict(dtype="f32" if f32 else "bf16", hq=hkv * g, hkv=hkv, d=rng.choice([64, 128]))
    sizes = rng.randrange(1 << 30)
    if kind == "append":
        c = _append("", **heads, page=rng.choice([8, 16, 32, 64, 128, 256]), batch=_log_int(rng, 1, 64), rows_lo=1,
                    rows_hi=_log_int(rng, 1, 128), ctx_lo=1, ctx_hi=_log_int(rng, 16, 2048), sizes=sizes)
    elif kind == "paged":
        rows_hi = rng.choice([1, _log_int(rng, 2, 16), _log_int(rng, 17, 300)])
        batch = _log_int(rng, 1, 48 if rows_hi < 17 else 4)
        c = _paged("", **heads, page=rng.choice([8, 16, 32, 64, 128, 256]), batch=batch, rows_lo=1, rows_hi=rows_hi,
                   ctx_lo=1, ctx_hi=_log_int(rng, 64, 2000 if f32 else 8000), causal=rng.random() < 0.8,
                   window=rng.choice([0, 0, _log_int(rng, 16, 4096)]), sizes=sizes)
    else:
        c = _prompt("", **heads, batch=_log_int(rng, 1, 12), rows_lo=1, rows_hi=_log_int(rng, 8, 900 if f32 else 3000),
                    causal=rng.random() < 0.85, window=rng.choice([0, 0, _log_int(rng, 16, 2048)]), sizes=sizes)
    del c["name"]
    return c


def _lengths(case):
    """New rows and cached length (the new rows among them) of every sequence, from the case alone."""
    rng = random.Random(case["sizes"])
    rows = [_log_int(rng, case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
    if case["kind"] == "prompt":
        if case["batch"] > 1:
            rows[rng.randrange(case["batch"])] = case["rows_hi"]
        return rows, list(rows)
    ctx = [_log_int(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    return rows, [c + r for c, r in zip(ctx, rows)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    st = dict(case=case)
    if case["kind"] == "logprobs":
        R, V = case["rows"], case["vocab"]
        logits = torch.empty((R, V), dtype=dt, device="cuda")
        for r0 in range(0, R, 256):   # in slices: the fp32 draw is larger than the rows kept
            n = min(256, R - r0)
            x = torch.randn((n, V), generator=gen, device="cuda") * 2.5
            if case["banned"]:
                x[torch.rand((n, V), generator=gen, device="cuda") < case["banned"]] = -math.inf
            # a confident model's rows: one token stands out by up to 12
            best = torch.randint(0, V, (n, 1), generator=gen, device="cuda")
            x.scatter_(1, best, 8.0 + 12.0 * torch.rand((n, 1), generator=gen, device="cuda"))
            logits[r0:r0 + n] = x
        # half of the given tokens are the likeliest, half any token
        tokens = torch.randint(0, V, (R,), generator=gen, device="cuda", dtype=torch.int32)
        pick = torch.rand(R, generator=gen, device="cuda") < 0.5
        tokens = torch.where(pick, logits.argmax(1).to(torch.int32), tokens)
        f = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")
        st.update(logits=logits, tokens=tokens, logprobs=f(R), entropy=f(R), top_logprobs=f(R, case["top"]),
                  top_ids=torch.empty((R, case["top"]), dtype=torch.int32, device="cuda"))
        return st
    rows, lens = _lengths(case)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    total, hq, hkv, d = starts[-1], case["hq"], case["hkv"], case["d"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st.update(host_rows=rows, host_lens=lens, host_starts=starts, starts=i32(starts))
    if case["kind"] != "append":
        st.update(q=normal(total, hq, d), out=torch.empty((total, hq, d), dtype=dt, device="cuda"),
                  lse=torch.empty((total, hq), dtype=torch.float32, device="cuda"))
    if case["kind"] != "paged":
        # K and V as the fused QKV product leaves them: column ranges of one row
        kv = normal(total, 2 * hkv, d)
        st.update(k=kv[:, :hkv], v=kv[:, hkv:])
    if case["kind"] != "prompt":
        page = case["page"]
        need = [(n + page - 1) // page for n in lens]
        spare = 3
        order = torch.randperm(sum(need) + spare, generator=gen, device="cuda")
        table = torch.zeros((case["batch"], max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        st.update(table=table, lens=i32(lens), k_pages=normal(sum(need) + spare, page, hkv, d),
                  v_pages=normal(sum(need) + spare, page, hkv, d))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import block_diffusion_speculative_flush_gb300 as D
    c = st["case"]
    if c["kind"] == "append":
        D.dflash_kv_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["starts"], st["lens"], st["table"])
        return st["k_pages"], st["v_pages"]
    if c["kind"] == "paged":
        D.dflash_paged_attention(st["q"], st["k_pages"], st["v_pages"], st["starts"], st["lens"], st["table"],
                                 st["out"], max_rows=max(st["host_rows"]), max_len=max(st["host_lens"]),
                                 causal=c["causal"], window=c["window"], lse=st["lse"])
        return st["out"], st["lse"]
    if c["kind"] == "prompt":
        D.dflash_prompt_attention(st["q"], st["k"], st["v"], st["starts"], st["out"], max_rows=max(st["host_rows"]),
                                  causal=c["causal"], window=c["window"], lse=st["lse"])
        return st["out"], st["lse"]
    top = c["top"] > 0
    D.dflash_token_logprobs(st["logits"], st["tokens"], st["logprobs"], entropy=st["entropy"],
                            top_ids=st["top_ids"] if top else None, top_logprobs=st["top_logprobs"] if top else None,
                            temperature=c["temperature"])
    return st["logprobs"], st["entropy"], st["top_ids"], st["top_logprobs"]


def _slots(st, b):
    """Pages and slots of sequence b's positions 0 .. len - 1."""
    pos = torch.arange(st["host_lens"][b], device="cuda")
    page = st["case"]["page"]
    return st["table"][b].long()[pos // page], pos % page


def _run_plain(st):
    c = st["case"]
    if c["kind"] == "append":
        for b, n in enumerate(st["host_rows"]):
            pg, sl = _slots(st, b)
            s = st["host_starts"][b]
            st["k_pages"][pg[-n:], sl[-n:]] = st["k"][s:s + n]
            st["v_pages"][pg[-n:], sl[-n:]] = st["v"][s:s + n]
        return st["k_pages"], st["v_pages"]
    if c["kind"] == "logprobs":
        return _plain_logprobs(st)
    for b, n in enumerate(st["host_rows"]):
        s = st["host_starts"][b]
        if c["kind"] == "paged":
            pg, sl = _slots(st, b)
            k, v = st["k_pages"][pg, sl], st["v_pages"][pg, sl]
        else:
            k, v = st["k"][s:s + n], st["v"][s:s + n]
        _plain_attention(c, st["q"][s:s + n], k, v, st["out"][s:s + n], st["lse"][s:s + n])
    return st["out"], st["lse"]


def _plain_attention(c, q, k, v, out, lse):
    n, L, g = q.shape[0], k.shape[0], c["hq"] // c["hkv"]
    qpos = torch.arange(L - n, L, device="cuda")[:, None]
    kpos = torch.arange(L, device="cuda")[None, :]
    hidden = torch.zeros((n, L), dtype=torch.bool, device="cuda")
    if c["causal"]:
        hidden |= kpos > qpos
    if c["window"]:
        hidden |= qpos - kpos >= c["window"]
    for h in range(c["hkv"]):
        kh, vh = k[:, h].float(), v[:, h].float()
        qh = q[:, h * g:(h + 1) * g].float().transpose(0, 1)             # [g, n, d]
        s = torch.matmul(qh, kh.t()) * (1.0 / math.sqrt(c["d"]))
        s.masked_fill_(hidden, -math.inf)
        m = s.amax(-1, keepdim=True)                                     # every row sees its own key
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        out[:, h * g:(h + 1) * g] = (torch.matmul(p, vh) / z).transpose(0, 1).to(out.dtype)
        lse[:, h * g:(h + 1) * g] = (m + torch.log(z))[..., 0].t()


def _plain_logprobs(st):
    c = st["case"]
    V, k = c["vocab"], c["top"]
    ids = torch.arange(V, device="cuda")
    for r0 in range(0, c["rows"], 512):
        sl = slice(r0, r0 + 512)
        raw = st["logits"][sl].float()
        z = raw * (1.0 / c["temperature"])
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(1, keepdim=True)
        logp = (z - m) - torch.log(total)
        st["logprobs"][sl] = logp.gather(1, st["tokens"][sl].long()[:, None])[:, 0]
        st["entropy"][sl] = -torch.where(e > 0, e * logp, 0.0).sum(1) / total[:, 0]
        if k:
            # one 64-bit key per entry: the value's order above, the id below (ties to the lowest)
            bits = torch.where(raw == 0, 0.0, raw).view(torch.int32).long()
            order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
            best = torch.topk(order * (1 << 20) - ids, k, dim=1).indices
            st["top_ids"][sl] = best.to(torch.int32)
            st["top_logprobs"][sl] = logp.gather(1, best)
    return st["logprobs"], st["entropy"], st["top_ids"], st["top_logprobs"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "append":
        K, W = st["k_pages"], st["v_pages"]
        for b, n in enumerate(st["host_rows"]):
            row = st["host_starts"][b]
            first = st["host_lens"][b] - n
            at = torch.arange(first, first + n, device="cuda")
            flat = st["table"][b].long().index_select(0, at.div(case["page"], rounding_mode="floor")) * case["page"] \
                + at.remainder(case["page"])
            K.view(-1, *K.shape[2:]).index_copy_(0, flat, st["k"][row:row + n].contiguous())
            W.view(-1, *W.shape[2:]).index_copy_(0, flat, st["v"][row:row + n].contiguous())
        return K, W
    if case["kind"] == "logprobs":
        k = case["top"]
        outs = []
        for r in torch.split(torch.arange(case["rows"], device="cuda"), 128):
            x = st["logits"][r].double()
            y = x / case["temperature"]
            lse = torch.logsumexp(y, 1)
            p = torch.exp(y - lse[:, None])
            plogp = torch.special.entr(p).sum(1)
            tok = y[torch.arange(len(r), device="cuda"), st["tokens"][r].long()] - lse
            by = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k] if k else \
                torch.empty((len(r), 0), dtype=torch.long, device="cuda")
            outs.append((tok, plogp, by.to(torch.int32), torch.gather(y, 1, by) - lse[:, None]))
        return tuple(torch.cat(o) for o in zip(*outs))
    total, hq, d = st["q"].shape
    out = torch.zeros((total, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64, device="cuda")
    g = hq // case["hkv"]
    for b, n in enumerate(st["host_rows"]):
        s0, L = st["host_starts"][b], st["host_lens"][b]
        if case["kind"] == "paged":
            used = st["table"][b, :(L + case["page"] - 1) // case["page"]].long()
            k64 = st["k_pages"].index_select(0, used).flatten(0, 1)[:L].double()
            v64 = st["v_pages"].index_select(0, used).flatten(0, 1)[:L].double()
        else:
            k64, v64 = st["k"][s0:s0 + n].double(), st["v"][s0:s0 + n].double()
        for h in range(hq):
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                first, last = L - n + i0, L - n + i1 - 1          # positions of this block of rows
                hi = last + 1 if case["causal"] else L
                lo = max(0, first - case["window"] + 1) if case["window"] else 0
                a = (st["q"][s0 + i0:s0 + i1, h].double() @ k64[lo:hi, h // g].t()) / math.sqrt(d)
                rel = torch.arange(first, last + 1, device="cuda")[:, None] - torch.arange(lo, hi, device="cuda")
                see = torch.ones_like(rel, dtype=torch.bool)
                if case["causal"]:
                    see &= rel >= 0
                if case["window"]:
                    see &= rel < case["window"]
                a = torch.where(see, a, -math.inf)
                z = torch.logsumexp(a, 1)
                out[s0 + i0:s0 + i1, h] = torch.exp(a - z[:, None]) @ v64[lo:hi, h // g]
                lse[s0 + i0:s0 + i1, h] = z
    return out, lse


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _visible(case, n, L):
    """(query, key) pairs that a head's rows see, and the distinct keys among them."""
    pairs = keys = 0
    W = case["window"]
    for p in range(L - n, L):
        hi = p + 1 if case["causal"] else L
        lo = max(0, p - W + 1) if W else 0
        pairs += hi - lo
    lo = max(0, L - n - W + 1) if W else 0
    keys = L - lo
    return pairs, keys


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * e + case["rows"] * (4 + 8 + 8 * case["top"]), "flops": 5 * n}
    rows, lens = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["kind"] == "append":
        return {"bytes": 4 * sum(rows) * hkv * d * e, "flops": 0}
    pairs = keys = 0
    for n, L in zip(rows, lens):
        p, k = _visible(case, n, L)
        pairs += p
        keys += k
    return {"bytes": 2 * sum(rows) * hq * d * e + 4 * sum(rows) * hq + 2 * keys * hkv * d * e,
            "flops": 4 * d * hq * pairs}
