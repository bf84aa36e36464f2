"""The workloads of the compressed cache's operators: cases, plain forms, definitions and work.

What a target's layer does around a K/V cache that is held in 8 bits, in the order
in which a serving step does it: rotary positions of the new queries and keys
(rope), the new rows into 8-bit pages with a scale for each page and KV head
(append8), attention over those pages (attn8), and the pages themselves as
sequences fork, grow, shrink and end (step) and as the pool is made dense again
(compact).

`own` chooses between the plain form (elementary torch operations in 32 bits, in
64 for angles and for values next to a border) and the library's calls.  `exact`
is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    qwen = dict(dtype="bf16", hq=32, hkv=8, d=128)      # the 8B-shaped draft's heads
    laguna = dict(dtype="bf16", hq=24, hkv=8, d=128)    # the windowed draft's heads
    return [
        # a decode step of a 64-sequence server: one new token each, far into long contexts
        _rope("rope_decode_64", **qwen, rot=128, layout="half", scaling="bands", batch=64, rows_lo=1, rows_hi=1,
              ctx_lo=1024, ctx_hi=1000000),
        # prompts being read in: neighbouring pairs, half of the head rotated, a stretched context
        _rope("rope_prompts", **qwen, rot=64, layout="interleaved", scaling="yarn", batch=7, rows_lo=301, rows_hi=4096,
              ctx_lo=1, ctx_hi=60000),
        # the decode step's 64 new rows into their pages
        _append8("append8_decode_64", **qwen, page=16, batch=64, rows_lo=1, rows_hi=1, ctx_lo=1024, ctx_hi=16384),
        # chunks of prompts into pages of 64: odd lengths, begun pages among them
        _append8("append8_chunks", **qwen, page=64, batch=7, rows_lo=301, rows_hi=2048, ctx_lo=1, ctx_hi=4096),
        # the block of one user's verify step at the headline context
        _attn8("attn8_verify_one_user", **qwen, page=16, batch=1, rows_lo=16, rows_hi=16, ctx_lo=4096, ctx_hi=4096),
        # a decode step of the serving mix: single tokens, contexts 1k to 16k
        _attn8("attn8_decode_mix_64", **qwen, page=16, batch=64, rows_lo=1, rows_hi=1, ctx_lo=1024, ctx_hi=16384),
        # verify steps of eight users of a sliding-window model, blocks of up to 8
        _attn8("attn8_verify_window", **laguna, page=32, batch=8, rows_lo=2, rows_hi=8, ctx_lo=257, ctx_hi=32768,
               window=512),
        # chunked prefill over long caches
        _attn8("attn8_chunked_prefill", **qwen, page=64, batch=6, rows_lo=129, rows_hi=512, ctx_lo=1000, ctx_hi=16000),
        # one user's four candidates dropped and forked anew from the committed tokens, eight tokens each to come
        _step("pages_step_one_user", hkv=8, d=128, page=16, layers=2, prompts=1, forks=4, len_lo=1000, len_hi=1000,
              grow=8),
        # 32 prompts with 8 samples each: the begun page of every fork is copied in all layers before it is written
        _step("pages_step_32x8", hkv=8, d=128, page=16, layers=8, prompts=32, forks=8, len_lo=301, len_hi=4096, grow=8),
        # a small pool made dense
        _compact("pages_compact_small", hkv=8, d=128, page=16, layers=2, batch=9, len_lo=17, len_hi=900, holes=0.5),
        # a pool of 64 long sequences made dense after half of its pages were freed here and there
        _compact("pages_compact_64", hkv=8, d=128, page=16, layers=8, batch=64, len_lo=128, len_hi=4096, holes=0.5),
    ]


def _rope(name, dtype, hq, hkv, d, rot, layout, scaling, batch, rows_lo, rows_hi, ctx_lo, ctx_hi, back=False, sizes=21):
    return dict(name=name, kind="rope", dtype=dtype, hq=hq, hkv=hkv, d=d, rot=rot, layout=layout, scaling=scaling,
                batch=batch, rows_lo=rows_lo, rows_hi=rows_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, back=back, sizes=sizes)


def _append8(name, dtype, hq, hkv, d, page, batch, rows_lo, rows_hi, ctx_lo, ctx_hi, sizes=22):
    return dict(name=name, kind="append8", dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, batch=batch, rows_lo=rows_lo,
                rows_hi=rows_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, sizes=sizes)


def _attn8(name, dtype, hq, hkv, d, page, batch, rows_lo, rows_hi, ctx_lo, ctx_hi, causal=True, window=0, sizes=23):
    return dict(name=name, kind="attn8", dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, batch=batch, rows_lo=rows_lo,
                rows_hi=rows_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, causal=causal, window=window, sizes=sizes)


def _step(name, hkv, d, page, layers, prompts, forks, len_lo, len_hi, grow, sizes=24):
    return dict(name=name, kind="step", hkv=hkv, d=d, page=page, layers=layers, prompts=prompts, forks=forks,
                len_lo=len_lo, len_hi=len_hi, grow=grow, sizes=sizes)


def _compact(name, hkv, d, page, layers, batch, len_lo, len_hi, holes, sizes=25):
    return dict(name=name, kind="compact", hkv=hkv, d=d, page=page, layers=layers, batch=batch, len_lo=len_lo,
                len_hi=len_hi, holes=holes, sizes=sizes)


def _log_int(rng, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the same ranges: any operator, head layout, page size and length."""
    kind = rng.choice(["rope", "append8", "attn8", "attn8", "attn8", "step", "compact"])
    hkv, d, sizes = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "step":
        c = _step("", hkv, d, page, layers=rng.choice([1, 2, 3, 5]), prompts=_log_int(rng, 1, 32),
                  forks=rng.randint(1, 8), len_lo=1, len_hi=_log_int(rng, 16, 4000), grow=_log_int(rng, 1, 40), sizes=sizes)
    elif kind == "compact":
        c = _compact("", hkv, d, page, layers=rng.choice([1, 2, 3, 5]), batch=_log_int(rng, 1, 64), len_lo=1,
                     len_hi=_log_int(rng, 16, 4000), holes=rng.uniform(0.1, 0.8), sizes=sizes)
    else:
        f32 = rng.random() < 0.25
        heads = dict(dtype="f32" if f32 else "bf16", hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), hkv=hkv, d=d)
        if kind == "rope":
            c = _rope("", **heads, rot=rng.choice([d, d // 2, 24]), layout=rng.choice(["half", "interleaved"]),
                      scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]), batch=_log_int(rng, 1, 64),
                      rows_lo=1, rows_hi=_log_int(rng, 1, 200), ctx_lo=1, ctx_hi=_log_int(rng, 16, 2000000),
                      back=rng.random() < 0.3, sizes=sizes)
        elif kind == "append8":
            c = _append8("", **heads, page=page, batch=_log_int(rng, 1, 64), rows_lo=1, rows_hi=_log_int(rng, 1, 128),
                         ctx_lo=1, ctx_hi=_log_int(rng, 16, 2048), sizes=sizes)
        else:
            rows_hi = rng.choice([1, _log_int(rng, 2, 16), _log_int(rng, 17, 300)])
            c = _attn8("", **heads, page=page, batch=_log_int(rng, 1, 48 if rows_hi < 17 else 4), rows_lo=1,
                       rows_hi=rows_hi, ctx_lo=1, ctx_hi=_log_int(rng, 64, 2000 if f32 else 8000),
                       causal=rng.random() < 0.8, window=rng.choice([0, 0, _log_int(rng, 16, 4096)]), sizes=sizes)
    del c["name"]
    return c


def _lengths(case):
    """New rows and length (the new rows among them) of every sequence, from the case alone."""
    rng = random.Random(case["sizes"])
    rows = [_log_int(rng, case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
    return rows, [r + _log_int(rng, case["ctx_lo"], case["ctx_hi"]) for r in rows]


def _step_lengths(case):
    rng = random.Random(case["sizes"])
    return [_log_int(rng, case["len_lo"], case["len_hi"]) for _ in range(case["prompts" if case["kind"] == "step" else "batch"])]


def _pages(n, page):
    return (n + page - 1) // page


# ---------------------------------------------------------------------------
# rotary frequencies
# ---------------------------------------------------------------------------
ROPE_THETA = 1000000.0
ROPE_SCALINGS = {
    "none": dict(),
    "linear": dict(factor=4.0),
    "ntk": dict(factor=4.0),
    "bands": dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0),
    "yarn": dict(factor=4.0, original_len=32768.0, low=1.0, high=32.0),
}


def _rope_freqs(rot, scaling):
    """Radians a position of each pair in 64 bits, and the factor on cos and sin."""
    p = ROPE_SCALINGS[scaling]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    theta, amplitude = ROPE_THETA, 1.0
    if scaling == "ntk":
        theta = theta * p["factor"] ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / p["factor"]
    elif scaling == "bands":
        turns = p["original_len"] * f / (2 * math.pi)      # in the original context
        s = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0.0, 1.0)
        f = f * ((1 - s) / p["factor"] + s)
    elif scaling == "yarn":
        at = [rot * math.log(p["original_len"] / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (p["high"], p["low"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = f / p["factor"] * ramp + f * (1 - ramp)
        amplitude = 0.1 * math.log(p["factor"]) + 1.0
    return f, amplitude


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["kind"] in ("step", "compact"):
        return _prepare_pages(case, gen)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    rows, lens = _lengths(case)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    total, hq, hkv, d = starts[-1], case["hq"], case["hkv"], case["d"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st = dict(case=case, max_rows=max(rows), max_len=max(lens), starts=i32(starts), lens=i32(lens))
    if case["kind"] == "rope":
        # Q, K and V as the fused product leaves them: column ranges of one row
        qkv = normal(total, hq + 2 * hkv, d)
        st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], q_out=torch.empty((total, hq, d), dtype=dt, device="cuda"),
                  k_out=torch.empty((total, hkv, d), dtype=dt, device="cuda"))
        if own:
            import block_diffusion_speculative_flush_gb300 as D
            scaling = None if case["scaling"] == "none" else dict(kind=case["scaling"], **ROPE_SCALINGS[case["scaling"]])
            st["rope"] = D.dflash_rope_table(case["rot"], ROPE_THETA, layout=case["layout"], scaling=scaling)
        return st
    page = case["page"]
    need = [_pages(n, page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = i32([0] + need).cumsum(0)
    col = torch.arange(max(need), device="cuda")[None, :]
    st["table"] = torch.where(col < i32(need)[:, None], order[(at[:-1, None] + col).clamp(max=n_pages - 1)], 0).to(torch.int32)
    for name in ("k", "v"):
        # pages of one head differ in size; codes and scales as a cache holds them
        x = torch.randn((n_pages, page, hkv, d), generator=gen, device="cuda")
        x *= torch.exp2(4.0 * torch.rand((n_pages, 1, hkv, 1), generator=gen, device="cuda") - 2.0)
        scale = x.abs().amax((1, 3)) / E4M3_MAX
        if case["kind"] == "append8":
            scale = torch.exp2(torch.ceil(torch.log2(scale)))
        x /= scale[:, None, :, None]
        st[name + "_pages"] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
        st[name + "_scale"] = scale.contiguous()
        del x
    if case["kind"] == "append8":
        kv = normal(total, 2 * hkv, d)
        # tokens of other sizes than what their page holds: scales grow at some of them
        kv *= torch.exp2(6.0 * torch.rand((total, 2 * hkv, 1), generator=gen, device="cuda") - 4.0).to(dt)
        st.update(k=kv[:, :hkv], v=kv[:, hkv:])
    else:
        st.update(q=normal(total, hq, d), out=torch.empty((total, hq, d), dtype=dt, device="cuda"),
                  lse=torch.empty((total, hq), dtype=torch.float32, device="cuda"))
    return st


def _prepare_pages(case, gen):
    page, layers, hkv, d = case["page"], case["layers"], case["hkv"], case["d"]
    lens = _step_lengths(case)
    need = [_pages(n, page) for n in lens]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    if case["kind"] == "step":
        n, f = case["prompts"], case["forks"]
        width = _pages(max(lens) + case["grow"], page)
        n_pages = sum(need) + n * f * (_pages(case["grow"], page) + 1) + 5
        rows = n * (1 + f)
    else:
        n, width, rows = case["batch"], max(need), case["batch"]
        n_pages = int(sum(need) / (1 - case["holes"])) + 2
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = i32([0] + need).cumsum(0)
    col = torch.arange(width, device="cuda")[None, :]
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    table[:n] = torch.where(col < i32(need)[:, None], order[(at[:-1, None] + col).clamp(max=n_pages - 1)], -1)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[order[:sum(need)].long()] = 1
    lens_dev = torch.zeros(rows, dtype=torch.int32, device="cuda")
    lens_dev[:n] = i32(lens)
    bytes_ = lambda *s: torch.randint(0, 256, s, generator=gen, device="cuda", dtype=torch.uint8)
    data = {"k": bytes_(layers, n_pages, page, hkv, d), "v": bytes_(layers, n_pages, page, hkv, d),
            "k_scale": torch.randn((layers, n_pages, hkv), generator=gen, device="cuda").view(torch.int32),
            "v_scale": torch.randn((layers, n_pages, hkv), generator=gen, device="cuda").view(torch.int32)}
    st = dict(case=case, refs=refs, table=table, lens=lens_dev, data=data, new_table=torch.empty_like(table),
              new_lens=torch.empty_like(lens_dev))
    if case["kind"] == "step":
        parents = list(range(n)) + [b for b in range(n) for _ in range(f)]
        st.update(parents=i32(parents), want=i32(lens + [lens[b] + case["grow"] for b in parents[n:]]))
    else:
        st.update(new_refs=torch.empty_like(refs), used=torch.empty(1, dtype=torch.int32, device="cuda"))
    if own:
        import block_diffusion_speculative_flush_gb300 as D
        st["buffers"] = D.dflash_page_buffers([x[i] for x in data.values() for i in range(layers)])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _PLAIN[state["case"]["kind"]])(state)


def _flip(st):
    """The step's tables change places: what the last pass wrote is what this one reads."""
    st["table"], st["new_table"] = st["new_table"], st["table"]
    st["lens"], st["new_lens"] = st["new_lens"], st["lens"]
    return st["table"], st["lens"], st["refs"], st["data"]


def _run_own(st):
    import block_diffusion_speculative_flush_gb300 as D
    c = st["case"]
    kind = c["kind"]
    if kind == "rope":
        D.dflash_rope(st["rope"], st["q"], st["k"], st["starts"], st["lens"], st["q_out"], st["k_out"],
                      transpose=c["back"])
        return st["q_out"], st["k_out"]
    if kind == "append8":
        D.dflash_kv8_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["starts"],
                            st["lens"], st["table"])
        return st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"]
    if kind == "attn8":
        D.dflash_kv8_attention(st["q"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["starts"],
                               st["lens"], st["table"], st["out"], max_rows=st["max_rows"], max_len=st["max_len"],
                               causal=c["causal"], window=c["window"], lse=st["lse"])
        return st["out"], st["lse"]
    if kind == "step":
        D.dflash_pages_reorder(st["refs"], st["table"], st["lens"], st["parents"], st["new_table"], st["new_lens"],
                               page_size=c["page"])
        D.dflash_pages_resize(st["refs"], st["new_table"], st["new_lens"], st["want"], st["buffers"],
                              page_size=c["page"])
        return _flip(st)
    D.dflash_pages_compact(st["refs"], st["table"], st["lens"], st["new_refs"], st["new_table"], st["buffers"],
                           page_size=c["page"], used=st["used"])
    return st["new_table"], st["new_refs"], st["used"], st["data"]


def _rows_of(st, total):
    """Sequence and position of every packed row."""
    row = torch.arange(total, device="cuda")
    starts = st["starts"].long()
    b = (row[:, None] >= starts[None, 1:]).sum(1)
    return b, st["lens"].long()[b] - starts[b + 1] + row


def _plain_rope(st):
    c = st["case"]
    rot, h = c["rot"], c["rot"] // 2
    f, amplitude = _rope_freqs(rot, c["scaling"])
    _, pos = _rows_of(st, st["q"].shape[0])
    angle = pos.double()[:, None] * f[None, :]              # 64 bits: far positions
    if c["back"]:
        angle = -angle
    cos = (torch.cos(angle) * amplitude).float()[:, None, :]
    sin = (torch.sin(angle) * amplitude).float()[:, None, :]

    def turn(x, out):
        out.copy_(x)
        r = x[..., :rot].float()
        if c["layout"] == "half":
            a, b = r[..., :h], r[..., h:]
            out[..., :rot] = torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(out.dtype)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            out[..., :rot] = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2).to(out.dtype)
        return out

    return turn(st["q"], st["q_out"]), turn(st["k"], st["k_out"])


def _plain_append8(st):
    page = st["case"]["page"]
    total = st["k"].shape[0]
    b, pos = _rows_of(st, total)
    pg, slot = st["table"][b, pos // page].long(), pos % page
    touched = torch.zeros(st["k_scale"].shape[0], dtype=torch.bool, device="cuda")
    touched[pg] = True
    first = torch.full(touched.shape, page, dtype=torch.long, device="cuda")    # first new slot of a page
    first.scatter_reduce_(0, pg, slot, "amin")
    t = touched.nonzero()[:, 0]
    at = torch.zeros_like(first)
    at[t] = torch.arange(len(t), device="cuda")
    held = torch.arange(page, device="cuda")[None, :] < first[t, None]          # slots that keep their rows

    def put(x, pages, scale):
        x = x.float()
        most = torch.zeros(scale.shape, device="cuda").scatter_reduce_(
            0, pg[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
        # the smallest power of two that holds it, found in 64 bits
        m, e = torch.frexp(most[t].double() / E4M3_MAX)
        want = torch.exp2(torch.where(m == 0.5, e - 1, e).clamp(-60, 60).double()).float()
        want = torch.where(most[t] > 0, want, 2.0 ** -60)
        new = torch.where(first[t, None] > 0, torch.maximum(want, scale[t]), want)
        codes = pages.view(torch.uint8)[t].view(E4M3)
        again = (codes.float() * (scale[t] / new)[:, None, :, None]).to(E4M3)
        kept = torch.where(held[:, :, None, None], again.view(torch.uint8), codes.view(torch.uint8))
        kept[at[pg], slot] = (x / new[at[pg]][..., None]).to(E4M3).view(torch.uint8)
        pages.view(torch.uint8)[t] = kept
        scale[t] = new

    put(st["k"], st["k_pages"], st["k_scale"])
    put(st["v"], st["v_pages"], st["v_scale"])
    return st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"]


def _plain_attn8(st):
    c = st["case"]
    total, hq, d = st["q"].shape
    page, hkv, g = c["page"], c["hkv"], hq // c["hkv"]
    n, L = st["max_rows"], st["max_len"]
    width = _pages(L, page)
    lens = st["lens"].long()
    table = st["table"][:, :width].long()

    def values(pages, scale):                                # [batch, hkv, L, d]
        x = pages.view(torch.uint8)[table].view(E4M3).float() * scale[table][:, :, None, :, None]
        return x.flatten(1, 2).transpose(1, 2)

    b, pos = _rows_of(st, total)
    i = pos - (lens - (st["starts"][1:] - st["starts"][:-1]).long())[b]
    q = torch.zeros((len(lens), n, hq, d), device="cuda")
    q[b, i] = st["q"].float()
    q = q.view(-1, n, hkv, g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)            # [batch, hkv, g n, d]
    k = values(st["k_pages"], st["k_scale"])
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    key = torch.arange(s.shape[-1], device="cuda")
    qpos = (lens - (st["starts"][1:] - st["starts"][:-1]).long())[:, None] + torch.arange(n, device="cuda")
    hidden = (key >= lens[:, None, None]) | (c["causal"] & (key > qpos[..., None]))
    if c["window"]:
        hidden = hidden | (qpos[..., None] - key >= c["window"])
    s = s.view(len(lens), hkv, g, n, -1).masked_fill_(hidden[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)            # (rows of padding see nothing)
    p = torch.exp_(s.sub_(m))
    z = p.sum(-1, keepdim=True)
    # pages that only fill the table up may hold anything
    v = values(st["v_pages"], st["v_scale"]).masked_fill_((key >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.flatten(2, 3), v).view(len(lens), hkv, g, n, d) / z
    st["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i])
    st["lse"].copy_((m + torch.log(z))[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[b, i])
    return st["out"], st["lse"]


def _held(table, lens, page):
    """Which entries of the table name a page that its row holds."""
    return torch.arange(table.shape[1], device="cuda")[None, :] * page < lens[:, None]


def _counts(table, held, n):
    return torch.bincount(table[held].long(), minlength=n).to(torch.int32)


def _move(data, src, dst):
    for x in data.values():
        x[:, dst] = x[:, src]


def _plain_step(st):
    c = st["case"]
    page, refs, n = c["page"], st["refs"], st["refs"].shape[0]
    old, parents = st["table"], st["parents"].long()
    # the rows of the step: forked, kept, dropped
    lens = st["lens"][parents]
    held = _held(old[parents], lens, page)
    table = torch.where(held, old[parents], -1)
    refs += _counts(table, held, n) - _counts(old, _held(old, st["lens"], page), n)
    # growth: begun pages that others hold too are copied, new pages are the lowest free ones
    want = st["want"]
    have, need = (lens + page - 1) // page, (want + page - 1) // page
    grows = (want > lens) & (lens % page != 0)
    last = table.gather(1, (have - 1).clamp(min=0).long()[:, None])[:, 0].clamp(min=0).long()
    writers = torch.bincount(last[grows], minlength=n)
    row = torch.arange(len(want), device="cuda")
    lowest = torch.full((n,), len(want), device="cuda").scatter_reduce_(0, last[grows], row[grows], "amin")
    keeps = (refs[last] == 1) | ((refs[last] == writers[last]) & (lowest[last] == row))
    copies = grows & ~keeps
    count = need - have + copies
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = ((col >= have[:, None]) & (col < need[:, None])) | (copies[:, None] & (col == have[:, None] - 1))
    free = (refs == 0).nonzero()[:, 0]
    given = free[:int(count.sum())]
    moved = table[copies[:, None] & (col == have[:, None] - 1)].long()
    refs -= torch.bincount(moved, minlength=n).to(torch.int32)
    table[fresh] = given.to(torch.int32)
    refs[given] = 1
    _move(st["data"], moved, table[copies[:, None] & (col == have[:, None] - 1)].long())
    st["new_table"].copy_(table)
    st["new_lens"].copy_(want)
    return _flip(st)


def _plain_compact(st):
    refs = st["refs"]
    used = int((refs > 0).sum())
    page = torch.arange(refs.shape[0], device="cuda")
    src, dst = page[(refs > 0) & (page >= used)], page[(refs == 0) & (page < used)]
    to = page.clone()
    to[src] = dst
    held = _held(st["table"], st["lens"], st["case"]["page"])
    st["new_table"].copy_(torch.where(held, to[st["table"].clamp(min=0).long()], -1))
    st["new_refs"].copy_(refs)
    st["new_refs"][dst] = refs[src]
    st["new_refs"][used:] = 0
    _move(st["data"], src, dst)
    st["used"].fill_(used)
    return st["new_table"], st["new_refs"], st["used"], st["data"]


_PLAIN = {"rope": _plain_rope, "append8": _plain_append8, "attn8": _plain_attn8, "step": _plain_step,
          "compact": _plain_compact}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["kind"] in ("step", "compact"):
        return None                                          # whole numbers and copies
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append8": _exact_append8, "attn8": _exact_attn8}[case["kind"]](case, st)


def _exact_rope(case, st):
    rows, lens = _lengths(case)
    rot = case["rot"]
    p = ROPE_SCALINGS[case["scaling"]]
    speed, size = [], 1.0
    for i in range(rot // 2):
        base = ROPE_THETA * (p["factor"] ** (rot / (rot - 2)) if case["scaling"] == "ntk" else 1.0)
        w = math.pow(base, -2.0 * i / rot)
        if case["scaling"] == "linear":
            w /= p["factor"]
        if case["scaling"] == "bands":
            t = p["original_len"] * w / (2 * math.pi)
            share = 0.0 if t < p["low"] else 1.0 if t > p["high"] else (t - p["low"]) / (p["high"] - p["low"])
            w = share * w + (1 - share) * w / p["factor"]
        if case["scaling"] == "yarn":
            dim = lambda turns: rot * math.log(p["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(0, math.floor(dim(p["high"]))), min(rot - 1, math.ceil(dim(p["low"])))
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = (1 - share) * w + share * w / p["factor"]
            size = 1.0 + 0.1 * math.log(p["factor"])
        speed.append(w)
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(rows, lens)]).cuda().double()
    angle = torch.outer(pos, torch.tensor(speed, dtype=torch.float64, device="cuda"))
    unit = torch.polar(torch.full_like(angle, size), -angle if case["back"] else angle)[:, None]
    outs = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        part = y[..., :rot]
        pairs = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(-1, (rot // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        part.copy_((z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2))
        outs.append(y)
    return tuple(outs)


def _exact_append8(case, st):
    page = case["page"]
    rows, lens = _lengths(case)
    outs = []
    for name in ("k", "v"):
        codes, scale = st[name + "_pages"].double(), st[name + "_scale"].double()
        at = 0
        for b, (n, L) in enumerate(zip(rows, lens)):
            p = L - n
            while p < L:
                pg, s0 = int(st["table"][b, p // page]), p % page
                m = min(page - s0, L - p)
                x = st[name][at:at + m].double()
                most = x.abs().amax((0, 2))
                # 448 times a power of two holds it: that power, no further from 1 than 2^60
                want = torch.exp2(torch.ceil(torch.log2(most / E4M3_MAX)).clamp(-60, 60))
                new = torch.maximum(want, scale[pg]) if s0 else want
                if s0:
                    codes[pg, :s0] = (codes[pg, :s0] * (scale[pg] / new)[:, None]).to(E4M3).double()
                codes[pg, s0:s0 + m] = (x / new[:, None]).to(E4M3).double()
                scale[pg] = new
                p, at = p + m, at + m
        outs.append((codes, scale))
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


def _exact_attn8(case, st):
    total, hq, d = st["q"].shape
    out = torch.zeros((total, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64, device="cuda")
    g, s0 = hq // case["hkv"], 0
    for b, (n, L) in enumerate(zip(*_lengths(case))):
        used = st["table"][b, :_pages(L, case["page"])].long()
        whole = lambda x, s: (x.view(torch.uint8).index_select(0, used).view(E4M3).double() *
                              s.index_select(0, used).double()[:, None, :, None]).flatten(0, 1)[:L]
        k64, v64 = whole(st["k_pages"], st["k_scale"]), whole(st["v_pages"], st["v_scale"])
        rel = torch.arange(L - n, L, device="cuda")[:, None] - torch.arange(L, device="cuda")
        see = torch.ones_like(rel, dtype=torch.bool)
        if case["causal"]:
            see &= rel >= 0
        if case["window"]:
            see &= rel < case["window"]
        for h in range(hq):
            a = (st["q"][s0:s0 + n, h].double() @ k64[:, h // g].t()) / math.sqrt(d)
            a = torch.where(see, a, -math.inf)
            z = torch.logsumexp(a, 1)
            out[s0:s0 + n, h] = torch.exp(a - z[:, None]) @ v64[:, h // g]
            lse[s0:s0 + n, h] = z
        s0 += n
    return out, lse


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    kind = case["kind"]
    if kind in ("step", "compact"):
        page, lens = case["page"], _step_lengths(case)
        entry = 2 * case["layers"] * case["hkv"] * (page * case["d"] + 4)        # bytes of a page, all layers
        held = sum(_pages(n, page) for n in lens)
        if kind == "step":
            f, grow = case["forks"], case["grow"]
            copied = f * sum(n % page != 0 for n in lens)
            rows = (1 + f) * held + f * sum(_pages(n + grow, page) - _pages(n, page) for n in lens)
            return {"bytes": 2 * copied * entry + 8 * rows, "flops": 0}
        # pages are spread evenly: as many lie behind the dense part as it has holes
        moved = held * case["holes"]
        return {"bytes": 2 * moved * entry + 8 * held + 8 * (int(held / (1 - case["holes"])) + 2), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    rows, lens = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if kind == "rope":
        n = sum(rows) * (hq + hkv)
        return {"bytes": 2 * n * d * e, "flops": 3 * n * case["rot"]}
    if kind == "append8":
        pages = sum(_pages(L, case["page"]) - (L - n) // case["page"] for n, L in zip(rows, lens))
        return {"bytes": 2 * sum(rows) * hkv * d * (e + 1) + 2 * 4 * pages * hkv, "flops": 4 * sum(rows) * hkv * d}
    pairs = keys = pages = 0
    W = case["window"]
    for n, L in zip(rows, lens):
        for p in range(L - n, L):
            pairs += (p + 1 if case["causal"] else L) - (max(0, p - W + 1) if W else 0)
        lo = max(0, L - n - W + 1) if W else 0
        keys += L - lo
        pages += _pages(L, case["page"]) - lo // case["page"]
    return {"bytes": 2 * sum(rows) * hq * d * e + 4 * sum(rows) * hq + 2 * hkv * (keys * d + 4 * pages),
            "flops": 4 * d * hq * pairs}
