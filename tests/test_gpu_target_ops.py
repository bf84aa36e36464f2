"""The target-side operators on the GPU against the fp64 oracle: append to
pages, attention of new rows over the paged cache, attention of packed
prompts, token log probabilities.  Bounds are the oracle module's."""
import math

import numpy as np
import pytest
import torch

from oracle import target_ops_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def lib():
    import block_diffusion_speculative_flush_gb300 as D
    return D


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(rows):
    return [0] + list(np.cumsum(rows))


class Batch:
    """A ragged batch over pages: rows[b] new rows, lens[b] tokens; every slot that holds no token of its
    sequence, every spare page and every row behind the last sequence is NaN."""

    def __init__(self, dtype, hq, hkv, d, page, rows, lens, seed=0, hnd=False, tail=3, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.hq, self.hkv, self.d, self.page, self.rows, self.lens = DT[dtype], hq, hkv, d, page, rows, lens
        self.starts = starts_of(rows)
        total = self.starts[-1] + tail
        rnd = lambda *s: torch.randn(s, generator=g).to(self.dt)
        self.q = rnd(total, hq, d)
        need = [(n + page - 1) // page for n in lens]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g)
        self.width = max(max(need), 1)
        self.table = torch.full((len(rows), self.width), -7, dtype=torch.int32)
        self.kp = torch.full((n_pages, page, hkv, d), math.nan, dtype=self.dt)
        self.vp = self.kp.clone()
        self.k, self.v = rnd(total, hkv, d), rnd(total, hkv, d)
        at = 0
        for b, L in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]].to(torch.int32)
            at += need[b]
            for p in range(L - rows[b]):
                self.kp[int(self.table[b, p // page]), p % page] = rnd(hkv, d)
                self.vp[int(self.table[b, p // page]), p % page] = rnd(hkv, d)
        self.hnd = hnd

    def appended(self):
        return (O.append(self.kp, self.k, self.starts, self.lens, self.table),
                O.append(self.vp, self.v, self.starts, self.lens, self.table))

    def pages_cuda(self, kp, vp):
        if self.hnd:   # [page][head][slot][d] in memory
            return tuple(x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (kp, vp))
        return kp.cuda(), vp.cuda()


def same_bits(a, b):
    a, b = a.contiguous(), b.contiguous()
    v = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.view(v), b.view(v))


def check_attention(o, lse, ref, rows):
    ro, rl, to, tl = ref
    err = (o[:rows].double().cpu() - ro[:rows]).abs()
    bad = ~(err <= to[:rows])
    assert not bad.any(), (int(bad.sum()), float(err[bad][0]), bad.nonzero()[:4].tolist())
    el = (lse[:rows].double().cpu() - rl[:rows]).abs()
    same_inf = torch.isneginf(lse[:rows].cpu()) & torch.isneginf(rl[:rows])
    assert bool((same_inf | (el <= tl[:rows])).all())


def run_paged(B, causal, window, scale=None, max_len=None, poison=False, append=True, status=None):
    """Append then attend; returns outputs (prefilled with 7 to see which rows were written)."""
    D = lib()
    kp, vp = B.pages_cuda(B.kp, B.vp)
    starts, lens, table = i32(B.starts), i32(B.lens), B.table.cuda()
    if append:
        D.dflash_kv_append(B.k.cuda(), B.v.cuda(), kp, vp, starts, lens, table, status=status)
    q = B.q.cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    D.dflash_paged_attention(q, kp, vp, starts, lens, table, out, max_rows=max(max(B.rows), 1), max_len=max_len,
                             causal=causal, window=window, scale=scale, lse=lse, status=status)
    torch.cuda.synchronize()
    return out, lse, kp, vp


def ref_paged(B, causal, window, scale=None):
    kp, vp = B.appended()
    return O.attention(B.q[:B.starts[-1]], O.gather(kp, B.lens, B.table), O.gather(vp, B.lens, B.table), B.starts,
                       B.lens, causal, window, scale if scale is not None else B.d ** -0.5, B.dt == torch.bfloat16)


SHAPES = [  # hq, hkv, page, rows, lens
    (4, 4, 8, [1], [1]),
    (8, 2, 16, [1, 1, 1], [1, 17, 300]),
    (6, 2, 16, [5, 0, 8, 1], [5, 0, 140, 64]),
    (5, 1, 32, [16], [129]),
    (8, 1, 64, [16, 3], [700, 128]),
    (7, 1, 128, [40, 33], [290, 33]),
    (4, 2, 8, [130, 1, 77], [130, 900, 205]),
    (16, 1, 256, [70], [513]),
]


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 37), (False, 130)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_and_paged_attention(dtype, d, causal, window, shape):
    hq, hkv, page, rows, lens = SHAPES[shape]
    B = Batch(dtype, hq, hkv, d, page, rows, lens, seed=shape, hnd=shape % 2 == 1)
    status = i32([0])
    out, lse, kp, vp = run_paged(B, causal, window, status=status)
    rk, rv = B.appended()
    assert same_bits(kp.cpu(), rk) and same_bits(vp.cpu(), rv)
    n = B.starts[-1]
    check_attention(out, lse, ref_paged(B, causal, window), n)
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())   # rows behind the last sequence
    lib().dflash_status_check(status)


@pytest.mark.parametrize("dtype,d", [("f32", 4), ("f32", 20), ("f32", 100)])
def test_paged_attention_of_other_fp32_head_dims(dtype, d):
    B = Batch(dtype, 6, 3, d, 16, [9, 1], [50, 400])
    out, lse, _, _ = run_paged(B, True, 0)
    check_attention(out, lse, ref_paged(B, True, 0), B.starts[-1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,lens", [([16], [5000]), ([1] * 9, [1, 4096, 5, 2999, 64, 128, 127, 129, 1000]),
                                       ([300, 2, 150], [2100, 3000, 150])])
def test_paged_attention_over_long_caches(dtype, rows, lens):
    B = Batch(dtype, 8, 2, 128, 16, rows, lens, seed=5)
    out, lse, _, _ = run_paged(B, True, 0)
    check_attention(out, lse, ref_paged(B, True, 0), B.starts[-1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,hq", [([1, 1, 1], 2), ([20, 9, 1], 4)])
def test_paged_attention_with_many_key_tiles_per_cta(rows, hq, d):
    """Enough keys that every CTA works through several tiles and more than one sequence."""
    B = Batch("bf16", hq, 2, d, 256, rows, [30011, 17, 16384], seed=7, tail=0)
    out, lse, _, _ = run_paged(B, True, 0)
    check_attention(out, lse, ref_paged(B, True, 0), B.starts[-1])


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50), (False, 20)])
@pytest.mark.parametrize("heads,rows", [((4, 4), [1]), ((8, 2), [37]), ((6, 2), [1, 0, 200, 129]),
                                        ((5, 1), [64, 300]), ((32, 1), [9, 100]), ((2, 2), [520, 3, 260])])
def test_prompt_attention(dtype, d, causal, window, heads, rows):
    D = lib()
    hq, hkv = heads
    g = torch.Generator().manual_seed(sum(rows) + hq)
    st = starts_of(rows)
    n, total = st[-1], st[-1] + 2
    # q, k and v as column ranges of one fused row, as a QKV product leaves them
    qkv = torch.randn((total, hq + 2 * hkv, d), generator=g).to(DT[dtype])
    qkv[n:] = math.nan
    dev = qkv.cuda()
    out = torch.full((total, hq, d), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((total, hq), 7.0, device="cuda")
    status = i32([0])
    D.dflash_prompt_attention(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], i32(st), out, max_rows=max(rows),
                              causal=causal, window=window, lse=lse, status=status)
    D.dflash_status_check(status)
    k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    ref = O.attention(qkv[:n, :hq], [k[st[b]:st[b + 1]] for b in range(len(rows))],
                      [v[st[b]:st[b + 1]] for b in range(len(rows))], st, rows, causal, window, d ** -0.5,
                      dtype == "bf16")
    check_attention(out, lse, ref, n)
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [math.nan, math.inf, -math.inf])
def test_hidden_keys_never_reach_a_row(dtype, bits):
    """K and V of position 150 are not finite: rows at 0 .. 149 do not see it and stay as they were."""
    D = lib()
    g = torch.Generator().manual_seed(3)
    n, hq, hkv, d = 200, 4, 2, 64
    q = torch.randn((n, hq, d), generator=g).to(DT[dtype])
    k = torch.randn((n, hkv, d), generator=g).to(DT[dtype])
    v = torch.randn((n, hkv, d), generator=g).to(DT[dtype])
    ref = O.attention(q, [k], [v], [0, n], [n], True, 0, d ** -0.5, dtype == "bf16")
    v[150, :, 3] = bits
    k[150, :, 5] = bits
    out = torch.empty((n, hq, d), dtype=DT[dtype], device="cuda")
    lse = torch.empty((n, hq), device="cuda")
    D.dflash_prompt_attention(q.cuda(), k.cuda(), v.cuda(), i32([0, n]), out, max_rows=n, lse=lse)
    check_attention(out[:150], lse[:150], tuple(x[:150] for x in ref), 150)
    if math.isnan(bits):   # ... and who sees it answers NaN
        assert bool(torch.isnan(out[150:, :, 3]).all())
    # behind the window it does not reach a row either
    D.dflash_prompt_attention(q.cuda(), k.cuda(), v.cuda(), i32([0, n]), out, max_rows=n, lse=lse, window=20)
    v2, k2 = v.clone(), k.clone()
    v2[150, :, 3], k2[150, :, 5] = 0, 0
    ref = O.attention(q, [k2], [v2], [0, n], [n], True, 20, d ** -0.5, dtype == "bf16")
    check_attention(out[170:], lse[170:], tuple(x[170:] for x in ref), 30)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,lens,hq", [([16], [3000], 4), ([1, 5], [900, 2000], 8), ([200, 90], [900, 700], 4),
                                          ([3] * 20, [1000 + 13 * b for b in range(20)], 8)])
def test_hidden_values_that_are_not_finite_in_every_layout_of_the_work(dtype, rows, lens, hq):
    """A window of 100 and K and V that are not finite outside it and behind the block's first row, in calls
    that run as a cluster, as ranges and as whole items: what a row does not see never reaches it."""
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=3)
    kp, vp = B.appended()
    for b, (n, L) in enumerate(zip(rows, lens)):
        for p in list(range(0, L - n - 100)) + ([L - 1] if n > 1 else []):
            pg, sl = int(B.table[b, p // 16]), p % 16
            vp[pg, sl, :, p % 64], kp[pg, sl, :, (p + 1) % 64] = (math.nan, math.inf)[p % 2], (math.inf, math.nan)[p % 2]
    B.kp, B.vp = kp, vp
    ref = O.attention(B.q[:B.starts[-1]], O.gather(kp.nan_to_num(0, 0, 0), lens, B.table),
                      O.gather(vp.nan_to_num(0, 0, 0), lens, B.table), B.starts, lens, True, 100, 0.125, dtype == "bf16")
    out, lse, _, _ = run_paged(B, True, 100, append=False)
    for b, n in enumerate(rows):   # the last row of a block of several sees the last key: not finite
        sl = slice(B.starts[b], B.starts[b + 1] - (1 if n > 1 else 0))
        check_attention(out[sl], lse[sl], tuple(x[sl] for x in ref), sl.stop - sl.start)
        if n > 1:
            assert not bool(torch.isfinite(out[B.starts[b + 1] - 1]).all())


@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 24, 1), ("bf16", 128, 1), ("bf16", 100, 2), ("f32", 24, 1)])
@pytest.mark.parametrize("rows,lens", [([1, 2], [200, 150]), ([7, 30], [77, 300])])
def test_wide_groups(dtype, hq, hkv, rows, lens):
    B = Batch(dtype, hq, hkv, 64, 32, rows, lens, seed=hq)
    out, lse, _, _ = run_paged(B, True, 0)
    check_attention(out, lse, ref_paged(B, True, 0), B.starts[-1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_beyond_two_to_the_31_elements(dtype):
    """Pages whose offsets pass 32 bits in elements."""
    D = lib()
    hkv, d, page, n_pages = 8, 128, 1024, 2100           # 2.2e9 elements each of K and V
    kp = torch.empty((n_pages, page, hkv, d), dtype=DT[dtype], device="cuda")
    vp = torch.empty_like(kp)
    g = torch.Generator().manual_seed(0)
    rows, lens, ids = [3, 1], [1500, 700], [[2099, 2090], [2080, 0]]
    table, starts = torch.tensor(ids, dtype=torch.int32), starts_of(rows)
    seq = [[torch.randn((L, hkv, d), generator=g).to(DT[dtype]) for L in lens] for _ in range(2)]
    for b, L in enumerate(lens):
        for j in range((L + page - 1) // page):
            m = min(page, L - j * page)
            kp[ids[b][j], :m], vp[ids[b][j], :m] = (x[b][j * page:j * page + m].cuda() for x in seq)
    new = [torch.cat([x[b][L - n:] for b, (n, L) in enumerate(zip(rows, lens))]).cuda() for x in seq]
    for b, (n, L) in enumerate(zip(rows, lens)):          # the new rows come back through the append
        kp[ids[b][(L - 1) // page], (L - n) % page:(L - 1) % page + 1] = 0
    q = torch.randn((4, 16, d), generator=g).to(DT[dtype])
    out, lse = torch.empty((4, 16, d), dtype=DT[dtype], device="cuda"), torch.empty((4, 16), device="cuda")
    args = (i32(starts), i32(lens), table.cuda())
    D.dflash_kv_append(*new, kp, vp, *args)
    D.dflash_paged_attention(q.cuda(), kp, vp, *args, out, max_rows=3, lse=lse)
    ref = O.attention(q, *seq, starts, lens, True, 0, d ** -0.5, dtype == "bf16")
    check_attention(out, lse, ref, 4)


def test_tensors_the_library_cannot_take_are_refused():
    D = lib()
    q = torch.zeros((4, 4, 64), device="cuda")
    kv = torch.zeros((4, 2, 64), device="cuda")
    out, st = torch.zeros_like(q), i32([0, 4])
    ok = lambda **k: D.dflash_prompt_attention(k.get("q", q), k.get("k", kv), k.get("v", kv), st, k.get("out", out), 4)
    ok()
    wide = torch.zeros((4, 4, 65), device="cuda")
    for bad in (dict(q=wide[..., 1:]), dict(out=wide[..., :64]), dict(k=kv[:1].expand(4, 2, 64)),
                dict(q=q.transpose(0, 2).contiguous().transpose(0, 2)), dict(out=q)):
        with pytest.raises((ValueError, D.DFlashError)):
            ok(**bad)
    with pytest.raises(ValueError):
        ok(k=kv.bfloat16(), v=kv.bfloat16())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_graphs_replayed_at_once(dtype):
    """Two captured calls (without a call before the capture) on two streams, each with its own workspace."""
    D = lib()
    Bs = [Batch(dtype, 8, 2, 128, 16, [6, 1], [2500 + 100 * i, 90], seed=i, tail=0) for i in range(2)]
    refs = [ref_paged(B, True, 0) for B in Bs]
    state, graphs = [], []
    for B in Bs:
        kp, vp = (x.cuda() for x in B.appended())
        q, st, ln, tb = B.q.cuda(), i32(B.starts), i32(B.lens), B.table.cuda()
        o, l = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        need = D.dflash_attention_workspace(q, o, st, ln, tb, 6, 2700, kp, vp)
        ws = torch.empty(max(need, 32), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            D.dflash_paged_attention(q, kp, vp, st, ln, tb, o, 6, max_len=2700, lse=l, workspace=ws)
        state.append((kp, vp, q, st, ln, tb, o, l, ws))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in Bs]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for x, r in zip(state, refs):
        check_attention(x[6], x[7], r, 7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_token_at_a_time_agrees_with_the_block(dtype):
    """The verified block's rows and the same tokens one by one."""
    B = Batch(dtype, 8, 2, 128, 16, [8], [300], seed=9, tail=0)
    ref = ref_paged(B, True, 0)
    out, lse, kp, vp = run_paged(B, True, 0)
    check_attention(out, lse, ref, 8)
    D = lib()
    one = torch.empty((1, 8, 128), dtype=B.dt, device="cuda")
    l1 = torch.empty((1, 8), device="cuda")
    for i in range(8):
        D.dflash_paged_attention(B.q[i:i + 1].cuda(), kp, vp, i32([0, 1]), i32([293 + i]), B.table.cuda(), one,
                                 max_rows=1, lse=l1)
        check_attention(one, l1, tuple(x[i:i + 1] for x in ref), 1)
        if dtype == "f32":   # the CUDA-core path's rows do not depend on the rows beside them
            assert torch.equal(one[0], out[i])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_sequences_and_pages_are_skipped_and_reported(dtype):
    D = lib()
    B = Batch(dtype, 4, 2, 64, 16, [4, 4, 4], [40, 60, 20], tail=0)
    ref = ref_paged(B, True, 0)
    kp0, vp0 = B.appended()
    q = B.q.cuda()

    def call(lens, table, max_rows=4, starts=B.starts):
        kp, vp = kp0.cuda(), vp0.cuda()
        st = i32([0])
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        D.dflash_paged_attention(q, kp, vp, i32(starts), i32(lens), table.cuda(), out, max_rows=max_rows, lse=lse,
                                 status=st)
        bits = int(st.item())
        if bits:
            with pytest.raises(D.DFlashError) as e:
                D.dflash_status_check(st)
            assert e.value.status == D.DFLASH_ERR_DEVICE
            D.dflash_status_check(st)   # cleared
        return out, lse, bits

    for lens in ([40, 3, 20], [40, -1, 20], [40, 1 << 29, 20], [40, 65, 20]):   # below its rows, or past the table
        out, lse, bits = call(lens, B.table)
        assert bits == 2 and bool((out[4:8] == 7).all())
        for sl in (slice(0, 4), slice(8, 12)):
            check_attention(out[sl], lse[sl], tuple(x[sl] for x in ref), 4)
    out, lse, bits = call(B.lens, B.table, starts=[0, 4, 13, 12])     # rows past the arrays, then a negative count
    assert bits == 2 and bool((out[4:] == 7).all())
    check_attention(out[:4], lse[:4], tuple(x[:4] for x in ref), 4)
    bad = B.table.clone()
    bad[0, 1] = kp0.shape[0]
    bad[2, 0] = -1
    out, lse, bits = call(B.lens, bad)
    assert bits == 4 and bool(torch.isfinite(out).all())
    check_attention(out[4:8], lse[4:8], tuple(x[4:8] for x in ref), 4)
    # a page that is not there holds zeros
    z = O.gather(kp0, B.lens, B.table)[0], O.gather(vp0, B.lens, B.table)[0]
    for x in z:
        x[16:32] = 0
    r0 = O.attention(B.q[:4], [z[0]], [z[1]], [0, 4], [40], True, 0, 64 ** -0.5, dtype == "bf16")
    check_attention(out[:4], lse[:4], r0, 4)
    # an append to it is dropped
    kp, vp = kp0.cuda(), vp0.cuda()
    st = i32([0])
    bad = B.table.clone()
    bad[1, 3] = -1
    D.dflash_kv_append(B.v.cuda(), B.k.cuda(), kp, vp, i32(B.starts), i32(B.lens), bad.cuda(), status=st)
    assert int(st.item()) == 4
    want = kp0.clone()
    for b in (0, 2):
        for i in range(4):
            p = B.lens[b] - 4 + i
            want[int(B.table[b, p // 16]), p % 16] = B.v[B.starts[b] + i]
    assert same_bits(kp.cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_steps_follow_the_lengths_on_the_device(dtype):
    """One captured append + attention, replayed as the sequences grow."""
    D = lib()
    hq, hkv, d, page, steps = 8, 2, 64, 16, 5
    B = Batch(dtype, hq, hkv, d, page, [1, 1, 1], [30, 126, 255], tail=0, spare=0)
    table = torch.arange(3 * 20, dtype=torch.int32).reshape(3, 20)
    g = torch.Generator().manual_seed(1)
    kp = torch.randn((60, page, hkv, d), generator=g).to(B.dt)
    vp = torch.randn((60, page, hkv, d), generator=g).to(B.dt)
    dk, dv, dt_ = kp.cuda(), vp.cuda(), table.cuda()
    q, k, v = (torch.zeros((3, h, d), dtype=B.dt, device="cuda") for h in (hq, hkv, hkv))
    starts, lens = i32([0, 1, 2, 3]), i32(B.lens)
    out, lse = torch.empty_like(q), torch.empty((3, hq), device="cuda")

    def step():
        D.dflash_kv_append(k, v, dk, dv, starts, lens, dt_)
        D.dflash_paged_attention(q, dk, dv, starts, lens, dt_, out, max_rows=1, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()   # warm-up; its append is repeated by the first replay
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        L = [x + i for x in B.lens]
        hq_, hk, hv = (torch.randn((3, h, d), generator=g).to(B.dt) for h in (hq, hkv, hkv))
        q.copy_(hq_), k.copy_(hk), v.copy_(hv), lens.copy_(i32(L))
        graph.replay()
        torch.cuda.synchronize()
        kp = O.append(kp, hk, [0, 1, 2, 3], L, table)
        vp = O.append(vp, hv, [0, 1, 2, 3], L, table)
        ref = O.attention(hq_, O.gather(kp, L, table), O.gather(vp, L, table), [0, 1, 2, 3], L, True, 0, d ** -0.5,
                          dtype == "bf16")
        check_attention(out, lse, ref, 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_on_two_streams_with_their_own_workspaces(dtype):
    D = lib()
    Bs = [Batch(dtype, 8, 2, 128, 16, [4, 1], [600 + 50 * i, 90], seed=i, tail=0) for i in range(2)]
    refs = [ref_paged(B, True, 0) for B in Bs]
    pages = [tuple(x.cuda() for x in B.appended()) for B in Bs]
    args = [(B.q.cuda(), i32(B.starts), i32(B.lens), B.table.cuda()) for B in Bs]
    outs = [(torch.empty_like(a[0]), torch.empty(a[0].shape[:2], device="cuda")) for a in args]
    streams = [torch.cuda.Stream() for _ in Bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (kp, vp), (q, st, ln, tb), (o, l) in zip(streams, pages, args, outs):
            D.dflash_paged_attention(q, kp, vp, st, ln, tb, o, max_rows=4, lse=l, stream=s)
    torch.cuda.synchronize()
    for (o, l), r in zip(outs, refs):
        check_attention(o, l, r, 5)


def test_results_do_not_change_from_run_to_run():
    B = Batch("bf16", 8, 2, 128, 16, [16, 1, 7], [3000, 900, 70], tail=0)
    first = run_paged(B, True, 0)
    for _ in range(5):
        again = run_paged(B, True, 0)
        assert same_bits(first[0].cpu(), again[0].cpu()) and torch.equal(first[1], again[1])


# ---------------------------------------------------------------------------
# token log probabilities
# ---------------------------------------------------------------------------
def run_logprobs(x, tokens, top, T, status=None):
    D = lib()
    R = x.shape[0]
    lp, ent = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    ids = torch.empty((R, top), dtype=torch.int32, device="cuda") if top else None
    tlp = torch.empty((R, top), device="cuda") if top else None
    D.dflash_token_logprobs(x, tokens, lp, ent, ids, tlp, temperature=T, status=status)
    torch.cuda.synchronize()
    return lp, ent, ids, tlp


def check_logprobs(got, ref):
    lp, ent, ids, tlp = got
    rlp, rent, rids, rtlp, t_lp, t_ent, t_top = ref

    def close(a, b, t):
        a = a.double().cpu()
        assert bool(((a == b) | ((a - b).abs() <= t)).all()), float((a - b).abs().max())
    close(lp, rlp, t_lp)
    close(ent, rent, t_ent)
    if ids is not None:
        assert torch.equal(ids.cpu().long(), rids)
        close(tlp, rtlp, t_top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V,top,T", [(1, 1, 1, 1.0), (3, 32, 32, 0.7), (16, 1000, 5, 1.0), (5, 32001, 20, 1.3),
                                          (2, 151936, 20, 1.0), (400, 999, 3, 0.5), (1, 100352, 0, 1.0),
                                          (700, 4099, 32, 1.0), (7, 50000, 1, 2.0)])
def test_token_logprobs(dtype, rows, V, top, T):
    g = torch.Generator().manual_seed(V + rows)
    x = (torch.randn((rows, V), generator=g) * 3).to(DT[dtype])   # bf16 rows hold many ties
    tok = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32)
    tok[0] = int(x[0].double().argmax())
    check_logprobs(run_logprobs(x.cuda(), tok.cuda(), top, T), O.logprobs(x, tok, top, T))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["ascending", "descending", "equal", "spikes"])
def test_token_logprobs_of_ordered_rows(dtype, order):
    """Rows whose order is the worst for a running selection, and rows of ties alone."""
    V, g = 20011, torch.Generator().manual_seed(2)
    x = torch.sort(torch.randn((3, V), generator=g) * 4, dim=1, descending=order == "descending").values
    if order == "equal":
        x = torch.full((3, V), -1.25)
    if order == "spikes":   # a top entry in the last place of every stretch of 512
        x[:, 511::512] = 30 + torch.arange(V // 512)[None, :] * 0.25
    x = x.to(DT[dtype])
    tok = torch.tensor([0, V - 1, 77], dtype=torch.int32)
    check_logprobs(run_logprobs(x.cuda(), tok.cuda(), 32, 1.0), O.logprobs(x, tok, 32, 1.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_of_padded_rows_masks_and_missing_tokens(dtype):
    D = lib()
    V, pad = 1501, 1544
    g = torch.Generator().manual_seed(4)
    wide = torch.randn((6, pad), generator=g).to(DT[dtype])
    x = wide[:, :V]
    x[1, 5:] = -math.inf          # five entries left: banned ones follow by id with -inf
    x[2, :-1] = -math.inf         # one entry left
    x[3, ::2] = torch.finfo(DT[dtype]).min
    wide[:, V:] = 100.0           # behind the vocabulary
    tok = torch.tensor([3, 700, V - 1, 1, -1, V], dtype=torch.int32)
    ref = list(O.logprobs(x, tok.clamp(max=V - 1), 8, 1.0))
    st = i32([0])
    dev = wide.cuda()[:, :V]
    lp, ent, ids, tlp = run_logprobs(dev, tok.cuda(), 8, 1.0, status=st)
    assert int(st.item()) == 1 and bool(torch.isnan(lp[5]))   # an id outside the vocabulary
    with pytest.raises(D.DFlashError):
        D.dflash_status_check(st)
    lp[5] = float(ref[0][5])
    check_logprobs((lp, ent, ids, tlp), ref)
    assert float(lp[4]) == 0.0 and float(ent[2]) == 0.0 and math.isinf(float(lp[1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_of_rows_without_a_distribution(dtype):
    x = torch.zeros((4, 3000), dtype=DT[dtype])
    x[0, 1234] = math.nan
    x[1] = -math.inf
    x[2] = math.nan
    x[3, 7] = math.inf
    lp, ent, ids, tlp = run_logprobs(x.cuda(), i32([5, 5, 5, 9]), 4, 1.0)
    assert bool(torch.isnan(lp).all()) and bool(torch.isnan(ent).all()) and bool(torch.isnan(tlp).all())
    assert ids.cpu().tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [-1] * 4, [7, 0, 1, 2]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 0.25, 4.0])
def test_token_logprobs_of_rows_masked_with_the_lowest_value(dtype, T):
    """Entries at the type's lowest value have probability zero and no share in the entropy, wherever they lie
    (their distance to the maximum is past the fp32 range once it is scaled)."""
    V, low = 40000, torch.finfo(DT[dtype]).min
    x = torch.randn((5, V), generator=torch.Generator().manual_seed(8)).to(DT[dtype])
    x[0, :30000] = low            # whole batches of a thread in front of the others,
    x[1, 9000:] = low             # behind them,
    x[2, ::2] = low               # between them,
    x[3, :] = low                 # one entry left,
    x[3, 31234] = 2.5
    x[4, :] = low                 # and none: a uniform row
    tok = torch.tensor([39999, 5, 33, 31234, -1], dtype=torch.int32)
    if T >= 1:                    # (below, a masked token's log probability leaves fp32)
        tok[2] = 34
    got = run_logprobs(x.cuda(), tok.cuda(), 5, T)
    ref = O.logprobs(x, tok, 5, T)
    check_logprobs(tuple(a[:3] for a in got), tuple(a[:3] for a in ref))
    lp, ent, ids, tlp = (a.cpu() for a in got)
    # one entry left: exact; the masked ones behind it, in the order of their ids
    assert float(lp[3]) == 0 and float(ent[3]) == 0 and ids[3].tolist() == [31234, 0, 1, 2, 3]
    assert float(tlp[3, 0]) == 0 and (T < 1 or bool(torch.isfinite(tlp[3]).all()))
    # a uniform row: sums of ones are exact, log2 and the product with ln 2 round (2 + 1 + 1 half steps at 11)
    tol = 4 * 2.0 ** -24 * 16
    assert abs(float(ent[4]) - math.log(V)) <= tol and float(lp[4]) == 0 and ids[4].tolist() == [0, 1, 2, 3, 4]
    assert float((tlp[4] + math.log(V)).abs().max()) <= tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_at_the_smallest_temperature(dtype):
    """1 / T close to the end of the fp32 range: scaled distances overflow, the distribution is its maximum's."""
    V = 20000
    x = torch.randn((3, V), generator=torch.Generator().manual_seed(9)).to(DT[dtype])
    x[:, 777] = 8.0
    tok = torch.tensor([777, -1, 777], dtype=torch.int32)
    lp, ent, ids, tlp = run_logprobs(x.cuda(), tok.cuda(), 1, 1e-38)
    assert lp.tolist() == [0, 0, 0] and ent.tolist() == [0, 0, 0] and tlp.flatten().tolist() == [0, 0, 0]
    assert ids.flatten().tolist() == [777] * 3


@pytest.mark.parametrize("heads", [1, 4])
def test_a_value_that_is_not_finite_in_the_last_tile_of_an_item(heads):
    """Items of two row tiles whose second one alone reaches the last key tile, which holds a NaN that only the
    sequence's last token sees: every other row, those of the first tile among them, is complete and right."""
    D = lib()
    n, d, seqs, hq, hkv = 256, 64, 40, heads, heads
    g = torch.Generator().manual_seed(12)
    t = n * seqs
    q, k, v = (torch.randn((t, h, d), generator=g).to(torch.bfloat16) for h in (hq, hkv, hkv))
    starts = [b * n for b in range(seqs + 1)]
    split = lambda x: [x[b * n:(b + 1) * n] for b in range(seqs)]
    ref = O.attention(q, split(k), split(v), starts, [n] * seqs, True, 0, d ** -0.5, True)
    v[n - 1::n, :, 7] = math.nan
    seen = torch.ones(t, dtype=torch.bool)
    seen[n - 1::n] = False
    dev = q.cuda(), k.cuda(), v.cuda()
    for _ in range(5):
        out, lse = torch.full((t, hq, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.empty((t, hq), device="cuda")
        D.dflash_prompt_attention(*dev, i32(starts), out, max_rows=n, lse=lse)
        check_attention(out.cpu()[seen], lse.cpu()[seen], tuple(x[seen] for x in ref), int(seen.sum()))
        assert bool(torch.isnan(out[n - 1::n, :, 7]).all()) and bool(torch.isfinite(out[n - 1::n, :, 8:]).all())


def test_a_value_that_is_not_finite_in_the_last_tile_of_a_paged_item():
    """The same with 8 heads a group: 32 new tokens over 112 cached ones, the first 16 of them end with a tile."""
    B = Batch("bf16", 8, 1, 128, 16, [32] * 40, [144] * 40, seed=5)
    ref = ref_paged(B, True, 0)
    B.v[31:32 * 40:32, :, 7] = math.nan
    seen = torch.ones(32 * 40, dtype=torch.bool)
    seen[31::32] = False
    for _ in range(5):
        out, lse, _, _ = run_paged(B, True, 0)
        check_attention(out[:1280].cpu()[seen], lse[:1280].cpu()[seen], tuple(x[seen] for x in ref), int(seen.sum()))
        assert bool(torch.isnan(out[31:1280:32, :, 7]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,lens", [(4, 40), (200, 300)])
def test_starts_that_decrease_are_reported(dtype, rows, lens):
    """64 sequences whose starts go back and forth: each of the good halves alone would be in bounds, together
    they are more rows than the arrays hold."""
    D = lib()
    q = torch.randn((rows, 4, 64), device="cuda").to(DT[dtype])
    pages = torch.zeros((20, 16, 1, 64), dtype=DT[dtype], device="cuda")
    out, st = torch.full_like(q, 7.0), i32([0])
    starts, table = i32([0, rows] * 32 + [0]), i32(list(range(20))).repeat(64, 1)
    D.dflash_paged_attention(q, pages, pages.clone(), starts, i32([lens] * 64), table, out, max_rows=rows, status=st)
    assert int(st.item()) == 2 and bool(((out == 7) | (out == 0)).all())
    with pytest.raises(D.DFlashError):
        D.dflash_status_check(st)


@pytest.mark.parametrize("d", [64, 100])
def test_fp32_rows_do_not_depend_on_the_bounds(d):
    """Splits that meet in a cluster (up to 2048 tokens) and in the workspace (a larger max_len): the same bits;
    and so for a block alone and beside a longer one (fewer and more rows to a CTA)."""
    B = Batch("f32", 4, 2, d, 16, [1, 4, 30], [2000, 900, 300], seed=21)
    B.table = torch.nn.functional.pad(B.table, (0, 200), value=-7)
    n = B.starts[-1]
    out, lse, _, _ = run_paged(B, True, 0, max_len=2000)
    check_attention(out, lse, ref_paged(B, True, 0), n)
    far, far_lse, _, _ = run_paged(B, True, 0, max_len=5000)
    assert same_bits(out[:n], far[:n]) and torch.equal(lse[:n], far_lse[:n])
    B.rows, B.lens, B.starts = B.rows[:2], B.lens[:2], B.starts[:3]
    B.table = B.table[:2].contiguous()
    few, few_lse, _, _ = run_paged(B, True, 0, max_len=2000)
    assert same_bits(out[:5], few[:5]) and torch.equal(lse[:5], few_lse[:5])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [[2, 4, 1], [90, 1, 70]])
def test_rows_in_front_of_the_first_sequence_are_left_alone(dtype, rows):
    """starts[0] > 0: those rows belong to no sequence, and nothing is wrong with that."""
    B = Batch(dtype, 4, 2, 64, 16, rows, [n + 40 for n in rows], seed=13)
    ref = ref_paged(B, True, 0)
    kp, vp = B.appended()
    n, pad = B.starts[-1], 3
    B.q, B.k, B.v = (torch.cat([torch.full_like(x[:pad], math.nan), x]) for x in (B.q, B.k, B.v))
    B.starts = [s + pad for s in B.starts]
    st = i32([0])
    out, lse, gk, gv = run_paged(B, True, 0, status=st)
    assert int(st.item()) == 0 and same_bits(gk.cpu(), kp) and same_bits(gv.cpu(), vp)
    check_attention(out[pad:], lse[pad:], ref, n)
    assert bool((out[:pad] == 7).all()) and bool((lse[:pad] == 7).all()) and bool((out[pad + n:] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,lens", [([b % 3 for b in range(75)], [5 + 31 * b for b in range(75)]),
                                       ([(37 * b) % 120 for b in range(70)], [130 + 3 * b for b in range(70)])])
def test_batches_of_more_than_32_sequences(dtype, rows, lens):
    """Sequences without rows among them, lengths from one key tile to many."""
    B = Batch(dtype, 4, 1, 64, 32, rows, lens, seed=17)
    st = i32([0])
    out, lse, _, _ = run_paged(B, True, 0, status=st)
    assert int(st.item()) == 0
    check_attention(out, lse, ref_paged(B, True, 0), B.starts[-1])
    assert bool((out[B.starts[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_largest_batch(dtype):
    """32768 sequences of one token over a page each."""
    D = lib()
    n, d, L = 32768, 64, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((n, 1, d), device="cuda", generator=g).to(DT[dtype])
    kp, vp = (torch.randn((n, 8, 1, d), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    out, st = torch.empty_like(q), i32([0])
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    D.dflash_paged_attention(q, kp, vp, torch.arange(n + 1, dtype=torch.int32, device="cuda"),
                             torch.full((n,), L, dtype=torch.int32, device="cuda"), table, out, max_rows=1, status=st)
    assert int(st.item()) == 0
    s = torch.einsum("nd,nld->nl", q[:, 0].double(), kp[:, :, 0].double()) * d ** -0.5
    p = torch.softmax(s, 1)
    ref = torch.einsum("nl,nld->nd", p, vp[:, :, 0].double())
    # fp32: a few steps of the sums; bf16: P and the output round, half a step each of |p| |v| summed and of the result
    av = torch.einsum("nl,nld->nd", p, vp[:, :, 0].double().abs())
    tol = av * 2.0 ** -18 + (av * 2.0 ** -8 + ref.abs() * 2.0 ** -8 if dtype == "bf16" else 0)
    assert bool(((out[:, 0].double() - ref).abs() <= tol).all())
