"""The compressed cache's operators without a GPU: refusals of the library and of the
binding before any device work, the rotary table, and the oracle's own arithmetic."""
import ctypes as C
import math

import pytest
import torch

import block_diffusion_speculative_flush_gb300 as D
from block_diffusion_speculative_flush_gb300 import _abi
from oracle import kv8_oracle as O

INVALID, SHAPE = _abi.DFLASH_ERR_INVALID_ARG, _abi.DFLASH_ERR_SHAPE
BASE = 4096   # stands for an aligned device pointer; refused calls never look at it


def make(cls, base, kw):
    f = dict(base)
    f.update(kw)
    return cls(**f)


def pages(**kw):
    return make(_abi.dflash_kv8_pages, dict(n_kv_heads=2, head_dim=64, page_size=16, reserved=0, n_pages=10, k=BASE, v=BASE,
                                            page_stride=2048, slot_stride=128, head_stride=64, k_scale=BASE, v_scale=BASE,
                                            scale_page_stride=2, scale_head_stride=1), kw)


def batch(**kw):
    return make(_abi.dflash_ragged, dict(batch=2, total_rows=8, max_rows=4, max_len=100, starts=BASE, lens=BASE, table=BASE,
                                         table_width=7, table_stride=7, status=None), kw)


def heads(data=BASE, row=256, head=64):
    return _abi.dflash_heads(data, row, head)


def attention(**kw):
    return make(_abi.dflash_attention, dict(dtype=1, n_q_heads=4, n_kv_heads=2, head_dim=64, causal=1, window=0, scale=0.125,
                                            q=heads(), out=heads(2 * BASE), lse=None, workspace=None, workspace_bytes=0), kw)


@pytest.mark.parametrize("bad,code", [
    (dict(n_kv_heads=0), SHAPE), (dict(n_kv_heads=1025), SHAPE), (dict(head_dim=72), SHAPE), (dict(head_dim=144), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=2048), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE), (dict(reserved=1), INVALID), (dict(k=None), INVALID),
    (dict(v=BASE + 8), INVALID), (dict(page_stride=2040), INVALID), (dict(slot_stride=48), INVALID),
    (dict(head_stride=32), INVALID), (dict(slot_stride=-128), INVALID), (dict(k_scale=None), INVALID),
    (dict(v_scale=BASE + 2), INVALID), (dict(scale_page_stride=0), INVALID), (dict(scale_head_stride=-1), INVALID)])
def test_bad_pages_are_refused(bad, code):
    p, b, h, a = pages(**bad), batch(), heads(), attention()
    assert D.lib.dflash_kv8_append(C.byref(p), C.byref(b), 1, C.byref(h), C.byref(h), None) == code
    assert D.lib.dflash_kv8_attention(C.byref(a), C.byref(b), C.byref(p), None) == code
    assert D.lib.dflash_kv8_attention_workspace(C.byref(a), C.byref(b), C.byref(p)) == code
    assert D.lib.dflash_last_error()


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(batch=32769), dict(total_rows=-1), dict(total_rows=(1 << 30) + 1), dict(max_rows=0),
    dict(max_rows=(1 << 24) + 1), dict(starts=None), dict(lens=None), dict(table=None), dict(max_len=0),
    dict(max_len=(1 << 30) + 1), dict(table_width=0), dict(table_stride=6)])
def test_bad_batches_are_refused(bad):
    p, b, h, a = pages(), batch(**bad), heads(), attention()
    assert D.lib.dflash_kv8_append(C.byref(p), C.byref(b), 1, C.byref(h), C.byref(h), None) == INVALID
    assert D.lib.dflash_kv8_attention(C.byref(a), C.byref(b), C.byref(p), None) == INVALID


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=2), INVALID), (dict(n_q_heads=3), SHAPE), (dict(n_q_heads=0), SHAPE), (dict(n_q_heads=258), SHAPE),
    (dict(head_dim=128), SHAPE), (dict(n_kv_heads=4), SHAPE), (dict(causal=2), INVALID), (dict(window=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(q=heads(None)), INVALID), (dict(q=heads(BASE + 8)), INVALID), (dict(q=heads(row=250)), INVALID),
    (dict(q=heads(head=32)), INVALID), (dict(out=heads(BASE)), INVALID), (dict(out=heads(None)), INVALID)])
def test_bad_attention_is_refused(bad, code):
    p, b, a = pages(), batch(), attention(**bad)
    assert D.lib.dflash_kv8_attention(C.byref(a), C.byref(b), C.byref(p), None) == code


def test_rows_of_nothing_need_no_device():
    p, b, h, a = pages(), batch(total_rows=0), heads(None), attention(q=heads(None), out=heads(None))
    assert D.lib.dflash_kv8_append(C.byref(p), C.byref(b), 1, C.byref(h), C.byref(h), None) == 0
    assert D.lib.dflash_kv8_attention(C.byref(a), C.byref(b), C.byref(p), None) == 0
    assert D.lib.dflash_kv8_append(C.byref(p), C.byref(b), 2, C.byref(h), C.byref(h), None) == INVALID


def config(**kw):
    return make(_abi.dflash_rope_config, dict(rot_dim=64, offset=0, layout=0, scaling=0, theta=10000.0, factor=4.0,
                                              original_len=4096.0, low=1.0, high=4.0, amplitude=0.0), kw)


@pytest.mark.parametrize("bad,code", [
    (dict(rot_dim=0), SHAPE), (dict(rot_dim=63), SHAPE), (dict(rot_dim=258), SHAPE), (dict(offset=-2), SHAPE),
    (dict(offset=1), SHAPE), (dict(offset=194), SHAPE), (dict(layout=2), INVALID), (dict(scaling=5), INVALID),
    (dict(scaling=-1), INVALID), (dict(theta=1.0), INVALID), (dict(theta=math.inf), INVALID), (dict(theta=math.nan), INVALID),
    (dict(amplitude=-1.0), INVALID), (dict(amplitude=1e300), INVALID), (dict(scaling=1, factor=0.0), INVALID),
    (dict(scaling=2, factor=math.nan), INVALID), (dict(scaling=2, rot_dim=2), SHAPE),
    (dict(scaling=2, factor=1e-9), INVALID), (dict(scaling=3, low=4.0), INVALID), (dict(scaling=3, original_len=0.0), INVALID),
    (dict(scaling=4, factor=0.5), INVALID), (dict(scaling=4, low=0.0), INVALID)])
def test_bad_rope_configs_are_refused(bad, code):
    t = _abi.dflash_rope_table()
    assert D.lib.dflash_rope_init(C.byref(config(**bad)), C.byref(t)) == code
    assert D.lib.dflash_rope_init(None, C.byref(t)) == INVALID


@pytest.mark.parametrize("scaling", [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=3.0),
                                     dict(kind="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
                                     dict(kind="yarn", factor=4.0, original_len=4096.0, low=1.0, high=32.0)])
@pytest.mark.parametrize("rot", [4, 64, 256])
def test_the_rope_table_holds_the_frequencies(scaling, rot):
    t = D.dflash_rope_table(rot, 500000.0, scaling=scaling)
    f, amp = O.rope_freqs(rot, 500000.0, scaling)
    got = torch.tensor([t.table.turns[i] / 2.0 ** 64 for i in range(rot // 2)], dtype=torch.float64)
    # a power and up to six products and sums in fp64
    assert bool(((got - f / (2 * math.pi)).abs() <= 2.0 ** -50 * f + 2.0 ** -64).all())
    assert abs(t.amplitude - amp) <= 2.0 ** -23 * amp
    assert all(t.table.turns[i] == 0 for i in range(rot // 2, 128))


def test_rope_options_of_the_binding():
    for bad in (dict(layout="other"), dict(scaling=dict(factor=2.0)), dict(scaling=dict(kind="linear")),
                dict(scaling=dict(kind="linear", factor=2.0, low=1.0)), dict(amplitude=0.0)):
        with pytest.raises(ValueError):
            D.dflash_rope_table(64, 10000.0, **bad)
    assert D.dflash_rope_table(64, 10000.0, amplitude=0.5).amplitude == 0.5


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=2), INVALID), (dict(head_dim=60), SHAPE), (dict(head_dim=32), SHAPE), (dict(head_dim=264), SHAPE),
    (dict(n_q_heads=-1), SHAPE), (dict(n_q_heads=0, n_k_heads=0), SHAPE), (dict(n_k_heads=1025), SHAPE),
    (dict(transpose=2), INVALID), (dict(q=heads(None)), INVALID), (dict(k=heads(BASE + 4)), INVALID),
    (dict(q_out=heads(row=32)), INVALID), (dict(q_out=heads(BASE, row=512)), INVALID)])
def test_bad_rope_calls_are_refused(bad, code):
    t = D.dflash_rope_table(64, 10000.0)
    a = make(_abi.dflash_rope_call, dict(dtype=1, head_dim=64, n_q_heads=4, n_k_heads=2, transpose=0, q=heads(), k=heads(),
                                         q_out=heads(2 * BASE), k_out=heads(3 * BASE)), bad)
    assert D.lib.dflash_rope(t.address, C.byref(batch()), C.byref(a), None) == code
    assert D.lib.dflash_rope(None, C.byref(batch()), C.byref(a), None) == INVALID
    assert D.lib.dflash_rope(t.address, C.byref(batch(starts=None)), C.byref(a), None) == INVALID
    ruined = _abi.dflash_rope_table.from_buffer_copy(t.table)
    ruined.rot_dim = 300
    good = make(_abi.dflash_rope_call, dict(dtype=1, head_dim=64, n_q_heads=4, n_k_heads=0, transpose=0, q=heads(), q_out=heads()), {})
    assert D.lib.dflash_rope(C.byref(ruined), C.byref(batch()), C.byref(good), None) == INVALID


def rows(**kw):
    return make(_abi.dflash_page_rows, dict(rows=3, width=4, stride=4, page_size=16, table=BASE, lens=2 * BASE), kw)


BAD_ROWS = [(dict(rows=0), INVALID), (dict(rows=32769), INVALID), (dict(width=0), INVALID), (dict(stride=3), INVALID),
            (dict(width=(1 << 20) + 1, stride=1 << 21), INVALID), (dict(page_size=12), SHAPE), (dict(page_size=4), SHAPE),
            (dict(page_size=2048), SHAPE), (dict(table=None), INVALID), (dict(lens=None), INVALID)]


@pytest.mark.parametrize("bad,code", BAD_ROWS)
def test_bad_rows_are_refused(bad, code):
    r, ok = C.byref(rows(**bad)), C.byref(rows(table=3 * BASE, lens=4 * BASE))
    assert D.lib.dflash_pages_reorder(BASE, 10, r, BASE, ok, None, None) == code
    assert D.lib.dflash_pages_reorder(BASE, 10, ok, BASE, r, None, None) == code
    assert D.lib.dflash_pages_resize(BASE, 10, r, BASE, None, 0, None, BASE, 1 << 20, None, None) == code
    assert D.lib.dflash_pages_compact(BASE, BASE, 10, r, ok, None, 0, None, BASE, 1 << 20, None, None) == code


def test_bad_pools_buffers_and_workspaces_are_refused():
    r, to = C.byref(rows()), C.byref(rows(table=3 * BASE, lens=4 * BASE))
    resize = lambda refs=BASE, n=10, new=BASE, bufs=None, nb=0, ws=BASE, size=1 << 20: D.lib.dflash_pages_resize(
        refs, n, r, new, bufs, nb, None, ws, size, None, None)
    assert resize(refs=None) == INVALID and resize(n=0) == SHAPE and resize(n=(1 << 30) + 1) == SHAPE
    assert resize(new=None) == INVALID and resize(new=2 * BASE) == INVALID
    assert resize(ws=None) == INVALID and resize(size=D.lib.dflash_pages_workspace(10, 3) - 1) == INVALID
    assert resize(nb=1) == INVALID and resize(nb=-1) == INVALID and resize(nb=4097) == INVALID
    for bad in ((0, 64, 64), (BASE + 2, 64, 64), (BASE, 62, 60), (BASE, 64, 62), (BASE, 60, 64), (BASE, 64, 0)):
        b = _abi.PACK_BUFFER(*bad)
        assert resize(bufs=b, nb=1) == INVALID
        assert D.lib.dflash_pages_copy(b, 1, 10, BASE, BASE, 1, None, None) == INVALID
    b = _abi.PACK_BUFFER(BASE, 64, 64)
    assert D.lib.dflash_pages_copy(b, 1, 0, BASE, BASE, 1, None, None) == SHAPE
    assert D.lib.dflash_pages_copy(b, 1, 10, None, BASE, 1, None, None) == INVALID
    assert D.lib.dflash_pages_copy(b, 1, 10, BASE, BASE, -1, None, None) == INVALID
    assert D.lib.dflash_pages_copy(b, 1, 10, None, None, 0, None, None) == 0
    assert D.lib.dflash_pages_reorder(BASE, 10, r, None, to, None, None) == INVALID
    assert D.lib.dflash_pages_reorder(BASE, 10, r, BASE, r, None, None) == INVALID
    assert D.lib.dflash_pages_reorder(BASE, 10, r, BASE, C.byref(rows(table=3 * BASE, lens=4 * BASE, page_size=32)), None, None) == SHAPE
    for bad in (dict(rows=4), dict(width=3), dict(page_size=32)):
        o = C.byref(rows(table=3 * BASE, **bad))
        assert D.lib.dflash_pages_compact(BASE, BASE, 10, r, o, None, 0, None, BASE, 1 << 20, None, None) == SHAPE
    assert D.lib.dflash_pages_compact(BASE, BASE, 10, r, C.byref(rows(stride=5)), None, 0, None, BASE, 1 << 20, None, None) == INVALID
    assert D.lib.dflash_pages_workspace(0, 1) == SHAPE and D.lib.dflash_pages_workspace(1, 0) == INVALID


def test_host_tensors_are_refused_by_the_binding():
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)
    i = lambda *s: z(*s, dtype=torch.int32)
    t = D.dflash_rope_table(16, 10000.0)
    for call in (lambda: D.dflash_rope(t, z(2, 1, 16), None, i(2), i(1)),
                 lambda: D.dflash_rope(t, None, None, i(2), i(1)),
                 lambda: D.dflash_kv8_append(z(1, 1, 16), z(1, 1, 16), z(2, 16, 1, 16, dtype=torch.uint8),
                                             z(2, 16, 1, 16, dtype=torch.uint8), z(2, 1), z(2, 1), i(2), i(1), i(1, 1)),
                 lambda: D.dflash_kv8_attention(z(1, 1, 16), z(2, 16, 1, 16, dtype=torch.uint8),
                                                z(2, 16, 1, 16, dtype=torch.uint8), z(2, 1), z(2, 1), i(2), i(1), i(1, 1),
                                                z(1, 1, 16), 1),
                 lambda: D.dflash_page_buffers([z(3, 4)]), lambda: D.dflash_page_buffers([]),
                 lambda: D.dflash_pages_reorder(i(3), i(1, 2), i(1), i(1), i(1, 2), i(1), 16),
                 lambda: D.dflash_pages_resize(i(3), i(1, 2), i(1), i(1), None, 16),
                 lambda: D.dflash_pages_compact(i(3), i(1, 2), i(1), i(3), i(1, 2), None, 16)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def test_the_scale_is_the_smallest_power_of_two():
    for most in (0.0, 1e-30, 0.5, 1.0, 1.75, 1.7500001, 447.9, 448.0, 448.1, 1e10, 3e38):
        s = O.needed_scale(most)
        assert most <= 448 * s or s == 2.0 ** 60
        assert s == 2.0 ** -60 or most > 448 * s / 2


def test_codes_are_the_nearest_ones():
    every = torch.arange(0x7F, dtype=torch.uint8).view(O.E4M3).double()      # 0 .. 448, ascending
    x = torch.linspace(-460, 460, 40001)
    v = O.encode(x).view(O.E4M3).double()
    at = torch.searchsorted(every, x.abs().double().clamp(max=448.0)).clamp(1, len(every) - 1)
    near = torch.minimum((every[at] - x.abs().clamp(max=448.0)).abs(), (every[at - 1] - x.abs().clamp(max=448.0)).abs())
    assert torch.equal((v.abs() - x.abs().clamp(max=448.0)).abs(), near)


def test_appending_one_by_one_and_at_once_hold_the_rows():
    """The codes may differ (a scale that grows rounds twice) by at most a step at the final scale."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn((20, 1, 16), generator=g) * torch.linspace(0.1, 9, 20)[:, None, None]
    tb = torch.tensor([[1, 0]], dtype=torch.int32)
    c, s = torch.zeros((2, 16, 1, 16), dtype=torch.uint8), torch.zeros((2, 1))
    at_once = O.append8(c, s, x, [0, 20], [20], tb)
    for i in range(20):
        c, s = O.append8(c, s, x[i:i + 1], [0, 1], [i + 1], tb)
    assert torch.equal(s, at_once[1])
    a, b = O.gather8(c, s, [20], tb)[0], O.gather8(*at_once, [20], tb)[0]
    step = (x.double().abs() * 2.0 ** -4).clamp(min=float(s.max()) * 2.0 ** -10)
    assert bool(((a - x).abs() <= 2 * step).all()) and bool(((b - x).abs() <= step).all())


def test_bookkeeping_keeps_the_counts():
    """After any calls, refs is how often the rows name each page."""
    import random
    rng = random.Random(0)
    page, width, n_pages = 8, 6, 60
    refs, table, lens = [0] * n_pages, [[-1] * width for _ in range(4)], [0] * 4
    for _ in range(60):
        if rng.random() < 0.4:
            parents = [rng.randrange(-1, len(lens)) for _ in range(rng.randrange(1, 7))]
            refs, table, lens = O.reorder(refs, table, lens, parents, page, width)
        else:
            want = [rng.randrange(0, width * page + 1) for _ in lens]
            refs, table, lens, copies, _ = O.resize(refs, table, lens, want, page)
        if rng.random() < 0.2:
            refs, table, used, _ = O.compact(refs, table, lens, page)
            assert all(c > 0 for c in refs[:used]) and not any(refs[used:])
        count = [0] * n_pages
        for t, n in zip(table, lens):
            for j, p in enumerate(t):
                assert (p >= 0) == (j < O.n_pages_of(n, page))
                if p >= 0:
                    count[p] += 1
        assert count == refs


def test_a_full_pool_leaves_no_page_with_a_writer_and_a_reader():
    """Rows that share begun pages at other lengths, all grown, any number of pages left: who is refused keeps length
    and pages, who grows writes to pages of its own, and what anyone holds is counted."""
    import random
    rng = random.Random(1)
    page, width, hit = 8, 4, 0
    for _ in range(400):
        heads, spare = rng.randrange(1, 4), rng.randrange(0, 5)
        lens = [rng.randrange(1, 2 * page + 1) for _ in range(heads)]
        refs, table = [], []
        for n in lens:
            table.append(list(range(len(refs), len(refs) + O.n_pages_of(n, page))))
            refs += [1] * O.n_pages_of(n, page)
        refs += [0] * spare
        table = [t + [-1] * (width - len(t)) for t in table]
        refs, table, lens = O.reorder(refs, table, lens, [rng.randrange(heads) for _ in range(rng.randrange(1, 6))], page, width)
        refs, table, lens, _, _ = O.resize(refs, table, lens, [n - rng.randrange(0, (n - 1) % page + 1) for n in lens], page)
        want = [n + rng.randrange(0, 2 * page) for n in lens]
        r, t, l, copies, refused = O.resize(refs, table, lens, want, page)
        assert all((l[i], t[i]) == (lens[i], table[i]) for i in refused)
        assert [l[i] for i in range(len(l)) if i not in refused] == [want[i] for i in range(len(l)) if i not in refused]
        count = [sum(p in row for row in t) for p in range(len(r))]
        assert count == r and len({b for _, b in copies}) == len(copies)
        for i in range(len(l)):
            if l[i] > lens[i] and lens[i] % page:
                assert r[t[i][(lens[i] - 1) // page]] == 1
        hit += len(refused) > 0
    assert hit > 20
