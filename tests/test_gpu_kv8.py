"""The 8-bit cache on the GPU against the oracle: append (bit by bit) and attention
(at the oracle's bounds)."""
import math

import pytest
import torch

from oracle import kv8_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def lib():
    import block_diffusion_speculative_flush_gb300 as D
    return D


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch8:
    """A ragged batch over 8-bit pages whose old rows and scales are there; every slot that holds no token, every
    spare page and its scale, and every row behind the last sequence is NaN."""

    def __init__(self, dtype, hq, hkv, d, page, rows, lens, seed=0, hnd=False, tail=3, spare=2, pow2=False):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.hq, self.hkv, self.d, self.page, self.rows, self.lens = DT[dtype], hq, hkv, d, page, rows, lens
        self.starts = [0]
        for n in rows:
            self.starts.append(self.starts[-1] + n)
        n, total = self.starts[-1], self.starts[-1] + tail
        rnd = lambda *s: torch.randn(s, generator=g)
        self.q = rnd(total, hq, d).to(self.dt)
        self.k, self.v = ((rnd(total, hkv, d) * torch.exp2(6 * torch.rand((total, hkv, 1), generator=g) - 3)).to(self.dt)
                          for _ in range(2))
        for x in (self.q, self.k, self.v):
            x[n:] = math.nan
        need = [O.n_pages_of(L, page) for L in lens]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g)
        self.table = torch.full((len(rows), max(max(need), 1)), -7, dtype=torch.int32)
        self.kp = torch.full((n_pages, page, hkv, d), 0x7F, dtype=torch.uint8)
        self.vp = self.kp.clone()
        self.ks = torch.full((n_pages, hkv), math.nan)
        self.vs = self.ks.clone()
        at = 0
        for b, L in enumerate(lens):
            ids = order[at:at + need[b]]
            self.table[b, :need[b]] = ids.to(torch.int32)
            at += need[b]
            old = L - rows[b]
            for j in range(O.n_pages_of(old, page)):
                m, pg = min(page, old - j * page), int(ids[j])
                for codes, scale in ((self.kp, self.ks), (self.vp, self.vs)):
                    x = rnd(m, hkv, d) * torch.exp2(4 * torch.rand((1, hkv, 1), generator=g) - 2)
                    s = x.abs().amax((0, 2)) / 448
                    if pow2:
                        s = torch.exp2(torch.ceil(torch.log2(s)))
                    codes[pg, :m] = O.encode(x / s[:, None])
                    scale[pg] = s
        self.hnd, self.pow2 = hnd, pow2

    def appended(self):
        a = O.append8(self.kp, self.ks, self.k, self.starts, self.lens, self.table)
        b = O.append8(self.vp, self.vs, self.v, self.starts, self.lens, self.table)
        return a[0], b[0], a[1], b[1]

    def cuda(self, kp, vp, ks, vs):
        if self.hnd:   # [page][head][slot][d] and [head][page] in memory
            kp, vp = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (kp, vp))
            ks, vs = (x.t().contiguous().cuda().t() for x in (ks, vs))
        return kp.cuda().view(torch.float8_e4m3fn), vp.cuda().view(torch.float8_e4m3fn), ks.cuda(), vs.cuda()


def same_codes(a, b):
    """Equal codes, any NaN for a NaN."""
    a, b = a.cpu().contiguous().view(torch.uint8), b.contiguous()
    return bool((((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F) | (a == b)).all())


def same_scales(a, b):
    return torch.equal(torch.nan_to_num(a.cpu(), nan=-1.0), torch.nan_to_num(b, nan=-1.0))


def check_attention(o, lse, ref, rows):
    ro, rl, to, tl = ref
    err = (o[:rows].double().cpu() - ro[:rows]).abs()
    bad = ~(err <= to[:rows])
    assert not bad.any(), (int(bad.sum()), float(err[bad][0]), bad.nonzero()[:4].tolist())
    el = (lse[:rows].double().cpu() - rl[:rows]).abs()
    same_inf = torch.isneginf(lse[:rows].cpu()) & torch.isneginf(rl[:rows])
    bad = ~(same_inf | (el <= tl[:rows]))
    assert not bad.any(), (int(bad.sum()), float(el[bad][0]), bad.nonzero()[:4].tolist())


def bound(B):
    """A bound of the new rows with which calls of more than 32 rows a group take the kernel of many rows, short ones too."""
    rows = max(max(B.rows), 1)
    return 1 << 15 if rows * (B.hq // B.hkv) > 32 else rows


WIDE = False


@pytest.fixture(params=["tight", "wide"])
def span(request):
    """wide: a table that could hold 200000 tokens a row, with which few rows' work is laid out as ranges."""
    global WIDE
    WIDE = request.param == "wide"
    yield
    WIDE = False


def widen(table, page):
    return torch.nn.functional.pad(table, (0, 200000 // page), value=-1) if WIDE else table


def run8(B, causal, window, scale=None, max_len=None, append=True, status=None, pages=None, max_rows=None):
    D = lib()
    P = B.cuda(B.kp, B.vp, B.ks, B.vs) if pages is None else pages
    starts, lens, table = i32(B.starts), i32(B.lens), widen(B.table, B.page).cuda()
    if append:
        D.dflash_kv8_append(B.k.cuda(), B.v.cuda(), *P, starts, lens, table, status=status)
    q = B.q.cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    D.dflash_kv8_attention(q, *P, starts, lens, table, out, max_rows=max_rows or bound(B), max_len=max_len, causal=causal,
                           window=window, scale=scale, lse=lse, status=status)
    torch.cuda.synchronize()
    return out, lse, P


def ref8(B, causal, window, scale=None, pages=None, many=None):
    kp, vp, ks, vs = B.appended() if pages is None else pages
    bf16 = B.dt == torch.bfloat16
    return O.attention8(B.q[:B.starts[-1]], O.gather8(kp, ks, B.lens, B.table), O.gather8(vp, vs, B.lens, B.table),
                        B.starts, B.lens, causal, window, scale if scale is not None else B.d ** -0.5, bf16,
                        bf16 and B.d in (64, 128), bf16 and B.d == 128 and (bound(B) > max(B.rows) if many is None else many))


SHAPES = [  # hq, hkv, page, rows, lens
    (4, 4, 16, [1], [1]),
    (8, 2, 16, [1, 1, 1], [1, 17, 300]),
    (6, 2, 16, [5, 0, 8, 1], [5, 0, 140, 64]),
    (5, 1, 32, [16], [129]),
    (8, 1, 64, [16, 3], [700, 128]),
    (7, 1, 128, [40, 33], [290, 33]),
    (4, 2, 16, [130, 1, 77], [130, 900, 205]),
    (16, 1, 256, [70], [513]),
]


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128), ("bf16", 48), ("f32", 16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 37), (False, 130)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_and_attention(dtype, d, causal, window, shape):
    hq, hkv, page, rows, lens = SHAPES[shape]
    B = Batch8(dtype, hq, hkv, d, page, rows, lens, seed=shape, hnd=shape % 2 == 1, pow2=shape % 3 == 0)
    status = i32([0])
    out, lse, P = run8(B, causal, window, status=status)
    want = B.appended()
    assert same_codes(P[0], want[0]) and same_codes(P[1], want[1])
    assert same_scales(P[2], want[2]) and same_scales(P[3], want[3])
    n = B.starts[-1]
    check_attention(out, lse, ref8(B, causal, window), n)
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())   # rows behind the last sequence
    lib().dflash_status_check(status)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,page,rows", [(128, 16, [200]), (64, 64, [64, 1, 130]), (80, 1024, [2500, 3]), (16, 256, [700])])
def test_append_of_long_chunks(dtype, d, page, rows):
    lens = [n + 5 * b for b, n in enumerate(rows)]
    B = Batch8(dtype, 3, 3, d, page, rows, lens, seed=d, pow2=True)
    D = lib()
    P = B.cuda(B.kp, B.vp, B.ks, B.vs)
    D.dflash_kv8_append(B.k.cuda(), B.v.cuda(), *P, i32(B.starts), i32(lens), B.table.cuda())
    want = B.appended()
    assert same_codes(P[0], want[0]) and same_codes(P[1], want[1])
    assert same_scales(P[2], want[2]) and same_scales(P[3], want[3])


def test_append_at_the_borders_of_a_scale():
    """Rows of exactly 448 and one step more, zeros, the largest and smallest numbers, NaN and infinities."""
    D = lib()
    vals = [448.0, 449.0, 0.0, 3.0e38, -3.0e38, 1e-40, math.nan, math.inf, -math.inf, 2.0 ** -60 * 448, 2.0 ** 60 * 448,
            1.0, 1.75, 1.7500001, 0.0625]
    for first in vals:
        for second in vals:
            x = torch.full((2, 1, 16), first)
            x[0, 0, 3] = 0.3
            x[1] = second
            kp = torch.zeros((1, 16, 1, 16), dtype=torch.uint8)
            ks = torch.full((1, 1), math.nan)
            dev = (kp.cuda(), kp.clone().cuda(), ks.cuda(), ks.clone().cuda())
            tb = torch.zeros((1, 1), dtype=torch.int32)
            codes, scale = kp, ks
            for i in range(2):   # one at a time: the second token meets the first one's scale
                D.dflash_kv8_append(x[i:i + 1].cuda(), x[i:i + 1].cuda(), *dev, i32([0, 1]), i32([i + 1]), tb.cuda())
                codes, scale = O.append8(codes, scale, x[i:i + 1], [0, 1], [i + 1], tb)
            assert same_codes(dev[0], codes) and same_codes(dev[1], codes), (first, second)
            assert same_scales(dev[2], scale) and same_scales(dev[3], scale), (first, second)


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 37)])
@pytest.mark.parametrize("rows,lens,hq,hkv", [([40], [600], 4, 1), ([33, 1, 90], [33, 1000, 400], 5, 1),
                                              ([200, 7], [900, 2000], 4, 2), ([16, 16], [4096, 300], 32, 8)])
def test_many_rows_of_short_calls(rows, lens, hq, hkv, causal, window, d):
    """Tight bounds: items that all run at once as clusters."""
    B = Batch8("bf16", hq, hkv, d, 16, rows, lens, seed=31)
    out, lse, _ = run8(B, causal, window, max_len=max(lens), max_rows=max(rows))
    check_attention(out, lse, ref8(B, causal, window, many=False), sum(rows))


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,lens", [([16], [5000]), ([1] * 9, [1, 4096, 5, 2999, 64, 128, 127, 129, 1000]),
                                       ([300, 2, 150], [2100, 3000, 150])])
def test_attention_over_long_caches(dtype, rows, lens):
    B = Batch8(dtype, 8, 2, 128, 16, rows, lens, seed=5)
    out, lse, _ = run8(B, True, 0)
    check_attention(out, lse, ref8(B, True, 0), B.starts[-1])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,hq", [([1, 1, 1], 2), ([20, 9, 1], 4), ([3, 3, 2], 16)])
def test_attention_with_many_key_tiles(rows, hq, d):
    B = Batch8("bf16", hq, 2, d, 256, rows, [30011, 17, 16384], seed=7, tail=0)
    out, lse, _ = run8(B, True, 0)
    check_attention(out, lse, ref8(B, True, 0), B.starts[-1])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows,lens,hq", [([16], [3000], 4), ([1, 5], [900, 2000], 8), ([200, 90], [900, 700], 4),
                                          ([3] * 20, [1000 + 13 * b for b in range(20)], 8)])
def test_hidden_codes_that_are_nan(dtype, d, rows, lens, hq):
    """A window of 100, NaN outside it and in the block's last key: what a row does not see never reaches it, and
    who sees the last key answers NaN where it is."""
    B = Batch8(dtype, hq, 2, d, 16, rows, lens, seed=3)
    kp, vp, ks, vs = B.appended()
    clean = tuple(x.clone() for x in (kp, vp, ks, vs))
    for b, (n, L) in enumerate(zip(rows, lens)):
        for p in list(range(0, L - n - 100)) + ([L - 1] if n > 1 else []):
            pg, sl = int(B.table[b, p // 16]), p % 16
            vp[pg, sl, :, p % d] = 0x7F
            if p < L - 1:
                kp[pg, sl, :, (p + 1) % d] = 0xFF
    ref = ref8(B, True, 100, pages=clean)
    out, lse, _ = run8(B, True, 100, append=False, pages=B.cuda(kp, vp, ks, vs))
    for b, n in enumerate(rows):
        last = B.starts[b + 1] - 1
        sl = slice(B.starts[b], last + (0 if n > 1 else 1))
        check_attention(out[sl], lse[sl], tuple(x[sl] for x in ref), sl.stop - sl.start)
        if n > 1:   # only that column of the last row
            c = (lens[b] - 1) % d
            assert bool(torch.isnan(out[last, :, c]).all())
            rest = [i for i in range(d) if i != c]
            check_attention(out[last:last + 1, :, rest], lse[last:last + 1],
                            (ref[0][last:last + 1, :, rest], ref[1][last:last + 1], ref[2][last:last + 1, :, rest],
                             ref[3][last:last + 1]), 1)


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [[1], [3], [40], [150]])
def test_a_nan_that_a_row_sees(dtype, d, rows):
    """A NaN in K makes all of a row NaN, one in V the columns where it is."""
    B = Batch8(dtype, 4, 1, d, 16, rows, [400], seed=11, tail=0)
    kp, vp, ks, vs = B.appended()
    pg = int(B.table[0, 3])
    v2 = vp.clone()
    v2[pg, 5, 0, 17] = 0x7F
    out, lse, _ = run8(B, True, 0, append=False, pages=B.cuda(kp, v2, ks, vs))
    assert bool(torch.isnan(out[..., 17]).all()) and bool(torch.isfinite(lse).all())
    rest = [c for c in range(d) if c != 17]
    ref = ref8(B, True, 0, pages=(kp, vp, ks, vs))
    check_attention(out[..., rest], lse, (ref[0][..., rest], ref[1], ref[2][..., rest], ref[3]), rows[0])
    kp[pg, 5, 0, 17] = 0x7F
    out, lse, _ = run8(B, True, 0, append=False, pages=B.cuda(kp, vp, ks, vs))
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [[1, 2], [30, 9], [140, 3]])
def test_scales_far_apart(dtype, d, rows):
    """Pages of V whose scales differ by 2^40 and keys whose scores are far apart, at the bounds' ends."""
    B = Batch8(dtype, 4, 2, d, 16, rows, [300, 200], seed=13)
    kp, vp, ks, vs = B.appended()
    for j in range(vs.shape[0]):
        vs[j] *= 2.0 ** [0, -40, 20, -3, 7][j % 5]
        ks[j] *= 2.0 ** [0, -30, 1, -3, -7][j % 5]
    out, lse, _ = run8(B, True, 0, append=False, pages=B.cuda(kp, vp, ks, vs))
    check_attention(out, lse, ref8(B, True, 0, pages=(kp, vp, ks, vs)), B.starts[-1])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [[1, 2], [30, 9], [140, 3]])
@pytest.mark.parametrize("far", [0, 60])
def test_scales_that_are_no_powers_of_two(dtype, d, rows, far):
    """Any positive scales (a cache that another program filled), within 2^-60 .. 2^60."""
    B = Batch8(dtype, 4, 2, d, 16, rows, [500, 200], seed=15)
    kp, vp, ks, vs = B.appended()
    g = torch.Generator().manual_seed(2)
    ks *= 1 + torch.rand(ks.shape, generator=g)
    vs *= (1 + torch.rand(vs.shape, generator=g)) * torch.exp2(torch.randint(-far // 2, far // 2 + 1, vs.shape, generator=g).float())
    out, lse, _ = run8(B, True, 0, append=False, pages=B.cuda(kp, vp, ks, vs))
    check_attention(out, lse, ref8(B, True, 0, pages=(kp, vp, ks, vs)), B.starts[-1])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [[3], [40], [150]])
@pytest.mark.parametrize("window", [0, 50])
def test_scores_that_vanish(dtype, d, rows, window):
    """Queries of 2^-100 and a small scale: every factor of a score underflows, the mask holds all the same."""
    B = Batch8(dtype, 4, 1, d, 16, rows, [300], seed=33)
    B.q = B.q * 2.0 ** -100
    kp, vp, ks, vs = B.appended()
    ks = ks * 0 + 2.0 ** -60
    out, lse, _ = run8(B, True, window, scale=2.0 ** -20, append=False, pages=B.cuda(kp, vp, ks, vs))
    check_attention(out, lse, ref8(B, True, window, scale=2.0 ** -20, pages=(kp, vp, ks, vs)), B.starts[-1])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 24, 1), ("bf16", 128, 1), ("bf16", 100, 2), ("f32", 24, 1)])
@pytest.mark.parametrize("rows,lens", [([1, 2], [200, 150]), ([7, 30], [77, 300])])
def test_wide_groups(dtype, hq, hkv, rows, lens):
    B = Batch8(dtype, hq, hkv, 64, 32, rows, lens, seed=hq)
    out, lse, _ = run8(B, True, 0)
    check_attention(out, lse, ref8(B, True, 0), B.starts[-1])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,scale,big", [("bf16", 1e-30, 1e30), ("bf16", 1e20, 1e-22), ("f32", 1e-30, 1e30)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[1], [40], [200]])
def test_queries_and_scales_of_any_size(dtype, scale, big, d, rows):
    B = Batch8(dtype, 4, 1, d, 16, rows, [300], seed=17, tail=0)
    B.q = (B.q.float() * big * 0.1).to(B.dt)
    out, lse, _ = run8(B, True, 0, scale=scale)
    check_attention(out, lse, ref8(B, True, 0, scale=scale), rows[0])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [[2, 1], [100, 20]])
def test_missing_pages_read_as_zeros_and_are_told(dtype, d, rows):
    D = lib()
    B = Batch8(dtype, 4, 2, d, 16, rows, [300, 200], seed=19)
    want = B.appended()
    B2 = B.table.clone()
    for bad in (-1, 1 << 30, int(want[0].shape[0])):
        B.table = B2.clone()
        B.table[0, 4] = bad
        status = i32([0])
        out, lse, _ = run8(B, True, 0, append=False, status=status, pages=B.cuda(*want))
        with pytest.raises(D.DFlashError, match="page id"):
            D.dflash_status_check(status)
        z = tuple(torch.cat((x, torch.zeros_like(x[:1]) if x.dtype == torch.uint8 else torch.ones_like(x[:1]))) for x in want)
        B.table[0, 4] = want[0].shape[0]    # the page of zeros
        check_attention(out, lse, ref8(B, True, 0, pages=z), B.starts[-1])
    # an append to it is dropped
    B.table = B2.clone()
    B.table[1, 12] = -1
    status = i32([0])
    P = B.cuda(B.kp, B.vp, B.ks, B.vs)
    D.dflash_kv8_append(B.k.cuda(), B.v.cuda(), *P, i32(B.starts), i32(B.lens), B.table.cuda(), status=status)
    with pytest.raises(D.DFlashError, match="page id"):
        D.dflash_status_check(status)
    lost = int(B2[1, 12])
    w2 = tuple(x.clone() for x in want)
    for x, y in zip(w2, (B.kp, B.vp, B.ks, B.vs)):
        x[lost] = y[lost]
    assert same_codes(P[0], w2[0]) and same_codes(P[1], w2[1]) and same_scales(P[2], w2[2]) and same_scales(P[3], w2[3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_outside_their_bounds_are_left_alone(dtype):
    D = lib()
    B = Batch8(dtype, 4, 2, 64, 16, [2, 3, 1], [40, 50, 60], seed=23, tail=0)
    want = B.appended()
    ref = ref8(B, True, 0)
    P = B.cuda(B.kp, B.vp, B.ks, B.vs)
    lens = i32([40, 2, 60])                       # the second has three rows
    status = i32([0])
    D.dflash_kv8_append(B.k.cuda(), B.v.cuda(), *P, i32(B.starts), lens, B.table.cuda(), status=status)
    out, lse = torch.full_like(B.q.cuda(), 7.0), torch.full((6, 4), 7.0, device="cuda")
    D.dflash_kv8_attention(B.q.cuda(), *P, i32(B.starts), lens, B.table.cuda(), out, max_rows=3, lse=lse, status=status)
    with pytest.raises(D.DFlashError, match="bounds"):
        D.dflash_status_check(status)
    assert bool((out[2:5] == 7).all()) and bool((lse[2:5] == 7).all())
    for sl in (slice(0, 2), slice(5, 6)):
        check_attention(out[sl], lse[sl], tuple(x[sl] for x in ref), sl.stop - sl.start)
    for b in (0, 2):
        ids = B.table[b, :4].long()
        ids = ids[ids >= 0]
        assert same_codes(P[0][ids], want[0][ids])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_beyond_two_to_the_31_codes(dtype):
    D = lib()
    hkv, d, page, n_pages = 8, 128, 1024, 4200            # 4.4e9 codes each of K and V
    kp = torch.empty((n_pages, page, hkv, d), dtype=torch.uint8, device="cuda")
    vp = torch.empty_like(kp)
    ks, vs = (torch.ones((n_pages, hkv), device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(0)
    rows, lens, ids = [3, 1], [1500, 700], [[4199, 4190], [4180, 0]]
    table = torch.tensor(ids, dtype=torch.int32)
    # the same sequences in a small cache are the reference
    sk, sv = (torch.zeros((4, page, hkv, d), dtype=torch.uint8) for _ in range(2))
    ss, s2 = torch.ones((4, hkv)), torch.ones((4, hkv))
    small = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    x = [torch.randn((sum(lens), hkv, d), generator=g).to(DT[dtype]) for _ in range(2)]
    sk, ss = O.append8(sk, ss, x[0], [0, 1500, 2200], lens, small)
    sv, s2 = O.append8(sv, s2, x[1], [0, 1500, 2200], lens, small)
    D.dflash_kv8_append(x[0].cuda(), x[1].cuda(), kp, vp, ks, vs, i32([0, 1500, 2200]), i32(lens), table.cuda())
    q = torch.randn((4, 16, d), generator=g).to(DT[dtype])
    out, lse = torch.empty((4, 16, d), dtype=DT[dtype], device="cuda"), torch.empty((4, 16), device="cuda")
    D.dflash_kv8_attention(q.cuda(), kp, vp, ks, vs, i32([0, 3, 4]), i32(lens), table.cuda(), out, max_rows=3, lse=lse)
    for b, L in enumerate(lens):
        for j in range(O.n_pages_of(L, page)):
            m = min(page, L - j * page)
            assert same_codes(kp[ids[b][j], :m], sk[int(small[b, j]), :m])
    ref = O.attention8(q, O.gather8(sk, ss, lens, small), O.gather8(sv, s2, lens, small), [0, 3, 4], lens, True, 0,
                       d ** -0.5, dtype == "bf16", dtype == "bf16")
    check_attention(out, lse, ref, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [[6, 1], [90, 1]])
def test_two_graphs_replayed_at_once(dtype, rows):
    """Two captured calls (without a call before the capture) on two streams, each with its own workspace."""
    D = lib()
    Bs = [Batch8(dtype, 8, 2, 128, 16, rows, [2500 + 100 * i, 90], seed=i, tail=0) for i in range(2)]
    refs = [ref8(B, True, 0) for B in Bs]
    state, graphs = [], []
    for B in Bs:
        P = B.cuda(*B.appended())
        q, st, ln, tb = B.q.cuda(), i32(B.starts), i32(B.lens), B.table.cuda()
        o, l = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        need = D.dflash_kv8_attention_workspace(q, o, st, ln, tb, bound(B), 2700, *P)
        ws = torch.empty(max(need, 32), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            D.dflash_kv8_attention(q, *P, st, ln, tb, o, bound(B), max_len=2700, lse=l, workspace=ws)
        state.append((P, q, st, ln, tb, o, l, ws))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in Bs]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for x, r in zip(state, refs):
        check_attention(x[5], x[6], r, sum(rows))


def test_a_workspace_that_is_too_small_is_refused():
    D = lib()
    B = Batch8("bf16", 8, 2, 128, 16, [1], [900], tail=0)
    P = B.cuda(*B.appended())
    q, st, ln, tb = B.q.cuda(), i32(B.starts), i32(B.lens), torch.nn.functional.pad(B.table, (0, 2500), value=-1).cuda()
    o = torch.empty_like(q)
    need = D.dflash_kv8_attention_workspace(q, o, st, ln, tb, 1, 40000, *P)
    assert need > 0
    with pytest.raises(D.DFlashError, match="workspace"):
        D.dflash_kv8_attention(q, *P, st, ln, tb, o, 1, max_len=40000,
                               workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[1], [12], [30], [200]])
def test_queries_with_elements_far_apart(d, rows):
    """Elements of q that differ by up to 2^20 within a row, and rows of zeros."""
    B = Batch8("bf16", 4, 1, d, 32, rows, [500], seed=29, tail=0)
    g = torch.Generator().manual_seed(1)
    B.q = (B.q.float() * torch.exp2(torch.randint(-20, 1, B.q.shape, generator=g).float())).bfloat16()
    B.q[0, 1] = 0
    out, lse, _ = run8(B, True, 0)
    check_attention(out, lse, ref8(B, True, 0), rows[0])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("bits", [math.nan, math.inf])
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [[1], [30], [150]])
def test_a_query_that_is_not_finite_is_its_rows_own(dtype, d, rows, bits):
    B = Batch8(dtype, 4, 1, d, 16, rows, [400], seed=31, tail=0)
    ref = ref8(B, True, 0)
    B.q[0, 2, 5] = bits
    out, lse, _ = run8(B, True, 0)
    assert bool(torch.isnan(out[0, 2]).all())
    out[0, 2], lse[0, 2] = ref[0][0, 2].to(out), ref[1][0, 2].to(lse)
    check_attention(out, lse, ref, rows[0])


def test_a_stream_of_its_own_and_a_strided_cache():
    """K, V and their scales side by side in one allocation each, another stream than the current one."""
    D = lib()
    B = Batch8("bf16", 8, 2, 128, 16, [5, 1], [700, 90], seed=37, tail=0)
    want = B.appended()
    n = B.kp.shape[0]
    codes = torch.zeros((n, 2, 16, 2, 128), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, 2, 2), device="cuda")
    codes[:, 0], codes[:, 1] = B.kp.cuda(), B.vp.cuda()
    scales[:, 0], scales[:, 1] = B.ks.cuda(), B.vs.cuda()
    P = (codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1])
    args = (i32(B.starts), i32(B.lens), B.table.cuda())
    q, k, v = B.q.cuda(), B.k.cuda(), B.v.cuda()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    D.dflash_kv8_append(k, v, *P, *args, stream=s)
    D.dflash_kv8_attention(q, *P, *args, out, max_rows=5, lse=lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert same_codes(codes[:, 0], want[0]) and same_codes(codes[:, 1], want[1])
    assert same_scales(scales[:, 0], want[2]) and same_scales(scales[:, 1], want[3])
    check_attention(out, lse, ref8(B, True, 0), 6)


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("rows,lens", [([1] * 5, [300, 1, 900, 17, 2000]), ([40, 90], [500, 400])])
def test_the_same_call_twice_gives_the_same_bits(rows, lens):
    B = Batch8("bf16", 8, 2, 128, 16, rows, lens, seed=41)
    P = B.cuda(*B.appended())
    a = run8(B, True, 0, append=False, pages=P)
    for _ in range(5):
        b = run8(B, True, 0, append=False, pages=P)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,hkv,most", [(90, 4, 3), (70, 8, 1), (50, 8, 12), (257, 2, 2)])
def test_items_that_take_turns(batch, hkv, most, d):
    """More items than run at once, of uneven lengths, some of them alike and some without rows."""
    rows = [(b * 5) % (most + 1) for b in range(batch)]
    lens = [max(r, (b * 131) % 700 // 50 * 50) for b, r in enumerate(rows)]
    B = Batch8("bf16", 2 * hkv, hkv, d, 16, rows, lens, seed=47)
    out, lse, _ = run8(B, True, 0)
    check_attention(out, lse, ref8(B, True, 0), B.starts[-1])
    out, lse, _ = run8(B, True, 100)
    check_attention(out, lse, ref8(B, True, 100), B.starts[-1])


@pytest.mark.usefixtures("span")
def test_many_short_sequences():
    """More sequences than a warp looks at in one go, most of them of a few tokens, some without new rows."""
    rows = [(b * 7) % 3 for b in range(300)]
    lens = [r + (b * 37) % 50 for b, r in enumerate(rows)]
    for dtype in ("bf16", "f32"):
        B = Batch8(dtype, 4, 2, 64, 16, rows, lens, seed=43)
        status = i32([0])
        out, lse, P = run8(B, True, 0, status=status)
        lib().dflash_status_check(status)
        want = B.appended()
        assert same_codes(P[0], want[0]) and same_scales(P[3], want[3])
        check_attention(out, lse, ref8(B, True, 0), B.starts[-1])


# ---- a NaN among V's codes in the last, partial tile of keys
@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("causal,window", [(False, 0), (False, 50), (True, 0), (True, 50)])
@pytest.mark.parametrize("rows,lens", [([40], [400]), ([65], [400]), ([150], [400]), ([1], [400]), ([33, 2], [130, 257])])
@pytest.mark.parametrize("back", [0, 7])
def test_a_nan_in_the_last_tile_reaches_who_sees_it(dtype, d, causal, window, rows, lens, back):
    B = Batch8(dtype, 4, 1, d, 16, rows, lens, seed=51, tail=0)
    kp, vp, ks, vs = B.appended()
    ref = ref8(B, causal, window, pages=(kp, vp, ks, vs))
    v2 = vp.clone()
    at = [L - 1 - back for L in lens]
    for b, p in enumerate(at):
        v2[int(B.table[b, p // 16]), p % 16, 0, 17] = 0x7F
    out, lse, _ = run8(B, causal, window, append=False, pages=B.cuda(kp, v2, ks, vs))
    for b, (n, L) in enumerate(zip(rows, lens)):
        pos = torch.arange(L - n, L)
        see = (pos >= at[b] if causal else torch.ones(n, dtype=torch.bool)) & (pos - at[b] < window if window else True)
        got = torch.isnan(out[B.starts[b]:B.starts[b + 1], :, 17].cpu())
        assert torch.equal(got, see[:, None].expand_as(got)), (b, got[:, 0].tolist(), see.tolist())
    o = torch.where(torch.isnan(out), ref[0].to(out), out)
    check_attention(o, lse, ref, sum(rows))
    rest = [c for c in range(d) if c != 17]
    assert bool(torch.isfinite(out[..., rest]).all())


# ---- scales of V that a row does not see, or that come with next to no probability
@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows,lens", [([3], [2266]), ([30], [2266]), ([3, 40], [2266, 2270]), ([150], [2266])])
@pytest.mark.parametrize("window", [0, 2010])
def test_scales_of_hidden_pages_do_not_matter(dtype, d, rows, lens, window):
    """Pages that only the later rows see (without a window), or only the earlier ones (with one), have scales 2^40
    above the others: the rows that do not see them keep all their bits."""
    B = Batch8(dtype, 4, 1, d, 16, rows, lens, seed=53, tail=0)
    kp, vp, ks, vs = B.appended()
    for b, (n, L) in enumerate(zip(rows, lens)):
        for j in range(O.n_pages_of(L, 16)):
            if 16 * j + 16 <= L - window if window else 16 * j > L - n:
                vs[int(B.table[b, j])] *= 2.0 ** 40
    out, lse, _ = run8(B, True, window, append=False, pages=B.cuda(kp, vp, ks, vs))
    check_attention(out, lse, ref8(B, True, window, pages=(kp, vp, ks, vs)), sum(rows))


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [[1], [3], [30], [150]])
@pytest.mark.parametrize("bits", [40, 120])
@pytest.mark.parametrize("where", [0, 17, 131])
def test_a_large_scale_of_small_probability(dtype, d, rows, bits, where):
    """One page whose values are 2^bits times the others' and whose probabilities are as much smaller: both matter."""
    B = Batch8(dtype, 4, 1, d, 16, rows, [2450], seed=57, tail=0)
    B.q = B.q.abs()
    kp, vp, ks, vs = B.appended()
    pg = int(B.table[0, where])
    vs = torch.exp2(torch.round(torch.log2(vs)) - bits // 2)
    ks = ks * 0.25
    vs[pg] *= 2.0 ** bits
    vs = vs.clamp(2.0 ** -60, 2.0 ** 60)
    kp[pg] = 0xB8                                                   # -1
    ks[pg] = bits * math.log(2) / (0.8 * d * d ** -0.5)             # the mean of |q| is 0.8
    out, lse, _ = run8(B, True, 0, append=False, pages=B.cuda(kp, vp, ks, vs))
    check_attention(out, lse, ref8(B, True, 0, pages=(kp, vp, ks, vs)), rows[0])


@pytest.mark.usefixtures("span")
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[1], [30], [150]])
def test_one_key_of_a_huge_score(d, rows):
    """Scores of some 2^17 apart: a row is its best key's value, whose scale is its own page's, to bf16's last bit."""
    B = Batch8("bf16", 4, 1, d, 16, rows, [300], seed=59, tail=0)
    B.q = B.q.abs() + 1
    kp, vp, ks, vs = B.appended()
    best = 100                                                       # a key that every row sees
    pg, sl = int(B.table[0, best // 16]), best % 16
    kp[:] = 0xB8
    kp[pg, sl] = 0x38                                                # 1 at one key, -1 elsewhere
    ks[:] = 2.0 ** 12
    vs *= torch.exp2(torch.arange(len(vs), dtype=torch.float32) % 7 - 3)[:, None]
    out, lse, _ = run8(B, True, 0, append=False, pages=B.cuda(kp, vp, ks, vs))
    want = (O.decode(vp, vs)[pg, sl, 0]).expand(rows[0], 4, d)
    err = (out.cpu().double() - want).abs()
    assert bool((err <= want.abs() * (2.0 ** -8 + 2.0 ** -11)).all()), float((err / want.abs().clamp(min=1e-30)).max())


# ---- a bad sequence behind the first 32
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,bad", [(64, 40), (64, 63), (300, 33), (300, 299), (33, 32), (20, 19)])
@pytest.mark.parametrize("rows", [1, 0, 40])
def test_append_tells_of_a_bad_sequence_anywhere(dtype, batch, bad, rows):
    """The sequence at index bad has `rows` new rows (the others one) and a length outside its bounds."""
    D = lib()
    n = [1] * batch
    n[bad] = rows
    lens = [5 + b % 40 for b in range(batch)]
    lens[bad] = 50
    B = Batch8(dtype, 2, 2, 64, 16, n, lens, seed=61, tail=0, pow2=True)
    want = B.appended()
    for length in (-1, 16 * B.table.shape[1] + 1) + ((rows - 1,) if rows > 1 else ()):
        P = B.cuda(B.kp, B.vp, B.ks, B.vs)
        told = list(lens)
        told[bad] = length
        status = i32([0])
        D.dflash_kv8_append(B.k.cuda(), B.v.cuda(), *P, i32(B.starts), i32(told), B.table.cuda(), status=status)
        with pytest.raises(D.DFlashError, match="bounds"):
            D.dflash_status_check(status)
        ids = B.table[bad].long()
        ids = ids[ids >= 0]
        w = [x.clone() for x in want]
        for x, y in zip(w, (B.kp, B.vp, B.ks, B.vs)):
            x[ids] = y[ids]                                          # its pages keep what they held
        assert same_codes(P[0], w[0]) and same_codes(P[1], w[1]) and same_scales(P[2], w[2]) and same_scales(P[3], w[3])
