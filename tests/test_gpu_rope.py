"""Rotary positions on the GPU against the fp64 oracle, at the oracle's bounds."""
import math

import pytest
import torch

from oracle import kv8_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=3.0),
            dict(kind="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
            dict(kind="yarn", factor=4.0, original_len=4096.0, low=1.0, high=32.0)]


def lib():
    import block_diffusion_speculative_flush_gb300 as D
    return D


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def positions(rows, lens):
    return torch.cat([torch.arange(L - n, L) for n, L in zip(rows, lens)])


def starts_of(rows):
    st = [0]
    for n in rows:
        st.append(st[-1] + n)
    return st


def check(y, x, pos, table, theta, scaling, layout, dtype, transpose=False):
    f, amp = O.rope_freqs(table.rot_dim, theta, scaling)
    ref, tol = O.rope(x, pos, f, amp, layout, table.offset, transpose)
    err = (y.cpu().double() - ref).abs()
    bad = ~(err <= tol + ref.abs() * HALF[dtype] + 1e-30)
    assert not bad.any(), (int(bad.sum()), float(err[bad].max()), bad.nonzero()[:3].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,offset", [(128, 128, 0), (64, 32, 0), (128, 24, 8), (64, 2, 62), (256, 256, 0), (8, 6, 2),
                                          (96, 40, 20)])
@pytest.mark.parametrize("rows,lens", [([1], [1]), ([3, 0, 9], [3, 5, 1000000]), ([700, 1, 30], [2100, 1 << 30, 31])])
def test_rope(dtype, layout, d, rot, offset, rows, lens):
    D = lib()
    g = torch.Generator().manual_seed(rot + d)
    st = starts_of(rows)
    n, total, hq, hk = st[-1], st[-1] + 2, 5, 2
    qkv = torch.randn((total, hq + 2 * hk, d), generator=g).to(DT[dtype])
    x = qkv.cuda()
    table = D.dflash_rope_table(rot, 10000.0, layout=layout, offset=offset)
    qo, ko = (torch.full((total, h, d), 7.0, dtype=DT[dtype], device="cuda") for h in (hq, hk))
    status = i32([0])
    D.dflash_rope(table, x[:, :hq], x[:, hq:hq + hk], i32(st), i32(lens), qo, ko, status=status)
    D.dflash_status_check(status)
    pos = positions(rows, lens)
    check(qo[:n], qkv[:n, :hq], pos, table, 10000.0, None, layout, dtype)
    check(ko[:n], qkv[:n, hq:hq + hk], pos, table, 10000.0, None, layout, dtype)
    assert bool((qo[n:] == 7).all()) and bool((ko[n:] == 7).all())
    assert torch.equal(x.cpu(), qkv)
    D.dflash_rope(table, x[:, :hq], x[:, hq:hq + hk], i32(st), i32(lens))      # in place: the same bits
    assert torch.equal(x[:n, :hq], qo[:n]) and torch.equal(x[:n, hq:hq + hk], ko[:n])
    assert torch.equal(x[:, hq + hk:].cpu(), qkv[:, hq + hk:]) and torch.equal(x[n:].cpu(), qkv[n:])


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scaled_frequencies_of_prompts(scaling, dtype):
    D = lib()
    g = torch.Generator().manual_seed(1)
    rows = [130, 1, 500]
    k = torch.randn((sum(rows), 3, 128), generator=g).to(DT[dtype])
    table = D.dflash_rope_table(64, 500000.0, scaling=scaling)
    out = torch.empty_like(k, device="cuda")
    D.dflash_rope(table, None, k.cuda(), i32(starts_of(rows)), None, None, out)
    check(out, k, positions(rows, rows), table, 500000.0, scaling, "half", dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_the_transposed_map_is_the_gradient(layout):
    """<g, R x> = <R^T g, x>, and R^T R is the amplitude squared: against the formula and by differences."""
    D = lib()
    scaling = SCALINGS[4]
    table = D.dflash_rope_table(32, 10000.0, layout=layout, scaling=scaling, offset=8)
    g = torch.Generator().manual_seed(2)
    x, up = torch.randn((40, 2, 64), generator=g), torch.randn((40, 2, 64), generator=g)
    st, ln = i32([0, 40]), i32([100])
    back = torch.empty((40, 2, 64), device="cuda")
    D.dflash_rope(table, up.cuda(), None, st, ln, back, transpose=True)
    check(back, up, positions([40], [100]), table, 10000.0, scaling, layout, "f32", transpose=True)
    # the loss <up, R x> is linear in x: its difference quotient is the gradient up to the fp32 sums
    step = torch.randn((40, 2, 64), generator=g)
    y0, y1 = torch.empty_like(back), torch.empty_like(back)
    D.dflash_rope(table, (x - step).cuda(), None, st, ln, y0)
    D.dflash_rope(table, (x + step).cuda(), None, st, ln, y1)
    quotient = ((y1 - y0).double().cpu() / 2 * up.double()).sum()
    # every output is off by at most 2^-20 of its pair's sizes (up to about 10, times an amplitude below 1.2)
    bound = float((up.abs() * (x.abs() + step.abs() + 10)).sum()) * 2.0 ** -20 * 1.2
    assert abs(float(quotient - (back.double().cpu() * step.double()).sum())) <= bound


def test_a_sequence_outside_its_bounds_is_left_alone():
    D = lib()
    q = torch.ones((6, 1, 64), device="cuda")
    out = torch.full_like(q, 7.0)
    status = i32([0])
    table = D.dflash_rope_table(64, 10000.0)
    D.dflash_rope(table, q, None, i32([0, 2, 4, 6]), i32([2, 1, 1 << 30]), out, status=status)
    with pytest.raises(D.DFlashError, match="bounds"):
        D.dflash_status_check(status)
    assert bool((out[2:4] == 7).all()) and not bool((out[:2] == 7).any()) and not bool((out[4:] == 7).any())


def test_a_captured_call_follows_the_lengths():
    D = lib()
    g = torch.Generator().manual_seed(4)
    q = torch.randn((3, 4, 128), generator=g)
    x, st, ln, out = q.cuda(), i32([0, 1, 3]), i32([1, 2]), torch.empty((3, 4, 128), device="cuda")
    table = D.dflash_rope_table(128, 1e6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dflash_rope(table, x, None, st, ln, out)
    for lens in ([1, 2], [900, 70000]):
        ln.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        check(out, q, positions([1, 2], lens), table, 1e6, None, "half", "f32")
