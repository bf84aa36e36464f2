"""Calls of the target-side operators that their documentation allows at its
edges: pages that a window has left behind, strides of one entry, workspaces
sized ahead, status words."""
import pytest
import torch

from tests.test_gpu_paged_target import fwd, pool, table_of, weights_on_gpu
from tests.test_gpu_target_ops import DT, Batch, check_attention, i32, lib, ref_paged, run_paged, same_bits
from synthetic.target import TARGET_TINY

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,lens,hq", [([16], [3000], 4), ([1, 5], [900, 2000], 8), ([200, 90], [900, 700], 4),
                                          ([1, 1, 1], [30011, 700, 16384], 8), ([300, 2, 150], [2100, 3000, 150], 8)])
def test_pages_behind_the_window_may_be_gone(dtype, rows, lens, hq):
    """A server gives the pages back that no row's window reaches any more: their table entries name no page, and
    that is not an error, although a tile of keys begins in front of the window."""
    W = 100
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=2)
    ref = ref_paged(B, True, W)
    B.kp, B.vp = B.appended()
    for b, (n, L) in enumerate(zip(rows, lens)):
        B.table[b, :max(0, L - n - W + 1) // 16] = -1
    status = i32([0])
    out, lse, _, _ = run_paged(B, True, W, append=False, status=status)
    check_attention(out, lse, ref, B.starts[-1])
    assert int(status.item()) == 0
    b = max(range(len(lens)), key=lambda i: lens[i])   # one page further: the first new row sees its last slots
    B.table[b, (lens[b] - rows[b] - W + 1) // 16] = -1
    run_paged(B, True, W, append=False, status=status)
    assert int(status.item()) == 4


@pytest.mark.parametrize("window", [0, 100, 1 << 20])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tiles", [7, 14, 27, 28, 29, 55, 56, 57, 111, 112, 113])
def test_a_workspace_of_the_reported_size_serves_the_call(tiles, causal, window):
    """bf16 blocks of 16 with 8 KV heads around the lengths (7 key tiles for each CTA of a cluster) where the
    layout of the work, and with it the workspace, changes."""
    D = lib()
    L, page, hkv, hq, d, n = tiles * 128, 256, 8, 16, 64, 16
    g = torch.Generator(device="cuda").manual_seed(tiles)
    kp, vp = (torch.randn((tiles // 2 + 1, page, hkv, d), device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn((n, hq, d), device="cuda", generator=g).bfloat16()
    table = torch.arange(tiles // 2 + 1, dtype=torch.int32, device="cuda")[None]
    args = i32([0, n]), i32([L]), table
    want, got = torch.empty_like(q), torch.empty_like(q)
    need = D.dflash_attention_workspace(q, got, *args, n, L, kp, vp, causal=causal, window=window)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    D.dflash_paged_attention(q, kp, vp, *args, got, n, max_len=L, causal=causal, window=window, workspace=ws)
    D.dflash_paged_attention(q, kp, vp, *args, want, n, max_len=L, causal=causal, window=window)
    assert same_bits(got.cpu(), want.cpu())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hq", [([9], 4), ([300, 1500], 8), ([2000], 2)])
def test_a_workspace_of_the_reported_size_serves_a_prompt(dtype, rows, hq):
    D = lib()
    n = sum(rows)
    q, k, v = (torch.randn((n, h, 64), device="cuda").to(DT[dtype]) for h in (hq, 2, 2))
    st = i32([0] + [sum(rows[:i + 1]) for i in range(len(rows))])
    for window in (0, 200):
        want, got = torch.empty_like(q), torch.empty_like(q)
        need = D.dflash_attention_workspace(q, got, st, None, None, max(rows), 0, k, v, window=window)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        D.dflash_prompt_attention(q, k, v, st, got, max(rows), window=window, workspace=ws)
        D.dflash_prompt_attention(q, k, v, st, want, max(rows), window=window)
        assert same_bits(got.cpu(), want.cpu())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_stride_of_a_single_entry_does_not_matter(dtype):
    """One row, one page, one sequence: torch may report any stride for such a dimension (a slice of a wider
    buffer keeps the buffer's), and nothing ever uses it."""
    D = lib()
    B = Batch(dtype, 4, 2, 64, 16, [1], [9], tail=0, spare=0)
    ref = ref_paged(B, True, 0)
    odd = lambda t: torch.as_strided(t.cuda().contiguous(), t.shape, (1003, *t.contiguous().stride()[1:]))
    q, k, v, kp, vp = (odd(t) for t in (B.q, B.k, B.v, B.kp, B.vp))
    assert q.stride(0) == 1003 and kp.stride(0) == 1003
    args = i32(B.starts), i32(B.lens), odd(B.table)
    out, lse = odd(torch.full_like(B.q, 7.0)), torch.empty((1, 4), device="cuda")
    D.dflash_kv_append(k, v, kp, vp, *args)
    D.dflash_paged_attention(q, kp, vp, *args, out, max_rows=1, lse=lse)
    check_attention(out, lse, ref, 1)
    D.dflash_prompt_attention(q, k, v, i32([0, 1]), out, max_rows=1, lse=lse)
    assert same_bits(out.cpu(), B.v.repeat_interleave(2, 1))   # its only key is itself


def test_an_append_of_more_rows_than_a_sequence_may_have():
    """2^24 + 16 rows of two sequences: the bound on a sequence's rows is not one on the call's."""
    D = lib()
    n, page = (1 << 23) + 8, 1024
    k, v = (torch.arange(2 * n * 4, device="cuda", dtype=torch.float32).view(2 * n, 1, 4) + i for i in range(2))
    per = (n + page - 1) // page
    kp, vp = (torch.zeros((2 * per, page, 1, 4), device="cuda") for _ in range(2))
    st = i32([0])
    D.dflash_kv_append(k, v, kp, vp, i32([0, n, 2 * n]), i32([n, n]), torch.arange(2 * per, dtype=torch.int32,
                                                                                  device="cuda").view(2, per), status=st)
    assert int(st.item()) == 0
    for x, p in ((k, kp), (v, vp)):
        p = p.view(2, per * page, 4)
        assert torch.equal(p[:, :n].reshape(2 * n, 1, 4), x) and not bool(p[:, n:].any())


def test_a_paged_target_reports_both_status_words():
    """A bad token id does not hide a bad page, before or after it; the page is reported once."""
    D = lib()
    _, dw = weights_on_gpu()
    shape = TARGET_TINY
    t = D.dflash_target_create_paged(shape.as_dict(), dw, pool(shape, 4, 16), table_of([0, 9, 2, 3]))
    fwd(D, t, [1, shape.vocab, 2], 0, shape)
    with pytest.raises(D.DFlashError) as e:
        D.dflash_target_device_status(t)
    assert "token id" in str(e.value) and "page" not in str(e.value)
    fwd(D, t, [1] * 20, 3, shape)
    with pytest.raises(D.DFlashError) as e:
        D.dflash_target_device_status(t)
    assert e.value.status == D.DFLASH_ERR_DEVICE and "page" in str(e.value) and "token id" in str(e.value)
    with pytest.raises(D.DFlashError) as e:
        D.dflash_target_device_status(t)
    assert "page" not in str(e.value)
