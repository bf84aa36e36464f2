"""Values that are not finite where a row sees them: the target-side
attention answers NaN (or an infinity) whatever the layout of the work, and
its rows beside them stay right.  What a row does not see never reaches it
(tests/test_gpu_target_ops.py); here is the other half."""
import math

import pytest
import torch

from oracle import target_ops_oracle as O
from tests.test_gpu_target_ops import DT, Batch, check_attention, i32, lib, ref_paged, run_paged

pytestmark = pytest.mark.gpu

# dtype, new rows, lengths, query heads: the bf16 calls run as a cluster, as ranges of one row tile, as whole items
# of two and as ranges of two; the fp32 ones as splits that meet in a cluster, in the workspace, and as row tiles
LAYOUTS = [("bf16", [16], [3000], 8), ("bf16", [1, 1, 1], [30011, 700, 16384], 8), ("bf16", [200, 90], [900, 700], 4),
           ("bf16", [300, 2, 150], [2100, 3000, 150], 8), ("f32", [8, 1], [1500, 300], 4), ("f32", [8, 1], [5000, 300], 4),
           ("f32", [90, 70], [700, 1100], 4)]
IDS = ["cluster", "ranges-1", "items", "ranges-2", "few-cluster", "few-workspace", "tiles"]


@pytest.mark.parametrize("layout", range(len(LAYOUTS)), ids=IDS)
@pytest.mark.parametrize("components", [1, 64])
def test_a_query_that_is_not_a_number(layout, components):
    """One head of some rows holds NaN (one component, or all): that head's output and lse are NaN, not the zeros
    and -inf of a row that sees no key; every other row is right."""
    dtype, rows, lens, hq = LAYOUTS[layout]
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=layout)
    ref = ref_paged(B, True, 0)
    n = B.starts[-1]
    hit = torch.zeros((n, hq), dtype=torch.bool)
    for b in range(len(rows)):
        hit[B.starts[b], 0] = hit[B.starts[b + 1] - 1, hq - 1] = True
    B.q[:n][hit] = torch.where(torch.arange(64) < components, math.nan, B.q[:n][hit].float()).to(DT[dtype])
    out, lse, _, _ = run_paged(B, True, 0)
    out, lse = out[:n].cpu(), lse[:n].cpu()
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    out, lse = out[~hit][:, None], lse[~hit][:, None]
    check_attention(out, lse, tuple(x[:n][~hit][:, None] for x in ref), out.shape[0])


@pytest.mark.parametrize("layout", range(len(LAYOUTS)), ids=IDS)
@pytest.mark.parametrize("which", ["first_half", "every_fourth_64"])
def test_a_part_of_the_keys_is_not_a_number(layout, which):
    """K of KV head 1 is NaN over whole parts of the key axis, finite elsewhere: every row of its query heads sees
    such a key and is NaN; the other head's rows are right."""
    dtype, rows, lens, hq = LAYOUTS[layout]
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=layout)
    ref = ref_paged(B, True, 0)
    n, half = B.starts[-1], hq // 2
    B.kp, B.vp = B.appended()
    for b, L in enumerate(lens):
        for p in range(L - rows[b] + 1):   # keys that the first new row sees too
            if (p < max(1, (L - rows[b]) // 2)) if which == "first_half" else p // 64 % 4 == (1 if L - rows[b] >= 64 else 0):
                B.kp[int(B.table[b, p // 16]), p % 16, 1] = math.nan
    out, lse, _, _ = run_paged(B, True, 0, append=False)
    assert bool(torch.isnan(out[:n, half:]).all()) and bool(torch.isnan(lse[:n, half:]).all())
    check_attention(out[:n, :half], lse[:n, :half], tuple(x[:n, :half] for x in ref), n)


@pytest.mark.parametrize("layout", range(len(LAYOUTS)), ids=IDS)
def test_scores_of_minus_infinity(layout):
    """Scores that overflow to -inf on a part of the keys have probability zero; where a row sees nothing else
    there is no distribution: NaN, and the log of an empty sum."""
    dtype, rows, lens, hq = LAYOUTS[layout]
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=layout)
    n, far = B.starts[-1], 3e38
    B.kp, B.vp = B.appended()
    B.q[:] = 1.0
    for b, L in enumerate(lens):
        for p in range(L):   # 64 x -3e38 is past the fp32 range; finite in fp64, where its exponential is 0 as well
            if b > 0 or p < (L - rows[b]) // 2:
                B.kp[int(B.table[b, p // 16]), p % 16] = -far
    s1 = B.starts[1]
    ref = O.attention(B.q[:s1], O.gather(B.kp, lens[:1], B.table), O.gather(B.vp, lens[:1], B.table), B.starts[:2],
                      lens[:1], True, 0, 0.125, dtype == "bf16")
    # (the oracle's bound takes its hidden weight's |q||k| along: here those keys count for nothing)
    near = B.kp.clone()
    near[near < -1e30] = -60.0
    tol = O.attention(B.q[:s1], O.gather(near, lens[:1], B.table), O.gather(B.vp, lens[:1], B.table), B.starts[:2],
                      lens[:1], True, 0, 0.125, dtype == "bf16")[2:]
    out, lse, _, _ = run_paged(B, True, 0, append=False)
    check_attention(out[:s1], lse[:s1], (*ref[:2], *tol), s1)
    assert bool(torch.isnan(out[s1:n]).all()) and bool(torch.isneginf(lse[s1:n]).all())


@pytest.mark.parametrize("layout", range(len(LAYOUTS)), ids=IDS)
@pytest.mark.parametrize("which", ["first_new", "last_cached", "first_half"])
def test_a_seen_value_whose_probability_underflows(layout, which):
    """V is NaN at a key that every row sees and whose probability is 0 in fp32 (its score is 256 below the
    others'): 0 x NaN is NaN in that column, in tiles with and without hidden keys and in parts of weight 0."""
    dtype, rows, lens, hq = LAYOUTS[layout]
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=layout)
    B.kp, B.vp = B.appended()
    B.q[:] = 8.0
    n = B.starts[-1]
    for b, L in enumerate(lens):
        first = L - rows[b]
        far = {"first_new": [first], "last_cached": [max(first - 1, 0)], "first_half": list(range(max(1, first // 2)))}[which]
        if first == 0 or (which == "first_new" and rows[b] == 1):
            far = []   # a row's only key, or no row beside it
        for p in range(L):
            pg, sl = int(B.table[b, p // 16]), p % 16
            B.kp[pg, sl] = -2.0 if p in far else 2.0
            if p in far[:1]:
                B.vp[pg, sl, :, 7] = math.nan
        rows_b = slice(B.starts[b], B.starts[b + 1])
        B.far = getattr(B, "far", torch.zeros(n, dtype=torch.bool))
        B.far[rows_b] = bool(far)
        if which == "first_new" and far:
            B.far[B.starts[b]] = False   # its own row may see nothing else
    fixed = B.vp.nan_to_num(0, 0, 0)
    ref = O.attention(B.q[:n], O.gather(B.kp, lens, B.table), O.gather(fixed, lens, B.table), B.starts, lens, True, 0,
                      0.125, dtype == "bf16")
    out, lse, _, _ = run_paged(B, True, 0, append=False)
    out, lse = out[:n].cpu(), lse[:n].cpu()
    assert bool(torch.isnan(out[B.far][..., 7]).all())
    keep = [c for c in range(64) if c != 7]
    check_attention(out[..., keep], lse, (ref[0][..., keep], ref[1], ref[2][..., keep], ref[3]), n)


def test_a_hidden_value_that_is_not_finite_in_a_long_cache():
    """15 chunks of 300 tokens as whole items over a million cached keys (one set of pages serves them all but for
    the last): the value of one new token is NaN. The rows in front of it are right, the ones that see it NaN, and
    the call takes no longer for it than its waits allow (status 0)."""
    D = lib()
    seqs, n, L, page, h, d = 15, 300, 1_000_000, 1024, 8, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    per = L // page + 1
    kp, vp = (torch.randn((per - 1 + seqs, page, h, d), device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn((seqs * n, h, d), device="cuda", generator=g).bfloat16()
    table = torch.arange(per, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    table[:, per - 1] += torch.arange(seqs, dtype=torch.int32, device="cuda")
    assert (L - n) // page == per - 1   # every sequence's new rows are in its own last page
    at = L - n + 255
    clean = vp[per - 1, at % page].clone()
    vp[per - 1, at % page, :, 9] = math.nan
    st, out, lse = i32([0]), torch.full_like(q, 7.0), torch.empty((seqs * n, h), device="cuda")
    D.dflash_paged_attention(q, kp, vp, i32([b * n for b in range(seqs + 1)]), i32([L] * seqs), table, out, max_rows=n,
                             max_len=L, lse=lse, status=st)
    assert int(st.item()) == 0
    assert bool(torch.isnan(out[255:n, :, 9]).all())
    assert int(torch.isnan(out).sum()) == (n - 255) * h
    vp[per - 1, at % page] = clean
    for head in (0, 7):
        k, v = (x[:per, :, head].reshape(-1, d)[:L].cpu().double() for x in (kp, vp))
        rows = torch.tensor([0, 127, 128, 254])
        ref = O.attention_row_block(q[:n][rows, head].cpu().double(), k, v, L - n + rows, L, True, 0, 0.125, True)
        check_attention(out[:n][rows, head][:, None], lse[:n][rows, head][:, None], tuple(x[:, None] for x in ref), 4)


@pytest.mark.parametrize("layout", range(4), ids=IDS[:4])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_infinities_beside_hidden_keys(layout, value):
    """V is infinite at every new key, in the column of its number: rows that see it answer that infinity there,
    all other columns and rows stay finite and right."""
    dtype, rows, lens, hq = LAYOUTS[layout]
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=layout)
    B.kp, B.vp = B.appended()
    ref = O.attention(B.q[:B.starts[-1]], O.gather(B.kp, lens, B.table), O.gather(B.vp, lens, B.table), B.starts, lens,
                      True, 0, 0.125, dtype == "bf16")
    seen = torch.zeros((B.starts[-1], 64), dtype=torch.bool)
    for b, (n, L) in enumerate(zip(rows, lens)):
        for i in range(min(n, 60)):
            p = L - n + i
            B.vp[int(B.table[b, p // 16]), p % 16, :, i] = value
            seen[B.starts[b] + i:B.starts[b + 1], i] = True
    out, lse, _, _ = run_paged(B, True, 0, append=False)
    out = out[:B.starts[-1]].cpu()
    hit = seen[:, None].expand_as(out)
    assert bool((out[hit] == value).all())
    out, o, tol = (torch.where(hit, 0.0, x.double()) for x in (out, ref[0], ref[2]))
    check_attention(out, lse, (o, ref[1], tol, ref[3]), B.starts[-1])
