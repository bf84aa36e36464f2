"""The target on a paged cache (dflash_target_create_paged): the target-side
operators run together as a server would run them: prompts, verified blocks
and rollbacks of several sequences over one pool of pages, and the log
probabilities of what was decoded."""
import math

import numpy as np
import pytest
import torch

import synthetic as S
from oracle import target_ops_oracle as O
from oracle.target_oracle import OracleTarget
from synthetic.target import TARGET_TINY, TargetShape, make_target_weights
from tests.gpu_util import Pair, lib

pytestmark = pytest.mark.gpu


def weights_on_gpu(seed=1, shape=TARGET_TINY):
    w = make_target_weights(seed, shape)
    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return w, dict(embed=f32(w["embed"]), unembed=f32(w["unembed"]), final_norm=f32(w["final_norm"]),
                   layers=[{k: f32(v) for k, v in lw.items()} for lw in w["layers"]])


def pool(shape, n_pages, page):
    """NaN everywhere: a row that nobody wrote would show."""
    f = lambda: torch.full((n_pages, page, shape.n_heads, shape.head_dim), math.nan, device="cuda")
    return [(f(), f()) for _ in range(shape.n_layers)]


def table_of(pages):
    return torch.tensor(pages, dtype=torch.int32, device="cuda")


def fwd(D, t, tokens, start, shape):
    tok = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    lg = torch.empty((len(tokens), shape.vocab), device="cuda")
    tp = torch.empty((len(tokens), shape.n_taps * shape.hidden), device="cuda")
    D.dflash_target_forward(t, tok, start, lg, tp)
    torch.cuda.synchronize()
    return lg.cpu().numpy(), tp.cpu().numpy()


def close(g, r, tol):
    assert np.all(np.abs(g - r) <= tol * np.maximum(1.0, np.abs(r))), float(np.max(np.abs(g - r)))


@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("shape", [TARGET_TINY, TargetShape(hidden=96, n_heads=6, head_dim=20, intermediate=64, vocab=50,
                                                            n_layers=3)])
def test_two_sequences_share_a_pool(page, shape):
    """Interleaved prompts (one longer than a forward's internal chunk), blocks and trims of two targets on
    interleaved pages; logits and taps within the target's bar, 1e-4."""
    D = lib()
    w, dw = weights_on_gpu(3, shape)
    n = 256 // page
    cache = pool(shape, 2 * n, page)
    seqs = []
    for b in range(2):
        t = D.dflash_target_create_paged(shape.as_dict(), dw, cache, table_of(list(range(b, 2 * n, 2))))
        seqs.append((t, OracleTarget(w, shape)))
    rng = S.rng_for(0, "paged")
    plan = [(0, 150, 0, None), (1, 5, 0, None), (0, 8, 150, 153), (1, 16, 5, 9), (0, 1, 153, None), (1, 70, 9, None),
            (0, 8, 154, None)]
    for b, rows, start, trim in plan:
        t, ref = seqs[b]
        tokens = [int(x) for x in rng.integers(0, shape.vocab, size=rows)]
        lg, tp = fwd(D, t, tokens, start, shape)
        rl, rt = ref.forward(tokens, start)
        close(lg, rl, 1e-4)
        close(tp, rt, 1e-4)
        if trim is not None:
            D.dflash_target_trim(t, trim)
            ref.trim(trim)
        D.dflash_target_device_status(t)


def test_blocks_and_single_tokens_give_the_same_bits():
    """The paged target passes the block-versus-chain gate at the start, across a page, a tile and a split
    of the key axis: no logit byte differs."""
    D = lib()
    _, dw = weights_on_gpu()
    shape = TARGET_TINY
    cache = pool(shape, 40, 16)
    t = D.dflash_target_create_paged(shape.as_dict(), dw, cache, table_of(list(range(39, -1, -1))))
    rng = S.rng_for(1, "chain")
    length = 0
    for start in (0, 13, 60, 250, 507):
        while length < start:
            rows = start - length
            fwd(D, t, [int(x) for x in rng.integers(0, shape.vocab, size=rows)], length, shape)
            length = start
        tok = torch.from_numpy(rng.integers(0, shape.vocab, size=9).astype(np.int32)).cuda()
        a, b = torch.empty((9, shape.vocab), device="cuda"), torch.empty((9, shape.vocab), device="cuda")
        rec = torch.empty(9 * D.EXACTNESS_ROW_BYTES, dtype=torch.uint8, device="cuda")
        s = D.dflash_target_exactness_probe(t, tok, start, a, b, rec)
        assert s["differing_bytes"] == 0 and s["allows"] == 1, (start, s)


def test_a_bad_page_is_reported_and_capacity_is_refused():
    D = lib()
    _, dw = weights_on_gpu()
    shape = TARGET_TINY
    cache = pool(shape, 4, 16)
    t = D.dflash_target_create_paged(shape.as_dict(), dw, cache, table_of([0, 9, 2, 3]))
    fwd(D, t, [1] * 20, 0, shape)
    with pytest.raises(D.DFlashError) as e:
        D.dflash_target_device_status(t)
    assert e.value.status == D.DFLASH_ERR_DEVICE and "page" in str(e.value)
    with pytest.raises(D.DFlashError) as e:
        fwd(D, t, [1] * 45, 20, shape)
    assert e.value.status == D.DFLASH_ERR_CAPACITY
    with pytest.raises(D.DFlashError) as e:
        D.dflash_target_create_paged(shape.as_dict(), dw, cache, table_of([0, 1]), max_ctx=33)
    assert e.value.status == D.DFLASH_ERR_CAPACITY
    wrong = [(k[..., :32], v[..., :32]) for k, v in cache]
    with pytest.raises(D.DFlashError) as e:
        D.dflash_target_create_paged(shape.as_dict(), dw, wrong, table_of([0, 1]))
    assert e.value.status == D.DFLASH_ERR_SHAPE


def test_speculative_decode_on_pages_with_log_probabilities():
    """Draft and paged target on the GPU: greedy speculative decoding equals plain greedy decoding of the
    CPU target, and the decoded tokens' log probabilities, entropies and alternatives equal the oracle's on
    the same logits."""
    D = lib()
    cfg, shape = S.CONFIGS["tiny_fp32"], TARGET_TINY
    w, dw = weights_on_gpu()
    pair = Pair(cfg)
    cache = pool(shape, 24, 16)
    t = D.dflash_target_create_paged(shape.as_dict(), dw, cache, table_of(list(np.random.default_rng(0).permutation(24))))
    sess = D.dflash_open(pair.model, max_ctx=512)
    prompt = [int(x) for x in S.rng_for(0, "prompt").integers(0, shape.vocab, size=70)]
    plain = OracleTarget(w, shape)
    lg, _ = plain.forward(prompt, 0)
    want, cur = [], int(np.argmax(lg[-1]))
    for i in range(64):
        want.append(cur)
        lg, _ = plain.forward([cur], 70 + i)
        cur = int(np.argmax(lg[-1]))
    lg, tp = fwd(D, t, prompt, 0, shape)
    D.dflash_committed(sess, torch.from_numpy(tp).cuda(), 0)
    got, pos, cur, rnd = [], 70, int(np.argmax(lg[-1])), 0
    n = cfg.block_size - 1
    acc = torch.empty(1, dtype=torch.int32, device="cuda")
    bon = torch.empty(1, dtype=torch.int32, device="cuda")
    tok = torch.empty((1, n), dtype=torch.int32, device="cuda")
    q = torch.empty((1, n), device="cuda")
    while len(got) < 64:
        D.dflash_propose([sess], torch.tensor([cur], dtype=torch.int32, device="cuda"), n, 0.0, 0, rnd, tok, q)
        block = torch.cat([torch.tensor([cur], dtype=torch.int32, device="cuda"), tok[0]])
        logits = torch.empty((n + 1, shape.vocab), device="cuda")
        taps = torch.empty((n + 1, shape.n_taps * shape.hidden), device="cuda")
        D.dflash_target_forward(t, block, pos, logits, taps)
        D.dflash_verify([sess], logits[None], tok, n, 0.0, 0, rnd, acc, bon)
        a, bonus = int(acc.item()), int(bon.item())
        # row r of the block scores the token after it: the accepted ones, then the bonus
        given = torch.cat([tok[0, :a], bon]).contiguous()
        lp, ent = torch.empty(a + 1, device="cuda"), torch.empty(a + 1, device="cuda")
        ids = torch.empty((a + 1, 5), dtype=torch.int32, device="cuda")
        tlp = torch.empty((a + 1, 5), device="cuda")
        D.dflash_token_logprobs(logits[:a + 1], given, lp, ent, ids, tlp)
        rlp, rent, rids, rtlp, t_lp, t_ent, t_top = O.logprobs(logits[:a + 1].cpu(), given.cpu(), 5, 1.0)
        assert bool(((lp.double().cpu() - rlp).abs() <= t_lp).all())
        assert bool(((ent.double().cpu() - rent).abs() <= t_ent).all())
        assert torch.equal(ids.cpu().long(), rids) and bool(((tlp.double().cpu() - rtlp).abs() <= t_top).all())
        assert torch.equal(ids[:, 0].cpu(), given.cpu())     # greedy: the given token is the first alternative
        got += [cur] + [int(x) for x in tok[0, :a].cpu()]
        D.dflash_target_trim(t, pos + a + 1)
        D.dflash_committed(sess, taps[:a + 1], pos)
        pos, cur, rnd = pos + a + 1, bonus, rnd + 1
    D.dflash_target_device_status(t)
    assert got[:64] == want
