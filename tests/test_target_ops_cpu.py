"""The target-side operators' refusals and host arithmetic, without a GPU: every
bad argument is answered with a status before any device work, and the binding
refuses tensors that the library would read or write out of bounds."""
import ctypes as C
import math
import os
import re

import pytest
import torch

import block_diffusion_speculative_flush_gb300 as D
from block_diffusion_speculative_flush_gb300 import _abi
from oracle import target_ops_oracle as O

INVALID, SHAPE = _abi.DFLASH_ERR_INVALID_ARG, _abi.DFLASH_ERR_SHAPE
BASE = 4096   # stands for an aligned device pointer; refused calls never look at it


def pages(**kw):
    f = dict(dtype=1, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, k=BASE, v=BASE, page_stride=2048,
             slot_stride=128, head_stride=64)
    f.update(kw)
    return _abi.dflash_kv_pages(**f)


def batch(**kw):
    f = dict(batch=2, total_rows=8, max_rows=4, max_len=100, starts=BASE, lens=BASE, table=BASE, table_width=7,
             table_stride=7, status=None)
    f.update(kw)
    return _abi.dflash_ragged(**f)


def heads(data=BASE, row=256, head=64):
    return _abi.dflash_heads(data, row, head)


def attention(**kw):
    f = dict(dtype=1, n_q_heads=4, n_kv_heads=2, head_dim=64, causal=1, window=0, scale=0.125, q=heads(),
             out=heads(2 * BASE), lse=None, workspace=None, workspace_bytes=0)
    f.update(kw)
    return _abi.dflash_attention(**f)


PAGES = [(dict(dtype=2), INVALID), (dict(n_kv_heads=0), SHAPE), (dict(head_dim=96), SHAPE),
         (dict(dtype=0, head_dim=66), SHAPE), (dict(dtype=0, head_dim=132), SHAPE), (dict(page_size=12), SHAPE),
         (dict(page_size=4), SHAPE), (dict(page_size=2048), SHAPE), (dict(n_pages=0), SHAPE),
         (dict(n_pages=1 << 31), SHAPE), (dict(k=None), INVALID), (dict(v=BASE + 2), INVALID),
         (dict(page_stride=2044), INVALID), (dict(slot_stride=32), INVALID), (dict(head_stride=8), INVALID),
         (dict(slot_stride=-128), INVALID)]
BATCHES = [dict(batch=0), dict(batch=32769), dict(total_rows=-1), dict(total_rows=(1 << 30) + 1), dict(max_rows=0),
           dict(max_rows=(1 << 24) + 1), dict(starts=None), dict(lens=None), dict(table=None), dict(max_len=0),
           dict(max_len=(1 << 30) + 1), dict(table_width=0), dict(table_stride=6)]
ATTENTION = [(dict(dtype=5), INVALID), (dict(n_q_heads=3), SHAPE), (dict(n_q_heads=0), SHAPE),
             (dict(n_q_heads=258), SHAPE), (dict(head_dim=32), SHAPE), (dict(causal=2), INVALID),
             (dict(window=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
             (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(q=heads(None)), INVALID),
             (dict(q=heads(BASE + 8)), INVALID), (dict(q=heads(row=250)), INVALID), (dict(q=heads(head=32)), INVALID),
             (dict(q=heads(row=32)), INVALID), (dict(out=heads(BASE)), INVALID), (dict(out=heads(None)), INVALID)]


@pytest.mark.parametrize("bad,code", PAGES)
def test_bad_pages_are_refused(bad, code):
    p, b, h, a = pages(**bad), batch(), heads(), attention()
    assert D.lib.dflash_kv_append(C.byref(p), C.byref(b), C.byref(h), C.byref(h), None) == code
    assert D.lib.dflash_paged_attention(C.byref(a), C.byref(b), C.byref(p), None) == code
    assert D.lib.dflash_last_error()


@pytest.mark.parametrize("bad", BATCHES)
def test_bad_batches_are_refused(bad):
    p, b, h, a = pages(), batch(**bad), heads(), attention()
    assert D.lib.dflash_kv_append(C.byref(p), C.byref(b), C.byref(h), C.byref(h), None) == INVALID
    assert D.lib.dflash_paged_attention(C.byref(a), C.byref(b), C.byref(p), None) == INVALID
    if not set(bad) & {"lens", "table", "max_len", "table_width", "table_stride"}:
        assert D.lib.dflash_prompt_attention(C.byref(a), C.byref(b), C.byref(h), C.byref(h), None) == INVALID


@pytest.mark.parametrize("bad,code", ATTENTION)
def test_bad_attention_is_refused(bad, code):
    p, b, h, a = pages(), batch(), heads(), attention(**bad)
    assert D.lib.dflash_paged_attention(C.byref(a), C.byref(b), C.byref(p), None) == code
    assert D.lib.dflash_prompt_attention(C.byref(a), C.byref(b), C.byref(h), C.byref(h), None) == code


def test_a_scale_that_overflows_in_the_exp2_domain_is_refused():
    p, b, h = pages(), batch(total_rows=0), heads()
    for scale, code in ((2.2e38, 0), (2.4e38, INVALID), (3.4e38, INVALID)):
        a = attention(scale=scale)
        assert D.lib.dflash_paged_attention(C.byref(a), C.byref(b), C.byref(p), None) == code
        assert D.lib.dflash_prompt_attention(C.byref(a), C.byref(b), C.byref(h), C.byref(h), None) == code


def test_null_and_mismatched_arguments_are_refused():
    p, b, h, a = pages(), batch(), heads(), attention()
    r = C.byref
    assert D.lib.dflash_kv_append(None, r(b), r(h), r(h), None) == INVALID
    assert D.lib.dflash_kv_append(r(p), None, r(h), r(h), None) == INVALID
    assert D.lib.dflash_kv_append(r(p), r(b), None, r(h), None) == INVALID
    assert D.lib.dflash_kv_append(r(p), r(b), r(h), r(heads(BASE + 4)), None) == INVALID
    assert D.lib.dflash_paged_attention(None, r(b), r(p), None) == INVALID
    assert D.lib.dflash_paged_attention(r(a), r(b), None, None) == INVALID
    assert D.lib.dflash_prompt_attention(r(a), r(b), None, r(h), None) == INVALID
    assert D.lib.dflash_prompt_attention(r(a), r(b), r(h), r(heads(row=8)), None) == INVALID
    assert D.lib.dflash_paged_attention(r(attention(dtype=0)), r(b), r(p), None) == SHAPE
    assert D.lib.dflash_paged_attention(r(attention(n_kv_heads=4)), r(b), r(p), None) == SHAPE
    assert D.lib.dflash_status_check(None, None) == INVALID
    assert D.lib.dflash_attention_workspace(None, r(b), None) == INVALID
    assert D.lib.dflash_attention_workspace(r(a), r(batch(batch=0)), r(p)) == INVALID


def test_empty_batches_are_no_work():
    p, b, h = pages(), batch(total_rows=0), heads(None)
    a = attention(q=heads(None), out=heads(None))
    assert D.lib.dflash_kv_append(C.byref(p), C.byref(b), C.byref(h), C.byref(h), None) == 0
    assert D.lib.dflash_paged_attention(C.byref(a), C.byref(b), C.byref(p), None) == 0
    assert D.lib.dflash_prompt_attention(C.byref(a), C.byref(b), C.byref(h), C.byref(h), None) == 0


def test_a_call_that_needs_a_workspace_is_refused_without_one():
    p, b = pages(dtype=0, head_stride=64, slot_stride=128), batch(max_len=100)
    f = dict(dtype=0, q=heads(row=256), out=heads(2 * BASE, row=256))
    b.max_len, b.table_width, b.table_stride = 4000, 300, 300
    need = D.lib.dflash_attention_workspace(C.byref(attention(**f)), C.byref(b), C.byref(p))
    assert need > 0
    for ws, n in ((None, 0), (BASE, need - 1), (BASE + 8, need)):
        a = attention(workspace=ws, workspace_bytes=n, **f)
        assert D.lib.dflash_paged_attention(C.byref(a), C.byref(b), C.byref(p), None) == INVALID


def test_a_paged_target_refuses_bad_pages():
    cfg = _abi.dflash_target_config(hidden=256, n_heads=4, head_dim=64, intermediate=512, vocab=32, n_layers=1,
                                    rope_theta=1e6, rms_eps=1e-6)
    w, out = _abi.dflash_target_weights(embed=16, unembed=16, final_norm=16), C.c_void_p()
    good = dict(dtype=0, n_kv_heads=4, head_dim=64, page_stride=4096, slot_stride=256, head_stride=64)

    def call(p, table=BASE, width=8, max_ctx=64, config=cfg):
        return D.lib.dflash_target_create_paged(C.byref(config), C.byref(w), C.byref(p), table, width, max_ctx, None,
                                                C.byref(out))
    for bad, code in PAGES:
        if "dtype" not in bad and "head_dim" not in bad and "n_kv_heads" not in bad:
            assert call(pages(**{**good, **bad})) == code, bad
    for bad in (dict(dtype=1, head_dim=64), dict(n_kv_heads=2), dict(head_dim=32)):
        assert call(pages(**{**good, **bad})) == SHAPE, bad
    assert call(pages(**good), table=None) == INVALID
    assert call(pages(**good), width=0) == INVALID
    assert call(pages(**good), max_ctx=129) == _abi.DFLASH_ERR_CAPACITY
    assert call(pages(**good)) == INVALID                      # no layer weights: refused as any target's
    assert D.lib.dflash_target_create_paged(C.byref(cfg), C.byref(w), None, BASE, 8, 64, None, C.byref(out)) == INVALID
    assert out.value is None


def logprobs(**kw):
    f = dict(logits=BASE, row_stride=1000, dtype=0, rows=3, vocab=1000, top=5, temperature=1.0, tokens=BASE,
             logprobs=BASE, entropy=None, top_ids=BASE, top_logprobs=BASE, status=None)
    f.update(kw)
    return _abi.dflash_logprobs(**f)


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 24) + 1),
                                 dict(row_stride=999), dict(top=-1), dict(top=33), dict(vocab=4), dict(temperature=0.0),
                                 dict(temperature=math.nan), dict(temperature=math.inf), dict(logits=None),
                                 dict(logits=BASE + 2), dict(tokens=None), dict(logprobs=None), dict(top_ids=None),
                                 dict(top_logprobs=None)])
def test_bad_logprobs_are_refused(bad):
    assert D.lib.dflash_token_logprobs(C.byref(logprobs(**bad)), None) == INVALID


def test_logprobs_null_and_empty():
    assert D.lib.dflash_token_logprobs(None, None) == INVALID
    assert D.lib.dflash_token_logprobs(C.byref(logprobs(rows=0, logits=None, tokens=None)), None) == 0


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    f = lambda *s: torch.zeros(s)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        D.dflash_kv_append(f(4, 2, 64), f(4, 2, 64), f(3, 16, 2, 64), f(3, 16, 2, 64), i(2), i(1), i(1, 3))
    with pytest.raises(ValueError):
        D.dflash_paged_attention(f(4, 4, 64), f(3, 16, 2, 64), f(3, 16, 2, 64), i(2), i(1), i(1, 3), f(4, 4, 64), 4)
    with pytest.raises(ValueError):
        D.dflash_prompt_attention(f(4, 4, 64), f(4, 2, 64), f(4, 2, 64), i(2), f(4, 4, 64), 4)
    with pytest.raises(ValueError):
        D.dflash_prompt_attention(f(4, 4, 64), f(5, 2, 64), f(5, 2, 64), i(2), f(4, 4, 64), 4)
    with pytest.raises(ValueError):
        D.dflash_token_logprobs(f(4, 100), i(4), f(4))
    with pytest.raises(ValueError):
        D.dflash_status_check(i(1))


def test_a_paged_target_refuses_pages_and_tables_of_another_device(monkeypatch):
    """The kernels would read them through this device's pointers."""
    class On:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    class Reached(Exception):
        pass

    def reached(*a):
        raise Reached
    monkeypatch.setattr(D, "_target_args", lambda cfg, weights: (None, None, [], []))
    monkeypatch.setattr(D, "_pages", reached)
    call = lambda w, k, v, t: D.dflash_target_create_paged(dict(n_layers=1), dict(embed=On(w)), [(On(k), On(v))], On(t))
    for bad in ((0, 0, 0, 1), (0, 1, 0, 0), (0, 0, 1, 0), (1, 0, 0, 0), (-1, -1, -1, -1)):
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(Reached):
        call(1, 1, 1, 1)


def test_the_packed_layouts_are_the_structs():
    for name, struct, n in (("PACK_HEADS", _abi.dflash_heads, 3), ("PACK_PAGES", _abi.dflash_kv_pages, 10),
                            ("PACK_RAGGED", _abi.dflash_ragged, 10), ("PACK_LOGPROBS", _abi.dflash_logprobs, 13)):
        values = list(range(1, n + 1))
        assert getattr(_abi, name)(*values) == bytes(struct(*values))
    h = _abi.dflash_heads(8, 9, 10)
    want = bytes(_abi.dflash_attention(1, 2, 3, 4, 5, 6, 7.0, h, h, 14, 15, 16))
    got = _abi.PACK_ATTENTION(1, 2, 3, 4, 5, 6, 7.0, 8, 9, 10, 8, 9, 10, 14, 15, 16)
    assert len(got) == len(want) and _abi.dflash_attention.from_buffer_copy(got).workspace_bytes == 16
    f = _abi.dflash_attention.from_buffer_copy(got)
    assert (f.dtype, f.window, f.scale, f.q.data, f.out.head_stride, f.lse, f.workspace) == (1, 6, 7.0, 8, 10, 14, 15)


def test_oracle_attention_by_hand():
    """Two keys, one query: the weights are the logistic function of the score difference."""
    q = torch.tensor([[[2.0, 0.0]]])
    k, v = torch.tensor([[[1.0, 0.0]], [[0.0, 5.0]]]), torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]]])
    o, lse, _, _ = O.attention(q, [k], [v], [0, 1], [2], True, 0, 0.5, False)
    w = 1 / (1 + math.exp(-1.0))
    assert torch.allclose(o[0, 0], torch.tensor([w, 1 - w], dtype=torch.float64))
    assert abs(float(lse[0, 0]) - math.log(math.e + 1)) < 1e-12
    o, lse, _, _ = O.attention(q, [k], [v], [0, 1], [2], True, 1, 0.5, False)   # the window leaves the second key
    assert torch.allclose(o[0, 0], torch.tensor([0.0, 1.0], dtype=torch.float64)) and float(lse[0, 0]) == 0.0


def test_oracle_logprobs_by_hand():
    x = torch.tensor([[0.0, math.log(3.0), -math.inf, 0.0]])
    lp, ent, ids, tlp, *_ = O.logprobs(x, torch.tensor([1]), 4, 1.0)
    assert abs(float(lp[0]) - math.log(0.6)) < 1e-7
    assert abs(float(ent[0]) + 0.6 * math.log(0.6) + 0.4 * math.log(0.2)) < 1e-7
    assert ids[0].tolist() == [1, 0, 3, 2] and math.isinf(float(tlp[0, 3]))


CSRC = os.path.join(os.path.dirname(D.__file__), "csrc")
# read-only loads of these are right: weights, and tables that the host copied before the first launch
CONSTANT = {"E", "W", "rope"}


def kernels(source):
    """(name, parameters, body) of every __global__ function of a file."""
    text = open(os.path.join(CSRC, source)).read()
    for m in re.finditer(r"__global__ void (?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s+)?(\w+)\(", text):
        end = text.index(") {\n", m.end())
        yield m.group(1), text[m.end():end], text[end:text.index("\n}\n", end)]


@pytest.mark.parametrize("source", ["ragged_attention.cu", "ragged_attention_tc.cu", "token_logprobs.cu", "target.cu"])
def test_kernels_read_a_predecessors_rows_after_their_wait(source):
    """A kernel starts while its predecessor still runs: what that one may write is never behind a const
    __restrict__ pointer (which permits read-only loads, and loads before the wait) unless the pointer passes
    through after_wait."""
    found = list(kernels(source))
    assert found
    for name, params, body in found:
        for p in re.findall(r"const [\w:]+\* __restrict__ (\w+)", params):
            assert p in CONSTANT or f"{p} = after_wait({p})" in body, (name, p)
