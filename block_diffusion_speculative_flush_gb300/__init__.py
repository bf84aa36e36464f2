"""Python binding of the GB300-native DFlash draft round (libdflash.so).

Each function has the name of the C entry point it marshals and does nothing
else: tensors become device pointers, lists of sessions become host arrays,
negative status codes become DFlashError.  Every step of the round runs in
the CUDA library; if the library is missing, importing this package fails.

PyTorch is used only for device memory (the tensors passed in) and streams.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _abi
from ._abi import (DFLASH_DTYPE_BF16, DFLASH_DTYPE_F32, DFLASH_ERR_CAPACITY, DFLASH_ERR_CONTEXT_GAP,
                   DFLASH_ERR_CUDA, DFLASH_ERR_DEVICE, DFLASH_ERR_INVALID_ARG, DFLASH_ERR_OOM, DFLASH_ERR_SHAPE,
                   DFLASH_ERR_STATE, DFLASH_FLAG_SIMT_GEMM, DFLASH_OK, DFLASH_PENDING_FLUSH_TOKENS,
                   DFLASH_VARIANT_DFLASH, DFLASH_VARIANT_DFLASH2, DFLASH2_DEPTH)

lib = _abi.load()

__all__ = [
    "DFlashError", "Model", "Session", "lib", "torch_dtype",
    "dflash_model_create", "dflash_model_destroy", "dflash_draft_limit", "dflash_device_status", "dflash_open",
    "dflash_committed", "dflash_committed_taps", "dflash_flush", "dflash_settle", "dflash_commit_block", "dflash_propose", "dflash_verify",
    "dflash_close", "dflash_set_sampler", "dflash_set_penalties", "dflash_candidates", "dflash_committed_batch", "dflash_stats", "dflash_session_state", "dflash_kv_export", "dflash_kv_import",
    "dflash_version", "dflash_last_error", "dflash_timing_enable", "dflash_timing_read", "dflash_verify_noalloc",
    "Target", "dflash_target_create", "dflash_target_destroy", "dflash_target_forward", "dflash_target_trim",
    "dflash_target_length", "dflash_target_argmax", "dflash_target_device_status",
    "dflash_logits_compare", "dflash_exactness_summarize", "dflash_target_exactness_probe", "exactness_rows",
    "dflash_target_create_paged", "dflash_kv_append", "dflash_paged_attention", "dflash_prompt_attention", "dflash_attention_workspace",
    "dflash_token_logprobs", "dflash_status_check",
    "RopeTable", "dflash_rope_table", "dflash_rope", "dflash_kv8_append", "dflash_kv8_attention",
    "dflash_kv8_attention_workspace", "PageBuffers", "dflash_page_buffers", "dflash_pages_copy", "dflash_pages_reorder",
    "dflash_pages_resize", "dflash_pages_compact",
]


class DFlashError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"dflash status {status}: {message}")
        self.status = status


def _check(rc: int) -> int:
    if rc < 0:
        raise DFlashError(rc, lib.dflash_last_error().decode(errors="replace"))
    return rc


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def torch_dtype(cfg) -> torch.dtype:
    return torch.bfloat16 if cfg.dtype == "bf16" else torch.float32


class Model:
    """Handle of a dflash_model; keeps the weight tensors alive."""

    def __init__(self, handle: int, cfg, tensors: dict, layer_structs):
        self.handle = handle
        self.cfg = cfg
        self._tensors = tensors
        self._layers = layer_structs

    def __del__(self):
        if getattr(self, "handle", None):
            lib.dflash_model_destroy(self.handle)
            self.handle = None


class Session:
    def __init__(self, handle: int, model: Model):
        self.handle = handle
        self.model = model


def _sessions(sessions):
    if isinstance(sessions, Session):
        sessions = [sessions]
    arr = (C.c_void_p * len(sessions))(*[s.handle for s in sessions])
    return arr, len(sessions)


def _need(t, dtypes, numel: int, what: str) -> None:
    """The library reads or writes numel elements of t from its data pointer:
    t must be a contiguous CUDA tensor of one of dtypes with at least that many."""
    if t is None:
        return
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if not t.is_cuda or t.dtype not in dtypes or not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{what}: a contiguous CUDA tensor of {'/'.join(str(d) for d in dtypes)} with at least "
                         f"{numel} elements")


def _model_of(sessions):
    first = sessions if isinstance(sessions, Session) else sessions[0]
    return first.model


def dflash_version() -> int:
    return lib.dflash_version()


def dflash_last_error() -> str:
    return lib.dflash_last_error().decode(errors="replace")


def dflash_model_create(cfg, weights: dict, flags: int = 0) -> Model:
    """cfg: an object with the fields of synthetic.DraftConfig; weights: name ->
    CUDA tensor in the storage type (names as synthetic.weight_shapes)."""
    c = _abi.dflash_config(
        dtype=DFLASH_DTYPE_BF16 if cfg.dtype == "bf16" else DFLASH_DTYPE_F32, n_taps=cfg.n_taps,
        target_hidden=cfg.target_hidden, hidden=cfg.hidden, n_layers=cfg.n_layers, n_q_heads=cfg.n_q_heads,
        n_kv_heads=cfg.n_kv_heads, head_dim=cfg.head_dim, intermediate=cfg.intermediate, vocab=cfg.vocab,
        block_size=cfg.block_size, mask_token=cfg.mask_token, window=cfg.window,
        causal_block=int(cfg.causal_block), gated_attention=int(cfg.gated_attention), flags=flags,
        rope_theta=cfg.rope_theta, rms_eps=cfg.rms_eps,
        variant=DFLASH_VARIANT_DFLASH2 if getattr(cfg, "variant", "dflash") == "dflash2" else DFLASH_VARIANT_DFLASH,
        conv_taps=getattr(cfg, "conv_taps", 0), sel_rank=getattr(cfg, "sel_rank", 0),
        sel_candidates=getattr(cfg, "sel_candidates", 0))
    t = {k: v.contiguous() for k, v in weights.items()}
    layers = (_abi.dflash_layer_weights * cfg.n_layers)()
    for l in range(cfg.n_layers):
        p = f"layers.{l}."
        g = t.get(p + "w_g")
        layers[l] = _abi.dflash_layer_weights(
            _ptr(t[p + "in_norm"]), _ptr(t[p + "w_qkv"]), _ptr(t[p + "q_norm"]), _ptr(t[p + "k_norm"]), _ptr(g),
            _ptr(t[p + "w_o"]), _ptr(t[p + "post_norm"]), _ptr(t[p + "w_gate"]), _ptr(t[p + "w_up"]),
            _ptr(t[p + "w_down"]), _ptr(t.get(p + "conv_norm")), _ptr(t.get(p + "w_dc")))
    w = _abi.dflash_weights(_ptr(t["aux_norms"]), _ptr(t["w_fc"]), _ptr(t["hidden_norm"]), _ptr(t["final_norm"]),
                            _ptr(t["embed"]), _ptr(t["unembed"]), layers, _ptr(t.get("sel_prev")),
                            _ptr(t.get("sel_next")))
    out = C.c_void_p()
    _check(lib.dflash_model_create(C.byref(c), C.byref(w), C.byref(out)))
    return Model(out.value, cfg, t, layers)


def dflash_model_destroy(model: Model) -> None:
    if model.handle:
        _check(lib.dflash_model_destroy(model.handle))
        model.handle = None


def dflash_draft_limit(model: Model) -> int:
    return _check(lib.dflash_draft_limit(model.handle))


def dflash_device_status(model: Model) -> None:
    _check(lib.dflash_device_status(model.handle))


def dflash_open(model: Model, restored_offset: int = 0, max_ctx: int = 4096, stream=None) -> Session:
    if stream is None:
        stream = torch.cuda.current_stream()
    out = C.c_void_p()
    _check(lib.dflash_open(model.handle, restored_offset, max_ctx, C.c_void_p(stream.cuda_stream), C.byref(out)))
    return Session(out.value, model)


def dflash_committed(session: Session, features: torch.Tensor, position: int) -> None:
    """features: CUDA tensor [n_rows, K*H_t] (row stride from the tensor)."""
    if features.dim() != 2 or features.stride(1) != 1:
        raise ValueError("features must be 2-D with unit column stride")
    cfg = session.model.cfg
    if not features.is_cuda or features.dtype != torch_dtype(cfg) or features.shape[1] != cfg.feature_width:
        raise ValueError(f"features: CUDA {torch_dtype(cfg)} rows of width {cfg.feature_width}")
    _check(lib.dflash_committed(session.handle, _ptr(features), features.stride(0), features.shape[0], position))


def dflash_committed_taps(session: Session, taps, position: int) -> None:
    """taps: n_taps CUDA tensors [n_rows, H_t] (unit column stride, one row stride for all)."""
    cfg = session.model.cfg
    taps = list(taps)
    if len(taps) != cfg.n_taps:
        raise ValueError(f"{cfg.n_taps} taps expected")
    rows, stride = taps[0].shape[0], taps[0].stride(0)
    for t in taps:
        if t.dim() != 2 or t.stride(1) != 1 or not t.is_cuda or t.dtype != torch_dtype(cfg) or \
                t.shape != (rows, cfg.target_hidden) or t.stride(0) != stride:
            raise ValueError(f"taps: CUDA {torch_dtype(cfg)} [{rows}, {cfg.target_hidden}] with one row stride")
    arr = (C.c_void_p * len(taps))(*[t.data_ptr() for t in taps])
    _check(lib.dflash_committed_taps(session.handle, arr, stride, rows, position))


def dflash_committed_batch(sessions, features, positions) -> None:
    """features: one CUDA tensor [n_rows_b, K*H_t] per session (one row stride
    for all); positions: the committed run's position per session.  Sessions
    that reach the flush threshold flush in one batched forward."""
    arr, b = _sessions(sessions)
    features, positions = list(features), [int(x) for x in positions]
    if len(features) != b or len(positions) != b:
        raise ValueError("one features tensor and one position per session")
    cfg = _model_of(sessions).cfg
    stride = features[0].stride(0)
    for f in features:
        if f.dim() != 2 or f.stride(1) != 1 or not f.is_cuda or f.dtype != torch_dtype(cfg) or \
                f.shape[1] != cfg.feature_width or (f.shape[0] > 1 and f.stride(0) != stride):
            raise ValueError(f"features: CUDA {torch_dtype(cfg)} rows of width {cfg.feature_width}, one row stride")
    ptrs = (C.c_void_p * b)(*[f.data_ptr() for f in features])
    rows = (C.c_int32 * b)(*[f.shape[0] for f in features])
    pos = (C.c_int64 * b)(*positions)
    _check(lib.dflash_committed_batch(arr, b, ptrs, stride, rows, pos))


def dflash_flush(sessions) -> None:
    arr, n = _sessions(sessions)
    _check(lib.dflash_flush(arr, n))


def dflash_settle(session: Session) -> None:
    _check(lib.dflash_settle(session.handle))


def dflash_commit_block(sessions) -> None:
    arr, n = _sessions(sessions)
    _check(lib.dflash_commit_block(arr, n))


def dflash_propose(sessions, current: torch.Tensor, max_tokens: int, temperature: float, seed: int, rnd: int,
                   out_tokens: torch.Tensor, out_q: torch.Tensor, out_logits: torch.Tensor | None = None) -> list:
    """Returns out_n per session (0 where the pages return nil)."""
    arr, n = _sessions(sessions)
    cfg = _model_of(sessions).cfg
    per = max(0, min(int(max_tokens), cfg.block_size - 1))
    if per and getattr(cfg, "variant", "dflash") == "dflash2":
        per = min(DFLASH2_DEPTH, cfg.block_size - 1)      # a DFlash2 proposal's fixed length
    rows = n * per
    _need(current, torch.int32, n, "current")
    _need(out_tokens, torch.int32, rows, "out_tokens")
    _need(out_q, torch.float32, rows, "out_q")
    _need(out_logits, torch.float32, rows * cfg.vocab, "out_logits")
    out_n = (C.c_int32 * n)()
    _check(lib.dflash_propose(arr, n, _ptr(current), max_tokens, float(temperature), seed, rnd, _ptr(out_tokens),
                              _ptr(out_q), _ptr(out_logits), out_n))
    return list(out_n)


def _verify_args(sessions, b, target_logits, draft_tokens, n, out_accept, out_bonus) -> None:
    V = _model_of(sessions).cfg.vocab
    n = max(0, int(n))
    _need(target_logits, (torch.float32, torch.bfloat16), b * (n + 1) * V, "target_logits [batch, n+1, V]")
    _need(draft_tokens, torch.int32, b * n, "draft_tokens [batch, n]")
    _need(out_accept, torch.int32, b, "out_accept")
    _need(out_bonus, torch.int32, b, "out_bonus")


def dflash_verify(sessions, target_logits: torch.Tensor, draft_tokens: torch.Tensor, n: int, temperature: float,
                  seed: int, rnd: int, out_accept: torch.Tensor, out_bonus: torch.Tensor) -> None:
    arr, b = _sessions(sessions)
    _verify_args(sessions, b, target_logits, draft_tokens, n, out_accept, out_bonus)
    dt = DFLASH_DTYPE_BF16 if target_logits.dtype == torch.bfloat16 else DFLASH_DTYPE_F32
    _check(lib.dflash_verify(arr, b, _ptr(target_logits), dt, _ptr(draft_tokens), n, float(temperature), seed, rnd,
                             _ptr(out_accept), _ptr(out_bonus)))


def dflash_verify_noalloc(sessions, target_logits: torch.Tensor, draft_tokens: torch.Tensor, n: int,
                          temperature: float, seed: int, rnd: int, out_accept: torch.Tensor,
                          out_bonus: torch.Tensor) -> None:
    """dflash_verify on the library's static scratch (no device allocation)."""
    arr, b = _sessions(sessions)
    _verify_args(sessions, b, target_logits, draft_tokens, n, out_accept, out_bonus)
    dt = DFLASH_DTYPE_BF16 if target_logits.dtype == torch.bfloat16 else DFLASH_DTYPE_F32
    _check(lib.dflash_verify_noalloc(arr, b, _ptr(target_logits), dt, _ptr(draft_tokens), n, float(temperature), seed,
                                     rnd, _ptr(out_accept), _ptr(out_bonus)))


def dflash_close(session: Session) -> None:
    if session.handle:
        _check(lib.dflash_close(session.handle))
        session.handle = None


def dflash_candidates(session: Session, out_ids: torch.Tensor, out_probs: torch.Tensor) -> None:
    """A DFlash2 session's last candidate distributions: ids int32 and
    probabilities fp32, each [n, sel_candidates] on the device."""
    cfg = session.model.cfg
    k, n = cfg.sel_candidates, min(DFLASH2_DEPTH, cfg.block_size - 1)
    _need(out_ids, torch.int32, n * k, "out_ids [n, sel_candidates]")
    _need(out_probs, torch.float32, n * k, "out_probs [n, sel_candidates]")
    _check(lib.dflash_candidates(session.handle, _ptr(out_ids), _ptr(out_probs)))


def dflash_set_penalties(session: Session, repeat: float = 1.0, presence: float = 0.0, frequency: float = 0.0,
                         history: torch.Tensor | None = None) -> None:
    """The sampler's penalties over a committed history (CUDA int32 [n] token ids)."""
    n = 0 if history is None else int(history.numel())
    if n and (not history.is_cuda or history.dtype != torch.int32 or not history.is_contiguous()):
        raise ValueError("history: contiguous CUDA int32 token ids")
    _check(lib.dflash_set_penalties(session.handle, float(repeat), float(presence), float(frequency),
                                    _ptr(history) if n else None, n))


def dflash_set_sampler(session: Session, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0) -> None:
    _check(lib.dflash_set_sampler(session.handle, top_k, top_p, min_p))


def dflash_stats(session: Session) -> dict:
    c = _abi.dflash_counters()
    _check(lib.dflash_stats(session.handle, C.byref(c)))
    return {k: getattr(c, k) for k, _ in c._fields_}


def dflash_session_state(session: Session) -> tuple:
    F, P, B = C.c_int64(), C.c_int32(), C.c_int32()
    _check(lib.dflash_session_state(session.handle, C.byref(F), C.byref(P), C.byref(B)))
    return F.value, P.value, bool(B.value)


def dflash_kv_export(session: Session, layer: int, first_slot: int, n_rows: int, k_out: torch.Tensor,
                     v_out: torch.Tensor) -> None:
    _check(lib.dflash_kv_export(session.handle, layer, first_slot, n_rows, _ptr(k_out), _ptr(v_out)))


def dflash_kv_import(session: Session, layer: int, first_slot: int, n_rows: int, k_in: torch.Tensor,
                     v_in: torch.Tensor) -> None:
    _check(lib.dflash_kv_import(session.handle, layer, first_slot, n_rows, _ptr(k_in), _ptr(v_in)))


def dflash_timing_enable(model: Model, on: bool) -> None:
    _check(lib.dflash_timing_enable(model.handle, 1 if on else 0))


def dflash_timing_read(model: Model) -> dict:
    """kernel class -> dict(launches, total_ms, bytes, flops); synchronises."""
    arr = (_abi.dflash_kernel_time * 16)()
    n = C.c_int32()
    _check(lib.dflash_timing_read(model.handle, arr, 16, C.byref(n)))
    return {arr[i].name.decode(): dict(launches=arr[i].launches, total_ms=arr[i].total_ms, bytes=arr[i].bytes,
                                       flops=arr[i].flops) for i in range(n.value)}


# ---------------------------------------------------------------------------
# synthetic target (fp32)
# ---------------------------------------------------------------------------
class Target:
    """Handle of a dflash_target; keeps the weight tensors alive."""

    def __init__(self, handle: int, cfg: dict, tensors: list, layer_structs):
        self.handle = handle
        self.cfg = cfg
        self._tensors = tensors
        self._layers = layer_structs

    def __del__(self):
        if getattr(self, "handle", None):
            lib.dflash_target_destroy(self.handle)
            self.handle = None


def _target_args(cfg: dict, weights: dict):
    c = _abi.dflash_target_config(hidden=cfg["hidden"], n_heads=cfg["n_heads"], head_dim=cfg["head_dim"],
                                  intermediate=cfg["intermediate"], vocab=cfg["vocab"], n_layers=cfg["n_layers"],
                                  rope_theta=cfg["rope_theta"], rms_eps=cfg["rms_eps"])
    keep = []
    H, qd, I, V = cfg["hidden"], cfg["n_heads"] * cfg["head_dim"], cfg["intermediate"], cfg["vocab"]
    shapes = dict(n1=(H,), wq=(qd, H), wk=(qd, H), wv=(qd, H), wo=(H, qd), n2=(H,), wg=(I, H), wu=(I, H),
                  wd=(H, I))

    def dev(t, shape, name):
        t = t.contiguous()
        if not t.is_cuda or t.dtype != torch.float32:
            raise ValueError("target weights are fp32 CUDA tensors")
        if tuple(t.shape) != shape:
            raise ValueError(f"target weight {name}: shape {tuple(t.shape)}, expected {shape}")
        keep.append(t)
        return t.data_ptr()

    if len(weights["layers"]) != cfg["n_layers"]:
        raise ValueError("target weights: one dict per layer")
    layers = (_abi.dflash_target_layer * cfg["n_layers"])()
    for l, lw in enumerate(weights["layers"]):
        for name, shape in shapes.items():
            setattr(layers[l], name, dev(lw[name], shape, name))
    w = _abi.dflash_target_weights(embed=dev(weights["embed"], (V, H), "embed"),
                                   unembed=dev(weights["unembed"], (V, H), "unembed"),
                                   final_norm=dev(weights["final_norm"], (H,), "final_norm"), layers=layers)
    return c, w, keep, layers


def dflash_target_create(cfg: dict, weights: dict, max_ctx: int = 4096, stream=None) -> Target:
    """cfg: hidden, n_heads, head_dim, intermediate, vocab, n_layers, rope_theta, rms_eps;
    weights: fp32 CUDA tensors embed, unembed, final_norm and layers = [dict n1, wq, wk,
    wv, wo, n2, wg, wu, wd]."""
    c, w, keep, layers = _target_args(cfg, weights)
    stream = stream if stream is not None else torch.cuda.current_stream()
    out = C.c_void_p()
    _check(lib.dflash_target_create(C.byref(c), C.byref(w), max_ctx, C.c_void_p(stream.cuda_stream), C.byref(out)))
    return Target(out.value, dict(cfg), keep, layers)


def dflash_target_create_paged(cfg: dict, weights: dict, pages, table: torch.Tensor, max_ctx: int | None = None,
                               stream=None) -> Target:
    """A target on a paged cache that it may share with others.  pages: one (k_pages, v_pages) pair per
    layer, fp32 [n_pages, page_size, n_heads, head_dim]; table: int32 CUDA vector, the page of position p
    at p // page_size; max_ctx: None is what the table can hold."""
    c, w, keep, layers = _target_args(cfg, weights)
    pages = list(pages)
    if len(pages) != cfg["n_layers"]:
        raise ValueError("pages: one (k_pages, v_pages) pair per layer")
    _same_device(weights["embed"], table, *(t for kv in pages for t in kv))
    arr = (_abi.dflash_kv_pages * len(pages))(*[_abi.dflash_kv_pages(*_pages(k, v)) for k, v in pages])
    width = table.numel()
    _int_vector(table, width, "table")
    if max_ctx is None:
        max_ctx = width * arr[0].page_size
    stream = stream if stream is not None else torch.cuda.current_stream()
    out = C.c_void_p()
    _check(lib.dflash_target_create_paged(C.byref(c), C.byref(w), arr, table.data_ptr(), width, max_ctx,
                                          C.c_void_p(stream.cuda_stream), C.byref(out)))
    return Target(out.value, dict(cfg), keep + [t for kv in pages for t in kv] + [table], layers)


def dflash_target_destroy(target: Target) -> None:
    if target.handle:
        _check(lib.dflash_target_destroy(target.handle))
        target.handle = None


def dflash_target_forward(target: Target, tokens: torch.Tensor, start: int, logits: torch.Tensor,
                          taps: torch.Tensor | None = None) -> None:
    """tokens: int32 CUDA [rows]; logits: fp32 CUDA [rows][vocab]; taps: fp32 CUDA [rows][(2L+1)*hidden]."""
    c = target.cfg
    rows = tokens.numel()
    if tokens.dtype != torch.int32 or not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous int32")
    if logits.dtype != torch.float32 or not logits.is_contiguous() or tuple(logits.shape) != (rows, c["vocab"]):
        raise ValueError("logits must be contiguous fp32 [rows, vocab]")
    if taps is not None and (taps.dtype != torch.float32 or not taps.is_contiguous() or
                             tuple(taps.shape) != (rows, (2 * c["n_layers"] + 1) * c["hidden"])):
        raise ValueError("taps must be contiguous fp32 [rows, (2 * n_layers + 1) * hidden]")
    _check(lib.dflash_target_forward(target.handle, _ptr(tokens), tokens.numel(), start, _ptr(logits), _ptr(taps)))


def dflash_target_trim(target: Target, length: int) -> None:
    _check(lib.dflash_target_trim(target.handle, length))


def dflash_target_length(target: Target) -> int:
    v = C.c_int64()
    _check(lib.dflash_target_length(target.handle, C.byref(v)))
    return v.value


def dflash_target_argmax(target: Target, logits: torch.Tensor, out: torch.Tensor) -> None:
    """logits: fp32 CUDA [rows][vocab]; out: int32 CUDA [rows], the greedy token of each row."""
    if logits.dtype != torch.float32 or not logits.is_contiguous() or logits.dim() != 2 or \
            logits.shape[1] != target.cfg["vocab"] or out.dtype != torch.int32 or out.numel() < logits.shape[0]:
        raise ValueError("logits must be contiguous fp32 [rows, vocab] and out int32 [rows]")
    _check(lib.dflash_target_argmax(target.handle, _ptr(logits), logits.shape[0], _ptr(out)))


def dflash_target_device_status(target: Target) -> None:
    _check(lib.dflash_target_device_status(target.handle))


EXACTNESS_ROW_BYTES = C.sizeof(_abi.dflash_exactness_row)


def _rows_buffer(out: torch.Tensor, rows: int) -> None:
    if out.dtype != torch.uint8 or not out.is_contiguous() or out.numel() < rows * EXACTNESS_ROW_BYTES:
        raise ValueError(f"out must be a contiguous uint8 CUDA buffer of rows * {EXACTNESS_ROW_BYTES} bytes")


def _logits_pair(a: torch.Tensor, b: torch.Tensor) -> tuple:
    if a.dtype != torch.float32 or b.dtype != torch.float32 or a.dim() != 2 or a.shape != b.shape or \
            not a.is_contiguous() or not b.is_contiguous():
        raise ValueError("block and chain logits must be contiguous fp32 [rows, vocab] of one shape")
    return a.shape[0], a.shape[1]


def dflash_logits_compare(block: torch.Tensor, chain: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """block, chain: fp32 CUDA [rows][vocab]; out: uint8 CUDA buffer of rows dflash_exactness_row records."""
    rows, V = _logits_pair(block, chain)
    _rows_buffer(out, rows)
    stream = stream if stream is not None else torch.cuda.current_stream()
    _check(lib.dflash_logits_compare(_ptr(block), _ptr(chain), rows, V, _ptr(out), C.c_void_p(stream.cuda_stream)))


def _records(buf):
    raw = bytes(buf.cpu().numpy().tobytes()) if isinstance(buf, torch.Tensor) else bytes(buf)
    n = len(raw) // EXACTNESS_ROW_BYTES
    return (_abi.dflash_exactness_row * n).from_buffer_copy(raw[:n * EXACTNESS_ROW_BYTES])


def exactness_rows(buf) -> list:
    """Decodes row records (the uint8 buffer, copied to the host) into dicts."""
    return [dict(differing_bytes=r.differing_bytes, block_top=list(r.block_top), chain_top=list(r.chain_top),
                 block_val=list(r.block_val), chain_val=list(r.chain_val)) for r in _records(buf)]


def dflash_exactness_summarize(buf) -> dict:
    arr = _records(buf)
    s = _abi.dflash_exactness_summary()
    _check(lib.dflash_exactness_summarize(arr, len(arr), C.byref(s)))
    return {k: getattr(s, k) for k, _ in s._fields_}


def dflash_target_exactness_probe(target: Target, tokens: torch.Tensor, start: int, block_logits: torch.Tensor,
                                  chain_logits: torch.Tensor, out: torch.Tensor) -> dict:
    """Block forward and one-token forwards of `tokens` at start, compared; the
    cache is left at `start`.  Returns the summary (the call synchronises)."""
    rows, V = _logits_pair(block_logits, chain_logits)
    if tokens.dtype != torch.int32 or not tokens.is_contiguous() or tokens.numel() != rows or \
            V != target.cfg["vocab"]:
        raise ValueError("tokens must be contiguous int32 [rows] and logits [rows, vocab]")
    _rows_buffer(out, rows)
    s = _abi.dflash_exactness_summary()
    _check(lib.dflash_target_exactness_probe(target.handle, _ptr(tokens), rows, start, _ptr(block_logits),
                                             _ptr(chain_logits), _ptr(out), C.byref(s)))
    return {k: getattr(s, k) for k, _ in s._fields_}


# ---------------------------------------------------------------------------
# target-side operators
# ---------------------------------------------------------------------------
_DTYPES = {torch.float32: DFLASH_DTYPE_F32, torch.bfloat16: DFLASH_DTYPE_BF16}


def _stream_of(stream, device: int) -> int:
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)


class _on_device:
    """torch.cuda.device(device) for the call, free when that device is current already."""

    def __init__(self, device: int):
        self.ctx = None if torch._C._cuda_getDevice() == device else torch.cuda.device(device)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _same_device(first: torch.Tensor, *others) -> int:
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors of a call live on one CUDA device")
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    return dev


def _heads(t: torch.Tensor, shape, dtype: torch.dtype, what: str) -> tuple:
    """(pointer, row stride, head stride) of [rows, heads, head_dim] with a dense last dimension."""
    st = t.stride()
    if t.dtype != dtype or len(shape) != 3 or (st[2] != 1 and shape[2] > 1):
        raise ValueError(f"{what}: a CUDA {dtype} tensor [rows, heads, head_dim] with a dense last dimension")
    # torch may report any stride for a dimension of one entry, and nothing uses it; the library asks for
    # one that is aligned and that a head fits in
    rows, heads, d = shape
    return (t.data_ptr() if rows else 0, st[0] if rows > 1 else heads * d, st[1] if heads > 1 else d)


def _pages(k_pages: torch.Tensor, v_pages: torch.Tensor) -> tuple:
    """The fields of dflash_kv_pages for [n_pages, page_size, n_kv_heads, head_dim] views of one shape and
    stride (a permuted [n_pages, n_kv_heads, page_size, head_dim] cache too)."""
    shape, st, dtype = k_pages.shape, k_pages.stride(), _DTYPES.get(k_pages.dtype)
    if not k_pages.is_cuda or dtype is None or len(shape) != 4 or st[3] != 1 or v_pages.dtype != k_pages.dtype or \
            v_pages.shape != shape or v_pages.stride() != st:
        raise ValueError("k_pages, v_pages: CUDA fp32 or bf16 [n_pages, page_size, n_kv_heads, head_dim] of one shape "
                         "and stride, with a dense last dimension")
    n, page, heads, d = shape
    return (dtype, heads, d, page, n, k_pages.data_ptr(), v_pages.data_ptr(), st[0] if n > 1 else d, st[1],
            st[2] if heads > 1 else d)


def _int_vector(t: torch.Tensor, n: int | None, what: str) -> int:
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.numel() != n) or \
            not t.is_cuda:
        raise ValueError(f"{what}: a contiguous CUDA int32 vector" + (f" of {n}" if n is not None else ""))
    return t.data_ptr()


def _ragged(starts, lens, table, total: int, max_rows: int, max_len: int, status) -> bytes:
    first = _int_vector(starts, None, "starts [batch + 1]")
    batch = starts.shape[0] - 1
    word = 0 if status is None else _int_vector(status, 1, "status")
    if lens is None:
        return _abi.PACK_RAGGED(batch, total, max_rows, 0, first, 0, 0, 0, 0, word)
    shape, st = table.shape, table.stride()
    if table.dtype != torch.int32 or len(shape) != 2 or shape[0] != batch or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"table: CUDA int32 [{batch}, pages per sequence] with a dense last dimension")
    return _abi.PACK_RAGGED(batch, total, max_rows, max_len, first, _int_vector(lens, batch, "lens"), table.data_ptr(),
                            shape[1], st[0] if batch > 1 else shape[1], word)


def _attention(q, out, n_kv_heads: int, causal, window: int, scale, lse, ragged: bytes, pages, workspace,
               stream, workspace_of=lib.dflash_attention_workspace) -> tuple:
    """The packed dflash_attention, and its workspace: the caller's, or one from torch's allocator on the
    call's stream."""
    dtype, shape = _DTYPES.get(q.dtype), q.shape
    if dtype is None:
        raise ValueError("q: fp32 or bf16")
    if out.shape != shape:
        raise ValueError("out: the shape of q")
    qh, oh = _heads(q, shape, q.dtype, "q"), _heads(out, shape, q.dtype, "out")
    rows, heads, d = shape
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != shape[:2]):
        raise ValueError("lse: contiguous CUDA fp32 [rows, n_q_heads]")
    head = (dtype, heads, n_kv_heads, d, 1 if causal else 0, int(window), d ** -0.5 if scale is None else float(scale),
            *qh, *oh, 0 if lse is None else lse.data_ptr())
    if workspace is None:
        need = workspace_of(_abi.PACK_ATTENTION(*head, 0, 0), ragged, pages)
        if need < 0:
            _check(need)
        if need == 0:
            return _abi.PACK_ATTENTION(*head, 0, 0), None
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous CUDA uint8 tensor")
    return _abi.PACK_ATTENTION(*head, workspace.data_ptr(), workspace.numel()), workspace


def dflash_kv_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                     starts: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, status=None, stream=None) -> None:
    """New rows k, v [rows, n_kv_heads, head_dim] of a ragged batch into their pages
    [n_pages, page_size, n_kv_heads, head_dim]: sequence b's rows starts[b] .. starts[b + 1] - 1
    become its last positions below lens[b]; table [batch, pages] names its pages."""
    device = _same_device(k_pages, k, v, v_pages, starts, lens, table, status)
    p = _pages(k_pages, v_pages)
    shape = k.shape
    if v.shape != shape or len(shape) != 3 or shape[1] != p[1] or shape[2] != p[2]:
        raise ValueError(f"k, v: [rows, {p[1]}, {p[2]}]")
    kh = _abi.PACK_HEADS(*_heads(k, shape, k_pages.dtype, "k"))
    vh = _abi.PACK_HEADS(*_heads(v, shape, k_pages.dtype, "v"))
    rows = shape[0]
    # (max_rows bounds the rows of a sequence, not of the call: the widest that the library takes)
    r = _ragged(starts, lens, table, rows, max(1, min(rows, 1 << 24)), 1 << 30, status)
    with _on_device(device):
        _check(lib.dflash_kv_append(_abi.PACK_PAGES(*p), r, kh, vh, _stream_of(stream, device)))


def dflash_attention_workspace(q, out, starts, lens, table, max_rows: int, max_len: int, k_pages, v_pages,
                               causal: bool = True, window: int = 0) -> int:
    """Bytes a dflash_paged_attention call of these tensors, bounds, causal and window needs. With lens and
    table None: those of a dflash_prompt_attention call, k_pages and v_pages being its k and v (max_len is
    not used)."""
    device = _same_device(q, out, starts, lens, table, k_pages, v_pages)
    shape = q.shape
    qh = _heads(q, shape, k_pages.dtype, "q")
    if (lens is None) != (table is None):
        raise ValueError("lens and table go together")
    if lens is None:
        if q.dtype not in _DTYPES or k_pages.dim() != 3:
            raise ValueError("k, v: fp32 or bf16 [rows, n_kv_heads, head_dim]")
        dtype, kv_heads, pages = _DTYPES[q.dtype], k_pages.shape[1], None
    else:
        p = _pages(k_pages, v_pages)
        dtype, kv_heads, pages = p[0], p[1], _abi.PACK_PAGES(*p)
    r = _ragged(starts, lens, table, shape[0], max_rows, max_len, None)
    a = _abi.PACK_ATTENTION(dtype, shape[1], kv_heads, shape[2], 1 if causal else 0, int(window), 1.0, *qh, *qh, 0, 0, 0)
    with _on_device(device):
        return _check(lib.dflash_attention_workspace(a, r, pages))


def dflash_paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, starts: torch.Tensor,
                           lens: torch.Tensor, table: torch.Tensor, out: torch.Tensor, max_rows: int,
                           max_len: int | None = None, causal: bool = True, window: int = 0,
                           scale: float | None = None, lse: torch.Tensor | None = None, workspace=None, status=None,
                           stream=None) -> None:
    """Attention of each sequence's new rows q [rows, n_q_heads, head_dim] over its pages, which already
    hold them.  max_rows and max_len bound the new rows and the length of every sequence (max_len: None
    takes what the table can hold); scale: None is head_dim ** -0.5."""
    device = _same_device(q, k_pages, v_pages, starts, lens, table, out, lse, workspace, status)
    p = _pages(k_pages, v_pages)
    if max_len is None:
        max_len = min(1 << 30, table.shape[-1] * p[3])
    r = _ragged(starts, lens, table, q.shape[0], max_rows, max_len, status)
    pages = _abi.PACK_PAGES(*p)
    with _on_device(device):
        # (keep: the workspace lives until the launches are enqueued; the allocator orders its reuse)
        a, keep = _attention(q, out, p[1], causal, window, scale, lse, r, pages, workspace, stream)
        _check(lib.dflash_paged_attention(a, r, pages, _stream_of(stream, device)))


def dflash_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor, out: torch.Tensor,
                            max_rows: int, causal: bool = True, window: int = 0, scale: float | None = None,
                            lse: torch.Tensor | None = None, workspace=None, status=None, stream=None) -> None:
    """Attention of whole packed prompts: sequence b is rows starts[b] .. starts[b + 1] - 1 of
    q [rows, n_q_heads, head_dim] and of k, v [rows, n_kv_heads, head_dim]."""
    device = _same_device(q, k, v, starts, out, lse, workspace, status)
    shape, qs = k.shape, q.shape
    if v.shape != shape or len(shape) != 3 or len(qs) != 3 or shape[0] != qs[0] or shape[2] != qs[2]:
        raise ValueError("k, v: [rows, n_kv_heads, head_dim] with q's rows and head_dim")
    kh = _abi.PACK_HEADS(*_heads(k, shape, q.dtype, "k"))
    vh = _abi.PACK_HEADS(*_heads(v, shape, q.dtype, "v"))
    r = _ragged(starts, None, None, shape[0], max_rows, 0, status)
    with _on_device(device):
        a, keep = _attention(q, out, shape[1], causal, window, scale, lse, r, None, workspace, stream)
        _check(lib.dflash_prompt_attention(a, r, kh, vh, _stream_of(stream, device)))


def dflash_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, logprobs: torch.Tensor,
                          entropy: torch.Tensor | None = None, top_ids: torch.Tensor | None = None,
                          top_logprobs: torch.Tensor | None = None, temperature: float = 1.0, status=None,
                          stream=None) -> None:
    """Log probability of tokens[r] (int32, -1: none) under softmax(logits[r] / temperature), the row's
    entropy, and its top entries: top_ids int32 and top_logprobs fp32 [rows, k], k at most 32."""
    device = _same_device(logits, tokens, logprobs, entropy, top_ids, top_logprobs, status)
    shape, st, dtype = logits.shape, logits.stride(), _DTYPES.get(logits.dtype)
    if dtype is None or len(shape) != 2 or (st[1] != 1 and shape[1] > 1):
        raise ValueError("logits: CUDA fp32 or bf16 [rows, vocab] with a dense last dimension")
    R, V = shape
    tok = _int_vector(tokens, R, "tokens [rows]")
    for t, what in ((logprobs, "logprobs"), (entropy, "entropy")):
        if t is not None and (t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != R or not t.is_contiguous()):
            raise ValueError(f"{what}: contiguous CUDA fp32 [rows]")
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    top = 0
    if top_ids is not None:
        if top_ids.dtype != torch.int32 or not top_ids.is_contiguous() or top_ids.dim() != 2 or \
                top_ids.shape[0] != R or top_logprobs.dtype != torch.float32 or not top_logprobs.is_contiguous() or \
                top_logprobs.shape != top_ids.shape:
            raise ValueError("top_ids int32 and top_logprobs fp32: contiguous CUDA [rows, k] of one shape")
        top = top_ids.shape[1]
    ptr = lambda t: 0 if t is None else t.data_ptr()
    a = _abi.PACK_LOGPROBS(logits.data_ptr(), st[0] if R > 1 else V, dtype, R, V, top, float(temperature),
                           tok, logprobs.data_ptr(), ptr(entropy), ptr(top_ids), ptr(top_logprobs),
                           0 if status is None else _int_vector(status, 1, "status"))
    with _on_device(device):
        _check(lib.dflash_token_logprobs(a, _stream_of(stream, device)))


# ---------------------------------------------------------------------------
# the compressed cache
# ---------------------------------------------------------------------------
def _vector(t: torch.Tensor, n: int, what: str) -> int:
    """The address of a contiguous int32 vector of n (a tensor that _same_device has seen)."""
    if t.dtype is not torch.int32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous CUDA int32 vector of {n}")
    return t.data_ptr()


def _word(t) -> int:
    return 0 if t is None else _vector(t, 1, "status")


_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_SCALINGS = {"linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


class RopeTable:
    """What dflash_rope_table made: the library's table (host memory), and its fields."""

    def __init__(self, table):
        self.table = table
        self.rot_dim, self.offset, self.amplitude = table.rot_dim, table.offset, table.amplitude
        self.address = C.addressof(table)


def dflash_rope_table(rot_dim: int, theta: float, layout: str = "half", scaling: dict | None = None, offset: int = 0,
                      amplitude: float | None = None) -> RopeTable:
    """The rotary table of a model, made once: rot_dim elements of each head from offset on, base theta,
    layout "half" (pairs i, i + rot_dim / 2) or "interleaved" (pairs 2i, 2i + 1).  scaling for long contexts:
    dict(kind="linear" or "ntk", factor=), dict(kind="bands" or "yarn", factor=, original_len=, low=, high=) with
    low and high in turns over the original context.  amplitude: the factor on cos and sin (None: 1, for
    "yarn" 0.1 ln(factor) + 1)."""
    if layout not in _ROPE_LAYOUTS:
        raise ValueError(f"layout: one of {sorted(_ROPE_LAYOUTS)}")
    p = dict(scaling or {})
    kind = p.pop("kind", None)
    if scaling is not None and kind not in _ROPE_SCALINGS:
        raise ValueError(f"scaling: a dict with kind, one of {sorted(_ROPE_SCALINGS)}")
    want = set() if kind is None else {"factor"} if kind in ("linear", "ntk") else {"factor", "original_len", "low", "high"}
    if set(p) != want:
        raise ValueError(f"scaling {kind}: takes {sorted(want)}")
    if amplitude is not None and not amplitude > 0:
        raise ValueError("amplitude: > 0")
    c = _abi.dflash_rope_config(rot_dim=rot_dim, offset=offset, layout=_ROPE_LAYOUTS[layout],
                                scaling=_ROPE_SCALINGS.get(kind, 0), theta=theta, amplitude=amplitude or 0.0, **p)
    t = _abi.dflash_rope_table()
    _check(lib.dflash_rope_init(C.byref(c), C.byref(t)))
    return RopeTable(t)


def _rope_ragged(starts, lens, total: int, status) -> bytes:
    batch = starts.numel() - 1
    return _abi.PACK_RAGGED(batch, total, 1 << 24, 1 << 30, _vector(starts, batch + 1, "starts [batch + 1]"),
                            0 if lens is None else _vector(lens, batch, "lens"), 0, 0, 0, _word(status))


def dflash_rope(table: RopeTable, q: torch.Tensor | None, k: torch.Tensor | None, starts: torch.Tensor,
                lens: torch.Tensor | None, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                transpose: bool = False, status=None, stream=None) -> None:
    """Turns q [rows, n_q_heads, head_dim] and k [rows, n_k_heads, head_dim] (either may be None) of a ragged
    batch by their positions: row i of sequence b is at lens[b] - n_b + i, or at i with lens None.  In place, or
    into q_out and k_out.  transpose: the transposed map, which takes a gradient back."""
    one = q if q is not None else k
    if one is None:
        raise ValueError("q or k")
    device = _same_device(one, q, k, starts, lens, q_out, k_out, status)
    dtype = _DTYPES.get(one.dtype)
    if dtype is None:
        raise ValueError("q, k: fp32 or bf16")
    packed, heads = [], []
    rows, d = one.shape[0], one.shape[-1]
    for x, y, what in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            if y is not None:
                raise ValueError(f"{what}_out without {what}")
            heads.append(0)
            packed.append(((0, 0, 0), (0, 0, 0)))
            continue
        shape = x.shape
        if len(shape) != 3 or shape[0] != rows or shape[2] != d or (y is not None and y.shape != shape):
            raise ValueError("q, k and their outputs: [rows, heads, head_dim] of the same rows and head_dim")
        xh = _heads(x, shape, one.dtype, what)
        heads.append(shape[1])
        packed.append((xh, xh if y is None else _heads(y, shape, one.dtype, what + "_out")))
    a = _abi.PACK_ROPE(dtype, d, heads[0], heads[1], 1 if transpose else 0, *packed[0][0], *packed[1][0], *packed[0][1],
                       *packed[1][1])
    r = _rope_ragged(starts, lens, rows, status)
    with _on_device(device):
        _check(lib.dflash_rope(table.address, r, a, _stream_of(stream, device)))


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _kv8_pages(k_pages, v_pages, k_scale, v_scale) -> tuple:
    """The fields of dflash_kv8_pages: codes [n_pages, page_size, n_kv_heads, head_dim] and scales
    [n_pages, n_kv_heads], each pair of one shape and stride."""
    shape, st, ss = k_pages.shape, k_pages.stride(), k_scale.stride()
    if k_pages.dtype not in _CODES or v_pages.dtype not in _CODES or len(shape) != 4 or st[3] != 1 or \
            v_pages.shape != shape or v_pages.stride() != st:
        raise ValueError("k_pages, v_pages: CUDA float8_e4m3fn (or uint8) [n_pages, page_size, n_kv_heads, head_dim] of "
                         "one shape and stride, with a dense last dimension")
    n, page, heads, d = shape
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or k_scale.shape != (n, heads) or \
            v_scale.shape != (n, heads) or v_scale.stride() != ss:
        raise ValueError("k_scale, v_scale: CUDA fp32 [n_pages, n_kv_heads] of one stride")
    return (heads, d, page, 0, n, k_pages.data_ptr(), v_pages.data_ptr(), st[0] if n > 1 else d, st[1],
            st[2] if heads > 1 else d, k_scale.data_ptr(), v_scale.data_ptr(), ss[0] if n > 1 else 1,
            ss[1] if heads > 1 else 1)


def dflash_kv8_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                      k_scale: torch.Tensor, v_scale: torch.Tensor, starts: torch.Tensor, lens: torch.Tensor,
                      table: torch.Tensor, status=None, stream=None) -> None:
    """dflash_kv_append into 8-bit pages: codes float8_e4m3fn [n_pages, page_size, n_kv_heads, head_dim] with
    fp32 scales [n_pages, n_kv_heads], which become the powers of two that their pages need."""
    device = _same_device(k_pages, k, v, v_pages, k_scale, v_scale, starts, lens, table, status)
    p = _kv8_pages(k_pages, v_pages, k_scale, v_scale)
    shape, dtype = k.shape, _DTYPES.get(k.dtype)
    if dtype is None or v.shape != shape or len(shape) != 3 or shape[1] != p[0] or shape[2] != p[1]:
        raise ValueError(f"k, v: fp32 or bf16 [rows, {p[0]}, {p[1]}]")
    kh = _abi.PACK_HEADS(*_heads(k, shape, k.dtype, "k"))
    vh = _abi.PACK_HEADS(*_heads(v, shape, k.dtype, "v"))
    rows = shape[0]
    r = _ragged(starts, lens, table, rows, max(1, min(rows, 1 << 24)), 1 << 30, status)
    with _on_device(device):
        _check(lib.dflash_kv8_append(_abi.PACK_KV8(*p), r, dtype, kh, vh, _stream_of(stream, device)))


def dflash_kv8_attention_workspace(q, out, starts, lens, table, max_rows: int, max_len: int, k_pages, v_pages, k_scale,
                                   v_scale, causal: bool = True, window: int = 0) -> int:
    """Bytes a dflash_kv8_attention call of these tensors, bounds, causal and window needs."""
    device = _same_device(q, out, starts, lens, table, k_pages, v_pages, k_scale, v_scale)
    shape, dtype = q.shape, _DTYPES.get(q.dtype)
    if dtype is None:
        raise ValueError("q: fp32 or bf16")
    qh = _heads(q, shape, q.dtype, "q")
    p = _kv8_pages(k_pages, v_pages, k_scale, v_scale)
    r = _ragged(starts, lens, table, shape[0], max_rows, max_len, None)
    a = _abi.PACK_ATTENTION(dtype, shape[1], p[0], shape[2], 1 if causal else 0, int(window), 1.0, *qh, *qh, 0, 0, 0)
    with _on_device(device):
        return _check(lib.dflash_kv8_attention_workspace(a, r, _abi.PACK_KV8(*p)))


def dflash_kv8_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, starts: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                         out: torch.Tensor, max_rows: int, max_len: int | None = None, causal: bool = True,
                         window: int = 0, scale: float | None = None, lse: torch.Tensor | None = None, workspace=None,
                         status=None, stream=None) -> None:
    """dflash_paged_attention over 8-bit pages (dflash_kv8_append): value = code * scale of its page and head."""
    device = _same_device(q, k_pages, v_pages, k_scale, v_scale, starts, lens, table, out, lse, workspace, status)
    p = _kv8_pages(k_pages, v_pages, k_scale, v_scale)
    if max_len is None:
        max_len = min(1 << 30, table.shape[-1] * p[2])
    r = _ragged(starts, lens, table, q.shape[0], max_rows, max_len, status)
    pages = _abi.PACK_KV8(*p)
    with _on_device(device):
        a, keep = _attention(q, out, p[0], causal, window, scale, lse, r, pages, workspace, stream,
                             lib.dflash_kv8_attention_workspace)
        _check(lib.dflash_kv8_attention(a, r, pages, _stream_of(stream, device)))


class PageBuffers:
    """What lies in a pool's pages: the library's list of buffers (host memory), made once, with the tensors
    that it points into."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("at least one tensor")
        self.device = _same_device(*self.tensors)
        self.n_pages = self.tensors[0].shape[0] if self.tensors[0].dim() else 0
        packed = []
        for t in self.tensors:
            if t.dim() < 1 or t.shape[0] != self.n_pages or self.n_pages < 1:
                raise ValueError("buffers: tensors [n_pages, ...] of one pool")
            if not t[0].is_contiguous():
                raise ValueError("buffers: a page is one dense run")
            size, es = t[0].numel() * t.element_size(), t.element_size()
            packed.append(_abi.PACK_BUFFER(t.data_ptr(), t.stride(0) * es if self.n_pages > 1 else size, size))
        self.packed, self.count = b"".join(packed), len(packed)


def dflash_page_buffers(tensors) -> PageBuffers:
    """The buffers of a pool: one tensor [n_pages, ...] for each run of bytes that a page has (a layer's K, V
    and their scales), each page dense and a multiple of 4 bytes."""
    return PageBuffers(tensors)


def _page_rows(table: torch.Tensor, lens: torch.Tensor, page_size: int, what: str) -> bytes:
    shape, st = table.shape, table.stride()
    if table.dtype != torch.int32 or len(shape) != 2 or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what}table: CUDA int32 [rows, pages of a row] with a dense last dimension")
    return _abi.PACK_ROWS(shape[0], shape[1], st[0] if shape[0] > 1 else shape[1], page_size, table.data_ptr(),
                          _vector(lens, shape[0], f"{what}lens"))


def _pages_workspace(workspace, n_pages: int, rows: int, like: torch.Tensor, stream):
    if workspace is not None:
        if not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace: a contiguous CUDA uint8 tensor")
        return workspace
    need = _check(lib.dflash_pages_workspace(n_pages, rows))
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=like.device)


def dflash_pages_copy(buffers: PageBuffers, src: torch.Tensor, dst: torch.Tensor, status=None, stream=None) -> None:
    """Copies page src[i] to page dst[i] (int32) in every buffer."""
    device = _same_device(src, dst, buffers.tensors[0], status)
    n = src.numel()
    s, t = _vector(src, n, "src"), _vector(dst, n, "dst")
    with _on_device(device):
        _check(lib.dflash_pages_copy(buffers.packed, buffers.count, buffers.n_pages, s, t, n,
                                     _word(status), _stream_of(stream, device)))


def dflash_pages_reorder(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
                         new_table: torch.Tensor, new_lens: torch.Tensor, page_size: int, status=None,
                         stream=None) -> None:
    """Rows of the next step: row i of new_table and new_lens becomes row parents[i] (int32, -1: empty) of table
    and lens; refs (int32 [n_pages]) follows.  A row named twice is forked, one that is not named is freed."""
    device = _same_device(refs, table, lens, parents, new_table, new_lens, status)
    a, b = _page_rows(table, lens, page_size, ""), _page_rows(new_table, new_lens, page_size, "new_")
    n_pages = refs.numel()
    with _on_device(device):
        _check(lib.dflash_pages_reorder(_vector(refs, n_pages, "refs [n_pages]"), n_pages, a,
                                        _vector(parents, new_table.shape[0], "parents"), b,
                                        _word(status),
                                        _stream_of(stream, device)))


def dflash_pages_resize(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor,
                        buffers: PageBuffers | None, page_size: int, free_pages: torch.Tensor | None = None,
                        workspace=None, status=None, stream=None) -> None:
    """Sets the rows' lengths to new_lens: pages behind them go back, new ones are the lowest free ids, and a
    begun last page that others hold too is copied before its row grows.  A row whose pages are not there, or whose
    begun page a row without its own copy still holds, stays as it is (status 16)."""
    device = _same_device(refs, table, lens, new_lens, free_pages, workspace, status,
                          None if buffers is None else buffers.tensors[0])
    rows = _page_rows(table, lens, page_size, "")
    n_pages = refs.numel()
    if buffers is not None and buffers.n_pages != n_pages:
        raise ValueError("refs: int32 [n_pages] of the buffers' pool")
    with _on_device(device):
        ws = _pages_workspace(workspace, n_pages, table.shape[0], refs, stream)
        _check(lib.dflash_pages_resize(_vector(refs, n_pages, "refs [n_pages]"), n_pages, rows,
                                       _vector(new_lens, table.shape[0], "new_lens"),
                                       None if buffers is None else buffers.packed, 0 if buffers is None else buffers.count,
                                       0 if free_pages is None else _vector(free_pages, 1, "free_pages"),
                                       ws.data_ptr(), ws.numel(),
                                       _word(status),
                                       _stream_of(stream, device)))


def dflash_pages_compact(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, new_refs: torch.Tensor,
                         new_table: torch.Tensor, buffers: PageBuffers | None, page_size: int,
                         new_lens: torch.Tensor | None = None, used: torch.Tensor | None = None, workspace=None,
                         status=None, stream=None) -> None:
    """Moves the pages in use to the lowest ids: new_refs and new_table (which may be refs and table) say where
    they are then, used (int32 [1]) how many.  new_lens None: lens stays what it is."""
    new_lens = lens if new_lens is None else new_lens
    device = _same_device(refs, table, lens, new_refs, new_table, new_lens, used, workspace, status,
                          None if buffers is None else buffers.tensors[0])
    n_pages = refs.numel()
    if buffers is not None and buffers.n_pages != n_pages:
        raise ValueError("refs: int32 [n_pages] of the buffers' pool")
    if new_table.shape != table.shape:
        raise ValueError("new_table: the shape of table")
    a, b = _page_rows(table, lens, page_size, ""), _page_rows(new_table, new_lens, page_size, "new_")
    with _on_device(device):
        ws = _pages_workspace(workspace, n_pages, table.shape[0], refs, stream)
        _check(lib.dflash_pages_compact(_vector(refs, n_pages, "refs [n_pages]"), _vector(new_refs, n_pages, "new_refs"),
                                        n_pages, a, b, None if buffers is None else buffers.packed,
                                        0 if buffers is None else buffers.count,
                                        0 if used is None else _vector(used, 1, "used"), ws.data_ptr(), ws.numel(),
                                        _word(status),
                                        _stream_of(stream, device)))


def dflash_status_check(status: torch.Tensor, stream=None) -> None:
    """Waits for the stream, clears the operators' status word and raises DFlashError if a bit was set."""
    word, device = _int_vector(status, 1, "status"), status.get_device()
    with _on_device(device):
        _check(lib.dflash_status_check(word, _stream_of(stream, device)))
