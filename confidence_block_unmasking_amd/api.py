"""Thin torch-facing binding of the C ABI: argument marshalling only.

Every function hands device pointers of caller-owned torch tensors to libdllm.so and enqueues work
on the current torch stream (or the stream given).  No part of the step, pack or compact
computation runs here.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MAX_TOP, DllmError, Meta, Queue, Reqs  # noqa: F401  (re-exported)

_DT = {torch.bfloat16: _lib.DLLM_BF16, torch.float32: _lib.DLLM_FP32}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _launch(fn, args, where, events, stream):
    """Call fn(*args) and check its status; with `events` (two timing events), they are recorded on
    the launch stream right before and right after the call, after every argument is marshalled."""
    if events is not None:
        s = torch.cuda.current_stream() if stream is None else stream
        events[0].record(s)
        rc = fn(*args)
        events[1].record(s)
    else:
        rc = fn(*args)
    _lib.check(rc, where)


def _need(t, dtype, name, numel=None, inner=()):
    """Refuse t unless it is a contiguous device tensor of this type with at least numel elements, and, where it has
    more than those, rows of `inner` (as far as it has dimensions behind the first; flat tensors have none)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        if t.numel() < numel:
            raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
        n = min(t.dim() - 1, len(inner))
        if n > 0 and tuple(t.shape[-n:]) != tuple(inner[-n:]):
            raise ValueError(f"{name} of shape {tuple(t.shape)} for rows of {tuple(inner)}")


def dllm_step_workspace_bytes(rows: int, L: int, V: int, dtype=torch.bfloat16) -> int:
    return int(_lib.lib().dllm_step_workspace_bytes(rows, L, V, _DT[dtype]))


def new_workspace(rows: int, L: int, V: int, dtype=torch.bfloat16, device="cuda"):
    """A step workspace for this shape (the step needs no particular contents; zero-filled here)."""
    n = dllm_step_workspace_bytes(rows, L, V, dtype)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def _logits_shape(logits, rows, L, V, pos_stride, row_stride):
    """Shape and strides (in elements) of the logits; the kernels read element (r, j, v) at
    r*row_stride + j*pos_stride + v, so the tensor's storage must reach that far."""
    if logits.dtype not in _DT:
        raise ValueError(f"logits dtype {logits.dtype} not supported")
    # the kernels read a slot's V elements as one contiguous run
    if logits.dim() >= 1 and logits.shape[-1] > 1 and logits.stride(-1) != 1:
        raise ValueError(f"logits must have unit stride along the vocabulary, got stride {logits.stride(-1)}")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    if rows is None:
        rows, L, V = logits.shape
    if pos_stride is None and row_stride is None and logits.dim() != 3 and not logits.is_contiguous():
        raise ValueError(f"logits of shape {tuple(logits.shape)} with strides {logits.stride()} need pos_stride and row_stride")
    cube = logits.dim() == 3
    if pos_stride is None:
        pos_stride = logits.stride(1) if cube else V
        if L == 1 and cube and not V <= pos_stride <= logits.stride(0):
            pos_stride = V                      # a dimension of size 1 has a stride of any value
    if row_stride is None:
        row_stride = logits.stride(0) if cube else L * pos_stride
        if rows == 1 and row_stride < L * pos_stride:
            row_stride = L * pos_stride
    if rows > 0 and L > 0 and V > 0:
        reach = (rows - 1) * row_stride + (L - 1) * pos_stride + V
        if reach > logits.numel() or not logits.is_contiguous():
            avail = logits.untyped_storage().nbytes() // logits.element_size() - logits.storage_offset()
            if reach > avail:
                raise ValueError(f"logits storage holds {avail} elements past its offset; rows={rows}, L={L}, V={V} "
                                 f"with strides ({row_stride}, {pos_stride}) reach {reach}")
    return rows, L, V, pos_stride, row_stride


def _decide_args(rows, L, input_ids, mask_in, mask_out, threshold, done, accept_len, workspace, status, p, b, conf,
                 argmax, need_tau=True):
    W = input_ids.shape[-1]
    _need(input_ids, torch.int32, "input_ids", rows * W)
    _need(mask_in, torch.uint8, "mask_in", rows * L)
    _need(mask_out, torch.uint8, "mask_out", rows * L)
    if need_tau:
        _need(threshold, torch.float32, "threshold", rows)
    _need(done, torch.uint8, "done", rows)
    _need(accept_len, torch.int32, "accept_len", rows)
    _need(workspace, torch.uint8, "workspace")
    _need(status, torch.int32, "status", 1)
    for t, dt, nm, n in ((p, torch.int32, "p", rows), (b, torch.int32, "b", rows),
                         (conf, torch.float32, "conf", rows * L), (argmax, torch.int32, "argmax", rows * L)):
        if t is not None:
            _need(t, dt, nm, n)
    return W


def dllm_step(logits, input_ids, mask_in, mask_out, threshold, done, accept_len, workspace, status,
              p=None, b=None, conf=None, argmax=None, rows=None, L=None, V=None, pos_stride=None,
              row_stride=None, stream=None, events=None):
    """One LowConfidence denoise step (see include/dllm.h).

    logits: [rows, L, V] bf16/fp32 device tensor, or any tensor whose storage holds element
    (r, j, v) at r*row_stride + j*pos_stride + v when the strides are given.  events: optional
    pair of timing events recorded right around the library call.
    """
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    W = _decide_args(rows, L, input_ids, mask_in, mask_out, threshold, done, accept_len, workspace, status, p, b,
                     conf, argmax)
    args = (_stream(stream), _ptr(logits), _DT[logits.dtype], pos_stride, row_stride, rows, L, V, _ptr(input_ids), W,
            _ptr(mask_in), _ptr(mask_out), _ptr(threshold), _ptr(p), _ptr(b), _ptr(conf), _ptr(argmax), _ptr(done),
            _ptr(accept_len), _ptr(workspace), workspace.numel(), _ptr(status))
    _launch(_lib.lib().dllm_step, args, "dllm_step", events, stream)


def dllm_step_noalloc(logits, input_ids, mask_in, mask_out, threshold, done, accept_len, status, p=None, b=None,
                      conf=None, argmax=None, rows=None, L=None, V=None, pos_stride=None, row_stride=None, stream=None):
    """dllm_step without a workspace: the library's fixed per-device scratch holds the partials
    (for callers that cannot allocate; calls on one GPU must not overlap).  See include/dllm.h."""
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    W = input_ids.shape[-1]
    _need(input_ids, torch.int32, "input_ids", rows * W)
    _need(mask_in, torch.uint8, "mask_in", rows * L)
    _need(mask_out, torch.uint8, "mask_out", rows * L)
    _need(threshold, torch.float32, "threshold", rows)
    _need(done, torch.uint8, "done", rows)
    _need(accept_len, torch.int32, "accept_len", rows)
    _need(status, torch.int32, "status", 1)
    for t, dt, nm, n in ((p, torch.int32, "p", rows), (b, torch.int32, "b", rows),
                         (conf, torch.float32, "conf", rows * L), (argmax, torch.int32, "argmax", rows * L)):
        if t is not None:
            _need(t, dt, nm, n)
    rc = _lib.lib().dllm_step_noalloc(_stream(stream), _ptr(logits), _DT[logits.dtype], pos_stride, row_stride, rows,
                                      L, V, _ptr(input_ids), W, _ptr(mask_in), _ptr(mask_out), _ptr(threshold),
                                      _ptr(p), _ptr(b), _ptr(conf), _ptr(argmax), _ptr(done), _ptr(accept_len),
                                      _ptr(status))
    _lib.check(rc, "dllm_step_noalloc")


def dllm_step_timed(logits, input_ids, mask_in, mask_out, threshold, done, accept_len, workspace, status, kernel_events,
                    p=None, b=None, conf=None, argmax=None, rows=None, L=None, V=None, pos_stride=None,
                    row_stride=None, stream=None):
    """dllm_step with `kernel_events` (a KernelEvents) bound to the scoring kernel's start and the
    deciding kernel's end."""
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    W = _decide_args(rows, L, input_ids, mask_in, mask_out, threshold, done, accept_len, workspace, status, p, b,
                     conf, argmax)
    args = (_stream(stream), _ptr(logits), _DT[logits.dtype], pos_stride, row_stride, rows, L, V, _ptr(input_ids), W,
            _ptr(mask_in), _ptr(mask_out), _ptr(threshold), _ptr(p), _ptr(b), _ptr(conf), _ptr(argmax), _ptr(done),
            _ptr(accept_len), _ptr(workspace), workspace.numel(), _ptr(status), kernel_events.start,
            kernel_events.stop)
    _launch(_lib.lib().dllm_step_timed, args, "dllm_step_timed", None, stream)


def dllm_step_score(logits, mask_in, workspace, status, rows=None, L=None, V=None, pos_stride=None,
                    row_stride=None, stream=None):
    """The scoring half of dllm_step: per-chunk partials of every masked slot into `workspace`."""
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    _need(mask_in, torch.uint8, "mask_in", rows * L)
    _need(workspace, torch.uint8, "workspace")
    _need(status, torch.int32, "status", 1)
    rc = _lib.lib().dllm_step_score(_stream(stream), _ptr(logits), _DT[logits.dtype], pos_stride, row_stride, rows,
                                    L, V, _ptr(mask_in), _ptr(workspace), workspace.numel(), _ptr(status))
    _lib.check(rc, "dllm_step_score")


class KernelEvents:
    """Two HIP events with timing enabled, for dllm_step_score_timed.  They are created through the
    HIP runtime that libdllm.so and torch share; elapsed_ms() waits for the second one."""

    def __init__(self):
        hip = _lib.lib()
        self._hip = hip
        self.start, self.stop = ctypes.c_void_p(), ctypes.c_void_p()
        for e in (self.start, self.stop):
            if hip.hipEventCreate(ctypes.byref(e)) != 0:
                raise RuntimeError("hipEventCreate failed")

    def elapsed_ms(self) -> float:
        if self._hip.hipEventSynchronize(self.stop) != 0:
            raise RuntimeError("hipEventSynchronize failed")
        ms = ctypes.c_float()
        if self._hip.hipEventElapsedTime(ctypes.byref(ms), self.start, self.stop) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return ms.value

    def __del__(self):
        for e in (getattr(self, "start", None), getattr(self, "stop", None)):
            if e is not None and e.value:
                self._hip.hipEventDestroy(e)


def dllm_step_score_timed(logits, mask_in, workspace, status, events, rows=None, L=None, V=None, pos_stride=None,
                          row_stride=None, stream=None):
    """dllm_step_score with the scoring kernel's own start and end recorded into `events`
    (a KernelEvents)."""
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    _need(mask_in, torch.uint8, "mask_in", rows * L)
    _need(workspace, torch.uint8, "workspace")
    _need(status, torch.int32, "status", 1)
    rc = _lib.lib().dllm_step_score_timed(_stream(stream), _ptr(logits), _DT[logits.dtype], pos_stride, row_stride,
                                          rows, L, V, _ptr(mask_in), _ptr(workspace), workspace.numel(),
                                          _ptr(status), events.start, events.stop)
    _lib.check(rc, "dllm_step_score_timed")


def dllm_step_decide(dtype, rows, L, V, input_ids, mask_in, mask_out, threshold, done, accept_len, workspace, status,
                     p=None, b=None, conf=None, argmax=None, unmasked=None, fallback=None, stream=None, events=None):
    """The deciding half of dllm_step, on the partials dllm_step_score left in `workspace`
    (same dtype, rows, L, V and mask_in).  unmasked (int32 [rows]) and fallback (uint8 [rows]),
    when given, receive each row's count of slots unmasked and whether the rule's single-slot
    fallback applied.  events: optional pair of timing events recorded right around the call."""
    if dtype not in _DT:
        raise ValueError(f"dtype {dtype} not supported")
    W = _decide_args(rows, L, input_ids, mask_in, mask_out, threshold, done, accept_len, workspace, status, p, b,
                     conf, argmax)
    if unmasked is not None:
        _need(unmasked, torch.int32, "unmasked", rows)
    if fallback is not None:
        _need(fallback, torch.uint8, "fallback", rows)
    args = (_stream(stream), _DT[dtype], rows, L, V, _ptr(input_ids), W, _ptr(mask_in), _ptr(mask_out),
            _ptr(threshold), _ptr(p), _ptr(b), _ptr(conf), _ptr(argmax), _ptr(done), _ptr(accept_len),
            _ptr(workspace), workspace.numel(), _ptr(status), _ptr(unmasked), _ptr(fallback))
    _launch(_lib.lib().dllm_step_decide, args, "dllm_step_decide", events, stream)


def dllm_step_quota(logits, input_ids, mask_in, mask_out, steps_per_block, done, accept_len, workspace, status,
                    p=None, b=None, conf=None, argmax=None, rows=None, L=None, V=None, pos_stride=None,
                    row_stride=None, stream=None):
    """One denoise step with the fixed per-step quota (steps_per_block diffusion steps per block)."""
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    W = _decide_args(rows, L, input_ids, mask_in, mask_out, None, done, accept_len, workspace, status, p, b, conf,
                     argmax, need_tau=False)
    rc = _lib.lib().dllm_step_quota(_stream(stream), _ptr(logits), _DT[logits.dtype], pos_stride, row_stride, rows,
                                    L, V, _ptr(input_ids), W, _ptr(mask_in), _ptr(mask_out), int(steps_per_block),
                                    _ptr(p), _ptr(b), _ptr(conf), _ptr(argmax), _ptr(done), _ptr(accept_len),
                                    _ptr(workspace), workspace.numel(), _ptr(status))
    _lib.check(rc, "dllm_step_quota")


def dllm_step_decide_quota(dtype, rows, L, V, input_ids, mask_in, mask_out, steps_per_block, done, accept_len,
                           workspace, status, p=None, b=None, conf=None, argmax=None, stream=None):
    """The deciding half of dllm_step_quota, on the partials dllm_step_score left in `workspace`."""
    if dtype not in _DT:
        raise ValueError(f"dtype {dtype} not supported")
    W = _decide_args(rows, L, input_ids, mask_in, mask_out, None, done, accept_len, workspace, status, p, b, conf,
                     argmax, need_tau=False)
    rc = _lib.lib().dllm_step_decide_quota(_stream(stream), _DT[dtype], rows, L, V, _ptr(input_ids), W,
                                           _ptr(mask_in), _ptr(mask_out), int(steps_per_block), _ptr(p), _ptr(b),
                                           _ptr(conf), _ptr(argmax), _ptr(done), _ptr(accept_len), _ptr(workspace),
                                           workspace.numel(), _ptr(status))
    _lib.check(rc, "dllm_step_decide_quota")


def new_triples(rows: int, L: int, n_shards: int, device="cuda"):
    """Buffer for the per-shard results of dllm_step_score_shard ([rows, L, n_shards] records of 16 B)."""
    n = _lib.lib().dllm_shard_triples_bytes(rows, L, n_shards)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def dllm_step_score_shard(logits, mask_in, workspace, triples, shard, n_shards, vocab_offset, status, rows=None,
                          L=None, V_shard=None, pos_stride=None, row_stride=None, stream=None):
    """Score one vocabulary shard (columns vocab_offset .. + V_shard - 1) of every masked slot."""
    rows, L, V_shard, pos_stride, row_stride = _logits_shape(logits, rows, L, V_shard, pos_stride, row_stride)
    _need(mask_in, torch.uint8, "mask_in", rows * L)
    _need(workspace, torch.uint8, "workspace")
    _need(triples, torch.uint8, "triples", _lib.lib().dllm_shard_triples_bytes(rows, L, n_shards))
    _need(status, torch.int32, "status", 1)
    rc = _lib.lib().dllm_step_score_shard(_stream(stream), _ptr(logits), _DT[logits.dtype], pos_stride, row_stride,
                                          rows, L, V_shard, int(vocab_offset), int(shard), int(n_shards),
                                          _ptr(mask_in), _ptr(workspace), workspace.numel(), _ptr(triples),
                                          _ptr(status))
    _lib.check(rc, "dllm_step_score_shard")


def dllm_step_decide_shards(n_shards, triples, rows, L, V, input_ids, mask_in, mask_out, threshold, done, accept_len,
                            status, p=None, b=None, conf=None, argmax=None, stream=None):
    """Combine the shards' results per masked slot and apply the LowConfidence rule."""
    W = _decide_args(rows, L, input_ids, mask_in, mask_out, threshold, done, accept_len, triples, status, p, b, conf,
                     argmax)
    _need(triples, torch.uint8, "triples", _lib.lib().dllm_shard_triples_bytes(rows, L, n_shards))
    rc = _lib.lib().dllm_step_decide_shards(_stream(stream), int(n_shards), _ptr(triples), rows, L, V,
                                            _ptr(input_ids), W, _ptr(mask_in), _ptr(mask_out), _ptr(threshold),
                                            _ptr(p), _ptr(b), _ptr(conf), _ptr(argmax), _ptr(done), _ptr(accept_len),
                                            _ptr(status))
    _lib.check(rc, "dllm_step_decide_shards")


N_FEATURES = 9


def dllm_step_features(rows, L, row_req, reqs: "ReqTable", conf, mask_out, features, status, stream=None):
    """Step-predictor features per row after a step: float32 [rows, 9] (see include/dllm.h)."""
    _need(row_req, torch.int32, "row_req", rows)
    _need(conf, torch.float32, "conf", rows * L)
    _need(mask_out, torch.uint8, "mask_out", rows * L)
    _need(features, torch.float32, "features", rows * N_FEATURES)
    _need(status, torch.int32, "status", 1)
    st = reqs.struct()
    rc = _lib.lib().dllm_step_features(_stream(stream), rows, L, _ptr(row_req), ctypes.byref(st), _ptr(conf),
                                       _ptr(mask_out), _ptr(features), _ptr(status))
    _lib.check(rc, "dllm_step_features")


# ---- log probabilities and embeddings: the two sides of the forward ------------------------------

_devices = 0          # GPUs this process sees (counted at the first call)


def _call(fn, where, stream, tensors, *args):
    """fn(stream, *args) on the device that all `tensors` share (None entries aside; each has been
    checked to be a device tensor), whatever the current device is; `stream`, when given, must be that
    device's.  The small calls take microseconds on the device, so this path avoids building stream
    objects, and with one GPU there is nothing to compare."""
    global _devices
    if not _devices:
        _devices = torch.cuda.device_count()
    dev = tensors[0].get_device()
    if _devices > 1:
        for t in tensors:
            if t is not None and t.get_device() != dev:
                raise ValueError(f"{where}: tensors on devices {dev} and {t.get_device()}; all must be on one device")
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"{where}: stream of {stream.device} for tensors on device {dev}")
        handle = stream.cuda_stream
    else:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    if _devices == 1 or dev == torch.cuda.current_device():
        rc = fn(handle, *args)
    else:
        with torch.cuda.device(dev):
            rc = fn(handle, *args)
    if rc != 0:
        _lib.check(rc, where)


def _adr(t):
    return None if t is None else t.data_ptr()


def _fits(where, *sizes):
    """Sizes past 32 bits are past every limit of the library, and would reach it modulo 2^32.  The callers
    ask only where (a | b | ...) >> 31 is not 0: past 31 bits, or negative (which the library refuses)."""
    for n in sizes:
        if not -(1 << 31) <= n < 1 << 31:
            raise DllmError(_lib.DLLM_ERR_SHAPE, where, f"size {n} is past 32 bits")


def _tokens_arg(tokens, rows, L):
    """Row stride of int32 tokens [rows, L]: a contiguous tensor, or a 2-D view with unit column
    stride (such as box[:, W - L:])."""
    if not tokens.is_cuda or tokens.dtype != torch.int32:
        raise ValueError(f"tokens must be an int32 device tensor, got {tokens.dtype} on {tokens.device}")
    if tokens.dim() != 2:
        _need(tokens, torch.int32, "tokens", rows * L)
        return L
    have, wide = tokens.shape
    if have < rows or wide < L:
        raise ValueError(f"tokens of shape {tuple(tokens.shape)}, needs [{rows}, {L}]")
    step, unit = tokens.stride()
    if L > 1 and unit != 1:
        raise ValueError("tokens must have unit stride along a row")
    return step if have > 1 else max(step, L)


def dllm_logprobs_workspace_bytes(rows: int, L: int, V: int, k: int = 0, dtype=torch.bfloat16) -> int:
    if max(rows, L, V, k) >> 31:                # past every limit
        return 0
    return int(_lib.lib().dllm_logprobs_workspace_bytes(rows, L, V, k, _DT[dtype]))


def new_logprobs_workspace(rows: int, L: int, V: int, k: int = 0, dtype=torch.bfloat16, device="cuda"):
    """A dllm_logprobs workspace for this shape (no particular contents are needed)."""
    return torch.empty(max(dllm_logprobs_workspace_bytes(rows, L, V, k, dtype), 256), dtype=torch.uint8, device=device)


def dllm_logprobs(logits, mask, tokens, logprob, workspace, status, entropy=None, stats=None, top_ids=None,
                  top_logprobs=None, k=None, exclude=None, rows=None, L=None, V=None, pos_stride=None, row_stride=None,
                  stream=None):
    """Log probabilities of `tokens` at the selected slots (mask nonzero, exclude zero), with entropy,
    softmax statistics and the top k alternatives where those outputs are given (see include/dllm.h).

    logits as for dllm_step, at any alignment; tokens int32 [rows, L] (a view of the box's block
    columns will do) or None with logprob None; logprob, entropy float32 [rows, L]; stats float32
    [rows, L, 2]; top_ids int32 and top_logprobs float32 [rows, L, k], or flat with k given (k:
    top_ids' last dimension unless given).  Slots that are not selected keep what the outputs held."""
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    _need(mask, torch.uint8, "mask", rows * L, (L,))
    _need(workspace, torch.uint8, "workspace")
    _need(status, torch.int32, "status", 1)
    if exclude is not None:
        _need(exclude, torch.uint8, "exclude", rows * L, (L,))
    token_stride = L
    if tokens is not None:
        token_stride = _tokens_arg(tokens, rows, L)
    if k is None:
        k = top_ids.shape[-1] if top_ids is not None else 0
    n = rows * L
    for t, dt, nm, each, inner in ((logprob, torch.float32, "logprob", 1, (L,)), (entropy, torch.float32, "entropy", 1, (L,)),
                                   (stats, torch.float32, "stats", 2, (L, 2)), (top_ids, torch.int32, "top_ids", k, (L, k)),
                                   (top_logprobs, torch.float32, "top_logprobs", k, (L, k))):
        if t is not None:
            _need(t, dt, nm, n * each, inner if each else ())
    if (rows | L | V | k) >> 31:
        _fits("dllm_logprobs", rows, L, V, k)
    _call(_lib.lib().dllm_logprobs, "dllm_logprobs", stream,
          (logits, mask, exclude, tokens, logprob, entropy, stats, top_ids, top_logprobs, workspace, status),
          _adr(logits), _DT[logits.dtype], pos_stride, row_stride, rows, L, V, _adr(mask), _adr(exclude), _adr(tokens),
          token_stride, int(k), _adr(logprob), _adr(entropy), _adr(stats), _adr(top_ids), _adr(top_logprobs),
          _adr(workspace), workspace.numel(), _adr(status))


def dllm_logprobs_grad(logits, mask, tokens, stats, grad_logprob, grad_logits, status, entropy=None, grad_entropy=None,
                       exclude=None, rows=None, L=None, V=None, pos_stride=None, row_stride=None, grad_pos_stride=None,
                       grad_row_stride=None, stream=None):
    """Gradient of dllm_logprobs' log probabilities (grad_logprob) and entropies (grad_entropy) with
    respect to the logits, into every slot of grad_logits (the logits' dtype; zeros where not
    selected).  stats and entropy are the forward's outputs.  grad_logits may be logits itself."""
    rows, L, V, pos_stride, row_stride = _logits_shape(logits, rows, L, V, pos_stride, row_stride)
    if grad_logits.dtype != logits.dtype:
        raise ValueError(f"grad_logits must be {logits.dtype}, got {grad_logits.dtype}")
    if grad_logits.dim() == 3 and tuple(grad_logits.shape) != (rows, L, V):
        raise ValueError(f"grad_logits of shape {tuple(grad_logits.shape)}, needs [{rows}, {L}, {V}]")
    own_strides = grad_pos_stride is None and grad_row_stride is None and grad_logits.dim() == 3
    _, _, _, grad_pos_stride, grad_row_stride = _logits_shape(grad_logits, rows, L, V, grad_pos_stride, grad_row_stride)
    if not own_strides and rows > 0:            # what is written has to lie in the tensor, not in its storage only
        reach = (rows - 1) * grad_row_stride + (L - 1) * grad_pos_stride + V
        own = 1 + sum((n - 1) * s for n, s in zip(grad_logits.shape, grad_logits.stride())) if grad_logits.numel() else 0
        if reach > own:
            raise ValueError(f"grad_logits of shape {tuple(grad_logits.shape)} spans {own} elements; rows={rows}, L={L}, V={V} "
                             f"with strides ({grad_row_stride}, {grad_pos_stride}) reach {reach}")
    _need(mask, torch.uint8, "mask", rows * L, (L,))
    _need(stats, torch.float32, "stats", rows * L * 2, (L, 2))
    _need(status, torch.int32, "status", 1)
    token_stride = L
    if tokens is not None:
        token_stride = _tokens_arg(tokens, rows, L)
    for t, dt, nm in ((exclude, torch.uint8, "exclude"), (grad_logprob, torch.float32, "grad_logprob"),
                      (entropy, torch.float32, "entropy"), (grad_entropy, torch.float32, "grad_entropy")):
        if t is not None:
            _need(t, dt, nm, rows * L, (L,))
    if (rows | L | V) >> 31:
        _fits("dllm_logprobs_grad", rows, L, V)
    _call(_lib.lib().dllm_logprobs_grad, "dllm_logprobs_grad", stream,
          (logits, mask, exclude, tokens, stats, grad_logprob, entropy, grad_entropy, grad_logits, status),
          _adr(logits), _DT[logits.dtype], pos_stride, row_stride, rows, L, V, _adr(mask), _adr(exclude), _adr(tokens),
          token_stride, _adr(stats), _adr(grad_logprob), _adr(entropy), _adr(grad_entropy), _adr(grad_logits),
          grad_pos_stride, grad_row_stride, _adr(status))


def _matrix(t, name):
    """(rows, columns, row stride) of a device matrix: a 2-D tensor with unit column stride, or a
    contiguous tensor of any shape taken as [-1, its last dimension]."""
    if t is None or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in _DT:
        raise ValueError(f"{name} dtype {t.dtype} not supported")
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    D = t.shape[-1]
    if t.dim() == 2:
        if D > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit stride along a row")
        return t.shape[0], D, t.stride(0) if t.shape[0] > 1 else max(t.stride(0), D)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, or 2-D")
    return (t.numel() // D if D else 0), D, D


def _ids_arg(ids, valid, status):
    _need(ids, torch.int32, "ids")
    n = ids.numel()
    if valid is not None:
        _need(valid, torch.uint8, "valid", n, () if valid.numel() == n else ids.shape[1:])
    _need(status, torch.int32, "status", 1)
    return n


def _same_box(t, name, ids, n):
    """Refuse a box [..., W', D] of more rows of D than the n ids whose rows of W' are not the ids' rows: its first n
    are used as one run.  (A matrix [n_rows, D] leaves no doubt; flat ids may be any whole rows.)"""
    if t.dim() > 2 and ((t.shape[1:-1] != ids.shape[1:]) if ids.dim() > 1 else (n % max(t.shape[-2], 1) != 0)):
        raise ValueError(f"{name} of shape {tuple(t.shape)} for ids of shape {tuple(ids.shape)}")


def dllm_embed(table, ids, out, status, valid=None, scale=1.0, stream=None):
    """out[n] = scale * table[ids[n]], zeros where valid[n] == 0 (see include/dllm.h).  table
    [n_vocab, D]; ids int32 and valid uint8 of any shape (a box's box_ids and box_valid); out
    [ids.numel(), D] or ids' shape with D appended, or more such rows; fp32 or bf16 each.  Rows of out
    past the last token keep what they held."""
    n = _ids_arg(ids, valid, status)
    n_vocab, D, ts = _matrix(table, "table")
    n_out, D_out, os_ = _matrix(out, "out")
    if D_out != D or n_out < n:
        raise ValueError(f"out holds {n_out} rows of {D_out}, needs {n} of {D}")
    if n_out != n:
        _same_box(out, "out", ids, n)
    if (n | n_vocab | D) >> 31:
        _fits("dllm_embed", n, n_vocab, D)
    _call(_lib.lib().dllm_embed, "dllm_embed", stream, (table, ids, valid, out, status),
          _adr(table), _DT[table.dtype], ts, n_vocab, D, _adr(ids), _adr(valid), n, float(scale), _adr(out),
          _DT[out.dtype], os_, _adr(status))


def dllm_embed_grad_workspace_bytes(n_tokens: int, n_vocab: int, D: int) -> int:
    if max(n_tokens, n_vocab, D) >> 31:         # past every limit
        return 0
    return int(_lib.lib().dllm_embed_grad_workspace_bytes(n_tokens, n_vocab, D))


def new_embed_grad_workspace(n_tokens: int, n_vocab: int, D: int, device="cuda"):
    """A dllm_embed_grad workspace for up to n_tokens tokens (no particular contents are needed)."""
    return torch.empty(max(dllm_embed_grad_workspace_bytes(n_tokens, n_vocab, D), 256), dtype=torch.uint8, device=device)


def dllm_embed_grad(grad_out, ids, grad_table, workspace, status, valid=None, scale=1.0, accumulate=False, stream=None):
    """The gradient of dllm_embed with respect to its table: grad_table[v] = scale * the sum of
    grad_out over the tokens of v, every row written; with accumulate, added to the rows that occur
    (see include/dllm.h)."""
    n = _ids_arg(ids, valid, status)
    n_vocab, D, ts = _matrix(grad_table, "grad_table")
    n_grad, D_grad, gs = _matrix(grad_out, "grad_out")
    if D_grad != D or n_grad < n:
        raise ValueError(f"grad_out holds {n_grad} rows of {D_grad}, needs {n} of {D}")
    if n_grad != n:
        _same_box(grad_out, "grad_out", ids, n)
    _need(workspace, torch.uint8, "workspace")
    if (n | n_vocab | D) >> 31:
        _fits("dllm_embed_grad", n, n_vocab, D)
    _call(_lib.lib().dllm_embed_grad, "dllm_embed_grad", stream,
          (grad_out, ids, valid, grad_table, workspace, status),
          _adr(grad_out), _DT[grad_out.dtype], gs, _adr(ids), _adr(valid), n, float(scale), n_vocab, D,
          _adr(grad_table), _DT[grad_table.dtype], ts, int(bool(accumulate)), _adr(workspace), workspace.numel(),
          _adr(status))


class ReqTable:
    """Device-resident request table (the fields of dllm_reqs), built from host numpy arrays."""

    def __init__(self, p, K, b, state, threshold, arena_off, arena, blk_mask, device="cuda"):
        def dev(a, dt):
            return torch.as_tensor(a).to(dtype=dt).contiguous().to(device)
        self.p = dev(p, torch.int32)
        self.K = dev(K, torch.int32)
        self.b = dev(b, torch.int32)
        self.state = dev(state, torch.int32)
        self.threshold = dev(threshold, torch.float32)
        self.arena_off = dev(arena_off, torch.int64)
        self.arena = dev(arena, torch.int32)
        self.blk_mask = dev(blk_mask, torch.uint8)
        self.L = int(self.blk_mask.shape[1])
        self.n_req = int(self.p.shape[0])

    def struct(self) -> Reqs:
        return Reqs(self.n_req, self.p.data_ptr(), self.K.data_ptr(), self.b.data_ptr(), self.state.data_ptr(),
                    self.threshold.data_ptr(), self.arena_off.data_ptr(), self.arena.data_ptr(),
                    self.blk_mask.data_ptr())


class DevQueue:
    """Device-resident pending queue (dllm_queue): ids [cap] and a device length."""

    def __init__(self, ids, device="cuda", cap=None):
        ids = torch.as_tensor(ids).to(torch.int32)
        cap = int(ids.numel()) if cap is None else int(cap)
        self.ids = torch.full((max(cap, 1),), -1, dtype=torch.int32, device=device)
        self.ids[:ids.numel()] = ids.to(device)
        self.len = torch.tensor([ids.numel()], dtype=torch.int32, device=device)
        self.cap = cap

    def struct(self) -> Queue:
        return Queue(self.ids.data_ptr(), self.len.data_ptr(), self.cap)


def dllm_pack(rows, L, W, pad_id, row_req, reqs: ReqTable, box_ids, mask, threshold, p, b, status,
              box_valid=None, box_pos=None, stream=None, events=None):
    """Gather the left-padded box for rows [0, rows) (see include/dllm.h).  events: optional pair
    of timing events recorded right around the library call."""
    if rows > 0:
        _need(row_req, torch.int32, "row_req", rows)
        _need(box_ids, torch.int32, "box_ids", rows * W)
        _need(mask, torch.uint8, "mask", rows * L)
        _need(threshold, torch.float32, "threshold", rows)
        _need(p, torch.int32, "p", rows)
        _need(b, torch.int32, "b", rows)
        _need(status, torch.int32, "status", 1)
        if box_valid is not None:
            _need(box_valid, torch.uint8, "box_valid", rows * W)
        if box_pos is not None:
            _need(box_pos, torch.int32, "box_pos", rows * W)
    st = reqs.struct()
    args = (_stream(stream), rows, L, W, pad_id, _ptr(row_req), ctypes.byref(st), _ptr(box_ids), _ptr(box_valid),
            _ptr(box_pos), _ptr(mask), _ptr(threshold), _ptr(p), _ptr(b), _ptr(status))
    _launch(_lib.lib().dllm_pack, args, "dllm_pack", events, stream)


def dllm_compact(rows, L, W, mask_id, eos_id, row_req, rows_cap, reqs: ReqTable, queue: DevQueue, budget, meta,
                 status, box_ids=None, mask=None, done=None, stream=None, events=None):
    """Commit finished blocks, evict, refill under the token budget (see include/dllm.h).
    meta: device uint8 tensor of 32 bytes (a dllm_meta).  events: optional pair of timing events
    recorded right around the library call."""
    _need(row_req, torch.int32, "row_req", rows_cap)
    _need(meta, torch.uint8, "meta", 32)
    _need(status, torch.int32, "status", 1)
    if box_ids is not None:
        _need(box_ids, torch.int32, "box_ids", rows * W)
        _need(mask, torch.uint8, "mask", rows * L)
        _need(done, torch.uint8, "done", rows)
    st = reqs.struct()
    q = queue.struct()
    args = (_stream(stream), rows, L, W, mask_id, eos_id, _ptr(box_ids), _ptr(mask), _ptr(done), _ptr(row_req),
            rows_cap, ctypes.byref(st), ctypes.byref(q), int(budget), _ptr(meta), _ptr(status))
    _launch(_lib.lib().dllm_compact, args, "dllm_compact", events, stream)


def read_meta(meta_tensor) -> dict:
    """Copy a device dllm_meta to the host (synchronises with the tensor's stream)."""
    raw = meta_tensor.cpu().numpy().tobytes()
    m = Meta.from_buffer_copy(raw)
    return dict(rows=m.rows, W=m.W, n_evicted=m.n_evicted, n_admitted=m.n_admitted, n_queued=m.n_queued,
                cost=m.cost)
