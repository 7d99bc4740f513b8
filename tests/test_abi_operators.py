"""Refusals of the log-probability and embedding calls, before anything reaches a device (CPU)."""
import ctypes

import pytest

from confidence_block_unmasking_amd import _lib

A = [ctypes.c_void_p(0x100000000 * (i + 1)) for i in range(12)]   # distinct, never dereferenced
ARG, SHAPE, DTYPE = _lib.DLLM_ERR_ARG, _lib.DLLM_ERR_SHAPE, _lib.DLLM_ERR_DTYPE


def test_workspace_sizes():
    L = _lib.lib()
    # V = 152064 bf16: 38 chunks per slot; a record of 16 bytes and 64 lane maxima of 2
    assert L.dllm_logprobs_workspace_bytes(64, 32, 152064, 0, 1) == 64 * 32 * 38 * 16
    assert L.dllm_logprobs_workspace_bytes(64, 32, 152064, 20, 1) == 64 * 32 * 38 * (16 + 128)
    assert L.dllm_logprobs_workspace_bytes(1, 1, 1, 1, 0) >= 24
    for bad in ((-1, 32, 100, 0, 1), (1, 0, 100, 0, 1), (1, 1, 0, 0, 1), (1, 1, 100, 33, 1), (1, 1, 100, -1, 1),
                (1, 1, 100, 0, 2)):
        assert L.dllm_logprobs_workspace_bytes(*bad) == 0, bad
    assert L.dllm_embed_grad_workspace_bytes(1000, 5000, 64) >= 2 * 1000 * 8 + 16 * 2 * 64 * 4
    for bad in ((-1, 5, 5), (5, 0, 5), (5, 5, 0), ((1 << 24) + 1, 5, 5), (5, (1 << 24) + 1, 5), (5, 5, (1 << 20) + 1)):
        assert L.dllm_embed_grad_workspace_bytes(*bad) == 0, bad


def logprobs(**kw):
    a = dict(logits=A[0], dtype=1, ps=1024, rs=32 * 1024, rows=4, L=32, V=1024, mask=A[1], exclude=None, tokens=A[2],
             ts=32, k=5, lp=A[3], ent=A[4], stats=A[5], ti=A[6], tl=A[7], ws=A[8], n=1 << 30, status=A[9])
    a.update(kw)
    return _lib.lib().dllm_logprobs(None, *a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(rows=-1), ARG), (dict(L=0), SHAPE), (dict(L=1025, rs=1025 * 1024, ts=1025), SHAPE),
    (dict(rows=4097), SHAPE), (dict(rows=4096, L=128, rs=128 * 1024, ts=128), SHAPE), (dict(V=0), ARG), (dict(ps=1023), ARG),
    (dict(rs=1024), ARG), (dict(ts=31), ARG), (dict(logits=None), ARG), (dict(mask=None), ARG), (dict(status=None), ARG),
    (dict(logits=ctypes.c_void_p(0x100000001)), ARG), (dict(logits=ctypes.c_void_p(0x100000002), dtype=0), ARG),
    (dict(k=-1), ARG), (dict(k=33), ARG), (dict(k=5, V=4), ARG), (dict(tokens=None), ARG), (dict(lp=None), ARG),
    (dict(ti=None), ARG), (dict(tl=None), ARG), (dict(tokens=None, lp=None, ent=None, stats=None, k=0), ARG),
    (dict(stats=ctypes.c_void_p(0x100000004)), ARG), (dict(ws=None), ARG), (dict(n=4 * 32 * (16 + 128) - 1), ARG),
    (dict(ws=ctypes.c_void_p(0x100000008)), ARG),
    (dict(V=2 ** 31 - 1, ps=2 ** 31, rs=2 ** 36, rows=4096, L=32), SHAPE),
])
def test_logprobs_refuses(kw, code):
    assert logprobs(**kw) == code
    assert "dllm_logprobs" in _lib.last_error()


def test_logprobs_of_no_rows_is_a_no_op():
    assert logprobs(rows=0, logits=None, mask=None, status=None, ws=None, n=0) == _lib.DLLM_OK


def grad(**kw):
    a = dict(logits=A[0], dtype=1, ps=1024, rs=32 * 1024, rows=4, L=32, V=1024, mask=A[1], exclude=None, tokens=A[2],
             ts=32, stats=A[3], gl=A[4], ent=A[5], gh=A[6], out=A[7], gps=1024, grs=32 * 1024, status=A[9])
    a.update(kw)
    return _lib.lib().dllm_logprobs_grad(None, *a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), DTYPE), (dict(rows=-3), ARG), (dict(V=0), ARG), (dict(ps=1000), ARG), (dict(gps=1000), ARG),
    (dict(grs=32 * 1024 - 1), ARG), (dict(stats=None), ARG), (dict(out=None), ARG), (dict(tokens=None), ARG),
    (dict(gl=None), ARG), (dict(ent=None), ARG), (dict(tokens=None, gl=None, gh=None), ARG), (dict(mask=None), ARG),
    (dict(stats=ctypes.c_void_p(0x300000004)), ARG), (dict(out=ctypes.c_void_p(0x700000001)), ARG),
    (dict(out=ctypes.c_void_p(0x100000002)), ARG),                         # overlaps the logits by an offset
    (dict(out=A[0], gps=2048, grs=64 * 1024), ARG),                        # the same address, other strides
    (dict(out=ctypes.c_void_p(0x100000000 - 2)), ARG),
    (dict(V=2 ** 31 - 1, ps=2 ** 31, gps=2 ** 31, rs=2 ** 36, grs=2 ** 36, rows=4096, L=32, out=ctypes.c_void_p(1 << 60)),
     SHAPE),
])
def test_logprobs_grad_refuses(kw, code):
    assert grad(**kw) == code
    assert "dllm_logprobs_grad" in _lib.last_error()


def embed(**kw):
    a = dict(table=A[0], td=1, ts=64, V=100, D=64, ids=A[1], valid=A[2], n=50, scale=1.0, out=A[3], od=0, os=64, status=A[4])
    a.update(kw)
    return _lib.lib().dllm_embed(None, *a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(td=5), DTYPE), (dict(od=-1), DTYPE), (dict(n=-1), ARG), (dict(n=(1 << 24) + 1), SHAPE), (dict(V=0), SHAPE),
    (dict(V=(1 << 24) + 1), SHAPE), (dict(D=0), SHAPE), (dict(D=(1 << 20) + 1), SHAPE), (dict(ts=63), ARG),
    (dict(os=63), ARG), (dict(table=None), ARG), (dict(ids=None), ARG), (dict(out=None), ARG), (dict(status=None), ARG),
    (dict(table=ctypes.c_void_p(0x100000001)), ARG), (dict(out=ctypes.c_void_p(0x400000002)), ARG),
    (dict(out=ctypes.c_void_p(0x100000000 + 4)), ARG), (dict(out=ctypes.c_void_p(0x200000000 - 4)), ARG),
    (dict(out=ctypes.c_void_p(0x300000000 - 4)), ARG),
])
def test_embed_refuses(kw, code):
    assert embed(**kw) == code
    assert "dllm_embed" in _lib.last_error()


def embed_grad(**kw):
    a = dict(g=A[0], gd=1, gs=64, ids=A[1], valid=A[2], n=50, scale=1.0, V=100, D=64, t=A[3], td=0, ts=64, acc=0, ws=A[4],
             nb=1 << 30, status=A[5])
    a.update(kw)
    return _lib.lib().dllm_embed_grad(None, *a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(gd=2), DTYPE), (dict(td=2), DTYPE), (dict(n=-1), ARG), (dict(n=(1 << 24) + 1), SHAPE), (dict(V=0), SHAPE),
    (dict(D=0), SHAPE), (dict(gs=63), ARG), (dict(ts=1), ARG), (dict(g=None), ARG), (dict(ids=None), ARG), (dict(t=None), ARG),
    (dict(status=None), ARG), (dict(ws=None), ARG), (dict(nb=16), ARG), (dict(ws=ctypes.c_void_p(0x500000010)), ARG),
    (dict(g=ctypes.c_void_p(0x100000001)), ARG), (dict(t=ctypes.c_void_p(0x400000002)), ARG),
    (dict(t=ctypes.c_void_p(0x100000000 + 64)), ARG), (dict(t=ctypes.c_void_p(0x200000000)), ARG),
    (dict(t=ctypes.c_void_p(0x500000000)), ARG), (dict(ws=ctypes.c_void_p(0x100000000)), ARG),
    (dict(ws=ctypes.c_void_p(0x200000000)), ARG),
])
def test_embed_grad_refuses(kw, code):
    assert embed_grad(**kw) == code
    assert "dllm_embed_grad" in _lib.last_error()


def test_embed_of_no_tokens_is_a_no_op():
    assert embed(n=0, table=None, ids=None, out=None, status=None) == _lib.DLLM_OK
    assert embed_grad(n=0, acc=1, g=None, ids=None, t=None, ws=None, nb=0, status=None) == _lib.DLLM_OK
