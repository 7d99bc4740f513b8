"""Sizes whose launch would need 2^32 threads are refused as shapes, before anything is launched (CPU)."""
import ctypes

import pytest

from confidence_block_unmasking_amd import _lib

A = [ctypes.c_void_p(1 << (44 + i)) for i in range(10)]           # far apart, never dereferenced


def _grad(rows, L, V, dtype, in_place):
    out = A[0] if in_place else A[9]
    return _lib.lib().dllm_logprobs_grad(None, A[0], dtype, V, L * V, rows, L, V, A[1], None, A[2], L, A[3], A[4], None, None,
                                         out, V, L * V, A[5])


@pytest.mark.parametrize("rows,L,V,dtype", [
    (1792, 128, 152064, 0),                                        # 75 workgroups of 256 threads per slot
    (4096, 64, 129025, 0), (4096, 64, 258049, 1),                  # 64 per slot: 2^24 exactly
    (4096, 64, 152064, 0), (1, 1024, 1 << 30, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_gradient_of_the_log_probabilities(rows, L, V, dtype, in_place):
    assert _grad(rows, L, V, dtype, in_place) == _lib.DLLM_ERR_SHAPE, _lib.last_error()
    assert "dllm_logprobs_grad" in _lib.last_error()


@pytest.mark.parametrize("n,D", [(1 << 24, 6145), (1 << 24, 8192), (1 << 20, 1 << 20), ((1 << 24) - 1, 10241)])
def test_lookup(n, D):
    rc = _lib.lib().dllm_embed(None, A[0], 1, D, 4, D, A[2], None, n, 1.0, A[9], 1, D, A[3])
    assert rc == _lib.DLLM_ERR_SHAPE, _lib.last_error()
    assert "dllm_embed" in _lib.last_error()
