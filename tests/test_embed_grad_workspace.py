"""dllm_embed_grad's workspace: one allocated for the largest box serves every smaller one."""
import numpy as np
import pytest

from confidence_block_unmasking_amd import _lib


def _bytes(n, D, V=152066):
    return _lib.lib().dllm_embed_grad_workspace_bytes(n, V, D)


@pytest.mark.parametrize("D", [1, 64, 512, 513, 1000, 1024, 2048, 4096, 5120, 8192, 1 << 20])
def test_size_never_falls_with_the_tokens(D):
    rng = np.random.default_rng(D)
    ns = set(range(0, 300)) | {int(2 ** e) for e in rng.uniform(0, 24, 4000)} | {1 << 24}
    for e in range(25):
        ns |= {n for n in range((1 << e) - 70, (1 << e) + 70) if 0 <= n <= 1 << 24}
    ns |= {n for m in range(1, 2100) for n in (64 * m - 1, 64 * m, 64 * m + 1)}
    last = 0
    for n in sorted(ns):
        got = _bytes(n, D)
        assert got >= last, (n, got, last)
        last = got


@pytest.mark.parametrize("D", [64, 1000, 4096])
def test_call_is_not_refused_for_a_larger_box_s_workspace(D):
    """The call's own need is within the size reported for any larger box (refusals come before the
    launch, so a null workspace of that size shows what the size check says)."""
    A = [np.uintp((i + 1) << 32).item() for i in range(5)]
    for big in (1 << 14, 1 << 15, 1 << 17):
        have = _bytes(big, D)
        for n in (1, 100, 1000, 5000, 10000, 16320, 16383, 16384):
            rc = _lib.lib().dllm_embed_grad(None, A[0], 1, D, A[1], None, n, 1.0, 152066, D, A[2], 1, D, 0,
                                            A[3] + 8, have, A[4])
            assert rc == _lib.DLLM_ERR_ARG and "256-byte aligned" in _lib.last_error(), (big, n, _lib.last_error())


@pytest.mark.gpu
@pytest.mark.parametrize("D,gd,td", [(1000, "bf16", "fp32"), (4096, "bf16", "bf16"), (64, "fp32", "fp32")])
def test_one_workspace_for_boxes_of_every_size(D, gd, td):
    """A session's boxes: the workspace of the widest serves the narrower ones, on both sides of the token
    count at which the layout changes, and the results are those of a workspace of their own."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from confidence_block_unmasking_amd import api
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}
    rng = np.random.default_rng(D)
    V, big = 500, 140000 if D == 64 else 20000
    ids = torch.from_numpy(np.where(rng.random(big) < 0.5, 7, rng.integers(0, V, big)).astype(np.int32)).cuda()
    grad = torch.randn((big, D), device="cuda").to(dt[gd])
    shared = api.new_embed_grad_workspace(big, V, D)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (big, 16384, 16320, 10000, 3100, 700, 13, 1):
        a, b = (torch.full((V, D), 9.0, dtype=dt[td], device="cuda") for _ in range(2))
        api.dllm_embed_grad(grad, ids[:n], a, shared, st)
        api.dllm_embed_grad(grad, ids[:n], b, api.new_embed_grad_workspace(n, V, D), st)
        assert torch.equal(a, b), n
    assert int(st.item()) == 0
