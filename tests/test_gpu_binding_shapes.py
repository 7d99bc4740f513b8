"""What the binding of the calls around the forward refuses because it would be read or written otherwise
than its shape says, on the GPU (device tensors); each refusal leaves the outputs alone."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _forward(rows=2, L=4, V=50, k=3):
    from confidence_block_unmasking_amd import api
    f = dict(dtype=torch.float32, device="cuda")
    return dict(logits=torch.randn((rows, L, V), **f), mask=torch.ones((rows, L), dtype=torch.uint8, device="cuda"),
                tokens=torch.zeros((rows, L), dtype=torch.int32, device="cuda"), logprob=torch.full((rows, L), 7.0, **f),
                workspace=api.new_logprobs_workspace(rows, L, V, 5, torch.float32),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _top(last_ids, last_lp, rows=2, L=4):
    return dict(top_ids=torch.full((rows, L, last_ids), -5, dtype=torch.int32, device="cuda"),
                top_logprobs=torch.full((rows, L, last_lp), 7.0, dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("k,last_ids,last_lp", [(3, 5, 3), (3, 3, 5), (3, 5, 5), (None, 3, 5), (None, 3, 4), (1, 2, 1)])
def test_alternatives_have_k_columns(k, last_ids, last_lp):
    from confidence_block_unmasking_amd import api
    a, top = _forward(), _top(last_ids, last_lp)
    with pytest.raises(ValueError):
        api.dllm_logprobs(**a, **top, k=k)
    torch.cuda.synchronize()
    assert (top["top_ids"] == -5).all() and (top["top_logprobs"] == 7.0).all() and (a["logprob"] == 7.0).all()


def test_alternatives_of_any_layout_that_holds_k_columns():
    """[rows, L, k], [rows * L, k], a flat buffer with k, and more rows than the call has."""
    from confidence_block_unmasking_amd import api
    a, top = _forward(), _top(3, 3)
    api.dllm_logprobs(**a, **top)
    for shape, k in (((8, 3), None), ((24,), 3), ((5, 4, 3), None), ((30,), 3)):
        ids = torch.full(shape, -5, dtype=torch.int32, device="cuda")
        lp = torch.full(shape, 7.0, dtype=torch.float32, device="cuda")
        api.dllm_logprobs(**a, top_ids=ids, top_logprobs=lp, k=k)
        assert torch.equal(ids.view(-1)[:24], top["top_ids"].view(-1))
        assert torch.equal(lp.view(-1)[:24], top["top_logprobs"].view(-1))
    assert int(a["status"].item()) == 0
