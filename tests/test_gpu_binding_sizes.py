"""Sizes past 32 bits reach the library's limits and are refused there; taken modulo 2^32 they would be
small sizes that it serves.  Device buffers of 17 and 9 GB, never filled."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BIG = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture()
def small():
    f = dict(dtype=torch.float32, device="cuda")
    return dict(table=torch.zeros((4, 4), **f), out=torch.full((8, 4), 7.0, **f), status=torch.zeros(1, dtype=torch.int32, device="cuda"),
                ids=torch.zeros(2, dtype=torch.int32, device="cuda"), ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


def _refused(call):
    from confidence_block_unmasking_amd import _lib, api
    with pytest.raises((api.DllmError, ValueError)) as e:
        call()
    torch.cuda.synchronize()
    assert isinstance(e.value, ValueError) or e.value.code == _lib.DLLM_ERR_SHAPE


def test_tokens(small):
    from confidence_block_unmasking_amd import api
    ids = torch.empty(BIG + 2, dtype=torch.int32, device="cuda")
    rows = torch.zeros((BIG + 2, 1), dtype=torch.bfloat16, device="cuda")
    table = torch.ones((4, 1), dtype=torch.float32, device="cuda")
    _refused(lambda: api.dllm_embed(table, ids, rows, small["status"]))
    _refused(lambda: api.dllm_embed_grad(rows, ids, table, small["ws"], small["status"]))
    assert not rows[:8].any() and (table == 1.0).all() and int(small["status"].item()) == 0
    assert api.dllm_embed_grad_workspace_bytes(BIG + 2, 4, 4) == 0


def test_table_rows_and_columns(small):
    from confidence_block_unmasking_amd import api
    flat = torch.empty(BIG + 4, dtype=torch.bfloat16, device="cuda")
    _refused(lambda: api.dllm_embed(flat.view(-1, 1), small["ids"], small["out"][:, :1], small["status"]))
    _refused(lambda: api.dllm_embed(flat.view(1, -1), small["ids"], flat.view(1, -1).expand(2, -1), small["status"]))
    _refused(lambda: api.dllm_embed_grad(small["out"][:, :1], small["ids"], flat.view(-1, 1), small["ws"], small["status"]))
    assert (small["out"] == 7.0).all()
    assert api.dllm_embed_grad_workspace_bytes(8, BIG + 4, 4) == 0 and api.dllm_embed_grad_workspace_bytes(8, 4, BIG + 4) == 0


def test_logits(small):
    from confidence_block_unmasking_amd import api
    flat = torch.zeros(BIG + 4, dtype=torch.bfloat16, device="cuda")
    f = dict(dtype=torch.float32, device="cuda")
    lp, one = torch.full((8,), 7.0, **f), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    mask, stats, gl = torch.ones(8, dtype=torch.uint8, device="cuda"), torch.zeros(16, **f), torch.ones(8, **f)
    _refused(lambda: api.dllm_logprobs(flat.view(1, 1, -1), mask, one, lp, small["ws"], small["status"]))
    _refused(lambda: api.dllm_logprobs_grad(flat.view(1, 1, -1), mask, one, stats, gl, flat.view(1, 1, -1), small["status"]))
    _refused(lambda: api.dllm_logprobs(flat[:4].view(1, 1, 4), mask, one, lp, small["ws"], small["status"], k=BIG))
    assert (lp == 7.0).all() and not flat.any() and int(small["status"].item()) == 0
    assert api.dllm_logprobs_workspace_bytes(1, 1, BIG + 4) == 0 and api.dllm_logprobs_workspace_bytes(1, 1, 4, BIG) == 0
    assert api.dllm_logprobs_workspace_bytes(BIG + 1, 1, 4) == 0
