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


@pytest.mark.parametrize("name,shape", [
    ("logprob", (2, 7)), ("logprob", (3, 2, 7)), ("entropy", (2, 5)), ("mask", (2, 6)), ("exclude", (4, 5)), ("stats", (2, 7, 2)),
    ("stats", (8, 3)), ("top_ids", (2, 7, 3)), ("top_logprobs", (2, 5, 3))])
def test_wider_rows_are_refused(name, shape):
    """Rows of more than L entries: the call would use them L apart."""
    from confidence_block_unmasking_amd import api
    a, top = _forward(), _top(3, 3)
    f = dict(dtype=torch.float32, device="cuda")
    kw = dict(a, **top, entropy=torch.full((2, 4), 7.0, **f), stats=torch.full((2, 4, 2), 7.0, **f))
    kw[name] = torch.full(shape, 7, dtype={"mask": torch.uint8, "exclude": torch.uint8, "top_ids": torch.int32}.get(name, torch.float32),
                          device="cuda")
    with pytest.raises(ValueError):
        api.dllm_logprobs(**kw)
    torch.cuda.synchronize()
    assert name == "logprob" or (a["logprob"] == 7.0).all()


@pytest.mark.parametrize("name,shape", [("mask", (2, 6)), ("exclude", (2, 5)), ("stats", (2, 7, 2)), ("grad_logprob", (2, 9)),
                                        ("entropy", (3, 5)), ("grad_entropy", (2, 2, 5))])
def test_wider_rows_are_refused_by_the_gradient(name, shape):
    from confidence_block_unmasking_amd import api
    a = _forward()
    f = dict(dtype=torch.float32, device="cuda")
    out = torch.full((2, 4, 50), 7.0, **f)
    kw = dict(logits=a["logits"], mask=a["mask"], tokens=a["tokens"], status=a["status"], grad_logits=out,
              stats=torch.zeros((2, 4, 2), **f), grad_logprob=torch.ones((2, 4), **f), entropy=torch.ones((2, 4), **f),
              grad_entropy=torch.ones((2, 4), **f))
    kw[name] = torch.ones(shape, dtype=torch.uint8 if name in ("mask", "exclude") else torch.float32, device="cuda")
    with pytest.raises(ValueError):
        api.dllm_logprobs_grad(**kw)
    torch.cuda.synchronize()
    assert (out == 7.0).all()


def test_more_rows_than_the_call_has_and_flat_buffers_are_taken():
    from confidence_block_unmasking_amd import api
    a, f = _forward(), dict(dtype=torch.float32, device="cuda")
    ref = dict(logprob=torch.zeros((2, 4), **f), entropy=torch.zeros((2, 4), **f), stats=torch.zeros((2, 4, 2), **f))
    api.dllm_logprobs(**{**a, **ref})
    for shapes in (((6, 4), (3, 4), (5, 4, 2)), ((11,), (9,), (17,)), ((1, 3, 4), (8, 1), (12, 2)), ((4, 2), (2, 4), (16, 1))):
        got = {n: torch.full(s, 7.0, **f) for n, s in zip(("logprob", "entropy", "stats"), shapes)}
        mask = torch.ones(9 if len(shapes[0]) == 1 else (4, 4), dtype=torch.uint8, device="cuda")
        api.dllm_logprobs(**{**a, **got, "mask": mask})
        for n, t in got.items():
            m = ref[n].numel()
            assert torch.equal(t.view(-1)[:m], ref[n].view(-1)) and (t.view(-1)[m:] == 7.0).all(), (n, shapes)
    assert int(a["status"].item()) == 0


def test_no_alternatives_into_buffers_for_some():
    """k = 0 leaves the buffers of another call alone."""
    from confidence_block_unmasking_amd import api
    a, top = _forward(), _top(5, 5)
    api.dllm_logprobs(**a, **top, k=0)
    torch.cuda.synchronize()
    assert (top["top_ids"] == -5).all() and (top["top_logprobs"] == 7.0).all() and (a["logprob"] <= 0).all()
