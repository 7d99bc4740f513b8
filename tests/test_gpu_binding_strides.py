"""Logits that are not [rows, L, V], padded between slots, and without strides given: what lies where is not
known, and the calls refuse them instead of reading them as packed."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_padded_matrix_of_logits_needs_its_strides():
    from confidence_block_unmasking_amd import api
    rows, L, V, pitch = 2, 3, 40, 48
    f = dict(dtype=torch.float32, device="cuda")
    buf = torch.randn((rows * L + 4, pitch), **f)
    lg = buf[:rows * L, :V]
    mask, tok = torch.ones((rows, L), dtype=torch.uint8, device="cuda"), torch.zeros((rows, L), dtype=torch.int32, device="cuda")
    lp, gl, sta = torch.full((rows, L), 7.0, **f), torch.ones((rows, L), **f), torch.zeros((rows, L, 2), **f)
    ws, st = api.new_logprobs_workspace(rows, L, V, 0, torch.float32), torch.zeros(1, dtype=torch.int32, device="cuda")
    size = dict(rows=rows, L=L, V=V)
    with pytest.raises(ValueError):
        api.dllm_logprobs(lg, mask, tok, lp, ws, st, **size)
    assert (lp == 7.0).all()
    grad = torch.full((rows * L + 4, pitch), 7.0, **f)
    packed = lg.contiguous()
    with pytest.raises(ValueError):
        api.dllm_logprobs_grad(packed, mask, tok, sta, gl, grad[:rows * L, :V], st, **size)
    with pytest.raises(ValueError):
        api.dllm_logprobs_grad(lg, mask, tok, sta, gl, torch.empty_like(packed), st, **size)
    assert (grad == 7.0).all()
    # packed, or with the strides, they are taken
    api.dllm_logprobs(packed, mask, tok, lp, ws, st, stats=sta, **size)
    again, s2 = torch.zeros_like(lp), torch.zeros_like(sta)
    api.dllm_logprobs(lg, mask, tok, again, ws, st, stats=s2, pos_stride=pitch, row_stride=L * pitch, **size)
    assert torch.equal(lp, again) and torch.equal(sta, s2)
    other = torch.empty_like(packed)
    api.dllm_logprobs_grad(packed, mask, tok, sta, gl, other, st, **size)
    api.dllm_logprobs_grad(lg, mask, tok, sta, gl, grad[:rows * L, :V], st, pos_stride=pitch, row_stride=L * pitch,
                           grad_pos_stride=pitch, grad_row_stride=L * pitch, **size)
    assert torch.equal(grad[:rows * L, :V], other) and (grad[:, V:] == 7.0).all() and (grad[rows * L:] == 7.0).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("make,strides", [
    (lambda b: b[:100], {}), (lambda b: b[:239], {}), (lambda b: b[:240], dict(grad_pos_stride=41, grad_row_stride=123)),
    (lambda b: b[:240].view(6, 40)[:5], {}), (lambda b: b[:240].view(2, 3, 40), dict(grad_pos_stride=48, grad_row_stride=144)),
    (lambda b: b[:0], {})])
def test_gradient_stays_in_its_tensor(make, strides):
    """A view too small for the gradient, in a storage that would hold it: what lies behind the view is
    not the call's."""
    from confidence_block_unmasking_amd import api
    rows, L, V = 2, 3, 40
    f = dict(dtype=torch.float32, device="cuda")
    buf = torch.full((4096,), 7.0, **f)
    mask, tok = torch.ones((rows, L), dtype=torch.uint8, device="cuda"), torch.zeros((rows, L), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        api.dllm_logprobs_grad(torch.randn((rows, L, V), **f), mask, tok, torch.zeros((rows, L, 2), **f), torch.ones((rows, L), **f),
                               make(buf), st, rows=rows, L=L, V=V, **strides)
    torch.cuda.synchronize()
    assert (buf == 7.0).all()


def test_gradient_into_views_that_hold_it():
    from confidence_block_unmasking_amd import api
    rows, L, V = 2, 3, 40
    f = dict(dtype=torch.float32, device="cuda")
    lg = torch.randn((rows, L, V), **f)
    mask, tok = torch.ones((rows, L), dtype=torch.uint8, device="cuda"), torch.zeros((rows, L), dtype=torch.int32, device="cuda")
    sta, one, st = torch.zeros((rows, L, 2), **f), torch.ones((rows, L), **f), torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = torch.empty((rows, L, V), **f)
    api.dllm_logprobs_grad(lg, mask, tok, sta, one, ref, st)
    for shape, strides, pitch in (((240,), {}, 40), ((6, 40), {}, 40), ((300,), {}, 40),
                                  ((286,), dict(grad_pos_stride=48, grad_row_stride=150), 48)):
        buf = torch.full((512,), 7.0, **f)
        n = 1
        for d in shape:
            n *= d
        api.dllm_logprobs_grad(lg, mask, tok, sta, one, buf[:n].view(shape), st, rows=rows, L=L, V=V, **strides)
        at = [(r * strides.get("grad_row_stride", L * pitch) + j * pitch, r, j) for r in range(rows) for j in range(L)]
        for a, r, j in at:
            assert torch.equal(buf[a:a + V], ref[r, j])
        assert (buf[at[-1][0] + V:] == 7.0).all()
    assert int(st.item()) == 0
