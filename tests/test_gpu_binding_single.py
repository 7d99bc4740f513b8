"""One row, or one slot per row: the stride of a dimension of size 1 says nothing (a tensor from numpy's
x[None] has 0 there, a transposed one a large one), and the calls take such tensors as any other."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _run(lg, grad):
    from confidence_block_unmasking_amd import api
    rows, L, V = lg.shape
    f = dict(dtype=torch.float32, device="cuda")
    mask, tok = torch.ones((rows, L), dtype=torch.uint8, device="cuda"), torch.zeros((rows, L), dtype=torch.int32, device="cuda")
    lp, sta, st = torch.zeros((rows, L), **f), torch.zeros((rows, L, 2), **f), torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dllm_logprobs(lg, mask, tok, lp, api.new_logprobs_workspace(rows, L, V, 0, lg.dtype), st, stats=sta)
    api.dllm_logprobs_grad(lg, mask, tok, sta, torch.ones((rows, L), **f), grad, st)
    out, done, acc = mask.clone(), torch.zeros(rows, dtype=torch.uint8, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    conf = torch.zeros((rows, L), **f)
    api.dllm_step(lg if grad is not lg else torch.zeros((rows, L, V), **f), tok.clone(), mask, out, torch.full((rows,), 0.5, **f), done, acc,
                  api.new_workspace(rows, L, V, lg.dtype), st, conf=conf)
    assert int(st.item()) == 0
    return lp.view(-1), sta.view(-1), grad.reshape(-1).clone(), conf.view(-1)


def _same(a, b, n=4):
    return all(torch.equal(x, y) for x, y in zip(a[:n], b[:n]))


def test_one_row():
    x = np.random.default_rng(0).standard_normal((6, 33), np.float32)
    ref = _run(torch.from_numpy(x).cuda().view(1, 6, 33), torch.empty((1, 6, 33), device="cuda"))
    odd = torch.from_numpy(x[None]).cuda()
    strange = odd.as_strided((1, 6, 33), (0, 33, 1))
    huge = odd.as_strided((1, 6, 33), (1 << 40, 33, 1))
    for t in (odd, strange, huge):
        assert _same(_run(t, torch.empty((1, 6, 33), device="cuda")), ref)
        assert _same(_run(t, torch.empty((6, 33), device="cuda").as_strided((1, 6, 33), (0, 33, 1))), ref)
    assert _same(_run(strange, strange), ref, 3)                 # in place


def test_one_slot_per_row():
    x = torch.randn((5, 40), device="cuda")
    ref = _run(x.view(5, 1, 40), torch.empty((5, 1, 40), device="cuda"))
    turned = x.view(1, 5, 40).transpose(0, 1)                     # strides (40, 200, 1)
    for t in (turned, x.as_strided((5, 1, 40), (40, 0, 1))):
        assert _same(_run(t, torch.empty((5, 1, 40), device="cuda")), ref)
        assert _same(_run(t, torch.empty((1, 5, 40), device="cuda").transpose(0, 1)), ref)
    one = x[:1].as_strided((1, 1, 40), (0, 0, 1))
    assert torch.equal(_run(one, torch.empty((1, 1, 40), device="cuda"))[0], ref[0][:1])
    padded = torch.randn((5, 3, 64), device="cuda")[:, 1:2, :40]
    assert _same(_run(padded, torch.empty((5, 1, 40), device="cuda")), _run(padded.contiguous(), torch.empty((5, 1, 40), device="cuda")))
