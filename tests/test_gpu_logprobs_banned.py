"""The gradient where columns are banned (-inf), the given token's own among them: 0 in every banned
column, and at the token gl (1 - 0), as the formula has it."""
import numpy as np
import pytest

from tests.test_gpu_logprobs import DT, check_grad, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("V,dtype", [(9, "fp32"), (4103, "bf16"), (20011, "fp32")])
@pytest.mark.parametrize("entropy", [False, True])
def test_banned_columns(V, dtype, entropy):
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(V)
    n = 6
    t = torch.from_numpy((rng.normal(size=(1, n, V)) * 2).astype(np.float32)).to(DT[dtype])
    t[0, :, V // 3:] = -float("inf")
    tokens = np.array([[0, V // 3 - 1, V // 3, V // 2, V - 2, V - 1]])
    g, st = run(t.view(-1).cuda(), 1, n, V, V, 0, np.ones((1, n), bool), tokens, 0)
    assert st == 0 and np.isneginf(g["logprob"][0, 2:]).all() and np.isfinite(g["logprob"][0, :2]).all()
    f = dict(dtype=torch.float32, device="cuda")
    gl = torch.from_numpy(rng.normal(size=(1, n)).astype(np.float32)).cuda()
    gh = torch.from_numpy(rng.normal(size=(1, n)).astype(np.float32)).cuda()
    out, st = torch.full((1, n, V), 9.0, dtype=DT[dtype], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ent = dict(entropy=torch.from_numpy(g["entropy"]).cuda(), grad_entropy=gh) if entropy else {}
    api.dllm_logprobs_grad(t.cuda(), torch.ones((1, n), dtype=torch.uint8, device="cuda"),
                           torch.from_numpy(tokens.astype(np.int32)).cuda(), torch.from_numpy(g["stats"]).cuda(), gl, out, st, **ent)
    assert int(st.item()) == 0
    got, x = out[0].double().cpu().numpy(), t[0].double().numpy()
    for i in range(n):
        tok = tokens[0, i]
        banned = np.isneginf(x[i])
        assert not got[i][banned & (np.arange(V) != tok)].any(), i
        if banned[tok]:
            assert got[i][tok] == gl[0, i].to(DT[dtype]).item(), i
        check_grad(got[i], x[i], tok, gl[0, i].item(), gh[0, i].item() if entropy else 0.0, dtype, f"{i}")
