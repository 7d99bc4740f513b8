"""The probabilities that the gradient is made of err to both sides of the formula's."""
import numpy as np
import pytest

from tests.test_gpu_logprobs import U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("V,sd", [(20011, 2.0), (126464, 4.0)])
def test_probabilities_err_to_both_sides(V, sd):
    """Over the columns of many slots the relative errors of p, roundings of either sign, average out.  With
    log2 e as one float, 0.224 u of itself too small, every p would be too large by 0.224 u |log p| of itself; at
    most half of that is left on average."""
    from confidence_block_unmasking_amd import api
    n = 48
    rng = np.random.default_rng(V)
    x = (rng.standard_normal((n, V), np.float32) * np.float32(sd)).astype(np.float32)
    u = x.astype(np.float64) - x.max(1, keepdims=True)
    ls = np.log(np.exp(u).sum(1))
    sta = np.stack([x.max(1), ls], 1).astype(np.float32)[None]
    f = dict(dtype=torch.float32, device="cuda")
    out, st = torch.zeros((1, n, V), **f), torch.zeros(1, dtype=torch.int32, device="cuda")
    tok = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    api.dllm_logprobs_grad(torch.from_numpy(x).cuda().view(1, n, V), torch.ones((1, n), dtype=torch.uint8, device="cuda"), tok,
                           torch.from_numpy(sta).cuda(), torch.ones((1, n), **f), out, st)
    assert int(st.item()) == 0
    got = -out[0, :, 1:].double().cpu().numpy()               # column 0 is the token's
    logp = (u - sta[0, :, 1:].astype(np.float64))[:, 1:]
    rel = (got / np.exp(logp) - 1) / U
    print(f"mean relative error {rel.mean():.2f} u, mean |log p| {-logp.mean():.1f}", flush=True)
    assert abs(rel.mean()) <= 0.112 * -logp.mean()
