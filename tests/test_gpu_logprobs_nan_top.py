"""Alternatives of slots that hold NaN (of either sign, quiet or signalling): their order is not
specified, but every place is written with a column of its own and reads NaN."""
import numpy as np
import pytest

from tests.test_gpu_logprobs import DT, check, run
from tests.test_gpu_logprobs_nan import _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("V,k,dtype", [(5, 5, "fp32"), (9, 9, "bf16"), (9, 4, "fp32"), (32, 32, "bf16"), (4097, 20, "bf16"),
                                       (6145, 32, "fp32"), (70000, 20, "fp32"), (152064, 20, "bf16")])
@pytest.mark.parametrize("rows", [1, 13])
def test_alternatives_of_slots_with_nan(V, k, dtype, rows):
    rng = np.random.default_rng(V + rows + k)
    print(f"nan alternatives V={V} k={k} {dtype} rows={rows}", flush=True)
    t, bad = _rows(V, dtype, rng)
    n = len(bad)
    mask = np.zeros((rows, n), bool)
    mask[rows // 2] = True
    box = torch.zeros((rows, n, V), dtype=DT[dtype])
    box[rows // 2] = t
    x = t.double().numpy()
    tokens = np.full((rows, n), V // 2)
    g, st = run(box.view(-1).cuda(), rows, n, V, V, 0, mask, tokens, k)
    assert st == 0
    got = {name: a[rows // 2] for name, a in g.items()}
    for i in range(n):
        ids = got["top_ids"][i]
        assert ((ids >= 0) & (ids < V)).all() and len(set(ids.tolist())) == k, (i, ids)
        if bad[i]:
            assert np.isnan(got["logprob"][i]) and np.isnan(got["entropy"][i]), i
            assert np.isnan(got["top_logprobs"][i]).all(), (i, got["top_logprobs"][i])
        else:
            one = {name: a[None, i:i + 1] for name, a in got.items()}
            check(one, x[None, i:i + 1], np.ones((1, 1), bool), tokens[:1, :1], k, f"row {i}")
    assert (g["top_ids"][~mask] == -5).all() and (g["top_logprobs"][~mask] == 55.0).all()
