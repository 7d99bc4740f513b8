"""Slots whose distribution is nearly all at one token (the ones a step unmasks): log probability, log S and
entropy to a relative error, however near 0 they are.

With r the sum of the other powers, log S = log(1 + r), and the token's log probability is its negative.
Terms of r are off by (2.3 |x - m| + 3) u of themselves (one FMA's rounding within a chunk, or those of a
difference and a product between chunks, the constant log2 e, the power), their sum by 51 u (additions, across lanes and chunks); where a chunk's own sum is 1.25 or more
the 24 roundings of up to u that beside the 1 go into it are at most 96 u of its r.  log(1 + r) adds a few.
The entropy is log S plus the sum of p |x - m| over the others, all of one sign, whose terms are off by
(2.3 |x - m| + 5) u of themselves: with E1 and E2 the means of |x - m| and (x - m)^2 under the others alone,
the relative errors are at most u (2.3 E1 + 155) and u (2.3 E2 / E1 + 160).  Beside that, a power below the
least normal float, 2^-126, reads 0: each of at most V - 1 takes less than 2^-126 off r, and its term p |x - m|,
which falls as |x - m| grows past 126 ln 2, less than 2^-126 88 off the entropy's sum.
"""
import numpy as np
import pytest

from tests.test_gpu_logprobs import DT, U, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _reference(x):
    at = int(x.argmax())
    u = np.delete(x, at) - x[at]
    e = np.exp(u)
    r = e.sum()
    q = e / r if r > 0 else e
    E1, E2 = (q * np.where(e > 0, -u, 0)).sum(), (q * np.where(e > 0, u * u, 0)).sum()
    ls = np.log1p(r)
    return at, ls, ls + r * E1 / (1 + r), E1, E2


@pytest.mark.parametrize("rows", [1, 20])                      # 30 and 600 slots: one kernel (short rows) and two
@pytest.mark.parametrize("V,dtype", [(2, "fp32"), (9, "bf16"), (40, "fp32"), (2049, "fp32"), (4097, "bf16"), (20011, "bf16"),
                                     (40000, "bf16"), (126464, "fp32")])
@pytest.mark.parametrize("offset,entropy,k", [(0.0, True, 0), (0.0, False, 3), (16384.0, True, 2), (-3.0e6, True, 0)])
def test_confident_slots(rows, V, dtype, offset, entropy, k):
    rng = np.random.default_rng(V)
    k = min(k, V)
    n = 30
    x = (rng.normal(size=(n, V)) * 2).astype(np.float32)
    at = rng.integers(0, V, n)
    at[:4] = [0, V - 1, V // 2, (V - 1) // 8 * 8]
    for i in range(n):
        x[i, at[i]] = x[i].max() + 1 + 3 * i                  # p from about 0.5 to 1 - 1e-38
    x[n - 1] = -np.inf
    x[n - 1, at[n - 1]] = 2.0                                  # p = 1
    x[n - 2, :] = x[n - 2, at[n - 2]]                          # no token apart from the others
    t = torch.from_numpy(x + np.float32(offset)).to(DT[dtype])
    x = t.double().numpy()
    mask = np.zeros((rows, n), bool)
    mask[rows // 2] = True
    box = torch.zeros((rows, n, V), dtype=DT[dtype])
    box[rows // 2] = t
    ref = [_reference(v) for v in x]
    tokens = np.tile(np.array([o[0] for o in ref]), (rows, 1))
    g, st = run(box.view(-1).cuda(), rows, n, V, V, 0, mask, tokens, k, entropy=entropy)
    assert st == 0
    got = {a: None if b is None else b[rows // 2] for a, b in g.items()}
    for i, (tok, ls, H, E1, E2) in enumerate(ref):
        tol = U * (2.3 * E1 + 155) * ls + TINY * V
        where = (i, ls, got["logprob"][i], got["stats"][i, 1], (got["stats"][i, 1] - ls) / (U * ls + 1e-45))
        assert abs(got["stats"][i, 1] - ls) <= tol, where
        assert abs(got["logprob"][i] + ls) <= tol, where
        if k:
            assert got["top_ids"][i, 0] == tok and abs(got["top_logprobs"][i, 0] + ls) <= tol, where
        if entropy:
            tolH = U * (2.3 * (E2 / E1 if E1 > 0 else 0.0) + 160) * H + TINY * V * 128
            assert abs(got["entropy"][i] - H) <= tolH, (i, H, got["entropy"][i], (got["entropy"][i] - H) / (U * H + 1e-45))


@pytest.mark.parametrize("d", [20, 30])
def test_log_sums_err_to_both_sides(d):
    """Over many slots the relative error of r averages out: roundings have no sign.  Powers of 2 with
    log2 e as one float, which is 1.33e-8 of itself (0.224 u) too small, would make every term too large
    by 0.224 u |x - m|: 0.224 d u on average.  At most half of that is left."""
    n, V = 200, 126464
    rng = np.random.default_rng(d)
    x = (rng.standard_normal((n, V), np.float32) - np.float32(d))
    x[np.arange(n), rng.integers(0, V, n)] = 0.0
    x += (8 * rng.random((n, 1)) - 4).astype(np.float32)
    t = torch.from_numpy(x)
    g, st = run(t.view(-1).cuda(), 1, n, V, V, 0, np.ones((1, n), bool), np.zeros((1, n)), 0)
    assert st == 0
    ls = np.array([_reference(v.astype(np.float64))[1] for v in x])
    rel = (g["stats"][0, :, 1] - ls) / (U * ls)
    print(f"mean relative error {rel.mean():.2f} u, std {rel.std():.2f} u", flush=True)
    assert abs(rel.mean()) <= 0.112 * d
