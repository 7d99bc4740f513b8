"""Slots that hold NaN or +inf beside columns of -inf, on the GPU: every log probability and the entropy
read NaN wherever in the row the NaN lies, and the slots beside them keep their values.  The widths
take the last column into a vector, and a chunk (2048 columns of fp32, 4096 of bf16), of its own; a box
of few slots and short rows is finished by one kernel, any other by two."""
import numpy as np
import pytest

from tests.test_gpu_logprobs import DT, check, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# sign set, quiet and signalling patterns
NANS = {"bf16": [0x7FC0, 0xFFC0, 0x7F81, 0xFF81, 0xFFFF], "fp32": [0x7FC00000, 0xFFC00000, 0x7F800001, 0xFF800001, 0xFFFFFFFF]}
CHUNK = {"bf16": 4096, "fp32": 2048}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rows(V, dtype, rng):
    """(host tensor [n, V], bad [n]): rows with a NaN or +inf in every kind of place, finite ones between."""
    C, inf = CHUNK[dtype], float("inf")
    x = (rng.normal(size=(64, V)) * 2).astype(np.float32)
    t = torch.from_numpy(x).to(DT[dtype])
    raw = t.view(torch.int16 if dtype == "bf16" else torch.int32)
    bits = [int(np.array(p, np.uint32).astype(np.int32)) if dtype == "fp32" else int(np.array(p, np.uint16).view(np.int16))
            for p in NANS[dtype]]
    bad, n = np.zeros(64, bool), 0

    def row(is_bad=True):
        nonlocal n
        bad[n] = is_bad
        n += 1
        return n - 1

    for b in bits:
        raw[row(), V - 1] = b                              # the last column
        r = row()                                          # the last chunk: one NaN, else banned
        t[r, (V - 1) // C * C:] = -inf
        raw[r, V - 1] = b
        r = row()                                          # the first chunk (all of a short row)
        t[r, :min(C, V)] = -inf
        raw[r, min(C, V) // 2] = b
        r = row()                                          # a chunk of NaN
        raw[r, V // (2 * C) * C:V // (2 * C) * C + C] = b
        r = row()                                          # nothing but NaN
        raw[r] = b
        r = row()                                          # a NaN among banned columns only
        t[r] = -inf
        raw[r, V // 3] = b
        r = row()                                          # NaN, a single finite column, else banned
        t[r] = -inf
        t[r, V // 2] = 1.0
        raw[r, V - 1 if V // 2 != V - 1 else 0] = b
        row(False)
    r = row()                                              # +inf alone in its chunk
    t[r, (V - 1) // C * C:] = -inf
    t[r, V - 1] = inf
    r = row()                                              # +inf and NaN
    t[r, 0] = inf
    raw[r, V - 1] = bits[0]
    t[row()] = -inf                                        # all banned
    r = row(False)                                         # all banned but the last column
    t[r] = -inf
    t[r, V - 1] = -3.0
    return t[:n], bad[:n]


@pytest.mark.parametrize("V,dtype", [(9, "fp32"), (4097, "bf16"), (6145, "fp32"), (20011, "bf16"), (70000, "fp32"), (152064, "bf16"),
                                     (300000, "bf16")])
@pytest.mark.parametrize("rows", [1, 13])
@pytest.mark.parametrize("entropy,k", [(True, 0), (False, 0)])
def test_nan_anywhere_in_a_slot(V, dtype, rows, entropy, k):
    rng = np.random.default_rng(V + rows)
    print(f"nan V={V} {dtype} rows={rows} entropy={entropy} k={k}", flush=True)
    t, bad = _rows(V, dtype, rng)
    n = len(bad)
    mask = np.zeros((rows, n), bool)
    mask[rows // 2] = True                                 # the other rows of a box are not selected
    box = torch.zeros((rows, n, V), dtype=DT[dtype])
    box[rows // 2] = t
    x = t.double().numpy()
    tokens = np.full((rows, n), V // 2)
    g, st = run(box.view(-1).cuda(), rows, n, V, V, 0, mask, tokens, k, entropy=entropy)
    assert st == 0
    got = {name: None if a is None else a[rows // 2] for name, a in g.items()}
    assert np.isnan(got["logprob"][bad]).all(), np.flatnonzero(bad & ~np.isnan(got["logprob"]))
    assert not entropy or np.isnan(got["entropy"][bad]).all()
    assert not np.isfinite(got["stats"][bad, 1]).any()
    for i in np.flatnonzero(~bad):
        one = {name: None if a is None else a[None, i:i + 1] for name, a in got.items()}
        check(one, x[None, i:i + 1], np.ones((1, 1), bool), tokens[:1, :1], k, f"row {i}")
    assert (g["logprob"][~mask] == 55.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_of_slots_without_a_distribution_is_nan(dtype):
    """From the forward's own statistics: every column of such a slot, and of no other."""
    from confidence_block_unmasking_amd import api
    V = CHUNK[dtype] + 1
    t, bad = _rows(V, dtype, np.random.default_rng(3))
    n = len(bad)
    g, _ = run(t.view(-1).cuda(), 1, n, V, V, 0, np.ones((1, n), bool), np.full((1, n), V // 2), 0)
    out = torch.zeros((1, n, V), dtype=DT[dtype], device="cuda")
    one = torch.ones((1, n), dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for ent in ({}, dict(entropy=torch.from_numpy(g["entropy"]).cuda(), grad_entropy=one)):
        api.dllm_logprobs_grad(t.view(1, n, V).cuda(), torch.ones((1, n), dtype=torch.uint8, device="cuda"),
                               torch.full((1, n), V // 2, dtype=torch.int32, device="cuda"),
                               torch.from_numpy(g["stats"]).cuda(), one, out, st, **ent)
        nan = out[0].isnan().cpu().numpy()
        assert nan[bad].all() and not nan[~bad].any()
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_of_a_nan_logit_is_nan_whatever_the_statistics(dtype, entropy):
    """Statistics of other logits (a caller's mistake) do not hide a NaN: its column reads NaN, the others
    the formula's values."""
    from confidence_block_unmasking_amd import api
    V, f = 1030, dict(dtype=torch.float32, device="cuda")
    t = torch.randn((1, 2, V), generator=torch.Generator().manual_seed(5)).to(DT[dtype])
    g, _ = run(t.view(-1).cuda(), 1, 2, V, V, 0, np.ones((1, 2), bool), np.zeros((1, 2)), 0)
    one, st = torch.ones((1, 2), **f), torch.zeros(1, dtype=torch.int32, device="cuda")
    ent = dict(entropy=torch.from_numpy(g["entropy"]).cuda(), grad_entropy=one) if entropy else {}
    out = []
    for plant in (False, True):
        x = t.clone()
        if plant:
            x[0, 1, [3, V - 1]] = float("nan")
        out.append(torch.zeros((1, 2, V), dtype=DT[dtype], device="cuda"))
        api.dllm_logprobs_grad(x.cuda(), torch.ones((1, 2), dtype=torch.uint8, device="cuda"),
                               torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.from_numpy(g["stats"]).cuda(), one, out[-1], st,
                               **ent)
    nan = torch.zeros((1, 2, V), dtype=torch.bool, device="cuda")
    nan[0, 1, [3, V - 1]] = True
    assert torch.equal(out[1].isnan(), nan) and torch.equal(out[1][~nan], out[0][~nan])
