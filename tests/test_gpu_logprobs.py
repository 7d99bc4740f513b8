"""dllm_logprobs and dllm_logprobs_grad on the GPU against the float64 oracle.

Tolerances count float32 roundings, u = 2^-24 each, from the arithmetic (y = (x - m) log2 e by one
FMA, 2^y to one unit in the last place, fixed summation trees):
  log S   every term is off by at most (1.3 |x - m| + 3) u of itself (the FMA's rounding, the constant
          log2 e, the power), the sum by 48 u (16 additions per accumulator, 2 to join four, 6 across
          lanes, the residual's factor, and at most 22 more across chunks for V <= 160000): in all
          (1.3 E1 + 51) u, E1 the mean of |x - m| under the distribution; the logarithm 2 u ln V.
  logprob that, plus one rounding each of x_t - m and of the result: 2 u |logprob| + 2 u |x_t - m|.
  entropy log S - T/S with T = sum e y: terms of T are off by (1.3 |x - m| + 5) u of themselves, the
          sums by 48 u, so u (1.3 E2 + 53 E1 + E1 (1.3 E1 + 51)) beside log S, and 2 u of the result.
  gradient p by the given statistics: (3 |log p| + 2 log S + 8) u of itself, its factor 4 u of
          |gl| + |gh| (|log p| + H), one rounding for the added gl, half a step of the type for the result.
"""
import math

import numpy as np
import pytest

from oracle import logprobs as olp

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U = 2.0 ** -24
FMAX = float(np.finfo(np.float32).max)
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import confidence_block_unmasking_amd  # noqa: F401  (fails loudly if the library is missing)


def tol_logS(o, V):
    return U * (1.3 * o["E1"] + 51 + 2 * math.log(max(V, 2)))


def tol_logprob(o, V, lp):
    return tol_logS(o, V) + U * (2 * abs(lp) + 2 * abs(lp + o["logS"]))


def tol_entropy(o, V):
    return tol_logS(o, V) + U * (1.3 * o["E2"] + 53 * o["E1"] + o["E1"] * (1.3 * o["E1"] + 51) + 2 * o["entropy"])


def make_logits(rng, rows, L, V, dtype, pos_stride=None, offset=0, x=None, sd=2.0):
    """(flat device tensor whose slots lie pos_stride apart from `offset`, host float64 [rows, L, V])."""
    ps = pos_stride or V
    if x is None:
        x = (rng.normal(size=(rows, L, V)) * sd).astype(np.float32)
        x[np.arange(rows)[:, None], np.arange(L)[None, :], rng.integers(0, V, (rows, L))] += (
            14 * rng.random((rows, L))).astype(np.float32)
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DT[dtype])
    buf = torch.full((offset + rows * L * ps,), 776.0, dtype=DT[dtype])
    buf[offset:].view(rows * L, ps)[:, :V] = t.view(rows * L, V)
    return buf.cuda(), t.double().numpy().reshape(rows, L, V), ps


def run(buf, rows, L, V, ps, offset, mask, tokens, k, exclude=None, entropy=True, stats=True, stream=None, ws=None):
    from confidence_block_unmasking_amd import api
    f = dict(dtype=torch.float32, device="cuda")
    out = dict(logprob=torch.full((rows, L), 55.0, **f), entropy=torch.full((rows, L), 55.0, **f) if entropy else None,
               stats=torch.full((rows, L, 2), 55.0, **f) if stats else None,
               top_ids=torch.full((rows, L, k), -5, dtype=torch.int32, device="cuda") if k else None,
               top_logprobs=torch.full((rows, L, k), 55.0, **f) if k else None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = api.new_logprobs_workspace(rows, L, V, k, buf.dtype) if ws is None else ws
    ws.fill_(0xA5)
    mt = torch.from_numpy(mask.astype(np.uint8)).cuda()
    tt = torch.from_numpy(tokens.astype(np.int32)).cuda()
    et = None if exclude is None else torch.from_numpy(exclude.astype(np.uint8)).cuda()
    torch.cuda.synchronize()
    api.dllm_logprobs(buf[offset:], mt, tt, out["logprob"], ws, status, entropy=out["entropy"], stats=out["stats"],
                      top_ids=out["top_ids"], top_logprobs=out["top_logprobs"], exclude=et, rows=rows, L=L, V=V,
                      pos_stride=ps, row_stride=L * ps, stream=stream)
    torch.cuda.synchronize()
    return {n: None if t is None else t.cpu().numpy() for n, t in out.items()}, int(status.item())


def check(g, x, on, tokens, k, where=""):
    rows, L, V = x.shape
    for r in range(rows):
        for j in range(L):
            if not on[r, j]:
                assert g["logprob"][r, j] == 55.0
                for n in ("entropy", "stats", "top_logprobs"):
                    assert g[n] is None or (g[n][r, j] == 55.0).all(), n
                assert g["top_ids"] is None or (g["top_ids"][r, j] == -5).all()
                continue
            o = olp.slot(x[r, j], token=tokens[r, j], k=k)
            at = f"{where} slot {r},{j}"
            assert g["logprob"][r, j] <= 0 and (g["entropy"] is None or g["entropy"][r, j] >= 0), at
            assert g["top_logprobs"] is None or (g["top_logprobs"][r, j] <= 0).all(), at
            if np.isneginf(o["logprob"]) or o["logprob"] < -FMAX:
                assert np.isneginf(g["logprob"][r, j]), at
            else:
                assert abs(g["logprob"][r, j] - o["logprob"]) <= tol_logprob(o, V, o["logprob"]), at
            if g["entropy"] is not None:
                assert abs(g["entropy"][r, j] - o["entropy"]) <= tol_entropy(o, V), at
            if g["stats"] is not None:
                assert g["stats"][r, j, 0] == np.float32(o["m"]), at
                assert abs(g["stats"][r, j, 1] - o["logS"]) <= tol_logS(o, V), at
            if k:
                assert np.array_equal(g["top_ids"][r, j], o["top_ids"]), at
                for a, b in zip(g["top_logprobs"][r, j], o["top_logprobs"]):
                    assert np.isneginf(a) if b < -FMAX else abs(a - b) <= tol_logprob(o, V, b), at


CASES = [  # rows, L, V, dtype, k, share selected, extra stride, offset
    (1, 1, 1, "fp32", 1, 1.0, 0, 0), (1, 1, 1, "bf16", 1, 1.0, 0, 1), (3, 5, 2, "bf16", 2, 1.0, 1, 0),
    (2, 3, 7, "fp32", 7, 1.0, 2, 1), (2, 3, 8, "bf16", 8, 1.0, 0, 0), (4, 9, 9, "bf16", 3, 0.7, 4, 3),
    (5, 7, 33, "fp32", 32, 0.6, 1, 2), (2, 2, 511, "bf16", 20, 1.0, 0, 0), (3, 4, 1024, "fp32", 5, 0.5, 0, 0),
    (2, 3, 2048, "fp32", 20, 1.0, 0, 0), (2, 3, 2049, "fp32", 20, 1.0, 0, 0), (2, 2, 4096, "bf16", 32, 1.0, 0, 0),
    (2, 2, 4097, "bf16", 32, 1.0, 0, 0), (2, 2, 4103, "bf16", 1, 1.0, 8, 5), (3, 7, 20011, "fp32", 20, 0.8, 2, 0),
    (2, 8, 20011, "bf16", 5, 0.8, 3, 7), (1, 32, 126464, "bf16", 5, 0.04, 0, 0), (2, 16, 152064, "bf16", 20, 0.5, 0, 0),
    (1, 5, 152064, "fp32", 20, 1.0, 0, 0), (1, 3, 152063, "bf16", 32, 1.0, 1, 1), (6, 6, 3000, "bf16", 0, 0.5, 0, 0),
]


@pytest.mark.parametrize("rows,L,V,dtype,k,share,extra,offset", CASES)
def test_against_the_oracle(rows, L, V, dtype, k, share, extra, offset):
    rng = np.random.default_rng(V * 7 + k)
    print(f"logprobs rows={rows} L={L} V={V} {dtype} k={k}", flush=True)
    buf, x, ps = make_logits(rng, rows, L, V, dtype, V + extra, offset)
    mask = rng.random((rows, L)) < share
    mask[0, 0] = True
    tokens = rng.integers(0, V, (rows, L))
    tokens[0, 0] = x[0, 0].argmax()
    g, st = run(buf, rows, L, V, ps, offset, mask, tokens, k)
    assert st == 0
    check(g, x, mask, tokens, k)


@pytest.mark.parametrize("entropy,stats,k", [(False, True, 0), (True, False, 4), (False, False, 4)])
def test_optional_outputs(entropy, stats, k):
    rng = np.random.default_rng(9)
    buf, x, ps = make_logits(rng, 2, 5, 5000, "bf16")
    tokens = rng.integers(0, 5000, (2, 5))
    mask = np.ones((2, 5), bool)
    g, st = run(buf, 2, 5, 5000, ps, 0, mask, tokens, k, entropy=entropy, stats=stats)
    assert st == 0
    check(g, x, mask, tokens, k)


@pytest.mark.parametrize("rows,L,V,share", [(2000, 8, 70, 0.3), (4096, 64, 5, 0.02), (4096, 64, 3, 1.0), (300, 64, 130, 1.0),
                                            (1024, 32, 9, 0.0)])
def test_many_slots(rows, L, V, share):
    """More slots than one pass of the mask scan covers (8192), dense, sparse and none at all."""
    rng = np.random.default_rng(rows)
    buf, x, ps = make_logits(rng, rows, L, V, "bf16")
    mask = rng.random((rows, L)) < share
    exclude = rng.random((rows, L)) < 0.5
    tokens = rng.integers(0, V, (rows, L))
    g, st = run(buf, rows, L, V, ps, 0, mask, tokens, 3, exclude=exclude)
    assert st == 0
    on = mask & ~exclude
    assert (g["logprob"][~on] == 55.0).all() and (g["top_ids"][~on] == -5).all() and (g["stats"][~on] == 55.0).all()
    m = x.max(2, keepdims=True)
    S = np.exp(x - m).sum(2)
    lp = np.take_along_axis(x, tokens[:, :, None], 2)[:, :, 0] - m[:, :, 0] - np.log(S)
    assert np.abs(g["logprob"] - lp)[on].max(initial=0) <= U * (100 + 4 * np.abs(x).max() + 2 * np.abs(lp).max())
    assert np.array_equal(g["top_ids"][on], np.argsort(-x, axis=2, kind="stable")[:, :, :3][on])


def _special(kind, V, rng):
    x = rng.normal(size=V) * 2
    lowest = float(torch.finfo(torch.bfloat16).min)
    if kind == "minus-inf-tail":
        x[V // 3:] = -np.inf
    elif kind == "one-finite":
        x[:] = -np.inf
        x[V // 2] = 1.5
    elif kind == "lowest-tail":
        x[V // 3:] = lowest
    elif kind == "all-lowest":
        x[:] = lowest
    elif kind == "equal":
        x[:] = 3.0
    elif kind == "zeros-of-both-signs":
        x[:] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    elif kind == "ties":
        x = np.round(x)
    elif kind == "offset":
        x += 16384.0
    elif kind == "negative-offset":
        x -= 16384.0
    elif kind == "huge":
        x[:] = -1.0e38
        x[[1, V - 1]] = 3.0e38
    elif kind == "wide":
        x *= 40.0
    elif kind == "descending":
        x = np.sort(x)[::-1].copy()
    elif kind == "ascending":
        x = np.sort(x)
    elif kind == "max-in-tail-vector":
        x[V - 1] = 50.0
    return x


SPECIALS = ["minus-inf-tail", "one-finite", "lowest-tail", "all-lowest", "equal", "zeros-of-both-signs", "ties", "offset",
            "negative-offset", "huge", "wide", "descending", "ascending", "max-in-tail-vector"]


@pytest.mark.parametrize("V,dtype", [(9, "fp32"), (6001, "fp32"), (20011, "bf16"), (152064, "bf16")])
def test_special_rows(V, dtype):
    rng = np.random.default_rng(V)
    n = len(SPECIALS)
    x = np.stack([_special(s, V, rng) for s in SPECIALS])[None].astype(np.float32)
    buf, xr, ps = make_logits(rng, 1, n, V, dtype, x=x)
    tokens = rng.integers(0, V, (1, n))
    k = min(V, 20)
    g, st = run(buf, 1, n, V, ps, 0, np.ones((1, n), bool), tokens, k)
    assert st == 0
    for i, s in enumerate(SPECIALS):
        sub = {a: None if b is None else b[:, i:i + 1] for a, b in g.items()}
        check(sub, xr[:, i:i + 1], np.ones((1, 1), bool), tokens[:, i:i + 1], k, s)


@pytest.mark.parametrize("V,dtype", [(100, "fp32"), (9001, "bf16"), (100001, "bf16"), (70000, "fp32")])
def test_slots_without_a_distribution_read_nan(V, dtype):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(1, 4, V)).astype(np.float32)
    x[0, 0] = -np.inf
    x[0, 1, V - 3] = np.inf
    x[0, 2, V // 2] = np.nan
    buf, xr, ps = make_logits(rng, 1, 4, V, dtype, x=x)
    tokens = np.full((1, 4), 2)
    g, st = run(buf, 1, 4, V, ps, 0, np.ones((1, 4), bool), tokens, 5)
    assert st == 0
    assert np.isnan(g["logprob"][0, :3]).all() and np.isnan(g["entropy"][0, :3]).all()
    assert np.isnan(g["top_logprobs"][0, :3]).all()
    assert list(g["top_ids"][0, 0]) == [0, 1, 2, 3, 4] and g["top_ids"][0, 1, 0] == V - 3
    one = {a: b[:, 3:] for a, b in g.items()}
    check(one, xr[:, 3:], np.ones((1, 1), bool), tokens[:, 3:], 5)


@pytest.mark.parametrize("V,k", [(300, 2), (140000, 2), (140000, 0)])
def test_tokens_out_of_range_report_and_read_nan(V, k):
    rng = np.random.default_rng(2)
    buf, x, ps = make_logits(rng, 1, 4, V, "fp32")
    tokens = np.array([[-1, V, 7, 1 << 30]])
    g, st = run(buf, 1, 4, V, ps, 0, np.ones((1, 4), bool), tokens, k)
    assert st == 1
    assert np.isnan(g["logprob"][0, [0, 1, 3]]).all()
    o = olp.slot(x[0, 2], token=7)
    assert abs(g["logprob"][0, 2] - o["logprob"]) <= tol_logprob(o, V, o["logprob"])
    for j in range(4):                          # everything else is unaffected
        o = olp.slot(x[0, j], k=k)
        assert abs(g["entropy"][0, j] - o["entropy"]) <= tol_entropy(o, V)
        assert k == 0 or np.array_equal(g["top_ids"][0, j], o["top_ids"])


def test_bits_depend_on_the_slot_alone():
    """A slot scored alone, in a full box and again gives the same bits."""
    rng = np.random.default_rng(5)
    rows, L, V = 24, 32, 20011
    buf, x, ps = make_logits(rng, rows, L, V, "bf16")
    tokens = rng.integers(0, V, (rows, L))
    full, _ = run(buf, rows, L, V, ps, 0, np.ones((rows, L), bool), tokens, 20)
    again, _ = run(buf, rows, L, V, ps, 0, np.ones((rows, L), bool), tokens, 20)
    for n in full:
        assert np.array_equal(full[n].view(np.uint32), again[n].view(np.uint32)), n
    mask = np.zeros((rows, L), bool)
    mask[17, 3] = True
    one, _ = run(buf, rows, L, V, ps, 0, mask, tokens, 20)
    for n in full:
        assert np.array_equal(full[n][17, 3].view(np.uint32), one[n][17, 3].view(np.uint32)), n
    # a box of one row is finished by one kernel, the box of 768 slots by two
    row, _ = run(buf[17 * L * V:], 1, L, V, ps, 0, np.ones((1, L), bool), tokens[17:18], 20)
    for n in full:
        assert np.array_equal(full[n][17].view(np.uint32), row[n][0].view(np.uint32)), n


def test_offsets_past_32_bits():
    """The last slots of a box whose logits exceed 4 GiB, tokens taken from a wider box."""
    from confidence_block_unmasking_amd import api
    rows, L, V, W = 230, 64, 152064, 90
    lg = torch.zeros(rows * L * V, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(8)
    box = torch.from_numpy(rng.integers(0, V, (rows, W)).astype(np.int32)).cuda()
    mask = torch.zeros((rows, L), dtype=torch.uint8, device="cuda")
    x = {}
    for r, j in ((0, 1), (rows - 1, 0), (rows - 1, L - 1)):
        h = torch.from_numpy((rng.normal(size=V) * 2).astype(np.float32)).to(torch.bfloat16)
        lg.view(rows, L, V)[r, j] = h.cuda()
        x[r, j] = h.double().numpy()
        mask[r, j] = 1
    f = dict(dtype=torch.float32, device="cuda")
    lp, ent, sta = torch.zeros((rows, L), **f), torch.zeros((rows, L), **f), torch.zeros((rows, L, 2), **f)
    ti, tl = torch.zeros((rows, L, 4), dtype=torch.int32, device="cuda"), torch.zeros((rows, L, 4), **f)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dllm_logprobs(lg.view(rows, L, V), mask, box[:, W - L:], lp, api.new_logprobs_workspace(rows, L, V, 4), st,
                      entropy=ent, stats=sta, top_ids=ti, top_logprobs=tl)
    gl = torch.ones((rows, L), **f)
    api.dllm_logprobs_grad(lg.view(rows, L, V), mask, box[:, W - L:], sta, gl, lg.view(rows, L, V), st)
    assert int(st.item()) == 0
    tok = box[:, W - L:].cpu().numpy()
    for (r, j), h in x.items():
        o = olp.slot(h, token=tok[r, j], k=4)
        assert abs(lp[r, j].item() - o["logprob"]) <= tol_logprob(o, V, o["logprob"])
        assert np.array_equal(ti[r, j].cpu().numpy(), o["top_ids"])
        check_grad(lg.view(rows, L, V)[r, j].double().cpu().numpy(), h, tok[r, j], 1.0, 0.0, "bf16")
    assert not lg.view(rows, L, V)[1].any()


# ---- gradient -------------------------------------------------------------------------------------

def check_grad(g, x, token, gl, gh, dtype, where=""):
    o = olp.slot(x)
    ref = olp.grad(x, token, gl, gh)
    p, lp = o["p"], np.where(o["p"] > 0, o["logp"], 0.0)
    coef = abs(gl) + abs(gh) * (np.abs(lp) + o["entropy"])
    tol = U * p * coef * (3 * np.abs(lp) + 2 * o["logS"] + 12) + U * abs(gl) * (np.arange(x.size) == token) + 1e-37
    tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(ref)
    err = np.abs(g - ref)
    assert (err <= tol).all(), (where, int((err - tol).argmax()), float((err - tol).max()))


def run_grad(buf, rows, L, V, ps, offset, mask, tokens, x, gl, gh, gextra=0, exclude=None, in_place=False):
    """Statistics from the oracle, rounded once."""
    from confidence_block_unmasking_amd import api
    sta, ent = np.full((rows, L, 2), np.nan, np.float32), np.full((rows, L), np.nan, np.float32)
    for r in range(rows):
        for j in range(L):
            if mask[r, j]:
                o = olp.slot(x[r, j])
                sta[r, j] = o["m"], o["logS"]
                ent[r, j] = o["entropy"]
    gs = V + gextra
    out = buf[offset:] if in_place else torch.full((rows * L * gs + 1,), 776.0, dtype=buf.dtype, device="cuda")[1:]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
           for a in (mask.astype(np.uint8), None if tokens is None else tokens.astype(np.int32), sta,
                     None if gl is None else gl.astype(np.float32), ent, None if gh is None else gh.astype(np.float32),
                     None if exclude is None else exclude.astype(np.uint8))]
    api.dllm_logprobs_grad(buf[offset:], dev[0], dev[1], dev[2], dev[3], out, st, entropy=dev[4], grad_entropy=dev[5],
                           exclude=dev[6], rows=rows, L=L, V=V, pos_stride=ps, row_stride=L * ps,
                           grad_pos_stride=ps if in_place else gs, grad_row_stride=L * (ps if in_place else gs))
    torch.cuda.synchronize()
    step = ps if in_place else gs
    return out[:rows * L * step].double().cpu().numpy().reshape(rows, L, step), int(st.item())


@pytest.mark.parametrize("rows,L,V,dtype,extra,offset,gextra,ent,in_place", [
    (1, 1, 1, "fp32", 0, 0, 0, True, False), (2, 3, 2, "bf16", 0, 0, 1, True, False), (2, 2, 7, "bf16", 1, 1, 0, False, False),
    (3, 4, 33, "fp32", 0, 3, 2, True, False), (4, 8, 1024, "fp32", 0, 0, 0, True, True),
    (2, 3, 4096, "fp32", 0, 0, 0, True, False), (2, 3, 8192, "bf16", 0, 0, 0, False, False),
    (2, 3, 8193, "bf16", 0, 0, 0, True, True), (2, 2, 20011, "bf16", 3, 1, 5, True, False),
    (1, 3, 20011, "fp32", 1, 1, 0, True, True), (1, 8, 152064, "bf16", 0, 0, 0, True, False),
    (1, 3, 126464, "fp32", 0, 0, 0, True, False)])
def test_gradient_against_the_oracle(rows, L, V, dtype, extra, offset, gextra, ent, in_place):
    rng = np.random.default_rng(V + rows)
    print(f"logprobs_grad rows={rows} L={L} V={V} {dtype}", flush=True)
    buf, x, ps = make_logits(rng, rows, L, V, dtype, V + extra, offset)
    mask = rng.random((rows, L)) < 0.7
    mask[0, 0] = True
    exclude = rng.random((rows, L)) < 0.2
    exclude[0, 0] = False
    tokens = rng.integers(0, V, (rows, L))
    gl, gh = rng.normal(size=(rows, L)), rng.normal(size=(rows, L)) if ent else None
    g, st = run_grad(buf, rows, L, V, ps, offset, mask, tokens, x, gl, gh, gextra, exclude, in_place)
    assert st == 0
    for r in range(rows):
        for j in range(L):
            assert (g[r, j, V:] == 776.0).all()
            if mask[r, j] and not exclude[r, j]:
                check_grad(g[r, j, :V], x[r, j], tokens[r, j], float(np.float32(gl[r, j])),
                           float(np.float32(gh[r, j])) if ent else 0.0, dtype, f"{r},{j}")
            else:
                assert not g[r, j, :V].any()


def test_gradient_of_one_output_alone_and_bad_tokens():
    rng = np.random.default_rng(4)
    rows, L, V = 2, 3, 700
    buf, x, ps = make_logits(rng, rows, L, V, "fp32")
    mask = np.ones((rows, L), bool)
    gh = rng.normal(size=(rows, L)).astype(np.float32)
    g, st = run_grad(buf, rows, L, V, ps, 0, mask, None, x, None, gh)
    assert st == 0
    for r in range(rows):
        for j in range(L):
            check_grad(g[r, j], x[r, j], None, 0.0, float(gh[r, j]), "fp32")
    tokens = np.full((rows, L), V)
    g, st = run_grad(buf, rows, L, V, ps, 0, mask, tokens, x, np.ones((rows, L)), gh)
    assert st == 1
    for r in range(rows):
        for j in range(L):
            check_grad(g[r, j], x[r, j], None, 0.0, float(gh[r, j]), "fp32")


def test_gradient_of_special_rows():
    V = 6001
    rng = np.random.default_rng(V)
    n = len(SPECIALS)
    x = np.stack([_special(s, V, rng) for s in SPECIALS])[None].astype(np.float32)
    buf, xr, ps = make_logits(rng, 1, n, V, "fp32", x=x)
    tokens = rng.integers(0, V, (1, n))
    gl, gh = rng.normal(size=(1, n)).astype(np.float32), rng.normal(size=(1, n)).astype(np.float32)
    g, st = run_grad(buf, 1, n, V, ps, 0, np.ones((1, n), bool), tokens, xr, gl, gh)
    assert st == 0
    for i, s in enumerate(SPECIALS):
        check_grad(g[0, i], xr[0, i], tokens[0, i], float(gl[0, i]), float(gh[0, i]), "fp32", s)
        assert not g[0, i][np.isneginf(xr[0, i]) & (np.arange(V) != tokens[0, i])].any()


def test_gradient_against_differences_of_the_forward():
    """The gradient from the library's own statistics against central differences of the oracle's
    forward (h^2 f'''/6 with h = 1e-4 and |f'''| < 10, plus the float32 bound above)."""
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(12)
    V = 40
    buf, x, ps = make_logits(rng, 1, 2, V, "fp32")
    tokens = np.array([[3, 17]])
    g, _ = run(buf, 1, 2, V, ps, 0, np.ones((1, 2), bool), tokens, 0)
    f32 = dict(dtype=torch.float32, device="cuda")
    gl, gh = torch.tensor([[1.0, -0.5]], **f32), torch.tensor([[0.25, 2.0]], **f32)
    grad = torch.empty((1, 2, V), **f32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dllm_logprobs_grad(buf.view(1, 2, V), torch.ones((1, 2), dtype=torch.uint8, device="cuda"),
                           torch.from_numpy(tokens.astype(np.int32)).cuda(), torch.from_numpy(g["stats"]).cuda(), gl, grad,
                           st, entropy=torch.from_numpy(g["entropy"]).cuda(), grad_entropy=gh)
    got = grad.cpu().numpy()
    h = 1e-4
    for j in range(2):
        def f(y):
            o = olp.slot(y, token=tokens[0, j])
            return gl[0, j].item() * o["logprob"] + gh[0, j].item() * o["entropy"]
        num = np.array([(f(x[0, j] + h * np.eye(V)[i]) - f(x[0, j] - h * np.eye(V)[i])) / (2 * h) for i in range(V)])
        assert np.abs(got[0, j] - num).max() <= 10 * h * h / 6 + 200 * U


def test_replays_of_a_captured_graph_and_another_stream():
    """Forward and gradient captured together; every replay on new inputs equals the eager result."""
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(6)
    rows, L, V, k = 3, 16, 20011, 5
    f = dict(dtype=torch.float32, device="cuda")
    lg = torch.empty((rows, L, V), dtype=torch.bfloat16, device="cuda")
    mask = torch.zeros((rows, L), dtype=torch.uint8, device="cuda")
    tok = torch.zeros((rows, L), dtype=torch.int32, device="cuda")
    gl = torch.ones((rows, L), **f)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def outputs():
        return dict(lp=torch.zeros((rows, L), **f), ent=torch.zeros((rows, L), **f), sta=torch.zeros((rows, L, 2), **f),
                    ti=torch.zeros((rows, L, k), dtype=torch.int32, device="cuda"), tl=torch.zeros((rows, L, k), **f),
                    grad=torch.empty((rows, L, V), dtype=torch.bfloat16, device="cuda"),
                    ws=api.new_logprobs_workspace(rows, L, V, k))

    def both(o, stream=None):
        api.dllm_logprobs(lg, mask, tok, o["lp"], o["ws"], st, entropy=o["ent"], stats=o["sta"], top_ids=o["ti"],
                          top_logprobs=o["tl"], stream=stream)
        api.dllm_logprobs_grad(lg, mask, tok, o["sta"], gl, o["grad"], st, stream=stream)

    def fill(seed):
        r = np.random.default_rng(seed)
        lg.copy_(torch.from_numpy((r.normal(size=(rows, L, V)) * 2).astype(np.float32)))
        mask.copy_(torch.from_numpy((r.random((rows, L)) < 0.6).astype(np.uint8)))
        tok.copy_(torch.from_numpy(r.integers(0, V, (rows, L)).astype(np.int32)))

    a, b, s = outputs(), outputs(), torch.cuda.Stream()
    fill(0)
    both(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(a)
    for seed in (1, 2, 3):
        fill(seed)
        for o in (a, b):
            for n in ("lp", "ent", "sta", "ti", "tl"):
                o[n].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        both(b, stream=s)
        torch.cuda.synchronize()
        for n in ("lp", "ent", "sta", "ti", "tl", "grad"):
            assert torch.equal(a[n], b[n]), (seed, n)
    assert int(st.item()) == 0


def test_binding_refuses_what_the_kernels_cannot_read():
    from confidence_block_unmasking_amd import api
    f = dict(dtype=torch.float32, device="cuda")
    lg, mask = torch.zeros((2, 4, 50), **f), torch.ones((2, 4), dtype=torch.uint8, device="cuda")
    tok, out = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros((2, 4), **f)
    ws, st = api.new_logprobs_workspace(2, 4, 50, 3, torch.float32), torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, tl = torch.zeros((2, 4, 3), dtype=torch.int32, device="cuda"), torch.zeros((2, 4, 3), **f)
    sta, grad = torch.zeros((2, 4, 2), **f), torch.zeros((2, 4, 50), **f)
    bad = [dict(tokens=tok.long()), dict(tokens=tok.t()), dict(tokens=tok[:, :3]), dict(tokens=tok.cpu()),
           dict(logprob=out[:1]), dict(logprob=out.double()), dict(mask=mask.bool()), dict(mask=mask[:1]),
           dict(logits=lg.half()), dict(logits=lg.transpose(1, 2)), dict(entropy=out.t()), dict(stats=out),
           dict(top_ids=ids.long()), dict(top_ids=ids, top_logprobs=tl[:1]), dict(exclude=mask[:1]), dict(status=st.long()),
           dict(logits=lg.cpu()), dict(V=60), dict(k=4, top_ids=ids, top_logprobs=tl)]
    for kw in bad:
        a = dict(logits=lg, mask=mask, tokens=tok, logprob=out, workspace=ws, status=st)
        if "V" in kw:
            a.update(rows=2, L=4, V=60, pos_stride=60, row_stride=240)
            kw = {}
        with pytest.raises(ValueError):
            api.dllm_logprobs(**{**a, **kw})
    for kw in (dict(top_ids=ids), dict(workspace=ws[:16]), dict(logprob=None)):
        with pytest.raises(api.DllmError):
            api.dllm_logprobs(**{**dict(logits=lg, mask=mask, tokens=tok, logprob=out, workspace=ws, status=st), **kw})
    good = dict(logits=lg, mask=mask, tokens=tok, stats=sta, grad_logprob=out, grad_logits=grad, status=st)
    for kw in (dict(grad_logits=grad.bfloat16()), dict(grad_logits=grad[:, :, :40]), dict(stats=out), dict(grad_logprob=out[:1]),
               dict(grad_entropy=out.double()), dict(grad_logits=grad.transpose(0, 1))):
        with pytest.raises(ValueError):
            api.dllm_logprobs_grad(**{**good, **kw})
    for kw in (dict(grad_entropy=out), dict(grad_logprob=None), dict(grad_logits=lg.view(-1)[1:], rows=1, L=4, V=49,
                                                                       pos_stride=49, row_stride=196)):
        with pytest.raises(api.DllmError):
            api.dllm_logprobs_grad(**{**good, **kw})
    torch.cuda.synchronize()


def test_calls_on_two_streams_at_once():
    """Two boxes scored at the same time on two streams, each with its own workspace."""
    rng = np.random.default_rng(21)
    V, k = 20011, 7
    from confidence_block_unmasking_amd import api
    boxes = []
    for rows, L in ((40, 32), (3, 16)):
        buf, x, ps = make_logits(rng, rows, L, V, "bf16")
        f = dict(dtype=torch.float32, device="cuda")
        boxes.append(dict(buf=buf, x=x, rows=rows, L=L, s=torch.cuda.Stream(),
                          tok=torch.from_numpy(rng.integers(0, V, (rows, L)).astype(np.int32)).cuda(),
                          mask=torch.ones((rows, L), dtype=torch.uint8, device="cuda"), lp=torch.zeros((rows, L), **f),
                          ti=torch.zeros((rows, L, k), dtype=torch.int32, device="cuda"), tl=torch.zeros((rows, L, k), **f),
                          ws=api.new_logprobs_workspace(rows, L, V, k), st=torch.zeros(1, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for b in boxes:
            api.dllm_logprobs(b["buf"], b["mask"], b["tok"], b["lp"], b["ws"], b["st"], top_ids=b["ti"], top_logprobs=b["tl"],
                              rows=b["rows"], L=b["L"], V=V, pos_stride=V, row_stride=b["L"] * V, stream=b["s"])
    torch.cuda.synchronize()
    for b in boxes:
        for r, j in ((0, 0), (b["rows"] - 1, b["L"] - 1)):
            o = olp.slot(b["x"][r, j], token=int(b["tok"][r, j].item()), k=k)
            assert np.array_equal(b["ti"][r, j].cpu().numpy(), o["top_ids"])
            assert abs(b["lp"][r, j].item() - o["logprob"]) <= tol_logprob(o, V, o["logprob"])
