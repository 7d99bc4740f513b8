"""dllm_embed and dllm_embed_grad on the GPU against the float64 oracle.

Tolerances: the lookup is one float32 product rounded once more to the output's type, u |ref| + half a
step.  The gradient sums c terms in float32 in chains: at most min(c, 64 + c/192 + 17) additions deep
(up to 64 tokens of a piece, a sixteenth of the pieces of at least 12 tokens, 16 slices), each off by u of the sum of absolute terms, then
one FMA with the scale (and the row it adds to) and half a step of the type.
"""
import numpy as np
import pytest

from oracle import embed as oembed

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import confidence_block_unmasking_amd  # noqa: F401  (fails loudly if the library is missing)


def _matrix(rng, n, D, dtype, extra=0, offset=0, sd=1.0):
    """A device matrix of n rows D + extra apart that starts `offset` elements into its storage, and
    its values."""
    t = torch.from_numpy((rng.normal(size=(n, D)) * sd).astype(np.float32)).to(DT[dtype])
    buf = torch.full((offset + n * (D + extra),), 776.0, dtype=DT[dtype], device="cuda")
    m = buf[offset:].view(n, D + extra)[:, :D]
    m.copy_(t)
    return m, t.double().numpy()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n,V,D,table,out,extra,offset", [
    (1, 1, 1, "fp32", "fp32", 0, 0), (1, 5, 4096, "bf16", "bf16", 0, 0), (3, 5, 7, "bf16", "fp32", 1, 1),
    (17, 40, 8, "fp32", "bf16", 0, 0), (33, 40, 9, "bf16", "bf16", 2, 3), (5, 300, 1000, "fp32", "fp32", 1, 2),
    (257, 1000, 129, "bf16", "bf16", 0, 1), (1023, 77, 2048, "bf16", "bf16", 0, 0), (70, 90, 2049, "fp32", "bf16", 3, 0),
    (4097, 20, 16, "bf16", "fp32", 0, 0), (64, 50, 5001, "bf16", "bf16", 0, 0)])
@pytest.mark.parametrize("masked", [False, True])
def test_lookup(n, V, D, table, out, extra, offset, masked):
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(n * 31 + D)
    print(f"embed n={n} V={V} D={D} {table}->{out}", flush=True)
    t, th = _matrix(rng, V, D, table, extra, offset)
    o, _ = _matrix(rng, n + 2, D, out, extra, offset)
    o.fill_(55.0)
    ids = rng.integers(0, V, n).astype(np.int32)
    valid = (rng.random(n) < 0.6).astype(np.uint8) if masked else None
    if masked:
        ids[valid == 0] = 1 << 30              # not looked at
    st = _status()
    api.dllm_embed(t, torch.from_numpy(ids).cuda(), o, st, valid=None if valid is None else torch.from_numpy(valid).cuda(),
                   scale=1.7)
    got = o.double().cpu().numpy()
    ref = oembed.lookup(th, ids, valid, 1.7)
    assert int(st.item()) == 0
    assert (np.abs(got[:n] - ref) <= (U + HALF[out] * (1 + U)) * np.abs(ref)).all()
    assert (got[n:] == 55.0).all()
    if extra:
        assert (o.as_strided((n, extra), (D + extra, 1), o.storage_offset() + D) == 776.0).all()


def test_lookup_of_bad_ids_reports_and_writes_zeros():
    from confidence_block_unmasking_amd import api
    t = torch.ones((10, 24), device="cuda")
    o = torch.full((4, 24), 5.0, device="cuda")
    st = _status()
    api.dllm_embed(t, torch.tensor([-1, 3, 10, 1 << 30], dtype=torch.int32, device="cuda"), o, st)
    assert int(st.item()) == 1
    assert o[:, 0].tolist() == [0.0, 1.0, 0.0, 0.0] and o.sum().item() == 24


def test_lookup_of_unscaled_special_values_is_exact():
    from confidence_block_unmasking_amd import api
    t = torch.tensor([[0.0, -0.0, float("inf"), float("-inf"), 1e-40, 3.0e38, 1.0, -2.5]], device="cuda")
    o = torch.empty((1, 8), device="cuda")
    api.dllm_embed(t, torch.zeros(1, dtype=torch.int32, device="cuda"), o, _status())
    assert torch.equal(o, t)


def test_lookup_past_32_bit_offsets():
    from confidence_block_unmasking_amd import api
    V, D = 300000, 8192                        # 4.6 GiB of bf16
    t = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    t[V - 1] = 3.0
    ids = torch.tensor([0, V - 1, 5], dtype=torch.int32, device="cuda")
    o = torch.empty((3, D), dtype=torch.bfloat16, device="cuda")
    st = _status()
    api.dllm_embed(t, ids, o, st)
    assert (o[1] == 3.0).all() and not o[0].any() and not o[2].any()
    g = torch.ones((3, D), dtype=torch.bfloat16, device="cuda")
    api.dllm_embed_grad(g, ids, t, api.new_embed_grad_workspace(3, V, D), st, scale=2.0, accumulate=True)
    assert (t[V - 1] == 5.0).all() and (t[0] == 2.0).all() and (t[5] == 2.0).all() and not t[V - 2].any()
    api.dllm_embed_grad(g, ids, t, api.new_embed_grad_workspace(3, V, D), st, scale=2.0)
    assert (t[V - 1] == 2.0).all() and int((t != 0).sum().item()) == 3 * D and int(st.item()) == 0


def _ids(kind, n, V, rng):
    if kind == "spread":
        return rng.integers(0, V, n)
    if kind == "one":
        return np.full(n, V - 1)
    if kind == "half-mask":
        a = rng.integers(0, V, n)
        a[rng.random(n) < 0.5] = V // 2
        return a
    if kind.startswith("runs-of-"):            # every id as long as a piece, or one token longer
        m = int(kind.split("-")[-1])
        return rng.permutation(np.repeat(np.arange((n + m - 1) // m) % V, m)[:n])
    if kind == "ascending":
        return np.arange(n) % V
    if kind == "descending":
        return (n - np.arange(n)) % V
    raise AssertionError(kind)


def check_grad(got, ref, size, count, dtype, base=None):
    depth = np.minimum(count, 64 + count // 192 + 17)[:, None]
    tol = U * (depth + 2) * size
    total = ref if base is None else ref + base
    tol = tol + HALF[dtype] * (np.abs(total) + tol) + 2 * U * np.abs(total)
    err = np.abs(got - total)
    assert (err <= tol).all(), (np.unravel_index((err - tol).argmax(), err.shape), float((err - tol).max()))


@pytest.mark.parametrize("n,V,D,kind,go,table,extra,offset", [
    (1, 1, 1, "spread", "fp32", "fp32", 0, 0), (1, 600, 8, "spread", "bf16", "bf16", 0, 0),
    (63, 10, 7, "spread", "bf16", "fp32", 1, 1), (64, 3, 33, "one", "fp32", "bf16", 0, 0),
    (65, 3, 33, "one", "fp32", "fp32", 2, 3), (200, 511, 64, "spread", "bf16", "bf16", 0, 0),
    (200, 512, 64, "spread", "bf16", "bf16", 0, 1), (1000, 20013, 1000, "half-mask", "bf16", "fp32", 0, 0),
    (640, 40, 130, "runs-of-64", "fp32", "fp32", 0, 0), (650, 40, 130, "runs-of-65", "fp32", "fp32", 0, 0),
    (4096, 700, 24, "ascending", "bf16", "bf16", 0, 0), (4097, 5000, 24, "descending", "bf16", "bf16", 1, 0),
    (9000, 3, 40, "spread", "bf16", "fp32", 0, 0), (20000, 152066, 72, "half-mask", "bf16", "bf16", 0, 0),
    (70001, 9, 16, "half-mask", "fp32", "fp32", 0, 0), (5000, 300000, 16, "half-mask", "bf16", "fp32", 0, 0),
    (33, 70, 2056, "spread", "bf16", "bf16", 0, 0), (300, 7, 4100, "half-mask", "bf16", "bf16", 0, 0),
    (150000, 50000, 8, "spread", "bf16", "fp32", 0, 0), (150000, 70, 8, "half-mask", "fp32", "fp32", 0, 0),
    (131200, 2100, 8, "runs-of-64", "bf16", "bf16", 0, 0), (133250, 2100, 8, "runs-of-65", "fp32", "bf16", 0, 1),
    (132000, 1, 8, "one", "fp32", "fp32", 0, 0), (600, 60, 24, "runs-of-12", "fp32", "fp32", 0, 0),
    (650, 60, 24, "runs-of-13", "bf16", "fp32", 0, 0)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(n, V, D, kind, go, table, extra, offset, accumulate):
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(n + V + D)
    print(f"embed_grad n={n} V={V} D={D} {kind} {go}->{table} accumulate={accumulate}", flush=True)
    g, gh = _matrix(rng, n, D, go, extra, offset)
    t, base = _matrix(rng, V, D, table, extra, offset)
    ids = _ids(kind, n, V, rng).astype(np.int32)
    valid = (rng.random(n) < 0.8).astype(np.uint8)
    ws = api.new_embed_grad_workspace(n, V, D)
    ws.fill_(0xA5)
    st = _status()
    api.dllm_embed_grad(g, torch.from_numpy(ids).cuda(), t, ws, st, valid=torch.from_numpy(valid).cuda(), scale=0.75,
                        accumulate=accumulate)
    got = t.double().cpu().numpy()
    assert int(st.item()) == 0
    ref, size, count = oembed.gradient(gh, ids, V, valid, 0.75)
    check_grad(got, ref, size, count, table, base if accumulate else None)
    absent = count == 0
    assert np.array_equal(got[absent], base[absent]) if accumulate else not got[absent].any()
    if extra:
        assert (t.as_strided((V, extra), (D + extra, 1), t.storage_offset() + D) == 776.0).all()


@pytest.mark.parametrize("n", [3000, 9000])
def test_gradient_of_a_large_table(n):
    """A table whose zeros hide the sort: every row that occurs against float64 sums of its
    tokens, every other row zero, the columns past D untouched."""
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(n)
    V, D, pitch = 210000, 2001, 2004
    buf = torch.full((V, pitch), 776.0, dtype=torch.bfloat16, device="cuda")
    t = buf[:, :D]
    ids = torch.from_numpy(_ids("half-mask", n, V, rng).astype(np.int32)).cuda()
    g = torch.randn((n, D), device="cuda").to(torch.bfloat16)
    st = _status()
    api.dllm_embed_grad(g, ids, t, api.new_embed_grad_workspace(n, V, D), st, scale=0.5)
    names, back = ids.long().unique(return_inverse=True)
    ref = torch.zeros((names.numel(), D), dtype=torch.float64, device="cuda").index_add_(0, back, 0.5 * g.double())
    size = torch.zeros_like(ref).index_add_(0, back, 0.5 * g.double().abs())
    depth = torch.bincount(back).clamp(max=81 + n // 192)[:, None]
    tol = U * (depth + 2) * size
    assert ((t[names].double() - ref).abs() <= tol + HALF["bf16"] * (ref.abs() + tol)).all()
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[names] = False
    assert not t[absent].any() and (buf[:, D:] == 776.0).all() and int(st.item()) == 0


@pytest.mark.parametrize("n,V,D,pitch,table", [(1, 60000, 1000, 1000, "fp32"), (160, 1600000, 33, 33, "fp32"),
                                               (700, 110000, 257, 259, "fp32"), (3000, 100001, 513, 515, "fp32"),
                                               (4096, 90001, 2050, 2052, "bf16"), (4097, 120000, 1001, 1001, "fp32"),
                                               (9000, 1100000, 200, 203, "bf16")])
def test_gradient_whose_zeros_outlast_the_sort(n, V, D, pitch, table):
    """Tables that the launches of the sort clear only in part: every row that occurs against float64 sums,
    every other row zero, the columns past D untouched."""
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(n)
    buf = torch.full((V, pitch), 776.0, dtype=torch.bfloat16 if table == "bf16" else torch.float32, device="cuda")
    t = buf[:, :D]
    ids = torch.from_numpy(_ids("half-mask", n, V, rng).astype(np.int32)).cuda()
    ids[0] = V - 1
    g = torch.randn((n, D), device="cuda").to(torch.bfloat16)
    st = _status()
    api.dllm_embed_grad(g, ids, t, api.new_embed_grad_workspace(n, V, D), st, scale=0.5)
    names, back = ids.long().unique(return_inverse=True)
    ref = torch.zeros((names.numel(), D), dtype=torch.float64, device="cuda").index_add_(0, back, 0.5 * g.double())
    size = torch.zeros_like(ref).index_add_(0, back, 0.5 * g.double().abs())
    depth = torch.bincount(back).clamp(max=81 + n // 192)[:, None]
    tol = U * (depth + 2) * size
    assert ((t[names].double() - ref).abs() <= tol + HALF[table] * (ref.abs() + tol)).all()
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[names] = False
    assert not t[absent].any() and (buf[:, D:] == 776.0).all() and int(st.item()) == 0


def test_gradient_of_a_large_table_without_tokens():
    from confidence_block_unmasking_amd import api
    t = torch.full((70000, 1025), 9.0, device="cuda")
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    api.dllm_embed_grad(torch.ones((1, 1025), device="cuda"), ids, t, api.new_embed_grad_workspace(0, 70000, 1025), _status())
    assert not t.any()


def test_gradient_without_tokens():
    from confidence_block_unmasking_amd import api
    for n, valid in ((0, None), (5, torch.zeros(5, dtype=torch.uint8, device="cuda"))):
        g = torch.ones((max(n, 1), 20), device="cuda")
        ids = torch.zeros(n, dtype=torch.int32, device="cuda")
        t = torch.full((70, 20), 9.0, device="cuda")
        ws = api.new_embed_grad_workspace(n, 70, 20)
        st = _status()
        api.dllm_embed_grad(g, ids, t, ws, st, valid=valid, accumulate=True)
        assert (t == 9.0).all()
        api.dllm_embed_grad(g, ids, t, ws, st, valid=valid)
        assert not t.any() and int(st.item()) == 0
    o = torch.full((2, 20), 4.0, device="cuda")
    api.dllm_embed(t, torch.zeros(0, dtype=torch.int32, device="cuda"), o, st)
    assert (o == 4.0).all()


def test_gradient_of_bad_ids_reports_and_leaves_them_out():
    from confidence_block_unmasking_amd import api
    g = torch.ones((5, 12), device="cuda")
    ids = torch.tensor([2, -7, 4, 2, 5], dtype=torch.int32, device="cuda")
    t = torch.full((5, 12), 9.0, device="cuda")
    st = _status()
    api.dllm_embed_grad(g, ids, t, api.new_embed_grad_workspace(5, 5, 12), st)
    assert int(st.item()) == 1 and t[:, 0].tolist() == [0.0, 0.0, 2.0, 0.0, 1.0]


def test_gradient_bits_do_not_depend_on_timing_or_workspace():
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(3)
    n, V, D = 40000, 5000, 136
    g, _ = _matrix(rng, n, D, "bf16")
    ids = torch.from_numpy(_ids("half-mask", n, V, rng).astype(np.int32)).cuda()
    outs = []
    for fill in (0, 255, 77):
        ws = api.new_embed_grad_workspace(n, V, D)
        ws.fill_(fill)
        t = torch.full((V, D), 3.0, device="cuda")
        st = _status()
        api.dllm_embed_grad(g, ids, t, ws, st)
        outs.append(t)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_gradient_is_the_lookups_transpose():
    """<lookup(T), G> = <T, gradient(G)> for fp32 values on a grid coarse enough that both sides are
    exact: the gradient against the forward's own linear map."""
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(2)
    n, V, D = 300, 50, 21
    T = torch.from_numpy(rng.integers(-8, 9, (V, D)).astype(np.float32)).cuda()
    G = torch.from_numpy(rng.integers(-8, 9, (n, D)).astype(np.float32)).cuda()
    ids = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    out, grad, st = torch.empty((n, D), device="cuda"), torch.empty((V, D), device="cuda"), _status()
    api.dllm_embed(T, ids, out, st, scale=0.5)
    api.dllm_embed_grad(G, ids, grad, api.new_embed_grad_workspace(n, V, D), st, scale=0.5)
    assert (out.double() * G.double()).sum().item() == (T.double() * grad.double()).sum().item()


def test_replays_of_a_captured_graph_and_another_stream():
    from confidence_block_unmasking_amd import api
    n, V, D = 9000, 3000, 264
    f = dict(device="cuda")
    table = torch.randn((V, D), **f)
    ids = torch.zeros(n, dtype=torch.int32, **f)
    valid = torch.zeros(n, dtype=torch.uint8, **f)
    st = _status()

    def outputs():
        return dict(out=torch.empty((n, D), dtype=torch.bfloat16, **f), grad=torch.empty((V, D), **f),
                    ws=api.new_embed_grad_workspace(n, V, D))

    def both(o, stream=None):
        api.dllm_embed(table, ids, o["out"], st, valid=valid, scale=3.0, stream=stream)
        api.dllm_embed_grad(o["out"], ids, o["grad"], o["ws"], st, valid=valid, scale=3.0, stream=stream)

    a, b, s = outputs(), outputs(), torch.cuda.Stream()
    both(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(a)
    for seed in (1, 2, 3):
        r = np.random.default_rng(seed)
        ids.copy_(torch.from_numpy(_ids("half-mask", n, V, r).astype(np.int32)))
        valid.copy_(torch.from_numpy((r.random(n) < 0.9).astype(np.uint8)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        both(b, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["grad"], b["grad"]), seed
    assert int(st.item()) == 0


def test_binding_refuses_what_the_kernels_cannot_read():
    from confidence_block_unmasking_amd import api
    t, ids, out, st = torch.zeros((9, 16), device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(
        (5, 16), device="cuda"), _status()
    ws = api.new_embed_grad_workspace(5, 9, 16)
    for kw in (dict(table=t.half()), dict(table=t.cpu()), dict(table=t.t()), dict(ids=ids.long()), dict(ids=ids[::2]),
               dict(out=out[:4]), dict(out=out[:, :8]), dict(out=out.t()), dict(valid=torch.ones(4, dtype=torch.uint8, device="cuda")),
               dict(valid=torch.ones(5, dtype=torch.bool, device="cuda")), dict(status=st.float())):
        with pytest.raises(ValueError):
            api.dllm_embed(**{**dict(table=t, ids=ids, out=out, status=st), **kw})
    with pytest.raises(api.DllmError):
        api.dllm_embed(t, ids, t[4:], st)          # out overlaps the table
    good = dict(grad_out=out, ids=ids, grad_table=t, workspace=ws, status=st)
    for kw in (dict(grad_out=out[:4]), dict(grad_out=out[:, :8]), dict(grad_table=t.double()), dict(ids=ids.float()),
               dict(workspace=ws.float())):
        with pytest.raises(ValueError):
            api.dllm_embed_grad(**{**good, **kw})
    for kw in (dict(workspace=ws[:64]), dict(workspace=ws[16:]), dict(grad_table=t[:1].expand(9, 16))):
        with pytest.raises(api.DllmError):
            api.dllm_embed_grad(**{**good, **kw})
    torch.cuda.synchronize()


def test_gradients_on_two_streams_at_once():
    """Two tables accumulated at the same time on two streams, each with its own workspace."""
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(17)
    jobs = []
    for n, V, D in ((20000, 3000, 264), (700, 90, 40)):
        g, gh = _matrix(rng, n, D, "bf16")
        ids = _ids("half-mask", n, V, rng).astype(np.int32)
        jobs.append(dict(g=g, gh=gh, ids=ids, d=torch.from_numpy(ids).cuda(), t=torch.empty((V, D), device="cuda"),
                         ws=api.new_embed_grad_workspace(n, V, D), st=_status(), s=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for j in jobs:
            api.dllm_embed_grad(j["g"], j["d"], j["t"], j["ws"], j["st"], stream=j["s"])
            api.dllm_embed_grad(j["g"], j["d"], j["t"], j["ws"], j["st"], accumulate=True, stream=j["s"])
    torch.cuda.synchronize()
    for j in jobs:
        V = j["t"].shape[0]
        ref, size, count = oembed.gradient(j["gh"], j["ids"], V)
        check_grad(j["t"].double().cpu().numpy(), ref, 2 * size, count, "fp32", ref)
