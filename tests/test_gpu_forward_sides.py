"""The calls around the forward used together on the GPU: a session that records the log probabilities
of the tokens it generates, and one training step from a packed box's ids to its table's gradient."""
import numpy as np
import pytest

from oracle import logprobs as olp
from tests.test_gpu_logprobs import tol_entropy, tol_logprob
from workload import configs, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _forward(w):
    def forward(s):
        synth.logits_gpu(s.logits, w.dtype, s.rows, w.L, w.V, s.row_req, s.b_rows, s.masks[s.cur], w.logit_seed, w.sigma,
                         w.umax)
    return forward


@pytest.mark.parametrize("mode,dtype,k", [("fdfo", "bf16", 5), ("sync", "fp32", 0), ("handback", "bf16", 1)])
def test_session_records_every_generated_token(mode, dtype, k):
    """Every unmasked token's entry against the oracle on the logits of the step that unmasked it; blocks
    that wait, move rows or span rounds included."""
    from confidence_block_unmasking_amd.driver import Session
    w = configs.small(L=8, V=700, n_act=5, n_q=9, K=3, seed=11, dtype=dtype, rows_cap=5, mode=mode)
    sess = Session.from_workload(w)
    sess.record_logprobs(k)
    seen = {}
    prev = {}

    def on_step(s, info):
        rr, bb = s.row_req[:s.rows].cpu().numpy(), s.b_rows[:s.rows].cpu().numpy()
        lg = s.logits[:s.rows].double().cpu().numpy()
        tok = s.box().cpu().numpy()[:, s.W - s.L:]
        old = s.masks[1 - s.cur][:s.rows * s.L].view(s.rows, s.L).cpu().numpy()
        for r in range(s.rows):
            for j in np.flatnonzero((old[r] != 0) & (info["mask"][r] == 0)):
                at = (int(rr[r]), int(bb[r]) * s.L + int(j))
                assert at not in seen
                seen[at] = olp.slot(lg[r, j], token=int(tok[r, j]), k=k)
                prev[at] = int(tok[r, j])

    sess.run(mode, _forward(w), on_step=on_step)
    got = {n: t.cpu().numpy() for n, t in sess.logprobs().items()}
    assert len(seen) == int((w.K * w.L).sum())
    arena = sess.reqs.arena.cpu().numpy()
    for (q, i), o in seen.items():
        assert arena[w.arena_off[q] + w.p[q] + i] == prev[q, i]
        assert abs(got["logprob"][q, i] - o["logprob"]) <= tol_logprob(o, w.V, o["logprob"])
        assert abs(got["entropy"][q, i] - o["entropy"]) <= tol_entropy(o, w.V)
        if k:
            assert np.array_equal(got["top_ids"][q, i], o["top_ids"])
            assert np.abs(got["top_logprobs"][q, i] - o["top_logprobs"]).max() <= tol_logprob(o, w.V, o["top_logprobs"][-1])
    missing = np.ones(got["logprob"].shape, bool)
    for q, i in seen:
        missing[q, i] = False
    assert np.isnan(got["logprob"][missing]).all() and np.isnan(got["entropy"][missing]).all()
    if k:
        assert (got["top_ids"][missing] == -1).all()


def test_record_survives_a_snapshot():
    from confidence_block_unmasking_amd.driver import Session
    w = configs.small(L=8, V=700, n_act=4, n_q=8, K=3, seed=12, dtype="bf16", rows_cap=4)
    whole = Session.from_workload(w)
    whole.record_logprobs(3)
    whole.run("fdfo", _forward(w))
    first = Session.from_workload(w)
    first.record_logprobs(3)
    first.run("fdfo", _forward(w), max_rounds=3)
    second = Session.from_snapshot(first.snapshot())
    second.run("fdfo", _forward(w))
    a, b = whole.logprobs(), second.logprobs()
    for n in a:
        assert torch.equal(a[n].view(torch.int32), b[n].view(torch.int32)), n
    with pytest.raises(ValueError):
        Session.from_workload(w).logprobs()


def test_session_embeds_its_box():
    from confidence_block_unmasking_amd.driver import Session
    w = configs.small(L=8, V=50, n_act=6, n_q=0, K=2, seed=3, dtype="fp32")
    sess = Session.from_workload(w)
    sess.compact(with_box=False)
    sess.pack()
    table = torch.randn((w.V + 1, 24), device="cuda")      # the mask token's row; padding (id V + 1) has none
    x = sess.embed(table, scale=0.5)
    sess.check_status("dllm_embed")
    n = sess.rows * sess.W
    ids, valid = sess.box_ids[:n].long(), sess.box_valid[:n].bool()
    ref = torch.where(valid[:, None], table[torch.where(valid, ids, 0)] * 0.5, 0.0)
    assert x.shape == (sess.rows, sess.W, 24) and torch.equal(x.view(n, 24), ref)
    buf = torch.empty((n, 24), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(sess.embed(table, scale=0.5, out=buf), ref.to(torch.bfloat16))


@pytest.mark.parametrize("replays", [0, 3])
def test_training_step_from_ids_to_table_gradient(replays):
    """Embedding, a linear layer tied to the table, the masked tokens' log probabilities with an entropy
    bonus, and back to the table's gradient (from the head and from the lookup), against float64
    autograd; also captured into a graph and replayed.  Tolerance: two passes of fp32 products over D
    and V terms, each element off by at most (D + V) u of the sum of its absolute terms, bounded here by
    the same computation on absolute values."""
    from confidence_block_unmasking_amd import api
    rng = np.random.default_rng(0)
    rows, W, L, V, D = 6, 30, 8, 90, 32
    f = dict(device="cuda")
    ids = torch.from_numpy(rng.integers(0, V, (rows, W)).astype(np.int32)).cuda()
    target = torch.from_numpy(rng.integers(0, V, (rows, L)).astype(np.int32)).cuda()
    valid = torch.ones((rows, W), dtype=torch.uint8, **f)
    valid[:, :5] = 0
    mask = torch.from_numpy((rng.random((rows, L)) < 0.6).astype(np.uint8)).cuda()
    ids[:, W - L:] = torch.where(mask != 0, torch.full_like(target, V), target)      # the mask token is row V
    table = torch.from_numpy(rng.normal(size=(V + 1, D)).astype(np.float32)).cuda()
    mix = torch.from_numpy((rng.normal(size=(D, D)) / np.sqrt(D)).astype(np.float32)).cuda()
    gl = torch.from_numpy(rng.normal(size=(rows, L)).astype(np.float32)).cuda()
    gh = torch.from_numpy(rng.normal(size=(rows, L)).astype(np.float32)).cuda()
    st = torch.zeros(1, dtype=torch.int32, **f)
    x, gx = torch.empty((rows, W, D), **f), torch.zeros((rows, W, D), **f)
    logprob, ent, sta = torch.zeros((rows, L), **f), torch.zeros((rows, L), **f), torch.zeros((rows, L, 2), **f)
    lw, ew = api.new_logprobs_workspace(rows, L, V, 0, torch.float32), api.new_embed_grad_workspace(rows * W, V + 1, D)
    grad = torch.empty((V + 1, D), **f)

    def step():
        api.dllm_embed(table, ids, x, st, valid=valid, scale=1.5)
        h = x[:, W - L:].reshape(-1, D) @ mix
        logits = (h @ table[:V].t().contiguous()).view(rows, L, V)
        api.dllm_logprobs(logits, mask, target, logprob, lw, st, entropy=ent, stats=sta)
        api.dllm_logprobs_grad(logits, mask, target, sta, gl, logits, st, entropy=ent, grad_entropy=gh)
        g = logits.view(-1, V)
        gx[:, W - L:] = ((g @ table[:V]) @ mix.t().contiguous()).view(rows, L, D)
        grad.zero_()
        grad[:V] = g.t().contiguous() @ h
        api.dllm_embed_grad(gx, ids, grad, ew, st, valid=valid, scale=1.5, accumulate=True)

    step()
    torch.cuda.synchronize()

    def reference(absolute):
        def v(t):
            return t.double().cpu().abs() if absolute else t.double().cpu()
        T = v(table).requires_grad_(True)
        e = (T[ids.cpu().long()] * 1.5) * valid.cpu().double()[:, :, None]
        lg = (e[:, W - L:] @ v(mix)) @ T[:V].t()
        lp = torch.log_softmax((table.double().cpu()[ids.cpu().long()] * 1.5 * valid.cpu().double()[:, :, None])[:, W - L:]
                               @ mix.double().cpu() @ table.double().cpu()[:V].t(), 2) if absolute else torch.log_softmax(lg, 2)
        p = lp.exp()
        H = -(p * lp).sum(2)
        on = mask.cpu().double()
        if not absolute:
            got = lp.gather(2, target.cpu().long()[:, :, None])[:, :, 0]
            ((got * gl.double().cpu() + H * gh.double().cpu()) * on).sum().backward()
            return T.grad, got.detach(), H.detach()
        one = torch.zeros_like(lp).scatter_(2, target.cpu().long()[:, :, None], 1.0)
        dl = (v(gl)[:, :, None] * (one + p) + v(gh)[:, :, None] * p * (lp.abs() + H[:, :, None])) * on[:, :, None]
        (lg * dl).sum().backward()
        return T.grad

    ref, lp_ref, H_ref = reference(False)
    size = reference(True)
    u = 2.0 ** -24

    def check():
        # logits are off by D u of their absolute terms (at most ~60 here), the probabilities by as much again
        assert ((grad.double().cpu() - ref).abs() <= (4 * D + V) * 64 * u * size).all()
        on = mask.cpu() != 0
        assert (logprob.double().cpu() - lp_ref)[on].abs().max() <= 4 * D * 64 * u
        assert (ent.double().cpu() - H_ref)[on].abs().max() <= 4 * D * 64 * u * 8
        assert int(st.item()) == 0

    check()
    if not replays:
        return
    eager = grad.clone()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()                                 # the library products' own first-use work stays out of the graph
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(replays):
        grad.fill_(9.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(grad, eager)
        grad.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, eager)
        check()
