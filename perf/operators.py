"""Cases for measuring the operators on either side of a diffusion language model's forward.

Four paths, each in a plain form (elementary torch operations) and, with `own` true, as the calls a
user makes of this library:

  logprobs    log probabilities of given tokens at selected slots of a box's logits, with the
              distribution's entropy and its top alternatives (dllm_logprobs)
  lossgrad    the gradient of those log probabilities and entropies with respect to the logits
              (dllm_logprobs_grad)
  embed       embedding lookup of a packed box's token ids, scaled (dllm_embed)
  embedgrad   the lookup's gradient: a dense table gradient from the box's output gradients
              (dllm_embed_grad)

Vocabularies, block lengths and row counts are those of the package's workloads (LLaDA-shaped
V = 126464, Dream-shaped V = 152064, L = 32 and 64, boxes of 64 to 256 rows); embedding widths are
generic.
"""
import math

import torch

own = False

MASK_RUN = 256          # generated columns at the end of a training row


def _case(op, name=None, **kw):
    c = dict(op=op, **kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one freshly unmasked token of a single request: the latency of a streamed answer
        _case("logprobs", "logprobs-one-token", rows=1, L=32, V=126464, selected=1, k=5, entropy=True, stats=False,
              dtype="bf16", pad=0, banned=0),
        # the tokens one denoise step unmasked over a batch, three per row, with five alternatives
        _case("logprobs", "logprobs-step-record", rows=64, L=32, V=152064, selected=192, k=5, entropy=True, stats=False,
              dtype="bf16", pad=0, banned=2),
        # every masked slot of the Dream-shaped step with twenty alternatives
        _case("logprobs", "logprobs-box-top20", rows=64, L=32, V=152064, selected=1005, k=20, entropy=True, stats=False,
              dtype="bf16", pad=0, banned=2),
        # an odd vocabulary in fp32, rows padded to an odd stride, so no row is 16-byte aligned
        _case("logprobs", "logprobs-odd-fp32", rows=33, L=7, V=20011, selected=231, k=20, entropy=True, stats=True,
              dtype="fp32", pad=2, banned=11),
        # the largest box scored whole: the forward half of a masked-token loss
        _case("logprobs", "logprobs-large-score", rows=256, L=64, V=152064, selected=16384, k=0, entropy=True, stats=True,
              dtype="bf16", pad=0, banned=0),
        # the backward half of that loss on the Dream-shaped box
        _case("lossgrad", "lossgrad-box", rows=64, L=32, V=152064, selected=1005, entropy=False, dtype="bf16", pad=0,
              banned=0),
        # a policy loss with an entropy bonus, in fp32, every slot selected
        _case("lossgrad", "lossgrad-entropy-fp32", rows=16, L=32, V=126464, selected=512, entropy=True, dtype="fp32",
              pad=0, banned=2),
        # the tiny step's box
        _case("lossgrad", "lossgrad-small", rows=4, L=32, V=1024, selected=64, entropy=True, dtype="fp32", pad=0,
              banned=0),
        # one token
        _case("embed", "embed-one-token", rows=1, W=1, V=126466, D=4096, distinct=1, prompt=1, masked=0, table="bf16",
              act="bf16"),
        # the mixed-state box: 128 requests, prompts up to 1024, 256 generated columns
        _case("embed", "embed-box", rows=128, W=1280, V=126466, D=4096, distinct=40000, prompt=1024, masked=128,
              table="bf16", act="bf16"),
        # a small box in two micro-batches, the second added to the first; odd sizes, fp32 master gradients
        _case("embedgrad", "embedgrad-two-batches", rows=8, W=200, V=20013, D=1000, distinct=300, prompt=100, masked=50,
              table="fp32", act="bf16", batches=2),
        # a training box: half of the 256 generated columns of every row hold the mask token
        _case("embedgrad", "embedgrad-box", rows=64, W=544, V=152066, D=4096, distinct=12000, prompt=288, masked=128,
              table="bf16", act="bf16", batches=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "lossgrad", "embed", "embedgrad"])
    if op in ("logprobs", "lossgrad"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        es = 2 if dtype == "bf16" else 4
        V = rng.choice([126464, 152064, _log(rng, 300, 160000), _log(rng, 300, 160000) | 1])
        L = rng.choice([32, 64, rng.randint(1, 100)])
        rows = max(1, min(_log(rng, 1, 256), int(6e8 // (L * V * es))))
        selected = rng.choice([rows * L, max(1, _log(rng, 1, rows * L))])
        c = dict(rows=rows, L=L, V=V, selected=selected, entropy=rng.random() < 0.7, dtype=dtype,
                 pad=rng.choice([0, 0, 8, rng.randint(1, 9)]), banned=rng.choice([0, 2, rng.randint(0, 100)]))
        if op == "logprobs":
            c.update(k=rng.choice([0, 1, 5, 20, rng.randint(1, 32)]), stats=rng.random() < 0.5)
        return _case(op, **c)
    D = rng.choice([1024, 2048, 4096, _log(rng, 8, 5000)])
    prompt = _log(rng, 1, 1024)
    gen = rng.choice([0, 32, 64, MASK_RUN])
    W = prompt + gen
    rows = max(1, min(_log(rng, 1, 128), int(2.0e8 // (W * D))))
    V = rng.choice([126466, 152066, _log(rng, 300, 160000)])
    c = dict(rows=rows, W=W, V=V, D=D, prompt=prompt, masked=rng.randint(0, gen), table=rng.choice(["bf16", "fp32"]),
             act=rng.choice(["bf16", "bf16", "fp32"]))
    c["distinct"] = max(1, min(V - 2, _log(rng, 1, max(1, _valid(c) - rows * c["masked"]))))
    if op == "embedgrad":
        c["batches"] = rng.choice([1, 1, 2])
    return _case(op, **c)


# ---- what a case holds, from the case alone ------------------------------------------------------

def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _widths(c):
    """Real columns of each row: prompts spread from a tenth of the longest to the longest, plus the
    generated columns; the rest is left padding."""
    gen = c["W"] - c["prompt"]
    lo = max(1, c["prompt"] // 10)
    n = c["rows"]
    return [(c["prompt"] if n == 1 else lo + (c["prompt"] - lo) * r // (n - 1)) + gen for r in range(n)]


def _valid(c):
    return sum(_widths(c))


def _distinct(c):
    """Distinct ids a box really holds (every drawn id is used where the columns suffice)."""
    plain = _valid(c) - c["rows"] * c["masked"]
    return min(c["distinct"], plain) + (1 if c["masked"] else 0)


def work(case):
    c = case
    if c["op"] in ("logprobs", "lossgrad"):
        es, M, slots = _size(c["dtype"]), c["selected"], c["rows"] * c["L"]
        if c["op"] == "logprobs":
            out = M * (4 + (4 if c["entropy"] else 0) + (8 if c["stats"] else 0) + 8 * c["k"])
            return {"bytes": M * c["V"] * es + slots + 4 * M + out, "flops": M * c["V"] * (6 if c["entropy"] else 4)}
        extra = M * (4 + 8 + 4 + (8 if c["entropy"] else 0))
        return {"bytes": M * c["V"] * es + slots * c["V"] * es + slots + extra,
                "flops": M * c["V"] * (8 if c["entropy"] else 5)}
    n, nv, D = c["rows"] * c["W"], _valid(c), c["D"]
    if c["op"] == "embed":
        return {"bytes": _distinct(c) * D * _size(c["table"]) + n * D * _size(c["act"]) + 5 * n, "flops": n * D}
    b = c["batches"]
    dense = c["V"] * D * _size(c["table"])
    again = (b - 1) * 2 * _distinct(c) * D * _size(c["table"])
    return {"bytes": b * (nv * D * _size(c["act"]) + 5 * n) + dense + again, "flops": b * nv * D}


# ---- inputs --------------------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BLOCK = 512            # slots widened to 32 bits at a time by the plain forms


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logit_inputs(c, seed):
    g = _gen(seed)
    rows, L, V, M = c["rows"], c["L"], c["V"], c["selected"]
    dt, slots, pitch = _DT[c["dtype"]], rows * L, V + c["pad"]
    buf = torch.empty(slots * pitch, dtype=dt, device="cuda")
    x = buf.view(slots, pitch)[:, :V]
    top = V - c["banned"]                       # the last `banned` columns can never be answered
    planted = torch.randint(0, top, (slots,), generator=g, device="cuda")
    lift = 14.0 * torch.rand(slots, generator=g, device="cuda")
    for a in range(0, slots, _BLOCK):
        n = min(_BLOCK, slots - a)
        y = 2.0 * torch.randn((n, V), generator=g, device="cuda")
        i = torch.arange(n, device="cuda")
        y[i, planted[a:a + n]] += lift[a:a + n]
        y[:, top:] = -math.inf
        x[a:a + n] = y.to(dt)
    pick = torch.randperm(slots, generator=g, device="cuda")[:M].sort().values
    mask = torch.zeros(slots, dtype=torch.uint8, device="cuda")
    mask[pick] = 1
    other = torch.randint(0, top, (slots,), generator=g, device="cuda")
    keep = torch.rand(slots, generator=g, device="cuda") < 0.7
    tokens = torch.where(keep, planted, other).to(torch.int32)
    s = dict(logits=buf, x=x, pick=pick, mask=mask.view(rows, L), tokens=tokens.view(rows, L), pitch=pitch)
    if c["op"] == "lossgrad":
        s["gl"] = (torch.randn(slots, generator=g, device="cuda") / M).view(rows, L)
        s["gh"] = (0.1 * torch.randn(slots, generator=g, device="cuda") / M).view(rows, L)
    return s


def _box_inputs(c, seed):
    g = _gen(seed)
    rows, W, V, D = c["rows"], c["W"], c["V"], c["D"]
    mask_id, pad_id = V - 2, V - 1
    widths = torch.tensor(_widths(c), device="cuda")
    col = torch.arange(W, device="cuda")
    valid = col[None, :] >= (W - widths)[:, None]
    gen = W - c["prompt"]
    hidden = torch.zeros((rows, W), dtype=torch.bool, device="cuda")
    if c["masked"]:
        order = torch.rand((rows, gen), generator=g, device="cuda").argsort(1)
        hidden[:, W - gen:] = order < c["masked"]
    plain = (valid & ~hidden).nonzero()
    n = plain.shape[0]
    names = torch.randperm(V - 2, generator=g, device="cuda")[:c["distinct"]]
    # frequencies fall off as in text: every id once where the columns suffice, the rest skewed to the first
    d = min(c["distinct"], n)
    rank = (d * torch.rand(n, generator=g, device="cuda") ** 3).long().clamp_(max=d - 1)
    rank[:d] = torch.arange(d, device="cuda")
    ids = torch.full((rows, W), pad_id, dtype=torch.int32, device="cuda")
    shuffle = torch.randperm(n, generator=g, device="cuda")
    ids[plain[:, 0], plain[:, 1]] = names[rank][shuffle].to(torch.int32)
    ids[hidden] = mask_id
    return ids, valid.to(torch.uint8), g


def _scale(c):
    return math.sqrt(c["D"])


def _embed_inputs(c, seed):
    ids, valid, g = _box_inputs(c, seed)
    table = torch.empty((c["V"], c["D"]), dtype=_DT[c["table"]], device="cuda")
    for a in range(0, c["V"], 16384):
        n = min(16384, c["V"] - a)
        table[a:a + n] = (0.02 * torch.randn((n, c["D"]), generator=g, device="cuda")).to(table.dtype)
    return dict(ids=ids, valid=valid, table=table)


def _embedgrad_inputs(c, seed):
    out = []
    for b in range(c["batches"]):
        ids, valid, g = _box_inputs(c, seed * 2 + b)
        go = torch.empty((c["rows"], c["W"], c["D"]), dtype=_DT[c["act"]], device="cuda")
        for r in range(c["rows"]):
            go[r] = (1e-3 * torch.randn((c["W"], c["D"]), generator=g, device="cuda")).to(go.dtype)
        out.append(dict(ids=ids, valid=valid, grad_out=go))
    return dict(batches=out)


def prepare(case, seed):
    c = case
    st = dict(case=c)
    if c["op"] in ("logprobs", "lossgrad"):
        st.update(_logit_inputs(c, seed))
        rows, L, V, dt = c["rows"], c["L"], c["V"], _DT[c["dtype"]]
        f32 = dict(dtype=torch.float32, device="cuda")
        if c["op"] == "logprobs":
            # a record that steps fill in: zero where nothing was asked for
            st["logprob"] = torch.zeros((rows, L), **f32)
            st["entropy"] = torch.zeros((rows, L), **f32) if c["entropy"] else None
            st["stats"] = torch.zeros((rows, L, 2), **f32) if c["stats"] else None
            st["top_ids"] = torch.zeros((rows, L, c["k"]), dtype=torch.int32, device="cuda") if c["k"] else None
            st["top_logprobs"] = torch.zeros((rows, L, c["k"]), **f32) if c["k"] else None
        else:
            # what the forward pass kept for its backward one
            m, s, h = _plain_stats(st, c, want_entropy=True)
            st["stats"] = torch.zeros((rows * L, 2), **f32)
            st["stats"][st["pick"], 0] = m
            st["stats"][st["pick"], 1] = s
            st["stats"] = st["stats"].view(rows, L, 2)
            st["entropy"] = torch.zeros(rows * L, **f32)
            st["entropy"][st["pick"]] = h
            st["entropy"] = st["entropy"].view(rows, L)
            if own:
                st["grad"] = torch.empty((rows, L, V), dtype=dt, device="cuda")
        if own:
            from confidence_block_unmasking_amd import api
            st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            if c["op"] == "logprobs":
                st["ws"] = api.new_logprobs_workspace(rows, L, V, c["k"], dt)
        return st
    if c["op"] == "embed":
        st.update(_embed_inputs(c, seed))
        if own:
            st["out"] = torch.empty((c["rows"], c["W"], c["D"]), dtype=_DT[c["act"]], device="cuda")
            st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return st
    st.update(_embedgrad_inputs(c, seed))
    if own:
        from confidence_block_unmasking_amd import api
        st["grad"] = torch.empty((c["V"], c["D"]), dtype=_DT[c["table"]], device="cuda")
        st["ws"] = api.new_embed_grad_workspace(c["rows"] * c["W"], c["V"], c["D"])
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _OWN[c["op"]](state, c)
    return _PLAIN[c["op"]](state, c)


def _own_logprobs(st, c):
    from confidence_block_unmasking_amd import api
    api.dllm_logprobs(st["logits"], st["mask"], st["tokens"], st["logprob"], st["ws"], st["status"],
                      entropy=st["entropy"], stats=st["stats"], top_ids=st["top_ids"],
                      top_logprobs=st["top_logprobs"], rows=c["rows"], L=c["L"], V=c["V"], pos_stride=st["pitch"],
                      row_stride=c["L"] * st["pitch"])
    return _logprob_outputs(st["logprob"], st["entropy"], st["stats"], st["top_ids"], st["top_logprobs"])


def _own_lossgrad(st, c):
    from confidence_block_unmasking_amd import api
    kw = dict(entropy=st["entropy"], grad_entropy=st["gh"]) if c["entropy"] else {}
    api.dllm_logprobs_grad(st["logits"], st["mask"], st["tokens"], st["stats"], st["gl"], st["grad"], st["status"],
                           rows=c["rows"], L=c["L"], V=c["V"], pos_stride=st["pitch"],
                           row_stride=c["L"] * st["pitch"], **kw)
    return st["grad"]


def _own_embed(st, c):
    from confidence_block_unmasking_amd import api
    api.dllm_embed(st["table"], st["ids"], st["out"], st["status"], valid=st["valid"], scale=_scale(c))
    return st["out"]


def _own_embedgrad(st, c):
    from confidence_block_unmasking_amd import api
    for i, b in enumerate(st["batches"]):
        api.dllm_embed_grad(b["grad_out"], b["ids"], st["grad"], st["ws"], st["status"], valid=b["valid"],
                            scale=_scale(c), accumulate=i > 0)
    return st["grad"]


_OWN = dict(logprobs=_own_logprobs, lossgrad=_own_lossgrad, embed=_own_embed, embedgrad=_own_embedgrad)


def _logprob_outputs(logprob, entropy, stats, top_ids, top_logprobs):
    out = dict(logprob=logprob)
    if entropy is not None:
        out["entropy"] = entropy
    if stats is not None:
        out["stats"] = stats
    if top_ids is not None:
        out["top_ids"] = top_ids
        out["top_logprobs"] = top_logprobs
    return out


def _order_key(y):
    """Distinct int64 keys whose descending order is: larger value first, lower column on ties."""
    b = (y + 0.0).view(torch.int32).long()      # + 0.0: the two zeros are one value
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    V = y.shape[1]
    return b * (1 << 24) + (V - 1 - torch.arange(V, device=y.device))


def _plain_stats(st, c, want_entropy):
    ms, ss, hs = [], [], []
    for a in range(0, st["pick"].numel(), _BLOCK):
        y = st["x"][st["pick"][a:a + _BLOCK]].float()
        m = y.max(1).values
        u = y - m[:, None]
        e = u.exp()
        S = e.sum(1)
        ms.append(m)
        ss.append(S.log())
        if want_entropy:
            hs.append(S.log() - torch.where(e > 0, e * u, torch.zeros_like(u)).sum(1) / S)
    return torch.cat(ms), torch.cat(ss), torch.cat(hs) if want_entropy else None


def _plain_logprobs(st, c):
    rows, L, k = c["rows"], c["L"], c["k"]
    pick = st["pick"]
    m, s, h = _plain_stats(st, c, c["entropy"])
    tok = st["tokens"].view(-1)[pick].long()
    lp = torch.zeros(rows * L, device="cuda")
    lp[pick] = st["x"][pick, tok].float() - m - s
    ent = stats = ti = tl = None
    if c["entropy"]:
        ent = torch.zeros(rows * L, device="cuda")
        ent[pick] = h
        ent = ent.view(rows, L)
    if c["stats"]:
        stats = torch.zeros((rows * L, 2), device="cuda")
        stats[pick] = torch.stack([m, s], 1)
        stats = stats.view(rows, L, 2)
    if k:
        ti = torch.zeros((rows * L, k), dtype=torch.int32, device="cuda")
        tl = torch.zeros((rows * L, k), device="cuda")
        for a in range(0, pick.numel(), _BLOCK):
            p = pick[a:a + _BLOCK]
            y = st["x"][p].float()
            at = _order_key(y).topk(k, dim=1).indices
            ti[p] = at.to(torch.int32)
            tl[p] = y.gather(1, at) - m[a:a + _BLOCK, None] - s[a:a + _BLOCK, None]
        ti, tl = ti.view(rows, L, k), tl.view(rows, L, k)
    return _logprob_outputs(lp.view(rows, L), ent, stats, ti, tl)


def _plain_lossgrad(st, c):
    rows, L, V = c["rows"], c["L"], c["V"]
    pick, dt = st["pick"], _DT[c["dtype"]]
    out = torch.zeros((rows * L, V), dtype=dt, device="cuda")
    stats, tok = st["stats"].view(-1, 2), st["tokens"].view(-1).long()
    gl, gh, ent = st["gl"].view(-1), st["gh"].view(-1), st["entropy"].view(-1)
    for a in range(0, pick.numel(), _BLOCK):
        p = pick[a:a + _BLOCK]
        i = torch.arange(p.numel(), device="cuda")
        u = st["x"][p].float() - stats[p, 0:1] - stats[p, 1:2]
        e = u.exp()
        g = -gl[p, None] * e
        if c["entropy"]:
            g = g - gh[p, None] * torch.where(e > 0, e * (u + ent[p, None]), torch.zeros_like(u))
        g[i, tok[p]] += gl[p]
        out[p] = g.to(dt)
    return out.view(rows, L, V)


def _plain_embed(st, c):
    ids = torch.where(st["valid"] != 0, st["ids"], torch.zeros_like(st["ids"])).long()
    out = torch.empty((c["rows"], c["W"], c["D"]), dtype=_DT[c["act"]], device="cuda")
    for a in range(0, c["rows"], 16):
        y = st["table"][ids[a:a + 16]].float() * _scale(c)
        out[a:a + 16] = (y * (st["valid"][a:a + 16] != 0)[:, :, None]).to(out.dtype)
    return out


def _plain_embedgrad(st, c):
    total = None
    for b in st["batches"]:
        part = torch.zeros((c["V"], c["D"]), device="cuda")
        keep = b["valid"].view(-1) != 0
        ids = torch.where(keep, b["ids"].view(-1), torch.zeros_like(b["ids"].view(-1))).long()
        part.index_add_(0, ids, b["grad_out"].view(-1, c["D"]).float() * (_scale(c) * keep.float())[:, None])
        # each micro-batch leaves the table in its own type
        total = (part if total is None else total.float() + part).to(_DT[c["table"]])
    return total


_PLAIN = dict(logprobs=_plain_logprobs, lossgrad=_plain_lossgrad, embed=_plain_embed, embedgrad=_plain_embedgrad)


# ---- the definitions in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] in ("logprobs", "lossgrad"):
        return _exact_logits(c, _logit_inputs(c, seed))
    if c["op"] == "embed":
        st = _embed_inputs(c, seed)
        out = torch.zeros((c["rows"], c["W"], c["D"]), dtype=torch.float64, device="cuda")
        for r in range(c["rows"]):
            on = st["valid"][r].bool()
            out[r, on] = st["table"].index_select(0, st["ids"][r, on].long()).double().mul(_scale(c))
        return out
    st = _embedgrad_inputs(c, seed)
    out = torch.zeros((c["V"], c["D"]), dtype=torch.float64, device="cuda")
    for b in st["batches"]:
        for r in range(c["rows"]):
            on = b["valid"][r].bool()
            out.index_add_(0, b["ids"][r, on].long(), b["grad_out"][r, on].double(), alpha=_scale(c))
    return out


def _exact_logits(c, st):
    rows, L, V = c["rows"], c["L"], c["V"]
    n, f64 = rows * L, dict(dtype=torch.float64, device="cuda")
    tok = st["tokens"].reshape(-1).long()
    grads = c["op"] == "lossgrad"
    if grads:
        out = torch.zeros((n, V), **f64)
    else:
        k = c["k"]
        lp, ent, stats = torch.zeros(n, **f64), torch.zeros(n, **f64), torch.zeros((n, 2), **f64)
        ti, tl = torch.zeros((n, k), dtype=torch.int32, device="cuda"), torch.zeros((n, k), **f64)
    for p in st["pick"].split(256):
        x = st["x"].index_select(0, p).double()
        lse = torch.logsumexp(x, 1, keepdim=True)
        logp = x - lse
        prob = logp.exp()
        H = -(prob * logp.clamp_min(-1e300)).sum(1, keepdim=True)
        t = tok[p].unsqueeze(1)
        if grads:
            gl = st["gl"].reshape(-1)[p].double().unsqueeze(1)
            g = -gl * prob
            g.scatter_add_(1, t, gl)
            if c["entropy"]:
                gh = st["gh"].reshape(-1)[p].double().unsqueeze(1)
                g -= gh * prob * (logp.clamp_min(-1e300) + H)
            out[p] = g
            continue
        lp[p] = logp.gather(1, t).squeeze(1)
        ent[p] = H.squeeze(1)
        top = x.max(1).values
        stats[p] = torch.stack([top, lse.squeeze(1) - top], 1)
        if k:
            at = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
            ti[p] = at.to(torch.int32)
            tl[p] = logp.gather(1, at)
    if grads:
        return out.view(rows, L, V)
    return _logprob_outputs(lp.view(rows, L), ent.view(rows, L) if c["entropy"] else None,
                            stats.view(rows, L, 2) if c["stats"] else None,
                            ti.view(rows, L, k) if k else None, tl.view(rows, L, k) if k else None)
