"""Log probabilities, entropy and alternatives of one slot's logits, and their gradient, in float64.

The distribution is the softmax of a masked slot's vocabulary logits ([DiLaServe] = page "DiLaServe:
High SLO Attainment Serving for Diffusion Language Models" §三 3.1).  -inf logits have probability 0;
a slot of -inf only, or with NaN or +inf, has no distribution (NaN).
"""
import numpy as np


def slot(x, token=None, k=0):
    """dict(m, logS, logprob, entropy, top_ids, top_logprobs, E1, E2) of one slot's logits x (any
    float array).  E1, E2: the means of |u| and u^2 under the distribution, u = x - m, from which the
    tests derive what float32 may lose."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        m = x.max() if not np.isnan(x).any() else np.nan
        u = x - m
        e = np.exp(u)
        S = e.sum()
        logp = u - np.log(S)
        p = e / S
        live = p > 0
        bad = not np.isfinite(S)
        H = np.nan if bad else -float((p[live] * logp[live]).sum())
        order = np.argsort(-x, kind="stable")[:k]
        return dict(m=m, logS=np.log(S) if not bad else np.nan, entropy=H,
                    logprob=np.nan if token is None or bad else logp[token], top_ids=order.astype(np.int32),
                    top_logprobs=logp[order], E1=float((p[live] * -u[live]).sum()),
                    E2=float((p[live] * u[live] ** 2).sum()), p=p, logp=logp)


def grad(x, token, gl, gh):
    """d/dx of gl * logprob(token) + gh * entropy."""
    o = slot(x)
    p, logp = o["p"], o["logp"]
    g = -gl * p
    live = p > 0
    g[live] -= gh * p[live] * (logp[live] + o["entropy"])
    if token is not None:
        g[token] += gl
    return g
