"""Embedding lookup of a packed box's token ids and its gradient, in float64 ([BlockServe] = page
"BlockServe: 块粒度连续批处理实现高吞吐扩散大语言模型服务" §II-E: the left-padded box; padding contributes
nothing)."""
import numpy as np


def _used(ids, valid, n_vocab):
    ids = np.asarray(ids).reshape(-1)
    on = np.ones(ids.shape, bool) if valid is None else np.asarray(valid).reshape(-1) != 0
    return ids, on & (ids >= 0) & (ids < n_vocab)


def lookup(table, ids, valid=None, scale=1.0):
    ids, on = _used(ids, valid, table.shape[0])
    out = np.zeros((ids.size, table.shape[1]))
    out[on] = float(np.float32(scale)) * np.asarray(table, np.float64)[ids[on]]
    return out


def gradient(grad_out, ids, n_vocab, valid=None, scale=1.0):
    """(gradient [n_vocab, D], the sums of absolute terms, tokens per id)."""
    ids, on = _used(ids, valid, n_vocab)
    g = np.asarray(grad_out, np.float64)[:ids.size]
    s = float(np.float32(scale))
    total = np.zeros((n_vocab, g.shape[1]))
    size = np.zeros_like(total)
    np.add.at(total, ids[on], s * g[on])
    np.add.at(size, ids[on], abs(s) * np.abs(g[on]))
    return total, size, np.bincount(ids[on], minlength=n_vocab)
