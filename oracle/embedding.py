"""Embedding lookup and its gradient in float64 (oracle; test infrastructure only).

  out[t] = scale table[id_t]   (zeros for id < 0, NaN for id >= vocab)
  d[v]   = scale sum of dout[t] over the tokens t with id_t = v, token by token
"""

import numpy as np


def lookup(table, ids, scale=1.0):
    table = np.asarray(table, np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, v in enumerate(ids):
        if v >= table.shape[0]:
            out[t] = np.nan
        elif v >= 0:
            out[t] = table[v] * scale
    return out


def grad(ids, dout, vocab, scale=1.0):
    """(gradient, sum of the magnitudes that were added up, tokens of each row)."""
    dout = np.asarray(dout, np.float64)
    d, size = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1]))
    count = np.zeros(vocab, np.int64)
    for t, v in enumerate(ids):
        if 0 <= v < vocab:
            d[v] += dout[t]
            size[v] += np.abs(dout[t])
            count[v] += 1
    return d * scale, size * abs(scale), count
