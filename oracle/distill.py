"""Distillation from a teacher's top logits: a plain fp64 CPU statement of what
the library's monarch_distill_* entry points compute. TEST INFRASTRUCTURE ONLY
(same rules as monarch_oracle; it shares no code with the HIP path).

Row by row, with student logits z [V], teacher entries (id, t), label c:

    p    = softmax(t / T) over the valid entries, spread over the vocabulary
    loss = mix T^2 sum_j p_j (log p_j - log softmax(z / T)_j) - (1 - mix) log softmax(z)_c
    dz   = w (mix T (softmax(z / T) - p) + (1 - mix) (softmax(z) - onehot(c)))

An entry is valid with 0 <= id < V and t > -inf, a label with 0 <= c < V. The first
term is absent without a valid entry, the second without a label; a row with
neither, or with z = -inf throughout, gives 0. p_j = 0 adds nothing.

p of entries that name one id is their sum; the loss counts every entry's own
p_k (log p_k - log q[id_k]).
"""
from __future__ import annotations

import numpy as np


def log_softmax(z):
    m = z.max()
    e = z - m
    return e - np.log(np.exp(e).sum())


def row(z, teacher, ids, label, T, mix):
    """(loss, dz at w = 1, S_loss, S_dz): the last two are the sums of absolute terms."""
    z = np.asarray(z, dtype=np.float64)
    V = z.size
    ok = (ids >= 0) & (ids < V) & (np.asarray(teacher, np.float64) > -np.inf)
    told = label is not None and 0 <= label < V and mix < 1.0
    some = bool(ok.any()) and mix > 0.0
    dz, sdz = np.zeros(V), np.zeros(V)
    loss = sloss = 0.0
    if (not some and not told) or np.all(np.isneginf(z)):
        return loss, dz, sloss, sdz
    if some:
        t, at = np.asarray(teacher, np.float64)[ok] / T, np.asarray(ids)[ok]
        lp, lq = log_softmax(t), log_softmax(z / T)
        p = np.exp(lp)
        use = p > 0
        loss += mix * T * T * float((p[use] * (lp[use] - lq[at[use]])).sum())
        sloss += mix * T * T * float((p[use] * (1 + np.abs(lp[use]) + np.abs(lq[at[use]]))).sum())
        spread = np.zeros(V)
        np.add.at(spread, at, p)
        dz += mix * T * (np.exp(lq) - spread)
        sdz += mix * T * (np.exp(lq) + spread)
    if told:
        ls = log_softmax(z)
        loss += -(1.0 - mix) * ls[label]
        sloss += (1.0 - mix) * (1 + abs(ls[label]))
        dz += (1.0 - mix) * np.exp(ls)
        dz[label] -= 1.0 - mix
        sdz += (1.0 - mix) * np.exp(ls)
        sdz[label] += 1.0 - mix
    return loss, dz, sloss, sdz


def rows(z, teacher, ids, labels=None, weight=None, T=1.0, mix=1.0):
    """(loss, dz, S_loss, S_dz) of every row."""
    out = [row(z[i], teacher[i], ids[i], None if labels is None else int(labels[i]), T, mix)
           for i in range(len(z))]
    loss, dz, sl, sd = (np.array([o[k] for o in out]) for k in range(4))
    w = np.ones(len(z)) if weight is None else np.asarray(weight, np.float64)
    return loss, dz * w[:, None], sl, sd * np.abs(w)[:, None]
