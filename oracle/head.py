"""The head loss: a plain fp64 statement of what the library's monarch_head_* entry
points compute, in torch on whatever device its inputs are. TEST INFRASTRUCTURE ONLY
(it shares no code with the HIP path).

    z = x w^T, q = softmax(z / T), s = softmax(z), p = softmax(t / T) over the valid entries
    loss = mix T^2 sum_k p_k (log p_k - log q[id_k]) - (1 - mix) log s[c]
    g = r (mix T (q - p spread) + (1 - mix) (s - onehot(c))), dx = g w, dw = g^T x

Without a teacher's columns mix is 0. A row without a label (mix < 1) and without a valid entry (mix > 0) gives 0 and adds
nothing to dw, whatever it holds.
"""
from __future__ import annotations

from typing import NamedTuple

import torch


class Head(NamedTuple):
    loss: torch.Tensor
    dx: torch.Tensor
    dw: torch.Tensor
    g: torch.Tensor       # gradient of the logits
    s_loss: torch.Tensor  # sums of absolute terms
    s_g: torch.Tensor
    s_z: torch.Tensor     # [rows]: the largest sum of |x||w| of a row's logits
    used: torch.Tensor    # [rows]


def head(x, w, labels=None, teacher=None, ids=None, weight=None, T=1.0, mix=0.0) -> Head:
    x, w = x.double(), w.double()
    rows, vocab, dev = x.shape[0], w.shape[0], x.device
    if teacher is None or not teacher.shape[1]:
        mix = 0.0
    zero = torch.zeros((rows,), dtype=torch.float64, device=dev)
    told = torch.zeros((rows,), dtype=torch.bool, device=dev)
    some = told.clone()
    if labels is not None and mix < 1.0:
        told = (labels >= 0) & (labels < vocab)
    if teacher is not None and teacher.shape[1] and mix > 0.0:
        ok = (ids >= 0) & (ids < vocab) & (teacher > float("-inf"))
        some = ok.any(dim=1)
    used = told | some
    x = torch.where(used[:, None], x, 0.0)
    r = torch.where(used, (zero + 1.0) if weight is None else weight.double(), 0.0)
    z = x @ w.T
    s_z = (x.abs() @ w.abs().T).amax(dim=1) if rows else zero
    loss, s_loss, g, s_g = zero.clone(), zero.clone(), torch.zeros_like(z), torch.zeros_like(z)
    if some.any():
        t = torch.where(ok, teacher.double() / T, float("-inf"))
        t = torch.where(some[:, None], t, 0.0)
        lp = torch.log_softmax(t, dim=1)
        p = torch.where(ok, lp.exp(), 0.0)
        lq = torch.log_softmax(z / T, dim=1)
        at = ids.clamp(0, vocab - 1)
        lqk = lq.gather(1, at)
        use = p > 0
        lp, lqk = torch.where(use, lp, 0.0), torch.where(use, lqk, 0.0)
        loss += mix * T * T * (p * (lp - lqk)).sum(dim=1)
        s_loss += mix * T * T * (p * (1 + lp.abs() + lqk.abs())).sum(dim=1)
        a = (mix * T * r * some)[:, None]
        spread = torch.zeros_like(z).scatter_add_(1, at, p)
        g += a * (lq.exp() - spread)
        s_g += a.abs() * (lq.exp() + spread)
    if told.any():
        ls = torch.log_softmax(z, dim=1)
        c = torch.where(told, labels, 0)[:, None]
        lc = ls.gather(1, c)[:, 0]
        loss -= torch.where(told, (1 - mix) * lc, 0.0)
        s_loss += torch.where(told, (1 - mix) * (1 + lc.abs()), 0.0)
        b = ((1 - mix) * r * told)[:, None]
        one = torch.zeros_like(z).scatter_(1, c, 1.0)
        g += b * (ls.exp() - one)
        s_g += b.abs() * (ls.exp() + one)
    return Head(loss, g @ w, g.T @ x, g, s_loss, s_g, s_z, used)


def bounds(o: Head, x, w, rounding: float, T=1.0):
    """(loss, dx, dw): how far fp32 sums and one rounding of g and of each result may be off.

    A logit: every addition of its sum rounds by at most 2^-24 of the absolute terms, and parts of
    fp32 operands leave out 2^-23 of them: e_z = (d + 2) 2^-24 s_z. Parts under bf16's least normal value
    2^-126 may count as 0: an operand v = v0 + v1 + v2 is then off by |v1| + |v2| < 2^-125 at
    most, and a product x w by 2^-125 (|x| + |w|), which e_z has as well. A loss moves by two logits and by
    2e-5 of its absolute terms (sums of exponentials of up to 2^17 terms joined in runs of at most
    256, and the logarithms). A value of g moves by 2 e_z / min(T, 1) of its absolute terms and by 3e-5 of
    them besides, and is rounded once (`rounding`, 0 where it is not). dx and dw add these up with their
    factors' absolute values, their own sums round by at most 2^-24 an addition, and they are
    rounded once."""
    rows, d = x.shape
    vocab = w.shape[0]
    x, w = torch.where(o.used[:, None], x.double(), 0.0), w.double()
    e_z = (d + 2) * 2.0 ** -24 * o.s_z
    if not rounding:
        e_z = e_z + 2.0 ** -125 * (x.abs().sum(dim=1) + w.abs().sum(dim=1).max())
    loss = 2 * e_z * max(T, 1.0) + 2e-5 * o.s_loss
    e_g = (2 * e_z / min(T, 1.0) + 3e-5)[:, None] * o.s_g + max(rounding, 2.0 ** -23) * o.g.abs()
    top = (o.g.abs() + e_g)
    dx = (e_g + vocab * 2.0 ** -24 * top) @ w.abs()
    dw = (e_g + (rows + 2) * 2.0 ** -24 * top).T @ x.abs()
    half = max(rounding, 2.0 ** -24)
    return loss, dx + half * (o.dx.abs() + dx), dw + half * (o.dw.abs() + dw)
