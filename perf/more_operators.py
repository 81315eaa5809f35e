"""A head's loss without its logits, and dropout, as measured cases: their plain
forms in elementary torch operations, the framework's calls, and their
definitions in 64 bits.

Head loss (rows i of hidden states x, a dense head w over a vocabulary, label c,
teacher entries (id_k, t_k), temperature T):
    z = x w^T, q = softmax(z / T), s = softmax(z), p = softmax(t / T) over the valid entries
    loss = mix T^2 sum_k p_k (log p_k - log q[id_k]) - (1 - mix) log s[c]
and, in a training step, its gradients by x and w under a weight for every row.
mix = 0 without a teacher is the cross entropy. Rows without label and entries
(padding, prompts) have loss 0 and gradient 0.

Dropout: y = residual + keep * x / (1 - t / 65536), and dx = keep * dy / (1 - t /
65536), where t = round(65536 p) and element i is kept when 16 bits of Philox4x32-10
(key: the seed; counter: i / 8 and the call's offset) are at least t.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _head(name, rows, d, vocab, dtype, top, temperature, mix, step, holes):
    return {"name": name, "op": "head", "rows": rows, "d": d, "vocab": vocab, "dtype": dtype, "top": top, "temperature": temperature, "mix": mix,
            "step": step, "holes": holes}


def _drop(name, rows, d, dtype, p, residual, step, state):
    return {"name": name, "op": "dropout", "rows": rows, "d": d, "dtype": dtype, "p": p, "residual": residual, "step": step, "state": state}


def listed():
    return [
        # one token's block output joined to its residual: latency alone
        _drop("dropout_one_token", 1, 768, "bf16", 0.1, True, False, False),
        # a training step of a 768-wide model: the join's dropout and its backward pass
        _drop("dropout_step", 16384, 768, "bf16", 0.1, True, True, False),
        # an odd width in 32 bits: the 625-feature blocks of the recommender, batch 10000, no residual
        _drop("dropout_step_odd_f32", 10000, 625, "f32", 0.5, False, True, False),
        # a training step of the widest layer, the generator's state on the GPU as a captured step keeps it
        _drop("dropout_step_wide", 8192, 16384, "bf16", 0.2, True, True, True),
        # the cross entropy of 8 tokens in an evaluation, 50257 words
        _head("ce_loss_8", 8, 768, 50257, "bf16", 0, 1.0, 0.0, False, False),
        # a training step of one sequence of 1024 tokens, prompt tokens without labels
        _head("ce_step_1024", 1024, 768, 50257, "bf16", 0, 1.0, 0.0, True, True),
        # a training step of 16 sequences of 1024 tokens
        _head("ce_step_16384", 16384, 768, 50257, "bf16", 0, 1.0, 0.0, True, False),
        # a wide model's step over a vocabulary of 131072
        _head("ce_step_wide", 4096, 4096, 131072, "bf16", 0, 1.0, 0.0, True, False),
        # the recommender's 10000 items from its 625-feature blocks in 32 bits, batch 1000
        _head("ce_step_odd_f32", 1000, 625, 10000, "f32", 0, 1.0, 0.0, True, True),
        # distillation: the loss alone over a validation batch, hard labels mixed in
        _head("distill_loss", 4096, 768, 50257, "bf16", 64, 2.0, 0.5, False, False),
        # a training step of 8 sequences of 1024 tokens, padded tokens and shorter lists, hard labels mixed in
        _head("distill_step_8192", 8192, 768, 50257, "bf16", 32, 2.0, 0.5, True, True),
        # the recommender's step in 32 bits, 512 hidden features, batch 1000
        _head("distill_step_f32", 1000, 512, 10000, "f32", 100, 1.0, 1.0, True, False),
    ]


def _log_between(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = rng.random() < 0.6
    if rng.random() < 0.3:
        d = _log_between(rng, 32, 16384)
        if rng.random() < 0.6:
            d = max(32, d // 32 * 32)
        rows = _log_between(rng, 1, min(65536, (1 << (27 if dtype == "bf16" else 26)) // d))
        c = _drop("", rows, d, dtype, rng.choice([0.1, 0.1, 0.5, round(rng.uniform(0.01, 0.9), 3)]), rng.random() < 0.6, step, rng.random() < 0.3)
    else:
        vocab = _log_between(rng, 512, 131072)
        d = _log_between(rng, 32, 4096)
        if rng.random() < 0.7:
            d = max(32, d // 32 * 32)
        limit = (1 << 40) if dtype == "bf16" else (1 << 38)
        rows = _log_between(rng, 1, max(1, min(16384, (1 << 29) // vocab, limit // (vocab * d))))
        top = 0 if rng.random() < 0.5 else min(vocab, _log_between(rng, 1, 256))
        c = _head("", rows, d, vocab, dtype, top, rng.choice([1.0, 1.0, 2.0, round(rng.uniform(0.5, 4.0), 2)]) if top else 1.0,
                  rng.choice([1.0, 0.5, 0.9]) if top else 0.0, step, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_head if case["op"] == "head" else _prepare_drop)(case, g, seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_drop(c, g, seed):
    t, shape = _TYPES[c["dtype"]], (c["rows"], c["d"])
    s = {"case": c, "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), "offset": seed % 1000003}
    s["x"] = _randn(g, *shape).to(t)
    s["residual"] = (2.0 * _randn(g, *shape)).to(t) if c["residual"] else None
    s["dy"] = _randn(g, *shape).to(t) if c["step"] else None
    s["state"] = torch.tensor([s["seed"], s["offset"]], dtype=torch.int64, device="cuda") if c["state"] else None
    return s


def _prepare_head(c, g, seed):
    rows, d, vocab, top, t = c["rows"], c["d"], c["vocab"], c["top"], _TYPES[c["dtype"]]
    # a head whose logits spread by about 1.5, words of different weight as in trained ones
    w = _randn(g, vocab, d) * (1.5 * d ** -0.5) * torch.exp(0.2 * _randn(g, vocab, 1))
    labels = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    x = _randn(g, rows, d)
    # normed hidden states that already point at their label in part
    x += (4.0 * torch.rand((rows, 1), generator=g, device="cuda")) * w[labels] / 1.5
    s = {"case": c, "w": w.to(t), "teacher": None, "ids": None}
    if top:
        # distinct entries a row: a random start and a step round the vocabulary; the teacher's logits in falling order
        start = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
        ids = (start + torch.arange(top, device="cuda") * max(1, vocab // top)) % vocab
        teacher = torch.sort(_randn(g, rows, top) * 2.0 + 6.0, dim=1, descending=True)[0].contiguous()
        x += w[ids[:, 0]] / 1.5
        hard = torch.rand((rows,), generator=g, device="cuda") < 0.7
        labels = torch.where(hard, ids[:, 0], labels)
    if c["holes"]:
        # prompts and padded tokens have no label (and no entry); shorter lists
        u = torch.rand((rows,), generator=g, device="cuda")
        labels = torch.where(u < 0.25, -100, labels)
        if top:
            kept = torch.where(u < 0.2, 0, torch.where(u < 0.4, (top + 1) // 2, top))
            ids = torch.where(torch.arange(top, device="cuda") < kept[:, None], ids, -1)
    s["x"] = x.to(t)
    if top:
        s["teacher"], s["ids"] = teacher, ids.contiguous()
    s["labels"] = labels if c["mix"] < 1.0 else None
    s["weight"] = (torch.rand((rows,), generator=g, device="cuda") * 0.5 + 0.75) if c["step"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if s["case"]["op"] == "head":
        return _own_head(s) if own else _plain_head(s)
    return _own_drop(s) if own else _plain_drop(s)


def _own_drop(s):
    from monarch_block_diagonal_amd import torch_api as T
    c = s["case"]
    how = dict(state=s["state"]) if c["state"] else dict(seed=s["seed"], offset=s["offset"])
    out = {"y": T.dropout_forward(s["x"], c["p"], residual=s["residual"], **how)}
    if c["step"]:
        out["dx"] = T.dropout_backward(s["dy"], c["p"], **how)
    return out


def _own_head(s):
    from monarch_block_diagonal_amd import torch_api as T
    c = s["case"]
    args, how = (s["x"], s["w"], s["labels"], s["teacher"], s["ids"]), dict(temperature=c["temperature"], mix=c["mix"])
    if c["step"]:
        loss, dx, dw = T.head_loss_step(*args, row_weight=s["weight"], **how)
        return {"loss": loss, "dx": dx, "dw": dw}
    return {"loss": T.head_loss_forward(*args, **how)[0]}


def _plain_keep(n, threshold, seed, offset):
    """Philox4x32-10 over whole tensors: the products of 32-bit words wrap in int64, which keeps their bits."""
    low = 0xFFFFFFFF
    at = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64)
    c0, c1 = at & low, at >> 32
    c2, c3 = torch.full_like(at, offset & low), torch.full_like(at, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), dim=1)
    halves = torch.stack((words & 0xFFFF, words >> 16), dim=2).reshape(-1)[:n]
    return halves >= threshold


def _plain_drop(s):
    c, t = s["case"], s["x"].dtype
    threshold = round(c["p"] * 65536)
    keep = _plain_keep(s["x"].numel(), threshold, s["seed"], s["offset"]).view(s["x"].shape)
    scale = 65536.0 / (65536 - threshold)
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if c["residual"]:
        y = s["residual"].float() + y
    out = {"y": y.to(t)}
    if c["step"]:
        out["dx"] = torch.where(keep, s["dy"].float() * scale, 0.0).to(t)
    return out


def _plain_head(s):
    c = s["case"]
    T, mix, vocab, t = c["temperature"], c["mix"], c["vocab"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    rows = torch.arange(c["rows"], device="cuda")
    z -= z.max(dim=1, keepdim=True)[0]
    loss = torch.zeros((c["rows"],), device="cuda")
    r = s["weight"]
    if c["step"]:
        grad = torch.zeros_like(z)
    if c["top"]:
        inside = (s["ids"] >= 0) & (s["ids"] < vocab) & (s["teacher"] > float("-inf"))
        some, ids = inside.any(dim=1), s["ids"].clamp(0, vocab - 1)
        e = torch.where(inside, s["teacher"] / T, float("-inf"))
        top = torch.where(some, e.max(dim=1)[0], 0.0)[:, None]
        e_exp = torch.exp(e - top)
        e_sum = torch.where(some, e_exp.sum(dim=1), 1.0)[:, None]
        p, log_p = e_exp / e_sum, e - top - torch.log(e_sum)
        q = torch.exp(z / T)
        q_sum = q.sum(dim=1, keepdim=True)
        log_q = torch.gather(z, 1, ids) / T - torch.log(q_sum)
        kl = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(dim=1)
        loss += mix * T * T * torch.where(some, kl, 0.0)
        if c["step"]:
            a = torch.where(some, mix * T * r, 0.0)[:, None]
            grad += q * (a / q_sum)
            grad.scatter_add_(1, ids, -a * p)
        del q
    if s["labels"] is not None:
        told, label = (s["labels"] >= 0) & (s["labels"] < vocab), s["labels"].clamp(0, vocab - 1)
        z_label = z[rows, label]
        e = torch.exp(z)
        e_sum = e.sum(dim=1)
        loss += (1.0 - mix) * torch.where(told, torch.log(e_sum) - z_label, 0.0)
        if c["step"]:
            b = torch.where(told, (1.0 - mix) * r, 0.0)
            grad += e * (b / e_sum)[:, None]
            grad[rows, label] -= b
        del e
    if not c["step"]:
        return {"loss": loss}
    return {"loss": loss, "dx": (grad @ w).to(t), "dw": (grad.t() @ x).to(t)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_head(s) if case["op"] == "head" else _exact_drop(s)


def _exact_drop(s):
    """The generator in 16-bit limbs, no product over 48 bits."""
    c, n = s["case"], s["x"].numel()

    def times(a, m):
        """(high, low) 32-bit words of a * m."""
        p0, p1 = a * (m & 0xFFFF), a * (m >> 16)
        low = p0 + ((p1 & 0xFFFF) << 16)
        return (p1 >> 16) + (low >> 32), low % (1 << 32)

    i = torch.arange(-(-n // 8), dtype=torch.int64, device="cuda")
    ctr = [i % (1 << 32), i // (1 << 32), torch.zeros_like(i) + s["offset"] % (1 << 32), torch.zeros_like(i) + s["offset"] // (1 << 32)]
    for r in range(10):
        key0 = (s["seed"] + r * 0x9E3779B9) % (1 << 32)
        key1 = (s["seed"] // (1 << 32) + r * 0xBB67AE85) % (1 << 32)
        (h0, l0), (h1, l1) = times(ctr[0], 0xD2511F53), times(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ key0, l1, h0 ^ ctr[3] ^ key1, l0]
    drawn = torch.cat([(v[:, None] // (1 << sh)) % 65536 for v in ctr for sh in (0, 16)], dim=1).flatten()[:n].reshape(s["x"].shape)
    cut = int(math.floor(c["p"] * 65536 + 0.5))
    factor = (drawn >= cut).double() / (1.0 - cut / 65536.0)
    y = s["x"].double() * factor
    if s["residual"] is not None:
        y += s["residual"].double()
    return {"y": y, "dx": s["dy"].double() * factor} if c["step"] else {"y": y}


def _exact_head(s):
    """Row blocks in 64 bits; log-probabilities instead of the plain form's quotients, a target distribution spread over the vocabulary."""
    c = s["case"]
    T, mix, vocab, rows = c["temperature"], c["mix"], c["vocab"], c["rows"]
    w = s["w"].double()
    loss = torch.empty((rows,), dtype=torch.float64, device="cuda")
    dx = torch.empty((rows, c["d"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((vocab, c["d"]), dtype=torch.float64, device="cuda")
    at = max(1, (1 << 27) // vocab)
    for first in range(0, rows, at):
        b = slice(first, min(rows, first + at))
        x = s["x"][b].double()
        z = torch.mm(x, w.t())
        val = torch.zeros((z.shape[0],), dtype=torch.float64, device="cuda")
        grad = torch.zeros_like(z)
        r = s["weight"][b].double() if c["step"] else val
        if s["ids"] is not None:
            ids = s["ids"][b]
            ok = (ids >= 0) & (ids < vocab)
            has = ok.any(dim=1)
            t = s["teacher"][b].double().div(T).masked_fill(~ok, float("-inf"))
            t[~has] = 0.0
            logp = torch.log_softmax(t, dim=1)
            p = torch.exp(logp)
            p[~has] = 0.0
            logq = torch.log_softmax(z / T, dim=1)
            cross = (p * torch.gather(logq, 1, ids.clamp(min=0))).masked_fill(p == 0, 0.0)
            val += mix * T ** 2 * (torch.special.xlogy(p, p) - cross).sum(dim=1)
            if c["step"]:
                target = torch.zeros_like(z).scatter_add_(1, ids.clamp(min=0), p)
                grad += (mix * T * r * has)[:, None] * (torch.exp(logq) - target)
                del target
            del logq
        if s["labels"] is not None:
            y = s["labels"][b]
            good = (y >= 0) & (y < vocab)
            logs = torch.log_softmax(z, dim=1)
            pick = torch.arange(z.shape[0], device="cuda")
            val -= (1 - mix) * torch.where(good, logs[pick, y.clamp(min=0)], 0.0)
            if c["step"]:
                part = torch.exp(logs)
                part[pick, y.clamp(min=0)] -= 1.0
                grad += ((1 - mix) * r * good)[:, None] * part
                del part
            del logs
        loss[b] = val
        if c["step"]:
            dx[b] = torch.mm(grad, w)
            dw += torch.mm(grad.t(), x)
    return {"loss": loss, "dx": dx, "dw": dw} if c["step"] else {"loss": loss}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "dropout":
        n = case["rows"] * case["d"]
        tensors = 2 + case["residual"] + (2 if case["step"] else 0)
        return {"bytes": n * size * tensors, "flops": n * (3 + 2 * case["step"])}
    rows, d, vocab, top = case["rows"], case["d"], case["vocab"], case["top"]
    # rows without label and entries need no product: on average a quarter of a case with holes, a fifth with a teacher
    busy = rows * (1.0 if not case["holes"] else 0.8 if top else 0.75)
    product = 2.0 * busy * vocab * d
    tensors = (rows + vocab) * d * size
    return {"bytes": int(tensors * (2 if case["step"] else 1) + rows * (top * 12 + 16)), "flops": int(product * (3 if case["step"] else 1))}
