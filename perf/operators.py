"""The sandwich norm and the distillation loss as measured cases: their plain
forms in elementary torch operations, the framework's calls, and their
definitions in 64 bits.

Sandwich norm (rows i, features j; norm is RMS, LAYER or none):
    u  = norm_post(y) * w_post + b_post
    h' = skip * h + branch * g * u         (gate g: one row for B/G rows of h)
    n  = norm_pre(h') * w_pre + b_pre
and, in a training step, the gradients of everything from dh' and dn.

Distillation from a teacher's top logits (student logits z, teacher entries
(id_k, t_k), label c, temperature T):
    p = softmax(t / T) over the valid entries, q = softmax(z / T), s = softmax(z)
    loss = mix T^2 sum_k p_k (log p_k - log q[id_k]) - (1 - mix) log s[c]
and, in a training step, its gradient by z under a weight for every row.
"""
import math

import torch

own = False

_NORMS = {"none": 0, "rms": 1, "layer": 2}
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(name, rows, d, dtype, post, pre, bias, gates, step):
    return {"name": name, "op": "sandwich", "rows": rows, "d": d, "dtype": dtype, "post": post, "pre": pre, "bias": bias, "gates": gates, "step": step}


def _distill(name, rows, vocab, ld, dtype, top, temperature, mix, step, holes):
    return {"name": name, "op": "distill", "rows": rows, "vocab": vocab, "ld": ld, "dtype": dtype, "top": top, "temperature": temperature, "mix": mix,
            "step": step, "holes": holes}


def listed():
    return [
        # one token through one block of a 768-wide model: latency alone
        _norm("norm_one_token", 1, 768, "bf16", "rms", "rms", False, 1, False),
        # a batch of 64 tokens being generated, 4096 features, a gate for every token
        _norm("norm_64_tokens", 64, 4096, "bf16", "layer", "layer", True, 64, False),
        # a prompt pass of 16 sequences of 1024 tokens, no norm after the block
        _norm("norm_prompt", 16384, 768, "bf16", "none", "layer", True, 1, False),
        # a training step of the same model, one gate for every sequence
        _norm("norm_step", 16384, 768, "bf16", "rms", "rms", False, 16, True),
        # an odd width in 32 bits: the 625-feature blocks of the recommender, batch 10000
        _norm("norm_step_odd_f32", 10000, 625, "f32", "layer", "layer", True, 1, True),
        # a training step of the widest layer, a gate for every token
        _norm("norm_step_wide", 8192, 16384, "bf16", "rms", "rms", False, 8192, True),
        # the loss of 8 tokens in an evaluation, 50257 words
        _distill("distill_loss_8", 8, 50257, 50257, "bf16", 16, 1.0, 1.0, False, False),
        # the loss alone over a validation batch
        _distill("distill_loss", 4096, 50257, 50304, "bf16", 64, 2.0, 0.5, False, False),
        # a training step of the recommender over its 10000 items, batch 1000
        _distill("distill_step_f32", 1000, 10000, 10000, "f32", 100, 1.0, 0.5, True, True),
        # a training step of one sequence of 1024 tokens, rows off every alignment, hard labels mixed in
        _distill("distill_step_1024", 1024, 50257, 50257, "bf16", 64, 2.0, 0.5, True, True),
        # a training step of 16 sequences of 1024 tokens
        _distill("distill_step_16384", 16384, 50257, 50304, "bf16", 32, 1.0, 1.0, True, False),
        # a vocabulary of 131072 in 32 bits, padded rows
        _distill("distill_step_wide_f32", 2048, 131072, 131200, "f32", 256, 1.5, 0.9, True, True),
    ]


def _log_between(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = rng.random() < 0.6
    if rng.random() < 0.5:
        d = _log_between(rng, 32, 16384)
        if rng.random() < 0.6:
            d = max(32, d // 32 * 32)
        rows = _log_between(rng, 1, min(65536, (1 << 25) // d))
        gates = rng.choice([0, 1, rows, max(1, rows // rng.randint(2, 1024))])
        if gates:
            rows = rows // gates * gates
        post, pre = rng.choice(["none", "rms", "layer"]), rng.choice(["none", "rms", "rms", "layer", "layer"])
        c = _norm("", rows, d, dtype, post, pre, rng.random() < 0.5, gates, step)
    else:
        vocab = _log_between(rng, 512, 131072)
        rows = _log_between(rng, 1, min(16384, (1 << 28) // vocab))
        ld = vocab if rng.random() < 0.5 else (vocab + 64 + 63) // 64 * 64
        c = _distill("", rows, vocab, ld, dtype, _log_between(rng, 1, 256), rng.choice([1.0, 1.0, 2.0, round(rng.uniform(0.5, 4.0), 2)]),
                     rng.choice([1.0, 0.5, 0.9]), step, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_norm if case["op"] == "sandwich" else _prepare_distill)(case, g)


def _normal(g, shape, std, dtype, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _prepare_norm(c, g):
    rows, d, t = c["rows"], c["d"], _TYPES[c["dtype"]]
    s = {"case": c, "skip": 1.0, "branch": 0.5, "eps": 1e-5}
    # a residual stream whose features differ in size, as they do in trained models, and a block's output
    s["h"] = (torch.randn((rows, d), generator=g, device="cuda") * torch.exp(0.5 * torch.randn((d,), generator=g, device="cuda"))).to(t)
    s["y"] = _normal(g, (rows, d), 0.7, t, 0.1)
    s["post_weight"] = _normal(g, (d,), 0.2, t, 1.0)
    s["post_bias"] = _normal(g, (d,), 0.1, t) if c["bias"] else None
    s["gate"] = _normal(g, (c["gates"], d), 0.3, t, 0.8) if c["gates"] else None
    s["pre_weight"] = _normal(g, (d,), 0.2, t, 1.0) if c["pre"] != "none" else None
    s["pre_bias"] = _normal(g, (d,), 0.1, t) if c["bias"] and c["pre"] != "none" else None
    if c["step"]:
        s["dh"] = _normal(g, (rows, d), 1.0, t)
        s["dn"] = _normal(g, (rows, d), 1.0, t) if c["pre"] != "none" else None
    return s


def _prepare_distill(c, g):
    rows, vocab, top, t = c["rows"], c["vocab"], min(c["top"], c["vocab"]), _TYPES[c["dtype"]]
    buf = torch.empty((rows, c["ld"]), device="cuda", dtype=t)
    buf.normal_(generator=g).mul_(2.5)
    z = buf[:, :vocab]
    # distinct teacher entries a row: a random start and an odd step round the vocabulary
    start = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
    stride = max(1, vocab // top)
    ids = (start + torch.arange(top, device="cuda") * stride) % vocab
    # a teacher's logits in falling order; the student agrees with it in part
    teacher = torch.sort(torch.randn((rows, top), generator=g, device="cuda") * 2.0 + 6.0, dim=1, descending=True)[0].contiguous()
    z.scatter_(1, ids, (0.6 * teacher + torch.randn((rows, top), generator=g, device="cuda")).to(t))
    labels = ids[:, 0].clone()
    other = torch.rand((rows,), generator=g, device="cuda") < 0.3
    labels = torch.where(other, torch.randint(0, vocab, (rows,), generator=g, device="cuda"), labels)
    if c["holes"]:
        # padded tokens (no entry, no label), shorter lists, logits masked out of the vocabulary
        u = torch.rand((rows,), generator=g, device="cuda")
        kept = torch.where(u < 0.05, 0, torch.where(u < 0.3, (top + 1) // 2, top))
        ids = torch.where(torch.arange(top, device="cuda") < kept[:, None], ids, -1)
        labels = torch.where(u < 0.1, -100, labels)
        last = torch.arange(vocab - vocab // 100, vocab, device="cuda")
        taken = torch.zeros((rows, vocab), dtype=torch.bool, device="cuda")
        taken.scatter_(1, ids.clamp(min=0), True)
        taken.scatter_(1, labels.clamp(min=0)[:, None], True)
        z[:, last] = torch.where(taken[:, last], z[:, last], float("-inf"))
    weight = torch.rand((rows,), generator=g, device="cuda") * 0.5 + 0.75
    return {"case": c, "z": z, "teacher": teacher, "ids": ids, "labels": labels if c["mix"] < 1.0 else None, "weight": weight}


# ---------------------------------------------------------------- one pass

def run(s):
    if s["case"]["op"] == "sandwich":
        return _own_norm(s) if own else _plain_norm(s)
    return _own_distill(s) if own else _plain_distill(s)


def _own_norm(s):
    from monarch_block_diagonal_amd import torch_api as T
    c = s["case"]
    how = dict(post_norm=_NORMS[c["post"]], pre_norm=_NORMS[c["pre"]], skip_scale=s["skip"], branch_scale=s["branch"], eps=s["eps"])
    affine = (s["post_weight"], s["post_bias"], s["gate"], s["pre_weight"], s["pre_bias"])
    h_out, n, stats = T.sandwich_forward(s["h"], s["y"], *affine, **how)
    out = {"h_out": h_out, "n": n}
    if c["step"]:
        out.update(T.sandwich_backward(s["dh"], s["dn"], h_out, s["y"], stats, *affine, **how)._asdict())
    return out


def _own_distill(s):
    from monarch_block_diagonal_amd import torch_api as T
    c = s["case"]
    args = (s["z"], s["teacher"], s["ids"], s["labels"])
    if c["step"]:
        loss, dz = T.distill_step(*args, row_weight=s["weight"], temperature=c["temperature"], mix=c["mix"])
        return {"loss": loss, "dz": dz}
    return {"loss": T.distill_forward(*args, temperature=c["temperature"], mix=c["mix"])[0]}


def _plain_stats(v, kind, eps):
    """(normalised v, rho); rho is None without a norm."""
    if kind == "none":
        return v, None
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    rho = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)
    return v * rho, rho


def _plain_norm_grad(q, hat, rho, kind):
    if kind == "none":
        return q
    q = q - hat * (q * hat).mean(dim=1, keepdim=True) - (q.mean(dim=1, keepdim=True) if kind == "layer" else 0.0)
    return q * rho


def _plain_norm(s):
    c, t = s["case"], s["h"].dtype
    rows, d, gates = c["rows"], c["d"], c["gates"]
    f = {k: v.float() for k, v in s.items() if isinstance(v, torch.Tensor)}
    yhat, rho_y = _plain_stats(f["y"], c["post"], s["eps"])
    u = yhat * f["post_weight"]
    if "post_bias" in f:
        u = u + f["post_bias"]
    gate = f["gate"].repeat_interleave(rows // gates, dim=0) if gates > 1 else f["gate"] if gates else 1.0
    h_out = s["skip"] * f["h"] + s["branch"] * (gate * u)
    n = None
    if c["pre"] != "none":
        hhat, rho_h = _plain_stats(h_out, c["pre"], s["eps"])
        n = hhat * f["pre_weight"]
        if "pre_bias" in f:
            n = n + f["pre_bias"]
    out = {"h_out": h_out.to(t), "n": None if n is None else n.to(t)}
    if not c["step"]:
        return out
    dh = f["dh"]
    if c["pre"] != "none":
        dh = dh + _plain_norm_grad(f["dn"] * f["pre_weight"], hhat, rho_h, c["pre"])
        out["dpre_weight"] = (f["dn"] * hhat).sum(dim=0).to(t)
        out["dpre_bias"] = f["dn"].sum(dim=0).to(t) if "pre_bias" in f else None
    else:
        out["dpre_weight"] = out["dpre_bias"] = None
    out["dh"] = (s["skip"] * dh).to(t)
    e = s["branch"] * gate * dh
    out["dgate"] = (s["branch"] * dh * u).reshape(gates, rows // gates, d).sum(dim=1).to(t) if gates else None
    out["dy"] = _plain_norm_grad(e * f["post_weight"], yhat, rho_y, c["post"]).to(t)
    out["dpost_weight"] = (e * yhat).sum(dim=0).to(t)
    out["dpost_bias"] = e.sum(dim=0).to(t) if "post_bias" in f else None
    return out


def _plain_distill(s):
    c, z = s["case"], s["z"].float()
    T, mix, vocab = c["temperature"], c["mix"], c["vocab"]
    ids, inside = s["ids"].clamp(0, vocab - 1), (s["ids"] >= 0) & (s["ids"] < vocab) & (s["teacher"] > float("-inf"))
    some = inside.any(dim=1)
    # teacher: softmax over the valid entries, 0 elsewhere
    t = torch.where(inside, s["teacher"] / T, float("-inf"))
    t_top = torch.where(some, t.max(dim=1)[0], 0.0)[:, None]
    t_exp = torch.exp(t - t_top)
    t_sum = torch.where(some, t_exp.sum(dim=1), 1.0)[:, None]
    p, log_p = t_exp / t_sum, t - t_top - torch.log(t_sum)
    # student
    top = z.max(dim=1, keepdim=True)[0]
    alive = top[:, 0] > float("-inf")
    z = z - torch.where(alive[:, None], top, 0.0)
    q = torch.exp(z / T)
    q_sum = torch.where(alive, q.sum(dim=1), 1.0)[:, None]
    log_q = torch.gather(z, 1, ids) / T - torch.log(q_sum)
    kl = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(dim=1)
    loss = mix * T * T * torch.where(some & alive, kl, 0.0)
    if s["labels"] is not None:
        told = (s["labels"] >= 0) & (s["labels"] < vocab) & alive
        label = s["labels"].clamp(0, vocab - 1)[:, None]
        e = torch.exp(z)
        e_sum = torch.where(alive, e.sum(dim=1), 1.0)[:, None]
        ce = torch.log(e_sum) - torch.gather(z, 1, label)
        loss = loss + (1.0 - mix) * torch.where(told, ce[:, 0], 0.0)
    if not c["step"]:
        return {"loss": loss}
    w = s["weight"]
    a = torch.where(some & alive, mix * T * w, 0.0)[:, None]
    dz = q * (a / q_sum)
    dz.scatter_add_(1, ids, -a * p)
    if s["labels"] is not None:
        b = torch.where(told, (1.0 - mix) * w, 0.0)[:, None]
        dz = dz + e * (b / e_sum)
        dz.scatter_add_(1, label, -b)
    return {"loss": loss, "dz": dz.to(s["z"].dtype)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "sandwich" else _exact_distill(s)


def _exact_norm(s):
    """Forward as written above; the gradients are those of sum(dh * h') + sum(dn * n), by the chain rule of autograd."""
    c = s["case"]
    x = {k: (v.double().requires_grad_(c["step"]) if isinstance(v, torch.Tensor) else v) for k, v in s.items()}

    def affine(v, kind, w, b):
        if kind != "none":
            mean = v.mean(dim=-1, keepdim=True) if kind == "layer" else torch.zeros((), dtype=v.dtype, device=v.device)
            v = (v - mean) / torch.sqrt((v - mean).pow(2).mean(dim=-1, keepdim=True) + s["eps"])
        v = v * w
        return v if b is None else v + b

    u = affine(x["y"], c["post"], x["post_weight"], x["post_bias"])
    if c["gates"]:
        u = (u.reshape(c["gates"], -1, c["d"]) * x["gate"][:, None, :]).reshape(c["rows"], c["d"])
    h_out = s["skip"] * x["h"] + s["branch"] * u
    n = affine(h_out, c["pre"], x["pre_weight"], x["pre_bias"]) if c["pre"] != "none" else None
    out = {"h_out": h_out.detach(), "n": None if n is None else n.detach()}
    if not c["step"]:
        return out
    total = (x["dh"].detach() * h_out).sum()
    if n is not None:
        total = total + (x["dn"].detach() * n).sum()
    names = [k for k in ("h", "y", "post_weight", "post_bias", "gate", "pre_weight", "pre_bias") if x[k] is not None]
    grads = dict(zip(names, torch.autograd.grad(total, [x[k] for k in names])))
    out.update({"d" + k: grads.get(k) for k in ("h", "y", "post_weight", "post_bias", "gate", "pre_weight", "pre_bias")})
    return out


def _exact_distill(s):
    """Row blocks in 64 bits; log-probabilities instead of the plain form's quotients."""
    c = s["case"]
    T, mix, vocab, rows = c["temperature"], c["mix"], c["vocab"], c["rows"]
    loss, dz = torch.empty((rows,), dtype=torch.float64, device="cuda"), None
    if c["step"]:
        dz = torch.empty((rows, vocab), dtype=torch.float64, device="cuda")
    at = max(1, (1 << 27) // vocab)
    for r in range(0, rows, at):
        b = slice(r, min(rows, r + at))
        z, ids = s["z"][b].double(), s["ids"][b]
        m = z.shape[0]
        ok = (ids >= 0) & (ids < vocab)
        # the teacher's distribution spread over the vocabulary
        t = s["teacher"][b].double().div(T).masked_fill(~ok, float("-inf"))
        has = ok.any(dim=1)
        t[~has] = 0.0
        logp = t - torch.logsumexp(t, dim=1, keepdim=True)
        p = torch.exp(logp)
        p[~has] = 0.0
        lq = z / T
        lq = lq - torch.logsumexp(lq, dim=1, keepdim=True)
        # p log p - p log q, with 0 log 0 = 0
        at_ids = torch.gather(lq, 1, ids.clamp(min=0))
        terms = (torch.special.xlogy(p, p) - (p * at_ids).masked_fill(p == 0, 0.0)).sum(dim=1)
        val = mix * T ** 2 * terms
        w = s["weight"][b].double()
        if dz is not None:
            grad = torch.exp(lq) * (mix * T * w * has)[:, None]
            grad.scatter_add_(1, ids.clamp(min=0), -mix * T * w[:, None] * p)
        if s["labels"] is not None:
            y = s["labels"][b]
            good = (y >= 0) & (y < vocab)
            ls = z - torch.logsumexp(z, dim=1, keepdim=True)
            val = val - (1 - mix) * torch.where(good, ls[torch.arange(m, device="cuda"), y.clamp(min=0)], 0.0)
            if dz is not None:
                grad += torch.exp(ls) * ((1 - mix) * w * good)[:, None]
                grad[torch.arange(m, device="cuda"), y.clamp(min=0)] -= (1 - mix) * w * good
        loss[b] = val
        if dz is not None:
            dz[b] = grad
    return {"loss": loss, "dz": dz} if dz is not None else {"loss": loss}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sandwich":
        n = case["rows"] * case["d"]
        pre = case["pre"] != "none"
        # h, y in; h', n out; a step also dh', dn in and dh, dy out
        tensors = (3 + pre) + ((3 + pre) if case["step"] else 0)
        small = case["d"] * (1 + pre) * (1 + case["bias"]) + case["gates"] * case["d"]
        return {"bytes": (tensors * n + small * (2 if case["step"] else 1)) * size, "flops": n * (35 if case["step"] else 10)}
    n = case["rows"] * case["vocab"]
    entries = case["rows"] * min(case["top"], case["vocab"]) * 12
    return {"bytes": n * size * (2 if case["step"] else 1) + entries + case["rows"] * 16,
            "flops": n * (4 if case["mix"] == 1.0 else 7) * (2 if case["step"] else 1)}
