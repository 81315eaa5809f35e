"""GPU parity of the sandwich norm against its fp64 oracle, and its refusals.

Bounds, element by element, derived from the formulas: a result may be off by
its own rounding (2^-8 of it in bf16, nothing to speak of in fp32) and by T
times the sum of the absolute values of its terms, where T is 1e-5 in fp32
(sums of up to 16384 terms, each partial sum of at most 100 terms in a row) and
in bf16 2^-8 for everything computed from h_out, which the backward pass reads
as it was rounded. The scales S below are those sums.
"""
import numpy as np
import pytest

from oracle import sandwich as O
from monarch_block_diagonal_amd import synthetic as S

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROUND = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8}
KINDS = {"none": 0, "rms": 1, "layer": 2}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    return torch_api


def dev(a, dtype):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda:0")
    return t if dtype == "f32" else t.to(torch.bfloat16)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def draw(rows, d, gates, bias, dtype, seed=7300, offset=0.1, pre="rms", y=True):
    n = lambda k, shape, var=1.0, mean=0.0: S.round_to_bf16(S.draw(seed + k, shape, "normal", var) + np.float32(mean)) \
        if dtype == "bf16" else S.draw(seed + k, shape, "normal", var) + np.float32(mean)  # noqa: E731
    a = dict(h=n(0, (rows, d)), y=n(1, (rows, d), 0.5, offset) if y else None,
             post_w=n(2, (d,), 0.04, 1.0) if y else None, post_b=n(3, (d,), 0.04) if bias and y else None,
             gate=n(4, (gates, d), 0.2, 0.7) if gates else None,
             pre_w=n(5, (d,), 0.04, 1.0) if pre != "none" else None,
             pre_b=n(6, (d,), 0.04) if bias and pre != "none" else None)
    return a, n(8, (rows, d)), (n(9, (rows, d)) if pre != "none" else None)


def scales(a, dh, dn, post, pre, skip, branch, eps):
    """Sums of absolute terms of every result (see the module's text)."""
    A, rows = np.abs, a["h"].shape[0]
    one = lambda v, d=1.0: d if v is None else A(np.asarray(v, np.float64))  # noqa: E731
    h_out, _ = O.forward(a["h"], a["y"], a["post_w"], a["post_b"], a["gate"], a["pre_w"], a["pre_b"], post, pre, skip,
                         branch, eps)

    def spread(v, kind):
        v = np.asarray(v, np.float64)
        if kind == "none":
            return A(v), 1.0
        _, _, rho = O.norm(v, kind, eps)
        mu = A(v).mean(axis=1, keepdims=True) if kind == "layer" else 0.0
        return rho * (A(v) + mu), rho

    s = {}
    g = 1.0
    if a["y"] is not None:
        Ay, rho_y = spread(a["y"], post)
        if a["gate"] is not None:
            g = A(np.repeat(np.asarray(a["gate"], np.float64), rows // a["gate"].shape[0], axis=0))
        Su = Ay * one(a["post_w"]) + one(a["post_b"], 0.0)
        s["h_out"] = abs(skip) * A(a["h"]) + abs(branch) * g * Su
    else:
        s["h_out"] = A(np.asarray(a["h"], np.float64))
    SD = np.zeros_like(s["h_out"]) if dh is None else A(np.asarray(dh, np.float64))
    if pre != "none":
        Ah, rho_h = spread(h_out, pre)
        Ah = Ah + rho_h * s["h_out"]
        s["n"] = Ah * one(a["pre_w"]) + one(a["pre_b"], 0.0)
        q = A(np.asarray(dn, np.float64)) * one(a["pre_w"])
        SD = SD + rho_h * (q + 2 * Ah * (q * Ah).mean(axis=1, keepdims=True) + q.mean(axis=1, keepdims=True))
        s["dpre_w"] = (A(dn) * Ah).sum(axis=0)
        s["dpre_b"] = A(dn).astype(np.float64).sum(axis=0)
    s["dh"] = abs(skip) * SD if a["y"] is not None else SD
    if a["y"] is not None:
        e = abs(branch) * g * SD
        q2 = e * one(a["post_w"])
        s["dy"] = q2
        if post != "none":
            s["dy"] = rho_y * (q2 + 2 * Ay * (q2 * Ay).mean(axis=1, keepdims=True) + q2.mean(axis=1, keepdims=True))
        if a["gate"] is not None:
            s["dgate"] = (abs(branch) * SD * Su).reshape(a["gate"].shape[0], -1, a["h"].shape[1]).sum(axis=1)
        s["dpost_w"], s["dpost_b"] = (e * Ay).sum(axis=0), e.sum(axis=0)
    return s


def check(name, got, want, scale, dtype, t):
    assert got.shape == want.shape, name
    over = np.abs(host(got) - want) - (ROUND[dtype] * np.abs(want) + t * scale)
    assert np.isfinite(over).all() and over.max() <= 0, (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


def compare(api, rows, d, gates, bias, dtype, post, pre, skip=1.0, branch=0.5, eps=1e-5, offset=0.1, y=True, with_dh=True):
    print(f"[sandwich] rows={rows} d={d} gates={gates} bias={bias} {dtype} {post}/{pre} y={y} dh={with_dh}", flush=True)
    a, dh, dn = draw(rows, d, gates, bias, dtype, offset=offset, pre=pre, y=y)
    if not with_dh:
        dh = None
    how = dict(post_norm=KINDS[post], pre_norm=KINDS[pre], skip_scale=skip, branch_scale=branch)
    D = {k: dev(v, dtype) for k, v in a.items()}
    par = (D["post_w"], D["post_b"], D["gate"], D["pre_w"], D["pre_b"])
    h_out, n, stats = api.sandwich_forward(D["h"], D["y"], *par, eps=eps, **how)
    g = api.sandwich_backward(dev(dh, dtype), dev(dn, dtype), h_out, D["y"], stats, *par, **how)
    torch.cuda.synchronize()
    par = (a["post_w"], a["post_b"], a["gate"], a["pre_w"], a["pre_b"])
    rh, rn = O.forward(a["h"], a["y"], *par, post, pre, skip, branch, eps)
    rg = O.backward(dh, dn, a["h"], a["y"], *par, post, pre, skip, branch, eps)
    s = scales(a, dh, dn, post, pre, skip, branch, eps)
    check("h_out", h_out, rh, s["h_out"], dtype, 1e-5)
    if pre == "none":
        assert n is None
    else:
        check("n", n, rn, s["n"], dtype, 1e-5)
    t = {"f32": 1e-5, "bf16": 2.0 ** -8}[dtype]
    for mine, theirs, given in (("dh", "dh", "h"), ("dy", "dy", "y"), ("dpost_weight", "dpost_w", "post_w"),
                                ("dpost_bias", "dpost_b", "post_b"), ("dgate", "dgate", "gate"),
                                ("dpre_weight", "dpre_w", "pre_w"), ("dpre_bias", "dpre_b", "pre_b")):
        got = getattr(g, mine)
        if a[given] is None:
            assert got is None, mine
        else:
            check(mine, got, rg[theirs], s[theirs], dtype, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,gates", [
    (1, 1, 0), (1, 1, 1), (3, 2, 3), (5, 7, 5), (2, 31, 1), (33, 128, 3), (17, 250, 17), (100, 256, 4), (10, 513, 10),
    (700, 625, 1), (1000, 768, 1000), (1024, 768, 16), (4096, 768, 0), (90, 1000, 3), (300, 1536, 100), (65, 2050, 65),
    (40, 4096, 40), (257, 4097, 1), (24, 6150, 2), (12, 8192, 6), (9, 16383, 3), (66, 16384, 2), (5, 16384, 5),
])
def test_shapes(api, rows, d, gates, dtype):
    compare(api, rows, d, gates, (rows + d) % 2 == 0, dtype, "rms", "layer" if d % 3 else "rms")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("post", list(KINDS))
@pytest.mark.parametrize("pre", list(KINDS))
@pytest.mark.parametrize("gates", [0, 2, 74])
def test_norm_kinds(api, post, pre, gates, bias, dtype):
    compare(api, 148, 136, gates, bias, dtype, post, pre, skip=0.75, branch=-1.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_a_block(api, dtype):
    compare(api, 50, 768, 0, True, dtype, "rms", "layer", y=False)
    compare(api, 50, 770, 0, False, dtype, "rms", "rms", y=False, with_dh=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_final_norm_has_no_residual_gradient(api, dtype):
    compare(api, 20, 96, 1, True, dtype, "layer", "rms", with_dh=False)


def test_a_mean_far_from_zero(api):
    # features around 100 with a spread of 0.7: the variance is that of the centred features
    compare(api, 64, 768, 1, True, "f32", "layer", "layer", offset=100.0)
    compare(api, 64, 4096, 64, False, "bf16", "layer", "layer", offset=100.0)


def test_gate_runs_longer_and_shorter_than_a_chunk(api):
    for rows, gates in ((33 * 5, 5), (32 * 5, 5), (600, 1), (3000, 3), (5000, 2500), (7, 7)):
        compare(api, rows, 72, gates, True, "f32", "rms", "rms")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("d", [135, 767, 1023, 4095, 12001])
def test_odd_widths_by_gate_run(api, d, bias, dtype):
    """One gate, long runs, short runs and a gate a row: each has its own kernel, with and without biases."""
    for gates in (0, 2, 35, 70):
        compare(api, 70, d, gates, bias, dtype, "layer", "rms")


@pytest.mark.parametrize("bias", [False, True])
def test_many_long_gate_runs(api, bias):
    """More runs than a launch has teams are taken whole, whatever their length; fewer are cut."""
    compare(api, 33 * 4096, 8, 4096, bias, "f32", "rms", "rms")
    compare(api, 33 * 4095, 8, 4095, bias, "f32", "rms", "rms")
    compare(api, 40 * 512, 1032, 512, bias, "bf16", "rms", "layer")
    compare(api, 40 * 1024, 129, 1024, bias, "f32", "layer", "rms")


def test_results_do_not_change_from_run_to_run(api):
    a, dh, dn = draw(5000, 768, 5, True, "bf16")
    D = {k: dev(v, "bf16") for k, v in a.items()}
    par = (D["post_w"], D["post_b"], D["gate"], D["pre_w"], D["pre_b"])
    DH, DN = dev(dh, "bf16"), dev(dn, "bf16")

    def step():
        h_out, n, stats = api.sandwich_forward(D["h"], D["y"], *par)
        return (h_out, n, *api.sandwich_backward(DH, DN, h_out, D["y"], stats, *par))

    first = step()
    for _ in range(3):
        for x, y in zip(first, step()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_row_stays_alone(api, value):
    rows, d = 64, 768
    a, dh, dn = draw(rows, d, rows, True, "f32")
    a["y"][7, 100] = value
    a["h"][20, 3] = value
    dn[33, 5] = value
    D = {k: dev(v, "f32") for k, v in a.items()}
    par = (D["post_w"], D["post_b"], D["gate"], D["pre_w"], D["pre_b"])
    h_out, n, stats = api.sandwich_forward(D["h"], D["y"], *par)
    g = api.sandwich_backward(dev(dh, "f32"), dev(dn, "f32"), h_out, D["y"], stats, *par)
    bad = lambda t: sorted(set(torch.nonzero(~torch.isfinite(t))[:, 0].tolist()))  # noqa: E731
    assert bad(n) == [7, 20]
    assert bad(h_out) == [7, 20]
    assert bad(g.dh) == [7, 20, 33] and bad(g.dy) == [7, 20, 33] and bad(g.dgate) == [7, 20, 33]


def test_zero_rows_of_a_block(api):
    # a row of zeros: rho = 1/sqrt(eps), results 0, gradients finite
    D = dict(h=torch.zeros(8, 64, device="cuda"), y=torch.zeros(8, 64, device="cuda"))
    h_out, n, stats = api.sandwich_forward(D["h"], D["y"])
    g = api.sandwich_backward(torch.ones_like(h_out), torch.ones_like(n), h_out, D["y"], stats)
    assert not h_out.any() and not n.any()
    assert torch.isfinite(g.dh).all() and torch.isfinite(g.dy).all()


def test_no_rows(api):
    w = torch.ones(64, device="cuda")
    h = torch.empty(0, 64, device="cuda")
    h_out, n, stats = api.sandwich_forward(h, h.clone(), w, w, None, w, w)
    assert h_out.shape == n.shape == (0, 64)
    g = api.sandwich_backward(h, h.clone(), h_out, h.clone(), stats, w, w, None, w, w)
    for t in (g.dpost_weight, g.dpost_bias, g.dpre_weight, g.dpre_bias):
        assert t.shape == (64,) and not t.any()


def test_in_place(api):
    """h_out in h's memory, n in y's; dh in dh_out's."""
    from monarch_block_diagonal_amd import binding as B
    rows, d = 300, 768
    a, dh, dn = draw(rows, d, 0, False, "bf16")
    D = {k: dev(v, "bf16") for k, v in a.items()}
    par = (D["post_w"], None, None, D["pre_w"], None)
    h_out, n, stats = api.sandwich_forward(D["h"], D["y"], *par)
    g = api.sandwich_backward(dev(dh, "bf16"), dev(dn, "bf16"), h_out, D["y"], stats, *par)
    h, y, st = D["h"].clone(), D["y"].clone(), torch.empty_like(stats)
    B.monarch_sandwich_fwd(h, y, *par, h, y, st, rows, d, 0, 1, 1, 1.0, 1.0, 1e-5, B.BF16)
    assert torch.equal(h, h_out) and torch.equal(y, n) and torch.equal(st, stats)
    need = B.monarch_sandwich_bwd_workspace_bytes(rows, d, 0, False, B.BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    DH, dy = dev(dh, "bf16"), torch.empty_like(D["y"])
    B.monarch_sandwich_bwd(DH, dev(dn, "bf16"), h_out, D["y"], stats, *par, DH, dy, None, None, None, None, None, ws, need,
                           rows, d, 0, 1, 1, 1.0, 1.0, B.BF16)
    assert torch.equal(DH, g.dh) and torch.equal(dy, g.dy)


def test_another_stream(api):
    a, dh, dn = draw(500, 768, 1, True, "f32")
    D = {k: dev(v, "f32") for k, v in a.items()}
    par = (D["post_w"], D["post_b"], D["gate"], D["pre_w"], D["pre_b"])
    want = api.sandwich_forward(D["h"], D["y"], *par)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = api.sandwich_forward(D["h"], D["y"], *par)
    s.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_offsets_past_32_bits(api):
    """2^31 elements and more in a tensor: the last rows come out as the same rows alone do."""
    rows, d, last = (1 << 17) + 40, 16384, 64
    t = torch.bfloat16
    w = torch.linspace(0.5, 1.5, d, device="cuda").to(t)
    h, y = torch.zeros(rows, d, dtype=t, device="cuda"), torch.zeros(rows, d, dtype=t, device="cuda")
    tail = slice(rows - last, rows)
    h[tail].normal_()
    y[tail].normal_()
    h_out, n, stats = api.sandwich_forward(h, y, w, None, None, w, None)
    small = api.sandwich_forward(h[tail].clone(), y[tail].clone(), w, None, None, w, None)
    assert torch.equal(h_out[tail], small[0]) and torch.equal(n[tail], small[1])
    assert not h_out[: rows - last].any() and not n[: rows - last].any()
    g = api.sandwich_backward(h, y, h_out, y, stats, w, None, None, w, None)
    sg = api.sandwich_backward(h[tail].clone(), y[tail].clone(), small[0], y[tail].clone(), small[2], w, None, None, w, None)
    assert torch.equal(g.dh[tail], sg.dh) and torch.equal(g.dy[tail], sg.dy)


def test_refusals(api):
    h = torch.zeros(6, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    bad = [
        dict(h=h[0]), dict(y=torch.zeros(5, 64, device="cuda")), dict(post_weight=torch.ones(63, device="cuda")),
        dict(gate=torch.ones(4, 64, device="cuda")), dict(gate=torch.ones(12, 64, device="cuda")),
        dict(gate=torch.ones(0, 64, device="cuda")), dict(gate=torch.ones(64, device="cuda")),
        dict(y=None, gate=torch.ones(1, 64, device="cuda")), dict(y=None, skip_scale=2.0),
        dict(pre_norm=0, pre_weight=w), dict(h=h.cpu()), dict(y=torch.zeros(64, 6, device="cuda").T),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            api.sandwich_forward(**{**dict(h=h, y=h.clone()), **kw})
    with pytest.raises(TypeError):
        api.sandwich_forward(h, h.to(torch.bfloat16))
    with pytest.raises(TypeError):
        api.sandwich_forward(h.half(), h.half())
    from monarch_block_diagonal_amd import MonarchError
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(branch_scale=float("inf")), dict(post_norm=3), dict(pre_norm=-1)):
        with pytest.raises(MonarchError):
            api.sandwich_forward(h, h.clone(), **kw)
    with pytest.raises(MonarchError):
        wide = torch.zeros(1, 16385, device="cuda")
        api.sandwich_forward(wide, wide.clone())
    h_out, n, stats = api.sandwich_forward(h, h.clone())
    for args in ((h, None, h_out, h, stats), (h, h[:5], h_out, h, stats), (h, h, h_out, h, stats[:5]),
                 (h, h, h_out, h, stats.double())):
        with pytest.raises(ValueError):
            api.sandwich_backward(*args)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("rows,d,gates", [(512, 768, 16), (64, 768, 2), (256, 16384, 8), (90, 767, 6), (28, 7, 4), (30, 4095, 3)])
def test_few_short_gate_runs(api, rows, d, gates, bias, dtype):
    """Cut into chunks over the whole chip."""
    compare(api, rows, d, gates, bias, dtype, "rms", "layer", branch=-0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("d,gates,run", [
    (7, 4096, 3), (72, 3000, 5), (135, 700, 2), (136, 700, 32), (767, 700, 2), (768, 1100, 9), (1023, 700, 3), (4095, 512, 2), (4096, 512, 3),
    (12001, 256, 2), (16384, 256, 2),
])
def test_many_short_gate_runs(api, d, gates, run, bias, dtype):
    """Each a team's own."""
    compare(api, gates * run, d, gates, bias, dtype, "layer", "rms", branch=-0.5)


@pytest.mark.parametrize("rows,d,gates,pre,mean", [
    (2048, 768, 16, "rms", 0.0), (2048, 768, 0, "layer", 24.0), (300, 767, 300, "layer", 24.0), (900, 2048, 300, "rms", 24.0),
    (700, 7, 1, "layer", 0.0), (257, 6151, 257, "rms", 0.0), (200, 16384, 4, "layer", 24.0),
])
def test_bf16_gradients_carry_one_rounding(api, rows, d, gates, pre, mean):
    """The gradients of h' itself: their own rounding, and no more of h_out's than the kept bits leave.

    In 2-norms, in units of a gradient's own rounding to bf16: a value of h' is off by at most 1/16 of what h_out's is (1/32
    but for ties), so with r the size of h' over that of the centred row a gradient that takes hhat value by value is off
    by r/16 besides; twice that for the spread of the mantissas, and a tenth of a rounding for everything in fp32.
    From h_out alone dpre_weight would be sqrt(1 + r^2) off."""
    a, dh, dn = draw(rows, d, gates, True, "bf16", pre=pre)
    a["h"] = S.round_to_bf16(a["h"] * np.float32(0.5) + np.float32(mean))
    how = dict(post_norm=KINDS["rms"], pre_norm=KINDS[pre], skip_scale=1.0, branch_scale=0.5)
    D = {k: dev(v, "bf16") for k, v in a.items()}
    par = (D["post_w"], D["post_b"], D["gate"], D["pre_w"], D["pre_b"])
    h_out, n, stats = api.sandwich_forward(D["h"], D["y"], *par, **how)
    g = api.sandwich_backward(dev(dh, "bf16"), dev(dn, "bf16"), h_out, D["y"], stats, *par, **how)
    par = (a["post_w"], a["post_b"], a["gate"], a["pre_w"], a["pre_b"])
    rh, _ = O.forward(a["h"], a["y"], *par, "rms", pre, 1.0, 0.5)
    rg = O.backward(dh, dn, a["h"], a["y"], *par, "rms", pre, 1.0, 0.5)
    _, c, _ = O.norm(rh, pre, 1e-5)
    r = float(np.linalg.norm(rh) / np.linalg.norm(c))
    for mine, theirs in (("dh", "dh"), ("dy", "dy"), ("dpre_weight", "dpre_w"), ("dgate", "dgate"), ("dpost_weight", "dpost_w")):
        if mine == "dgate" and not gates:
            continue
        want = rg[theirs]
        own = np.linalg.norm(host(torch.from_numpy(want).to(torch.bfloat16)) - want)
        off = np.linalg.norm(host(getattr(g, mine)) - want)
        print(f"[rounding] {rows}x{d} {pre} mean={mean} r={r:.1f} {mine}: {off / own:.2f} roundings", flush=True)
        assert off <= np.hypot(1.1, r / 8) * own, (mine, off / own, r)
