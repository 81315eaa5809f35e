"""GPU parity of the distillation loss and gradient against the fp64 oracle, and
its refusals.

Bounds, derived from the formulas: sums of exponentials are off by at most
2e-5 of themselves (a thread adds up to 256 terms in a row in fp32, 256 * 2^-24;
an exponent of up to 100 rounded to 2^-24 of itself adds 0.7e-5 to terms that
small), so a loss by 2e-5 of the sum of its absolute terms (a logarithm counted
as 1 more) and a gradient by 3e-5 of its own, besides the rounding of the result
(2^-8 of it in bf16) and 1e-37 for what is flushed to zero.
"""
import numpy as np
import pytest

from oracle import distill as O
from monarch_block_diagonal_amd import synthetic as S

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROUND = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    return torch_api


def draw(rows, V, K, dtype, seed=8100, scale=2.5):
    z = S.draw(seed, (rows, V), "normal", scale * scale, dtype)
    t = S.draw(seed + 1, (rows, K), "normal", 4.0)
    r = np.random.default_rng(seed + 2)
    if rows * V <= 1 << 22:
        ids = np.stack([r.permutation(V)[:K] for _ in range(rows)]) if V >= K else r.integers(0, V, (rows, K))
    else:
        ids = (r.integers(0, V, (rows, 1)) + np.arange(K) * (V // K)) % V
    labels = np.where(r.random(rows) < 0.5, ids[:, 0] if K else 0, r.integers(0, V, rows))
    return z, t, ids.astype(np.int64), labels.astype(np.int64), (0.5 + r.random(rows)).astype(np.float32)


def place(z, dtype, ld, shift=0):
    """The rows on the GPU, `ld` elements apart, `shift` elements into their memory; NaN between them."""
    rows, V = z.shape
    buf = torch.full((rows * ld + shift + 64,), float("nan"), dtype=TYPES[dtype], device="cuda")
    view = torch.as_strided(buf, (rows, V), (ld, 1), shift)
    view.copy_(torch.from_numpy(z))
    return view, buf


def cu(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(what, got, want, scale, rounding, t):
    got = host(got)
    # a result past the range of fp32 (the loss of a label at the type's lowest value) is an infinity there
    with np.errstate(over="ignore"):
        want = np.where(np.isinf(want.astype(np.float32)), want.astype(np.float32), want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        over = np.abs(got - want) - (rounding * np.abs(want) + t * scale + 1e-37)
    over = np.where(same, -1.0, over)
    assert not np.isnan(over).any() and over.max() <= 0, (what, float(over.max()), np.unravel_index(over.argmax(), over.shape))


def compare(api, z, t, ids, labels, w, dtype, T, mix, ld=None, shift=0):
    rows, V = z.shape
    ld = ld or V
    print(f"[distill] rows={rows} V={V} ld={ld}+{shift} K={t.shape[1]} {dtype} T={T} mix={mix} labels={labels is not None}", flush=True)
    Z, buf = place(z, dtype, ld, shift)
    before = buf.clone()
    args = (Z, cu(t), cu(ids), cu(labels))
    how = dict(temperature=T, mix=mix)
    W = cu(w)
    loss, stats = api.distill_forward(*args, **how)
    dz = api.distill_backward(W if W is not None else torch.ones(rows, device="cuda"), *args, stats, **how)
    loss2, dz2 = api.distill_step(*args, row_weight=W, **how)
    torch.cuda.synchronize()
    assert torch.equal(buf.view(torch.uint8), before.view(torch.uint8)), "the logits changed"
    rl, rd, sl, sd = O.rows(z, t, ids, labels, w, T, mix)
    for what, l, g in (("fwd/bwd", loss, dz), ("step", loss2, dz2)):
        check(what + " loss", l, rl, sl, 0.0, 2e-5)
        check(what + " dz", g, rd, sd, ROUND[dtype], 3e-5)
    # in the logits' own memory: the same values, and nothing beside the rows touched
    loss3, dz3 = api.distill_step(*args, row_weight=W, out=Z, **how)
    torch.cuda.synchronize()
    assert dz3.data_ptr() == Z.data_ptr()
    assert torch.equal(loss3.view(torch.int32), loss2.view(torch.int32))
    assert torch.equal(dz3.contiguous().view(torch.uint8), dz2.contiguous().view(torch.uint8))
    torch.as_strided(buf, (rows, V), (ld, 1), shift).copy_(torch.as_strided(before, (rows, V), (ld, 1), shift))
    assert torch.equal(buf.view(torch.uint8), before.view(torch.uint8)), "columns outside the vocabulary changed"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V,K,pad,shift", [
    (1, 1, 1, 0, 0), (3, 2, 1, 0, 1), (4, 7, 7, 1, 3), (5, 100, 16, 0, 0), (9, 512, 33, 64, 5), (17, 1000, 100, 0, 0),
    (33, 1023, 10, 0, 1), (7, 4096, 512, 0, 0), (6, 4097, 64, 3, 2), (20, 10000, 100, 0, 0), (3, 16385, 50, 0, 7),
    (4, 32768, 64, 0, 0), (5, 50257, 64, 0, 0), (3, 50257, 256, 47, 0), (2, 65537, 16, 0, 0), (3, 131072, 128, 128, 0),
    (2, 262147, 512, 0, 3), (300, 640, 5, 0, 0),
])
def test_shapes(api, rows, V, K, pad, shift, dtype):
    z, t, ids, labels, w = draw(rows, V, K, dtype)
    compare(api, z, t, ids, labels, w, dtype, 2.0, 0.5, V + pad, shift)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,mix,with_labels", [
    (1.0, 1.0, False), (1.0, 0.5, True), (1.0, 0.0, True), (2.0, 0.5, False), (0.5, 0.9, True), (3.7, 0.0, True),
    (10.0, 1.0, True), (0.05, 0.5, True),
])
@pytest.mark.parametrize("V", [333, 20000])
def test_terms(api, V, T, mix, with_labels, dtype):
    z, t, ids, labels, w = draw(6, V, 20, dtype, seed=8200)
    compare(api, z, t, ids, labels if with_labels else None, None if T == 1.0 else w, dtype, T, mix)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [200, 9001, 70001])
def test_holes(api, V, dtype):
    """Rows without entries, without labels, without either; entries out of range, -inf, NaN or twice; masked logits."""
    z, t, ids, labels, w = draw(12, V, 24, dtype, seed=8300)
    low = float(torch.finfo(TYPES[dtype]).min)
    ids[0] = -1
    ids[1], labels[1] = -1, -100
    labels[2] = V
    ids[3, 5:] = -1
    ids[4, 3] = V
    ids[4, 4] = 1 << 40
    ids[4, 6] = -(1 << 40)
    t[5, 2:9] = -np.inf
    t[5, 10] = np.nan
    ids[6, 7] = ids[6, 2]
    ids[6, 20] = ids[6, 2]
    labels[6] = ids[6, 2]
    t[7] = -np.inf
    free = np.setdiff1d(np.arange(V), np.append(ids[8], labels[8]))
    z[8, free[: len(free) // 2]] = -np.inf
    z[8, free[len(free) // 2]] = low
    z[9] = low
    z[10] = -np.inf
    z[11, 1:] = low
    compare(api, z, t, ids, labels, w, dtype, 2.0, 0.5)
    compare(api, z, t, ids, labels, w, dtype, 0.5, 0.5)
    compare(api, z, t, ids, None, w, dtype, 1.0, 1.0)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("V", [500, 80000])
def test_a_bad_row_stays_alone(api, V, value):
    z, t, ids, labels, w = draw(8, V, 10, "f32", seed=8400)
    z[3, V // 2] = value
    z[5, V - 1] = value
    ids[5], labels[5] = -1, -100      # padding: nothing to learn, whatever its logits hold
    args = (cu(z), cu(t), cu(ids), cu(labels))
    loss, dz = api.distill_step(*args, temperature=2.0, mix=0.5)
    loss2, stats = api.distill_forward(*args, temperature=2.0, mix=0.5)
    dz2 = api.distill_backward(torch.ones(8, device="cuda"), *args, stats, temperature=2.0, mix=0.5)
    for l, g in ((loss, dz), (loss2, dz2)):
        bad = [i for i in range(8) if not torch.isfinite(l[i]) or not torch.isfinite(g[i]).all()]
        assert bad == [3]
        assert torch.isnan(l[3]) and torch.isnan(g[3]).all()
        assert l[5] == 0 and not g[5].any()


def test_a_wish_for_a_masked_word(api):
    z, t, ids, labels, w = draw(2, 300, 4, "f32", seed=8500)
    z[1, ids[1, 2]] = -np.inf
    compare(api, z, t, ids, None, None, "f32", 2.0, 1.0)


def test_gradient_against_differences(api):
    z, t, ids, labels, w = draw(3, 65, 8, "f32", seed=8600)
    args = (cu(t), cu(ids), cu(labels))
    loss, dz = api.distill_step(cu(z), *args, cu(w), temperature=2.0, mix=0.5)
    h = 0.05
    for j in range(0, 65, 4):
        up, down = z.copy(), z.copy()
        up[:, j] += h
        down[:, j] -= h
        a = host(api.distill_forward(cu(up), *args, temperature=2.0, mix=0.5)[0])
        b = host(api.distill_forward(cu(down), *args, temperature=2.0, mix=0.5)[0])
        # central difference of a loss of about 10 in fp32 (1e-6 / h), third derivatives below 1 (h^2 / 6)
        assert np.abs((a - b) / (2 * h) * w - host(dz)[:, j]).max() < 1e-3


def test_results_do_not_change_from_run_to_run(api):
    z, t, ids, labels, w = draw(64, 20001, 200, "bf16", seed=8700)
    ids[:, 100] = ids[:, 3]
    args = (cu(z).bfloat16(), cu(t), cu(ids), cu(labels), cu(w))
    first = api.distill_step(*args, temperature=2.0, mix=0.5)
    for _ in range(3):
        for x, y in zip(first, api.distill_step(*args, temperature=2.0, mix=0.5)):
            assert torch.equal(x, y)


def test_no_rows_and_no_entries(api):
    z = torch.randn(4, 100, device="cuda")
    e = torch.empty(0, 5, device="cuda")
    loss, dz = api.distill_step(z[:0], e, e.long())
    assert loss.shape == (0,) and dz.shape == (0, 100)
    none = torch.empty(4, 0, device="cuda")
    labels = torch.tensor([1, 99, -1, 100], device="cuda")
    loss, dz = api.distill_step(z, none, none.long(), labels, mix=0.25)
    want = 0.75 * torch.nn.functional.cross_entropy(z[:2].double(), labels[:2], reduction="none")
    assert torch.allclose(loss[:2].double(), want, rtol=2e-5) and not loss[2:].any() and not dz[2:].any()
    loss, dz = api.distill_step(z, none, none.long())
    assert not loss.any() and not dz.any()


def test_offsets_past_32_bits(api):
    rows, V = 17000, 131072
    z = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    z[-3:].normal_()
    t = torch.randn(rows, 8, device="cuda")
    ids = torch.arange(8, device="cuda").repeat(rows, 1) * 1000 + 5
    loss, dz = api.distill_step(z, t, ids)
    few = api.distill_step(z[-3:].clone(), t[-3:].clone(), ids[-3:].clone())
    assert torch.equal(loss[-3:], few[0]) and torch.equal(dz[-3:], few[1])
    lo, stats = api.distill_forward(z, t, ids)
    assert torch.equal(lo[-3:], api.distill_forward(z[-3:].clone(), t[-3:].clone(), ids[-3:].clone())[0])


def test_another_stream(api):
    z, t, ids, labels, w = draw(50, 5000, 20, "f32", seed=8800)
    args = (cu(z), cu(t), cu(ids), cu(labels), cu(w))
    want = api.distill_step(*args, mix=0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = api.distill_step(*args, mix=0.5)
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_refusals(api):
    z = torch.zeros(4, 50, device="cuda")
    t, ids = torch.zeros(4, 3, device="cuda"), torch.zeros(4, 3, dtype=torch.int64, device="cuda")
    lab = torch.zeros(4, dtype=torch.int64, device="cuda")
    w = torch.ones(4, device="cuda")
    good = dict(logits=z, teacher=t, ids=ids, labels=lab, row_weight=w)
    api.distill_step(**good)
    wide = torch.zeros(4, 513, device="cuda")
    for kw in (dict(logits=z[0]), dict(logits=torch.zeros(50, 4, device="cuda").T), dict(logits=z[:1].expand(4, 50)),
               dict(logits=z.cpu()), dict(teacher=t[:3]), dict(teacher=t[:, 0]), dict(ids=ids[:, :2]), dict(labels=lab[:3]),
               dict(row_weight=w[:2]), dict(teacher=torch.zeros(3, 4, device="cuda").T), dict(labels=lab.cpu()),
               dict(teacher=wide, ids=wide.long()), dict(out=z[:3]), dict(out=z.bfloat16()), dict(out=z.T.contiguous().T)):
        with pytest.raises(ValueError):
            api.distill_step(**{**good, **kw})
    for kw in (dict(teacher=t.bfloat16()), dict(ids=ids.int()), dict(labels=lab.int()), dict(row_weight=w.double()), dict(logits=z.half())):
        with pytest.raises(TypeError):
            api.distill_step(**{**good, **kw})
    from monarch_block_diagonal_amd import MonarchError
    for kw in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=1e30),
               dict(mix=-0.1), dict(mix=1.5), dict(mix=float("nan"))):
        with pytest.raises(MonarchError):
            api.distill_step(**{**good, **kw})
    loss, stats = api.distill_forward(z, t, ids, lab)
    for args in ((w[:2], z, t, ids, lab, stats), (w, z, t, ids, lab, stats[:2]), (w, z, t, ids, lab, stats.double())):
        with pytest.raises(ValueError):
            api.distill_backward(*args)
