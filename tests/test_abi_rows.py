"""Host-side checks of the sandwich norm's and the distillation loss's C entries:
bad arguments are rejected before any HIP call, in the documented order."""
import pytest

import monarch_block_diagonal_amd as M
from monarch_block_diagonal_amd import binding as B

A, A2 = 0x10000, 0x20000     # fake 16-byte aligned device addresses (never dereferenced)
MIS = 0x10008


def sandwich_fwd(h=A, y=A, pw=A, pb=A, g=A, w=A, b=A, ho=A2, n=A2, st=A2, rows=6, d=64, gates=2, post=1, pre=2,
                 skip=1.0, branch=1.0, eps=1e-5, dt=B.F32):
    return M.load_library().monarch_sandwich_fwd(h, y, pw, pb, g, w, b, ho, n, st, rows, d, gates, post, pre, skip, branch,
                                                 eps, dt, None, None, 0)


def sandwich_bwd(dho=A, dn=A, ho=A, y=A, st=A, pw=A, pb=A, g=A, w=A, b=A, dh=A2, dy=A2, dpw=A2, dpb=A2, dg=A2, dw=A2,
                 db=A2, ws=A2, wsb=1 << 40, rows=6, d=64, gates=2, post=1, pre=2, skip=1.0, branch=1.0, dt=B.F32):
    return M.load_library().monarch_sandwich_bwd(dho, dn, ho, y, st, pw, pb, g, w, b, dh, dy, dpw, dpb, dg, dw, db, ws, wsb,
                                                 rows, d, gates, post, pre, skip, branch, dt, None, None, 0)


@pytest.mark.parametrize("kw", [dict(dt=2), dict(dt=-1), dict(post=3), dict(post=-1), dict(pre=3)])
def test_sandwich_dtype_and_norms(kw):
    assert sandwich_fwd(**kw) == B.MONARCH_ERR_DTYPE
    assert sandwich_bwd(**kw) == B.MONARCH_ERR_DTYPE


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=16385), dict(gates=-1), dict(gates=4),
                                dict(gates=12), dict(gates=7)])
def test_sandwich_shapes(kw):
    assert sandwich_fwd(**kw) == B.MONARCH_ERR_SHAPE
    assert sandwich_bwd(**kw) == B.MONARCH_ERR_SHAPE
    sizes = {k: kw.get(k, v) for k, v in dict(rows=6, d=64, gates=2).items()}
    assert M.monarch_sandwich_bwd_workspace_bytes(sizes["rows"], sizes["d"], sizes["gates"], True, B.F32) == 0


@pytest.mark.parametrize("kw", [dict(skip=float("nan")), dict(branch=float("inf"))])
def test_sandwich_scales(kw):
    assert sandwich_fwd(**kw) == B.MONARCH_ERR_VALUE
    assert sandwich_bwd(**kw) == B.MONARCH_ERR_VALUE


def test_sandwich_eps():
    for eps in (-1.0, float("nan"), float("inf")):
        assert sandwich_fwd(eps=eps) == B.MONARCH_ERR_VALUE


@pytest.mark.parametrize("kw", [dict(h=None), dict(ho=None), dict(n=None), dict(st=None), dict(g=None)])
def test_sandwich_fwd_null(kw):
    assert sandwich_fwd(**kw) == B.MONARCH_ERR_NULL


@pytest.mark.parametrize("kw", [dict(dn=None), dict(ho=None), dict(st=None), dict(dh=None), dict(dy=None), dict(g=None),
                                dict(ws=None), dict(pre=0, dho=None), dict(y=None), dict(pw=None), dict(pb=None),
                                dict(w=None), dict(b=None), dict(gates=0)])
def test_sandwich_bwd_null(kw):
    # the last ones: a gradient is asked for of a parameter that there is not
    assert sandwich_bwd(**kw) == B.MONARCH_ERR_NULL


@pytest.mark.parametrize("name", ["h", "y", "pw", "pb", "g", "w", "b", "ho", "n", "st"])
def test_sandwich_fwd_align(name):
    assert sandwich_fwd(**{name: MIS}) == B.MONARCH_ERR_ALIGN


@pytest.mark.parametrize("name", ["dho", "dn", "ho", "y", "st", "pw", "pb", "g", "w", "b", "dh", "dy", "dpw", "dpb", "dg",
                                  "dw", "db", "ws"])
def test_sandwich_bwd_align(name):
    assert sandwich_bwd(**{name: MIS}) == B.MONARCH_ERR_ALIGN


def test_sandwich_workspace():
    need = M.monarch_sandwich_bwd_workspace_bytes(6, 64, 2, True, B.F32)
    assert need > 0 and sandwich_bwd(wsb=need - 256) == B.MONARCH_ERR_WORKSPACE
    assert M.monarch_sandwich_bwd_workspace_bytes(0, 64, 0, False, B.F32) == 0
    a = M.monarch_sandwich_bwd_workspace_bytes(10000, 768, 0, False, B.BF16)
    assert M.monarch_sandwich_bwd_workspace_bytes(10000, 768, 0, True, B.BF16) == 2 * a
    # bounded by the number of chunks or gate rows, not by the rows
    assert M.monarch_sandwich_bwd_workspace_bytes(1 << 24, 768, 0, False, B.BF16) <= 512 * 2 * 768 * 4 + 256
    assert M.monarch_sandwich_bwd_workspace_bytes(40 << 24, 8, 1 << 24, False, B.BF16) <= 8192 * 2 * 8 * 4 + 256


def test_sandwich_no_rows_and_description():
    assert sandwich_fwd(rows=0, gates=0, h=None, y=None, ho=None, n=None, st=None) == B.MONARCH_OK
    assert M.monarch_sandwich_describe(0, 6, 64, 2, B.F32) == ["sandwich_fwd"]
    assert M.monarch_sandwich_describe(1, 6, 64, 2, B.F32) == ["sandwich_bwd", "sandwich_join"]
    assert M.monarch_sandwich_describe(0, 0, 64, 0, B.F32) == []
    with pytest.raises(M.MonarchError):
        M.monarch_sandwich_describe(0, 6, 0, 0, B.F32)


def distill(kind, z=A, ld=100, t=A, ids=A, lab=A, per=A, loss=A2, st=A2, dz=A2, dld=100, rows=4, vocab=100, top=8, T=2.0,
            mix=0.5, dt=B.F32):
    lib = M.load_library()
    if kind == "fwd":
        return lib.monarch_distill_fwd(z, ld, t, ids, lab, loss, st, rows, vocab, top, T, mix, dt, None, None, 0)
    if kind == "bwd":
        return lib.monarch_distill_bwd(per, z, ld, t, ids, lab, st, dz, dld, rows, vocab, top, T, mix, dt, None, None, 0)
    return lib.monarch_distill_step(z, ld, t, ids, lab, per, loss, dz, dld, rows, vocab, top, T, mix, dt, None, None, 0)


KINDS = ("fwd", "bwd", "step")


@pytest.mark.parametrize("kind", KINDS)
def test_distill_sizes_and_values(kind):
    for dt in (-1, 2):
        assert distill(kind, dt=dt) == B.MONARCH_ERR_DTYPE
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=1 << 31, ld=1 << 31), dict(vocab=(1 << 30) + 1, ld=1 << 31), dict(ld=99), dict(top=-1),
               dict(top=513)):
        assert distill(kind, **kw) == B.MONARCH_ERR_SHAPE, kw
    for kw in (dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=1e7), dict(T=1e-7), dict(mix=-0.5), dict(mix=1.1),
               dict(mix=float("nan"))):
        assert distill(kind, **kw) == B.MONARCH_ERR_VALUE, kw
    assert distill(kind, rows=0, z=None, t=None, ids=None, lab=None, loss=None, dz=None, per=None, st=None) == B.MONARCH_OK


def test_distill_null_and_align():
    for kind, names in (("fwd", ("z", "t", "ids", "loss")), ("bwd", ("z", "t", "ids", "per", "st", "dz")),
                        ("step", ("z", "t", "ids", "loss", "dz"))):
        for name in names:
            assert distill(kind, **{name: None}) == B.MONARCH_ERR_NULL, (kind, name)
    for kind in ("bwd", "step"):
        assert distill(kind, dld=99) == B.MONARCH_ERR_SHAPE
    # logits are aligned to their elements only
    assert distill("fwd", z=A + 2) == B.MONARCH_ERR_ALIGN
    assert distill("fwd", z=A + 1, dt=B.BF16) == B.MONARCH_ERR_ALIGN
    for name, by in (("t", 2), ("ids", 4), ("lab", 4), ("loss", 2), ("st", 8)):
        assert distill("fwd", **{name: A + by}) == B.MONARCH_ERR_ALIGN, name
    assert distill("step", dz=A + 2) == B.MONARCH_ERR_ALIGN
    assert distill("step", per=A + 2) == B.MONARCH_ERR_ALIGN


def test_sandwich_bwd_gradients_of_an_absent_norm():
    """Without norm_pre its parameters are not used: asking for their gradients is an error, not memory left as it was."""
    gone = dict(pre=0, dn=None, ho=None)
    for rows, gates in ((6, 2), (0, 0)):
        for kw in (dict(dw=A2, db=None), dict(dw=None, db=A2)):
            assert sandwich_bwd(**gone, rows=rows, gates=gates, dg=A2 if gates else None, **kw) == B.MONARCH_ERR_NULL


def test_sandwich_gate_rows_of_no_rows():
    """rows == 0 zeroes dgate, whose rows are counted in workgroups: a count past a launch is refused, not cut."""
    none = dict(rows=0, h=None, y=None, ho=None, n=None, st=None)
    assert sandwich_fwd(**none, gates=1 << 21) == B.MONARCH_OK
    for gates in ((1 << 21) + 1, 1 << 31, 1 << 33):
        assert sandwich_fwd(**none, gates=gates) == B.MONARCH_ERR_SHAPE
        assert sandwich_bwd(rows=0, gates=gates) == B.MONARCH_ERR_SHAPE


def chunks(rows, d, gates, dtype=B.BF16):
    """Workgroups of the backward kernel: each leaves two partial rows of d."""
    return M.monarch_sandwich_bwd_workspace_bytes(rows, d, gates, False, dtype) // (2 * d * 4)


def test_few_gate_runs_are_cut():
    """Short gate runs are a team's own where there are enough of them; a few are cut over the chip as long ones are."""
    for dtype in (B.F32, B.BF16):
        for rows, d, gates in ((512, 768, 16), (64, 768, 2), (256, 16384, 8), (32 * 256, 768, 256), (128, 64, 4), (2048, 2048, 64), (16 * 16, 8192, 16)):
            # a row a team (at most 8 a workgroup), or a workgroup a CU
            assert chunks(rows, d, gates, dtype) >= min(rows // 8, 256), (rows, d, gates, dtype)
        # many: no partial rows of their own, at most as many chunks as a launch has workgroups
        for rows, d, gates in ((16384, 768, 2048), (32 * 4096, 768, 4096), (4096, 64, 2048), (4096, 16384, 512)):
            assert chunks(rows, d, gates, dtype) <= 512, (rows, d, gates, dtype)


def test_sandwich_stats():
    """Statistics of a row, and in bf16 behind them half a byte for each value of a joined and normed h_out."""
    from monarch_block_diagonal_amd import torch_api as T
    torch = pytest.importorskip("torch")
    for rows, d in ((1, 1), (6, 64), (1000, 767), (3, 16384), (1 << 20, 9), (0, 64)):
        for dtype, code in ((torch.float32, B.F32), (torch.bfloat16, B.BF16)):
            for y in (None, True):
                for pre in (0, 1, 2):
                    kept = (d + 7) // 8 if y and pre and code == B.BF16 else 0
                    need = M.monarch_sandwich_stats_bytes(rows, d, y is not None, pre, code)
                    assert need == rows * (16 + 4 * kept)
                    shape, kind = T._sandwich_stats(rows, d, y, pre, dtype)
                    assert shape[0] * shape[1] * kind.itemsize == need
    for bad in ((-1, 64, 1, 1, B.F32), (6, 0, 1, 1, B.F32), (6, 16385, 1, 1, B.F32), (6, 64, 1, 3, B.F32), (6, 64, 1, 1, 2)):
        assert M.monarch_sandwich_stats_bytes(*bad) == 0
