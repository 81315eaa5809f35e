"""Host-side checks of the head loss's and dropout's C entries: bad arguments are
rejected before any HIP call, in the documented order."""
import pytest

import monarch_block_diagonal_amd as M
from monarch_block_diagonal_amd import binding as B

A, A2 = 0x10000, 0x20000     # fake 16-byte aligned device addresses (never dereferenced)
KINDS = ("fwd", "bwd", "step")


def head(kind, x=A, ldx=64, w=A, lab=A, t=A, ids=A, per=A, loss=A2, st=A2, dx=A2, dw=A2, ws=A2, wsb=1 << 40, rows=4, d=64,
         vocab=100, top=8, T=2.0, mix=0.5, dt=B.F32):
    lib = M.load_library()
    tail = (ws, wsb, rows, d, vocab, top, T, mix, dt, None, None, 0)
    if kind == "fwd":
        return lib.monarch_head_fwd(x, ldx, w, lab, t, ids, loss, st, *tail)
    if kind == "bwd":
        return lib.monarch_head_bwd(per, x, ldx, w, lab, t, ids, st, dx, dw, *tail)
    return lib.monarch_head_step(x, ldx, w, lab, t, ids, per, loss, dx, dw, *tail)


@pytest.mark.parametrize("kind", KINDS)
def test_head_sizes_and_values(kind):
    for dt in (-1, 2):
        assert head(kind, dt=dt) == B.MONARCH_ERR_DTYPE
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=(1 << 20) + 1, ldx=1 << 21), dict(vocab=0),
               dict(vocab=(1 << 30) + 1), dict(ldx=63), dict(top=-1), dict(top=513)):
        assert head(kind, **kw) == B.MONARCH_ERR_SHAPE, kw
    for kw in (dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=1e7), dict(T=1e-7), dict(mix=-0.5), dict(mix=1.1),
               dict(mix=float("nan"))):
        assert head(kind, **kw) == B.MONARCH_ERR_VALUE, kw


def test_head_null_and_align():
    for kind, names in (("fwd", ("x", "w", "t", "ids", "loss", "st", "ws")), ("bwd", ("x", "w", "t", "ids", "per", "st", "dx", "dw", "ws")),
                        ("step", ("x", "w", "t", "ids", "loss", "dx", "dw", "ws"))):
        for name in names:
            assert head(kind, **{name: None}) == B.MONARCH_ERR_NULL, (kind, name)
    # x is aligned to its elements only
    assert head("fwd", x=A + 2) == B.MONARCH_ERR_ALIGN
    assert head("fwd", x=A + 1, dt=B.BF16) == B.MONARCH_ERR_ALIGN
    for name, by in (("w", 8), ("t", 2), ("ids", 4), ("lab", 4), ("loss", 2), ("st", 8), ("ws", 8)):
        assert head("fwd", **{name: A + by}) == B.MONARCH_ERR_ALIGN, name
    for name, by in (("dx", 8), ("dw", 8), ("per", 2)):
        assert head("step", **{name: A + by}) == B.MONARCH_ERR_ALIGN, name


def test_head_workspace():
    for k, kind in enumerate(KINDS):
        need = M.monarch_head_workspace_bytes(k, 4, 64, 100, 8, B.F32)
        assert need > 0 and head(kind, wsb=need - 256) == B.MONARCH_ERR_WORKSPACE
        assert M.monarch_head_workspace_bytes(k, 0, 64, 100, 8, B.F32) == 0
        for bad in ((-1, 64, 100, 8, B.F32), (4, 0, 100, 8, B.F32), (4, 64, 0, 8, B.F32), (4, 64, 100, 513, B.F32), (4, 64, 100, 8, 2)):
            assert M.monarch_head_workspace_bytes(k, *bad) == 0
    assert M.monarch_head_workspace_bytes(3, 4, 64, 100, 8, B.F32) == 0
    assert M.monarch_head_stats_bytes(5, 8) == 5 * 12 * 4 and M.monarch_head_stats_bytes(-1, 8) == 0
    # the gradient of the logits is held a piece at a time: at most 2 GiB of it and 1 GiB of each split sum, copies of
    # x, and a tile's sums of every 128 words at least
    for dt, es in ((B.BF16, 2), (B.F32, 4)):
        for rows, d, vocab in ((16384, 768, 50257), (4096, 4096, 131072), (65536, 1024, 131072), (8, 768, 50257), (1000, 625, 10000)):
            parts = 3 if es == 4 else 1
            np_, dp = (rows + 255) // 256 * 256, (d + 63) // 64 * 64
            copies = parts * (np_ + (vocab + 64 if es == 4 or d % 8 else 0)) * dp * 2
            sums = 3 * 4 * np_ * ((vocab + 127) // 128)
            assert M.monarch_head_workspace_bytes(B.HEAD_STEP, rows, d, vocab, 0, dt) <= copies + sums + (4 << 30) + np_ * dp * 4 + (np_ + rows) * 64


def test_head_no_rows():
    none = dict(rows=0, x=None, w=None, lab=None, t=None, ids=None, loss=None, st=None, ws=None, per=None)
    assert head("fwd", **none) == B.MONARCH_OK
    for kind in ("bwd", "step"):
        assert head(kind, **none, dx=None, dw=None) == B.MONARCH_ERR_NULL


def dropout(x=A, r=A, y=A2, n=100, p=0.5, seed=1, offset=2, state=None, dt=B.F32):
    return M.load_library().monarch_dropout(x, r, y, n, p, seed, offset, state, dt, None, None, 0)


def test_dropout_arguments():
    for dt in (-1, 2):
        assert dropout(dt=dt) == B.MONARCH_ERR_DTYPE
    for n in (-1, (1 << 41) + 1):
        assert dropout(n=n) == B.MONARCH_ERR_SHAPE
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert dropout(p=p) == B.MONARCH_ERR_VALUE
    for name in ("x", "y"):
        assert dropout(**{name: None}) == B.MONARCH_ERR_NULL
    for name in ("x", "r", "y"):
        assert dropout(**{name: A + 8}) == B.MONARCH_ERR_ALIGN
    assert dropout(state=A + 4) == B.MONARCH_ERR_ALIGN
    assert dropout(n=0, x=None, r=None, y=None) == B.MONARCH_OK


def test_tensor_calls_refuse():
    torch = pytest.importorskip("torch")
    from monarch_block_diagonal_amd import torch_api as T
    x = torch.zeros(4, 8)
    for seed in (-1, 1 << 64):
        with pytest.raises(ValueError):
            T._dropout_args(0.5, seed, 0, None, 0)
    with pytest.raises(ValueError):
        T._dropout_args(0.5, None, 0, None, 0)
    with pytest.raises(ValueError):
        T.Dropout(1.5)
    drop = T.Dropout(0.5).eval()
    assert torch.equal(drop(x + 1.0, x + 2.0), x + 3.0) and drop.calls == 0
