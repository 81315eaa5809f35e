"""monarch_head_describe: the kernels of a call, by the rules that choose between them."""
import pytest

import monarch_block_diagonal_amd as M
from monarch_block_diagonal_amd import binding as B


def test_kernels_of_a_call():
    assert M.monarch_head_describe(B.HEAD_FWD, 8, 768, 50257, 0, B.BF16) == ["head_rows", "head_thin", "head_loss"]
    assert M.monarch_head_describe(B.HEAD_STEP, 8, 768, 50257, 4, B.BF16) == [
        "head_flag", "head_rows", "head_entries", "head_thin", "head_loss", "head_few", "head_taught", "head_products_32", "head_dx_out"]
    assert M.monarch_head_describe(B.HEAD_BWD, 8, 768, 50257, 0, B.F32) == [
        "head_rows", "head_copy_x", "head_factors", "head_thin_grad", "head_few_products", "head_dx_out"]
    assert M.monarch_head_describe(B.HEAD_STEP, 8, 6, 500, 0, B.F32)[:4] == ["head_rows", "head_copy_x", "head_copy_w", "head_sums_32"]
    assert M.monarch_head_describe(B.HEAD_STEP, 16384, 768, 50257, 0, B.BF16) == [
        "head_rows", "head_copy_x", "head_sums_256", "head_loss", "head_grad_256*2", "head_products_256*2", "head_dx_out"]
    assert M.monarch_head_describe(B.HEAD_STEP, 65536, 1024, 131072, 0, B.BF16)[4:6] == ["head_grad_256*17", "head_products_256*17"]


@pytest.mark.parametrize("dt", [B.F32, B.BF16])
def test_large_tiles_from_enough_work_on(dt):
    for rows, d, vocab in ((1024, 768, 50257), (4096, 4096, 131072), (8192, 768, 50257)):
        for call in (B.HEAD_FWD, B.HEAD_BWD, B.HEAD_STEP):
            tiles = [n.split("*")[0] for n in M.monarch_head_describe(call, rows, d, vocab, 0, dt) if n.startswith(("head_sums", "head_grad", "head_prod"))]
            assert tiles and all(n.endswith("_256") for n in tiles)
    assert "head_products_128" in M.monarch_head_describe(B.HEAD_STEP, 1000, 625, 10000, 0, dt)


def test_no_rows_and_refusals():
    assert M.monarch_head_describe(B.HEAD_FWD, 0, 8, 9, 0, B.F32) == []
    assert M.monarch_head_describe(B.HEAD_STEP, 0, 8, 9, 0, B.F32) == ["zero_dw"]
    for bad in ((3, 4, 8, 9, 0, B.F32), (-1, 4, 8, 9, 0, B.F32), (0, -1, 8, 9, 0, B.F32), (0, 4, 0, 9, 0, B.F32), (0, 4, 8, 9, 513, B.F32),
                (0, 4, 8, 9, 0, 2)):
        with pytest.raises(M.MonarchError):
            M.monarch_head_describe(*bad)


def test_memory():
    """A step takes less than the logits would in the call's own type, from 1 GiB of them on; few rows take what they have."""
    for rows, d, vocab in ((16384, 768, 50257), (4096, 4096, 131072), (65536, 1024, 131072)):
        assert M.monarch_head_workspace_bytes(B.HEAD_STEP, rows, d, vocab, 0, B.BF16) < 0.62 * rows * vocab * 2
    # two parts of g of 32 rows each in bf16, the logits, a copy of the rows and partial sums
    assert M.monarch_head_workspace_bytes(B.HEAD_STEP, 8, 768, 50257, 0, B.BF16) < (64 * 2 + 32 * 4) * 50688 + (32 << 20)
