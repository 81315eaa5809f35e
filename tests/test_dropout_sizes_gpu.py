"""Dropout of tensors that take more than one launch (32 GiB each)."""
import numpy as np
import pytest

from oracle import dropout as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype,n", [(torch.float32, (1 << 33) + 4099), (torch.bfloat16, (1 << 34) + 4099)], ids=["f32", "bf16"])
def test_past_one_launch(dtype, n):
    """In place: the last element of the first launch, the first one of the second, and an end inside a piece."""
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import binding as B
    from monarch_block_diagonal_amd import torch_api as T
    x = torch.ones((n,), dtype=dtype, device="cuda")
    B.monarch_dropout(x, None, x, n, 0.5, 21, 3, None, T.dtype_code(x))
    per = (32 << 30) // x.element_size()
    for first in (0, per - 2000, n - 4000):
        want = O.draws(4000, 21, 3, first=first) >= 32768
        assert np.array_equal(x[first:first + 4000].float().cpu().numpy(), 2.0 * want)
    # every element was reached once: 0 or 2
    for at in range(0, n, 1 << 30):
        part = x[at:at + (1 << 30)]
        assert not (part == 1).any() and part.amax() == 2.0
    del x, part
    torch.cuda.empty_cache()
