"""A word whose logit is -inf: in bf16 the loss is that without the word; fp32's three parts turn infinity times
zero up, and the logits are NaN, which comes out."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from oracle import head as H  # noqa: E402
from test_head_gpu import U, api, draw, near  # noqa: E402,F401


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,d,vocab", [(5, 64, 500), (40, 40, 300), (300, 72, 4000)])
def test_a_word_at_minus_infinity(api, rows, d, vocab, dtype):  # noqa: F811
    x, w, labels, _, _, _ = draw(rows, d, vocab, dtype, seed=61)
    x[:, 3] = 1.0
    labels = torch.where(labels == 17, 18, labels)
    rest = torch.cat((w[:17], w[18:]))
    w[17, 3] = float("-inf")
    loss, _ = api.head_loss_forward(x, w, labels)
    if dtype == torch.float32:
        assert torch.isnan(loss).all()
        return
    o = H.head(x, rest, labels - (labels > 17).long())
    near(loss, o.loss, H.bounds(o, x, rest, U[dtype])[0], "loss")
