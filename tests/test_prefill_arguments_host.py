"""What Decoder.prefill refuses, before any kernel and without a change of the
decoder; a stack of no layers needs no GPU."""
import pytest
import torch

import bit_ternary_weight_b200 as bl
from bit_ternary_weight_b200.decoder import Decoder, DecoderConfig

BF16 = torch.bfloat16


def _decoder():
    cfg = DecoderConfig(hidden=64, layers=0, max_seq=8)
    return Decoder(cfg, [], torch.full((64,), 5.0, dtype=BF16), torch.tensor([3], dtype=torch.int32))


@pytest.mark.parametrize("x,start,status", [
    (torch.zeros(4, 64), 0, bl.BL_ERR_DTYPE), (torch.zeros(4, 64, dtype=torch.float16), 0, bl.BL_ERR_DTYPE),
    (torch.zeros((), dtype=BF16), 0, bl.BL_ERR_SHAPE), (torch.zeros(64, dtype=BF16), 0, bl.BL_ERR_SHAPE),
    (torch.zeros(1, 4, 64, dtype=BF16), 0, bl.BL_ERR_SHAPE), (torch.zeros(0, 64, dtype=BF16), 0, bl.BL_ERR_SHAPE),
    (torch.zeros(4, 65, dtype=BF16), 0, bl.BL_ERR_SHAPE), (torch.zeros(4, 64, dtype=BF16), 5, bl.BL_ERR_SHAPE),
    (torch.zeros(4, 64, dtype=BF16), -1, bl.BL_ERR_SHAPE)])
def test_refusals(x, start, status):
    d = _decoder()
    with pytest.raises(bl.BitLinearError) as e:
        d.prefill(x, start)
    assert e.value.status == status
    assert d.pos.item() == 3 and (d.h == 5.0).all()


def test_a_prompt_up_to_the_last_row():
    d, x = _decoder(), torch.arange(4 * 64).view(4, 64).to(BF16)
    assert torch.equal(d.prefill(x, 4), x)
    assert d.pos.item() == 8 and torch.equal(d.h, x[-1])


def test_streams_that_require_gradients_leave_no_graph_behind():
    """An embedding's output, for example: nothing of its graph is kept."""
    d, x = _decoder(), torch.ones(4, 64, dtype=BF16).requires_grad_()
    y = d.prefill(x * 2)
    assert not y.requires_grad and not d.h.requires_grad and d.h.grad_fn is None
    assert torch.equal(d.h, torch.full((64,), 2.0, dtype=BF16))
