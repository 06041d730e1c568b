"""A prompt through the decoder stack at once, against the same tokens stepped
one by one.

The keys and values of the first layer depend on the tokens alone, and every
kernel on their way (RMSNorm + quantisation, products, rotation) gives the bits
of the one-token kernels, so these cache rows are equal, and so is everything
that a further step() of a one-layer stack computes.  What the attention
returns differs in rounding (2^-8 relative); the int8 quantiser behind it turns
that into a step of 1/127 of the token's maximum where a value crosses a
rounding border: with maxima of four to five standard deviations a step is 3 to
4 % of one, one value in ten crosses (2^-8 against 2^-5), so about 1 % of the
output product's size in the mean, and the squared-ReLU block behind it at most
multiplies by four (a square times a linear factor, and its own quantiser): a
relative 2-norm of 0.1 of the streams holds with room and is missed by any wrong
row, mask or position.
"""
import pytest
import torch

import synth_inputs as si
from parity_helpers import dev
from test_decoder_gpu import _layers_cpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_ternary_weight_b200 as b
    return b


def _stepped(dec, x, start=0):
    dec.set_position(start)
    out = []
    for t in range(x.shape[0]):
        dec.h.copy_(x[t])
        dec.step()
        out.append(dec.h.clone())
    return torch.stack(out)


@pytest.mark.parametrize("cuts", [[37], [1], [20, 17], [5, 1, 31]])
def test_prefill_leaves_the_caches_of_the_steps(bl, cuts):
    from bit_ternary_weight_b200.decoder import Decoder, DecoderConfig
    cfg = DecoderConfig(layers=1, max_seq=64)
    w = _layers_cpu(1, cfg, seed=5)
    a, b = Decoder.from_weights(cfg, w, device=dev()), Decoder.from_weights(cfg, w, device=dev())
    T = sum(cuts)
    x = si.activations(T + 1, cfg.hidden, seed=11).to(dev())
    want = _stepped(a, x[:T])
    got, at = [], 0
    for n in cuts:
        got.append(b.prefill(x[at:at + n], at))
        at += n
    got = torch.cat(got)
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0
    assert int(b.pos.item()) == T == int(a.pos.item()) and torch.equal(b.h, got[-1])
    for ca, cb in ((a.layers[0].cache_k, b.layers[0].cache_k), (a.layers[0].cache_v, b.layers[0].cache_v)):
        assert torch.equal(ca, cb)
    diff = (got.double() - want.double()).norm() / want.double().norm()
    assert diff <= 0.1, float(diff)
    # decoding goes on: the same token on equal caches
    for d in (a, b):
        d.h.copy_(x[T])
        d.step()
    assert torch.equal(a.h, b.h)


def test_prefill_of_two_layers_and_its_refusals(bl):
    from bit_ternary_weight_b200.decoder import Decoder, DecoderConfig
    cfg = DecoderConfig(layers=2, max_seq=48)
    w = _layers_cpu(2, cfg, seed=6)
    a, b = Decoder.from_weights(cfg, w, device=dev()), Decoder.from_weights(cfg, w, device=dev())
    x = si.activations(40, cfg.hidden, seed=12).to(dev())
    want, got = _stepped(a, x), b.prefill(x)
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0
    # two layers: the first one's difference enters the second once more
    diff = (got.double() - want.double()).norm() / want.double().norm()
    assert diff <= 0.2, float(diff)
    for bad, start in ((x, 9), (x[:, :-1], 0), (x[:0], 0), (x[:3], -1), (x[:3], 46)):
        with pytest.raises(bl.BitLinearError) as e:
            b.prefill(bad, start)
        assert e.value.status == bl.BL_ERR_SHAPE
