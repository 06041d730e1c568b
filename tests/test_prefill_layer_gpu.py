"""Decoder.prefill's attention token by token against 64 bits, in a layer whose
stream is mostly what its attention adds; and a stack as the sequence of its
layers, bit for bit."""
import dataclasses

import numpy as np
import pytest
import torch

import prefill_layer as pl
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


def _check(layer, out):
    y, tol = layer.gain()
    off = np.linalg.norm(out.double().cpu().numpy() - layer.x - y, axis=-1)
    assert (off <= tol).all(), (off / tol).max()
    return (off / tol).max()


@pytest.mark.parametrize("hidden,heads,kv_heads", [(512, 4, 2), (2560, 20, 5)])
@pytest.mark.parametrize("cuts", [[37], [1, 36], [20, 17], [5, 1, 31], [36, 1], [1] * 37])
def test_gain_of_every_token(bl, hidden, heads, kv_heads, cuts):
    from bit_ternary_weight_b200.decoder import Decoder
    cfg = pl.config(hidden, heads, kv_heads)
    w, x = pl.weights(cfg, 5), pl.prompt(cfg, 37, 11)
    dec = Decoder.from_weights(cfg, [w], device=dev())
    got, at = [], 0
    for n in cuts:
        got.append(dec.prefill(x[at:at + n].to(dev()), at))
        at += n
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0
    _check(pl.Layer(cfg, w, x), torch.cat(got))


def test_gain_of_the_steps_and_of_a_piece_behind_steps(bl):
    """The bound holds for step() too, and for a piece behind its tokens."""
    from bit_ternary_weight_b200.decoder import Decoder
    cfg = pl.config(512, 4, 2)
    w, x = pl.weights(cfg, 6), pl.prompt(cfg, 80, 13)
    dec = Decoder.from_weights(cfg, [w], device=dev())
    got = []
    for t in range(9):
        dec.h.copy_(x[t])
        dec.step()
        got.append(dec.h.clone()[None])
    got.append(dec.prefill(x[9:].to(dev()), 9))
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0 and dec.pos.item() == 80
    _check(pl.Layer(cfg, w, x), torch.cat(got))


def test_a_stack_is_the_sequence_of_its_layers(bl):
    from bit_ternary_weight_b200.decoder import Decoder, DecoderConfig
    cfg = DecoderConfig(layers=3, max_seq=64)
    w = _layers_cpu(3, cfg, seed=8)
    stack = Decoder.from_weights(cfg, w, device=dev())
    one = dataclasses.replace(cfg, layers=1)
    layers = [Decoder.from_weights(one, [wl], device=dev()) for wl in w]
    x = si.activations(45, cfg.hidden, seed=14).to(dev())
    for at, end in ((0, 30), (30, 45)):
        h = x[at:end]
        got = stack.prefill(h, at)
        for d in layers:
            h = d.prefill(h, at)
        torch.cuda.synchronize()
        assert bl.last_device_status() == 0 and torch.equal(got, h)
    for L, d in zip(stack.layers, layers):
        assert torch.equal(L.cache_k, d.layers[0].cache_k) and torch.equal(L.cache_v, d.layers[0].cache_v)
