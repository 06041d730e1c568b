"""The bound of ``prefill_layer`` is one that the mistakes a prompt's attention
can make do not meet."""
import numpy as np
import pytest

import prefill_layer as pl


@pytest.fixture(scope="module")
def layer():
    cfg = pl.config(512, 4, 2)
    return pl.Layer(cfg, pl.weights(cfg, 5), pl.prompt(cfg, 37, 11))


def test_the_bound_is_a_small_part_of_the_gain(layer):
    y, tol = layer.gain()
    part = tol / np.linalg.norm(y, axis=-1)
    assert part.max() < 0.2 and np.median(part) < 0.1
    # and the gain most of the stream
    assert (np.linalg.norm(y, axis=-1) > np.linalg.norm(layer.x, axis=-1)).all()


@pytest.mark.parametrize("mistake", pl.MISTAKES)
def test_mistakes_are_outside_the_bound(layer, mistake):
    y, tol = layer.gain()
    wrong, _ = layer.gain(mistake, cut=20)
    ratio = np.linalg.norm(wrong - y, axis=-1) / tol
    assert ratio.max() > 3 and (ratio > 1.5).sum() >= 4, (ratio.max(), ratio)
