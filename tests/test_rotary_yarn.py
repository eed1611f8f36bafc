"""YaRN's frequencies against the formula written out, for original lengths short and long."""

import math

import pytest
import torch

from trainable_block_sparse_pooled_b200.rotary import rotary_frequencies


def yarn(rd, theta, factor, length, fast=32.0, slow=1.0):
    """Pair p stays below low, is divided by the factor from high on, and moves linearly in p between: low and high
    are the pairs that turn `fast` and `slow` times over the length, rounded outwards, within 0 .. rd - 1."""
    pair = lambda turns: rd * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rd - 1)
    out = []
    for p in range(rd // 2):
        f = theta ** (-2 * p / rd)
        share = min(max((p - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append(f * (1 - share) + f / factor * share)
    return out


@pytest.mark.parametrize("rd", [64, 128])
@pytest.mark.parametrize("theta,length", [(10000.0, 2048), (10000.0, 4096), (10000.0, 32768), (10000.0, 65536),
                                          (10000.0, 131072), (10000.0, 1048576), (1e6, 32768), (500.0, 8192)])
def test_yarn_follows_its_formula(rd, theta, length):
    for factor in (1.0, 4.0, 32.0):
        f, scale = rotary_frequencies(rd, theta=theta, scaling="yarn", factor=factor, original_length=length)
        assert f.tolist() == pytest.approx(yarn(rd, theta, factor, length), rel=1e-12)
        assert scale == pytest.approx(0.1 * math.log(factor) + 1.0)


def test_pairs_that_turn_more_often_are_not_divided_in_full():
    """Over 131072 positions the slowest of 64 pairs turns 2.4 times: between once and 32 times."""
    f, _ = rotary_frequencies(128)
    g, _ = rotary_frequencies(128, scaling="yarn", factor=4.0, original_length=131072)
    turns = 131072 * f / (2 * math.pi)
    assert turns.min() > 1 and ((g > f / 4) | (turns <= 1)).all()
    assert torch.equal(g[turns > 40], f[turns > 40])
