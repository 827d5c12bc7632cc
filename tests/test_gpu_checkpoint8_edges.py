"""8-bit activation checkpoints where pre-activations are not finite."""
import pytest
import torch

import mixture_experts_layer_60_b200 as moe
from tests.test_gpu_checkpoint8 import _ffn, _save8, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("col", [0, 33, 100, 127, 300])
def test_save8_of_a_nan_is_its_whole_tile(col):
    """A NaN is the largest of its tile: the scale and every code are NaN, so no finite value of
    the tile comes back changed; the other tiles are what they were."""
    sizes, d, I = [40, 0, 65], 256, 256
    x, off, Wgu, _, _ = _ffn(sizes, d, I, 21)
    h, q, sc = _save8(x, off, Wgu)
    bad = Wgu.clone()
    bad[0, col] = float("nan")                     # one gate or up column of expert 0
    h2, q2, s2 = _save8(x, off, bad)
    tile = col // 128
    assert torch.isnan(s2[:40, tile]).all()
    assert torch.isnan(_values(q2)[:40, tile * 128:tile * 128 + 128]).all()
    keep = [t for t in range(2 * I // 128) if t != tile]
    assert torch.equal(s2[:40, keep], sc[:40, keep]) and torch.equal(s2[40:], sc[40:])
    mask = torch.ones(2 * I, dtype=torch.bool, device="cuda")
    mask[tile * 128:tile * 128 + 128] = False
    assert torch.equal(q2[:40][:, mask], q[:40][:, mask]) and torch.equal(q2[40:], q[40:])


def test_save8_of_an_infinity():
    """An infinite pre-activation takes its tile's scale with it: finite values are 0 of it."""
    x, off, Wgu, _, _ = _ffn([50], 256, 256, 22)
    Wgu = Wgu.clone()
    Wgu[0, 5] = 0
    Wgu[0, 5, 0] = float("inf")
    x = x.clone()
    x[:, 0] = 1
    _, q, sc = _save8(x, off, Wgu)
    v = _values(q)
    assert torch.isinf(sc[:, 0]).all() and torch.isfinite(sc[:, 1:]).all()
    assert torch.isnan(v[:, 5]).all()
    rest = [c for c in range(128) if c != 5]
    assert (v[:, rest] == 0).all()
