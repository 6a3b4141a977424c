"""Rotary angles of far positions: 64 bits of the turns, so fp32's own error, for any frequency up to 1."""
import numpy as np
import pytest
import torch

from test_gpu_rope import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("low", [0.5, 0.999, 1e-6])
@pytest.mark.parametrize("sign", [1, -1])
def test_any_frequency_at_far_positions(fx, sign, low, layout):
    """pairs (0, 1) and (1, 0) become sine and cosine themselves. fp32's part: the remainder of the turns rounds by 2^-26
    of a turn (2^-23.3 rad) and sine and cosine by 2^-23 (one is multiplied by one, the other by zero: exact), together
    2.2e-7, below 2^-22: the angle's 64 bits may leave 2^-25 rad."""
    rng = np.random.default_rng(3)
    tokens, rot = 4096, 64
    freq = rng.uniform(low, min(2 * low, 1.0), rot // 2)
    pos = sign * (2 ** 31 - rng.integers(0, 1 << 20, tokens))
    x = np.zeros((tokens, 2, rot), np.float32)
    first = np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2)
    x[:, 0, first] = 1.0
    x[:, 1, first + (rot // 2 if layout == "half" else 1)] = 1.0
    want, size = reference(x, pos, freq, 0, layout, 1.0, False)
    got = fx.idx_rope(torch.from_numpy(x).cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), offset=0,
                      layout=layout)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -22 * size).all(), err.max()
