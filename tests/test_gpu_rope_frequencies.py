"""Rotary frequencies at the ends of their range: radians a position by the thousands of millions and by nearly none."""
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_rope import DEV, DT, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dt", list(DT))
def test_frequencies_of_any_size(dt, interleaved):
    """Exact modulo a turn below 2^64; from there on, where no two positions can be told apart, a pair stays as it is."""
    pk = require_gpu()
    below = [3.0, -1e6, 2.0 ** 40, 1.2345e15, 2.0 ** 53 + 2, 9e17, 2.0 ** 63, 2.0 ** 64 - 2048, 1e-30, -2.0 ** -70, 0.0, 5e-324]
    past = [2.0 ** 64, 3e19, -2.0 ** 70, 1e25, 1e30, 2.0 ** 115, 2.0 ** 116, 1e300, -1.7e308]
    inv = torch.tensor(below + past, dtype=torch.float64)
    pos = [0, 1, 2, 1000, -77, 2 ** 30 + 1]
    x = torch.randn(len(pos), 3, 2 * len(inv) + 6, generator=torch.Generator().manual_seed(1)).to(DT[dt]).to(DEV)
    got, _ = pk.rope(x, None, torch.tensor(pos, device=DEV), inv.to(DEV), interleaved=interleaved)
    close(got, x, pos, below + [0.0] * len(past), interleaved, 1.0)
