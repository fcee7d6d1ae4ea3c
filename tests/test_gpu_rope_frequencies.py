"""rope_append's angles for frequencies well above one radian a position, at far positions: against exact arithmetic."""
from fractions import Fraction

import pytest
import torch

from tests.test_gpu_rope import Case

pytestmark = pytest.mark.gpu
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Exact(Case):
    """The rotation by an angle whose whole turns are taken off exactly, in rational numbers."""

    def turned(self, x, w):
        assert w is None and not self.inter
        turns = [[Fraction(int(p)) * Fraction(float(f)) / (2 * PI) % 1 for f in self.inv_freq] for p in self.positions]
        t = torch.tensor([[float(2 * PI * f) for f in row] for row in turns], dtype=torch.float64)[:, None]
        c, s = t.cos(), t.sin()
        x = x.double()
        y, half = x.clone(), self.rot // 2
        a, b = x[..., :half], x[..., half:self.rot]
        y[..., :half], y[..., half:self.rot] = a * c - b * s, b * c + a * s
        return y


@pytest.mark.parametrize("far", [1000, 131071, 10 ** 6, 2 ** 30 + 3, 2 ** 31 - 10, -77, -2 ** 31 + 10])
@pytest.mark.parametrize("low,high", [(-9, 0), (0, 3), (3, 6), (6, 12)])
def test_large_frequencies_at_far_positions(low, high, far):
    """Frequencies of 10^low to 10^high, some negative; the tolerances of Case.check()."""
    c = Exact([7], [0], 4, 2, seed=3, dtype="f16")
    c.positions = (torch.arange(7, dtype=torch.int64) + far).to(torch.int32)
    c.inv_freq = torch.logspace(low, high, 64, dtype=torch.float64).float()
    c.inv_freq[::7] *= -1
    c.check(c.run())
