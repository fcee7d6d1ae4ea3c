"""rope_append into an FP8 cache: rows so small that 448 over their largest magnitude is beyond FP32 are rows of zeros."""
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_rope import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("size", [1e-34, 2e-36, 1e-37, 1e-38])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32)])
def test_tiny_rows(d, rot, size):
    """Zeros stay zeros, the others their values; a row up to 2^-119 becomes zeros. As Case.check(): half a step of e4m3 and
    the value's own error, here besides FP32's smallest step (2^-149): half of it in the scale, which up to 448 multiply, and
    a few in the rotation."""
    c = Case([9, 5], [3, 40], 4, 4, d=d, rot=rot, fp8=True, seed=d, dtype="bf16")
    g = torch.Generator().manual_seed(1)
    c.x = (c.x.double() * size * (torch.rand(c.x.shape, generator=g) < 0.7)).to(c.dt)
    _, cache, scales = c.run()
    page, off = (torch.tensor([w[i] for w in c.rows()], dtype=torch.long) for i in (0, 1))
    _, k, v = c.views(c.x)
    for kv, ref in ((0, c.turned(k, None)), (1, v.double())):
        s = scales[page, kv, :, off].double()
        value = cache[page, kv, :, off].view(torch.float8_e4m3fn).double() * s[..., None]
        top = ref.abs().amax(-1, keepdim=True)
        assert (value.isfinite()).all()
        assert (value[ref == 0] == 0).all()
        assert (s[(top <= 2.0 ** -120)[..., 0]] == 0).all() and (s[(top >= 2.0 ** -118)[..., 0]] > 0).all()
        tol = ref.abs() * 2.0 ** -4 * 1.001 + top / 448 * (2.0 ** -10 + 448 * 2.0 ** -19) + (224 + 8) * 2.0 ** -149
        assert ((value - ref).abs() <= torch.where(s[..., None] > 0, tol, 2.0 ** -119 * 1.001)).all()
    assert pkv.get_device_error() == 0
