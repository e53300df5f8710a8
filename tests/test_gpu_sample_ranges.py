"""Draws from rows whose logits lie closer together than the quotient of a bucket's share of their
range holds in fp32."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import DEV, _built, cache, check  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def narrow(V):
    """Rows whose finite logits differ by less than 1.5e-36 in all."""
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.empty(7, V, device=DEV)
    x[0] = 1e-42
    x[0, V // 3] = 2e-42
    x[1] = 1e-37 * torch.rand(V, generator=g, device=DEV)
    x[2] = -1e-44 * torch.randint(1, 5, (V,), generator=g, device=DEV)
    x[3] = 1e-40 * torch.randn(V, generator=g, device=DEV)
    x[3, ::3] = -torch.inf
    x[4] = 0.0
    x[4, V - 1] = 1e-45
    x[5] = -1.4e-36 * torch.rand(V, generator=g, device=DEV)
    x[6] = 1e-38
    x[6, 1::2] = -1e-38
    return x


@pytest.mark.parametrize("kw", [dict(t=0.0), dict(k=1), dict(k=2), dict(k=40), dict(k=700),
                                dict(p=0.3), dict(p=0.0), dict(k=40, p=0.55, m=0.5), dict(m=0.9),
                                dict()], ids=str)
@pytest.mark.parametrize("V", [100, 500, 3000, 40000])
def test_narrow_rows(cache, V, kw):  # noqa: F811
    x = narrow(V)
    u = np.array([0.0, 0.2, 0.4, 0.55, 0.7, 0.9, 0.999], np.float32)
    check(cache, x, u, **{name: [v] * 7 for name, v in kw.items()})


@pytest.mark.parametrize("t", [1e-29, 1e-20, 1e-3])
def test_narrow_rows_at_low_temperatures(cache, t):  # noqa: F811
    """Where the temperature is as small as the rows' spread."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(6, 5000, generator=g, device=DEV) * t
    x[5] *= 1e-5
    u = np.array([0.1, 0.3, 0.5, 0.7, 0.9, 0.99], np.float32)
    check(cache, x, u, t=[t] * 6, k=[0, 40, 0, 1, 700, 0], p=[0.9, 1.0, 1.0, 0.5, 0.8, 0.2],
          m=[0.0, 0.1, 0.2, 0.0, 0.01, 0.0])
