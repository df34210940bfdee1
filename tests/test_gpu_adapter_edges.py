"""The adapter calls at the edges of what they accept: arguments that only some outputs need."""
import pytest

from test_gpu_adapter import Case, pm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_down_has_to_be_on_the_device_without_dx_too(pm):  # noqa: F811
    import torch
    c = Case(20, 2, 64, 64, 8)
    down, up, scale = c.weights()
    x, ids, dy, v = c.d("x"), c.d("ids"), c.d("dy"), torch.zeros(20, 8, device="cuda")
    with pytest.raises(pm.PmoeError, match="down is not"):
        pm.adapter_backward(dy, x, v, ids, down.cpu(), up, scale, need_dx=False)
    _, d_down, d_up = pm.adapter_backward(dy, x, v, ids, down, up, scale, need_dx=False)
    assert d_down.shape == down.shape and d_up.shape == up.shape
