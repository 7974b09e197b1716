"""dropout's seed and offset as whole numbers of other types than Python's."""
import numpy as np
import pytest
import torch

import glu_mlp_gemv_amd as glu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [np.int64, np.int32, np.uint8])
def test_numpy_seed_and_offset(kind):
    x = torch.randn(5, 33, device="cuda:0")
    want = glu.dropout(x, 0.5, 7, 3)
    assert torch.equal(glu.dropout(x, 0.5, kind(7), kind(3)), want)
    assert torch.equal(glu.dropout(x, 0.5, np.int64(-1)), glu.dropout(x, 0.5, -1))
    y = x.clone().requires_grad_()
    (g,) = torch.autograd.grad(glu.dropout(y, 0.5, kind(7), kind(3)).sum(), y)
    assert torch.equal(g, glu.dropout(torch.ones_like(x), 0.5, 7, 3))
