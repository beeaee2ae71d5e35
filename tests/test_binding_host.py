"""The binding's own refusals of tensors without values."""
import types

import pytest
import torch


@pytest.fixture(scope="module")
def ic():
    from cross_layer_top_b200 import build
    build.build()
    from cross_layer_top_b200 import indexcache
    return indexcache


@pytest.mark.parametrize("shape", [(4, 0, 64), (4, 2, 0), (0, 0, 64)])
@pytest.mark.parametrize("listed", [list, tuple])
def test_heads_without_values(ic, shape, listed):
    ctx = types.SimpleNamespace(handle=None, device=-1)
    x = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no values"):
        ic.ic_qk_norm_rope(ctx, listed([dict(x=x, out=torch.zeros_like(x))]))
