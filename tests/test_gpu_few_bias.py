"""moe_forward_few's selection where the bias holds infinities or NaN."""
import pytest
import torch

import sparse_moe_transformer_fwd_b200 as moe

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def _layer(E):
    g = torch.Generator(DEV).manual_seed(E)
    n = lambda *s: (torch.randn(*s, generator=g, device=DEV) / s[-1] ** 0.5).bfloat16()
    return moe.MoELayer(n(E, 512), torch.rand(E, generator=g, device=DEV) - 0.5, n(E + 1, 256, 512), n(E + 1, 512, 128), top_k=6), \
        torch.randn(7, 512, generator=g, device=DEV).bfloat16()


@pytest.mark.parametrize("E", [40, 300])
def test_infinite_bias_routes_as_the_layer(E):
    """Infinities are values like others: an expert that is always, or never, chosen."""
    layer, x = _layer(E)
    layer.bias[3], layer.bias[E - 1], layer.bias[7] = float("inf"), float("inf"), float("-inf")
    a, b = (torch.empty(7, 6, dtype=torch.int32, device=DEV) for _ in range(2))
    layer.forward_few(x, topk_idx_out=a)
    layer(x, topk_idx_out=b)
    assert torch.equal(a, b)
    assert (a[:, 0] == 3).all() and (a[:, 1] == E - 1).all() and not (a == 7).any()
    assert layer.check_status(7) == 0


@pytest.mark.parametrize("E", [6, 40, 300])
def test_nan_in_the_bias_still_chooses_different_experts(E):
    """Which ones is not specified; that they are experts, and different, is, and the
    gates are of the scores, so the output is finite."""
    layer, x = _layer(E)
    for at in (0, E - 1, 5):
        layer.bias[at] = float("nan")
        idx = torch.empty(7, 6, dtype=torch.int32, device=DEV)
        out = layer.forward_few(x, topk_idx_out=idx)
        assert all(len(set(r)) == 6 and 0 <= min(r) and max(r) < E for r in idx.tolist())
        assert torch.isfinite(out).all()
        assert torch.equal(layer.forward_few(x), out)
    assert layer._few_ws.status() == 0
