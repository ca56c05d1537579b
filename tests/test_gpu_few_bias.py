"""moe_forward_few where the bias or a token holds infinities or NaN."""
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


@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0", "bf16"])
@pytest.mark.parametrize("layout", ["tiled", "rowmajor"])
def test_infinite_tokens_keep_to_their_rows(precision, layout):
    g = torch.Generator(DEV).manual_seed(1)
    n = lambda *s: (torch.randn(*s, generator=g, device=DEV) / s[-1] ** 0.5).bfloat16()
    layer = moe.MoELayer(n(24, 512), torch.zeros(24, device=DEV), n(25, 256, 512), n(25, 512, 128), top_k=4,
                         precision=precision, weight_layout=layout)
    x, gamma = torch.randn(9, 512, generator=g, device=DEV).bfloat16(), torch.ones(512, dtype=torch.bfloat16, device=DEV)
    y = x.clone()
    y[2, 5], y[4, 9], y[8] = float("inf"), float("nan"), float("-inf")
    keep = [0, 1, 3, 5, 6, 7]
    for call in (layer.forward_few, lambda t: layer.forward_few_prenorm(t, gamma)):
        want, got = call(x), call(y)
        assert torch.equal(got[keep], want[keep])
        assert not torch.isfinite(got[[2, 4, 8]]).any()
    assert layer.check_status(9) == 0
