"""The serving layer of latent attention: what its router is given."""
import pytest
import torch

from test_gpu_serve_latent import _layer, _lib, _set  # noqa: F401

pytestmark = pytest.mark.gpu


def test_the_router_gets_logits_of_32_bits(monkeypatch):
    """The choice of experts is exact on the logits it is given, so these are not rounded to 16 bits: they are the product of the
    layer's activations and router weights, summed in fp32 (|err| <= 2 H 2^-24 sum |y w|: the order of the sum is the library's)."""
    from bit_moe_expert_router_gb300 import binding
    layer = _layer()
    seen = {}
    route, experts = binding.moe_w4a8_route_scored, binding.moe_w4a8_forward_bf16_routed

    def see_route(logits, *args, **kw):
        seen["logits"] = logits.clone()
        return route(logits, *args, **kw)

    def see_experts(y, *args, **kw):
        seen["y"] = y.clone()
        return experts(y, *args, **kw)

    monkeypatch.setattr(binding, "moe_w4a8_route_scored", see_route)
    monkeypatch.setattr(binding, "moe_w4a8_forward_bf16_routed", see_experts)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(6)
    for q in ((20, 9), (1, 1)):
        _set(layer, q, (20 + q[0] % 20, 9 + q[1] % 9))
        layer.forward(torch.randn(sum(q), 256, generator=g, device="cuda:0").bfloat16(), max(q))
        y, w = seen["y"].double(), layer.w["router"].double()
        assert seen["logits"].dtype == torch.float32
        assert ((seen["logits"].double() - y @ w).abs() <= 2 * 256 * 2.0 ** -24 * (y.abs() @ w.abs())).all()
