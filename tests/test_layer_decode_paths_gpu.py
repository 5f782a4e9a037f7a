"""moe_layer_decode on the paths that a call reaches by its size: router blocks
of each form, several rounds of tiles."""
import pytest
import torch

import mixture_experts_routed_sigmoid_b200 as moe
import serving_reference as ref

pytestmark = pytest.mark.gpu


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def make(m, hidden, inter, E, top_k, inter_sh=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + m + hidden + inter + E)
    c = {"x": normal(g, m, hidden), "W_router": normal(g, E, hidden, std=hidden ** -0.5),
         "bias": (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.2, "top_k": top_k,
         "W_gate": normal(g, E, inter, hidden, std=hidden ** -0.5), "W_up": normal(g, E, inter, hidden, std=hidden ** -0.5),
         "W_down": normal(g, E, hidden, inter, std=inter ** -0.5), "shared": ()}
    if inter_sh:
        c["shared"] = (normal(g, hidden, std=hidden ** -0.5), normal(g, inter_sh, hidden, std=hidden ** -0.5),
                       normal(g, inter_sh, hidden, std=hidden ** -0.5), normal(g, hidden, inter_sh, std=inter_sh ** -0.5))
    return c


def call(c, **out):
    return moe.moe_layer_decode(c["x"], c["W_router"], c["bias"], c["top_k"], c["W_gate"], c["W_up"], c["W_down"],
                                *c["shared"], **out)


@pytest.mark.parametrize("hidden", [1000, 8192])
def test_logits_have_the_same_bits_in_every_batch(hidden):
    """The f64 additions of a logit keep their order: products over 120 powers of
    two whose exact sum is zero leave only the roundings, which show any other."""
    g = torch.Generator(device="cuda").manual_seed(hidden)
    c = make(32, hidden, 8, 30, 2, inter_sh=8, seed=1)
    half = hidden // 2
    c["W_router"] = c["W_router"] * 2.0 ** torch.randint(-30, 31, (hidden,), generator=g, device="cuda")
    c["x"] = c["x"] * 2.0 ** torch.randint(-30, 31, (hidden,), generator=g, device="cuda")
    order = torch.randperm(hidden, generator=g, device="cuda")
    near, far = order[:half], order[half:]
    c["x"][:, far] = c["x"][:, near]
    c["W_router"][:, far] = -c["W_router"][:, near]
    c = {k: v.bfloat16() if k in ("x", "W_router") else v for k, v in c.items()}
    whole = call(c)[3]
    for m in (1, 4, 5, 8, 9, 16, 17):
        part = call(dict(c, x=c["x"][:m].contiguous()))[3]
        assert torch.equal(part, whole[:m])
