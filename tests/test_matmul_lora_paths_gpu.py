"""moe_matmul_lora on the paths that a call reaches by its size: the first
product in several passes, row tiles one after another on a CTA pair, the
adapters' part added token by token, K split over clusters."""
import pytest
import torch

import mixture_experts_routed_sigmoid_b200 as moe
import serving_reference as ref

pytestmark = pytest.mark.gpu


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def make(m, n, k, rank, D, ids, seed=0):
    """ids: the adapter of each token, as a list or a function of the token."""
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + m + n + k + rank)
    ids = [ids(t) for t in range(m)] if callable(ids) else ids
    return {"x": normal(g, m, k), "W": normal(g, n, k, std=k ** -0.5), "A": normal(g, D, rank, k, std=k ** -0.5),
            "B": normal(g, D, n, rank, std=rank ** -0.5), "scales": torch.rand(D, generator=g, device="cuda") * 2 - 0.5,
            "ids": torch.tensor(ids, dtype=torch.int32, device="cuda")}


def call(c, **kw):
    return moe.moe_matmul_lora(c["x"], c["W"], c["ids"], c["A"], c["B"], c["scales"], **kw)


def check(c, got):
    y, bound = ref.lora(c["x"], c["W"], c["ids"], c["A"], c["B"], c["scales"], got.dtype == torch.bfloat16)
    off = (got.double() - y).abs()
    assert (off <= bound).all(), f"worst {(off / bound).max():.3g} of the bound"


@pytest.mark.parametrize("m, n, k, rank, D", [
    (2600, 300, 1000, 8, 40),     # five passes of four adapters to each of two adapter lanes, K over four CTAs
    (2600, 300, 1000, 24, 21),    # a rank that is no multiple of 16
    (150, 260, 4096, 24, 60),     # two passes of four adapters to each of nine lanes, K over eight CTAs
    (150, 260, 4096, 128, 30),    # passes of one adapter
])
def test_first_product_in_several_passes(m, n, k, rank, D):
    c = make(m, n, k, rank, D, lambda t: (t * 7) % (D + 1) - 1)
    check(c, call(c))
