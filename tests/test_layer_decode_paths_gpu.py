"""moe_layer_decode on the paths that a call reaches by its size: router blocks
of each form, several rounds of tiles.

serving_reference.dot_gamma(k, parts) is 4 ceil(k / 1024) * 4 parts + 16 u (u =
2^-24) of the sum of magnitudes.  A warp sums units of 64 columns in 4 * parts
instructions of at most 4 u each, 16 parts u in all, and adds ceil(k / 64) of them,
u each.  With c = ceil(k / 64) that is 16 parts + c, and the bound is at least 16
parts ceil(c / 16) + 16: not below it for parts 1 and 3 at any c."""
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


def check(c, got):
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    y, bound, ids, w, logits = ref.layer(cpu(c["x"]), cpu(c["W_router"]), cpu(c["bias"]), c["top_k"], cpu(c["W_gate"]),
                                         cpu(c["W_up"]), cpu(c["W_down"]), tuple(map(cpu, c["shared"])) or None)
    gy, gids, gw, gl = map(cpu, got)
    # f64 sums rounded once: the exact sum's rounding but for ties, one step apart at most
    assert ((gl.double() - logits.double()).abs() <= 2 * ref.U * logits.double().abs() + ref.TINY).all()
    assert torch.equal(gids.long(), ids)
    assert ((gw.double() - w).abs() <= 2 * ref.U * w).all()
    off = (gy.double() - y).abs()
    assert (off <= bound).all(), f"worst {(off / bound).max():.3g} of the bound"


@pytest.mark.parametrize("m, hidden, inter, E, top_k, inter_sh", [
    (1, 136, 5000, 24, 16, 0),       # 16 x 5000 gate/up rows: more than 16 rows for each of 148 x 16 warps
    (1, 136, 5000, 24, 16, 5000),
    (8, 136, 5000, 24, 8, 0),
    (8, 136, 5000, 24, 8, 2504),
    (13, 136, 5000, 24, 8, 0),
    (13, 136, 5000, 24, 8, 2504),
    (13, 2056, 64, 24, 8, 0),        # and of down rows
    (13, 2056, 64, 24, 8, 64),
    (24, 2056, 64, 24, 8, 64),
    (8, 2056, 64, 32, 32, 64),       # more routed rows than the combining form holds
])
def test_several_rounds_of_tiles(m, hidden, inter, E, top_k, inter_sh):
    c = make(m, hidden, inter, E, top_k, inter_sh)
    check(c, call(c))
    # a row has its bits alone and in the batch
    part = call(dict(c, x=c["x"][m - 1:].contiguous()))
    for a, b in zip(call(c), part):
        assert torch.equal(a[m - 1:].view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("m", [2, 12])
def test_experts_past_32_bit_offsets(m):
    """Weights of more than 2^31 values each; the experts that no token chooses hold whatever was there."""
    hidden, inter, E = 2048, 1032, 1024
    assert E * inter * hidden > 2 ** 31
    used = [3, 700, 1020, 1023]
    small = make(m, hidden, inter, len(used), 3)
    c = dict(small, W_router=torch.zeros(E, hidden, device="cuda").bfloat16(), bias=torch.full((E,), -5.0, device="cuda"))
    c["W_router"][used], c["bias"][used] = small["W_router"], small["bias"]
    for name in ("W_gate", "W_up", "W_down"):
        c[name] = torch.empty((E, *small[name].shape[1:]), dtype=torch.bfloat16, device="cuda")
        c[name][used] = small[name]
    y, ids, w, logits = call(c)
    back = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    back[used] = torch.arange(len(used), dtype=torch.int32, device="cuda")
    check(small, (y, back[ids.long()], w, logits[:, used]))
