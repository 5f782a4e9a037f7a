"""moe_layer_decode (the whole layer for a few tokens) against its plain
64-bit form, element by element within derived bounds."""
import pytest
import torch

import mixture_experts_routed_sigmoid_b200 as moe
import moe_inputs
import serving_reference as ref
from helpers import GUARD, POISON_BITS, poisoned_f32

pytestmark = pytest.mark.gpu

# m, hidden, inter, experts, top_k, inter_sh
SHAPES = [
    (1, 512, 256, 32, 8, 0),
    (1, 8, 8, 1, 1, 0),            # the smallest sizes; one expert
    (1, 16, 24, 2, 2, 8),
    (2, 64, 64, 4, 1, 0),          # top-1
    (3, 72, 40, 7, 3, 16),         # K tails inside a 64-column step
    (5, 1000, 520, 60, 6, 264),
    (7, 2048, 768, 16, 8, 768),    # more rows than experts
    (8, 128, 96, 1024, 32, 0),     # the limits of experts, top_k and routed rows
    (9, 264, 136, 24, 5, 0),       # just over one group of 8 tokens
    (16, 1024, 512, 12, 4, 128),
    (17, 320, 72, 9, 9, 40),       # every expert chosen by every token
    (32, 256, 128, 8, 8, 64),      # 32 tokens, each on all experts
    (32, 4104, 200, 40, 8, 0),     # hidden over 4096, not a multiple of 64
    (4, 9480, 64, 6, 2, 0),        # more than two 32-row passes per SM
    (31, 512, 2056, 100, 8, 72),
]


def make(m, hidden, inter, E, top_k, inter_sh, seed=0, with_bias=True):
    g = moe_inputs.generator(seed)
    n = lambda *s, std=1.0: moe_inputs.bf16_normal(s, std, g)  # noqa: E731
    c = {"x": n(m, hidden), "W_router": n(E, hidden, std=hidden ** -0.5),
         "bias": moe_inputs.uniform_bias(E, 0.1, g) if with_bias else None, "top_k": top_k,
         "W_gate": n(E, inter, hidden, std=hidden ** -0.5), "W_up": n(E, inter, hidden, std=hidden ** -0.5),
         "W_down": n(E, hidden, inter, std=inter ** -0.5)}
    sh = moe_inputs.shared_expert_inputs(hidden, inter_sh, seed) if inter_sh else None
    c["shared"] = (sh["w_sh"], sh["W_sh_gate"], sh["W_sh_up"], sh["W_sh_down"]) if sh else None
    return c


def call(c, **out):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    return moe.moe_layer_decode(d(c["x"]), d(c["W_router"]), d(c["bias"]), c["top_k"], d(c["W_gate"]),
                                d(c["W_up"]), d(c["W_down"]), *(d(t) for t in c["shared"] or ()), **out)


def check(c, got):
    y, bound, ids, w, logits = ref.layer(c["x"], c["W_router"], c["bias"], c["top_k"], c["W_gate"],
                                         c["W_up"], c["W_down"], c["shared"])
    gy, gids, gw, gl = (t.cpu() for t in got)
    # f64 sums rounded once: equal but for ties of the rounding, one ulp apart at most
    assert ((gl.double() - logits.double()).abs() <= 2 * ref.U * logits.double().abs() + ref.TINY).all()
    assert torch.equal(gids.long(), ids)
    assert ((gw.double() - w).abs() <= 2 * ref.U * w).all()
    off = (gy.double() - y).abs()
    assert (off <= bound).all(), f"worst {(off / bound).max():.3g} of the bound"


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_matches_the_plain_form(shape):
    c = make(*shape, seed=sum(shape))
    m, hidden = c["x"].shape
    buf, y = poisoned_f32((m, hidden))
    lbuf, logits = poisoned_f32((m, shape[3]))
    got = call(c, y=y, logits=logits)
    torch.cuda.synchronize()
    for b, n in ((buf, m * hidden), (lbuf, m * shape[3])):
        raw = b.view(torch.int32)
        assert not (raw[:n] == POISON_BITS).any() and (raw[n:] == POISON_BITS).all() and b.numel() == n + GUARD
    check(c, got)


def test_without_bias_and_with_crowded_experts():
    c = make(12, 256, 128, 64, 4, 0, seed=3, with_bias=False)
    check(c, call(c))
    c["bias"] = torch.zeros(64)
    c["bias"][[5, 9, 17, 40, 63]] = 2.0  # every token goes to four of five experts
    got = call(c)
    assert set(got[1].unique().tolist()) <= {5, 9, 17, 40, 63}
    check(c, got)


@pytest.mark.parametrize("m, crowd", [(10, 1), (16, 2), (24, 1), (25, 2), (32, 1), (32, 3)])
def test_crowded_experts_at_ragged_sizes(m, crowd):
    """All tokens on `crowd` experts (2 to 4 groups of 8 tokens each) and one of the others' choice."""
    c = make(m, 328, 200, 20, crowd + 1, 24, seed=40 + m + crowd)
    c["bias"][:crowd] = 2.0
    got = call(c)
    for e in range(crowd):
        assert ((got[1] == e).sum(1) == 1).all()
    check(c, got)


def test_a_row_has_the_same_bits_alone_and_in_a_crowd():
    c = make(32, 328, 200, 12, 3, 24, seed=50)
    whole = call(c)
    for m in (1, 5, 8, 9, 16, 17, 25):
        part = call(dict(c, x=c["x"][:m].contiguous()))
        for a, b in zip(whole, part):
            assert torch.equal(a[:m].view(torch.int32), b.view(torch.int32))


def test_equal_keys_take_the_lower_expert():
    c = make(6, 128, 64, 48, 5, 0, seed=4, with_bias=False)
    c["W_router"][:] = c["W_router"][0]       # all logits of a token are equal
    ids = call(c)[1].cpu()
    assert torch.equal(ids, torch.arange(5, dtype=torch.int32).expand(6, 5))
    c["x"][2] = 0
    check(c, call(c))


def test_rows_do_not_depend_on_each_other():
    """A row's bits stay when every other token changes (other experts active,
    other groups), also when another token holds NaN or infinities."""
    c = make(11, 328, 200, 30, 4, 24, seed=5)
    y0, ids0, w0, l0 = call(c)
    for fill in (None, float("nan"), float("inf")):
        d = dict(c, x=make(11, 328, 200, 30, 4, 24, seed=6)["x"].clone())
        d["x"][4] = c["x"][4]
        if fill is not None:
            d["x"][7] = fill
        y1, ids1, w1, l1 = call(d)
        for a, b in ((y0, y1), (ids0, ids1), (w0, w1), (l0, l1)):
            assert torch.equal(a[4].view(torch.int32), b[4].view(torch.int32))
        if fill is not None:
            assert torch.isnan(y1[7]).all()
            others = [t for t in range(11) if t != 7]
            assert torch.isfinite(y1[others]).all()


def test_infinite_weights_reach_their_own_tokens_only():
    c = make(6, 64, 64, 8, 2, 0, seed=8)
    ids = call(c)[1].cpu()
    e = ids[0, 0].item()
    c["W_down"][e, 3, 5] = float("inf")
    y = call(c)[0].cpu()
    hit = (ids == e).any(1)
    assert not torch.isfinite(y[hit][:, 3]).any()
    y[:, 3] = torch.where(hit, 0.0, y[:, 3])
    assert torch.isfinite(y).all()


def test_repeats_give_the_same_bits_and_the_workspace_needs_no_reset():
    c = make(10, 512, 256, 32, 8, 64, seed=9)
    ws = torch.full((moe.moe_layer_decode_workspace(10, 512, 256, 64, 8, 32),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    first = [t.clone() for t in call(c, ws=ws)]
    assert moe.moe_check_status(ws) == 0
    for _ in range(3):
        for a, b in zip(first, call(c, ws=ws)):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_agrees_with_the_calls_it_replaces():
    """moe_router_topk + moe_ffn_forward_shared on the same inputs: the same
    choice (no near ties in these inputs) and outputs within the bound."""
    c = make(8, 512, 256, 32, 4, 128, seed=10)
    y, ids, w, _ = call(c)
    x, d = c["x"].cuda(), lambda k: c[k].cuda()
    ids2, w2, _ = moe.moe_router_topk(x, d("W_router"), d("bias"), 4)
    assert torch.equal(ids, ids2)
    y2 = moe.moe_ffn_forward_shared(x, ids2, w2, d("W_gate"), d("W_up"), d("W_down"),
                                    *(t.cuda() for t in c["shared"]))
    bound = ref.layer(c["x"], c["W_router"], c["bias"], 4, c["W_gate"], c["W_up"], c["W_down"], c["shared"])[1]
    # both are within a bound of the exact value; the other one sums K in longer chains
    assert ((y - y2).abs().cpu().double() <= 8 * bound).all()


def test_replays_from_a_graph_with_new_inputs():
    c = make(4, 512, 256, 32, 8, 64, seed=11)
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in c.items() if k != "shared"}
    sh = [t.cuda() for t in c["shared"]]
    out = {"y": torch.empty((4, 512), device="cuda"), "ids": torch.empty((4, 8), dtype=torch.int32, device="cuda"),
           "weights": torch.empty((4, 8), device="cuda"), "logits": torch.empty((4, 32), device="cuda"),
           "ws": torch.empty(moe.moe_layer_decode_workspace(4, 512, 256, 64, 8, 32), dtype=torch.uint8, device="cuda")}

    def step():
        moe.moe_layer_decode(dev["x"], dev["W_router"], dev["bias"], 8, dev["W_gate"], dev["W_up"], dev["W_down"],
                             *sh, **out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (12, 13):
        c["x"] = make(4, 512, 256, 32, 8, 64, seed=seed)["x"]
        dev["x"].copy_(c["x"])
        graph.replay()
        torch.cuda.synchronize()
        check(c, (out["y"], out["ids"], out["weights"], out["logits"]))
    del graph


def test_two_streams_with_workspaces_of_their_own():
    cases = [make(8, 1024, 512, 64, 8, 0, seed=s) for s in (14, 15)]
    dev = [{k: v.cuda() for k, v in c.items() if torch.is_tensor(v)} for c in cases]
    want = [[t.clone() for t in call(c)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = dev[i]
                got[i] = moe.moe_layer_decode(d["x"], d["W_router"], d["bias"], 8, d["W_gate"], d["W_up"], d["W_down"])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_empty_batch():
    c = make(1, 64, 64, 8, 2, 0)
    c["x"] = c["x"][:0].contiguous()
    y, ids, w, logits = call(c)
    assert y.shape == (0, 64) and ids.shape == (0, 2) and w.shape == (0, 2) and logits.shape == (0, 8)
