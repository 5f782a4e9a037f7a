"""moe_matmul_lora (a shared projection with the low-rank adapter of each
token's request) against its plain 64-bit form, within derived bounds."""
import pytest
import torch

import mixture_experts_routed_sigmoid_b200 as moe
import moe_inputs
import serving_reference as ref
from helpers import GUARD

pytestmark = pytest.mark.gpu

# m, k, n, rank, adapters
SHAPES = [
    (1, 8, 1, 8, 1),               # the smallest sizes
    (1, 4096, 4096, 16, 8),
    (1, 2048, 300, 128, 3),        # the largest rank; K split over blocks
    (2, 72, 33, 8, 2),
    (7, 1000, 1001, 24, 5),
    (8, 512, 256, 16, 64),
    (9, 264, 4736, 40, 4),         # 32 columns per SM
    (20, 520, 5000, 16, 20),       # more than one tile per SM
    (32, 1024, 512, 64, 32),
    (32, 256, 513, 32, 64),        # the largest streamed batch
    (33, 136, 100, 16, 7),         # the smallest batch on tcgen05
    (65, 256, 513, 32, 64),
    (100, 4096, 512, 16, 10),      # K of one tile over a cluster of four CTA pairs
    (260, 2048, 2300, 16, 5),      # over two
    (128, 64, 256, 8, 3),
    (201, 1000, 1501, 24, 40),
    (300, 2048, 130, 128, 2),
    (513, 72, 70, 88, 9),
    (1500, 512, 768, 16, 12),
]


def make(m, k, n, rank, D, seed=0, mode="mixed"):
    g = moe_inputs.generator(seed)
    b = lambda *s, std=1.0: moe_inputs.bf16_normal(s, std, g)  # noqa: E731
    c = {"x": b(m, k), "W": b(n, k, std=k ** -0.5), "A": b(D, rank, k, std=k ** -0.5),
         "B": b(D, n, rank, std=rank ** -0.5), "scales": torch.rand(D, generator=g) * 2 - 0.5}
    if mode == "mixed":            # any order, any repetition, some without an adapter
        ids = torch.randint(-1, D, (m,), generator=g)
    elif mode == "runs":           # runs of ragged lengths
        cuts = torch.randint(0, 5, (m,), generator=g) == 0
        ids = torch.randint(-1, D, (m,), generator=g)[cuts.long().cumsum(0).clamp(max=m - 1)]
    elif mode == "none":
        ids = torch.full((m,), -1)
    else:                          # all tokens on the last adapter
        ids = torch.full((m,), D - 1)
    c["ids"] = ids.to(torch.int32)
    return c


def call(c, **kw):
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in c.items()}
    return moe.moe_matmul_lora(d["x"], d["W"], d["ids"], d["A"], d["B"], d["scales"], **kw)


def check(c, got):
    y, bound = ref.lora(c["x"], c["W"], c["ids"], c["A"], c["B"], c["scales"], got.dtype == torch.bfloat16)
    off = (got.cpu().double() - y).abs()
    assert (off <= bound).all(), f"worst {(off / bound).max():.3g} of the bound"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_matches_the_plain_form(shape, dtype):
    c = make(*shape, seed=sum(shape))
    m, n = shape[0], shape[2]
    buf = torch.full((m * n + GUARD,), -7777.0, dtype=dtype, device="cuda")
    y = buf[:m * n].view(m, n)
    got = call(c, y=y)
    torch.cuda.synchronize()
    assert got is y and (buf[m * n:] == -7777.0).all()
    check(c, y)


@pytest.mark.parametrize("m", [5, 40, 150, 700])
@pytest.mark.parametrize("mode", ["runs", "none", "one"])
def test_orders_of_adapters(m, mode):
    c = make(m, 320, 200, 16, 6, seed=m, mode=mode)
    check(c, call(c))


@pytest.mark.parametrize("m", [6, 150])
def test_without_scales(m):
    c = make(m, 320, 200, 16, 6, seed=m + 1)
    c["scales"] = None
    check(c, call(c))


@pytest.mark.parametrize("m", [12, 64, 140, 600])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_broken_adapter_reaches_its_own_requests_only(m, bad):
    """NaN or infinities in one adapter's A or B, in a row of x, or in an
    unused adapter leave every other row's bits as they were."""
    c = make(m, 192, 136, 16, 5, seed=m)
    c["ids"][:2] = torch.tensor([1, 2])
    want = call(c).cpu()
    for part in ("A", "B"):
        d = dict(c, **{part: c[part].clone()})
        d[part][1] = bad
        got = call(d).cpu()
        others = c["ids"] != 1
        assert torch.equal(got[others], want[others])
        assert not torch.isfinite(got[~others]).any()
    d = dict(c, B=c["B"].clone())
    d["B"][1, 7] = bad              # one output column of one adapter
    got = call(d).cpu()
    hit = c["ids"] == 1
    assert not torch.isfinite(got[hit][:, 7]).any()
    got[hit, 7] = want[hit, 7]
    assert torch.equal(got, want)
    d = dict(c, x=c["x"].clone())
    d["x"][3] = bad
    got = call(d).cpu()
    assert not torch.isfinite(got[3]).any()
    others = torch.arange(m) != 3
    assert torch.equal(got[others], want[others])


@pytest.mark.parametrize("m", [1, 30, 100, 400])
def test_repeats_give_the_same_bits_and_the_workspace_needs_no_reset(m):
    c = make(m, 2304, 300, 48, 9, seed=m)
    ws = torch.full((moe.moe_matmul_lora_workspace(m, 300, 2304, 48, 9),), 0xFF, dtype=torch.uint8, device="cuda")
    first = call(c, ws=ws).clone()
    assert moe.moe_check_status(ws) == 0
    for _ in range(3):
        assert torch.equal(call(c, ws=ws), first)


@pytest.mark.parametrize("m", [3, 64, 100, 2000])
@pytest.mark.parametrize("bad", [-2, 6, 2 ** 31 - 1, -2 ** 31])
def test_a_bad_id_is_reported_and_nothing_is_written(m, bad):
    c = make(m, 128, 72, 16, 6, seed=m)
    ws = torch.empty(moe.moe_matmul_lora_workspace(m, 72, 128, 16, 6), dtype=torch.uint8, device="cuda")
    good = c["ids"][m - 1].item()
    c["ids"][m - 1] = bad
    y = torch.full((m, 72), 5.0, device="cuda")
    call(c, y=y, ws=ws)
    assert moe.load_library().moe_check_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 6
    assert (y == 5.0).all()
    c["ids"][m - 1] = good          # the next call on the same workspace is a good one
    check(c, call(c, y=y, ws=ws))
    assert moe.moe_check_status(ws) == 0


@pytest.mark.parametrize("m", [6, 130])
def test_replays_from_a_graph_with_new_ids(m):
    c = make(m, 512, 384, 16, 8, seed=m)
    dev = {k: v.cuda() for k, v in c.items()}
    y = torch.empty((m, 384), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_matmul_lora_workspace(m, 384, 512, 16, 8), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_matmul_lora(dev["x"], dev["W"], dev["ids"], dev["A"], dev["B"], dev["scales"], y=y, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        new = make(m, 512, 384, 16, 8, seed=100 * m + seed)
        for k in ("x", "ids"):
            c[k] = new[k]
            dev[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        check(c, y)
    del graph


def test_two_streams_with_workspaces_of_their_own():
    cases = [make(m, 1024, 1000, 32, 8, seed=m) for m in (24, 300)]
    want = [call(c).clone() for c in cases]
    dev = [{k: v.cuda() for k, v in c.items()} for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = dev[i]
                got[i] = moe.moe_matmul_lora(d["x"], d["W"], d["ids"], d["A"], d["B"], d["scales"])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w, g)


@pytest.mark.parametrize("m, n", [(300, 512), (2100, 4096)])
def test_long_sums_in_f32(m, n):
    """An f32 output does not lose more with a longer K: the tensor core truncates its sums, so they
    are taken from it every 768 columns.  48 instructions of at most 2^-23 each to a partial sum,
    whose errors are independent of the next ones', then k / 768 roundings of 2^-24."""
    k = 16384
    g = torch.Generator(device="cuda").manual_seed(5)
    x, W = (torch.randn(r, k, device="cuda", generator=g).bfloat16() for r in (m, n))
    A, B = torch.zeros(1, 8, k, device="cuda").bfloat16(), torch.zeros(1, n, 8, device="cuda").bfloat16()
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    y = moe.moe_matmul_lora(x, W, ids, A, B, None, out_dtype=torch.float32).double()
    want = x.double() @ W.double().T
    off = ((y - want).norm() / want.norm()).item()
    assert off <= (48 * 2 + k // 768) * ref.U


def test_empty_batch():
    c = make(1, 64, 40, 8, 2)
    c["x"], c["ids"] = c["x"][:0].contiguous(), c["ids"][:0].contiguous()
    assert call(c).shape == (0, 40)


def test_decode_step_projection_then_layer():
    """The two operators as a decode step uses them: the bf16 output of the
    projection with adapters is the layer's input."""
    m, hidden, inter, E, top_k = 10, 512, 256, 16, 4
    c = make(m, 640, hidden, 16, 6, seed=21)
    h = call(c, out_dtype=torch.bfloat16)
    check(c, h)
    g = moe_inputs.generator(22)
    n = lambda *s, std: moe_inputs.bf16_normal(s, std, g)  # noqa: E731
    Wr, Wg, Wu, Wd = (n(E, hidden, std=0.05), n(E, inter, hidden, std=0.05), n(E, inter, hidden, std=0.05),
                      n(E, hidden, inter, std=0.05))
    y, ids, w, logits = moe.moe_layer_decode(h, Wr.cuda(), None, top_k, Wg.cuda(), Wu.cuda(), Wd.cuda())
    want, bound, wids, _, _ = ref.layer(h.cpu(), Wr, None, top_k, Wg, Wu, Wd)
    assert torch.equal(ids.cpu().long(), wids)
    assert ((y.cpu().double() - want).abs() <= bound).all()
