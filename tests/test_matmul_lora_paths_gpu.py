"""moe_matmul_lora on the paths that a call reaches by its size: the first
product in several passes, row tiles one after another on a CTA pair, the
adapters' part added token by token, K split over clusters.

serving_reference.lora's bound counts one chain of k / 16 instructions of at most
4 u (u = 2^-24) of the sum of magnitudes each, 16 u for what follows.  The kernels'
chains are shorter.  Above 32 tokens: 64 or 48 instructions to a partial sum (256 u
at most), whose k / 768 additions round by u each: below k / 4 u from k = 1024 on,
and one chain of k / 16 before; the parts of up to 4 CTA pairs (8 CTAs in the first
product) add by u each.  Up to 32: 4 instructions to a unit of 64 columns (16 u),
k / 64 additions, 16 warps."""
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


@pytest.mark.parametrize("m, n, D", [
    (20, 100, 5),                 # streamed
    (33, 100, 5), (200, 700, 3),  # joined tiles
    (200, 700, 120),              # joined, the adapters' part token by token
    (5000, 2100, 3),              # several tiles to a CTA pair
])
def test_an_f32_output_keeps_all_bits_of_the_first_product(m, n, D):
    """Whole numbers: A x has up to 21 bits, every sum of it is below 2^24, and a
    row of B picks one of its columns, so that y is A x exactly or has lost bits."""
    k, rank = 512, 16
    g = torch.Generator(device="cuda").manual_seed(m + D)
    whole = lambda top, *shape: torch.randint(-top, top + 1, shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, A = whole(255, m, k), whole(127, D, rank, k)
    B = torch.zeros(D, n, rank, device="cuda")
    B[:, torch.arange(n), torch.arange(n) % rank] = 1.0
    ids = (torch.arange(m, device="cuda") % (D + 1) - 1).int()
    scales = 2.0 ** torch.randint(-3, 4, (D,), generator=g, device="cuda")
    c = {"x": x, "W": torch.zeros(n, k, device="cuda").bfloat16(), "A": A, "B": B.bfloat16(), "ids": ids, "scales": scales}
    h = torch.einsum("tk,drk->tdr", x.double(), A.double())[torch.arange(m), ids.long().clamp(min=0)]
    assert 2 ** 18 < h.abs().max() < 2 ** 23
    want = torch.where(ids[:, None] >= 0, h[:, torch.arange(n) % rank] * scales.double()[ids.long().clamp(min=0), None], 0.0)
    assert torch.equal(call(c).double(), want)


@pytest.mark.parametrize("m, k", [(8, 2 ** 18), (200, 2 ** 20), (1100, 2 ** 18)])
def test_the_first_product_of_a_long_k(m, k):
    """The tensor core truncates: an instruction loses up to 2^-23 of its sum, 48
    of them (768 columns) at most 96 u of a partial sum, u = 2^-24.  The errors of
    the partial sums are independent: in the 2-norm 96 u of the whole, and their
    additions round, sqrt(k / 768) u of it.  (One sum of 32768 columns would be off
    by 4e-5.)  x and A are random, the projection is zero, B picks columns of A x."""
    n, rank, D = 48, 16, 2
    g = torch.Generator(device="cuda").manual_seed(m)
    c = {"x": normal(g, m, k), "W": torch.zeros(n, k, device="cuda").bfloat16(), "A": normal(g, D, rank, k, std=k ** -0.5),
         "ids": (torch.arange(m, device="cuda") % D).int(), "scales": None}
    B = torch.zeros(D, n, rank, device="cuda")
    B[:, torch.arange(n), torch.arange(n) % rank] = 1.0
    c["B"] = B.bfloat16()
    h = sum(torch.einsum("tk,drk->tdr", c["x"][:, i:i + 2 ** 16].double(), c["A"][:, :, i:i + 2 ** 16].double())
            for i in range(0, k, 2 ** 16))[torch.arange(m), c["ids"].long()]
    want = h[:, torch.arange(n) % rank]
    y = call(c).double()
    off = ((y - want).norm() / want.norm()).item()
    assert off <= (96 + (k / 768) ** 0.5) * ref.U, off
    # a bf16 output rounds by at most 2^-8 of its value, A x by 2^-17, and each of the k / 768
    # partial sums, about sqrt(768 / k) of x's size, loses at most 96 u
    y = call(c, out_dtype=torch.bfloat16).double()
    more = (y - want).abs() - (2.0 ** -8 + 2.0 ** -17) * want.abs()
    assert (more <= 96 * ref.U * (k / 768) ** 0.5 * c["x"].double().square().mean().sqrt()).all()


@pytest.mark.parametrize("m, n, k", [
    (20, 64, 2 ** 17),            # streamed
    (40, 64, 2 ** 18),            # K over four CTA pairs
    (2000, 2400, 2 ** 15),        # a tile or two to a CTA pair, each its whole K
])
def test_a_bf16_output_of_a_long_k_is_the_rounding_of_its_sum(m, n, k):
    """All products are positive, so that the tensor core's truncation (up to 2^-23
    = 2 u of the sum per instruction of 16 products) adds up: by 128 u of a partial
    sum of 1024 columns, and the k / 1024 additions of partial sums, which round,
    by u of the whole each.  What is left is the output's half step.  (A sum over
    all of K lost up to k / 8 u, 2^-9 at k = 2^18.)"""
    g = torch.Generator(device="cuda").manual_seed(m)
    c = {"x": normal(g, m, k).abs(), "W": normal(g, n, k, std=1 / k).abs(), "scales": None,
         "A": torch.zeros(1, 8, k, device="cuda").bfloat16(), "B": torch.zeros(1, n, 8, device="cuda").bfloat16(),
         "ids": torch.full((m,), -1, dtype=torch.int32, device="cuda")}
    want = sum(c["x"][:, i:i + 2 ** 13].double() @ c["W"][:, i:i + 2 ** 13].double().T for i in range(0, k, 2 ** 13))
    y = call(c, out_dtype=torch.bfloat16).double()
    step = 2.0 ** (torch.floor(torch.log2(want)) - 7)
    assert ((y - want).abs() <= step / 2 + (128 + k / 1024) * ref.U * want).all()


def varied_ids(m, D, seed):
    """Row tiles of 256 tokens without an adapter, with one, with a few in runs, with all."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.empty(m, dtype=torch.int64)
    for at in range(0, m, 256):
        n, kind = min(256, m - at), at // 256 % 4
        ids[at:at + n] = (torch.full((n,), -1) if kind == 0 else torch.full((n,), at % D) if kind == 1
                          else (torch.arange(n) // 50 + at) % D if kind == 2 else torch.randint(-1, D, (n,), generator=g))
    return ids.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m, n, k, rank, D", [
    (5000, 4100, 1000, 24, 7),    # 20 x 17 tiles of 256 x 256 or more of fewer columns
    (4700, 4100, 264, 128, 5),    # more columns of adapters than of k
    (9000, 2500, 72, 8, 40),
])
def test_row_tiles_one_after_another(m, n, k, rank, D, dtype):
    """Several tiles to each of the 74 CTA pairs, whose adapters differ in number:
    barriers, adapter lists and the adapters' buffers go from tile to tile."""
    assert -(-m // 256) * -(-n // 256) > 4 * 74
    c = make(m, n, k, rank, D, varied_ids(m, D, m))
    y = torch.full((m + 1, n), -7777.0, dtype=dtype, device="cuda")
    check(c, call(c, y=y[:m]))
    assert (y[m:] == -7777.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_broken_adapter_of_many_row_tiles(dtype, bad):
    """B of one adapter is not finite in some columns, x in a row: the other
    values keep their bits."""
    m, n, k, rank, D = 5000, 4100, 264, 24, 7
    c = make(m, n, k, rank, D, varied_ids(m, D, 3))
    want = call(c, out_dtype=dtype)
    columns = torch.tensor([0, 31, 200, 1777, 4099], device="cuda")
    d = dict(c, B=c["B"].clone())
    d["B"][2, columns, rank - 1] = bad
    got = call(d, out_dtype=dtype)
    hit = c["ids"] == 2
    assert hit.any() and not torch.isfinite(got[hit][:, columns]).any()
    got[:, columns] = torch.where(hit[:, None], want[:, columns], got[:, columns])
    assert torch.equal(got, want)
    d = dict(c, x=c["x"].clone())
    d["x"][4444, 5] = bad
    got = call(d, out_dtype=dtype)
    assert not torch.isfinite(got[4444]).any()
    got[4444] = want[4444]
    assert torch.equal(got, want)


BY_TOKEN = [
    # m, n, k, rank: one tile per cluster, of 1, 2 or 4 CTA pairs
    (65, 513, 256, 32), (251, 700, 512, 16),
    (200, 1300, 2048, 40), (90, 1000, 2048, 16),
    (150, 520, 4096, 24), (47, 300, 4096, 8), (200, 2300, 1024, 128), (300, 520, 2048, 16), (250, 4000, 2048, 16),
    (260, 2300, 2048, 40),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [15, 17, 21, 25, 31, 37, 45, 70, 250])
@pytest.mark.parametrize("m, n, k, rank", BY_TOKEN)
def test_numbers_of_adapters_around_the_by_token_border(m, n, k, rank, D, dtype):
    c = make(m, n, k, rank, D, lambda t: (t * 3) % (D + 1) - 1, seed=D)
    check(c, call(c, out_dtype=dtype))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("m, n, k, rank", BY_TOKEN)
def test_a_broken_adapter_by_token(m, n, k, rank, bad):
    D = 200
    c = make(m, n, k, rank, D, lambda t: (t * 3) % (D + 1) - 1)
    want = call(c)
    a = c["ids"][m // 2].item()
    hit = c["ids"] == a
    for part in ("A", "B"):
        d = dict(c, **{part: c[part].clone()})
        d[part][a] = bad
        got = call(d)
        assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).any()
    d = dict(c, B=c["B"].clone())
    d["B"][a, 7, rank - 1] = bad
    got = call(d)
    assert not torch.isfinite(got[hit][:, 7]).any()
    got[hit, 7] = want[hit, 7]
    assert torch.equal(got, want)
    d = dict(c, x=c["x"].clone())
    d["x"][5] = bad
    got = call(d)
    assert not torch.isfinite(got[5]).any()
    got[5] = want[5]
    assert torch.equal(got, want)


@pytest.mark.parametrize("m, k, rank, D", [(32, 1024, 128, 32), (32, 4096, 120, 40), (29, 72, 128, 29)])
def test_streamed_adapters_beyond_a_block_each(m, k, rank, D):
    """Eight blocks of 16 rank rows to an adapter leave 18 adapters at once."""
    c = make(m, 300, k, rank, D, lambda t: t % D)
    check(c, call(c))


@pytest.mark.parametrize("m, n, k, rank, D", [(33, 1, 8, 8, 1), (40, 24, 8, 128, 3), (257, 1, 24, 8, 2), (256, 7, 16, 16, 1)])
def test_smallest_sizes_of_larger_batches(m, n, k, rank, D):
    c = make(m, n, k, rank, D, lambda t: t % (D + 1) - 1)
    check(c, call(c))
    check(c, call(c, out_dtype=torch.bfloat16))


def test_adapters_past_32_bit_offsets():
    """A and B of more than 2^31 values each; the adapters that no token uses hold whatever was there."""
    n, k, rank, D = 4096, 4096, 16, 33000
    assert D * rank * k > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    used = [0, 20000, D - 1]
    A, B = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((D, rank, k), (D, n, rank)))
    for a in used:
        A[a], B[a] = normal(g, rank, k, std=k ** -0.5), normal(g, n, rank, std=0.25)
    for m in (20, 100, 2500):
        pick = torch.arange(m, device="cuda") % 4 - 1
        c = {"x": normal(g, m, k), "W": normal(g, n, k, std=k ** -0.5), "A": A[used], "B": B[used], "scales": None, "ids": pick.int()}
        ids = torch.where(pick >= 0, torch.tensor(used, device="cuda")[pick.clamp(min=0)], -1).int()
        check(c, moe.moe_matmul_lora(c["x"], c["W"], ids, A, B))


def test_rows_past_32_bit_offsets():
    m, n, k, rank, D = 263000, 8200, 64, 8, 3
    assert m * n > 2 ** 31
    c = make(m, n, k, rank, D, lambda t: t % (D + 1) - 1)
    y = call(c, out_dtype=torch.bfloat16)
    for at in (0, 131072, 261888, m - 300):
        rows = slice(at, at + 300)
        check(dict(c, x=c["x"][rows], ids=c["ids"][rows]), y[rows])


@pytest.mark.parametrize("at", [0, 300, 4999])
def test_a_bad_id_among_many_row_tiles_leaves_y_unwritten(at):
    m, n, k, rank, D = 5000, 4100, 72, 16, 7
    c = make(m, n, k, rank, D, varied_ids(m, D, 5))
    ws = torch.empty(moe.moe_matmul_lora_workspace(m, n, k, rank, D), dtype=torch.uint8, device="cuda")
    y = torch.full((m, n), 5.0, device="cuda")
    good = c["ids"][at].item()
    c["ids"][at] = D
    call(c, y=y, ws=ws)
    assert moe.moe_check_status(ws) == 6 and (y == 5.0).all()
    c["ids"][at] = good
    check(c, call(c, y=y, ws=ws))
    assert moe.moe_check_status(ws) == 0


@pytest.mark.parametrize("m, n", [(100, 520), (2500, 4100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_replays_with_other_numbers_of_adapters(m, n, dtype):
    """How a tile's adapters are added is decided on the device, by the ids of the replay."""
    k, rank, D = 1024, 16, 64
    c = make(m, n, k, rank, D, [-1] * m)
    y = torch.empty((m, n), dtype=dtype, device="cuda")
    ws = torch.empty(moe.moe_matmul_lora_workspace(m, n, k, rank, D), dtype=torch.uint8, device="cuda")
    call(c, y=y, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, y=y, ws=ws)
    for used in (3, 64, 1, 20, 0):
        c["ids"].copy_(torch.arange(m) % used if used else torch.full((m,), -1))
        graph.replay()
        torch.cuda.synchronize()
        check(c, y)
        assert torch.equal(call(c, out_dtype=dtype), y)
    del graph
