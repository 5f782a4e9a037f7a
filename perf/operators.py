"""The serving operators' cases: what they compute in plain form, and the calls a user makes of them.

Two operators of a decode step around a routed mixture-of-experts layer:

* ``layer``: the whole layer for a few tokens, from the hidden states to the layer's output (router projection,
  sigmoid + selection-bias top-k, the chosen experts' SwiGLU FFN, the weighted combine, and an optional shared
  expert with a sigmoid gate):
      logits = x . W_router^T (rounded once to f32),  s = sigmoid(logits),  ids = top_k of s + bias (lower index
      wins ties),  w_j = s[ids_j] / sum_j s[ids_j],
      y = sum_j w_j W_down[e_j] (silu(W_gate[e_j] x) * W_up[e_j] x)
          + sigmoid(w_sh . x) W_sh_down (silu(W_sh_gate x) * W_sh_up x)
* ``lora``: a projection that all requests share, with the low-rank adapter of each token's own request beside it:
      y[t] = W x[t] + scales[a] B[a] (A[a] x[t]),  a = adapter_ids[t]  (a = -1: the projection alone)
"""
import math

import torch

own = False


def listed():
    return [
        # one token of a small layer (the sizes that the graph tests use): latency alone counts
        layer("layer m1 small", m=1, hidden=512, inter=256, experts=32, top_k=8),
        # one request decoding: the weights of 8 of 256 experts are read once
        layer("layer m1", m=1, hidden=4096, inter=1536, experts=256, top_k=8),
        # a decode batch of 8 requests, and one with a shared expert beside 128 routed ones
        layer("layer m8", m=8, hidden=4096, inter=1536, experts=256, top_k=8),
        layer("layer m13 shared", m=13, hidden=2048, inter=768, experts=128, top_k=8, shared=768),
        # ragged sizes: nothing is a multiple of a tile
        layer("layer m5 ragged", m=5, hidden=1000, inter=520, experts=60, top_k=6, shared=264),
        # the largest batch, and the same batch with its tokens crowded on 16 popular experts
        layer("layer m32", m=32, hidden=4096, inter=1536, experts=256, top_k=8),
        layer("layer m32 hot", m=32, hidden=4096, inter=1536, experts=256, top_k=8, hot=16),
        # one token of one request beside its adapter
        lora("lora m1", m=1, k=4096, n=4096, rank=16, adapters=8, requests=1, out="bf16"),
        # a decode batch, every token of another request
        lora("lora m32", m=32, k=4096, n=4096, rank=16, adapters=64, requests=32, out="bf16"),
        # a mixed batch of odd sizes: short pieces of prompts between single tokens
        lora("lora m201 ragged", m=201, k=1000, n=1501, rank=24, adapters=40, requests=23, out="f32"),
        # prompts of a few requests, and the largest: long prompts at a high rank
        lora("lora m4096", m=4096, k=4096, n=4096, rank=16, adapters=8, requests=6, out="bf16"),
        lora("lora m16384", m=16384, k=2048, n=4096, rank=64, adapters=16, requests=9, out="f32"),
    ]


def layer(name, m, hidden, inter, experts, top_k, shared=0, hot=0):
    """hot: that many experts, at random, get a selection bias that all tokens follow (0: the router alone decides)."""
    c = {"op": "layer", "m": m, "hidden": hidden, "inter": inter, "experts": experts, "top_k": top_k, "shared": shared, "hot": hot}
    return c if name is None else {"name": name, **c}


def lora(name, m, k, n, rank, adapters, requests, out):
    """requests: the tokens are that many runs of ragged lengths; one in eight of them takes no adapter."""
    c = {"op": "lora", "m": m, "k": k, "n": n, "rank": rank, "adapters": adapters, "requests": requests, "out": out}
    return c if name is None else {"name": name, **c}


def spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    if rng.random() < 0.5:
        m = spread(rng, 1, 32)
        experts = spread(rng, 8, 256)
        top_k = rng.randint(1, min(8, experts))
        return layer(None, m=m, hidden=8 * spread(rng, 32, 512), inter=8 * spread(rng, 16, 192), experts=experts, top_k=top_k,
                     shared=rng.choice([0, 8 * spread(rng, 16, 192)]), hot=rng.choice([0, 0, max(top_k, experts // 8)]))
    k, n, rank = 8 * spread(rng, 32, 512), spread(rng, 256, 4096), 8 * rng.randint(1, 16)
    most = 16384 * 2048 * 4096 // (n * (k + 4 * rank))
    m = min(spread(rng, 1, 16384), most)
    return lora(None, m=m, k=k, n=n, rank=rank, adapters=spread(rng, 1, 64), requests=spread(rng, 1, min(m, 256)), out=rng.choice(["f32", "bf16"]))


def distinct(case):
    """Experts that at least one token is expected to choose, tokens choosing apart and evenly."""
    of = case["hot"] or case["experts"]
    return of * (1 - (1 - case["top_k"] / of) ** case["m"])


def adapted(case):
    """(requests with an adapter, adapters that they use)."""
    with_one = case["requests"] - case["requests"] // 8
    return with_one, min(with_one, case["adapters"])


def normal(g, shape, std):
    """Seeded bf16 normals, drawn in pieces so that a large stack needs no f32 copy of itself."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        piece = flat[at:at + (1 << 28)]
        piece.copy_(torch.randn(piece.numel(), generator=g, device="cuda") * std)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = case
    if c["op"] == "layer":
        m, hidden, inter, E, sh = c["m"], c["hidden"], c["inter"], c["experts"], c["shared"]
        s = {"case": c, "x": normal(g, (m, hidden), 1.0), "W_router": normal(g, (E, hidden), hidden ** -0.5),
             "bias": (torch.rand(E, generator=g, device="cuda") * 2 - 1) * 0.1,
             "W_gate": normal(g, (E, inter, hidden), 0.02), "W_up": normal(g, (E, inter, hidden), 0.02), "W_down": normal(g, (E, hidden, inter), 0.02)}
        if c["hot"]:
            s["bias"][torch.randperm(E, generator=g, device="cuda")[:c["hot"]]] += 1.0
        s["sh"] = (normal(g, (hidden,), 0.02), normal(g, (sh, hidden), 0.02), normal(g, (sh, hidden), 0.02), normal(g, (hidden, sh), 0.02)) if sh else None
        if own:
            import mixture_experts_routed_sigmoid_b200 as moe
            s["ws"] = torch.empty(moe.moe_layer_decode_workspace(m, hidden, inter, sh, c["top_k"], E), dtype=torch.uint8, device="cuda")
        return s
    m, k, n, r, D = c["m"], c["k"], c["n"], c["rank"], c["adapters"]
    s = {"case": c, "x": normal(g, (m, k), 1.0), "W": normal(g, (n, k), 0.02), "A": normal(g, (D, r, k), 0.02), "B": normal(g, (D, n, r), 0.02),
         "scales": torch.rand(D, generator=g, device="cuda") * 1.5 + 0.5}
    # the runs of tokens: requests - 1 cuts at distinct places, and the adapter of each run
    q = c["requests"]
    starts = torch.zeros(m, dtype=torch.int64, device="cuda")
    starts[1 + torch.randperm(m - 1, generator=g, device="cuda")[:q - 1]] = 1
    run_of = starts.cumsum(0)
    with_one, used = adapted(c)
    pick = torch.randperm(D, generator=g, device="cuda")[:used].repeat(q // used + 1)[:q]
    pick[with_one:] = -1
    s["ids"] = pick[torch.randperm(q, generator=g, device="cuda")][run_of].to(torch.int32)
    if own:
        import mixture_experts_routed_sigmoid_b200 as moe
        s["ws"] = torch.empty(moe.moe_matmul_lora_workspace(m, n, k, r, D), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    c = s["case"]
    if own:
        import mixture_experts_routed_sigmoid_b200 as moe
        if c["op"] == "layer":
            y, ids, weights, logits = moe.moe_layer_decode(s["x"], s["W_router"], s["bias"], c["top_k"], s["W_gate"], s["W_up"], s["W_down"],
                                                           *(s["sh"] or ()), ws=s["ws"])
            return {"y": y, "ids": ids, "weights": weights, "logits": logits}
        return moe.moe_matmul_lora(s["x"], s["W"], s["ids"], s["A"], s["B"], s["scales"], out_dtype=out_type(c), ws=s["ws"])
    return plain_layer(s) if c["op"] == "layer" else plain_lora(s)


def out_type(case):
    return torch.bfloat16 if case["out"] == "bf16" else torch.float32


def swiglu(x, gate, up, down):
    """down (silu(gate x) * up x) in 32 bits; x [..., hidden, 1], weights [..., out, in]."""
    a = gate.float() @ x
    return down.float() @ (a * torch.sigmoid(a) * (up.float() @ x))


def plain_layer(s):
    c, x = s["case"], s["x"]
    # in 64 bits, rounded once: which experts are chosen depends on the last bits of near-equal scores
    logits = (x.double() @ s["W_router"].double().T).float()
    score = torch.sigmoid(logits.double()).float()
    ids = (score + s["bias"]).sort(dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    chosen = score.gather(1, ids).double()
    weights = (chosen / chosen.sum(1, keepdim=True)).float()
    xf = x.float()
    rows = xf.repeat_interleave(c["top_k"], 0).unsqueeze(2)
    e = ids.reshape(-1)
    d = swiglu(rows, s["W_gate"][e], s["W_up"][e], s["W_down"][e]).view(c["m"], c["top_k"], c["hidden"])
    y = (weights.unsqueeze(2) * d).sum(1)
    if s["sh"]:
        w_sh, gate, up, down = s["sh"]
        y = y + torch.sigmoid(xf @ w_sh.float()).unsqueeze(1) * swiglu(xf.unsqueeze(2), gate, up, down).squeeze(2)
    return {"y": y, "ids": ids.to(torch.int32), "weights": weights, "logits": logits}


def plain_lora(s):
    c, x, ids = s["case"], s["x"].float(), s["ids"].long()
    D, r = c["adapters"], c["rank"]
    h = (x @ s["A"].float().view(D * r, -1).T).view(-1, D, r)
    # every token keeps its own adapter's part, times its scale
    mine = (ids.unsqueeze(1) == torch.arange(D, device="cuda")).float() * s["scales"]
    h = (h * mine.unsqueeze(2)).view(-1, D * r)
    return (x @ s["W"].float().T + h @ s["B"].float().transpose(0, 1).reshape(-1, D * r).T).to(out_type(c))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "layer":
        x = s["x"].double()
        logits = torch.einsum("th,eh->te", x, s["W_router"].double())
        score = 1 / (1 + torch.exp(-logits.float().double()))
        # the choice goes by the rounded scores: that is the operator's definition
        key = score.float() + s["bias"]
        order = sorted_by_key(key)[:, :c["top_k"]]
        w = score.gather(1, order)
        w = w / w.sum(1, keepdim=True)
        y = torch.zeros_like(x)

        def ffn(rows, gate, up, down):
            g = torch.einsum("th,ih->ti", rows, gate.double())
            u = torch.einsum("th,ih->ti", rows, up.double())
            return torch.einsum("ti,hi->th", g / (1 + torch.exp(-g)) * u, down.double())

        for e in order.unique().tolist():
            t, j = (order == e).nonzero(as_tuple=True)
            y[t] += w[t, j].unsqueeze(1) * ffn(x[t], s["W_gate"][e], s["W_up"][e], s["W_down"][e])
        if s["sh"]:
            w_sh, gate, up, down = s["sh"]
            y += (1 / (1 + torch.exp(-torch.einsum("th,h->t", x, w_sh.double())))).unsqueeze(1) * ffn(x, gate, up, down)
        return {"y": y, "ids": None, "weights": w, "logits": logits}
    x = s["x"].double()
    y = torch.einsum("tk,nk->tn", x, s["W"].double())
    for a in s["ids"].unique().tolist():
        if a >= 0:
            t = (s["ids"] == a).nonzero().squeeze(1)
            h = torch.einsum("tk,rk->tr", x[t], s["A"][a].double())
            y[t] += s["scales"][a].double() * torch.einsum("tr,nr->tn", h, s["B"][a].double())
    return y


def sorted_by_key(key):
    """Indices by falling key, the lower index first where keys are equal."""
    m, E = key.shape
    index = torch.arange(E, device=key.device)
    before = (key.unsqueeze(1) > key.unsqueeze(2)) | ((key.unsqueeze(1) == key.unsqueeze(2)) & (index[None, :] < index[:, None]))
    rank = before.sum(2)
    return torch.empty_like(rank).scatter_(1, rank, index.expand(m, E).contiguous())


def work(case):
    c = case
    m = c["m"]
    if c["op"] == "layer":
        hidden, per, k, E, sh = c["hidden"], 3 * c["hidden"] * c["inter"], c["top_k"], c["experts"], c["shared"]
        weights = distinct(c) * per + E * hidden + (3 * hidden * sh + hidden if sh else 0)
        return {"bytes": 2 * weights + 4 * E + m * (2 * hidden + 4 * hidden + 8 * k + 4 * E),
                "flops": 2 * m * (k * per + E * hidden + 3 * hidden * sh + (hidden if sh else 0))}
    n, kk, r = c["n"], c["k"], c["rank"]
    share = adapted(c)[0] / c["requests"]
    return {"bytes": 2 * n * kk + adapted(c)[1] * 2 * r * (kk + n) + m * (2 * kk + 4 + n * (2 if c["out"] == "bf16" else 4)),
            "flops": 2 * m * (n * kk + share * r * (kk + n))}
