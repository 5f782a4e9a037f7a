"""Plain 64-bit forms of the serving operators (the whole layer for a few
tokens, the projection with adapters) with element-wise error bounds.

A bound is derived, not tuned: every step's forward error is carried along
with the value.  Units: u = 2^-24 is the relative error of one f32 rounding.
One tensor-core instruction adds 16 products and the accumulator; its f32
result is off by at most 4 u of the sum of their magnitudes (products of
bf16 values are exact; alignment and the final step lose below 2^-22 of the
largest magnitude).
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -120  # covers results that underflow


def dot_gamma(k: int, parts: int = 1) -> float:
    """Relative error, against the sum of magnitudes, of a dot product of
    length k whose 64-column steps go over 16 warps (4 instructions per step
    and part in a warp's chain), the 16 partial sums added in f32."""
    chain = 4 * parts * -(-(-(-k // 64)) // 16)
    return (4 * chain + 16) * U


def silu(g):
    return g / (1 + torch.exp(-g))


def route(logits64, bias, top_k):
    """ids (ties: lower index), weights and f32 logits from exact logits."""
    logits = logits64.float()
    score = (1 / (1 + torch.exp(-logits.double()))).float()
    key = score + (bias.float() if bias is not None else 0.0)
    key = torch.where(torch.isnan(key), torch.full_like(key, float("-inf")), key)
    ids = torch.stack([torch.tensor(sorted(range(key.shape[1]), key=lambda e, t=t: (-key[t, e].item(), e))[:top_k])
                       for t in range(key.shape[0])]) if key.shape[0] else torch.zeros((0, top_k), dtype=torch.int64)
    s = score.gather(1, ids).double()
    return ids, (s / s.sum(1, keepdim=True)), logits


def ffn(x, gate, up, down):
    """down (silu(gate x) * up x) for one expert's rows x [t, hidden], with its bound."""
    gate, up, down = gate.double(), up.double(), down.double()
    g, u = x @ gate.T, x @ up.T
    dg = dot_gamma(x.shape[1]) * (x.abs() @ gate.abs().T)
    du = dot_gamma(x.shape[1]) * (x.abs() @ up.abs().T)
    a = silu(g) * u
    # |silu'| <= 1.1; expf, the division and two products: 8 u
    da = 1.1 * dg * (u.abs() + du) + silu(g).abs() * du + 8 * U * a.abs()
    d = a @ down.T
    mag = a.abs() @ down.abs().T
    return d, da @ down.abs().T + (dot_gamma(a.shape[1], 3) + 2 * U) * mag


def layer(x, W_router, bias, top_k, W_gate, W_up, W_down, shared=None):
    """(y, bound, ids, weights, logits) of the whole layer; CPU tensors."""
    xd = x.double()
    ids, w, logits = route(xd @ W_router.double().T, bias, top_k)
    y, dy, mag = torch.zeros_like(xd), torch.zeros_like(xd), torch.zeros_like(xd)
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        d, dd = ffn(xd[t], W_gate[e], W_up[e], W_down[e])
        ww = w[t, j].unsqueeze(1)
        y[t] += ww * d
        dy[t] += ww * dd
        mag[t] += (ww * d).abs()
    if shared is not None:
        w_sh, sg, su, sd = shared
        gate = 1 / (1 + torch.exp(-(xd @ w_sh.double())))
        d, dd = ffn(xd, sg, su, sd)
        y += gate.unsqueeze(1) * d
        dy += gate.unsqueeze(1) * dd
        mag += (gate.unsqueeze(1) * d).abs()
    # each weight, product and addition of the combine rounds once
    return y, dy + (top_k + 4) * U * mag + TINY, ids, w, logits


def lora(x, W, ids, A, B, scales, bf16_out):
    """(y, bound) of the projection with adapters; CPU tensors."""
    xd, Wd = x.double(), W.double()
    k, rank = x.shape[1], A.shape[1]
    y = xd @ Wd.T
    # the tcgen05 projection accumulates its k / 16 instructions in one chain
    dy = (4 * -(-k // 16) + 16) * U * (xd.abs() @ Wd.abs().T)
    for a in ids.unique().tolist():
        if a < 0:
            continue
        t = (ids == a).nonzero().squeeze(1)
        Ad, Bd = A[a].double(), B[a].double()
        s = scales[a].double() if scales is not None else torch.tensor(1.0, dtype=torch.float64)
        h = xd[t] @ Ad.T
        dh = (4 * -(-k // 16) + 24) * U * (xd[t].abs() @ Ad.abs().T)  # one chain, as the projection
        y[t] += s * (h @ Bd.T)
        # h enters its product with 16 significant bits or more; rank sequential additions
        dy[t] += s.abs() * (dh @ Bd.abs().T + (2.0 ** -17 + (rank + 8) * U) * (h.abs() @ Bd.abs().T))
    dy += 4 * U * y.abs() + TINY
    if bf16_out:
        dy += 2.0 ** -8 * (y.abs() + dy)
    return y, dy
