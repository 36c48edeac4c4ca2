"""Plain 64-bit forms of the few-token operators, with error bounds, for their tests.

Written from the header's definitions with elementary torch operations; shares nothing with the
library.  Every ``*_ref`` returns (value, bound): the FP64 result and, element by element, how far
an implementation may be from it that holds products exactly (BF16 or code operands), sums in
FP32 and rounds where the definition says so.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24   # half a step of FP32, relative
U16 = 2.0 ** -8    # of BF16
# FP32 roundings on the way of one product into an output: 4 MMAs of a 64-element block, each of
# which may truncate (2 half steps), up to 32 scaled additions per warp, 16 warps, 8 CTAs
DEPTH = 4 * 2 + 32 + 16 + 8


def codes(w: torch.Tensor, group: int):
    """(q float64 [.., R, K], s float64 [.., R, K / group]) of BF16 weights."""
    x = w.float().unflatten(-1, (-1, group))
    s = (x.abs().amax(-1) / 7.0).to(torch.bfloat16).float()
    q = torch.where(s[..., None] > 0, x / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    q = q.round().clamp(-8, 7)
    return q.flatten(-2).double(), s.double()


def values(w: torch.Tensor, group: int):
    """The FP64 weights that an operator multiplies with; group 0: BF16 weights as they are."""
    if group == 0:
        return w.double()
    q, s = codes(w, group)
    return (q.unflatten(-1, (-1, group)) * s[..., None]).flatten(-2)


def interleave(a: torch.Tensor, b: torch.Tensor):
    """Rows of a and b in 8-row chunks, as beam_int4_quantize(a, b) stores them."""
    g, r, k = a.shape
    return torch.stack([a.view(g, r // 8, 8, k), b.view(g, r // 8, 8, k)], dim=2).reshape(g, 2 * r, k)


def unpack(packed: torch.Tensor, rows: int, cols: int, group: int):
    """(q [groups, rows16, cols], s [groups, rows16, cols / group]) read from packed bytes by the
    documented layout, one column and row at a time in index form; rows16: whole tiles."""
    groups = packed.shape[0]
    tiles, sbs, per = (rows + 15) // 16, cols // 128, 128 // group
    unit = 1024 + 32 * per
    p = packed.cpu().view(groups, tiles, sbs, unit)
    words = p[..., :1024].contiguous().view(torch.int32).long() & 0xffffffff   # [.., 256]
    words = words.view(groups, tiles, sbs, 2, 32, 4)                           # block, lane, v
    scales = p[..., 1024:].contiguous().view(torch.bfloat16).view(groups, tiles, sbs, per, 16)
    q = torch.empty(groups, tiles, 16, sbs, 128, dtype=torch.float64)
    s = torch.empty(groups, tiles, 16, sbs, per, dtype=torch.float64)
    for g in range(8):
        for c in range(4):
            for blk in range(2):
                for v in range(4):
                    w = words[:, :, :, blk, 4 * g + c, v]
                    for i in range(4):
                        k = 64 * blk + 32 * (v // 2) + 8 * c + 4 * (v % 2) + i
                        for half, at in ((0, 8 * i + 4), (8, 8 * i)):
                            n = (w >> at) & 15
                            q[:, :, g + half, :, k] = torch.where(n >= 8, n - 16, n).double()
        s[:, :, g] = scales[..., 2 * g].double()
        s[:, :, g + 8] = scales[..., 2 * g + 1].double()
    return q.reshape(groups, tiles * 16, cols), s.reshape(groups, tiles * 16, sbs * per)


def matmul_ref(x: torch.Tensor, w: torch.Tensor, dx=None, pieces=False):
    """x [n, K] FP64, w [R, K] FP64 -> (x w^T, bound); dx: bound of x's own error; pieces: x enters
    as 23-bit integers (4-bit weights), where elements below 2^-14 of the largest are off by up to
    2^-22 of it."""
    y = x @ w.T
    bound = DEPTH * U32 * (x.abs() @ w.abs().T)
    if pieces:
        top = x.abs().amax(1, keepdim=True)
        small = (x.abs() < 2.0 ** -14 * top * (1 + U16)) * top * 2.0 ** -22
        bound = bound + small @ w.abs().T
    if dx is not None:
        bound = bound + dx @ w.abs().T
    return y, bound


def linear_ref(x: torch.Tensor, w: torch.Tensor, group: int, fp32: bool):
    y, b = matmul_ref(x.double(), values(w, group), pieces=True)
    return y, b + (0 if fp32 else U16 * y.abs()) + 1e-37


def mlp_ref(x: torch.Tensor, gate, up, down, pieces=False):
    """SwiGLU MLP of x [n, d] FP64 with FP64 weights -> (y, bound); the activation is rounded to
    BF16 by definition, which the bound counts (the value leaves it out)."""
    g, dg = matmul_ref(x, gate, pieces=pieces)
    u, du = matmul_ref(x, up, pieces=pieces)
    sig = torch.sigmoid(g)
    a = g * sig * u
    # |silu'| <= 1.1; expf, the division and the two products: at most 8 half steps
    da = 1.1 * u.abs() * dg + (g * sig).abs() * du + 1.1 * dg * du + 8 * U32 * a.abs()
    da = da + U16 * (a.abs() + da)
    return matmul_ref(a, down, da, pieces)


def dense_ref(x, gate, up, down, group):
    y, b = mlp_ref(x.double(), values(gate, group), values(up, group), values(down, group), True)
    return y, b + U16 * y.abs() + 1e-37


def route_ref(h, router_w, bias, n_group, topk_group, k, scale=2.5, norm=True):
    """(idx [T, k] int64, w [T, k] float64): FP64 logits rounded to FP32, FP64 sigmoid rounded to
    FP32, selection on FP32 scores, the lower index on ties."""
    logit = (h.double().cpu() @ router_w.double().cpu().T).float()
    s = (1.0 / (1.0 + torch.exp(-logit.double()))).float()
    sb = s + bias.cpu().float()
    T, E = sb.shape
    P = E // n_group
    idx = []
    for t in range(T):
        v = sb[t].tolist()
        tot = []
        for g in range(n_group):
            two = sorted(v[g * P:(g + 1) * P], reverse=True)[:2]
            tot.append(torch.tensor(two).sum().item())
        kept = sorted(range(n_group), key=lambda g: (-tot[g], g))[:topk_group]
        cand = [e for g in kept for e in range(g * P, (g + 1) * P)]
        idx.append(sorted(sorted(cand, key=lambda e: (-v[e], e))[:k]))
    idx = torch.tensor(idx)
    w = s.double().gather(1, idx)
    if norm:
        w = w / w.sum(1, keepdim=True)
    return idx, w * scale


def layer_ref(h, idx, w, gate, up, down, group):
    """(out [T, d], bound) of the MoE layer on chosen experts idx with weights w."""
    x = h.double()
    out = torch.zeros_like(x)
    bound = torch.zeros_like(x)
    mag = torch.zeros_like(x)
    idx, w = idx.to(h.device), w.to(h.device)
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        y, b = mlp_ref(x[t], values(gate[e], group), values(up[e], group), values(down[e], group), group > 0)
        wt = w[t, j][:, None]
        out.index_add_(0, t, wt * y)
        bound.index_add_(0, t, wt * b)
        mag.index_add_(0, t, wt * y.abs())
    # the weights' own roundings (score, sum of k, product, quotient) and the sum over slots
    bound = bound + 2 * (idx.shape[1] + 6) * U32 * (mag + bound)
    return out, bound + U16 * (out.abs() + bound) + 1e-37


def assert_within(got, ref, bound, what=""):
    got, ref, bound = got.double().cpu(), ref.cpu(), bound.cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    err = (got - ref).abs()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of its bound (max abs {err.max().item():.3e})"
    return worst
