"""The MoE layer for a few tokens (BF16 and 4-bit experts) against plain 64-bit forms
(tests/int4_ref.py, whose error bounds are the tolerances) and the oracle's routing."""
import numpy as np
import pytest
import torch

import oracle
from sparse_moe_transformer_fp32_b200 import beam_moe as bm
from sparse_moe_transformer_fp32_b200 import workloads as W
from tests import int4_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def normal(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)


class Layer:
    def __init__(self, d, E, G, Gk, k, I, group=0, seed=0, bias=None, norm=True, scale=2.5):
        self.cfg = (d, E, G, Gk, k, I)
        self.group, self.norm, self.scale = group, norm, scale
        self.router_w = normal(seed + 1, E, d, std=0.7 * d ** -0.5, dtype=torch.float32)
        self.bias = normal(seed + 2, E, std=0.05, dtype=torch.float32) if bias is None else bias
        self.gate = normal(seed + 3, E, I, d, std=d ** -0.5)
        self.up = normal(seed + 4, E, I, d, std=d ** -0.5)
        self.down = normal(seed + 5, E, d, I, std=I ** -0.5)
        if group:
            self.gu = bm.beam_int4_quantize(self.gate, self.up, group_size=group)
            self.dn = bm.beam_int4_quantize(self.down, group_size=group)

    def shape(self, T):
        d, E, G, Gk, k, I = self.cfg
        return bm.make_shape(T, d, E, G, Gk, k, I, self.scale, self.norm)

    def call(self, h, out, idx=None, w=None, ws=None, stream=None):
        s = self.shape(h.shape[0])
        if self.group:
            return bm.beam_moe_forward_few_int4(s, self.group, h, self.router_w, self.bias, self.gu,
                                                self.dn, out, idx, w, ws=ws, stream=stream)
        return bm.beam_moe_forward_few(s, h, self.router_w, self.bias, self.gate, self.up, self.down,
                                       out, idx, w, ws=ws, stream=stream)

    def run(self, h, ws=None):
        T, (d, E, G, Gk, k, I) = h.shape[0], self.cfg
        # rows before and behind the outputs stay as they were
        flat = torch.full((T + 2, d), 7.0, device="cuda", dtype=torch.bfloat16)
        out = flat[1:T + 1]
        idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), -1.0, device="cuda")
        ws = self.call(h, out, idx, w, ws)
        assert bm.beam_moe_sync_status(ws) == bm.BEAM_OK
        assert (flat[0] == 7).all() and (flat[T + 1] == 7).all()
        return out, idx, w, ws

    def check(self, h, out, idx, w):
        d, E, G, Gk, k, I = self.cfg
        ridx, rw = R.route_ref(h, self.router_w, self.bias, G, Gk, k, self.scale, self.norm)
        assert torch.equal(idx.cpu().long(), ridx)
        # score (rounded twice to FP32), k - 1 additions, product and quotient
        assert ((w.cpu().double() - rw).abs() <= (k + 6) * R.U32 * rw).all()
        ref, bound = R.layer_ref(h, ridx, rw, self.gate, self.up, self.down, self.group)
        return R.assert_within(out, ref, bound, f"T={h.shape[0]} {self.cfg} g={self.group}")


SHAPES = [  # T, d, E, G, Gk, k, I
    (1, 256, 16, 4, 2, 4, 128),
    (7, 256, 16, 4, 2, 4, 128),
    (16, 256, 4, 1, 1, 1, 128),
    (5, 512, 32, 8, 8, 8, 384),
    (3, 768, 64, 2, 1, 3, 640),
    (16, 1280, 128, 4, 3, 5, 256),
    (2, 2560, 40, 8, 5, 7, 1408),
    (9, 4096, 8, 2, 2, 2, 2048),
    (4, 5120, 16, 4, 2, 8, 2560),
    (2, 8192, 4, 1, 1, 2, 8192),
    (6, 256, 256, 32, 3, 8, 128),
]


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("T,d,E,G,Gk,k,I", SHAPES)
def test_layer_matches_64_bits(T, d, E, G, Gk, k, I, group):
    m = Layer(d, E, G, Gk, k, I, group)
    h = normal(99, T, d)
    out, idx, w, _ = m.run(h)
    m.check(h, out, idx, w)


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count(T, group):
    m = Layer(512, 16, 4, 2, 4, 384, group, seed=T)
    h = normal(99 + T, T, 512)
    out, idx, w, _ = m.run(h)
    m.check(h, out, idx, w)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T", [8, 9, 16])
def test_all_tokens_on_the_same_experts(T, group):
    """More than eight tokens on an expert open a second entry for it."""
    bias = torch.zeros(32, device="cuda")
    bias[[3, 4, 9, 30]] = 5.0
    m = Layer(512, 32, 4, 4, 4, 256, group, bias=bias)
    h = normal(3, T, 512)
    out, idx, w, _ = m.run(h)
    assert (idx.cpu() == torch.tensor([3, 4, 9, 30])).all()
    m.check(h, out, idx, w)
    # identical tokens give identical rows
    h[1:] = h[0]
    out, idx, w, _ = m.run(h)
    assert (out == out[0]).all()


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_layer_loses_nothing_before_the_output_is_rounded(T, group):
    """The activations stay FP32 (two BF16 pieces with BF16 weights): the whole error has the mean square
    of the output's rounding to within some percent; BF16 activations would double it."""
    m = Layer(1280, 32, 4, 2, 4, 640, group)
    h = normal(11, T, 1280)
    out, idx, w, _ = m.run(h)
    ridx, rw = R.route_ref(h, m.router_w, m.bias, 4, 2, 4, m.scale, m.norm)
    ref, _ = R.layer_ref(h, ridx, rw, m.gate, m.up, m.down, group)
    rounding = (ref.to(torch.bfloat16).double() - ref).square().mean()
    assert (out.double() - ref).square().mean() <= 1.1 * rounding


def test_ties_go_to_the_lower_index():
    m = Layer(256, 32, 4, 2, 4, 128)
    m.router_w.zero_()
    m.bias.zero_()
    h = normal(3, 5, 256)
    out, idx, w, _ = m.run(h)
    assert (idx.cpu() == torch.arange(4)).all()
    assert (w == 2.5 / 4).all()
    m.check(h, out, idx, w)
    # equal groups and equal experts across lanes of 32
    m = Layer(256, 256, 8, 4, 8, 128)
    m.router_w.zero_()
    m.bias.zero_()
    m.bias[[5, 37, 69, 101, 133, 165, 197, 229]] = 1.0  # one per group: groups tie, lowest four stay
    out, idx, w, _ = m.run(h)
    assert idx[0].tolist() == [0, 1, 2, 3, 5, 37, 69, 101]
    m.check(h, out, idx, w)


def test_near_ties_follow_the_definition():
    """Router rows that differ in their last bits: FP32 sums in another order would choose others."""
    m = Layer(5120, 64, 8, 4, 8, 128)
    base = normal(8, 1, 5120, std=0.01, dtype=torch.float32)
    m.router_w.copy_(base * (1 + 1e-6 * torch.rand(64, 1, device="cuda", generator=torch.Generator(
        device="cuda").manual_seed(4))))
    m.bias.zero_()
    for seed in range(8):
        h = normal(200 + seed, 16, 5120)
        out, idx, w, _ = m.run(h)
        m.check(h, out, idx, w)


def test_routing_equals_the_oracle_without_removing_near_ties():
    wl = W.WORKLOADS["decode"].with_tokens(16)
    h, router_w, bias = W.hidden(wl), W.router_weight(wl), W.router_bias(wl)
    _, ridx, rw, _, _ = oracle.layer_routing(h, router_w, bias, wl)
    m = Layer(wl.d, wl.E, wl.n_group, wl.topk_group, wl.top_k, 128)
    m.router_w, m.bias = router_w.cuda(), bias.cuda()
    out, idx, w, _ = m.run(h.cuda())
    assert np.array_equal(idx.cpu().numpy(), ridx)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-6)


def test_unnormalised_weights_and_another_scale():
    m = Layer(512, 16, 4, 2, 4, 256, norm=False, scale=1.25)
    h = normal(4, 6, 512)
    out, idx, w, _ = m.run(h)
    m.check(h, out, idx, w)


@pytest.mark.parametrize("group", [0, 32])
def test_a_nan_token_stays_alone(group):
    m = Layer(512, 16, 4, 2, 4, 256, group)
    h = normal(4, 6, 512)
    h[2, 9] = float("nan")
    h[4, 0] = float("inf")
    out, idx, w, _ = m.run(h)
    assert torch.isnan(out[2]).all()
    assert ((idx >= 0) & (idx < 16)).all()
    rest = [0, 1, 3, 5]
    m.check(h[rest], out[rest], idx[rest], w[rest])


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("T", [2, 3, 4])
def test_a_nan_token_stays_alone_where_columns_are_the_tokens(T, group):
    m = Layer(512, 16, 4, 2, 4, 256, group)
    h = normal(4, T, 512)
    h[1, 9] = float("nan")
    out, idx, w, _ = m.run(h)
    assert torch.isnan(out[1]).all()
    rest = [t for t in range(T) if t != 1]
    m.check(h[rest], out[rest], idx[rest], w[rest])


@pytest.mark.parametrize("T,d,I", [(3, 5376, 256), (5, 5376, 256), (4, 512, 6144), (16, 512, 6144)])
def test_wide_layers_hold_two_tokens_to_an_entry(T, d, I):
    m = Layer(d, 8, 2, 2, 3, I, 64)
    h = normal(8, T, d)
    out, idx, w, _ = m.run(h)
    m.check(h, out, idx, w)


@pytest.mark.parametrize("T", [5, 8, 13])
def test_rows_do_not_depend_on_how_entries_are_cut(T):
    """All tokens on the same experts: entries of four tokens and a rest, and each token alone."""
    bias = torch.zeros(32, device="cuda")
    bias[[3, 4, 9, 30]] = 5.0
    m = Layer(512, 32, 4, 4, 4, 256, 64, bias=bias)
    h = normal(13, T, 512)
    out = m.run(h)[0]
    for t in range(T):
        one = torch.empty_like(out[:1])
        m.call(h[t:t + 1].clone(), one)
        assert torch.equal(one[0], out[t])


@pytest.mark.parametrize("group", [0, 64])
def test_same_bits_every_time_and_without_optional_outputs(group):
    m = Layer(2560, 64, 8, 4, 8, 1280, group)
    h = normal(4, 5, 2560)
    out, idx, w, ws = m.run(h)
    for _ in range(10):
        again = torch.empty_like(out)
        m.call(h, again, ws=ws)
        assert torch.equal(again, out)
    # a token alone has the bits that it has among others
    for t in range(5):
        one = torch.empty_like(out[:1])
        m.call(h[t:t + 1].clone(), one)
        assert torch.equal(one[0], out[t])


@pytest.mark.parametrize("group", [0, 128])
def test_graph_replay_two_graphs_on_one_workspace(group):
    m = Layer(1280, 32, 4, 2, 4, 640, group)
    h1, h2 = normal(1, 3, 1280), normal(2, 9, 1280)
    o1, o2 = torch.empty_like(h1), torch.empty_like(h2)
    ws = bm.few_workspace(m.shape(9))
    m.call(h1, o1, ws=ws)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        m.call(h1, o1, ws=ws)
        m.call(h1, o1, ws=ws)
    with torch.cuda.graph(g2):
        m.call(h2, o2, ws=ws)
    for seed in (10, 20, 30):
        h1.copy_(normal(seed, 3, 1280))
        h2.copy_(normal(seed + 1, 9, 1280))
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert bm.beam_moe_sync_status(ws) == bm.BEAM_OK
        for h, o in ((h1, o1), (h2, o2)):
            got = o.clone()
            again, idx, w, _ = m.run(h)
            assert torch.equal(got, again)
            m.check(h, got, idx, w)


def test_two_streams_at_once_with_their_own_workspaces():
    ms = [Layer(1280, 32, 4, 2, 4, 640, 0, seed=1), Layer(1280, 32, 4, 2, 4, 640, 64, seed=2)]
    hs = [normal(5, 4, 1280), normal(6, 7, 1280)]
    want = [m.run(h)[0].clone() for m, h in zip(ms, hs)]
    streams = [torch.cuda.Stream() for _ in ms]
    wss = [bm.few_workspace(m.shape(h.shape[0])) for m, h in zip(ms, hs)]
    outs = [[torch.empty_like(h) for _ in range(10)] for h in hs]
    torch.cuda.synchronize()
    for i in range(10):
        for m, h, o, ws, st in zip(ms, hs, outs, wss, streams):
            m.call(h, o[i], ws=ws, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)


@pytest.mark.parametrize("group", [0, 64])
def test_wait_that_runs_out_is_reported_and_the_context_survives(group):
    m = Layer(1280, 32, 4, 2, 4, 640, group)
    h = normal(5, 4, 1280)
    out, idx, w, ws = m.run(h)
    good = out.clone()
    old = bm.beam_moe_get_wait_limit_ns()
    bm.beam_moe_set_wait_limit_ns(0)
    try:
        m.call(h, out, ws=ws)
        assert bm.beam_moe_sync_status(ws) == bm.BEAM_ERR_TIMEOUT
    finally:
        bm.beam_moe_set_wait_limit_ns(old)
    m.call(h, out, ws=ws)
    assert bm.beam_moe_sync_status(ws) == bm.BEAM_OK
    assert torch.equal(out, good)


def test_agrees_with_the_many_token_layer():
    """The same layer through beam_moe_forward, whose BF16 expert outputs its tolerance counts."""
    wl = W.WORKLOADS["tiny"]
    m = Layer(wl.d, wl.E, wl.n_group, wl.topk_group, wl.top_k, wl.I)
    h = normal(3, 16, wl.d)
    out, idx, w, _ = m.run(h)
    other = torch.empty_like(out)
    oidx = torch.empty_like(idx)
    bm.beam_moe_forward(m.shape(16), h, m.router_w, m.bias, m.gate, m.up, m.down, other, oidx)
    torch.cuda.synchronize()
    same = (idx == oidx).all(dim=1).cpu()
    assert same.sum() >= 12
    ref, bound = R.layer_ref(h, idx.cpu().long(), w.cpu().double(), m.gate, m.up, m.down, 0)
    # expert outputs rounded to BF16 before the weighted sum: another half step of each
    assert ((other.double() - ref).abs().cpu() <= 2 * bound.cpu() + 2.5 * R.U16 * 4 *
            ref.abs().amax().cpu())[same].all()


def test_a_decode_step_of_dense_moe_and_head():
    """Dense 4-bit MLP, the MoE layer with 4-bit experts, and an LM head, back to back on a stream:
    each stage against the 64-bit form on the stage before."""
    T, d, I, V = 4, 512, 1280, 1001
    m = Layer(d, 32, 4, 2, 4, 384, 64)
    h = normal(1, T, d)
    g, u = (normal(s, 1, I, d, std=d ** -0.5) for s in (2, 3))
    dn, head = normal(4, 1, d, I, std=I ** -0.5), normal(5, 1, V, d, std=d ** -0.5)
    gu, dq = bm.beam_int4_quantize(g, u, group_size=64), bm.beam_int4_quantize(dn, group_size=64)
    hq = bm.beam_int4_quantize(head, group_size=64)
    x1, x2 = torch.empty_like(h), torch.empty_like(h)
    idx = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 4, device="cuda")
    logits = torch.empty(T, V, device="cuda")
    dws, ws = bm.dense_int4_workspace(bm.dense_shape(T, d, I)), bm.few_workspace(m.shape(T))
    for _ in range(3):
        bm.beam_dense_forward_int4(bm.dense_shape(T, d, I), 64, h, gu, dq, x1, ws=dws)
        m.call(x1, x2, idx, w, ws=ws)
        bm.beam_int4_linear(bm.int4_shape(T, V, d, 64), x2, hq, logits)
    assert bm.beam_moe_sync_status(ws) == bm.BEAM_OK
    R.assert_within(x1, *R.dense_ref(h, g[0], u[0], dn[0], 64), "dense")
    m.check(x1, x2, idx, w)
    R.assert_within(logits, *R.linear_ref(x2, head[0], 64, True), "head")


@pytest.mark.parametrize("group", [0, 128])
def test_beam_layer(group):
    """The full Beam shape: expert rows beyond 32-bit element offsets."""
    m = Layer(5120, 256, 8, 4, 8, 2560, group)
    for T in (1, 16):
        h = normal(7 + T, T, 5120)
        out, idx, w, _ = m.run(h)
        assert T == 1 or int(idx.max()) > 200
        m.check(h, out, idx, w)


def pair_layer(T, I, k, E):
    """Experts whose activations come in nearly equal pairs, with outputs that are their differences.  Gate
    and up sums hold two terms, exact in FP32, and a pair's differ by 2^-16: what is lost of an activation
    on its way into the second product shows in the output."""
    d = 256
    m = Layer(d, E, 1, 1, k, I, bias=torch.linspace(1, 0, E, device="cuda"))
    h = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    h[:, 0] = 1.0 + torch.arange(T, device="cuda") / 64
    h[:, 1] = 2.0 ** -8
    for w in (m.gate, m.up, m.down):
        w.zero_()
    m.gate[..., 0] = normal(31, E, I // 2, std=0.7).abs().clamp(0.25, 2).repeat_interleave(2, dim=1)
    m.up[..., 0] = normal(32, E, I // 2).abs().clamp(0.5, 2).repeat_interleave(2, dim=1)
    m.up[:, 0::2, 1] = 1.0
    m.up[:, 1::2, 1] = 1.0 + 2.0 ** -7
    r = torch.arange(d, device="cuda")
    pair = r * (I // 2) // d
    m.down[:, r, 2 * pair] = 1.0
    m.down[:, r, 2 * pair + 1] = -1.0
    return m, h


@pytest.mark.parametrize("T,I,k", [(1, 128, 1), (2, 384, 3), (3, 128, 1), (4, 256, 2), (5, 1280, 1), (16, 128, 2),
                                   (4, 4096, 1), (3, 4224, 1), (7, 8192, 2)])
def test_bf16_layer_keeps_every_bit_of_the_activation(T, I, k):
    m, h = pair_layer(T, I, k, 4)
    out, idx, w, _ = m.run(h)
    ridx, rw = R.route_ref(h, m.router_w, m.bias, 1, 1, k)
    assert torch.equal(idx.cpu().long(), ridx)
    x = h.double()
    ref, mag = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e, wt = int(ridx[t, j]), rw[t, j].item()
            g, u = m.gate[e].double() @ x[t], m.up[e].double() @ x[t]
            a = g * torch.sigmoid(g) * u
            ref[t] += wt * (m.down[e].double() @ a)
            mag[t] += wt * (m.down[e].double().abs() @ a.abs())
    # of each activation: its product's rounding (the SiLU's error is the pair's alike, 8 half steps of the
    # difference), and one each of the three columns' sums and the two additions of columns; then the
    # weights' and the combine's roundings, and the output's
    bound = 8 * R.U32 * mag + 16 * R.U32 * ref.abs() + R.U16 * ref.abs()
    R.assert_within(out, ref, bound + 1e-37, f"T={T} I={I} k={k}")


MASKS = {  # of 32 experts in 4 groups: one expert; all but one of a group; a group; one of each group; all but two of each
    "one": [5], "all but one of a group": list(range(1, 8)), "a group": list(range(8, 16)),
    "one of each group": [0, 9, 18, 27], "all but two of each": [e for e in range(32) if e % 8 not in (2, 5)]}


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [1, 3, 6, 16])
@pytest.mark.parametrize("mask", MASKS)
def test_a_bias_of_minus_infinity_masks_experts(mask, T, group):
    bias = normal(2, 32, std=0.05, dtype=torch.float32)
    bias[MASKS[mask]] = -float("inf")
    m = Layer(512, 32, 4, 2, 4, 128, group, bias=bias)
    h = normal(3, T, 512)
    out, idx, w, _ = m.run(h)
    assert not torch.isin(idx.cpu(), torch.tensor(MASKS[mask])).any()
    m.check(h, out, idx, w)
    # and as in the many-token layer, whose experts' outputs are not looked at here
    oidx, ow = torch.empty_like(idx), torch.empty_like(w)
    bm.beam_moe_route(m.shape(T), h, m.router_w, m.bias, oidx, ow)
    torch.cuda.synchronize()
    assert torch.equal(idx, oidx)


def test_masked_experts_fill_up_where_no_other_is_left():
    """All groups but one masked and more experts to choose than are left open: the lowest masked ones."""
    bias = torch.full((32,), -float("inf"), device="cuda")
    bias[[17, 21]] = 0.0
    m = Layer(512, 32, 4, 2, 4, 128, bias=bias)
    h = normal(3, 5, 512)
    out, idx, w, _ = m.run(h)
    assert (idx.cpu() == torch.tensor([0, 1, 17, 21])).all()
    m.check(h, out, idx, w)


def test_a_bias_of_plus_infinity_forces_experts():
    bias = normal(2, 32, std=0.05, dtype=torch.float32)
    bias[[6, 30]] = float("inf")
    bias[[1, 2, 3]] = -float("inf")
    m = Layer(512, 32, 4, 2, 4, 128, bias=bias)
    h = normal(3, 7, 512)
    out, idx, w, _ = m.run(h)
    assert (idx == 6).any(dim=1).all() and (idx == 30).any(dim=1).all()
    m.check(h, out, idx, w)


@pytest.mark.parametrize("T,d,I,group", [(1, 256, 128, 0), (10, 8192, 256, 0), (4, 5120, 2560, 64), (16, 512, 1280, 32)])
def test_short_wait_limits_give_the_right_output_or_are_reported(T, d, I, group):
    """Whichever wait runs out, the router's or one of the layer's: never a wrong output with BEAM_OK."""
    m = Layer(d, 16, 4, 2, 4, I, group)
    h = normal(5, T, d)
    out, idx, w, ws = m.run(h)
    want = out.clone()
    old = bm.beam_moe_get_wait_limit_ns()
    seen = set()
    try:
        for limit in (0, 0, 1, 500, 2000, 5000, 10_000, 20_000, 50_000, 100_000, 1_000_000):
            bm.beam_moe_set_wait_limit_ns(limit)
            out.fill_(7.0)
            m.call(h, out, ws=ws)
            status = bm.beam_moe_sync_status(ws)
            assert status in (bm.BEAM_OK, bm.BEAM_ERR_TIMEOUT)
            if status == bm.BEAM_OK:
                assert torch.equal(out, want), limit
            else:
                seen.add(bm.last_cuda_error())
    finally:
        bm.beam_moe_set_wait_limit_ns(old)
    assert seen  # a limit of 0 gives up at once
    if d == 8192:  # 224 KB of copies a CTA are not there at once: the router's wait (site 26)
        assert any("site 26" in s for s in seen), seen
    m.call(h, out, ws=ws)
    assert bm.beam_moe_sync_status(ws) == bm.BEAM_OK
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 2, 5, 9])
def test_router_sums_of_zeros_and_huge_values(T):
    """Zero weights with tokens of 2^120, and zero tokens with weights of 2^125: logits of exactly zero."""
    m = Layer(256, 16, 4, 2, 4, 128, norm=False)
    m.bias.zero_()
    m.router_w.zero_()
    m.gate.zero_()
    h = (normal(3, T, 256).abs().double() * 2.0 ** 120).bfloat16()
    out, idx, w, _ = m.run(h)
    assert (w == 2.5 * 0.5).all() and (idx.cpu() == torch.arange(4)).all() and (out == 0).all()
    m.router_w.fill_(2.0 ** 125)
    out, idx, w, _ = m.run(torch.zeros_like(h))
    assert (w == 2.5 * 0.5).all() and (idx.cpu() == torch.arange(4)).all() and (out == 0).all()
    # zeros among others
    h = normal(4, T, 256)
    h[:, 1::2] = 0
    m.router_w.copy_(normal(5, 16, 256, std=0.05, dtype=torch.float32))
    m.router_w[:, 1::2] = 2.0 ** 125
    m.gate.copy_(normal(6, 16, 128, 256, std=1 / 16))
    out, idx, w, _ = m.run(h)
    m.check(h, out, idx, w)


def test_router_subnormals_count():
    """Subnormal weights against tokens of 2^126: logits of 2^-5 for one expert, 2^-6 for the next."""
    m = Layer(256, 4, 1, 1, 2, 128, norm=False)
    m.bias.zero_()
    m.router_w.zero_()
    m.router_w[2, 9], m.router_w[1, 9] = 2.0 ** -131, 2.0 ** -132
    m.gate.zero_()
    h = torch.zeros(3, 256, device="cuda", dtype=torch.bfloat16)
    h[:, 9] = 2.0 ** 126
    out, idx, w, _ = m.run(h)
    assert (idx.cpu() == torch.tensor([1, 2])).all()
    want = 2.5 * torch.sigmoid(torch.tensor([2.0 ** -6, 2.0 ** -5], dtype=torch.float64))
    assert ((w.cpu().double() - want).abs() <= 4 * R.U32 * want).all()


@pytest.mark.parametrize("group", [0, 64])
def test_a_nan_router_row_is_not_hidden(group):
    m = Layer(512, 16, 4, 2, 4, 128, group)
    m.router_w[11, 100] = float("nan")
    h = normal(3, 5, 512)
    out, idx, w, _ = m.run(h)
    assert (idx == 11).any(dim=1).all()
    assert torch.isnan(out).all() and torch.isnan(w).all()


def test_infinite_router_weights_decide():
    m = Layer(512, 16, 4, 2, 4, 128)
    m.router_w[11, 100], m.router_w[3, 200] = float("inf"), -float("inf")
    h = normal(3, 8, 512)
    assert (h[:, [100, 200]] != 0).all()
    out, idx, w, _ = m.run(h)
    m.check(h, out, idx, w)


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [1, 4, 11, 16])
def test_loads_and_the_bias_update_from_a_few_token_workspace(T, group):
    m = Layer(512, 32, 4, 2, 4, 128, group)
    out, idx, w, ws = m.run(normal(3, T, 512))
    loads = torch.bincount(idx.flatten().cpu().long(), minlength=32)
    assert torch.equal(bm.beam_moe_expert_counts(m.shape(T), ws).long(), loads)
    want = m.bias.cpu() + 0.25 * torch.sign(T * 4 / 32 - loads.double()).float()
    bm.beam_moe_bias_update(m.shape(T), ws, m.bias, 0.25)
    torch.cuda.synchronize()
    assert torch.equal(m.bias.cpu(), want)


def test_slot_rows_are_refused_after_a_few_token_forward():
    m = Layer(512, 32, 4, 2, 4, 128)
    h = normal(3, 11, 512)
    ws = bm.workspace(m.shape(11))  # larger than a few-token one
    out, idx = torch.empty_like(h), torch.empty(11, 4, dtype=torch.int32, device="cuda")

    def many():
        bm.beam_moe_forward(m.shape(11), h, m.router_w, m.bias, m.gate, m.up, m.down, out, idx, ws=ws)
        return bm.beam_moe_slot_rows(m.shape(11), ws)

    rows = many()
    m.call(h, out, ws=ws)
    with pytest.raises(bm.BeamError) as e:
        bm.beam_moe_slot_rows(m.shape(11), ws)
    assert e.value.status == bm.BEAM_ERR_WORKSPACE and "few-token" in bm.last_cuda_error()
    assert torch.equal(many(), rows)


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T,d", [(16, 5888), (11, 8192), (16, 8192)])
def test_router_of_wide_layers_in_one_and_two_launches(T, d, group):
    """16 token rows of 5888 do not fit beside the router's weights in shared memory, nor 11 of 8192."""
    m = Layer(d, 16, 4, 2, 4, 128, group)
    h = normal(9, T, d)
    before = bm.beam_moe_launch_count()
    out, idx, w, ws = m.run(h)
    assert bm.beam_moe_launch_count() - before == 3
    m.check(h, out, idx, w)
    assert bm.beam_moe_expert_counts(m.shape(T), ws).sum() == T * 4


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T,d,I", [(4, 512, 256), (5, 512, 256), (8, 512, 256), (9, 512, 256), (2, 5376, 256),
                                   (3, 5376, 256), (5, 5376, 256), (2, 256, 4224), (3, 256, 4224), (5, 256, 4224)])
def test_entries_of_the_same_experts_at_their_limits(T, d, I, group):
    """An entry holds 4 tokens, 2 in wide layers; one more token of an expert opens another."""
    bias = torch.zeros(8, device="cuda")
    bias[[2, 7]] = 5.0
    m = Layer(d, 8, 2, 2, 2, I, group, bias=bias)
    h = normal(3, T, d)
    out, idx, w, _ = m.run(h)
    assert (idx.cpu() == torch.tensor([2, 7])).all()
    m.check(h, out, idx, w)
    one = torch.empty_like(out[:1])
    for t in range(T):
        m.call(h[t:t + 1].clone(), one)
        assert torch.equal(one[0], out[t])


def test_a_captured_step_that_forks_and_joins():
    """Products on two streams that join before the layer, which forks again into two heads."""
    T, d, V = 3, 512, 1001
    m = Layer(d, 32, 4, 2, 4, 384, 64)
    h = normal(1, T, d)
    ws_ = [normal(s, 1, n, d, std=d ** -0.5) for s, n in ((2, d), (3, d), (4, V), (5, V))]
    qs = [bm.beam_int4_quantize(w, group_size=64) for w in ws_]
    a, b, x = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    idx = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 4, device="cuda")
    l1, l2 = torch.empty(T, V, device="cuda"), torch.empty(T, V, device="cuda")
    ws = bm.few_workspace(m.shape(T))
    square, head = bm.int4_shape(T, d, d, 64), bm.int4_shape(T, V, d, 64)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        bm.beam_int4_linear(square, h, qs[0], a)
        with torch.cuda.stream(side):
            bm.beam_int4_linear(square, h, qs[1], b)
        main.wait_stream(side)
        bm.beam_int4_linear(square, b, qs[0], x)   # behind both
        m.call(x, a, idx, w, ws=ws)
        side.wait_stream(main)
        bm.beam_int4_linear(head, a, qs[2], l1)
        with torch.cuda.stream(side):
            bm.beam_int4_linear(head, a, qs[3], l2)
        main.wait_stream(side)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for seed in (11, 12):
        h.copy_(normal(seed, T, d))
        for t in (a, b, x, l1, l2):
            t.fill_(9.0)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert bm.beam_moe_sync_status(ws) == bm.BEAM_OK
        R.assert_within(b, *R.linear_ref(h, ws_[1][0], 64, False), "second branch")
        R.assert_within(x, *R.linear_ref(b, ws_[0][0], 64, False), "after the join")
        m.check(x, a, idx, w)
        R.assert_within(l1, *R.linear_ref(a, ws_[2][0], 64, True), "head")
        R.assert_within(l2, *R.linear_ref(a, ws_[3][0], 64, True), "other head")


def test_two_host_threads_at_once():
    import threading
    ms = [Layer(1280, 32, 4, 2, 4, 640, 0, seed=1), Layer(1280, 32, 4, 2, 4, 640, 64, seed=2)]
    hs = [normal(5, 4, 1280), normal(6, 7, 1280)]
    want = [m.run(h)[0].clone() for m, h in zip(ms, hs)]
    lw = normal(7, 1, 999, 1280, std=0.03)
    lq = bm.beam_int4_quantize(lw, group_size=64)
    logits = []
    for o, h in zip(want, hs):
        logits.append(torch.empty(h.shape[0], 999, device="cuda"))
        bm.beam_int4_linear(bm.int4_shape(h.shape[0], 999, 1280, 64), o, lq, logits[-1])
    torch.cuda.synchronize()
    bad = []

    def work(m, h, o, l):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ws, out = bm.few_workspace(m.shape(h.shape[0])), torch.empty_like(h)
            got = torch.empty_like(l)
            for _ in range(40):
                m.call(h, out, ws=ws)
                bm.beam_int4_linear(bm.int4_shape(h.shape[0], 999, 1280, 64), out, lq, got)
                stream.synchronize()
                if not (torch.equal(out, o) and torch.equal(got, l)):
                    bad.append(m.group)
            if bm.beam_moe_sync_status(ws) != bm.BEAM_OK:
                bad.append("status")

    threads = [threading.Thread(target=work, args=a) for a in zip(ms, hs, want, logits)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
