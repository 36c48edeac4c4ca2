"""4-bit weights with group scales: conversion, the linear product and the dense MLP against
plain 64-bit forms (tests/int4_ref.py, whose error bounds are the tolerances)."""
import pytest
import torch

from sparse_moe_transformer_fp32_b200 import beam_moe as bm
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


# ------------------------------------------------------------------ conversion

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("groups,rows,cols,pair", [
    (1, 1, 128, False), (1, 17, 256, False), (3, 16, 384, False), (2, 8, 128, True),
    (2, 24, 640, True), (1, 1283, 2560, False)])
def test_quantize_matches_definition(group, groups, rows, cols, pair):
    a = normal(1, groups, rows, cols)
    b = normal(2, groups, rows, cols, std=3.0) if pair else None
    # a zero group, a zero row, an outlier, tiny values, and elements exactly between two codes
    a[0, 0, :group] = 0
    if rows > 2:
        a[0, 2] = 0
        a[0, 1, 5] = 300.0
        a[-1, 1, -group:] *= 1e-30
        s = 2.0 ** -3
        a[-1, rows - 1, :16] = torch.arange(-7, 9, device="cuda").to(torch.bfloat16) * s + s / 2
        a[-1, rows - 1, 15] = 7 * s
    packed = bm.beam_int4_quantize(a, b, group_size=group)
    m = (R.interleave(a, b) if pair else a).cpu()
    q, s = R.codes(m, group)
    got_q, got_s = R.unpack(packed, m.shape[1], cols, group)
    n = m.shape[1]
    assert torch.equal(got_q[:, :n], q)
    assert torch.equal(got_s[:, :n], s)
    assert not got_q[:, n:].any() and not got_s[:, n:].any()  # rows that only fill the last tile
    # the value is within half a step of the weight, unless the code saturates at 7 by the
    # rounding of s (then within s * 7 * 2^-8 more)
    v = (q.unflatten(-1, (-1, group)) * s[..., None]).flatten(-2)
    step = s[..., None].expand(*s.shape, group).flatten(-2)
    assert ((v - m.double()).abs() <= step * (0.5 + 7 * R.U16) + 2.0 ** -133).all()


def test_quantize_writes_only_its_bytes():
    a = normal(3, 2, 24, 256)
    n = bm.beam_int4_packed_size(1, 24, 256, 64)
    buf = torch.full((4, n), 0xA5, dtype=torch.uint8, device="cuda")
    bm.beam_int4_quantize(a, group_size=64, out=buf[1:3])
    assert (buf[0] == 0xA5).all() and (buf[3] == 0xA5).all()
    assert torch.equal(buf[1:3], bm.beam_int4_quantize(a, group_size=64))


# ------------------------------------------------------------------ linear product

def run_linear(T, N, K, group, fp32, seed=0, x=None, w=None):
    x = normal(seed + 1, T, K) if x is None else x
    w = normal(seed + 2, 1, N, K, std=K ** -0.5) if w is None else w
    packed = bm.beam_int4_quantize(w, group_size=group)
    # rows before and behind the outputs stay as they were
    pad = torch.full((T + 2, N), 7.0, device="cuda", dtype=torch.float32 if fp32 else torch.bfloat16)
    off = (-N * pad.element_size()) % 16  # 16-byte aligned start
    flat = torch.full((T * N + 64,), 7.0, device="cuda", dtype=pad.dtype)
    out = flat[16:16 + T * N].view(T, N)
    assert off >= 0
    bm.beam_int4_linear(bm.int4_shape(T, N, K, group), x, packed, out)
    assert (flat[:16] == 7).all() and (flat[16 + T * N:] == 7).all()
    return x, w, packed, out


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K,fp32", [
    (1, 1, 128, True), (1, 16, 128, False), (3, 40, 256, True), (8, 33, 384, False),
    (9, 129, 640, True), (16, 250, 1408, False), (2, 1283, 2560, False), (7, 2048, 2176, True),
    (16, 2400, 5120, True), (5, 2600, 8192, False), (11, 1000, 8320, True), (1, 640, 20480, True),
    (16, 500, 20480, False), (4, 100, 32768, True), (16, 100, 32768, True)])
def test_linear_matches_64_bits(T, N, K, fp32, group):
    x, w, _, out = run_linear(T, N, K, group, fp32)
    ref, bound = R.linear_ref(x, w[0], group, fp32)
    R.assert_within(out, ref, bound, f"T={T} N={N} K={K} g={group}")


@pytest.mark.parametrize("T", range(1, 17))
def test_linear_every_token_count(T):
    x, w, _, out = run_linear(T, 272, 1280, 128, True, seed=T)
    ref, bound = R.linear_ref(x, w[0], 128, True)
    R.assert_within(out, ref, bound, f"T={T}")


@pytest.mark.parametrize("T", [3, 12])
def test_linear_keeps_tokens_apart(T):
    """Infinities and NaN in one token's input reach that token's outputs only."""
    x = normal(5, T, 1280)
    x[1, 7] = float("inf")
    x[2, 100] = float("nan")
    w = normal(6, 1, 272, 1280, std=0.03)
    packed = bm.beam_int4_quantize(w, group_size=64)
    out = torch.empty(T, 272, device="cuda")
    bm.beam_int4_linear(bm.int4_shape(T, 272, 1280, 64), x, packed, out)
    assert not torch.isfinite(out[1]).any() and torch.isnan(out[2]).all()
    rest = [t for t in range(T) if t not in (1, 2)]
    ref, bound = R.linear_ref(x[rest], w[0], 64, True)
    R.assert_within(out[rest], ref, bound)


@pytest.mark.parametrize("spread", [4, 12, 24, 60])
def test_linear_with_a_wide_range_of_magnitudes(spread):
    """Elements spread over 2^-spread .. 1 of the largest, and tokens of very different size."""
    T, N, K = 6, 300, 2560
    x = normal(1, T, K)
    e = torch.randint(-spread, 1, (T, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    x = (x.double() * 2.0 ** e).to(torch.bfloat16)
    x = (x.double() * (2.0 ** torch.tensor([0, 90, -60, 7, -100, 30], device="cuda").double())[:, None])
    x = x.to(torch.bfloat16)
    x, w, _, out = run_linear(T, N, K, 64, True, x=x)
    ref, bound = R.linear_ref(x, w[0], 64, True)
    R.assert_within(out, ref, bound)


def test_linear_zero_tokens_and_extremes():
    x = torch.zeros(3, 256, device="cuda", dtype=torch.bfloat16)
    x[1, 3] = 2.0 ** -130   # subnormal
    x[2, 200] = 1e38
    x, w, _, out = run_linear(3, 64, 256, 32, True, x=x)
    assert (out[0] == 0).all()
    ref, bound = R.linear_ref(x, w[0], 32, True)
    R.assert_within(out, ref, bound + 2.0 ** -126)


def test_linear_same_bits_every_time():
    for T, N, K in ((1, 2571, 5120), (16, 5120, 20480)):
        x, w, packed, out = run_linear(T, N, K, 128, True)
        for _ in range(5):
            again = torch.empty_like(out)
            bm.beam_int4_linear(bm.int4_shape(T, N, K, 128), x, packed, again)
            assert torch.equal(again, out)


def test_linear_token_rows_do_not_depend_on_the_batch():
    """A token's outputs are the same bits alone and among up to eight tokens."""
    x, w, packed, out = run_linear(8, 1283, 2560, 64, True)
    one = torch.empty(1, 1283, device="cuda")
    for t in range(8):
        bm.beam_int4_linear(bm.int4_shape(1, 1283, 2560, 64), x[t:t + 1].clone(), packed, one)
        assert torch.equal(one[0], out[t])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K,fp32", [
    (1, 20011, 640, True), (2, 16000, 1408, False), (3, 20483, 256, True), (4, 11000, 5120, False),
    (8, 20011, 640, True), (16, 11000, 1408, False)])
def test_linear_with_many_tiles_to_a_cta(T, N, K, fp32, group):
    """Steps of two tiles, even and odd numbers of tiles to a CTA."""
    x, w, _, out = run_linear(T, N, K, group, fp32)
    ref, bound = R.linear_ref(x, w[0], group, fp32)
    R.assert_within(out, ref, bound, f"T={T} N={N} K={K} g={group}")


def test_linear_rows_of_steps_of_two_tiles_have_the_same_bits():
    x, w, packed, out = run_linear(8, 20011, 1280, 64, True)
    for first, n in ((0, 1), (3, 2), (4, 4), (1, 5)):
        part = torch.empty(n, 20011, device="cuda")
        bm.beam_int4_linear(bm.int4_shape(n, 20011, 1280, 64), x[first:first + n].clone(), packed, part)
        assert torch.equal(part, out[first:first + n])


def test_linear_chain_back_to_back():
    """Each product reads what the one before wrote, without a wait between them; and weights
    converted right before their first use."""
    x = normal(7, 4, 1280)
    ws = [normal(20 + i, 1, 1280, 1280, std=1280 ** -0.5) for i in range(6)]
    torch.cuda.synchronize()
    sh = bm.int4_shape(4, 1280, 1280, 64)
    bufs = [torch.empty(4, 1280, device="cuda", dtype=torch.bfloat16) for _ in ws]
    src = x
    for w, o in zip(ws, bufs):
        bm.beam_int4_linear(sh, src, bm.beam_int4_quantize(w, group_size=64), o)
        src = o
    packed = [bm.beam_int4_quantize(w, group_size=64) for w in ws]
    again = [torch.empty_like(o) for o in bufs]
    src = x
    for p, o in zip(packed, again):
        bm.beam_int4_linear(sh, src, p, o)
        src = o
    torch.cuda.synchronize()
    src = x
    for w, o, a in zip(ws, bufs, again):
        assert torch.equal(o, a)
        ref, bound = R.linear_ref(src, w[0], 64, False)
        R.assert_within(o, ref, bound)
        src = o


# ------------------------------------------------------------------ dense MLP

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,d,I", [(1, 256, 128), (5, 1024, 2816), (8, 512, 640), (9, 256, 1408),
                                   (16, 2560, 1280), (3, 5120, 20480), (16, 256, 32768)])
def test_dense_matches_64_bits(T, d, I, group):
    h = normal(1, T, d)
    g, u = (normal(s, 1, I, d, std=d ** -0.5) for s in (2, 3))
    dn = normal(4, 1, d, I, std=I ** -0.5)
    sh = bm.dense_shape(T, d, I)
    out = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    gu, dq = bm.beam_int4_quantize(g, u, group_size=group), bm.beam_int4_quantize(dn, group_size=group)
    ws = bm.beam_dense_forward_int4(sh, group, h, gu, dq, out)
    ref, bound = R.dense_ref(h, g[0], u[0], dn[0], group)
    R.assert_within(out, ref, bound, f"T={T} d={d} I={I} g={group}")
    again = torch.empty_like(out)
    bm.beam_dense_forward_int4(sh, group, h, gu, dq, again, ws=ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("T", [1, 3, 8])
def test_dense_loses_nothing_before_the_output_is_rounded(T):
    """Up to 8 tokens the activation stays FP32: what is ahead of the output's rounding to BF16 is off by
    less than 2^-15 of it, against a rounding of 2^-9 half the time, so the whole error has the
    rounding's mean square to within some percent (a BF16 activation would double it)."""
    d, I = 1024, 2816
    h = normal(1, T, d)
    g, u = (normal(s, 1, I, d, std=d ** -0.5) for s in (2, 3))
    dn = normal(4, 1, d, I, std=I ** -0.5)
    out = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    gu, dq = bm.beam_int4_quantize(g, u, group_size=64), bm.beam_int4_quantize(dn, group_size=64)
    bm.beam_dense_forward_int4(bm.dense_shape(T, d, I), 64, h, gu, dq, out)
    ref, _ = R.dense_ref(h, g[0], u[0], dn[0], 64)
    rounding = (ref.to(torch.bfloat16).double() - ref).square().mean()
    assert (out.double() - ref).square().mean() <= 1.1 * rounding


# ------------------------------------------------------------------ streams, graphs, waits

def test_linear_and_dense_replay_from_a_graph_and_run_on_other_streams():
    T, d, I = 3, 512, 1280
    h = normal(1, T, d)
    g, u = (normal(s, 1, I, d, std=d ** -0.5) for s in (2, 3))
    dn = normal(4, 1, d, I, std=I ** -0.5)
    head = normal(5, 1, 999, d, std=d ** -0.5)
    gu, dq = bm.beam_int4_quantize(g, u, group_size=64), bm.beam_int4_quantize(dn, group_size=64)
    hq = bm.beam_int4_quantize(head, group_size=64)
    sh, lin = bm.dense_shape(T, d, I), bm.int4_shape(T, 999, d, 64)
    ws = bm.dense_int4_workspace(sh)
    mid = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(T, 999, device="cuda")

    def step():
        bm.beam_dense_forward_int4(sh, 64, h, gu, dq, mid, ws=ws)
        bm.beam_int4_linear(lin, mid, hq, out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for seed in (11, 12):
        h.copy_(normal(seed, T, d))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        assert torch.equal(got, out)
        ref, bound = R.dense_ref(h, g[0], u[0], dn[0], 64)
        R.assert_within(mid, ref, bound)
        ref, bound = R.linear_ref(mid, head[0], 64, True)
        R.assert_within(out, ref, bound)


def test_two_streams_at_once():
    sh = bm.int4_shape(2, 4000, 2560, 128)
    w = [normal(s, 1, 4000, 2560, std=0.02) for s in (1, 2)]
    q = [bm.beam_int4_quantize(m, group_size=128) for m in w]
    x = [normal(s, 2, 2560) for s in (3, 4)]
    outs = [[torch.empty(2, 4000, device="cuda") for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(10):
        for s in range(2):
            bm.beam_int4_linear(sh, x[s], q[s], outs[s][i], stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        ref, bound = R.linear_ref(x[s], w[s][0], 128, True)
        R.assert_within(outs[s][0], ref, bound)
        assert all(torch.equal(o, outs[s][0]) for o in outs[s])


@pytest.mark.parametrize("T,N,K", [(1, 2571, 2560), (16, 320, 20480)])
def test_wait_that_runs_out_shows_as_nan_and_the_context_survives(T, N, K):
    x, w, packed, out = run_linear(T, N, K, 128, True)
    sh = bm.int4_shape(T, N, K, 128)
    good = out.clone()
    old = bm.beam_moe_get_wait_limit_ns()
    bm.beam_moe_set_wait_limit_ns(0)
    try:
        bm.beam_int4_linear(sh, x, packed, out)
        torch.cuda.synchronize()
    finally:
        bm.beam_moe_set_wait_limit_ns(old)
    assert torch.isnan(out).any()
    ok = ~torch.isnan(out)
    assert torch.equal(out[ok], good[ok])  # what is not NaN is right
    bm.beam_int4_linear(sh, x, packed, out)
    assert torch.equal(out, good)


@pytest.mark.parametrize("T,d,I,group", [(9, 1024, 2816, 64), (12, 1024, 2816, 32), (16, 1024, 2816, 128),
                                         (16, 2560, 640, 64), (11, 512, 8320, 64)])
def test_dense_of_9_to_16_tokens_loses_nothing_before_the_output_is_rounded(T, d, I, group):
    """As for up to 8 tokens: the whole error has the rounding's mean square to within some percent."""
    h = normal(1, T, d)
    g, u = (normal(s, 1, I, d, std=d ** -0.5) for s in (2, 3))
    dn = normal(4, 1, d, I, std=I ** -0.5)
    flat = torch.full((T + 2, d), 7.0, device="cuda", dtype=torch.bfloat16)
    out = flat[1:T + 1]
    gu, dq = bm.beam_int4_quantize(g, u, group_size=group), bm.beam_int4_quantize(dn, group_size=group)
    bm.beam_dense_forward_int4(bm.dense_shape(T, d, I), group, h, gu, dq, out)
    assert (flat[0] == 7).all() and (flat[T + 1] == 7).all()
    ref, bound = R.dense_ref(h, g[0], u[0], dn[0], group)
    R.assert_within(out, ref, bound, f"T={T} d={d} I={I} g={group}")
    rounding = (ref.to(torch.bfloat16).double() - ref).square().mean()
    assert (out.double() - ref).square().mean() <= 1.1 * rounding


LATE_COPY = """
extern "C" __global__ void late_copy(const unsigned* src, unsigned* dst, int n) {
  asm volatile("griddepcontrol.launch_dependents;");  // the successor may start now
  for (long long t = clock64(); clock64() - t < 200000;) {}
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) dst[i] = src[i];
}
"""


@pytest.mark.parametrize("T,N,K", [(2, 1283, 1280), (12, 640, 20480)])
def test_weights_written_by_a_kernel_that_lets_its_successor_start_early(T, N, K):
    late = torch.cuda._compile_kernel(LATE_COPY, "late_copy")
    x, old, new = normal(1, T, K), normal(2, 1, N, K, std=K ** -0.5), normal(3, 1, N, K, std=K ** -0.5)
    src, packed = bm.beam_int4_quantize(new, group_size=64), bm.beam_int4_quantize(old, group_size=64)
    out = torch.empty(T, N, device="cuda")
    torch.cuda.synchronize()
    late(grid=(32, 1, 1), block=(256, 1, 1), args=[src, packed, src.numel() // 4])
    bm.beam_int4_linear(bm.int4_shape(T, N, K, 64), x, packed, out)
    torch.cuda.synchronize()
    ref, bound = R.linear_ref(x, new[0], 64, True)
    R.assert_within(out, ref, bound, f"T={T} N={N} K={K}")


@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("which", ["gate_up", "down"])
def test_dense_weights_written_by_a_kernel_that_lets_its_successor_start_early(which, T):
    late = torch.cuda._compile_kernel(LATE_COPY, "late_copy")
    d, I = 512, 1280
    h = normal(1, T, d)
    g, u = (normal(s, 1, I, d, std=d ** -0.5) for s in (2, 3))
    dn = normal(4, 1, d, I, std=I ** -0.5)
    packed = {"gate_up": bm.beam_int4_quantize(g, u, group_size=64), "down": bm.beam_int4_quantize(dn, group_size=64)}
    src = packed[which].clone()
    packed[which].zero_()
    out = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    ws = bm.dense_int4_workspace(bm.dense_shape(T, d, I))
    torch.cuda.synchronize()
    late(grid=(32, 1, 1), block=(256, 1, 1), args=[src, packed[which], src.numel() // 4])
    bm.beam_dense_forward_int4(bm.dense_shape(T, d, I), 64, h, packed["gate_up"], packed["down"], out, ws=ws)
    torch.cuda.synchronize()
    R.assert_within(out, *R.dense_ref(h, g[0], u[0], dn[0], 64), which)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T", [4, 8, 9, 16])
def test_linear_of_tokens_whose_unscaled_sums_would_overflow(T, group):
    """Elements up to 1e38 against weights of 0.04: the codes alone, up to 7, would take the sums of a group
    beyond FP32; the outputs are 2^123 at most."""
    x = normal(1, T, 512)
    x[2, 200] = 1e38
    x[3] = (normal(2, 512).double() * 2.0 ** 118).bfloat16()
    x[0] = (normal(3, 512).double() * 2.0 ** -100).bfloat16()
    x, w, _, out = run_linear(T, 80, 512, group, True, x=x)
    ref, bound = R.linear_ref(x, w[0], group, True)
    assert ref.abs().max() < 2.0 ** 124
    R.assert_within(out, ref, bound)


@pytest.mark.parametrize("as_handle", [False, True])
def test_quantize_on_another_stream_does_not_take_memory_that_is_still_written(as_handle):
    """Memory freed on the current stream while a write to it is queued there."""
    a = normal(1, 4, 512, 512)
    want = bm.beam_int4_quantize(a, group_size=64)
    side = torch.cuda.Stream()
    old = torch.empty_like(want)
    old.fill_(3)  # loads the kernel
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # 50 ms
    old.fill_(3)
    del old
    got = bm.beam_int4_quantize(a, group_size=64, stream=side.cuda_stream if as_handle else side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_workspaces_of_calls_on_another_stream_come_from_its_pool():
    T, d, I = 3, 512, 1280
    h = normal(1, T, d)
    g, u = (normal(s, 1, I, d, std=d ** -0.5) for s in (2, 3))
    dn = normal(4, 1, d, I, std=I ** -0.5)
    gu, dq = bm.beam_int4_quantize(g, u, group_size=64), bm.beam_int4_quantize(dn, group_size=64)
    sh = bm.dense_shape(T, d, I)
    layer = bm.make_shape(T, d, 4, 1, 1, 1, I)
    router_w, bias = normal(5, 4, d, std=0.02, dtype=torch.float32), torch.zeros(4, device="cuda")
    gu4, dq4 = gu.expand(4, -1).contiguous(), dq.expand(4, -1).contiguous()
    w = [t.expand(4, -1, -1).contiguous() for t in (g, u, dn)]
    out, side = torch.empty_like(h), torch.cuda.Stream()
    calls = [
        (lambda: bm.dense_int4_workspace(sh), lambda: bm.beam_dense_forward_int4(sh, 64, h, gu, dq, out, stream=side)),
        (lambda: bm.few_workspace(layer),
         lambda: bm.beam_moe_forward_few(layer, h, router_w, bias, *w, out, stream=side)),
        (lambda: bm.few_workspace(layer),
         lambda: bm.beam_moe_forward_few_int4(layer, 64, h, router_w, bias, gu4, dq4, out, stream=side))]
    torch.cuda.synchronize()
    for allocate, call in calls:
        free = [allocate() for _ in range(4)]  # what the current stream's pool would hand out
        at = [t.data_ptr() for t in free]
        del free
        ws = call()
        torch.cuda.synchronize()
        assert ws.data_ptr() not in at
