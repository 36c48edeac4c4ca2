"""Host-side checks of the few-token and 4-bit entry points: sizes, refusals before anything is
launched (fake pointers are never dereferenced), and the binding's argument checks."""
import ctypes

import pytest
import torch

from sparse_moe_transformer_fp32_b200 import beam_moe as bm
from sparse_moe_transformer_fp32_b200 import workloads as W

A = 0x7f0000000000  # 4 KB aligned fake address
q = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from sparse_moe_transformer_fp32_b200 import build
    build.build()
    return bm.lib()


def beam(T, **kw):
    s = bm.shape_of(W.WORKLOADS["prefill"], T)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("group", [32, 64, 128])
def test_packed_size(L, group):
    per = 1024 + 32 * (128 // group)
    assert bm.beam_int4_packed_size(1, 16, 128, group) == per
    assert bm.beam_int4_packed_size(1, 17, 128, group) == 2 * per      # whole 16-row tiles
    assert bm.beam_int4_packed_size(256, 5120, 5120, group) == 256 * 320 * 40 * per  # over 2^31
    assert bm.beam_int4_packed_size(0, 16, 128, group) == 0
    for bad in ((1, 0, 128, group), (1, 16, 64, group), (1, 16, 192, group), (-1, 16, 128, group),
                (1, 16, 0, group), (1, 16, 128, 16), (1, 16, 128, 256), (1, 16, 128, 0)):
        assert bm.beam_int4_packed_size(*bad) == 0, bad


def test_quantize_refuses(L):
    f = L.beam_int4_quantize
    far = A + (1 << 32)
    assert f(q(A), None, 0, 16, 128, 64, q(far), None) == bm.BEAM_OK  # nothing to convert
    for b, groups, rows, cols, group, out, want in (
            (None, -1, 16, 128, 64, far, bm.BEAM_ERR_INVALID_ARG),
            (None, 1, 0, 128, 64, far, bm.BEAM_ERR_INVALID_ARG),
            (None, 1, 16, 0, 64, far, bm.BEAM_ERR_INVALID_ARG),
            (None, 1, 16, 192, 64, far, bm.BEAM_ERR_UNSUPPORTED),
            (None, 1, 16, 128, 48, far, bm.BEAM_ERR_UNSUPPORTED),
            (A + (1 << 30), 1, 12, 128, 64, far, bm.BEAM_ERR_UNSUPPORTED),  # pairs: rows % 8
            (A + (1 << 30) + 8, 1, 16, 128, 64, far, bm.BEAM_ERR_INVALID_ARG),
            (None, 1, 16, 128, 64, far + 8, bm.BEAM_ERR_INVALID_ARG),
            (None, 1, 16, 128, 64, None, bm.BEAM_ERR_INVALID_ARG),
            (None, 2, 16, 128, 64, A + 16 * 128 * 2, bm.BEAM_ERR_INVALID_ARG),  # over the input
            (A + (1 << 30), 1, 16, 128, 64, A + (1 << 30) - 16, bm.BEAM_ERR_INVALID_ARG)):
        assert f(q(A), q(b) if b else None, groups, rows, cols, group, q(out) if out else None,
                 None) == want, (b, groups, rows, cols, group)


def test_linear_refuses(L):
    f = L.beam_int4_linear
    far, out = A + (1 << 32), A + (1 << 33)

    def call(T, N, K, group, x=A, w=far, o=out):
        s = bm.int4_shape(T, N, K, group)
        return f(ctypes.byref(s), q(x) if x else None, q(w) if w else None, q(o) if o else None, 0, None)
    assert call(0, 64, 256, 64, None, None, None) == bm.BEAM_OK
    assert f(None, q(A), q(far), q(out), 0, None) == bm.BEAM_ERR_INVALID_ARG
    for args in ((-1, 64, 256, 64), (1, 0, 256, 64), (1, 64, 0, 64), (1, -5, 256, 64)):
        assert call(*args) == bm.BEAM_ERR_INVALID_ARG, args
    for args in ((17, 64, 256, 64), (1, 64, 192, 64), (1, 64, 256, 96), (1, 64, 32768 + 128, 64)):
        assert call(*args) == bm.BEAM_ERR_UNSUPPORTED, args
        assert bm.last_cuda_error() != ""
    for kw in (dict(x=None), dict(w=None), dict(o=None), dict(x=A + 8), dict(w=far + 4), dict(o=out + 2),
               dict(o=A + 256), dict(o=far + 1024)):  # the last two overlap x and the weights
        assert call(2, 64, 256, 64, **kw) == bm.BEAM_ERR_INVALID_ARG, kw


def test_dense_refuses(L):
    f = L.beam_dense_forward_int4
    s = bm.dense_shape(4, 512, 640)
    n = int(L.beam_dense_int4_workspace_size(ctypes.byref(s)))
    assert n >= 4 * 640 * 2
    p = [q(A + (i << 32)) for i in range(5)]
    assert f(ctypes.byref(bm.dense_shape(0, 512, 640)), 64, None, None, None, None, None, 0, None) == bm.BEAM_OK
    for bad in (bm.dense_shape(17, 512, 640), bm.dense_shape(4, 500, 640), bm.dense_shape(4, 512, 600),
                bm.dense_shape(4, 512, 32768 + 128), bm.dense_shape(4, 8448, 640)):
        assert f(ctypes.byref(bad), 64, *p, n, None) == bm.BEAM_ERR_UNSUPPORTED
        assert L.beam_dense_int4_workspace_size(ctypes.byref(bad)) == 0
    assert f(ctypes.byref(s), 16, *p, n, None) == bm.BEAM_ERR_UNSUPPORTED
    assert f(ctypes.byref(bm.dense_shape(-1, 512, 640)), 64, *p, n, None) == bm.BEAM_ERR_INVALID_ARG
    assert f(ctypes.byref(s), 64, *p, n - 1, None) == bm.BEAM_ERR_WORKSPACE
    assert f(ctypes.byref(s), 64, *p[:4], None, n, None) == bm.BEAM_ERR_WORKSPACE
    assert f(ctypes.byref(s), 64, *p[:4], q(A + 128), n, None) == bm.BEAM_ERR_WORKSPACE
    for i in range(4):
        for v in (None, q(A + 8)):
            args = list(p)
            args[i] = v
            assert f(ctypes.byref(s), 64, *args, n, None) == bm.BEAM_ERR_INVALID_ARG, i


def test_few_workspace_size(L):
    sizes = [int(L.beam_moe_few_workspace_size(ctypes.byref(beam(T)))) for T in (0, 1, 8, 16)]
    assert 0 < sizes[0] < sizes[1] < sizes[2] < sizes[3]
    assert sizes[3] >= 16 * 8 * (2560 * 2 + 5120 * 4)
    assert L.beam_moe_few_workspace_size(None) == 0
    for bad in (dict(T=17), dict(T=-1), dict(I=8192 + 128), dict(d=100), dict(n_group=7), dict(top_k=9)):
        assert L.beam_moe_few_workspace_size(ctypes.byref(beam(**{"T": 4, **bad}))) == 0, bad
    # the activation and outputs of 16 tokens, not the many-token layout's buffers
    assert sizes[3] < bm.beam_moe_workspace_size(beam(16))


@pytest.mark.parametrize("int4", [False, True])
def test_few_layer_refuses(L, int4):
    s = beam(4)
    n = int(L.beam_moe_few_workspace_size(ctypes.byref(s)))
    names = ["hidden", "router_w", "bias"] + (["gate_up", "down"] if int4 else ["w_gate", "w_up", "w_down"]) + ["out"]

    def call(shape=s, group=64, ws=A, nbytes=n, idx=None, w=None, **ptr):
        args = [q(ptr.get(m, A)) if ptr.get(m, A) else None for m in names]
        args += [idx, w, q(ws) if ws else None, nbytes, None]
        if int4:
            return L.beam_moe_forward_few_int4(ctypes.byref(shape), group, *args)
        return L.beam_moe_forward_few(ctypes.byref(shape), *args)

    nothing = {m: None for m in names}
    assert call(beam(0), ws=None, nbytes=0, **nothing) == bm.BEAM_OK
    assert call(beam(17)) == bm.BEAM_ERR_UNSUPPORTED
    assert "16 tokens" in bm.last_cuda_error()
    assert call(beam(4, I=8320)) == bm.BEAM_ERR_UNSUPPORTED
    assert call(beam(4, d=100)) == bm.BEAM_ERR_UNSUPPORTED
    assert call(beam(-1)) == bm.BEAM_ERR_INVALID_ARG
    if int4:
        for g in (0, 16, 100, 256):
            assert call(group=g) == bm.BEAM_ERR_UNSUPPORTED
    for m in names:
        assert call(**{m: None}) == bm.BEAM_ERR_INVALID_ARG, m
        if m != "bias":
            assert call(**{m: A + 8}) == bm.BEAM_ERR_INVALID_ARG, m
    assert call(idx=q(A + 4)) == bm.BEAM_ERR_INVALID_ARG
    assert call(w=q(A + 4)) == bm.BEAM_ERR_INVALID_ARG
    assert call(ws=None) == bm.BEAM_ERR_WORKSPACE
    assert call(ws=A + 128) == bm.BEAM_ERR_WORKSPACE
    assert call(nbytes=n - 1) == bm.BEAM_ERR_WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device_report_cuda_errors(L):
    s = beam(4)
    n = int(L.beam_moe_few_workspace_size(ctypes.byref(s)))
    assert L.beam_moe_forward_few(ctypes.byref(s), *[q(A)] * 7, None, None, q(A), n, None) == bm.BEAM_ERR_CUDA
    sh = bm.int4_shape(1, 64, 256, 64)
    assert L.beam_int4_linear(ctypes.byref(sh), q(A), q(A + (1 << 32)), q(A + (1 << 33)), 0,
                              None) == bm.BEAM_ERR_CUDA


def test_binding_refuses(L):
    w = torch.zeros(1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bm.beam_int4_quantize(w)                     # a CPU tensor
    with pytest.raises(ValueError):
        bm.beam_int4_quantize(w[0])                  # not [groups, rows, cols]
    with pytest.raises(bm.BeamError):
        bm.beam_int4_quantize(w, group_size=48)
    with pytest.raises(bm.BeamError):
        bm.few_workspace(beam(17), "cpu")
    with pytest.raises(bm.BeamError):
        bm.dense_int4_workspace(bm.dense_shape(17, 512, 640), "cpu")
    x = torch.zeros(1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bm.beam_int4_linear(bm.int4_shape(1, 16, 128, 64), x, torch.zeros(10, dtype=torch.uint8), x)


class _FakeTensor:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert bm._one_device(5, _FakeTensor(0), None, _FakeTensor(0)) == 5
    with pytest.raises(ValueError, match="cuda:1"):
        bm._one_device(5, _FakeTensor(0), _FakeTensor(1))


def test_workspaces_hold_fp32_activations(L):
    s = bm.dense_shape(4, 512, 640)
    assert int(L.beam_dense_int4_workspace_size(ctypes.byref(s))) >= 4 * 640 * 4
    for T in (1, 8, 16):
        n = int(L.beam_moe_few_workspace_size(ctypes.byref(beam(T))))
        assert n >= T * 8 * (2560 + 5120) * 4 + T * 256 * 8 + 256 * 4


class _OnDevice(torch.Tensor):
    """A CPU tensor that says it is on CUDA device `index`."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


def test_launch_refuses_tensors_of_another_device(monkeypatch):
    def entry(index):
        t = torch.zeros(4).as_subclass(_OnDevice)
        t.index = index
        return t, torch.float32, "t", (4,)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    st, ptrs = bm._launch(5, entry(0), (None, torch.float32, "none", (4,), True), entry(0))
    assert st == 5 and ptrs[1] is None and len(ptrs) == 3
    for devices in ((1,), (1, 1), (0, 1), (1, 0)):
        with pytest.raises(ValueError, match="cuda:1"):
            bm._launch(5, *(entry(d) for d in devices))


def test_sizes_beyond_64_bits_are_refused(L):
    big = 1 << 31
    assert bm.beam_int4_packed_size(1 << 62, 16, 128, 64) == 0
    assert bm.beam_int4_packed_size(1 << 40, big - 1, big - 128, 64) == 0
    assert bm.beam_int4_packed_size(1, big - 1, big - 128, 64) == (1 << 27) * ((1 << 24) - 1) * 1088
    f = L.beam_int4_quantize
    for groups, rows, cols in ((1 << 62, 16, 128), (1 << 40, big - 1, big - 128), (1 << 24, 1 << 15, 128),
                               ((1 << 63) - 1, 1, 128)):
        for b in (None, q(A + (1 << 30))):
            if b and (rows % 8 or rows > 1 << 30):
                continue
            assert f(q(A), b, groups, rows, cols, 64, q(A + (1 << 46)), None) == bm.BEAM_ERR_UNSUPPORTED
    s = bm.int4_shape(1, big - 16, 128, 64)
    assert L.beam_int4_linear(ctypes.byref(s), q(A), q(A + (1 << 44)), q(A + (1 << 45)), 0,
                              None) == bm.BEAM_ERR_UNSUPPORTED
    assert "2^31" in bm.last_cuda_error()
