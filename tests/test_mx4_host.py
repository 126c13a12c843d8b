"""MX4 operators on the CPU: the reference against closed forms, and the refusals of the C entry points
and the binding (they return before touching a device)."""
import ctypes

import numpy as np
import pytest

import int8_expert_weight_b200 as jm
import mx4_reference as ref
from int8_expert_weight_b200 import build as jbuild

FAKE = 0x10000  # a 256-aligned non-null value; never dereferenced because validation fails first


@pytest.fixture(scope="module")
def lib():
    jbuild.build()
    return jm.load_library()


def one_block(values):
    q, s = ref.quantize(ref.bf16_bits(np.array(values + [0.0] * (32 - len(values)), np.float32))[None])
    return ref.values(q, s)[0][:len(values)], int(s[0, 0])


def test_reference_grid_ties_and_saturation():
    # 4 makes the scale 1: the grid itself, every midpoint (to the even code), and what is past 6
    got, s = one_block([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.75, 6.0, 7.5, 0.24, 0.26, -5.0625])
    assert s == 127
    assert got.tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -1.0, 6.0, 6.0, 0.0, 0.5, -6.0]


def test_reference_scales():
    assert one_block([0.0, -0.0])[1] == 127
    assert one_block([1.0])[1] == 125 and one_block([7.96875])[1] == 127 and one_block([8.0])[1] == 128
    assert one_block([2.0 ** 127])[1] == 252
    assert one_block([2.0 ** -124])[1] == 1 and one_block([2.0 ** -126])[1] == 0 and one_block([2.0 ** -133])[1] == 0
    for bad in (np.inf, -np.inf, np.nan):
        q, s = ref.quantize(np.array([[0x3F80] * 31 + [0x7FC0 if np.isnan(bad) else 0x7F80]], np.uint16))
        assert s[0, 0] == 255 and not q.any() and np.isnan(ref.values(q, s)).all()


def test_reference_round_trip_of_grid_values():
    rng = np.random.default_rng(3)
    q = rng.integers(0, 256, (5, 64), np.uint8)
    q[:, ::16] = (q[:, ::16] & 0x80) | 0x06  # element 0 of every block is 4: the block keeps its scale
    s = rng.integers(1, 250, (5, 4)).astype(np.uint8)
    v = ref.values(q, s)
    q2, s2 = ref.quantize(ref.bf16_bits(v))
    assert np.array_equal(s, s2) and np.array_equal(q, q2)


def quant(lib, fn, a=FAKE, b=FAKE, c=FAKE, n=1, rows=4, cols=64):
    f = getattr(lib, fn)
    return f(a, n, rows, cols, b, c, None) if fn == "jamba_moe_quantize_mx4" else f(b, c, n, rows, cols, a, None)


@pytest.mark.parametrize("fn", ["jamba_moe_quantize_mx4", "jamba_moe_dequantize_mx4"])
def test_quantize_refusals(lib, fn):
    assert quant(lib, fn, a=None) == 1 and quant(lib, fn, b=None) == 1 and quant(lib, fn, c=None) == 1
    for bad in (dict(n=0), dict(n=-1), dict(rows=0), dict(cols=0), dict(cols=48), dict(cols=(1 << 20) + 32),
                dict(n=1 << 40, rows=1 << 40), dict(n=1 << 20, rows=1 << 20, cols=64)):
        assert quant(lib, fn, **bad) == 2, bad
    assert quant(lib, fn, a=FAKE + 8) == 7 and quant(lib, fn, b=FAKE + 4) == 7 and quant(lib, fn, c=FAKE + 1) == 7


def grouped(lib, xq=FAKE, xs=FAKE, off=FAKE, N=8, rows=100, cols=256, E=4, Q=FAKE, S=FAKE, y=FAKE, out=0, ws=FAKE,
            wsb=1 << 40):
    return lib.jamba_moe_grouped_mx4(xq, xs, off, N, rows, cols, E, Q, S, y, out, ws, wsb, None)


def test_grouped_refusals(lib):
    for name in ("xq", "xs", "off", "Q", "S", "y", "ws"):
        assert grouped(lib, **{name: None}) == 1, name
    for bad in (dict(N=-1), dict(N=(1 << 20) + 1), dict(rows=0), dict(rows=65537), dict(cols=64), dict(cols=192),
                dict(cols=32896), dict(E=0), dict(E=257), dict(out=2), dict(out=-1)):
        assert grouped(lib, **bad) == 2, bad
    for name, off in (("xq", 8), ("Q", 8), ("y", 8), ("xs", 2), ("S", 2), ("off", 2)):
        assert grouped(lib, **{name: FAKE + off}) == 7, name
    assert grouped(lib, ws=FAKE + 64) == 3
    need = jm.jamba_moe_grouped_mx4_workspace_size(8, 100, 256, 4)
    assert need >= 4096 and grouped(lib, wsb=need - 1) == 3
    assert grouped(lib, N=0, xq=None, xs=None, off=None, Q=None, S=None, y=None, ws=None, wsb=0) == 0
    assert grouped(lib, N=0, cols=100) == 2  # sizes are still checked
    assert jm.jamba_moe_grouped_mx4_workspace_size(8, 100, 200, 4) == 0


def test_layer_refusals(lib):
    size = jm.jamba_moe_workspace_size_mx4
    need = size(8, 256, 512)
    assert need > 0 and need % 256 == 0 and size(8, 200, 512) == 0 and size(8, 256, 512, 8, 2) == 0

    def fwd(T=8, d=256, ffn=512, E=16, K=2, ws=FAKE, wsb=need, **at):
        names = ("x", "router", "bias", "Q1", "S1", "Q3", "S3", "Q2", "S2")
        p = [at.get(n, None if n == "bias" else FAKE) for n in names]
        return lib.jamba_moe_forward_mx4(*p, T, d, ffn, E, K, at.get("y", FAKE), at.get("ids"), at.get("w"), ws, wsb,
                                         None)

    for name in ("x", "router", "Q1", "S1", "Q3", "S3", "Q2", "S2", "y"):
        assert fwd(**{name: None}) == 1, name
    for bad in (dict(T=-1), dict(d=200), dict(ffn=100), dict(E=8), dict(K=1)):
        assert fwd(**bad) == 2, bad
    for name, off in (("x", 8), ("Q1", 8), ("Q3", 4), ("Q2", 2), ("y", 2), ("S1", 1), ("S3", 2), ("S2", 3), ("bias", 2),
                      ("ids", 2), ("w", 1)):
        assert fwd(**{name: FAKE + off}) == 7, name
    assert fwd(ws=None) == 1 and fwd(ws=FAKE + 128) == 3 and fwd(wsb=need - 1) == 3
    assert fwd(T=0, x=None, y=None, ws=None, wsb=0) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        jm.jamba_moe_quantize_mx4(cpu)
    with pytest.raises(ValueError, match="CUDA"):
        jm.jamba_moe_dequantize_mx4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        jm.jamba_moe_quantize_mx4(np.zeros((4, 64)))


class FakeStream:
    def __init__(self, device, handle=0x5151):
        self.device, self.cuda_stream = device, handle


@pytest.fixture
def fake(monkeypatch, lib):
    """A stand-in library that records its calls, checked against the declared argument lists; tensors on the CPU
    stand for the device's, `fake.current` is the current device's index."""
    import contextlib

    import torch

    class Recorder:
        calls, devices, current = [], [], 7

        def __getattr__(self, name):
            declared = getattr(lib, name).argtypes

            def call(*args):
                assert len(args) == len(declared), name
                self.calls.append((name, args))
                return 4096 if "workspace_size" in name else 0

            return call

    rec = Recorder()
    rec.calls, rec.devices = [], []

    @contextlib.contextmanager
    def switched(dev):
        rec.devices.append(dev)
        yield

    monkeypatch.setattr(jm, "_lib", rec)
    monkeypatch.setattr(jm, "_check", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "device", switched)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: rec.current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: FakeStream(dev))
    monkeypatch.setattr(jm, "_current_raw_stream", lambda index: 0x7777)
    return rec


def test_binding_marshals_and_switches_devices(fake):
    import torch
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    xq, xs, Q, S = u8(5, 64), u8(5, 4), u8(3, 40, 64), u8(3, 40, 4)
    off = torch.zeros(4, dtype=torch.int32)
    for current, stream in ((7, 0x5151), (None, 0x7777)):  # another device is current; the tensors' own is
        fake.current = current
        fake.calls.clear()
        q, s = jm.jamba_moe_quantize_mx4(torch.zeros(2, 3, 64, dtype=torch.bfloat16))
        assert tuple(q.shape) == (2, 3, 32) and tuple(s.shape) == (2, 3, 2) and q.dtype == s.dtype == torch.uint8
        w = jm.jamba_moe_dequantize_mx4(q, s)
        assert tuple(w.shape) == (2, 3, 64) and w.dtype == torch.bfloat16
        y = jm.jamba_moe_grouped_mx4(xq, xs, off, Q, S, out_dtype=torch.float32)
        assert tuple(y.shape) == (5, 40) and y.dtype == torch.float32
        out = jm.jamba_moe_forward_mx4(torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(16, 128), None,
                                       u8(16, 256, 64), u8(16, 256, 4), u8(16, 256, 64), u8(16, 256, 4),
                                       u8(16, 128, 128), u8(16, 128, 8))
        assert [tuple(t.shape) for t in out] == [(4, 128), (4, 2), (4, 2)]
        calls = [(n, a) for n, a in fake.calls if "workspace_size" not in n]
        assert [n for n, _ in calls] == ["jamba_moe_quantize_mx4", "jamba_moe_dequantize_mx4", "jamba_moe_grouped_mx4",
                                         "jamba_moe_forward_mx4"]
        assert calls[0][1][1:4] == (2, 3, 64) and calls[1][1][2:5] == (2, 3, 64)
        assert calls[2][1][3:7] == (5, 40, 128, 3) and calls[2][1][10] == jm.OUT_FP32
        assert calls[3][1][9:14] == (4, 128, 256, 16, 2)
        assert all(a[-1] == stream for _, a in calls)
    assert fake.devices == [torch.device("cpu")] * 4  # switched for the first four calls only


def test_binding_refuses_mixed_devices_and_streams(fake):
    import torch
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    args = [u8(5, 64), u8(5, 4), torch.zeros(4, dtype=torch.int32), u8(3, 40, 64), u8(3, 40, 4)]
    with pytest.raises(ValueError, match="S is on meta"):
        jm.jamba_moe_grouped_mx4(*args[:4], args[4].to("meta"))
    with pytest.raises(ValueError, match="stream belongs to"):
        jm.jamba_moe_grouped_mx4(*args, stream=FakeStream(torch.device("meta")))
    with pytest.raises(TypeError, match="out_dtype"):
        jm.jamba_moe_grouped_mx4(*args, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="xq must be"):
        jm.jamba_moe_grouped_mx4(args[0][None], *args[1:])
    assert not [n for n, _ in fake.calls if n == "jamba_moe_grouped_mx4"]


def test_kernel_names(lib):
    lib.jamba_moe_kernel_name.restype = ctypes.c_char_p
    assert [lib.jamba_moe_kernel_name(k).decode() for k in range(len(jm.KERNEL_NAMES))] == jm.KERNEL_NAMES
