"""Where the binding's wrappers get the memory that they allocate for a call on a given stream, on the CPU against a
stand-in library: from that stream's own pool.  (From the current stream's pool a call could be given a block that
kernels queued there have yet to read or write.)  What a call returns is marked as used by the caller's stream too."""
import contextlib

import pytest
import torch

import int8_expert_weight_b200 as jm
from int8_expert_weight_b200 import build as jbuild

CPU = torch.device("cpu")


class FakeStream:
    def __init__(self, name, device=CPU):
        self.name, self.device, self.cuda_stream = name, device, 0x5151

    def __repr__(self):
        return self.name


class FakeLibrary:
    def __getattr__(self, name):
        return lambda *args: 4096 if "workspace_size" in name else 0


@pytest.fixture
def pools(monkeypatch):
    """`pools.made`: (stream that was current, tensor) of every allocation; `pools.marked`: (tensor, stream)."""
    jbuild.build()

    class Pools:
        caller, made, marked = FakeStream("caller"), [], []

    p = Pools()
    p.made, p.marked = [], []
    current = [p.caller]

    @contextlib.contextmanager
    def entered(stream):
        current.append(stream)
        yield
        current.pop()

    @contextlib.contextmanager
    def device(dev):
        yield

    def recorded(make):
        def empty(*args, **kwargs):
            p.made.append((current[-1], make(*args, **kwargs)))
            return p.made[-1][1]
        return empty

    monkeypatch.setattr(jm, "_lib", FakeLibrary())
    monkeypatch.setattr(jm, "_check", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: current[-1])
    monkeypatch.setattr(jm, "_current_raw_stream", lambda index: 0x7777)
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch.Tensor, "new_empty", recorded(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: p.marked.append((t, s)))
    return p


def z(*shape, dt=torch.uint8, device="cpu"):
    return torch.zeros(*shape, dtype=dt, device=device)


def x():
    return z(4, 128, dt=torch.bfloat16)


def mx4_weights():
    return [z(16, 256, 64), z(16, 256, 4), z(16, 256, 64), z(16, 256, 4), z(16, 128, 128), z(16, 128, 8)]


def weights(dt, n=16):
    f = torch.float32
    return [z(n, 256, 128, dt=dt), z(n, 256, dt=f), z(n, 256, 128, dt=dt), z(n, 256, dt=f), z(n, 128, 256, dt=dt),
            z(n, 128, dt=f)]


def router():
    return z(16, 128, dt=torch.float32)


GROUPED = [z(5, 64), z(5, 4), z(4, dt=torch.int32), z(3, 40, 64), z(3, 40, 4)]
CALLS = {
    "quantize_mx4": lambda s: jm.jamba_moe_quantize_mx4(x(), stream=s),
    "dequantize_mx4": lambda s: jm.jamba_moe_dequantize_mx4(z(3, 32), z(3, 2), stream=s),
    "grouped_mx4": lambda s: jm.jamba_moe_grouped_mx4(*GROUPED, stream=s),
    "forward_mx4": lambda s: jm.jamba_moe_forward_mx4(x(), z(16, 128, dt=torch.float32), None, *mx4_weights(),
                                                      stream=s),
    "quantize": lambda s: jm.jamba_moe_quantize(x(), stream=s),
    "quantize_fp8": lambda s: jm.jamba_moe_quantize_fp8(x(), stream=s),
    "forward": lambda s: jm.jamba_moe_forward(x(), router(), None, *weights(torch.int8), stream=s),
    "forward_fp8": lambda s: jm.jamba_moe_forward_fp8(x(), router(), None, *weights(torch.uint8), stream=s),
    "forward_bf16w": lambda s: jm.jamba_moe_forward_bf16w(x(), router(), None, *weights(torch.bfloat16)[::2], stream=s),
    "mlp_forward": lambda s: jm.jamba_mlp_forward(x(), *[t[0] for t in weights(torch.int8)], stream=s),
    "ep_dispatch": lambda s: jm.jamba_moe_ep_dispatch(x(), router(), None, 2, stream=s),
    "ep_experts": lambda s: jm.jamba_moe_ep_experts(x(), z(4, dt=torch.int32), z(4, dt=torch.float32),
                                                    *weights(torch.int8, 8), stream=s),
    "ep_combine": lambda s: jm.jamba_moe_ep_combine(z(8, 128, dt=torch.float32), z(4, 2, dt=torch.int32), stream=s),
}


def tensors(out):
    return [t for t in (out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,))]


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_given_streams_pool(pools, name):
    side = FakeStream("side")
    out = tensors(CALLS[name](side))
    assert pools.made and [s for s, _ in pools.made] == [side] * len(pools.made)
    for t in out:
        assert any(t is m for _, m in pools.made)
        assert any(t is m and s is pools.caller for m, s in pools.marked), "not kept for the caller's stream"


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_it_is_the_current_ones(pools, name):
    CALLS[name](None)
    assert pools.made and [s for s, _ in pools.made] == [pools.caller] * len(pools.made)
    assert not pools.marked


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(pools, name):
    with pytest.raises(ValueError, match="stream belongs to"):
        CALLS[name](FakeStream("far", torch.device("meta")))
    assert not pools.made
