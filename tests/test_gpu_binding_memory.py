"""Calls on a given stream while the current stream is behind: what a call allocates for itself is no memory that
kernels queued on the current stream have yet to read or write (the mirror image: tests/test_gpu_mx4.py,
test_memory_of_calls_on_a_given_stream)."""
import dataclasses

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import int8_expert_weight_b200 as jm  # noqa: E402
import synth  # noqa: E402
from gpu_layer import bf16_to_dev  # noqa: E402
from helpers import gap_inputs, workload  # noqa: E402


@pytest.fixture(scope="module")
def calls():
    """{name: call(stream)}, their inputs long ready on the device."""
    from int8_expert_weight_b200 import build
    build.build()
    jm.load_library()
    wl = dataclasses.replace(workload("tiny"), T=40, d=256, F=384)
    inp = gap_inputs(wl)
    x, wr = bf16_to_dev(inp["x"]), torch.from_numpy(inp["wr"]).cuda()
    bias = None if inp["bias"] is None else torch.from_numpy(inp["bias"]).cuda()
    w = [bf16_to_dev(synth.gen_experts(wl, which)) for which in ("w1", "w3", "w2")]
    mx4 = [t for v in w for t in jm.jamba_moe_quantize_mx4(v)]
    xq, xs = jm.jamba_moe_quantize_mx4(x)
    int8 = [t for v in w for t in jm.jamba_moe_quantize(v)]
    fp8 = [t for v in w for t in jm.jamba_moe_quantize_fp8(v)]
    mlp = [t[0] for t in int8]
    sent = jm.jamba_moe_ep_dispatch(x, wr, bias, 1)
    sent = [sent["send_x"], sent["send_expert"], sent["send_w"], sent["pos"]]
    ret = jm.jamba_moe_ep_experts(*sent[:3], *int8)
    off = torch.tensor([0, 30, 30, 40] + [40] * 13, dtype=torch.int32, device="cuda")
    return {
        "quantize_mx4": lambda s: jm.jamba_moe_quantize_mx4(x, stream=s),
        "dequantize_mx4": lambda s: jm.jamba_moe_dequantize_mx4(xq, xs, stream=s),
        "grouped_mx4": lambda s: jm.jamba_moe_grouped_mx4(xq, xs, off, *mx4[:2], stream=s),
        "forward_mx4": lambda s: jm.jamba_moe_forward_mx4(x, wr, bias, *mx4, stream=s),
        "quantize": lambda s: jm.jamba_moe_quantize(x, stream=s),
        "quantize_fp8": lambda s: jm.jamba_moe_quantize_fp8(x, stream=s),
        "forward": lambda s: jm.jamba_moe_forward(x, wr, bias, *int8, stream=s),
        "forward_fp8": lambda s: jm.jamba_moe_forward_fp8(x, wr, bias, *fp8, stream=s),
        "forward_bf16w": lambda s: jm.jamba_moe_forward_bf16w(x, wr, bias, *w, stream=s),
        "mlp_forward": lambda s: jm.jamba_mlp_forward(x, *mlp, stream=s),
        "ep_dispatch": lambda s: tuple(v for k, v in jm.jamba_moe_ep_dispatch(x, wr, bias, 1, stream=s).items()
                                       if k != "workspace"),
        "ep_experts": lambda s: jm.jamba_moe_ep_experts(*sent[:3], *int8, stream=s),
        "ep_combine": lambda s: jm.jamba_moe_ep_combine(ret, sent[3], stream=s),
    }


NAMES = ["quantize_mx4", "dequantize_mx4", "grouped_mx4", "forward_mx4", "quantize", "quantize_fp8", "forward",
         "forward_fp8", "forward_bf16w", "mlp_forward", "ep_dispatch", "ep_experts", "ep_combine"]


@pytest.mark.parametrize("name", NAMES)
def test_call_beside_a_current_stream_that_is_behind(calls, name):
    def outputs(s):
        r = calls[name](s)
        return r if isinstance(r, tuple) else (r,)

    want = [t.clone() for t in outputs(None)]
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want]
    sizes += [4096, jm.jamba_moe_workspace_size_mx4(40, 256, 384), jm.jamba_moe_workspace_size(40, 256, 384),
              jm.jamba_moe_workspace_size_fp8(40, 256, 384), jm.jamba_mlp_workspace_size(40, 256, 384),
              jm.jamba_moe_ep_dispatch_workspace_size(40, 256), jm.jamba_moe_ep_experts_workspace_size(80, 256, 384)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the sizes that the call allocates, still to be read and then overwritten by the current stream when
    # they are dropped: the next ones of these sizes in its pool
    blocks = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes]
    kept = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for k, b in zip(kept, blocks):
        k.copy_(b)
        b.fill_(7)
    del b, blocks
    got = outputs(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all((k == 3).all() for k in kept), "the call wrote to memory that was still to be read"
    for a, b in zip(got, want):
        assert torch.equal(a, b)
