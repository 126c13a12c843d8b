"""A step (or an expert-parallel rank) without rows: the conversions take it as the products and the layer do."""
import pytest

torch = pytest.importorskip("torch")

import int8_expert_weight_b200 as jm
from int8_expert_weight_b200 import build as jbuild

EMPTY = [(0, 64), (0, 5, 96), (3, 0, 32), (0, 1 << 20)]


class NoLibrary:
    """Every call is refused, as the C entry points refuse no rows."""

    def __getattr__(self, name):
        return lambda *args: 2


@pytest.fixture
def on_cpu(monkeypatch):
    jbuild.build()
    jm.load_library()
    real = jm._lib
    fake = NoLibrary()
    fake.jamba_moe_status_string = real.jamba_moe_status_string
    monkeypatch.setattr(jm, "_lib", fake)
    monkeypatch.setattr(jm, "_check", lambda *a, **k: None)
    monkeypatch.setattr(jm, "_launch", lambda fn, dev, stream, *args: fn(*args))


@pytest.mark.parametrize("shape", EMPTY)
def test_conversions_of_no_rows(on_cpu, shape):
    cols = shape[-1]
    q, s = jm.jamba_moe_quantize_mx4(torch.zeros(shape, dtype=torch.bfloat16))
    assert q.shape == shape[:-1] + (cols // 2,) and s.shape == shape[:-1] + (cols // 32,)
    assert q.dtype == s.dtype == torch.uint8
    w = jm.jamba_moe_dequantize_mx4(q, s)
    assert w.shape == shape and w.dtype == torch.bfloat16
    out = (q.clone(), s.clone())
    assert jm.jamba_moe_quantize_mx4(w, out=out) is not None and jm.jamba_moe_dequantize_mx4(q, s, out=w) is w


@pytest.mark.parametrize("shape", [(0, 48), (4, 0), (0, (1 << 20) + 32), (2, 0, 16)])
def test_widths_are_still_checked(on_cpu, shape):
    with pytest.raises(jm.JmoeError):
        jm.jamba_moe_quantize_mx4(torch.zeros(shape, dtype=torch.bfloat16))
    with pytest.raises(jm.JmoeError):
        jm.jamba_moe_dequantize_mx4(torch.zeros(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8),
                                    torch.zeros(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [False, True])
def test_operators_together_without_rows(stream):
    jbuild.build()
    d, ffn = 256, 512
    s = torch.cuda.Stream() if stream else None
    w = torch.randn(16, ffn, d, device="cuda").bfloat16()
    q, sc = jm.jamba_moe_quantize_mx4(w)
    q2, s2 = jm.jamba_moe_quantize_mx4(w.transpose(1, 2).contiguous())
    torch.cuda.synchronize()
    sent = jm.jamba_moe_ep_dispatch(torch.zeros(0, d, dtype=torch.bfloat16, device="cuda"),
                                    torch.zeros(16, d, device="cuda"), None, 1, stream=s)
    off = torch.zeros(17, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    xq, xs = jm.jamba_moe_quantize_mx4(sent["send_x"], stream=s)
    g = jm.jamba_moe_grouped_mx4(xq, xs, off, q, sc, stream=s)
    assert g.shape == (0, ffn) and g.dtype == torch.bfloat16
    assert jm.jamba_moe_dequantize_mx4(xq, xs, stream=s).shape == (0, d)
    o = jm.jamba_moe_grouped_mx4(*jm.jamba_moe_quantize_mx4(g, stream=s), off, q2, s2, out_dtype=torch.float32, stream=s)
    assert o.shape == (0, d)
    y = jm.jamba_moe_ep_combine(o, sent["pos"], stream=s)
    assert y.shape == (0, d) and sent["send_counts"].tolist() == [0]
    assert jm.jamba_moe_forward_mx4(sent["send_x"], torch.zeros(16, d, device="cuda"), None, q, sc, q, sc, q2, s2,
                                    stream=s)[0].shape == (0, d)
