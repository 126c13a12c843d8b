"""The status word of the grouped MX4 product is each call's own, also of a call without rows."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import int8_expert_weight_b200 as jm  # noqa: E402


def call(n, offsets, ws):
    g = torch.Generator("cuda").manual_seed(n)
    code = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda")  # noqa: E731
    scale = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    jm.jamba_moe_grouped_mx4(code(n, 64), scale(n, 4), off, code(2, 40, 64), scale(2, 40, 4), workspace=ws)


def test_status_of_a_call_without_rows():
    from int8_expert_weight_b200 import build
    build.build()
    ws = torch.full((jm.jamba_moe_grouped_mx4_workspace_size(0, 40, 128, 2),), 0x11, dtype=torch.uint8, device="cuda")
    call(0, [0, 0, 0], ws)
    assert jm.jamba_moe_read_device_status(ws) == 0  # whatever was there
    call(9, [0, 12, 9], ws)
    assert jm.jamba_moe_read_device_status(ws) == 6
    call(0, [0, 0, 0], ws)
    assert jm.jamba_moe_read_device_status(ws) == 0  # not the last call's
    call(9, [0, 12, 9], ws)
    call(9, [0, 3, 9], ws)
    assert jm.jamba_moe_read_device_status(ws) == 0
